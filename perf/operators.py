"""Cases of the low-bit operators of the shard step, with their plain forms.

Four operators, as one rank of a ZeRO-3 step meets them:

* ``adamw``   one AdamW step over a list of tensors, states in 32 or in 8 bits
              (the 8-bit moments are read back with the call that a checkpoint uses);
* ``gather``  the coalesced all-gather of a bucket over a 4-bit wire: the own
              shard is quantised, the N chunks are widened into the parameters;
* ``send``    the send side of the 4-bit gradient wire: the rank's whole
              gradients are quantised for their owners (and widened again);
* ``reduce``  its owner side: N received 4-bit chunks are averaged.

Formats.  A wire block is 32 consecutive elements of one parameter's
partition: 16 bytes of e2m1 codes (element 2i in the low half of byte i) and
one scale byte s that stands for 2**(s - 127) (255: the block holds a value
that is not finite).  A chunk is the codes of all its blocks, then their scale
bytes, rounded up to 16 bytes.  An 8-bit moment of n elements is n codes
rounded up to whole blocks of 32, then one scale byte a block, rounded up to
16 bytes; the first moment's codes are e4m3, the second's are unsigned with
4 exponent and 4 mantissa bits (bias 7).  Rounding to 8 bits, and to 4 on
the gradient wire, is stochastic with bits from a counter hash of the seed.

``run`` computes the plain form with elementary torch operations where
``own`` is false, and calls the library where it is true.
"""

import numpy as np
import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
HP = {"lr": 1e-3, "beta1": 0.9, "beta2": 0.999, "eps": 1e-8}
SEED = 20240607
M32 = 0xFFFFFFFF
M64 = 0xFFFFFFFFFFFFFFFF

# ------------------------------------------------------------------- cases

# Parameter sets as "count x numel" lists, in ds_id order.
TOY = "1x2048,1x32,1x512,1x16"                                                       # a two-layer toy model
SMALL = "1x38597376,1x786432,12x1769472,12x589824,24x2359296,50x768,12x2304"         # GPT-2-small-shaped matrices and vectors
RAGGED = "1x3215666,1x131040,36x786000,36x262008,36x1048256,36x1048257,75x4095"      # rank 63's share of a width-4095 set, N = 64
LAYER = "1x2097152,2x524288,1x2097152,3x7340032,2x4096"                              # an eighth of a Llama-3-8B-shaped layer


def listed():
    return [
        # the two-layer toy model's parameters: a call that is all latency
        {"name": "adamw32 toy", "op": "adamw", "bits": 32, "dtype": "fp16", "grad": "fp16", "sizes": TOY, "wd": 0.0, "step": 1},
        # a whole small model in one call, bf16 gradients, decay on
        {"name": "adamw32 small model", "op": "adamw", "bits": 32, "dtype": "bf16", "grad": "bf16", "sizes": SMALL, "wd": 0.1, "step": 100},
        # the toy model with 8-bit states: odd blocks, latency
        {"name": "adamw8 toy", "op": "adamw", "bits": 8, "dtype": "fp16", "grad": "fp16", "sizes": TOY, "wd": 0.01, "step": 1},
        # one rank's share of a decoder layer with gradients accumulated in fp32
        {"name": "adamw8 layer fp32 grads", "op": "adamw", "bits": 8, "dtype": "bf16", "grad": "fp32", "sizes": LAYER, "wd": 0.1, "step": 10},
        # one rank's share of a 7.5B ragged set: hundreds of odd-sized tensors
        {"name": "adamw8 ragged share", "op": "adamw", "bits": 8, "dtype": "fp16", "grad": "fp16", "sizes": RAGGED, "wd": 0.0, "step": 1000},
        # the toy model's bucket
        {"name": "gather toy", "op": "gather", "dtype": "fp16", "world": 4, "rank": 1, "sizes": TOY},
        # a prefetch bucket: one MLP matrix of a Llama-3-8B-shaped layer over 8 ranks
        {"name": "gather mlp bucket", "op": "gather", "dtype": "bf16", "world": 8, "rank": 0, "sizes": "1x58720256"},
        # a ragged bucket over 64 ranks (width 4095): no partition starts at a whole vector
        {"name": "gather ragged bucket", "op": "gather", "dtype": "fp16", "world": 64, "rank": 63, "sizes": "1x16769025,1x67088385"},
        # a layer's attention gradients on their way to 8 owners
        {"name": "send attention bucket", "op": "send", "dtype": "bf16", "world": 8, "rank": 0, "sizes": "1x16777216,2x4194304,1x16777216", "stochastic": True},
        # the toy model's gradients, to the nearest
        {"name": "send toy", "op": "send", "dtype": "fp16", "world": 4, "rank": 2, "sizes": TOY, "stochastic": False},
        # the owner's average of an MLP gradient over 8 ranks
        {"name": "reduce mlp bucket", "op": "reduce", "dtype": "bf16", "world": 8, "rank": 7, "sizes": "3x58720256"},
        # the same over 64 ranks, ragged
        {"name": "reduce ragged bucket", "op": "reduce", "dtype": "fp16", "world": 64, "rank": 63, "sizes": "1x16769025,2x67088385"},
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["adamw32", "adamw8", "adamw8", "gather", "send", "reduce"])
    total = _log(rng, 3000, 80_000_000)
    kinds = rng.randint(1, 6)
    sizes = ",".join("%dx%d" % (c, max(1, int(total * rng.random() / (kinds * c)))) for c in (_log(rng, 1, 40) for _ in range(kinds)))
    dtype = rng.choice(["bf16", "fp16"])
    if op.startswith("adamw"):
        return {"op": "adamw", "bits": int(op[5:]), "dtype": dtype, "grad": rng.choice([dtype, dtype, "fp32"]), "sizes": sizes,
                "wd": rng.choice([0.0, 0.01, 0.1]), "step": _log(rng, 1, 10000)}
    world = rng.choice([1, 2, 3, 4, 8, 16, 48, 64])
    case = {"op": op, "dtype": dtype, "world": world, "rank": rng.randrange(world), "sizes": sizes}
    return dict(case, stochastic=rng.random() < 0.7) if op == "send" else case


def _numels(case):
    return [int(n) for c, n in (p.split("x") for p in case["sizes"].split(",")) for _ in range(int(c))]


def _ceil(a, b):
    return -(-a // b)


def _wire(case):
    """Per parameter: partition size and blocks; in all: blocks and bytes of a chunk."""
    ps = [_ceil(n, case["world"]) for n in _numels(case)]
    nb = [_ceil(p, 32) for p in ps]
    return ps, nb, sum(nb), _ceil(17 * sum(nb), 16) * 16


def _moment_bytes(n):
    return _ceil(33 * _ceil(n, 32), 16) * 16


def work(case):
    n = sum(_numels(case))
    if case["op"] == "adamw":
        per = (4 if case["grad"] == "fp32" else 2) + 8 + 2 + (16 if case["bits"] == 32 else 4 + 4 / 32 + 2 + 2 / 32 + 4)
        return {"bytes": per * n, "flops": 18 * n}
    ps, nb, blocks, _ = _wire(case)
    c, wire, N = sum(ps), 17 * blocks, case["world"]
    if case["op"] == "gather":
        return {"bytes": 2 * c + N * wire + 2 * n, "flops": n + 2 * c}
    if case["op"] == "send":
        return {"bytes": 2 * n + 2 * N * wire + 2 * n, "flops": 4 * n}
    return {"bytes": N * wire + 2 * c, "flops": 2 * N * c}


# ------------------------------------------------------------------ inputs

def _starts(sizes):
    return [0] + list(np.cumsum(sizes, dtype=np.int64))[:-1]


def _long(v):
    return torch.tensor([int(x) for x in v], dtype=torch.int64, device=DEV)


def _blocks_plan(real, nb):
    """Positions of a list of runs padded to whole blocks: (run of each padded
    position, its element within the run, whether it holds one)."""
    run = torch.repeat_interleave(torch.arange(len(nb), device=DEV), _long([32 * b for b in nb]))
    k = torch.arange(run.numel(), device=DEV) - _long(_starts([32 * b for b in nb]))[run]
    return run, k, k < _long(real)[run]


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _gradients(n, g, dtype):
    x = torch.randn(n, device=DEV, generator=g) * 1e-3
    x = torch.where(torch.rand(n, device=DEV, generator=g) < 0.01, x * 100, x)   # outliers
    return x.to(dtype)


def prepare(case, seed):
    g, sizes = _gen(seed), _numels(case)
    dt, n = DTYPES[case["dtype"]], sum(_numels(case))
    st = {"case": case, "sizes": sizes}
    if case["op"] == "adamw":
        nb = [_ceil(s, 32) for s in sizes]
        w = torch.randn(n, device=DEV, generator=g) * 0.02
        st.update(master=w, param=w.to(dt), grad=_gradients(n, g, DTYPES[case["grad"]]), t=case["step"],
                  scale=torch.full((1,), 0.5, device=DEV), nonfinite=torch.zeros(1, dtype=torch.int32, device=DEV))
        # every other tensor of the list decays at its own rate, as norms and biases are kept from it
        st["wd"] = [case["wd"] * (1 - i % 2) for i in range(len(sizes))]
        st["lr_scale"] = [1.0 if i % 3 else 0.5 for i in range(len(sizes))]
        m = torch.randn(n, device=DEV, generator=g) * 3e-4
        v = (torch.randn(n, device=DEV, generator=g) * 1e-3).square() + 1e-8
        if case["bits"] == 32:
            st["run_of"] = torch.repeat_interleave(torch.arange(len(sizes), device=DEV), _long(sizes))
            return dict(st, exp_avg=m, exp_avg_sq=v)
        run, k, live = _blocks_plan(sizes, nb)
        at = _long(_starts([_moment_bytes(s) for s in sizes]))
        st["off8"] = _starts([_moment_bytes(s) for s in sizes])
        st["codes_at"] = (at[run] + k).to(torch.int64)                             # of each padded position
        b = torch.arange(run.numel() // 32, device=DEV) * 32
        st["scales_at"] = at[run[b]] + 32 * _long(nb)[run[b]] + torch.div(k[b], 32, rounding_mode="floor")
        st["padded_of"] = torch.nonzero(live).reshape(-1)                          # of each element
        st["run_of"], st["k_of"] = run[st["padded_of"]], k[st["padded_of"]]
        total = sum(_moment_bytes(s) for s in sizes)
        for name, x, enc, half in (("exp_avg", m, _encode_m, 1 << 19), ("exp_avg_sq", v, _encode_v, 1 << 15)):   # to the nearest
            buf = torch.zeros(total, dtype=torch.uint8, device=DEV)
            code, s = enc(_pad(st, x), half)
            buf[st["codes_at"]], buf[st["scales_at"]] = code, s
            st[name] = buf
            st[name + "_values"] = torch.empty(n, dtype=torch.bfloat16, device=DEV)
        return st

    N, rank = case["world"], case["rank"]
    ps, nb, blocks, chunk = _wire(case)
    run, k, live = _blocks_plan(ps, nb)
    f = _long(_starts(sizes))
    v = torch.arange(N, device=DEV)[:, None]
    e = v * _long(ps)[run] + k                                                      # element of the parameter
    st["live"] = live & (e < _long(sizes)[run])                                     # [N, padded positions]
    st["full_at"] = (f[run] + e)[st["live"]]
    st["shard_at"] = (_long(_starts(ps))[run] + k)[st["live"][rank]]
    c = sum(ps)
    if case["op"] == "gather":
        full = (torch.randn(n, device=DEV, generator=g) * 0.02).to(dt)
        x = _spread(st, full)
        st["wires"] = _encode_wire(x, case["dtype"], None).reshape(N, chunk)        # what the ranks sent
        st["wires"][rank] = 0                                                       # the own chunk is the call's to write
        st["shard"] = torch.zeros(c, dtype=dt, device=DEV)
        st["shard"][st["shard_at"]] = full[st["full_at"][_own_part(st, rank)]]
        st["full"] = torch.empty(n, dtype=dt, device=DEV)
    elif case["op"] == "send":
        st["grads"] = _gradients(n, g, dt)
        st["wires"] = torch.zeros((N, chunk), dtype=torch.uint8, device=DEV)
        st["full"] = torch.empty(n, dtype=dt, device=DEV)
    else:
        st["wires"] = torch.empty((N, chunk), dtype=torch.uint8, device=DEV)
        for r in range(N):
            x = torch.zeros(run.numel(), device=DEV)
            x[st["live"][rank]] = _gradients(st["shard_at"].numel(), g, dt).float()
            st["wires"][r] = _encode_wire(x[None], case["dtype"], None)[0]
        st["grad_flat"] = torch.empty(c, dtype=dt, device=DEV)
    return st


def _own_part(st, rank):
    """Where rank's elements are among the live ones."""
    before = int(st["live"][:rank].sum())
    return slice(before, before + int(st["live"][rank].sum()))


def _spread(st, flat):
    """The parameters' elements at their padded places, [N, positions], zeros elsewhere."""
    x = torch.zeros(st["live"].shape, device=DEV)
    x[st["live"]] = flat.float()[st["full_at"]]
    return x


def _pad(st, x):
    out = torch.zeros(st["codes_at"].numel(), device=DEV)
    out[st["padded_of"]] = x
    return out


# -------------------------------------------------------------- plain forms

def _mix64(z):
    z ^= z >> 32
    z = z * 0xD6E8FEB86659FD93 & M64
    z ^= z >> 29
    z = z * 0xA0761D6478BD642F & M64
    return z ^ z >> 32


def _keys(seed, step, ident):
    """Two 32-bit keys of a tensor's random words."""
    z = _mix64((_mix64((seed + 0x9E3779B97F4A7C15 * step) & M64) + 0x9E3779B97F4A7C15 * ident) & M64)
    return z & M32, z >> 32


def _words(e, k0, k1):
    """The random word of element e (int64 tensors; the keys may be tensors too)."""
    x = ((e & M32) * 0x9E3779B1 + k0 + (e >> 32) * 0x85157AF5) & M32
    x = x ^ (x >> 16)
    x = (x * 0x761BCE4B) & M32
    x = x ^ (x >> 15) ^ k1
    x = (x * 0xA0D73955) & M32
    return x ^ (x >> 16)


def _scales(x, carry, emax, lowest=1, highest=254):
    """Scale byte of each block of 32: the smallest power of two under which
    the block's largest magnitude keeps to the code's range."""
    top = x.abs().reshape(-1, 32).amax(1).view(torch.int32).to(torch.int64)
    s = (((top + carry) >> 23) - emax).clamp(lowest, highest)
    return torch.where(top >= 0x7F800000, 255, s)


def _pow2(e):
    """2.0**e in 32 bits, e from -126 to 127."""
    return ((e.clamp(-126, 127) + 127) << 23).to(torch.int32).view(torch.float32)


def _over_scale(x, s):
    return (x.reshape(-1, 32) / _pow2(s - 127)[:, None]).reshape(-1)


def _exponent(a):
    return (a.view(torch.int32) >> 23) - 127


def _encode_m(x, u20):
    """e4m3; u20: 20 random bits that decide between the two codes around a value."""
    s = _scales(x, 0x1FFFFF, 8)
    a = _over_scale(x.abs(), s)
    e = _exponent(a).clamp(min=-6)
    t = a * _pow2(3 - e)
    lo = t.floor()
    part = ((t - lo) * 2.0**20).floor().to(torch.int64) + u20
    mag = ((e + 6) << 3) + lo.to(torch.int64) + (part >> 20)
    code = mag | (torch.signbit(x).to(torch.int64) << 7)
    code = torch.where(torch.repeat_interleave(s, 32) == 255, 0x7F, code)
    return code.to(torch.uint8), s.to(torch.uint8)


def _encode_v(x, u16):
    """Unsigned, 4 exponent and 4 mantissa bits; u16: 16 random bits; what is
    not zero never becomes zero."""
    s = _scales(x, 0x07FFFF, 8)
    a = _over_scale(x, s)
    e = _exponent(a).clamp(min=-6)
    t = torch.round(a * _pow2(4 - e + 19)).to(torch.int64)
    code = ((e + 6) << 4) + ((t + (u16 << 3)) >> 19)
    code = torch.maximum(code, (x > 0).to(torch.int64))
    code = torch.where(torch.repeat_interleave(s, 32) == 255, 0xFF, code)
    return code.to(torch.uint8), s.to(torch.uint8)


def _decode8(code, s, mant):
    """Values of 8-bit codes with `mant` mantissa bits (the sign bit of e4m3 apart)."""
    c = code.to(torch.int64)
    mag = c & 0x7F if mant == 3 else c
    e, m = mag >> mant, mag & ((1 << mant) - 1)
    m = torch.where(e > 0, m + (1 << mant), m).float()
    val = m * _pow2(e.clamp(min=1) - 7 - mant)
    val = (val.reshape(-1, 32) * _pow2(s.to(torch.int64) - 127)[:, None]).reshape(-1)
    return torch.where(c > 0x7F, -val, val) if mant == 3 else val


def _encode_wire(x, dtype, key):
    """Chunks [N, bytes] of padded values [N, positions]; `key`: None for the nearest."""
    N = x.shape[0]
    cap = 140 if dtype == "fp16" else 252               # so that 6 * scale is still finite in 16 bits
    s = _scales(x.reshape(-1), 0x200000 if key is None else 0x3FFFFF, 2, 1, cap)
    a = _over_scale(x.abs().reshape(-1), s)
    if key is None:                                     # ties to the even code
        code = sum(((a > b) if k % 2 == 0 else (a >= b)).to(torch.uint8) for k, b in enumerate((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)))
    else:
        at = torch.arange(a.numel(), device=DEV)
        word = _words(at >> 1, *key)
        word = torch.where(at % 2 == 0, word, ((word << 1) & M32) | (word >> 31))   # the pair's second: rotated by one
        e = _exponent(a).clamp(0, 2)
        t = a * _pow2(1 - e)                            # in steps of the code at a
        lo = t.floor()
        part = torch.floor((t - lo).double() * 2.0**32).to(torch.int64) + word
        code = ((e << 1) + lo.to(torch.int64) + (part >> 32)).clamp(max=7).to(torch.uint8)
    code = code | (torch.signbit(x.reshape(-1)).to(torch.uint8) << 3)
    pair = code.reshape(N, -1, 2)
    codes, s = pair[..., 0] | (pair[..., 1] << 4), s.to(torch.uint8).reshape(N, -1)
    fill = _ceil(17 * s.shape[1], 16) * 16 - 17 * s.shape[1]
    return torch.cat([codes, s, torch.zeros((N, fill), dtype=torch.uint8, device=DEV)], 1)


def _decode_wire(wires, blocks):
    """Values [N, positions] in 32 bits."""
    b = wires[:, :16 * blocks]
    code = torch.stack([b & 15, b >> 4], -1).reshape(wires.shape[0], -1).to(torch.int64)
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=DEV)
    s = wires[:, 16 * blocks:17 * blocks].to(torch.int64)
    one = torch.where(s == 255, float("nan"), _pow2(s - 127))
    return (table[code].reshape(-1, 32) * one.reshape(-1, 1)).reshape(wires.shape[0], -1)


def _per_element(st, values):
    return torch.tensor(values, dtype=torch.float64, device=DEV).float()[st["run_of"]]


def _adamw_plain(st):
    case, b1, b2 = st["case"], HP["beta1"], HP["beta2"]
    t = st["t"]
    w, gr = st["master"], st["grad"].float() * st["scale"]
    lr = [HP["lr"] * a for a in st["lr_scale"]]
    if case["bits"] == 32:
        m, v = st["exp_avg"], st["exp_avg_sq"]
    else:
        m, v = (_decode8(st[k][st["codes_at"]], st[k][st["scales_at"]], mant)[st["padded_of"]] for k, mant in (("exp_avg", 3), ("exp_avg_sq", 4)))
    w = w - _per_element(st, [a * d for a, d in zip(lr, st["wd"])]) * w
    m = b1 * m + (1 - b1) * gr
    v = b2 * v + (1 - b2) * (gr * gr)
    den = (v / (1 - b2**t)).sqrt() + HP["eps"]
    w = w - _per_element(st, lr) * ((m / (1 - b1**t)) / den)
    st["master"].copy_(w)
    st["param"].copy_(w)
    if case["bits"] == 32:
        st["exp_avg"].copy_(m)
        st["exp_avg_sq"].copy_(v)
        return
    k0, k1 = zip(*(_keys(SEED, t, i) for i in range(len(st["sizes"]))))
    word = _words(st["k_of"], _long(k0)[st["run_of"]], _long(k1)[st["run_of"]])
    bits = torch.zeros(st["codes_at"].numel(), dtype=torch.int64, device=DEV)
    bits[st["padded_of"]] = word
    live = torch.zeros(bits.numel(), dtype=torch.bool, device=DEV)
    live[st["padded_of"]] = True
    for name, x, enc, u, mant in (("exp_avg", m, _encode_m, bits >> 12, 3), ("exp_avg_sq", v, _encode_v, bits & 0xFFFF, 4)):
        code, s = enc(_pad(st, x), u)
        st[name][st["codes_at"][live]], st[name][st["scales_at"]] = code[live], s
        st[name + "_values"].copy_(_decode8(code, s, mant)[st["padded_of"]])


def _adamw_own(st):
    import zero_sharded_state_amd as zs3
    case = st["case"]
    if "list" not in st:
        g_bytes = st["grad"].element_size()
        starts = _starts(st["sizes"])
        moment = [4 * s for s in starts] if case["bits"] == 32 else st["off8"]
        st["list"] = zs3.zs3_adamw_tensor_list([
            dict(numel=n, id=i, master=st["master"].data_ptr() + 4 * s, grad=st["grad"].data_ptr() + g_bytes * s,
                 param=st["param"].data_ptr() + 2 * s, exp_avg=st["exp_avg"].data_ptr() + o,
                 exp_avg_sq=st["exp_avg_sq"].data_ptr() + o, lr_scale=a, weight_decay=d)
            for i, (n, s, o, a, d) in enumerate(zip(st["sizes"], starts, moment, st["lr_scale"], st["wd"]))])
        if case["bits"] == 8:
            st["reads"] = zs3.zs3_moment8_list(
                [dict(numel=n, kind=kind, moment=st[name].data_ptr() + o, out=st[name + "_values"].data_ptr() + 2 * s)
                 for name, kind in (("exp_avg", zs3.ZS3_EXP_AVG), ("exp_avg_sq", zs3.ZS3_EXP_AVG_SQ))
                 for n, s, o in zip(st["sizes"], starts, st["off8"])])
    zs3.zs3_adamw_tensors(case["dtype"], case["grad"], case["bits"], st["list"], st["scale"], st["nonfinite"],
                          dict(HP, step=st["t"]), SEED)
    if case["bits"] == 8:
        zs3.zs3_moment8_read("bf16", st["reads"])


def _wire_own(st):
    import zero_sharded_state_amd as zs3
    case, N, rank = st["case"], st["case"]["world"], st["case"]["rank"]
    if "layout" not in st:
        st["ids"] = list(range(len(st["sizes"])))
        st["layout"] = zs3.zs3_layout_create(N, 0, st["ids"], st["sizes"])
        chunk = st["wires"].shape[1]
        st["chunks"] = [st["wires"].data_ptr() + chunk * r for r in range(N)]
        if case["op"] == "send":
            st["each"] = [st["grads"].data_ptr() + 2 * s for s in _starts(st["sizes"])]
    if case["op"] == "gather":
        zs3.zs3_gather_coalesced_mx4(st["layout"], rank, case["dtype"], zs3.ZS3_PACK | zs3.ZS3_UNPACK, st["ids"], st["shard"],
                                     st["chunks"][rank], st["chunks"], st["full"])
    elif case["op"] == "send":
        zs3.zs3_reduce_scatter_coalesced_mx4(st["layout"], rank, case["dtype"], zs3.ZS3_PACK, st["ids"], grads=st["each"], send=st["wires"],
                                             rounding=zs3.ZS3_ROUND_STOCHASTIC if case["stochastic"] else zs3.ZS3_ROUND_NEAREST, seed=SEED)
        zs3.zs3_gather_coalesced_mx4(st["layout"], rank, case["dtype"], zs3.ZS3_UNPACK, st["ids"], rank_chunks=st["chunks"], full_flat=st["full"])
    else:
        zs3.zs3_reduce_scatter_coalesced_mx4(st["layout"], rank, case["dtype"], zs3.ZS3_REDUCE, st["ids"], recv_chunks=st["chunks"],
                                             grad_flat=st["grad_flat"])


def _wire_plain(st):
    case, rank = st["case"], st["case"]["rank"]
    blocks = _wire(case)[2]
    if case["op"] == "reduce":
        x = _decode_wire(st["wires"], blocks)
        total = torch.zeros(x.shape[1], device=DEV)
        for r in range(case["world"]):                  # in rank order
            total = total + x[r]
        st["grad_flat"].zero_()
        st["grad_flat"][st["shard_at"]] = (total / torch.tensor(float(case["world"]), device=DEV))[st["live"][rank]].to(st["grad_flat"].dtype)
        return
    if case["op"] == "gather":
        x = torch.zeros(st["live"].shape[1], device=DEV)
        x[st["live"][rank]] = st["shard"].float()[st["shard_at"]]
        st["wires"][rank] = _encode_wire(x[None], case["dtype"], None)[0]
    else:
        key = _keys(SEED, 0, 0) if case["stochastic"] else None
        st["wires"].copy_(_encode_wire(_spread(st, st["grads"]), case["dtype"], key))
    st["full"][st["full_at"]] = _decode_wire(st["wires"], blocks)[st["live"]].to(st["full"].dtype)


def run(state):
    if state["case"]["op"] == "adamw":
        if own:
            _adamw_own(state)
        else:
            _adamw_plain(state)
        names = ("master", "param") + (("exp_avg", "exp_avg_sq") if state["case"]["bits"] == 32 else ("exp_avg_values", "exp_avg_sq_values"))
        return {k.replace("_values", ""): state[k] for k in names}
    if own:
        _wire_own(state)
    else:
        _wire_plain(state)
    return state["grad_flat" if state["case"]["op"] == "reduce" else "full"]


# ------------------------------------------------------- the definition in 64 bits

_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _times_pow2(x, e):
    return x * torch.exp2(e.double())


def _magnitude(x):
    """floor(log2(x)) of positive doubles, and the mantissa in [1, 2)."""
    m, e = torch.frexp(x)
    return e.to(torch.int64) - 1, m * 2


def _block_scale(x, largest, emax, low=-126, high=127):
    """log2 of each block's scale, one per element; `largest`: the mantissa up to which a block of exponent k gets 2**(k - emax)."""
    pad = torch.zeros(_ceil(x.numel(), 32) * 32, dtype=torch.float64, device=x.device)
    pad[:x.numel()] = x.abs()
    top = pad.reshape(-1, 32).amax(1)
    k, m = _magnitude(top)
    e = torch.where(top > 0, k - emax + (~largest(m)).to(torch.int64), torch.full_like(k, low)).clamp(low, high)
    return torch.repeat_interleave(e, 32)[:x.numel()]


def _random_word(index, key):
    """The hash again, in numpy's modular integers."""
    i = index.astype(np.uint64)
    with np.errstate(over="ignore"):
        x = i.astype(np.uint32) * np.uint32(0x9E3779B1) + np.uint32(key[0]) + (i >> np.uint64(32)).astype(np.uint32) * np.uint32(0x85157AF5)
        x = (x ^ (x >> np.uint32(16))) * np.uint32(0x761BCE4B)
        x = (x ^ (x >> np.uint32(15)) ^ np.uint32(key[1])) * np.uint32(0xA0D73955)
    return x ^ (x >> np.uint32(16))


def _unit(index, key, shift, bits):
    """The word's `bits` bits from `shift` on as a fraction."""
    w = (_random_word(index, key) >> np.uint32(shift)) & np.uint32((1 << bits) - 1)
    return torch.from_numpy(w.astype(np.float64)).to(DEV) / 2.0**bits


def _stochastic(x, scale, mant, unit, floor):
    """x on the grid of `mant` mantissa bits, 4 exponent bits of bias 7, scaled."""
    a = _times_pow2(x.abs(), -scale)
    k, _ = _magnitude(a)
    step = _times_pow2(torch.ones_like(a), torch.where(a > 0, k, torch.full_like(k, -6)).clamp(min=-6) - mant)
    q = torch.floor(a / step + unit) * step
    if floor:
        q = torch.where(a > 0, q.clamp(min=2.0**-10), q)
    return _times_pow2(q, scale) * torch.sign(x)


def _read_moment(buf, n, mant):
    codes, s = buf[:n].to(torch.float64), buf[_ceil(n, 32) * 32:_ceil(n, 32) * 33].to(torch.int64)
    sign = torch.where((codes >= 128) & (mant == 3), -1.0, 1.0)
    mag = codes % 128 if mant == 3 else codes
    e, f = torch.floor(mag / 2**mant), mag % 2**mant
    val = torch.where(e == 0, f * 2.0**(-6 - mant), (1 + f / 2**mant) * 2.0**(e - 7))
    return sign * _times_pow2(val, torch.repeat_interleave(s, 32)[:n] - 127)


def _exact_adamw(case, st):
    b1, b2, t, out = HP["beta1"], HP["beta2"], case["step"], []
    at = 0
    for i, n in enumerate(st["sizes"]):
        here = slice(at, at + n)
        at += n
        lr = HP["lr"] * st["lr_scale"][i]
        w, g = st["master"][here].double(), st["grad"][here].double() * 0.5
        if case["bits"] == 32:
            m, v = st["exp_avg"][here].double(), st["exp_avg_sq"][here].double()
        else:
            o = st["off8"][i]
            m, v = (_read_moment(st[k][o:o + _moment_bytes(n)], n, mant) for k, mant in (("exp_avg", 3), ("exp_avg_sq", 4)))
        m, v = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g * g
        w = w * (1 - lr * st["wd"][i]) - lr * (m / (1 - b1**t)) / (torch.sqrt(v / (1 - b2**t)) + HP["eps"])
        if case["bits"] == 8:
            index, key = np.arange(n), _keys(SEED, t, i)
            m = _stochastic(m, _block_scale(m, lambda f: f <= 1.75, 8), 3, _unit(index, key, 12, 20), False)
            v = _stochastic(v, _block_scale(v, lambda f: f <= 1.9375, 8), 4, _unit(index, key, 0, 16), True)
        out.append((w, m, v))
    w, m, v = (torch.cat(x) for x in zip(*out))
    return {"master": w, "param": w, "exp_avg": m, "exp_avg_sq": v}


def _exact_block4(x, case, unit):
    """x rounded to the wire's values, in 64 bits."""
    s = _block_scale(x, (lambda f: f < 1.75) if unit is None else (lambda f: f <= 1.5), 2, -126, 13 if case["dtype"] == "fp16" else 125)
    a = _times_pow2(x.abs(), -s)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).double()
    q = (torch.round(a / step) if unit is None else torch.floor(a / step + unit)) * step
    return _times_pow2(q.clamp(max=6.0), s) * torch.sign(x)


def _exact_chunk(wire, first, count, blocks):
    """`count` values of a chunk from block `first` on."""
    nb = _ceil(count, 32)
    b = wire[16 * first:16 * (first + nb)].to(torch.int64)
    code = torch.stack([b % 16, torch.div(b, 16, rounding_mode="floor")], 1).reshape(-1)
    val = torch.tensor(_E2M1, dtype=torch.float64, device=DEV)[code % 8] * torch.where(code >= 8, -1.0, 1.0)
    s = wire[16 * blocks + first:16 * blocks + first + nb].to(torch.int64) - 127
    return _times_pow2(val, torch.repeat_interleave(s, 32))[:count]


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "adamw":
        return _exact_adamw(case, st)
    N, rank = case["world"], case["rank"]
    ps, nb, blocks, _ = _wire(case)
    first, f, o = _starts(nb), _starts(st["sizes"]), _starts(ps)
    out = torch.zeros(sum(ps) if case["op"] == "reduce" else sum(st["sizes"]), dtype=torch.float64, device=DEV)
    for j, n in enumerate(st["sizes"]):
        for r in range(N):
            lo, hi = min(n, r * ps[j]), min(n, (r + 1) * ps[j])
            mine = (min(n, rank * ps[j]), min(n, (rank + 1) * ps[j]))
            if case["op"] == "reduce":
                c = mine[1] - mine[0]
                out[o[j]:o[j] + c] += _exact_chunk(st["wires"][r], first[j], c, blocks) / N
            elif lo == hi:
                continue
            elif case["op"] == "gather":
                x = _exact_block4(st["shard"][o[j]:o[j] + hi - lo].double(), case, None) if r == rank else _exact_chunk(st["wires"][r], first[j], hi - lo, blocks)
                out[f[j] + lo:f[j] + hi] = x
            else:
                unit = None
                if case["stochastic"]:
                    at = (r * blocks + first[j]) * 32 + np.arange(hi - lo)
                    w = _random_word(at // 2, _keys(SEED, 0, 0))
                    w = np.where(at % 2 == 0, w, (w << np.uint32(1)) | (w >> np.uint32(31)))
                    unit = torch.from_numpy(w.astype(np.float64)).to(DEV) / 2.0**32
                out[f[j] + lo:f[j] + hi] = _exact_block4(st["grads"][f[j] + lo:f[j] + hi].double(), case, unit)
    return out
