"""Cases of the gradient-list operators of the shard step, with their plain forms.

Three operators over a list of gradient tensors that lie anywhere, as one rank of a ZeRO-3
step meets them between the reduce-scatter and AdamW, and the three in a row:

* ``norm``        the global norm (root of the sum of squares, or the largest magnitude), the clip
                  scale and the overflow flag, with the peers' sums and, where asked, every tensor's own norm;
* ``clip``        the gradients times the scale, in place or into another type;
* ``accumulate``  a micro-batch's gradients into fp32 accumulators, the norm of the sum with the last one;
* ``update``      the last micro-batch accumulated, the norm of the sum, the clipped sum in 16 bits.

The tensors of one type lie one behind the other in a flat buffer, as in a rank's flat
gradient, so odd sizes put the next ones at odd places.  Tensors under 100,000 elements are the
persistent ones (norms, biases), whole on every rank, and come last.

``run`` computes the plain form with elementary torch operations where ``own`` is false, and
calls the library where it is true.
"""

import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
PERSISTENT = 100_000

# ------------------------------------------------------------------- cases

# Tensor lists as "count x numel".
TOY = "1x2048,1x512,1x32,1x16"                                                       # a two-layer toy model
LAYER = "2x2097152,2x524288,3x7340032,2x4096"                                        # an eighth of a Llama-3-8B-shaped layer
RAGGED = "1x3215666,1x131040,36x786000,36x262008,36x1048256,36x1048257,75x4095"      # rank 63's share of a width-4095 set, N = 64
SHARE = "2x65667072,64x2097152,64x524288,96x7340032,65x4096"                         # rank 0's share of a Llama-3-8B-shaped set, N = 8


def listed():
    return [
        # the toy model's gradients, a norm for each tensor: a call that is all latency
        _norm("norm toy", TOY, "fp16", "fp16", 4, 1, per_tensor=True),
        # one decoder layer's share: the norm of a layer, looked at while training
        _norm("norm layer", LAYER, "bf16", "bf16", 8, 0),
        # a whole rank's share of a ragged set, every tensor's norm logged
        _norm("norm ragged share per tensor", RAGGED, "fp16", "fp16", 64, 63, per_tensor=True, loss_scale=1024.0),
        # a whole rank's share of the 8B set, norms' gradients kept in fp32: two types in one list
        _norm("norm 8B share", SHARE, "bf16", "fp32", 8, 0),
        # the largest magnitude, to set a loss scale by
        _norm("norm inf ragged share", RAGGED, "fp16", "fp32", 64, 63, kind="inf", loss_scale=1024.0),
        # the toy model's gradients clipped in place
        {"name": "clip toy", "op": "clip", "sizes": TOY, "dtype": "fp16", "small": "fp16", "out": "in place"},
        # a ragged share clipped in place, for an optimizer that takes no scale
        {"name": "clip ragged share", "op": "clip", "sizes": RAGGED, "dtype": "fp16", "small": "fp16", "out": "in place"},
        # fp32 sums handed on as bf16 gradients
        {"name": "clip fp32 layer to bf16", "op": "clip", "sizes": LAYER, "dtype": "fp32", "small": "fp32", "out": "bf16"},
        # the second of four micro-batches of the toy model
        _norm("accumulate toy", TOY, "fp16", "fp16", 4, 1, op="accumulate", first=False, norm=False, factor=0.25),
        # the first of four micro-batches of a ragged share: the accumulators' old contents do not count
        _norm("accumulate first ragged share", RAGGED, "fp16", "fp16", 64, 63, op="accumulate", first=True, norm=False, factor=0.25),
        # the last micro-batch of the 8B share, with the norm of the sum
        _norm("accumulate last 8B share", SHARE, "bf16", "bf16", 8, 0, op="accumulate", first=False, norm=True, factor=0.125),
        # a layer's last micro-batch, the norm of the sum and the clipped sum, as a trainer runs them
        _norm("update layer", LAYER, "bf16", "fp32", 8, 3, op="update", first=False, norm=True, factor=0.5, out="bf16"),
    ]


def _norm(name, sizes, dtype, small, world, rank, op="norm", kind="2", per_tensor=False, loss_scale=1.0, **more):
    return {"name": name, "op": op, "sizes": sizes, "dtype": dtype, "small": small, "world": world, "rank": rank,
            "kind": kind, "per_tensor": per_tensor, "loss_scale": loss_scale, **more}


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["norm", "norm", "clip", "accumulate", "accumulate", "update"])
    total = _log(rng, 3000, 400_000_000)
    kinds = rng.randint(1, 6)
    sizes = ",".join("%dx%d" % (c, max(1, int(total * rng.random() / (kinds * c)))) for c in (_log(rng, 1, 60) for _ in range(kinds)))
    dtype = rng.choice(["bf16", "fp16", "fp32"]) if op in ("norm", "clip") else rng.choice(["bf16", "fp16"])
    small = rng.choice([dtype, "fp32"])
    if op == "clip":
        return {"op": op, "sizes": sizes, "dtype": dtype, "small": small, "out": rng.choice(["in place", "bf16", "fp16", "fp32"])}
    world = rng.choice([1, 2, 4, 8, 48, 64])
    kind = rng.choice(["2", "2", "inf"])
    case = _norm("", sizes, dtype, small, world, rng.randrange(world), op=op, kind=kind, per_tensor=kind == "2" and rng.random() < 0.4,
                 loss_scale=rng.choice([1.0, 1024.0]))
    del case["name"]
    if op == "accumulate":
        case.update(first=rng.random() < 0.3, norm=rng.random() < 0.5, factor=1.0 / rng.choice([1, 2, 3, 8]))
    if op == "update":
        case.update(first=False, norm=True, factor=1.0 / rng.choice([1, 2, 3, 8]), out=dtype)
    return case


def _numels(case):
    """The persistent tensors come last."""
    n = [int(n) for c, n in (p.split("x") for p in case["sizes"].split(",")) for _ in range(int(c))]
    return [x for x in n if x >= PERSISTENT] + [x for x in n if x < PERSISTENT]


def _types(case):
    return [case["small"] if n < PERSISTENT else case["dtype"] for n in _numels(case)]


def work(case):
    """Bytes: the gradients once, the accumulators' old and new contents, the clipped gradients."""
    total = flops = 0
    for n, t in zip(_numels(case), _types(case)):
        total += n * BYTES[t]
        flops += 2 * n
        if case["op"] in ("accumulate", "update"):
            total += n * (4 if case["first"] else 8)
            flops += 2 * n
        if case["op"] in ("clip", "update"):
            total += n * BYTES[t if case["out"] == "in place" else case["out"]]
    return {"bytes": total, "flops": flops}


# ------------------------------------------------------------------ inputs

def _gradients(n, g, dtype):
    """Bell-shaped, one in a hundred a hundred times as large."""
    x = torch.randn(n, device=DEV, generator=g) * 1e-3
    x = torch.where(torch.rand(n, device=DEV, generator=g) < 0.01, x * 100, x)
    return x.to(dtype)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    sizes, types = _numels(case), _types(case)
    total = sum(sizes)
    st = {"case": case, "sizes": sizes, "types": types, "flat": {}}
    # where each tensor starts in its type's buffer, and in one over all of them
    used, st["start"], st["place"] = {}, [], []
    for n, t in zip(sizes, types):
        st["start"].append(used.get(t, 0))
        st["place"].append(st["place"][-1] + last if st["place"] else 0)
        used[t] = used.get(t, 0) + n
        last = n
    for t in used:
        st["flat"][t] = _gradients(used[t], g, DTYPES[t])
    if case["op"] in ("accumulate", "update"):
        st["acc"] = _gradients(total, g, torch.float32)
    if case["op"] == "clip":
        st["scale"] = torch.full((1,), 0.9375, device=DEV)
        st["nonfinite"] = torch.zeros(1, dtype=torch.int32, device=DEV)
        if case["out"] != "in place":
            st["out"] = torch.empty(total, dtype=DTYPES[case["out"]], device=DEV)
    else:
        # what the peers' all-reduce holds: sums of squares, or largest magnitudes, like the own one
        unit = total * 1e-4 if case["kind"] == "2" else 0.3
        st["sums"] = (unit * (0.5 + torch.rand(case["world"] + 1, device=DEV, generator=g))).double()
        st["norm"] = torch.zeros(1, dtype=torch.float64, device=DEV)
        st["scale"] = torch.zeros(1, device=DEV)
        st["nonfinite"] = torch.zeros(1, dtype=torch.int32, device=DEV)
        st["tensor_norms"] = torch.zeros(len(sizes), dtype=torch.float64, device=DEV)
        st["ends"] = torch.tensor([0] + [p + n for p, n in zip(st["place"], sizes)], device=DEV)
        st["partitioned"] = sum(n for n in sizes if n >= PERSISTENT)
        if case["op"] == "update":
            st["out"] = torch.empty(total, dtype=DTYPES[case["out"]], device=DEV)
    return st


# -------------------------------------------------------------- plain forms

def _all(st):
    """Every gradient in list order, in 32 bits."""
    case, flat = st["case"], st["flat"]
    if len(flat) == 1:
        return flat[st["types"][0]].float()
    return torch.cat([flat[case["dtype"]].float(), flat[case["small"]].float()])


def _norm_plain(st, x):
    case, rank, world, k = st["case"], st["case"]["rank"], st["case"]["world"], st["partitioned"]
    if case["kind"] == "2":
        sq = x.double().square()
        if case["per_tensor"]:
            upto = torch.cat([torch.zeros(1, dtype=torch.float64, device=DEV), sq.cumsum(0)])[st["ends"]]
            st["tensor_norms"].copy_((upto[1:] - upto[:-1]).clamp(min=0).sqrt())
        st["sums"][rank], st["sums"][world] = sq[:k].sum(), sq[k:].sum()
        total = st["sums"].sum()
        norm = total.sqrt() / case["loss_scale"]
    else:
        x = torch.cat([torch.zeros(1, device=DEV), x.abs(), torch.zeros(1, device=DEV)])
        st["sums"][rank], st["sums"][world] = x[:k + 1].max(), x[k + 1:].max()
        total = st["sums"].max()
        norm = total / case["loss_scale"]
    st["norm"].copy_(norm)
    st["nonfinite"].copy_(~torch.isfinite(total))
    coef = torch.clamp(1.0 / (norm + 1e-6), max=1.0) / case["loss_scale"]
    st["scale"].copy_(torch.where(torch.isfinite(total), coef, float("nan")))


def _plain(st):
    case, flat = st["case"], st["flat"]
    if case["op"] == "norm":
        _norm_plain(st, _all(st))
    elif case["op"] == "clip":
        if case["out"] != "in place":
            st["out"].copy_(_all(st) * st["scale"])
            return
        first, last = st["types"][0], st["types"][-1]
        flat[first].copy_(flat[first].float() * st["scale"])
        if last != first:
            flat[last].copy_(flat[last].float() * st["scale"])
    else:
        if case["first"]:
            torch.mul(_all(st), case["factor"], out=st["acc"])
        else:
            st["acc"].add_(_all(st), alpha=case["factor"])      # rounded once
        if case["norm"]:
            _norm_plain(st, st["acc"])
        if case["op"] == "update":
            st["out"].copy_(st["acc"] * st["scale"])


def _own_list(st):
    import zero_sharded_state_amd as zs3
    case, out = st["case"], []
    for n, t, s, p in zip(st["sizes"], st["types"], st["start"], st["place"]):
        d = dict(numel=n, grad=st["flat"][t].data_ptr() + BYTES[t] * s, dtype=t, shared=n < PERSISTENT)
        if "acc" in st:
            d.update(out=st["acc"].data_ptr() + 4 * p, out_dtype="fp32")
        elif "out" in st:
            d.update(out=st["out"].data_ptr() + BYTES[case["out"]] * p, out_dtype=case["out"])
        out.append(d)
    st["list"] = zs3.zs3_grad_tensor_list(out)
    if case["op"] == "update":
        st["clip_list"] = zs3.zs3_grad_tensor_list([
            dict(numel=n, grad=st["acc"].data_ptr() + 4 * p, dtype="fp32", out=st["out"].data_ptr() + 2 * p, out_dtype=case["out"])
            for n, p in zip(st["sizes"], st["place"])])
    if case["op"] != "clip":
        st["workspace"] = torch.zeros(zs3.zs3_norm_workspace_bytes(st["list"]), dtype=torch.uint8, device=DEV)
        st["norm_args"] = zs3.zs3_norm_args_of(
            kind=zs3.ZS3_NORM_2 if case["kind"] == "2" else zs3.ZS3_NORM_INF, rank=case["rank"], world=case["world"], max_norm=1.0,
            loss_scale=case["loss_scale"], sums=st["sums"], norm=st["norm"], scale=st["scale"], nonfinite=st["nonfinite"],
            tensor_norms=st["tensor_norms"] if case["per_tensor"] else None, workspace=st["workspace"])


def _own(st):
    import zero_sharded_state_amd as zs3
    case = st["case"]
    if "list" not in st:
        _own_list(st)
    if case["op"] == "norm":
        zs3.zs3_grad_norm_tensors(st["list"], st["norm_args"])
    elif case["op"] == "clip":
        zs3.zs3_clip_tensors(st["list"], st["scale"], st["nonfinite"])
    else:
        zs3.zs3_accumulate_tensors(st["list"], case["factor"], first=case["first"], norm=st["norm_args"] if case["norm"] else None)
        if case["op"] == "update":
            zs3.zs3_clip_tensors(st["clip_list"], st["scale"], st["nonfinite"])


def run(state):
    case = state["case"]
    if own:
        _own(state)
    else:
        _plain(state)
    out = {}
    if case["op"] != "clip" and case.get("norm", True):
        out = {k: state[k] for k in ("norm", "scale", "nonfinite", "sums") + (("tensor_norms",) if case["per_tensor"] else ())}
    if case["op"] in ("accumulate", "update"):
        out["acc"] = state["acc"]
    if "out" in state:
        out["out"] = state["out"]
    elif case["op"] == "clip":
        out.update(state["flat"])
    return out


# ------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    x = [st["flat"][t][s:s + n].double() for n, t, s in zip(st["sizes"], st["types"], st["start"])]
    if case["op"] == "clip":
        y = [0.9375 * v for v in x]
        if case["out"] != "in place":
            return {"out": torch.cat(y)}
        return {t: torch.cat([v for v, u in zip(y, st["types"]) if u == t]) for t in st["flat"]}
    out = {}
    if case["op"] != "norm":
        factor = float(torch.tensor(case["factor"], dtype=torch.float32))
        x = [v * factor + (0.0 if case["first"] else st["acc"][p:p + n].double()) for v, n, p in zip(x, st["sizes"], st["place"])]
    if case.get("norm", True):
        held = x if case["op"] == "norm" else [v.float().double() for v in x]      # the norm is that of the accumulators, 32 bits each
        each = [float(torch.dot(v, v)) if case["kind"] == "2" else float(v.abs().max()) for v in held]
        join = math.fsum if case["kind"] == "2" else lambda v: max(v, default=0.0)
        sums = [float(v) for v in st["sums"]]
        sums[case["rank"]] = join([e for e, n in zip(each, st["sizes"]) if n >= PERSISTENT])
        sums[case["world"]] = join([e for e, n in zip(each, st["sizes"]) if n < PERSISTENT])
        root = math.sqrt if case["kind"] == "2" else float
        norm = root(join(sums)) / case["loss_scale"]
        scale = min(1.0, 1.0 / (norm + 1e-6)) / case["loss_scale"]
        t64 = lambda v: torch.tensor(v, dtype=torch.float64, device=DEV)  # noqa: E731
        out = {"norm": t64([norm]), "scale": t64([scale]), "nonfinite": None, "sums": t64(sums)}
        if case["per_tensor"]:
            out["tensor_norms"] = t64([root(e) for e in each])
    if case["op"] != "norm":
        out["acc"] = torch.cat(x)
    if case["op"] == "update":
        out["out"] = out["acc"] * scale
    return out
