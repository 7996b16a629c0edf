"""Pins of the low-bit oracle (``oracle/lowbit.py``): the code tables against
torch's e4m3 type, rounding against exhaustive search over the codes,
stochastic rounding's mean over random words, the counter hash's uniformity,
AdamW against ``torch.optim.AdamW`` and the flat Adam oracle, and the wire's
places against the 16-bit wire's oracle."""

import numpy as np
import pytest
import torch

import oracle
from oracle import lowbit as lb

RNG = np.random.default_rng


def test_code_tables():
    t = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(lb.E4M3, t)
    # unsigned codes of 4 + 4 bits: from 0 to 31/16 * 2^8, each binade in 16 steps
    assert lb.E4M4[0] == 0 and lb.E4M4[1] == 2.0 ** -10 and lb.E4M4[255] == 496 and len(lb.E4M4) == 256
    assert np.all(np.diff(lb.E4M4) > 0) and np.array_equal(lb.E4M4[16:] * 2, np.append(lb.E4M4[32:], 512 * (1 + np.arange(16) / 16)))


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_nearest_wire_codes_by_exhaustive_search(dtype):
    """The scale is the smallest power of two with |x| < 7 of it, and every
    element's code is a nearest one: |error| <= half of the spacing (0.5, 1 or 2
    scales by binade), with the even code on ties."""
    rng = RNG(1)
    x = oracle.to_f32(oracle.from_f32((rng.standard_normal(32 * 300) * np.exp(rng.standard_normal(32 * 300) * 2)).astype(np.float32), dtype), dtype)
    x[64:96] = 0
    x[96:128] = oracle.to_f32(oracle.from_f32(np.linspace(-7, 7, 32, dtype=np.float32), dtype), dtype)
    x[128:160] = np.tile([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], 4) * np.repeat([1, -1, 1, -1], 8)   # ties
    code, s = lb.encode4(x, dtype)
    e = s.astype(int) - 127
    top = np.abs(x.reshape(-1, 32)).max(1)
    live = top > 0
    assert np.all(top[live] < 7 * 2.0 ** e[live]) and np.all(top[live] >= 7 * 2.0 ** (e[live] - 1))
    assert np.all(e[~live] == -126)
    y = np.abs(x.astype(np.float64)) / np.repeat(2.0 ** e, 32)
    dist = np.abs(y[:, None] - lb.E2M1[None])
    best = dist.min(1)
    got = dist[np.arange(len(y)), code & 7]
    assert np.array_equal(got, best)
    tie = (dist == best[:, None]).sum(1) == 2
    assert tie[128:160].sum() == 28 and np.all((code[tie] & 1) == 0)
    spacing = np.where(y < 2, 0.5, np.where(y < 4, 1.0, 2.0))
    assert np.all(got <= spacing / 2)
    assert np.array_equal((code >> 3) == 1, np.signbit(x))
    # what the codes stand for is exact in 16 bits
    v = lb.decode4(code, s)
    assert np.array_equal(oracle.to_f32(oracle.from_f32(v, dtype), dtype), v)


def test_wire_range_ends():
    """Magnitudes at the 16-bit types' ends stay finite, and a block that holds a
    value that is not finite is NaN as a whole."""
    for dtype, big, e in (("fp16", 65504.0, 13), ("bf16", 3.3895314e38, 125)):
        x = np.zeros(64, np.float32)
        x[0], x[1] = big, -1.0
        code, s = lb.encode4(x, dtype)
        assert s[0] == e + 127 and np.isfinite(oracle.to_f32(oracle.from_f32(lb.decode4(code, s), dtype), dtype)).all()
        x[40] = np.inf
        x[1] = np.nan
        code, s = lb.encode4(x, dtype)
        assert list(s) == [255, 255] and np.isnan(lb.decode4(code, s)).all()
    x = np.full(32, 2.0 ** -24, np.float32)            # the smallest fp16
    assert np.array_equal(lb.decode4(*lb.encode4(x, "fp16")), x)


@pytest.mark.parametrize("kind", ["first", "second", "wire"])
def test_stochastic_rounding_keeps_the_mean(kind):
    """Over 4096 random words, the average of a value's codes is the value: its
    distance has a standard deviation of at most spacing / 2 / sqrt(4096), and
    6 of those are allowed (the chance of one of 640 values past 6 is 1e-6)."""
    rng = RNG(2)
    x = np.abs(rng.standard_normal(32)).astype(np.float32) * np.exp(rng.uniform(-3, 0, 32)).astype(np.float32)
    if kind == "wire":
        x = oracle.to_f32(oracle.from_f32(x, "bf16"), "bf16")
    n, total = 4096, np.zeros(32)
    for k in range(n):
        word = lb.words(lb.keys(7, k, 3), np.arange(32))
        if kind == "wire":
            total += lb.decode4(*lb.encode4(x, "bf16", word))
        else:
            second = kind == "second"
            total += lb.decode_moment(*lb.encode_moment(x, word, second), second)
    top = float(x.max())
    table = {"first": lb.E4M3, "second": lb.E4M4, "wire": lb.E2M1}[kind]
    e = float(np.floor(np.log2(top / table[-1])) + 1)
    y = x / 2.0 ** e
    i = np.searchsorted(table, y, side="right") - 1
    spacing = (table[np.minimum(i + 1, len(table) - 1)] - table[i]) * 2.0 ** e
    assert np.all(np.abs(total / n - x) <= 6 * spacing / 2 / np.sqrt(n) + 1e-12)


def test_moments_round_to_a_neighbour_and_never_to_zero():
    rng = RNG(3)
    x = (np.abs(rng.standard_normal(32 * 200)) * np.exp(rng.uniform(-12, 0, 32 * 200))).astype(np.float32)
    x[:5] = [0, 1e-30, 1e-8, 1.0, 0]
    for second in (False, True):
        table = lb.E4M4 if second else lb.E4M3
        code, s = lb.encode_moment(x, lb.words(5, np.arange(len(x))), second)
        e = s.astype(int) - 127
        top = x.reshape(-1, 32).max(1).astype(np.float64)
        assert np.all(top <= table[-1] * 2.0 ** e) and np.all(top > table[-1] * 2.0 ** (e - 1))
        y = x / np.repeat(2.0 ** e, 32)
        lo = np.searchsorted(table, y, side="right") - 1
        up = code.astype(int) - lo
        assert set(np.unique(up)) <= {0, 1} and np.all(up[table[lo] == y] == 0)
        if second:
            assert np.all((code == 0) == (x == 0))
    neg, _ = lb.encode_moment(-x, lb.words(5, np.arange(len(x))), False)
    pos, _ = lb.encode_moment(x, lb.words(5, np.arange(len(x))), False)
    assert np.array_equal(neg, pos | 0x80)
    bad = np.ones(64, np.float32)
    bad[33] = np.nan
    for second in (False, True):
        code, s = lb.encode_moment(bad, np.zeros(64, np.uint32), second)
        v = lb.decode_moment(code, s, second)
        assert np.isfinite(v[:32]).all() and not np.isfinite(v[32:]).any() and s[1] == 255


def test_random_words_are_uniform():
    """Chi-square of the bits that rounding takes (upper 8 of the upper 20,
    upper 8 of the lower 16) over 2^18 consecutive indices: 255 degrees of
    freedom, under mean + 6 standard deviations; neighbours' correlation under
    6 / sqrt(n); other seeds, steps and ids give other words."""
    n = 1 << 18
    for key in (lb.keys(0, 1, 0), lb.keys(1, 1, 0), lb.keys(0, 2, 0), lb.keys(0, 1, 1)):
        w = lb.words(key, np.arange(n))
        for part in (w >> np.uint32(24), (w >> np.uint32(8)) & np.uint32(255)):
            chi = ((np.bincount(part.astype(int), minlength=256) - n / 256) ** 2 / (n / 256)).sum()
            assert chi < 255 + 6 * np.sqrt(2 * 255)
        u = w / 2.0 ** 32 - 0.5
        for lag in (1, 2, 32, 64):
            assert abs(np.mean(u[lag:] * u[:-lag]) * 12) < 6 / np.sqrt(n)
        lo = (w & np.uint32(0xFFFF)) / 65536.0 - 0.5
        assert abs(np.mean(lo * u) * 12) < 6 / np.sqrt(n)
    a, b = lb.words(lb.keys(0, 1, 0), np.arange(n)), lb.words(lb.keys(0, 2, 0), np.arange(n))
    assert np.mean(a == b) < 1e-4
    far = lb.words(lb.keys(0, 1, 0), np.arange(n) + (1 << 32))
    assert np.mean(a == far) < 1e-4


@pytest.mark.parametrize("wd", [0.0, 0.1])
def test_adamw_is_the_flat_adam_and_torchs(wd):
    rng = RNG(4)
    n = 257
    L = oracle.make_layout(1, 0, [0], [n])
    w0 = rng.standard_normal(n).astype(np.float32)
    w, m, v = w0.copy(), np.zeros(n, np.float32), np.zeros(n, np.float32)
    fw, fm, fv = w0.copy(), np.zeros(n, np.float32), np.zeros(n, np.float32)
    p = torch.nn.Parameter(torch.from_numpy(w0.astype(np.float64)))
    opt = torch.optim.AdamW([p], lr=1e-3, betas=(0.9, 0.99), eps=1e-8, weight_decay=wd)
    for step in range(1, 6):
        g = oracle.from_f32(rng.standard_normal(n).astype(np.float32), "bf16")
        w, m, v, _, _ = lb.adamw(w, m, v, oracle.to_f32(g, "bf16"), scale=1.0, lr=1e-3, wd=wd, beta1=0.9, beta2=0.99, eps=1e-8, step=step)
        oracle.adam_step(L, 0, "bf16", 0, n, fw, fm, fv, g, np.zeros(n, np.uint16), np.float32(1.0), False,
                         oracle.AdamHParams(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=wd, step=step))
        p.grad = torch.from_numpy(oracle.to_f32(g, "bf16").astype(np.float64))
        opt.step()
        for a, b in ((w, fw), (m, fm), (v, fv)):
            assert np.array_equal(a.view(np.uint32), b.view(np.uint32))
    # 5 steps of about 5 roundings each, relative to weights of up to 4
    assert np.abs(w - p.detach().numpy()).max() <= 5 * 5 * 2.0 ** -24 * 4


def test_8bit_second_moment_follows_its_mean():
    """Over 3000 steps of gradients with variance s^2 and beta2 = 0.99, the
    stored second moment stays near s^2 on average (stochastic rounding adds
    noise and no drift); rounded to the nearest, it stands still."""
    rng = RNG(5)
    n, b2, sigma = 1024, 0.99, 1e-3
    v = np.full(n, (4 * sigma) ** 2, np.float32)           # starts 16 times too large
    stuck = v.copy()
    sums = np.zeros(n)
    for k in range(3000):
        g2 = ((rng.standard_normal(n) * sigma) ** 2).astype(np.float32)
        v = np.float32(b2) * v + np.float32(1 - b2) * g2
        v = lb.decode_moment(*lb.encode_moment(v, lb.words(lb.keys(1, k, 0), np.arange(n)), True), True)
        stuck = np.float32(b2) * stuck + np.float32(1 - b2) * g2
        stuck = lb.decode_moment(*lb.encode_moment(stuck, np.full(n, 1 << 15, np.uint32), True), True)
        if k >= 1000:
            sums += v
    # the mean over 1024 x 2000 correlated samples: 1024 * 2000 / 100 independent
    # ones, each within 2 sigma^2, so 1% is over 6 standard deviations
    assert abs(sums.mean() / 2000 / sigma ** 2 - 1) < 0.01
    assert stuck.mean() > 2 * sigma ** 2


@pytest.mark.parametrize("world,sizes", [(1, [5]), (3, [100, 1, 33]), (4, [64, 7, 1000]), (8, [3, 4095])])
def test_wire_places(world, sizes):
    """With values that 4 bits hold exactly, the 4-bit wire carries what the
    16-bit wire does, whatever the padding positions of the shard hold."""
    rng = RNG(6)
    ids = [10 + 3 * i for i in range(len(sizes))]
    L = oracle.make_layout(world, 0, ids, sizes)
    full = {d: oracle.from_f32((rng.choice(lb.E2M1, n) * rng.choice([-1, 1], n)).astype(np.float32), "fp16") for d, n in zip(ids, sizes)}
    for d in ids:                      # +0 and -0 as the codes give them; a 4 so that the scale is 1 for all blocks
        full[d][::16] = oracle.from_f32(np.full(len(full[d][::16]), 4, np.float32), "fp16")
    request = ids[::-1]
    chunks = []
    for r in range(world):
        shard = oracle.partition(L, r, full)
        for p in L.params:
            lo, hi = L.own_range(p, r)
            shard[p.shard_offset + hi - lo:p.shard_offset + p.partition_size] = 0x7E00
        chunks.append(lb.pack4(L, r, request, shard, "fp16"))
    got = lb.unpack4(L, request, chunks, "fp16")
    assert np.array_equal(got, np.concatenate([full[d] for d in ids]))
    send = lb.send4(L, request, full, "fp16")
    assert np.array_equal(send, np.stack(chunks))
    for r in range(world):             # identical gradients from every rank average to themselves (powers of two)
        if world & (world - 1):
            continue
        flat = np.full(L.shard_numel, 0x1234, np.uint16)
        lb.reduce4(L, r, request, [lb.send4(L, request, full, "fp16")[r]] * world, "fp16", flat)
        ref = oracle.partition(L, r, full)
        assert np.array_equal(oracle.to_f32(flat, "fp16"), oracle.to_f32(ref, "fp16"))


@pytest.mark.parametrize("f", [0.05, 0.1, 0.25, 0.5, 0.75, 0.95])
def test_pairs_of_the_stochastic_wire_correlate_as_stated(f):
    """Two neighbours a fraction f of the way to the next code: each goes up with
    probability f, and the two correlate by (0.5 - f) / (1 - f), from f = 0.5 on
    by (f - 0.5) / f, since the second's word is the first's rotated by a bit
    (2u mod 1 beside u).  Within five deviations of a million pairs: sqrt(f(1-f)
    / n) of a mean, and at most sqrt(1 / min(f, 1-f) / n) of a correlation."""
    n = 1 << 21
    x = np.full(n, 0.5 * f, np.float32)
    x[31::32] = 6.0                                     # a scale of 1
    at = np.arange(n)
    word = lb.words(lb.keys(123, 0, 0), at // 2)
    word = np.where(at % 2 == 0, word, (word << np.uint32(1)) | (word >> np.uint32(31)))
    code, s = lb.encode4(x, "bf16", word)
    assert np.all(s == 127) and np.all(code[31::32] == 7)
    pairs = code.reshape(-1, 16, 2)[:, :15].reshape(-1, 2).astype(np.float64)       # the last pair of a block apart
    assert set(np.unique(pairs)) <= {0, 1}
    k = len(pairs)
    assert np.all(np.abs(pairs.mean(0) - f) <= 5 * np.sqrt(f * (1 - f) / k) + 2.0 ** -24)
    want = (0.5 - f) / (1 - f) if f <= 0.5 else (f - 0.5) / f
    assert abs(np.corrcoef(pairs.T)[0, 1] - want) <= 5 * np.sqrt(1 / min(f, 1 - f) / k)


def test_seed_zero_draws_a_zero_first():
    """The wire's first word of seed 0 is 0, of others it is not: the first pair
    of a send buffer then rounds toward zero."""
    assert lb.keys(0, 0, 0) == 0 and lb.words(0, np.arange(1))[0] == 0
    assert all(lb.words(lb.keys(s, 0, 0), np.arange(1))[0] != 0 for s in range(1, 1000))
