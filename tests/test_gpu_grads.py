"""GPU: the norm, clip and accumulation of gradient lists against the oracle
(``oracle.grads``).

Norms: all terms are positive, so a sum of n of them in binary64 is within n *
2^-53 of itself, whatever its order, and squares of fp32 values are off by 2^-53 at most; the root
halves that and adds an ulp.  The largest magnitude, clipped gradients and
accumulators are compared bit for bit."""

import math

import numpy as np
import pytest

import oracle
import zero_sharded_state_amd as zs
from gpu_util import Buf16, Buf32, note, require_gpu, sync
from oracle import grads as og

pytestmark = pytest.mark.gpu
KINDS = {"2": zs.ZS3_NORM_2, "inf": zs.ZS3_NORM_INF}
SIZES = [1, 2, 3, 4, 5, 7, 8, 9, 31, 63, 64, 65, 255, 257, 1023, 2047, 2048, 2049, 4095, 4096, 4097, 10007]


def _buf(n, dtype, shift=0, fill=None):
    return (Buf32 if dtype == "fp32" else Buf16)(n, shift, fill)


def _bits(x, dtype):
    return np.asarray(x, np.float32) if dtype == "fp32" else oracle.from_f32(np.asarray(x, np.float32), dtype)


def _same(a, b):
    """Bit for bit, NaN as NaN."""
    a, b = np.asarray(a), np.asarray(b)
    assert a.dtype == b.dtype and a.shape == b.shape
    if a.dtype == np.float32:
        ok = (a.view(np.uint32) == b.view(np.uint32)) | (np.isnan(a) & np.isnan(b))
        assert ok.all(), (int((~ok).sum()), int((~ok).argmax()))
    else:
        assert np.array_equal(a, b), (int((a != b).sum()), int((a != b).argmax()))


class Tensor:
    def __init__(self, rng, n, dtype, shift=0, shared=False, out=None, out_shift=0, mag=1e-3, special=()):
        self.n, self.dtype, self.shared, self.out_dtype = n, dtype, shared, out
        x = rng.standard_normal(n).astype(np.float32) * np.float32(mag)
        for i, v in special:
            x[i] = v
        self.bits = _bits(x, dtype)
        self.x = og.widened(self.bits, dtype)
        self.g = _buf(n, dtype, shift, self.bits)
        self.acc = None
        self.o = None
        if out == "acc":
            self.acc = (rng.standard_normal(n) * 1e-3).astype(np.float32)
            self.o = Buf32(n, out_shift, self.acc)
        elif out is not None:
            self.o = _buf(n, out, out_shift)

    def entry(self):
        d = dict(numel=self.n, grad=self.g.ptr(), dtype=self.dtype, shared=self.shared)
        if self.o is not None:
            d.update(out=self.o.ptr(), out_dtype="fp32" if self.out_dtype == "acc" else self.out_dtype)
        return d

    def guards(self):
        self.g.check_guards()
        if self.o is not None:
            self.o.check_guards()


class Norm:
    """The outputs of a norm, between canaries."""

    def __init__(self, entries, kind="2", rank=0, world=1, peers=None, max_norm=1.0, loss_scale=1.0, per_tensor=True, finalize=True):
        import torch
        n = len(entries)
        self.kind, self.rank, self.world, self.max_norm, self.loss_scale = kind, rank, world, max_norm, loss_scale
        self.peers = list(peers) if peers is not None else [0.0] * (world + 1)
        self.base = torch.full((world + 1 + n + 12,), -7.5, dtype=torch.float64, device="cuda")
        self.sums, self.norm, self.each = self.base[2:world + 3], self.base[world + 5:world + 6], self.base[world + 8:world + 8 + n]
        self.sums.copy_(torch.tensor(self.peers, dtype=torch.float64))
        self.scale = torch.full((3,), -7.5, dtype=torch.float32, device="cuda")
        self.flag = torch.full((3,), -7, dtype=torch.int32, device="cuda")
        self.ws = torch.zeros(zs.zs3_norm_workspace_bytes(entries), dtype=torch.uint8, device="cuda")
        self.per_tensor, self.n = per_tensor, n
        self.args = zs.zs3_norm_args_of(kind=KINDS[kind], rank=rank, world=world, finalize=finalize, max_norm=max_norm,
                                        loss_scale=loss_scale, sums=self.sums, norm=self.norm, scale=self.scale[1:2],
                                        nonfinite=self.flag[1:2], tensor_norms=self.each if per_tensor else None, workspace=self.ws)

    def got(self):
        return dict(sums=self.sums.cpu().numpy().copy(), norm=float(self.norm.cpu()), scale=float(self.scale[1].cpu()),
                    flag=int(self.flag[1].cpu()), each=self.each.cpu().numpy().copy())

    def check(self, tensors):
        """``tensors``: (fp32 values, shared)."""
        g = self.got()
        count = sum(len(x) for x, _ in tensors) + self.world + 2
        tol = count * 2.0 ** -53 if self.kind == "2" else 0.0
        want = og.sums(tensors, self.kind, self.peers, self.rank)
        np.testing.assert_allclose(g["sums"], want, rtol=tol, atol=0)
        norm, scale, bad = og.finalize(want, self.kind, self.max_norm, self.loss_scale)
        np.testing.assert_allclose(g["norm"], norm, rtol=tol + 2.0 ** -51, atol=0)
        assert g["flag"] == int(bad)
        # rounded to fp32: by 2^-24 of itself at most, or, below 2^-126, by half of the
        # subnormals' spacing of 2^-149
        np.testing.assert_allclose(g["scale"], scale, rtol=tol + 2.0 ** -24 + 2.0 ** -50, atol=2.0 ** -150)
        if self.per_tensor:
            each = [og.part(x, self.kind) for x, _ in tensors]
            each = [math.sqrt(e) if self.kind == "2" and not math.isnan(e) else e for e in each]
            np.testing.assert_allclose(g["each"], each, rtol=tol + 2.0 ** -51, atol=0)
        b = self.base.cpu().numpy()
        assert np.all(b[:2] == -7.5) and np.all(b[self.world + 3:self.world + 5] == -7.5)
        assert np.all(b[self.world + 6:self.world + 8] == -7.5) and np.all(b[self.world + 8 + self.n:] == -7.5)
        assert self.scale[0] == -7.5 and self.scale[2] == -7.5 and self.flag[0] == -7 and self.flag[2] == -7


def _norm(tensors, **kw):
    entries = [t.entry() for t in tensors]
    n = Norm(entries, **kw)
    zs.zs3_grad_norm_tensors(entries, n.args)
    sync()
    n.check([(t.x, t.shared) for t in tensors])
    for t in tensors:
        t.guards()
        _same(t.g.host(), t.bits)
    return n


# ------------------------------------------------------------------ the norm

@pytest.mark.parametrize("kind", ["2", "inf"])
@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("shift", [0, 1, 3])
def test_norm_of_lists(kind, dtype, shift):
    require_gpu()
    note(f"norm {kind} {dtype} shift {shift}")
    rng = np.random.default_rng(shift)
    for k in range(0, len(SIZES), 4):
        _norm([Tensor(rng, n, dtype, shift + i, shared=i % 3 == 1) for i, n in enumerate(SIZES[k:k + 4])], kind=kind, rank=1, world=3,
              peers=[0.25, 9.0, 0.5, 9.0])
    _norm([Tensor(rng, n, dtype, shift, shared=n % 2 == 0) for n in SIZES], kind=kind)


@pytest.mark.parametrize("n", SIZES)
def test_norm_of_one_tensor(n):
    require_gpu()
    note(f"one tensor of {n}")
    rng = np.random.default_rng(n)
    for dtype in ("fp16", "fp32"):
        _norm([Tensor(rng, n, dtype, n % 5)])


def test_norm_of_mixed_types_many_tensors():
    """More tensors than a launch holds, empty ones among them, in the three types."""
    require_gpu()
    note("600 mixed tensors")
    rng = np.random.default_rng(3)
    sizes = [int(rng.integers(1, 3000)) for _ in range(600)]
    ts = [Tensor(rng, n, ("fp16", "bf16", "fp32")[i % 3], i % 7, shared=i % 5 == 0) for i, n in enumerate(sizes)]
    entries = [t.entry() for t in ts]
    values = [(t.x, t.shared) for t in ts]
    for at in (0, 1, 224, 225, 300, 606):
        entries.insert(at, dict(numel=0, grad=0, dtype="fp16", shared=at % 2))
        values.insert(at, (np.zeros(0, np.float32), False))
    for kind in ("2", "inf"):
        n = Norm(entries, kind=kind, rank=0, world=2, peers=[0.0, 0.125, 0.0])
        zs.zs3_grad_norm_tensors(entries, n.args)
        sync()
        n.check(values)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_norm_of_large_tensors(dtype):
    """Many tiles a workgroup, tensors that span many workgroups and workgroups that span tensors."""
    require_gpu()
    note(f"large {dtype}")
    rng = np.random.default_rng(4)
    sizes = [9_000_001, 5, 4095, 3_000_000, 1, 700_001] + [1000 + 17 * i for i in range(40)]
    _norm([Tensor(rng, n, dtype, i % 3, shared=i % 4 == 2) for i, n in enumerate(sizes)])
    _norm([Tensor(rng, n, dtype, i % 3) for i, n in enumerate(sizes)], kind="inf")


@pytest.mark.parametrize("count,numel", [(1, 40_000_000), (700, 20_001), (1500, 20_001), (3000, 20_001)])
@pytest.mark.parametrize("kind", ["2", "inf"])
def test_joins_of_many_partial_sums(kind, count, numel):
    """Lists past what the last workgroup and what one workgroup join, over several launches.
    Small whole numbers: every sum of their squares is exact, in any order."""
    import torch
    require_gpu()
    note(f"{count} tensors of {numel}, {kind}")
    g = torch.Generator(device="cuda")
    g.manual_seed(count)
    flat = torch.randint(-8, 9, (count * numel,), device="cuda", generator=g).to(torch.bfloat16)
    flat[-1] = 15.0
    acc = torch.full((count * numel,), math.nan, device="cuda")
    entries = [dict(numel=numel, grad=flat.data_ptr() + 2 * numel * i, dtype="bf16", out=acc.data_ptr() + 4 * numel * i,
                    out_dtype="fp32", shared=i % 3 == 1) for i in range(count)]
    x = flat.view(count, numel).double()
    each = x.square().sum(1) if kind == "2" else x.abs().amax(1)
    shared = torch.arange(count, device="cuda") % 3 == 1
    join = (lambda v: float(v.sum())) if kind == "2" else (lambda v: float(v.max()) if v.numel() else 0.0)
    want = [join(each[~shared]), join(each[shared])]
    total = sum(want) if kind == "2" else max(want)
    arr = zs.zs3_grad_tensor_list(entries)
    for f in (1.0, 2.0):                # acc = x, then 2 x + x
        n = Norm(entries, kind=kind, max_norm=math.inf)
        zs.zs3_grad_norm_tensors(arr, n.args)
        fused = Norm(entries, kind=kind, max_norm=math.inf)
        zs.zs3_accumulate_tensors(arr, f, first=f == 1.0, norm=fused.args)
        torch.cuda.synchronize()
        for got, k in ((n.got(), 1), (fused.got(), 1 if f == 1.0 else 3)):
            power = k * k if kind == "2" else k
            assert got["sums"].tolist() == [power * w for w in want] and got["flag"] == 0
            assert got["norm"] == (math.sqrt(power * total) if kind == "2" else power * total)
            root = torch.sqrt(power * each) if kind == "2" else power * each
            np.testing.assert_allclose(got["each"], root.cpu().numpy(), rtol=2.0 ** -52 if kind == "2" else 0.0)
    assert torch.equal(acc, 3 * flat.float())


def test_norm_without_elements():
    require_gpu()
    note("empty lists")
    for entries in ([], [dict(numel=0, grad=0, dtype="bf16")] * 3):
        n = Norm(entries, rank=0, world=2, peers=[5.0, 4.0, 5.0])
        zs.zs3_grad_norm_tensors(entries, n.args)
        sync()
        n.check([(np.zeros(0, np.float32), False)] * len(entries))
        assert n.got()["norm"] == 2.0 and n.got()["scale"] == np.float32(1.0 / (2.0 + 1e-6))


@pytest.mark.parametrize("kind", ["2", "inf"])
@pytest.mark.parametrize("value", [np.inf, -np.inf, np.nan])
@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
def test_norm_flags_what_is_not_finite(kind, value, dtype):
    require_gpu()
    note(f"{value} in {dtype}, {kind}")
    rng = np.random.default_rng(5)
    for n, at in ((1, 0), (9, 0), (9, 8), (5000, 0), (5000, 2500), (5000, 4999), (300_000, 299_999)):
        n_ = _norm([Tensor(rng, 7, dtype), Tensor(rng, n, dtype, 1, special=[(at, value)]), Tensor(rng, 7, dtype)], kind=kind)
        assert n_.got()["flag"] == 1 and math.isnan(n_.got()["scale"])


def test_norm_of_extreme_values():
    """fp32 values whose squares are far outside fp32, both ways, and zeros."""
    require_gpu()
    note("extremes")
    rng = np.random.default_rng(6)
    for mag in (1e30, 3e38, 1e-30, 1e-44, 0.0):
        t = Tensor(rng, 3000, "fp32", mag=1.0)
        x = np.clip(t.x.astype(np.float64) * mag, -3.4e38, 3.4e38).astype(np.float32)
        t = Tensor(rng, 3000, "fp32", special=list(enumerate(x)))
        n = _norm([t], max_norm=1.0)
        assert n.got()["flag"] == 0
        _norm([t], kind="inf")


@pytest.mark.parametrize("kind", ["2", "inf"])
def test_norm_finalize_alone_and_measured_only(kind):
    import torch
    require_gpu()
    note(f"finalize alone {kind}")
    rng = np.random.default_rng(7)
    ts = [Tensor(rng, 5000, "fp16", shared=i == 1) for i in range(3)]
    entries, values = [t.entry() for t in ts], [(t.x, t.shared) for t in ts]
    whole = Norm(entries, kind=kind, rank=2, world=4, peers=[0.1, 0.2, 9, 0.3, 9], max_norm=0.01, loss_scale=64.0)
    zs.zs3_grad_norm_tensors(entries, whole.args)
    sync()
    whole.check(values)
    parts = Norm(entries, kind=kind, rank=2, world=4, peers=[0, 0, 9, 0, 9], max_norm=0.01, loss_scale=64.0, finalize=False)
    zs.zs3_grad_norm_tensors(entries, parts.args)
    sync()
    assert parts.scale[1] == -7.5 and parts.flag[1] == -7 and parts.norm[0] == -7.5      # not touched
    parts.sums[0], parts.sums[1], parts.sums[3] = 0.1, 0.2, 0.3
    zs.zs3_norm_finalize(parts.args)
    sync()
    a, b = whole.got(), parts.got()
    assert a["norm"] == b["norm"] and a["scale"] == b["scale"] and b["flag"] == 0 and np.array_equal(a["sums"], b["sums"])
    open_ = Norm(entries, kind=kind, max_norm=math.inf)
    zs.zs3_grad_norm_tensors(entries, open_.args)
    sync()
    assert open_.got()["scale"] == 1.0
    assert torch.cuda.current_stream() is not None


@pytest.mark.parametrize("kind", ["2", "inf"])
@pytest.mark.parametrize("world", [64, 65, 300])
def test_norm_of_many_ranks(kind, world):
    """More peers than a wave has lanes; one whose sum is not finite."""
    require_gpu()
    note(f"{world} ranks, {kind}")
    rng = np.random.default_rng(world)
    for sizes in ((500, 40), (30_000, 7, 9000)):
        ts = [Tensor(rng, n, "fp32", i, shared=i == 1) for i, n in enumerate(sizes)]
        peers = list(rng.random(world + 1) * 1e-3)
        for rank in (0, world - 1, 17):
            _norm(ts, kind=kind, rank=rank, world=world, peers=peers)
        assert _norm(ts, kind=kind, rank=1, world=world, peers=[math.inf if v == 20 else p for v, p in enumerate(peers)]).got()["flag"] == 1
        assert _norm(ts, kind=kind, rank=1, world=world, peers=[math.nan if v == 33 else p for v, p in enumerate(peers)]).got()["flag"] == 1


def test_norm_counts_a_tensor_twice_where_the_list_does():
    require_gpu()
    note("a tensor twice, and parts of one")
    rng = np.random.default_rng(9)
    for n in (700, 50_000):
        t = Tensor(rng, n, "bf16", 3)
        parts = [t.entry(), t.entry(), dict(numel=n // 2, grad=t.g.ptr(), dtype="bf16", shared=True)]
        nm = Norm(parts)
        zs.zs3_grad_norm_tensors(parts, nm.args)
        sync()
        nm.check([(t.x, False), (t.x, False), (t.x[:n // 2], True)])


def test_norm_agrees_with_the_flat_norm():
    """One flat gradient of a layout, by the layout's call and as a list."""
    import torch
    require_gpu()
    note("list against flat")
    ids, numels = list(range(6)), [5000, 33, 9000, 7, 1200, 64]
    h = zs.zs3_layout_create(2, 100, ids, numels)
    try:
        S = zs.zs3_layout_info(h)["shard_numel"]
        rng = np.random.default_rng(8)
        g = Buf16(S, 1, oracle.from_f32(rng.standard_normal(S).astype(np.float32), "bf16"))
        entries = []
        for d in ids:
            p, (lo, hi) = zs.zs3_layout_param(h, d), zs.zs3_layout_own_range(h, d, 1)
            entries.append(dict(numel=hi - lo, grad=g.ptr() + 2 * p["shard_offset"], dtype="bf16", shared=p["persistent"]))
        n = Norm(entries, rank=1, world=2, peers=[2.0, 0, 0])
        zs.zs3_grad_norm_tensors(entries, n.args)
        sums = torch.tensor([2.0, 0, 0], dtype=torch.float64, device="cuda")
        outs = torch.zeros(2, dtype=torch.float64, device="cuda")
        zs.zs3_grad_norm(h, 1, "bf16", g.ptr(), sums, True, 1.0, 1.0, outs.data_ptr(), outs.data_ptr() + 8, outs.data_ptr() + 12)
        sync()
        # two sums of the same S positive terms
        np.testing.assert_allclose(n.got()["sums"], sums.cpu().numpy(), rtol=2 * S * 2.0 ** -53)
        assert n.got()["scale"] == pytest.approx(float(outs.view(torch.float32)[2].cpu()), rel=2.0 ** -23)
    finally:
        zs.zs3_layout_destroy(h)


# ------------------------------------------------------------------ the clip

def _scalar(x, dtype):
    import torch
    return torch.full((1,), x, dtype=dtype, device="cuda")


def _clip(ts, scale=0.3, flag=0, use_flag=True):
    import torch
    zs.zs3_clip_tensors([t.entry() for t in ts], _scalar(scale, torch.float32), _scalar(flag, torch.int32) if use_flag else None)
    sync()
    for t in ts:
        out = t.out_dtype or t.dtype
        if flag == 0:
            _same((t.o or t.g).host(), og.clip(t.x, scale, out))
        if t.o is not None or flag != 0:
            _same(t.g.host(), t.bits)
        t.guards()


@pytest.mark.parametrize("out", [None, "fp16", "bf16", "fp32"])
@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
def test_clip_lists(dtype, out):
    require_gpu()
    note(f"clip {dtype} to {out}")
    rng = np.random.default_rng(10)
    for shift, out_shift in ((0, 0), (1, 0), (0, 1), (5, 3)):
        for k in range(0, len(SIZES), 5):
            _clip([Tensor(rng, n, dtype, shift, out=out, out_shift=out_shift + i) for i, n in enumerate(SIZES[k:k + 5])])
    _clip([Tensor(rng, n, dtype, 1, out=out) for n in (1_000_003, 3, 400_000)], use_flag=False)


@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
def test_clip_rounds_and_keeps_what_is_not_finite(dtype):
    """Overflow on the way to a narrower type, subnormal results, infinities, NaN, -0."""
    require_gpu()
    note(f"clip special values {dtype}")
    rng = np.random.default_rng(11)
    special = list(enumerate([np.inf, -np.inf, np.nan, 0.0, -0.0, 65504.0, -65504.0, 1e-7, 6e-8, 3e38, 1e-40, 65519.0, 65520.0]))
    for out in (None, "fp16", "bf16", "fp32"):
        for scale in (0.5, 1.0, 3.0, 1e-3, 0.0):
            t = Tensor(rng, 3000, dtype, 1, out=out, special=special)
            _clip([t], scale)


def test_clip_of_many_types_and_tensors():
    require_gpu()
    note("clip 400 mixed tensors")
    rng = np.random.default_rng(12)
    kinds = ("fp16", "bf16", "fp32")
    _clip([Tensor(rng, int(rng.integers(1, 4000)), kinds[i % 3], i % 5, out=(None, *kinds)[i // 3 % 4], out_shift=i % 3) for i in range(400)])


def test_clip_does_nothing_where_the_flag_is_set():
    require_gpu()
    note("clip flagged")
    rng = np.random.default_rng(13)
    a, b = Tensor(rng, 5000, "bf16"), Tensor(rng, 5000, "bf16", out="fp32")
    before = b.o.host()
    _clip([a, b], scale=float("nan"), flag=1)
    _same(b.o.host(), before)


def test_clip_by_one_in_place_keeps_every_bit():
    require_gpu()
    note("clip by one")
    rng = np.random.default_rng(14)
    ts = [Tensor(rng, 9000, d, special=[(3, np.nan), (8999, np.inf)]) for d in ("fp16", "bf16", "fp32")]
    _clip(ts, 1.0)
    for t in ts:
        _same(t.g.host(), t.bits)
    # an output that is the gradient itself is in place, too
    import torch
    t = Tensor(rng, 9000, "bf16")
    zs.zs3_clip_tensors([dict(t.entry(), out=t.g.ptr(), out_dtype="bf16")], _scalar(0.5, torch.float32))
    sync()
    _same(t.g.host(), og.clip(t.x, 0.5, "bf16"))


# ------------------------------------------------------------------ accumulation

def _accumulate(ts, factor, first, **norm):
    entries = [t.entry() for t in ts]
    n = Norm(entries, **norm) if norm else None
    zs.zs3_accumulate_tensors(entries, factor, first, norm=n.args if n else None)
    sync()
    for t in ts:
        t.acc = og.accumulate(t.acc, t.x, factor, first)
        _same(t.o.host(), t.acc)
        _same(t.g.host(), t.bits)
        t.guards()
    if n:
        n.check([(t.acc, t.shared) for t in ts])
    return n


@pytest.mark.parametrize("first", [False, True])
@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
def test_accumulate_lists(dtype, first):
    require_gpu()
    note(f"accumulate {dtype} first={first}")
    rng = np.random.default_rng(20)
    for shift, out_shift in ((0, 0), (1, 0), (0, 1), (5, 3)):
        for k in range(0, len(SIZES), 5):
            ts = [Tensor(rng, n, dtype, shift, out="acc", out_shift=out_shift + i, shared=i == 1) for i, n in enumerate(SIZES[k:k + 5])]
            _accumulate(ts, 1 / 3, first)
            _accumulate(ts, 0.25, False, kind="2", rank=0, world=2, peers=[0, 0.5, 0])
            _accumulate(ts, -1.0, first, kind="inf")


def test_accumulate_many_and_large():
    require_gpu()
    note("accumulate 400 tensors, and large ones")
    rng = np.random.default_rng(21)
    kinds = ("fp16", "bf16", "fp32")
    ts = [Tensor(rng, int(rng.integers(1, 4000)), kinds[i % 3], i % 5, out="acc", out_shift=i % 3, shared=i % 2 == 0) for i in range(400)]
    _accumulate(ts, 0.5, False, kind="2")
    _accumulate(ts, 0.5, False)
    ts = [Tensor(rng, n, "bf16", i, out="acc", out_shift=i) for i, n in enumerate((8_000_001, 5, 1_000_000, 33))]
    _accumulate(ts, 1.0, True, kind="2")
    _accumulate(ts, 1.0, False, kind="inf")


def test_first_micro_batch_clears_and_values_that_are_not_finite_reach_the_flag():
    require_gpu()
    note("accumulate nan")
    rng = np.random.default_rng(22)
    t = Tensor(rng, 5000, "fp16", out="acc", special=[(4999, np.inf)])
    assert _accumulate([t], 1.0, False, kind="2").got()["flag"] == 1
    assert not np.isfinite(t.acc[4999])
    t.bits = _bits(rng.standard_normal(5000), "fp16")
    t.x = og.widened(t.bits, "fp16")
    import torch
    t.g.view.copy_(torch.from_numpy(t.bits.view(np.int16)).cuda())
    assert _accumulate([t], 1.0, True, kind="2").got()["flag"] == 0


# ------------------------------------------------------------------ together

def test_micro_batches_to_adamw():
    """Four micro-batches accumulated, the norm of the sum with the last, the same norm by
    itself, the sum clipped to bf16, and AdamW on the sum with the scale."""
    import torch
    from oracle import lowbit as lb
    require_gpu()
    note("accumulate, norm, clip, AdamW")
    rng = np.random.default_rng(30)
    sizes = [4099, 1, 2048, 777]
    acc = [Buf32(n, 1) for n in sizes]
    want = [np.full(n, np.nan, np.float32) for n in sizes]
    out = [Buf16(n, 1) for n in sizes]
    norms = None
    for k in range(4):
        x = [_bits(rng.standard_normal(n), "bf16") for n in sizes]
        gs = [Buf16(n, 1, b) for n, b in zip(sizes, x)]
        entries = [dict(numel=n, grad=g.ptr(), dtype="bf16", out=a.ptr(), out_dtype="fp32", shared=i == 1)
                   for i, (n, g, a) in enumerate(zip(sizes, gs, acc))]
        norms = Norm(entries, max_norm=1.0) if k == 3 else None
        zs.zs3_accumulate_tensors(entries, 0.25, first=k == 0, norm=norms.args if norms else None)
        want = [og.accumulate(w, og.widened(b, "bf16"), 0.25, k == 0) for w, b in zip(want, x)]
        sync()
    norms.check([(w, i == 1) for i, w in enumerate(want)])
    held = [dict(numel=n, grad=a.ptr(), dtype="fp32", out=o.ptr(), out_dtype="bf16", shared=i == 1)
            for i, (n, a, o) in enumerate(zip(sizes, acc, out))]
    alone = Norm(held)
    zs.zs3_grad_norm_tensors(held, alone.args)
    zs.zs3_clip_tensors(held, alone.scale[1:2], alone.flag[1:2])
    sync()
    alone.check([(w, i == 1) for i, w in enumerate(want)])
    scale = alone.got()["scale"]
    assert scale == norms.got()["scale"] < 1.0
    for w, a, o in zip(want, acc, out):
        _same(a.host(), w)
        _same(o.host(), og.clip(w, scale, "bf16"))
        a.check_guards(), o.check_guards()
    masters = [rng.standard_normal(n).astype(np.float32) for n in sizes]
    ws, ms, vs = ([Buf32(n, 0, f) for n, f in zip(sizes, fill)] for fill in (masters, *([[np.zeros(n, np.float32) for n in sizes]] * 2)))
    zs.zs3_adamw_tensors("bf16", "fp32", 32, [dict(numel=n, id=i, master=w.ptr(), grad=a.ptr(), exp_avg=m.ptr(), exp_avg_sq=v.ptr())
                                              for i, (n, w, a, m, v) in enumerate(zip(sizes, ws, acc, ms, vs))],
                         norms.scale[1:2], norms.flag[1:2], dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, step=1))
    sync()
    for n, w0, g, w in zip(sizes, masters, want, ws):
        z = np.zeros(n, np.float32)
        ref = lb.adamw(w0, z, z, g, scale=scale, lr=1e-3, wd=0.0, beta1=0.9, beta2=0.999, eps=1e-8, step=1)[0]
        _same(w.host(), ref)
    assert torch.isfinite(norms.norm).all()


def test_same_bits_again_and_in_a_workspace_of_other_lists():
    """One workspace serves lists of other sizes, kinds and calls in turn."""
    import torch
    require_gpu()
    note("determinism")
    rng = np.random.default_rng(31)
    lists = [[Tensor(rng, n, "bf16", i, out="acc", shared=i == 1) for i, n in enumerate(sizes)]
             for sizes in ((2_000_001, 300, 40_000), (5,), (7_000_000, 1, 900), [700] * 260, (33_000_000,))]
    entries = [[t.entry() for t in ts] for ts in lists]
    ws = torch.zeros(max(zs.zs3_norm_workspace_bytes(e) for e in entries), dtype=torch.uint8, device="cuda")
    seen = [set() for _ in lists]
    for k in range(3):
        for i, (ts, e) in enumerate(zip(lists, entries)):
            for kind in ("2", "inf"):
                n = Norm(e, kind=kind)
                n.args.workspace, n.args.workspace_bytes = ws.data_ptr(), ws.numel()
                zs.zs3_grad_norm_tensors(e, n.args)
                sync()
                if k == 0:
                    n.check([(t.x, t.shared) for t in ts])
                seen[i].add((kind, n.got()["norm"], n.got()["scale"], n.got()["each"].tobytes(), n.got()["sums"].tobytes()))
            zs.zs3_accumulate_tensors(e, 1.0, True, norm=Norm(e).args if k else n.args)
    sync()
    assert all(len(s) == 2 for s in seen)


def test_every_call_sees_its_own_partial_results():
    """Calls in a row on one workspace, the gradients a power of two larger each time:
    norm, sums and single norms are the first call's times that, bit for bit, so no partial result of an earlier call is read."""
    import torch
    require_gpu()
    note("200 calls in a row")
    rng = np.random.default_rng(34)
    ts = [Tensor(rng, n, "fp32", i, shared=i == 1) for i, n in enumerate((3_000_001, 300, 40_000, 250_000))]
    entries = zs.zs3_grad_tensor_list([t.entry() for t in ts])
    n = Norm([t.entry() for t in ts], max_norm=math.inf)
    got = []
    for k in range(200):
        zs.zs3_grad_norm_tensors(entries, n.args)
        got.append([x.clone() for x in (n.norm, n.sums, n.each)])
        for t in ts:
            t.g.view.mul_(2.0 if k % 20 < 10 else 0.5)
    torch.cuda.synchronize()
    for k, (norm, sums, each) in enumerate(got):
        f = 2.0 ** (k % 20 if k % 20 <= 10 else 20 - k % 20)
        assert torch.equal(norm, got[0][0] * f) and torch.equal(each, got[0][2] * f), k
        assert torch.equal(sums, got[0][1] * f * f), k


@pytest.mark.parametrize("sizes", [(200_001, 300, 4000), (700,) * 330, (9, 5)], ids=["few", "many", "tiny"])
def test_captured_and_replayed(sizes):
    """Accumulation with the norm, the clip and the per-tensor norms in one graph, replayed on new values between eager calls."""
    import torch
    require_gpu()
    note(f"graph of {len(sizes)} tensors")
    rng = np.random.default_rng(32)
    ts = [Tensor(rng, n, "bf16", i % 9, out="acc", shared=i == 2) for i, n in enumerate(sizes)]
    entries = [t.entry() for t in ts]
    outs = [Buf16(t.n, 1) for t in ts]
    held = zs.zs3_grad_tensor_list([dict(numel=t.n, grad=t.o.ptr(), dtype="fp32", out=o.ptr(), out_dtype="bf16") for t, o in zip(ts, outs)])
    arr = zs.zs3_grad_tensor_list(entries)
    n = Norm(entries)
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        zs.zs3_accumulate_tensors(arr, 0.5, first=False, norm=n.args)
        zs.zs3_clip_tensors(held, n.scale[1:2], n.flag[1:2])
    for k in range(4):
        for t in ts:
            t.bits = _bits(rng.standard_normal(t.n) * (k + 1), "bf16")
            t.x = og.widened(t.bits, "bf16")
            t.g.view.copy_(torch.from_numpy(t.bits.view(np.int16)).cuda())
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for t, o in zip(ts, outs):
            t.acc = og.accumulate(t.acc, t.x, 0.5, False)
            _same(t.o.host(), t.acc)
            _same(o.host(), og.clip(t.acc, n.got()["scale"], "bf16"))
        n.check([(t.acc, t.shared) for t in ts])
        eager = Norm(entries)            # eager work between the replays
        zs.zs3_grad_norm_tensors(entries, eager.args)
        torch.cuda.synchronize()
        eager.check([(t.x, t.shared) for t in ts])


def test_two_streams_at_once():
    import torch
    require_gpu()
    note("two streams")
    rng = np.random.default_rng(33)
    sets = [[Tensor(rng, n, d, out="acc") for n in (900_000, 33, 70_000)] for d in ("bf16", "fp16")]
    streams = [torch.cuda.Stream() for _ in sets]
    norms, alone = ([Norm([t.entry() for t in ts]) for ts in sets] for _ in range(2))
    torch.cuda.synchronize()
    for _ in range(10):
        for ts, n, s in zip(sets, norms, streams):
            zs.zs3_accumulate_tensors([t.entry() for t in ts], 0.5, False, norm=n.args, stream=s)
            for t in ts:
                t.acc = og.accumulate(t.acc, t.x, 0.5, False)
        # and the lists' own norms, on the other stream each: workspaces of their own
        for ts, n, s in zip(sets, alone, reversed(streams)):
            zs.zs3_grad_norm_tensors([t.entry() for t in ts], n.args, stream=s)
    torch.cuda.synchronize()
    for ts, n in zip(sets, alone):
        n.check([(t.x, t.shared) for t in ts])
    for ts, n in zip(sets, norms):
        n.check([(t.acc, t.shared) for t in ts])
        for t in ts:
            _same(t.o.host(), t.acc)


def test_a_tensor_past_32_bits():
    """2^31 + 4099 elements: norm, clip in place and accumulation reach both ends and nothing else."""
    import torch
    require_gpu()
    note("2^31 + 4099 elements")
    n = (1 << 31) + 4099
    base = torch.zeros(n + 256, dtype=torch.bfloat16, device="cuda")
    g = base[129:129 + n]
    at = [0, 1, 4095, 1 << 30, (1 << 31) - 1, 1 << 31, (1 << 31) + 1, n - 1]
    for i, k in enumerate(at):
        g[k] = float(i + 1)
    base[128], base[129 + n] = 64.0, 64.0                      # neighbours that no call may touch or count
    entry = dict(numel=n, grad=g.data_ptr(), dtype="bf16")
    nm = Norm([entry], max_norm=1e9)
    zs.zs3_grad_norm_tensors([entry], nm.args)
    zs.zs3_clip_tensors([entry], _scalar(2.0, torch.float32))
    torch.cuda.synchronize()
    assert nm.got()["norm"] == math.sqrt(sum((i + 1) ** 2 for i in range(len(at)))) == nm.got()["each"][0]
    assert [float(g[k]) for k in at] == [2.0 * (i + 1) for i in range(len(at))]
    assert float(base[128]) == 64.0 and float(base[129 + n]) == 64.0
    acc = torch.full((n + 2,), -3.0, device="cuda")
    entry.update(out=acc[1:1 + n].data_ptr(), out_dtype="fp32")
    nm = Norm([entry], max_norm=1e9)
    zs.zs3_accumulate_tensors([entry], 0.5, first=True, norm=nm.args)
    torch.cuda.synchronize()
    assert [float(acc[1 + k]) for k in at] == [i + 1.0 for i in range(len(at))]
    assert float(acc[0]) == -3.0 and float(acc[n + 1]) == -3.0
    assert int(torch.count_nonzero(acc[1:1 + n])) == len(at)
    assert nm.got()["norm"] == math.sqrt(sum((i + 1) ** 2 for i in range(len(at))))


def test_lists_made_of_tensors():
    """Device tensors, their bits and pinned host memory; ordinary host memory is refused before a launch."""
    import torch
    require_gpu()
    note("lists of tensors")
    rng = np.random.default_rng(40)
    x = rng.standard_normal(5000).astype(np.float32)
    g = torch.from_numpy(x).cuda().bfloat16()
    held = og.widened(g.view(torch.int16).cpu().numpy().view(np.uint16), "bf16")
    scale, flag = _scalar(0.5, torch.float32), _scalar(0, torch.int32)
    for grad in (g, g.view(torch.int16)):
        for acc in (torch.zeros(5000, device="cuda"), torch.zeros(5000, pin_memory=True)):
            arr = zs.zs3_grad_tensor_list([dict(numel=5000, grad=grad, dtype="bf16", out=acc, out_dtype="fp32")] * 1)
            n = Norm(arr, max_norm=math.inf, per_tensor=False)
            zs.zs3_accumulate_tensors(arr, 0.5, first=True, norm=n.args)
            torch.cuda.synchronize()
            want = og.accumulate(held, held, 0.5, True)
            _same(acc.cpu().numpy(), want)
            n.check([(want, False)])
            zs.zs3_clip_tensors([dict(numel=5000, grad=acc, dtype="fp32")], scale, flag)
            torch.cuda.synchronize()
            _same(acc.cpu().numpy(), og.clip(want, 0.5, "fp32"))
    for call in (lambda: zs.zs3_accumulate_tensors([dict(numel=9, grad=g, dtype="bf16", out=torch.zeros(9), out_dtype="fp32")]),
                 lambda: zs.zs3_clip_tensors([dict(numel=9, grad=g.cpu(), dtype="bf16")], scale, flag),
                 lambda: zs.zs3_clip_tensors([dict(numel=9, grad=g, dtype="bf16")], scale.cpu(), flag),
                 lambda: zs.zs3_grad_norm_tensors([dict(numel=9, grad=g, dtype="bf16")], zs.zs3_norm_args_of(sums=torch.zeros(2, dtype=torch.float64)))):
        with pytest.raises(ValueError, match="host memory"):
            call()
