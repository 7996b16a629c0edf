"""GPU: AdamW over a list of tensors (32- and 8-bit states) and the moments'
read against the oracle (``oracle.lowbit``).

Moments: bit for bit (every operation on them is one IEEE fp32 operation, and
rounding to 8 bits is decided by integers).  32-bit states: master and the
16-bit copy bit for bit too.  8-bit states: the master's update is formed
within a few ulps of fp32, bounded in ``_check8``."""

import numpy as np
import pytest

import oracle
import zero_sharded_state_amd as zs
from gpu_util import Buf16, Buf32, note, require_gpu, sync
from oracle import lowbit as lb

pytestmark = pytest.mark.gpu
HP = {"lr": 1e-3, "beta1": 0.9, "beta2": 0.99, "eps": 1e-8, "step": 3}
GUARD8 = 64


class Buf8:
    """Bytes between canaries, 16-byte aligned."""

    def __init__(self, data):
        import torch
        self.n = len(data)
        self.base = torch.full((self.n + 2 * GUARD8,), 0xA5, dtype=torch.uint8, device="cuda")
        self.view = self.base[GUARD8:GUARD8 + self.n]
        self.view.copy_(torch.from_numpy(np.ascontiguousarray(data, np.uint8)).cuda())

    def ptr(self):
        return self.view.data_ptr()

    def host(self):
        return self.view.cpu().numpy().copy()

    def check_guards(self):
        b = self.base.cpu().numpy()
        assert np.all(b[:GUARD8] == 0xA5) and np.all(b[GUARD8 + self.n:] == 0xA5), "write outside the moment"


class Case:
    """One tensor: its arrays on the host, its buffers on the device."""

    def __init__(self, rng, n, ident, dtype, grad, bits, shift=0, wd=0.0, lr_scale=1.0, param=True, spread=1.0):
        self.n, self.id, self.dtype, self.grad, self.bits, self.wd, self.lr_scale = n, ident, dtype, grad, bits, wd, lr_scale
        self.w = (rng.standard_normal(n) * 0.02).astype(np.float32)
        g = (rng.standard_normal(n) * 1e-3 * np.exp(rng.uniform(-spread, spread, n))).astype(np.float32)
        self.g_bits = None if grad == "fp32" else oracle.from_f32(g, grad)
        self.g = g if grad == "fp32" else oracle.to_f32(self.g_bits, grad)
        m = (rng.standard_normal(n) * 3e-4).astype(np.float32)
        v = (rng.standard_normal(n) ** 2 * 1e-6 * np.exp(rng.uniform(-spread, spread, n))).astype(np.float32)
        self.dw = Buf32(n, shift, self.w)
        self.dg = Buf32(n, shift, g) if grad == "fp32" else Buf16(n, shift, self.g_bits)
        self.dp = Buf16(n, shift) if param else None
        if bits == 32:
            self.m, self.v = m, v
            self.dm, self.dv = Buf32(n, shift, m), Buf32(n, shift, v)
        else:
            half = np.full(n, 0x8000_8000, np.uint32)
            mc, vc = lb.encode_moment(m, half, False), lb.encode_moment(v, half, True)
            self.m, self.v = lb.decode_moment(*mc, False), lb.decode_moment(*vc, True)
            self.dm, self.dv = Buf8(lb.moment_buffer(*mc, fill=0xFF)), Buf8(lb.moment_buffer(*vc, fill=0xFF))

    def entry(self):
        return dict(numel=self.n, id=self.id, master=self.dw.ptr(), grad=self.dg.ptr(), param=self.dp.ptr() if self.dp else None,
                    exp_avg=self.dm.ptr(), exp_avg_sq=self.dv.ptr(), lr_scale=self.lr_scale, weight_decay=self.wd)

    def expect(self, scale, hp, seed):
        return lb.adamw(self.w, self.m, self.v, self.g, scale=scale, lr=hp["lr"] * self.lr_scale, wd=self.wd, beta1=hp["beta1"],
                        beta2=hp["beta2"], eps=hp["eps"], step=hp["step"])

    def check(self, scale=1.0, hp=HP, seed=0):
        w, m, v, decayed, upd = self.expect(scale, hp, seed)
        got = self.dw.host()
        if self.bits == 32:
            assert np.array_equal(got.view(np.uint32), w.view(np.uint32)), "master"
            assert np.array_equal(self.dm.host().view(np.uint32), m.view(np.uint32)), "exp_avg"
            assert np.array_equal(self.dv.host().view(np.uint32), v.view(np.uint32)), "exp_avg_sq"
        else:
            # given m, v and the decayed weight in fp32, the update lr/bc1 * m *
            # rcp(sqrt(v) * rsqrt_bc2 + eps) takes, in units of 2^-24 of itself:
            # the two constants 1 + 1, eps 1, root 2 (one ulp), its product 1, the
            # sum 1, the reciprocal 2, the products 1 + 1: 11; the last subtraction
            # rounds to half an ulp of the result, at most 2^-24 of it
            exact = decayed.astype(np.float64) - upd
            bound = 2.0 ** -24 * (11 * 1.001 * np.abs(upd) + 1.001 * np.abs(exact)) + 2.0 ** -149
            err = np.abs(got.astype(np.float64) - exact)
            assert np.all(err <= bound), (float((err / bound).max()), int((err / bound).argmax()))
            word = lb.words(lb.keys(seed, hp["step"], self.id), np.arange(self.n))
            for buf, x, second in ((self.dm, m, False), (self.dv, v, True)):
                code, s = lb.split_moment(buf.host(), self.n)
                rc, rs = lb.encode_moment(x, word, second)
                assert np.array_equal(s, rs), ("scales", second)
                assert np.array_equal(code, rc), ("codes", second, int((code != rc).sum()))
                tail = buf.host()[self.n:-(-self.n // 32) * 32]
                assert np.all(tail == 0xFF), "codes past the end were written"
                buf.check_guards()
        if self.dp is not None:
            assert np.array_equal(self.dp.host(), oracle.from_f32(got, self.dtype)), "param"
        for b in (self.dw, self.dg, self.dp, self.dm, self.dv):
            if b is not None:
                b.check_guards()

    def unchanged(self):
        assert np.array_equal(self.dw.host().view(np.uint32), self.w.view(np.uint32))


def _scale(x):
    import torch
    return torch.full((1,), x, dtype=torch.float32, device="cuda")


def _step(cases, bits, scale=None, flag=None, hp=HP, seed=0, stream=None):
    zs.zs3_adamw_tensors(cases[0].dtype, cases[0].grad, bits, [c.entry() for c in cases], scale, flag, hp, seed, stream=stream)


SIZES = [1, 2, 3, 4, 5, 31, 32, 33, 63, 255, 256, 257, 511, 512, 513, 2047, 2048, 2049, 4095, 10007]


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("grad", ["fp16", "bf16", "fp32"])
def test_sizes_and_types(bits, dtype, grad):
    require_gpu()
    note(f"adamw{bits} {dtype} grad {grad}, sizes {SIZES}")
    rng = np.random.default_rng(1)
    cases = [Case(rng, n, i, dtype, grad, bits, wd=0.1 * (i % 3), lr_scale=1 / (1 + i % 2)) for i, n in enumerate(SIZES)]
    _step(cases, bits, _scale(0.37), seed=9)
    sync()
    for c in cases:
        c.check(float(np.float32(0.37)), seed=9)


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("shift", [1, 2, 3, 5, 7])
def test_views_at_any_offset(bits, shift):
    """Gradients and parameters at 2-byte, masters at 4-byte aligned addresses."""
    require_gpu()
    note(f"adamw{bits} shift {shift}")
    rng = np.random.default_rng(shift)
    cases = [Case(rng, n, i, "bf16", "bf16", bits, shift=shift, param=i != 1) for i, n in enumerate((513, 1500, 4099))]
    _step(cases, bits)
    sync()
    for c in cases:
        c.check()


@pytest.mark.parametrize("bits", [8, 32])
def test_long_lists_split_and_reordered_calls_agree(bits):
    """130 tensors (more than a launch's 48), some empty, in one call; the same
    in reverse order over three calls gives the same bits."""
    require_gpu()
    note(f"adamw{bits} 130 tensors")
    out = []
    for k in range(2):
        rng = np.random.default_rng(5)
        cases = [Case(rng, int(rng.integers(1, 3000)), 1000 + i, "fp16", "fp16", bits, wd=0.01 * (i % 2)) for i in range(130)]
        empty = dict(numel=0, id=0, master=0, grad=0, exp_avg=0, exp_avg_sq=0)
        if k == 0:
            zs.zs3_adamw_tensors("fp16", "fp16", bits, [empty] + [c.entry() for c in cases] + [empty], None, None, HP, 4)
        else:
            e = [c.entry() for c in cases][::-1]
            for part in (e[:1], e[1:60], e[60:]):
                zs.zs3_adamw_tensors("fp16", "fp16", bits, part, None, None, HP, 4)
        sync()
        if k == 0:
            for c in cases:
                c.check(seed=4)
        out.append([(c.dw.host().view(np.uint32), c.dm.host(), c.dv.host(), c.dp.host()) for c in cases])
    for a, b in zip(*out):
        assert all(np.array_equal(x.view(np.uint8), y.view(np.uint8)) for x, y in zip(a, b))


def test_wide_ranges_in_a_block():
    """Second moments over 30 binades inside blocks: subnormal codes, and none
    that is not zero becomes zero."""
    require_gpu()
    note("adamw8 wide ranges")
    rng = np.random.default_rng(8)
    cases = [Case(rng, 4096, 0, "bf16", "fp32", 8, spread=s) for s in (5.0,)] + [Case(rng, 999, 1, "bf16", "fp32", 8, spread=10.0)]
    _step(cases, 8, seed=2)
    sync()
    for c in cases:
        c.check(seed=2)


def test_zero_gradients_and_fresh_moments():
    """All bytes 0 is the start; a zero gradient leaves zero moments zero and the
    weight to its decay alone."""
    require_gpu()
    note("adamw8 fresh moments")
    rng = np.random.default_rng(9)
    c = Case(rng, 1000, 0, "bf16", "fp32", 8, wd=0.1)
    c.dm.view.zero_()
    c.dv.view.zero_()
    c.m[:] = 0
    c.v[:] = 0
    c.dg.view[500:].zero_()
    c.g = c.g.copy()
    c.g[500:] = 0
    _step([c], 8, hp=dict(HP, step=1))
    sync()
    w, m, v, decayed, upd = c.expect(1.0, dict(HP, step=1), 0)
    code, s = lb.split_moment(c.dv.host(), c.n)
    got = lb.decode_moment(code, s, True)
    assert np.all(got[512:] == 0) and np.all(lb.decode_moment(*lb.split_moment(c.dm.host(), c.n), False)[512:] == 0)
    assert np.array_equal(c.dw.host()[512:], decayed[512:])
    assert np.all(got[:500] > 0)
    assert np.all(np.abs(c.dw.host()[:500] - decayed[:500]) <= 1.001e-3)         # |update| <= lr at step 1


def test_tiny_gradients():
    """Gradients whose squares leave fp32's normal range, at the smallest eps: the
    update is m / (sqrt(v) + eps) of the fp32 moments, where a root that counts
    as 0 is at most 1.1e-19 of 1e-12: 2 of the 11 half-ulps more.  Codes under
    2^-126 are not pinned; the moments read back finite."""
    require_gpu()
    import torch
    note("adamw8 tiny gradients")
    rng = np.random.default_rng(14)
    c = Case(rng, 2048, 0, "bf16", "fp32", 8)
    g = (rng.standard_normal(2048) * 10.0 ** rng.uniform(-24, -10, 2048)).astype(np.float32)
    c.g = g
    c.dg.view.copy_(torch.from_numpy(g))
    c.dm.view.zero_()
    c.dv.view.zero_()
    c.m[:] = 0
    c.v[:] = 0
    hp = dict(HP, eps=1e-12, step=1)
    _step([c], 8, hp=hp)
    sync()
    _, m, v, decayed, upd = c.expect(1.0, hp, 0)
    exact = decayed.astype(np.float64) - upd
    bound = 2.0 ** -24 * (13 * 1.001 * np.abs(upd) + 1.001 * np.abs(exact)) + 2.0 ** -149
    assert np.all(np.abs(c.dw.host().astype(np.float64) - exact) <= bound)
    for buf, second in ((c.dm, False), (c.dv, True)):
        assert np.isfinite(lb.decode_moment(*lb.split_moment(buf.host(), c.n), second)).all()


@pytest.mark.parametrize("bits", [8, 32])
def test_nonfinite_flag_writes_nothing(bits):
    require_gpu()
    import torch
    note(f"adamw{bits} flag")
    rng = np.random.default_rng(3)
    cases = [Case(rng, n, i, "bf16", "bf16", bits) for i, n in enumerate((100, 3000))]
    before = [(c.dm.host(), c.dv.host()) for c in cases]
    _step(cases, bits, flag=torch.ones(1, dtype=torch.int32, device="cuda"))
    sync()
    for c, (m, v) in zip(cases, before):
        c.unchanged()
        assert np.array_equal(c.dm.host(), m) and np.array_equal(c.dv.host(), v)
        assert np.all(c.dp.host() == 0x5A5A)
    _step(cases, bits, flag=torch.zeros(1, dtype=torch.int32, device="cuda"))
    sync()
    for c in cases:
        c.check()


def test_nonfinite_gradients_mark_their_block_only():
    """Without a flag, a NaN and an infinity reach their own element's weight and
    their block's moments, and nothing else."""
    require_gpu()
    note("adamw8 non-finite gradients")
    rng = np.random.default_rng(4)
    c = Case(rng, 1024, 0, "bf16", "fp32", 8)
    c.dg.view[70] = float("nan")
    c.dg.view[300] = float("inf")
    _step([c], 8)
    sync()
    w = c.dw.host()
    assert np.isnan(w[70]) and not np.isfinite(w[300])
    assert np.isfinite(np.delete(w, [70, 300])).all()
    for buf, second in ((c.dm, False), (c.dv, True)):
        x = lb.decode_moment(*lb.split_moment(buf.host(), c.n), second).reshape(-1, 32)
        bad = ~np.isfinite(x).any(1)
        assert list(np.nonzero(bad)[0]) == [2, 9] and np.isfinite(np.delete(x, [2, 9], 0)).all()


def test_32_bit_states_give_the_flat_adams_bits():
    """The same parameters stepped by zs3_adam_step on the flat shard."""
    require_gpu()
    import torch
    note("adamw32 against the flat step")
    rng = np.random.default_rng(6)
    ids, sizes, world, rank = [3, 1, 8], [5000, 77, 12345], 3, 1
    h = zs.zs3_layout_create(world, 100, ids, sizes)
    try:
        n = zs.zs3_layout_info(h)["shard_numel"]
        mk = lambda s: torch.from_numpy((rng.standard_normal(n) * s).astype(np.float32)).cuda()     # noqa: E731
        w, m, v, g = mk(0.02), mk(1e-4), mk(1e-3).square(), mk(1e-3).bfloat16()
        a = [w, m, v, torch.zeros(n, dtype=torch.bfloat16, device="cuda")]
        b = [x.clone() for x in a]
        scale = _scale(0.7)
        hp = dict(HP, weight_decay=0.05, step=11)
        zs.zs3_adam_step(h, rank, "bf16", 0, n, a[0], a[1], a[2], g, a[3], scale, None, hp)
        tensors = []
        for d in ids:
            p = zs.zs3_layout_param(h, d)
            lo, hi = zs.zs3_layout_own_range(h, d, rank)
            o, k = p["shard_offset"], hi - lo
            tensors.append(dict(numel=k, id=d, master=b[0][o:], grad=g[o:], param=b[3][o:], exp_avg=b[1][o:], exp_avg_sq=b[2][o:],
                                weight_decay=0.05))
        zs.zs3_adamw_tensors("bf16", "bf16", 32, tensors, scale, None, hp)
        sync()
        for x, y in zip(a, b):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    finally:
        zs.zs3_layout_destroy(h)


@pytest.mark.parametrize("n", [1, 3, 4, 33, 256, 1000, 4097, 70001])
@pytest.mark.parametrize("shift", [0, 1, 3])
@pytest.mark.parametrize("out", ["bf16", "fp32"])
def test_moment_read(n, shift, out):
    """Every code under many scales, at any offset of the output."""
    require_gpu()
    note(f"moment read {n} {shift} {out}")
    rng = np.random.default_rng(n)
    reads, checks = [], []
    for second in (False, True):
        code = rng.integers(0, 256, n).astype(np.uint8)
        scale = rng.integers(90, 170, -(-n // 32)).astype(np.uint8)
        buf = Buf8(lb.moment_buffer(code, scale, fill=0xFF))
        dst = Buf32(n, shift) if out == "fp32" else Buf16(n, shift)
        reads.append(dict(numel=n, kind=zs.ZS3_EXP_AVG_SQ if second else zs.ZS3_EXP_AVG, moment=buf.ptr(), out=dst.ptr()))
        checks.append((buf, dst, lb.decode_moment(code, scale, second)))
    zs.zs3_moment8_read(out, reads)
    sync()
    for buf, dst, ref in checks:
        got = dst.host() if out == "fp32" else oracle.to_f32(dst.host(), "bf16")
        assert np.array_equal(got, ref, equal_nan=True)
        dst.check_guards()


def test_moment_read_of_a_long_list():
    require_gpu()
    note("moment read of 150")
    rng = np.random.default_rng(2)
    reads, checks = [], []
    for i in range(150):
        n = int(rng.integers(1, 500))
        code, scale = rng.integers(0, 127, n).astype(np.uint8), rng.integers(100, 150, -(-n // 32)).astype(np.uint8)
        buf, dst = Buf8(lb.moment_buffer(code, scale)), Buf32(n)
        reads.append(dict(numel=n, kind=1 + i % 2, moment=buf.ptr(), out=dst.ptr()))
        checks.append((buf, dst, lb.decode_moment(code, scale, i % 2 == 1)))
    zs.zs3_moment8_read("fp32", reads)
    sync()
    for _, dst, ref in checks:
        assert np.array_equal(dst.host(), ref)
        dst.check_guards()


@pytest.mark.parametrize("bits", [8, 32])
def test_captured_and_replayed(bits):
    """Captured on the first call that is ever made with these buffers; each
    replay, with eager work and synchronisation between, is one more step."""
    require_gpu()
    import torch
    note(f"adamw{bits} captured")
    rng = np.random.default_rng(12)
    cases = [Case(rng, n, i, "bf16", "bf16", bits, wd=0.1) for i, n in enumerate([700] * 60)]
    tensors = zs.zs3_adamw_tensor_list([c.entry() for c in cases])
    start = [(c.dw.base.clone(), c.dm.base.clone(), c.dv.base.clone()) for c in cases]
    eager = []
    for _ in range(3):
        zs.zs3_adamw_tensors("bf16", "bf16", bits, tensors, None, None, HP, 5)
        sync()
        eager.append([(c.dw.host(), c.dm.host(), c.dv.host(), c.dp.host()) for c in cases])
    for c, (w, m, v) in zip(cases, start):
        c.dw.base.copy_(w)
        c.dm.base.copy_(m)
        c.dv.base.copy_(v)
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        zs.zs3_adamw_tensors("bf16", "bf16", bits, tensors, None, None, HP, 5, stream=torch.cuda.current_stream())
    for k in range(3):
        graph.replay()
        sync()
        other = torch.randn(1 << 20, device="cuda").sum().item()
        assert other == other
        for c, ref in zip(cases, eager[k]):
            for x, y in zip((c.dw.host(), c.dm.host(), c.dv.host(), c.dp.host()), ref):
                assert np.array_equal(x.view(np.uint8), y.view(np.uint8))


@pytest.mark.parametrize("bits", [8, 32])
def test_two_streams_at_once(bits):
    """Two lists on two streams, launched in turn, give the bits of one after the other."""
    require_gpu()
    import torch
    note(f"adamw{bits} two streams")
    rng = np.random.default_rng(13)
    groups = [[Case(rng, 200_003, 10 * k + i, "bf16", "fp32", bits) for i in range(2)] for k in range(2)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    sync()
    for c, s in zip(groups, streams):
        _step(c, bits, seed=3, stream=s)
    sync()
    for group in groups:
        for c in group:
            c.check(seed=3)


def test_a_tensor_past_32_bit_offsets():
    """2^32 + 70,001 elements, 8-bit states: elements on both sides of 2^32 and
    the last ones against the oracle."""
    require_gpu()
    import torch
    note("adamw8 2^32 + 70001 elements")
    n = (1 << 32) + 70001
    w = torch.full((n,), 0.02, dtype=torch.float32, device="cuda")
    p = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    m = torch.zeros(zs.zs3_moment8_bytes(n), dtype=torch.uint8, device="cuda")
    v = torch.zeros_like(m)
    spots = [0, (1 << 31) - 96, (1 << 32) - 96, (1 << 32), n - 96 - n % 32]
    rng = np.random.default_rng(1)
    grads = [oracle.from_f32((rng.standard_normal(96) * 1e-3).astype(np.float32), "bf16") for _ in spots]
    for s, x in zip(spots, grads):
        g[s:s + 96] = torch.from_numpy(x.view(np.int16)).cuda().view(torch.bfloat16)
    hp = dict(HP, step=1)
    zs.zs3_adamw_tensors("bf16", "bf16", 8, [dict(numel=n, id=2, master=w, grad=g, param=p, exp_avg=m, exp_avg_sq=v)], None, None, hp, 1)
    sync()
    nb = -(-n // 32)
    for s, x in zip(spots, grads):
        zero = np.zeros(96, np.float32)
        _, rm, rv, decayed, upd = lb.adamw(np.full(96, 0.02, np.float32), zero, zero, oracle.to_f32(x, "bf16"), scale=1.0, lr=hp["lr"], wd=0.0,
                                           beta1=hp["beta1"], beta2=hp["beta2"], eps=hp["eps"], step=1)
        word = lb.words(lb.keys(1, 1, 2), s + np.arange(96))
        for buf, ref, second in ((m, rm, False), (v, rv, True)):
            rc, rs = lb.encode_moment(ref, word, second)
            assert np.array_equal(buf[s:s + 96].cpu().numpy(), rc)
            assert np.array_equal(buf[32 * nb + s // 32:32 * nb + s // 32 + 3].cpu().numpy(), rs)
        assert np.abs(w[s:s + 96].cpu().numpy() - (decayed - upd)).max() <= 2.0 ** -24 * (11 * 1.1e-3 + 0.03)
    assert float(w[n - 1]) == np.float32(0.02) and float(w[12345]) == np.float32(0.02)
    out = torch.empty(n, dtype=torch.bfloat16, device="cuda")
    zs.zs3_moment8_read("bf16", [dict(numel=n, kind=1, moment=m, out=out)])
    sync()
    s = spots[3]
    code, sc = m[s:s + 96].cpu().numpy(), m[32 * nb + s // 32:32 * nb + s // 32 + 3].cpu().numpy()
    assert np.array_equal(out[s:s + 96].float().cpu().numpy(), lb.decode_moment(code, sc, False))


@pytest.mark.parametrize("beta2", [0.9, 0.99, 0.999, 0.9999])
@pytest.mark.parametrize("step", [1, 50])
@pytest.mark.parametrize("eps", [1e-12, 1e-8])
def test_updates_where_the_root_counts_as_zero(beta2, step, eps):
    """Weights of 0, so that the update itself is what is measured, and second
    moments on both sides of fp32's normal range.  Where one lies under it the
    root may count as 0: the denominator loses sqrt(v) / sqrt(1 - b2^t) of at
    least eps, at most 2^-63 / (eps * sqrt(1 - b2^t)) of the update, beside
    the 11 half-ulps that ``check`` counts and the half ulp of the result."""
    require_gpu()
    import torch
    note(f"adamw8 roots that count as 0, beta2 {beta2} step {step} eps {eps}")
    rng = np.random.default_rng(17)
    n = 4096
    c = Case(rng, n, 0, "bf16", "fp32", 8)
    c.w[:] = 0
    c.g = (rng.standard_normal(n) * 10.0 ** rng.uniform(-24, -15, n)).astype(np.float32)
    c.m[:] = 0
    c.v[:] = 0
    c.dw.view.zero_()
    c.dg.view.copy_(torch.from_numpy(c.g))
    c.dm.view.zero_()
    c.dv.view.zero_()
    hp = dict(HP, beta2=beta2, eps=eps, step=step)
    _step([c], 8, hp=hp)
    sync()
    _, m, v, decayed, upd = c.expect(1.0, hp, 0)
    assert np.all(decayed == 0) and 1000 < np.count_nonzero(v < 2.0 ** -126) < n - 500
    root = np.sqrt(v.astype(np.float64) / (1 - beta2 ** step))
    lost = np.where(v < 2.0 ** -126, root / eps, 0.0)
    assert lost.max() <= 2.0 ** -63 / (eps * np.sqrt(1 - beta2 ** step))
    err = np.abs(c.dw.host().astype(np.float64) + upd)
    bound = np.abs(upd) * (1.001 * 2.0 ** -24 * 12 * (1 + lost) + lost) + 2.0 ** -149
    assert np.all(err <= bound), float((err / bound).max())
