"""Whole shard steps over several micro-batches, as ``ShardStep(accumulate=K)`` runs them,
against a chain of the oracle's: every micro-batch's flat gradient, the accumulators, master,
moments and shard bit for bit, the norm within its sum's rounding; a step with an
infinite gradient in one micro-batch sets the flag and changes nothing, and the next one goes on."""

import gc
import math

import numpy as np
import pytest

import oracle
import zero_sharded_state_amd as zs
from gpu_util import note, require_gpu, sync
from oracle import grads as og
from oracle import lowbit as lb
from zero_sharded_state_amd.shard_step import AdamConfig, ShardStep

pytestmark = pytest.mark.gpu
IDS, SIZES = [4, 9, 1, 30, 12, 7], [4097, 64, 5000, 33, 8191, 130]


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()
    yield
    import torch
    gc.collect()
    torch.cuda.empty_cache()


def _h16(t):
    return t.cpu().numpy().view(np.uint16).copy()


def _make(world, rank, dtype, **k):
    return ShardStep(world_size=world, rank=rank, threshold=100, ds_ids=IDS, numels=SIZES, dtype=dtype, prefetch_bucket_size=9000,
                     reduce_bucket_size=7000, sub_group_size=3000, adam=AdamConfig(lr=1e-3, beta2=0.99, weight_decay=0.1),
                     rs_streams=2, gather_streams=2, **k)


def _start(step, rng):
    import torch
    full = {}
    for p in step.params:
        d, n = p["ds_id"], p["numel"]
        full[d] = oracle.from_f32((rng.standard_normal(n) * 0.02).astype(np.float32), step.dtype)
        t = torch.from_numpy(full[d].view(np.int16)).cuda()
        if p["persistent"]:
            step.pers_full[step.pers_off[d]:step.pers_off[d] + n] = t
        else:
            step.full[step.full_off[d]:step.full_off[d] + n] = t
    step.init_from_full()
    sync()


def _send(step, grads, rank):
    """The ranks' gradients where the step expects them."""
    import torch
    for p in step.params:
        lo, hi = p["own"]
        d = p["ds_id"]
        if step.reduce_path == "coalesced" and not p["persistent"]:
            step.own_grads[step.grad_off[d]:step.grad_off[d] + p["numel"]] = torch.from_numpy(grads[rank][d].view(np.int16)).cuda()
            continue
        for v in range(step.N):
            i = step.recv_index(v, d)
            step.recv[i:i + hi - lo] = torch.from_numpy(grads[v][d][lo:hi].view(np.int16)).cuda()
    if step.reduce_path == "coalesced":
        for bi, (part, _, C, _, chunks) in enumerate(step.coalesced):
            for v, o in chunks.items():
                x = np.zeros(C, np.uint16)
                at = 0
                for d in part:
                    p = step.by_id[d]
                    lo, hi = p["own"]
                    x[at:at + hi - lo] = grads[v][d][lo:hi]
                    at += p["partition_size"]
                step.xbuf[o:o + C] = torch.from_numpy(x.view(np.int16)).cuda()


@pytest.mark.parametrize("dtype,world,rank,path,fuse,K", [("bf16", 4, 0, "contiguous", True, 3), ("fp16", 3, 1, "contiguous", False, 2),
                                                          ("bf16", 4, 3, "coalesced", True, 2), ("fp16", 1, 0, "contiguous", True, 4)])
def test_accumulated_steps_against_the_oracle(dtype, world, rank, path, fuse, K):
    import torch
    note(f"accumulated steps {dtype} N={world} rank {rank} {path} fuse_norm={fuse} K={K}")
    rng = np.random.default_rng(world * 10 + rank)
    step = _make(world, rank, dtype, reduce_path=path, fuse_norm=fuse, accumulate=K, no_decay=[9, 30, 7])
    try:
        L = oracle.make_layout(world, 100, IDS, SIZES)
        _start(step, rng)
        own = {p.ds_id: (p.shard_offset, p.shard_offset + L.own_range(p, rank)[1] - L.own_range(p, rank)[0]) for p in L.params}
        w = step.master.cpu().numpy().copy()
        m, v2 = np.zeros_like(w), np.zeros_like(w)
        stepped = 0
        for t in (1, 2, 3):
            acc = np.full(L.shard_numel, np.nan, np.float32)
            before = [x.clone() for x in (step.master, step.exp_avg, step.exp_avg_sq, step.shard)]
            for k in range(K):
                grads = [{p.ds_id: oracle.from_f32((rng.standard_normal(p.numel) * 1e-1).astype(np.float32), dtype) for p in L.params}
                         for _ in range(world)]
                if t == 2 and k == 0:
                    p = next(p for p in L.params if p.ds_id == 12)
                    grads[0][12][L.own_range(p, rank)[0] + 5] = 0x7C00 if dtype == "fp16" else 0x7F80
                flat = np.zeros(L.shard_numel, np.uint16)
                oracle.reduce_scatter(L, rank, dtype, IDS, grads, flat)
                _send(step, grads, rank)
                peers = [0.125 * (v + 1) for v in range(world)] + [0.0]
                step.sumsq.copy_(torch.tensor(peers, dtype=torch.float64))
                (step.step if k == K - 1 else step.micro_step)()
                sync()
                assert np.array_equal(_h16(step.grad), flat), "flat gradient"
                for lo, hi in own.values():
                    acc[lo:hi] = og.accumulate(acc[lo:hi], oracle.to_f32(flat[lo:hi], dtype), 1.0 / K, k == 0)
                    got = step.acc[lo:hi].cpu().numpy()
                    assert np.array_equal(got, acc[lo:hi], equal_nan=True), "accumulators"
            assert (step.t, step.micro) == (t, 0)
            flag = int(step.outs.view(torch.int32)[3])
            if t == 2:
                assert flag == 1
                for a, b in zip(before, (step.master, step.exp_avg, step.exp_avg_sq, step.shard)):
                    assert torch.equal(a, b)
                continue
            assert flag == 0
            parts = [(acc[slice(*own[p.ds_id])], p.persistent) for p in L.params]
            s = og.sums(parts, "2", peers, rank)
            norm, scale, _ = og.finalize(s, "2", 1.0, 1.0)
            # n positive terms in binary64, then a root
            tol = (sum(SIZES) + world + 2) * 2.0 ** -53 + 2.0 ** -51
            assert abs(float(step.outs[0]) - norm) <= tol * norm
            got = float(step.outs.view(torch.float32)[2])
            assert abs(got - scale) <= (2.0 ** -24 + tol) * scale
            each = step.grad_norms().cpu().numpy()
            top = step.grad_norms(inf=True).cpu().numpy()
            for i, (x, _) in enumerate(parts):
                assert abs(each[i] - math.sqrt(og.part(x, "2"))) <= tol * each[i]
                assert top[i] == og.part(x, "inf")
            stepped = t
            for p in L.params:
                lo, hi = own[p.ds_id]
                wd = 0.0 if p.ds_id in (9, 30, 7) else 0.1
                w[lo:hi], m[lo:hi], v2[lo:hi] = lb.adamw(w[lo:hi], m[lo:hi], v2[lo:hi], acc[lo:hi], scale=got, lr=1e-3, wd=wd,
                                                         beta1=0.9, beta2=0.99, eps=1e-8, step=t)[:3]
                for buf, want in ((step.master, w), (step.exp_avg, m), (step.exp_avg_sq, v2)):
                    assert np.array_equal(buf[lo:hi].cpu().numpy(), want[lo:hi])
                assert np.array_equal(_h16(step.shard[lo:hi]), oracle.from_f32(w[lo:hi], dtype))
        assert stepped == 3
        # the sum clipped for an optimizer of the caller's own
        step.clip_grads()
        sync()
        for lo, hi in own.values():
            assert np.array_equal(step.acc[lo:hi].cpu().numpy(), og.clip(acc[lo:hi], got, "fp32"))
    finally:
        step.destroy()


def test_accumulation_over_the_4_bit_wire():
    """Every micro-batch's average crosses the 4-bit wire with words of its own, and its flat gradient is what is accumulated."""
    note("4-bit gradients, three micro-batches")
    rng = np.random.default_rng(6)
    step = _make(4, 2, "bf16", reduce_path="coalesced", reduce_bits=4, gather_bits=4, state_bits=8, fuse_norm=True, accumulate=3, seed=2)
    try:
        _start(step, rng)
        for p in step.params:
            x = oracle.from_f32((rng.standard_normal(p["numel"]) * 1e-1).astype(np.float32), "bf16").view(np.int16)
            t = step.torch.from_numpy(x).cuda()
            if p["persistent"]:
                for v in range(4):
                    i = step.recv_index(v, p["ds_id"])
                    step.recv[i:i + p["numel"]] = t
            else:
                step.own_grads[step.grad_off[p["ds_id"]]:step.grad_off[p["ds_id"]] + p["numel"]] = t
        want, flats = np.zeros(step.S, np.float32), []
        for k in range(3):
            (step.step if k == 2 else step.micro_step)()
            sync()
            flats.append(_h16(step.grad))
            for p in step.params:
                lo, hi = p["shard_offset"], p["shard_offset"] + p["own"][1] - p["own"][0]
                want[lo:hi] = og.accumulate(want[lo:hi], oracle.to_f32(flats[k][lo:hi], "bf16"), 1 / 3, k == 0)
                assert np.array_equal(step.acc[lo:hi].cpu().numpy(), want[lo:hi])
        # the same gradients, rounded by other words: the own chunk's part of the averages differs
        assert not np.array_equal(flats[0], flats[1]) and not np.array_equal(flats[1], flats[2])
        assert int(step.outs.view(step.torch.int32)[3]) == 0 and float(step.outs[0]) > 0
    finally:
        step.destroy()


@pytest.mark.parametrize("bits", [32, 8])
def test_one_micro_batch_accumulated_is_the_sum_of_its_halves(bits):
    """Two equal micro-batches accumulate to their gradient itself (halving is exact): the norm is
    that of a step that takes it at once, and so is all that follows from it."""
    import torch
    note(f"two equal micro-batches, {bits}-bit states")
    rng = np.random.default_rng(3)
    a = _make(4, 1, "bf16", state_bits=bits, fuse_norm=True, accumulate=2, no_decay=[9], seed=3)
    b = _make(4, 1, "bf16", state_bits=bits, fuse_norm=True, no_decay=[9], seed=3)
    try:
        for st in (a, b):
            _start(st, np.random.default_rng(9))
        grads = [{d: oracle.from_f32((rng.standard_normal(n) * 1e-1).astype(np.float32), "bf16") for d, n in zip(IDS, SIZES)}
                 for _ in range(4)]
        for st in (a, b):
            _send(st, grads, 1)
        a.micro_step()
        a.step()
        b.step()
        sync()
        tol = 2 * (sum(SIZES) + 6) * 2.0 ** -53 + 2.0 ** -50
        na, nb = float(a.outs[0]), float(b.outs[0])
        assert abs(na - nb) <= tol * nb
        assert float(a.outs.view(torch.float32)[2]) == pytest.approx(float(b.outs.view(torch.float32)[2]), rel=2.0 ** -23)
        if float(a.outs.view(torch.float32)[2]) == float(b.outs.view(torch.float32)[2]):
            assert torch.equal(a.master, b.master) and torch.equal(a.exp_avg, b.exp_avg) and torch.equal(a.shard, b.shard)
        # and the flat gradient of a step without accumulators has norms and can be clipped, too
        flat, scale = _h16(b.grad), float(b.outs.view(torch.float32)[2])
        each = b.grad_norms().cpu().numpy()
        b.clip_grads()
        sync()
        for i, p in enumerate(b.params):
            o, n = p["shard_offset"], p["own"][1] - p["own"][0]
            x = oracle.to_f32(flat[o:o + n], "bf16")
            assert abs(each[i] - math.sqrt(og.part(x, "2"))) <= tol * each[i]
            assert np.array_equal(_h16(b.grad[o:o + n]), og.clip(x, scale, "bf16"))
    finally:
        a.destroy(), b.destroy()


def test_a_trace_scheduled_step_over_micro_batches():
    """The coordinator's gathers in every micro-batch."""
    import bench
    from synth import get_config
    from synth.modules import module_table, step_order
    from zero_sharded_state_amd.trace_schedule import TraceGatherPass
    note("c1 by trace, two micro-batches")
    cfg = get_config("c1")
    step = ShardStep(world_size=cfg.world_size, rank=1, threshold=cfg.threshold, ds_ids=cfg.ds_ids, numels=cfg.numels, dtype=cfg.dtype,
                     prefetch_bucket_size=cfg.prefetch_bucket_size, reduce_bucket_size=cfg.reduce_bucket_size,
                     sub_group_size=cfg.sub_group_size, fuse_norm=True, accumulate=2)
    try:
        bench.fill_inputs(step, cfg)
        _, mods = module_table(cfg)
        trace = TraceGatherPass(step, mods, step_order(cfg), {"prefetch_bucket_size": cfg.prefetch_bucket_size,
                                                              "max_live_parameters": int(1e9), "max_reuse_distance": int(1e9)})
        trace.plan()
        trace.fill_peer_chunks()
        phases = []
        step.micro_step(trace_pass=trace, on_phase=phases.append)
        step.step(trace_pass=trace, on_phase=phases.append)
        sync()
        assert phases == ["gather_trace", "reduce_scatter", "accumulate", None, "gather_trace", "reduce_scatter", "accumulate", "adam", None]
        for p in step.params:
            o, n = p["shard_offset"], p["own"][1] - p["own"][0]
            flat = oracle.to_f32(_h16(step.grad[o:o + n]), cfg.dtype)
            assert np.array_equal(step.acc[o:o + n].cpu().numpy(), flat)        # twice the half of one gradient
        assert np.array_equal(_h16(step.shard), oracle.from_f32(step.master.cpu().numpy(), cfg.dtype))
    finally:
        step.destroy()
    assert zs.zs3_abi_version() == 3


def _values(step, rng):
    """Random contents of the gradient that the step holds, and each parameter's real elements of it."""
    import torch
    x = (rng.standard_normal(step.S) * 1e-1).astype(np.float32)
    if step.acc is None:
        bits = oracle.from_f32(x, step.dtype)
        step.grad.copy_(torch.from_numpy(bits.view(np.int16)))
        x = oracle.to_f32(bits, step.dtype)
    else:
        step.acc.copy_(torch.from_numpy(x))
    return [x[p["shard_offset"]:p["shard_offset"] + p["own"][1] - p["own"][0]] for p in step.params]


def _check_each(each, parts, kind="2"):
    # sums of n positive terms in binary64, then a root
    tol = (sum(SIZES) * 2.0 ** -53 + 2.0 ** -51) if kind == "2" else 0.0
    want = [math.sqrt(og.part(x, kind)) if kind == "2" else og.part(x, kind) for x in parts]
    np.testing.assert_allclose(each.cpu().numpy(), want, rtol=tol, atol=0)


@pytest.mark.parametrize("accumulate", [1, 2])
@pytest.mark.parametrize("handle", [False, True], ids=["stream", "handle"])
def test_single_norms_and_clip_on_another_stream(accumulate, handle):
    """The step's first such calls, on a stream that is behind: their results, and that what is allocated
    and written on the current stream meanwhile stays as it was."""
    import torch
    note(f"norms and clip on another stream, accumulate={accumulate}")
    rng = np.random.default_rng(12)
    step = _make(4, 1, "bf16", accumulate=accumulate)
    try:
        s = torch.cuda.Stream()
        on = int(s.cuda_stream) if handle else s
        for k in range(4):
            parts = _values(step, rng)
            step.outs.zero_()
            step.outs.view(torch.float32)[2] = 0.75
            torch.cuda.synchronize()
            with torch.cuda.stream(s):
                torch.cuda._sleep(20_000_000)       # about 10 ms
            each, top = step.grad_norms(stream=on), step.grad_norms(inf=True, stream=on)
            step.clip_grads(stream=on)
            mine = [torch.full((2,), -7.0, dtype=torch.float64, device="cuda") for _ in range(200)]
            s.synchronize()
            _check_each(each, parts)
            _check_each(top, parts, "inf")
            assert all(bool((x == -7.0).all()) for x in mine)
            for x, p in zip(parts, step.params):
                o = p["shard_offset"]
                if accumulate == 1:
                    assert np.array_equal(_h16(step.grad[o:o + len(x)]), og.clip(x, 0.75, "bf16"))
                else:
                    assert np.array_equal(step.acc[o:o + len(x)].cpu().numpy(), og.clip(x, 0.75, "fp32"))
    finally:
        step.destroy()


@pytest.mark.parametrize("accumulate", [1, 2])
def test_single_norms_captured_at_once(accumulate):
    """A step's first call of them is captured, then replayed between eager ones."""
    import torch
    note(f"norms captured first, accumulate={accumulate}")
    rng = np.random.default_rng(13)
    step = _make(4, 1, "fp16", accumulate=accumulate)
    try:
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            each = step.grad_norms()
        for k in range(4):
            eager = step.grad_norms()
            parts = _values(step, rng)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            _check_each(each, parts)
            eager = step.grad_norms()
            torch.cuda.synchronize()
            assert torch.equal(eager, each)
    finally:
        step.destroy()


@pytest.mark.parametrize("K,fuse,phases", [(1, True, False), (1, False, False), (3, True, False), (3, False, False), (3, True, True)])
def test_an_optimizer_of_the_callers_own(K, fuse, phases):
    """Two steps in a row that stop before AdamW: the clipped sum of each, nothing of the step before in it,
    master and moments as they were, and parameters that the caller has written to the shard gathered next."""
    import torch
    note(f"own optimizer, K={K} fuse_norm={fuse} phases={phases}")
    world, rank, rng = 4, 1, np.random.default_rng(21)
    step = _make(world, rank, "bf16", fuse_norm=fuse, accumulate=K)
    try:
        L = oracle.make_layout(world, 100, IDS, SIZES)
        _start(step, rng)
        own = [(p.shard_offset, p.shard_offset + L.own_range(p, rank)[1] - L.own_range(p, rank)[0]) for p in L.params]
        before = [x.clone() for x in (step.master, step.exp_avg, step.exp_avg_sq)]
        for t in (1, 2):
            acc = np.full(L.shard_numel, np.nan, np.float32)
            for k in range(K):
                grads = [{p.ds_id: oracle.from_f32(rng.standard_normal(p.numel).astype(np.float32), "bf16") for p in L.params}
                         for _ in range(world)]
                flat = np.zeros(L.shard_numel, np.uint16)
                oracle.reduce_scatter(L, rank, "bf16", IDS, grads, flat)
                _send(step, grads, rank)
                step.sumsq.zero_()
                if phases:
                    step.gather_pass()
                    step.reduce_scatter()
                    step.accumulate_grads(norm=k == K - 1)
                else:
                    (step.gradient_step if k == K - 1 else step.micro_step)()
                for lo, hi in own:
                    x = oracle.to_f32(flat[lo:hi], "bf16")
                    acc[lo:hi] = x if K == 1 else og.accumulate(acc[lo:hi], x, 1.0 / K, k == 0)
            step.clip_grads()
            sync()
            assert (step.t, step.micro) == (t, 0)
            scale = float(step.outs.view(torch.float32)[2])
            s = og.sums([(acc[lo:hi], p.persistent) for (lo, hi), p in zip(own, L.params)], "2", [0.0] * (world + 1), rank)
            # sums of positive terms in binary64, a root, and the rounding to fp32
            want = og.finalize(s, "2", 1.0, 1.0)[1]
            assert scale < 1.0 and abs(scale - want) <= (2.0 ** -24 + (sum(SIZES) + 6) * 2.0 ** -53 + 2.0 ** -50) * want
            for lo, hi in own:
                if K == 1:
                    assert np.array_equal(_h16(step.grad[lo:hi]), og.clip(acc[lo:hi], scale, "bf16"))
                else:
                    assert np.array_equal(step.acc[lo:hi].cpu().numpy(), og.clip(acc[lo:hi], scale, "fp32"))
            for a, b in zip(before, (step.master, step.exp_avg, step.exp_avg_sq)):
                assert torch.equal(a, b)
            # the caller's own update
            held = step.grad.view(torch.bfloat16) if K == 1 else step.acc
            step.shard.view(torch.bfloat16).sub_(held, alpha=0.5)
            step.gather_pass()
            sync()
            for p in step.params:
                if not p["persistent"]:
                    o, (lo, hi) = step.full_off[p["ds_id"]], p["own"]
                    assert torch.equal(step.full[o + lo:o + hi], step.shard[p["shard_offset"]:p["shard_offset"] + hi - lo])
    finally:
        step.destroy()


@pytest.mark.parametrize("accumulate", [1, 2])
def test_a_norm_that_waits_for_the_other_ranks(accumulate):
    """The sums first, the end of the norm after the others' have come: the norm that has them at once, bit for bit
    where the same kernel ends it."""
    import torch
    note(f"norm in two parts, accumulate={accumulate}")
    rng = np.random.default_rng(31)
    step = _make(4, 2, "bf16", accumulate=accumulate)
    try:
        _start(step, rng)
        step.recv.copy_(torch.from_numpy(oracle.from_f32(rng.standard_normal(step.recv.numel()).astype(np.float32), "bf16").view(np.int16)))
        peers = [0.5, 7.0, 0.0, 11.0, 0.0]
        outs = []
        for parts in (True, False):
            step.outs.fill_(-1.0)
            step.sumsq.copy_(torch.tensor([0.0] * 5 if parts else peers, dtype=torch.float64))
            for k in range(accumulate):
                step.reduce_scatter()
                if accumulate > 1:
                    step.accumulate_grads(norm=k == accumulate - 1, finalize=not parts)
            if accumulate == 1:
                step.grad_norm(finalize=not parts)
            if parts:
                sync()
                assert bool((step.outs == -1.0).all())
                for v in (0, 1, 3):
                    step.sumsq[v] = peers[v]
                step.finalize_norm()
            sync()
            outs.append((float(step.outs[0]), float(step.outs.view(torch.float32)[2]), int(step.outs.view(torch.int32)[3])))
        (na, sa, fa), (nb, sb, fb) = outs
        # two sums of the same world + 1 positive terms, a root; the scale rounded to fp32 from these
        assert abs(na - nb) <= 8 * 2.0 ** -53 * nb and abs(sa - sb) <= 2.0 ** -23 * sb and fa == fb == 0
        if accumulate > 1:
            assert na == nb and sa == sb
    finally:
        step.destroy()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_equal_halves_step_to_the_same_bits(bits, dtype):
    """Two equal micro-batches accumulate to their gradient itself (halving is exact); with a clip norm that
    is not reached both scales are 1, and master, moments and shard are those of the step that takes it at once."""
    import torch
    note(f"equal halves, {bits}-bit states, {dtype}")
    rng = np.random.default_rng(41)
    a = _make(4, 1, dtype, state_bits=bits, fuse_norm=True, accumulate=2, no_decay=[9], seed=3, max_norm=1e9)
    b = _make(4, 1, dtype, state_bits=bits, fuse_norm=True, no_decay=[9], seed=3, max_norm=1e9)
    try:
        for st in (a, b):
            _start(st, np.random.default_rng(9))
        for _ in range(3):
            grads = [{d: oracle.from_f32((rng.standard_normal(n) * 1e-1).astype(np.float32), dtype) for d, n in zip(IDS, SIZES)}
                     for _ in range(4)]
            for st in (a, b):
                _send(st, grads, 1)
            a.micro_step()
            a.step()
            b.step()
            sync()
            assert float(a.outs.view(torch.float32)[2]) == float(b.outs.view(torch.float32)[2]) == 1.0
            for x, y in ((a.master, b.master), (a.exp_avg, b.exp_avg), (a.exp_avg_sq, b.exp_avg_sq), (a.shard, b.shard)):
                assert torch.equal(x, y)
    finally:
        a.destroy(), b.destroy()
