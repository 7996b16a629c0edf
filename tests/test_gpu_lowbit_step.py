"""Whole shard steps with 8-bit moments and 4-bit wires, the operators run
together as ``ShardStep`` runs them, against a chain of the oracle's: the
gathered parameters, own send chunks and flat gradient bit for bit, the norm
within 1e-12, moments bit for bit, the master within the bound of its update,
the shard its rounding; then a step with an infinite gradient, which crosses
the 4-bit wire, sets the flag and changes nothing."""

import gc

import numpy as np
import pytest

import oracle
import zero_sharded_state_amd as zs
from gpu_util import note, require_gpu, sync
from oracle import lowbit as lb
from zero_sharded_state_amd.shard_step import AdamConfig, ShardStep

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()
    yield
    import torch
    gc.collect()
    torch.cuda.empty_cache()


def _h16(t):
    return t.cpu().numpy().view(np.uint16).copy()


def _make(world, rank, dtype, ids, sizes, **k):
    return ShardStep(world_size=world, rank=rank, threshold=100, ds_ids=ids, numels=sizes, dtype=dtype, prefetch_bucket_size=9000,
                     reduce_bucket_size=7000, sub_group_size=3000, adam=AdamConfig(lr=1e-3, beta2=0.99, weight_decay=0.1),
                     fuse_norm=True, rs_streams=2, gather_streams=2, **k)


def _fill(step, rng):
    """Random full parameters; returns them by ds_id as 16-bit patterns."""
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
    return full


IDS, SIZES = [4, 9, 1, 30, 12, 7], [4097, 64, 5000, 33, 8191, 130]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("world,rank", [(4, 0), (4, 3), (3, 1)])
def test_low_bit_steps_against_the_oracle(dtype, world, rank):
    import torch
    note(f"low-bit steps N={world} rank {rank} {dtype}")
    rng = np.random.default_rng(world * 10 + rank)
    step = _make(world, rank, dtype, IDS, SIZES, reduce_path="coalesced", state_bits=8, gather_bits=4, reduce_bits=4,
                 no_decay=[9, 30, 7], seed=5)
    try:
        L = oracle.make_layout(world, 100, IDS, SIZES)
        full = _fill(step, rng)
        step.init_from_full()
        sync()
        shards = [oracle.partition(L, v, full) for v in range(world)]
        master = {p.ds_id: oracle.to_f32(shards[rank][p.shard_offset:p.shard_offset + np.subtract(*L.own_range(p, rank)[::-1])], dtype)
                  for p in L.params}
        mom = {d: (np.zeros(len(w), np.float32), np.zeros(len(w), np.float32)) for d, w in master.items()}
        pos = {p.ds_id: p for p in L.params}
        for t in (1, 2, 3):
            last = t == 3
            # this rank's gradients and what the peers send it
            grads = {v: {p.ds_id: oracle.from_f32((rng.standard_normal(p.numel) * 1e-3).astype(np.float32), dtype) for p in L.params}
                     for v in range(world)}
            if last:                        # an overflow in a peer's gradient of this rank's elements
                p = pos[12]
                grads[(rank + 1) % world][12][L.own_range(p, rank)[0] + 5] = 0x7C00 if dtype == "fp16" else 0x7F80
            ref = np.zeros(L.shard_numel, np.uint16)
            sent = {}
            for bi, (part, pers, C, send, _) in enumerate(step.coalesced):
                if not part:
                    continue
                seeds = {v: (5 << 32) + ((t * world + v) << 16) + [i for i, b in enumerate(step.coalesced) if b[0]].index(bi) for v in range(world)}
                sends = [lb.send4(L, part, grads[v], dtype, lb.keys(seeds[v], 0, 0)) for v in range(world)]
                sent[bi] = sends[rank]
                for v in range(world):
                    if v != rank:
                        o = step.recv_chunk_ptr(bi, v) - step.xbuf.data_ptr()
                        step.xbuf[o:o + C] = torch.from_numpy(sends[v][rank]).cuda()
                lb.reduce4(L, rank, part, [s[rank] for s in sends], dtype, ref)
            for p in L.params:
                d = p.ds_id
                if p.persistent:
                    oracle.reduce_scatter(L, rank, dtype, [d], [grads[v] for v in range(world)], ref)
                    for v in range(world):
                        i = step.recv_index(v, d)
                        step.recv[i:i + p.numel] = torch.from_numpy(grads[v][d].view(np.int16)).cuda()
                else:
                    o = step.grad_off[d]
                    step.own_grads[o:o + p.numel] = torch.from_numpy(grads[rank][d].view(np.int16)).cuda()
            before = (step.master.clone(), step.exp_avg.clone(), step.exp_avg_sq.clone(), step.shard.clone())
            step.sumsq.zero_()              # no peers' norms: this rank's alone
            step.step()
            sync()
            # gathered parameters: everybody's codes, the own ones from the shard as it was
            for bi, b in enumerate(step.gather_buckets):
                chunks = [lb.pack4(L, v, b, shards[v], dtype) for v in range(world)]
                f, n, _, _ = step.bucket_meta[bi]
                assert np.array_equal(_h16(step.full[f:f + n]), lb.unpack4(L, b, chunks, dtype)), "gathered"
            for bi, (part, _, C, send, _) in enumerate(step.coalesced):
                if part:
                    got = step.xbuf[send:send + world * C].cpu().numpy().reshape(world, C)
                    blocks = lb.bucket_places(L, part)[2]
                    assert np.array_equal(got[:, :17 * blocks], sent[bi][:, :17 * blocks]), "send"
            flat = _h16(step.grad)
            if last:
                assert int(step.outs.view(torch.int32)[3]) == 1, "flag"
                for a, b in zip(before, (step.master, step.exp_avg, step.exp_avg_sq, step.shard)):
                    assert torch.equal(a, b)
                assert np.isnan(oracle.to_f32(flat, dtype)).any()
                break
            assert np.array_equal(flat, ref), "flat gradient"
            x = oracle.to_f32(ref, dtype).astype(np.float64)
            norm = float(np.sqrt((x * x).sum()))
            assert abs(float(step.outs[0]) - norm) <= 1e-12 * norm
            scale = float(step.outs.view(torch.float32)[2])
            assert scale == np.float32(min(1.0, 1.0 / (norm + 1e-6)))
            got_w, got_s = step.master.cpu().numpy(), _h16(step.shard)
            for p in L.params:
                d, n, o = p.ds_id, len(master[p.ds_id]), p.shard_offset
                if n == 0:
                    continue
                wd = 0.0 if d in (9, 30, 7) else 0.1
                _, m, v, decayed, upd = lb.adamw(master[d], *mom[d], oracle.to_f32(flat[o:o + n], dtype), scale=scale, lr=1e-3, wd=wd,
                                                 beta1=0.9, beta2=0.99, eps=1e-8, step=t)
                exact = decayed.astype(np.float64) - upd
                # 11 half-ulps of the update and one of the result, as the list step's own test counts them
                assert np.all(np.abs(got_w[o:o + n] - exact) <= 2.0 ** -24 * (11 * 1.001 * np.abs(upd) + 1.001 * np.abs(exact)) + 2.0 ** -149)
                word = lb.words(lb.keys(5, t, d), np.arange(n))
                mom[d] = tuple(lb.decode_moment(*lb.encode_moment(y, word, k == 1), k == 1) for k, y in enumerate((m, v)))
                for a, b in zip(step.moments(d), mom[d]):
                    assert np.array_equal(a.cpu().numpy(), b), "moments"
                master[d] = got_w[o:o + n].copy()
                assert np.array_equal(got_s[o:o + n], oracle.from_f32(master[d], dtype)), "shard"
            shards[rank] = got_s
    finally:
        step.destroy()


def test_decay_by_parameter():
    """32-bit state: parameters in no_decay step as without decay, the others as
    the flat step does."""
    import torch
    note("no_decay")
    out = {}
    for name, wd, off in (("with", 0.1, ()), ("without", 0.0, ()), ("mixed", 0.1, (9, 30, 1))):
        rng = np.random.default_rng(3)
        step = _make(4, 2, "bf16", IDS, SIZES, no_decay=off)
        step.adam = AdamConfig(lr=1e-3, beta2=0.99, weight_decay=wd)
        step._marshal()
        _fill(step, rng)
        step.init_from_full()
        step.recv.copy_(torch.from_numpy(oracle.from_f32((rng.standard_normal(step.recv.numel()) * 1e-3).astype(np.float32), "bf16").view(np.int16)))
        for _ in range(2):
            step.sumsq.zero_()
            step.step()
        sync()
        out[name] = {p["ds_id"]: [x[p["shard_offset"]:p["shard_offset"] + p["own"][1] - p["own"][0]].cpu().numpy().copy()
                                  for x in (step.master, step.exp_avg, step.exp_avg_sq, step.shard)] for p in step.params}
        a, b = step.moments(4)
        assert np.array_equal(a.cpu().numpy(), out[name][4][1]) and np.array_equal(b.cpu().numpy(), out[name][4][2])
        step.destroy()
    for d in IDS:
        ref = out["without" if d in (9, 30, 1) else "with"][d]
        for a, b in zip(out["mixed"][d], ref):
            assert np.array_equal(a.view(np.uint8), b.view(np.uint8)), d


def test_low_bit_bytes_and_refusals():
    step = _make(4, 0, "bf16", IDS, SIZES, reduce_path="coalesced", state_bits=8, gather_bits=4, reduce_bits=4)
    plain = _make(4, 0, "bf16", IDS, SIZES, reduce_path="coalesced")
    a, b = step.algorithmic_bytes(), plain.algorithmic_bytes()
    own = step.own_real
    assert a["adam"] == 16 * own + own // 8 and b["adam"] == 28 * own
    assert a["pack"] < 0.7 * b["pack"] and a["unpack"] < 0.7 * b["unpack"]       # 2 + 17/32 bytes for 4
    assert a["scatter_pack"] < 0.7 * b["scatter_pack"] and a["reduce_scatter"] < 0.5 * b["reduce_scatter"]
    step.destroy()
    plain.destroy()
    for bad in (dict(state_bits=16), dict(gather_bits=8), dict(reduce_bits=4), dict(state_bits=8, offload=True),
                dict(no_decay=[5]), dict(gather_bits=4, single_launch="gather")):
        with pytest.raises(ValueError):
            _make(4, 0, "bf16", IDS, SIZES, **bad)


@pytest.mark.parametrize("dtype,world,rank", [("bf16", 300, 150), ("fp16", 300, 299), ("bf16", 257, 0)])
def test_a_step_over_more_ranks_than_a_launch_has_pointers(dtype, world, rank):
    """The 4-bit gradient wire past 256 ranks: a whole step's send chunks, flat
    gradient and norm against the oracle (peers send one of three sets)."""
    import torch
    note(f"low-bit step N={world} rank {rank} {dtype}")
    rng = np.random.default_rng(world + rank)
    step = _make(world, rank, dtype, IDS, SIZES, reduce_path="coalesced", state_bits=8, gather_bits=4, reduce_bits=4, seed=9)
    try:
        L = oracle.make_layout(world, 100, IDS, SIZES)
        _fill(step, rng)
        step.init_from_full()
        mk = lambda: {p.ds_id: oracle.from_f32((rng.standard_normal(p.numel) * 1e-3).astype(np.float32), dtype) for p in L.params}   # noqa: E731
        mine, peers = mk(), [mk() for _ in range(3)]
        ref = np.zeros(L.shard_numel, np.uint16)
        sent = {}
        step.t = 1                          # the seeds of the step under way
        for bi, (part, _, C, send, _) in enumerate(step.coalesced):
            if not part:
                continue
            i = [k for k, b in enumerate(step.coalesced) if b[0]].index(bi)
            sent[bi] = lb.send4(L, part, mine, dtype, lb.keys(step.wire_seed(i), 0, 0))
            theirs = [lb.send4(L, part, g, dtype, lb.keys(100 + k, 0, 0))[rank] for k, g in enumerate(peers)]
            chunks = [sent[bi][rank] if v == rank else theirs[v % 3] for v in range(world)]
            for v in range(world):
                if v != rank:
                    o = step.recv_chunk_ptr(bi, v) - step.xbuf.data_ptr()
                    step.xbuf[o:o + C] = torch.from_numpy(chunks[v]).cuda()
            lb.reduce4(L, rank, part, chunks, dtype, ref)
        step.t = 0
        for p in L.params:
            d = p.ds_id
            if p.persistent:
                every = [mine if v == rank else peers[v % 3] for v in range(world)]
                oracle.reduce_scatter(L, rank, dtype, [d], every, ref)
                for v in range(world):
                    k = step.recv_index(v, d)
                    step.recv[k:k + p.numel] = torch.from_numpy(every[v][d].view(np.int16)).cuda()
            else:
                o = step.grad_off[d]
                step.own_grads[o:o + p.numel] = torch.from_numpy(mine[d].view(np.int16)).cuda()
        step.sumsq.zero_()
        step.step()
        sync()
        for bi, (part, _, C, send, _) in enumerate(step.coalesced):
            if part:
                got = step.xbuf[send:send + world * C].cpu().numpy().reshape(world, C)
                blocks = lb.bucket_places(L, part)[2]
                assert np.array_equal(got[:, :17 * blocks], sent[bi][:, :17 * blocks]), "send"
        assert np.array_equal(_h16(step.grad), ref), "flat gradient"
        x = oracle.to_f32(ref, dtype).astype(np.float64)
        norm = float(np.sqrt((x * x).sum()))
        assert abs(float(step.outs[0]) - norm) <= 1e-12 * norm
    finally:
        step.destroy()


def test_settings_changed_between_steps():
    """Learning rate and weight decay changed between steps, in place and by a new
    AdamConfig: the list step (a parameter without decay makes it one) gives the
    flat step's bits for every parameter that decays."""
    import torch
    note("settings changed between steps")
    out = {}
    for name, off in (("flat", ()), ("listed", (9,))):
        rng = np.random.default_rng(23)
        step = _make(4, 1, "bf16", IDS, SIZES, no_decay=off)
        _fill(step, rng)
        step.init_from_full()
        step.recv.copy_(torch.from_numpy(oracle.from_f32((rng.standard_normal(step.recv.numel()) * 1e-3).astype(np.float32), "bf16").view(np.int16)))
        step.adam = AdamConfig(lr=1e-3, beta2=0.99, weight_decay=0.1)
        for lr, wd in ((1e-3, 0.1), (5e-4, 0.4), (2e-3, 0.0)):
            step.adam.lr, step.adam.weight_decay = lr, wd
            step.sumsq.zero_()
            step.step()
        step.adam = AdamConfig(lr=3e-3, beta2=0.9, weight_decay=0.2)
        step.sumsq.zero_()
        step.step()
        sync()
        out[name] = {p["ds_id"]: [x[p["shard_offset"]:p["shard_offset"] + p["own"][1] - p["own"][0]].cpu().numpy().copy()
                                  for x in (step.master, step.exp_avg, step.exp_avg_sq, step.shard)] for p in step.params}
        step.destroy()
    for d in IDS:
        if d == 9:
            continue
        for a, b in zip(out["flat"][d], out["listed"][d]):
            assert np.array_equal(a.view(np.uint8), b.view(np.uint8)), d
