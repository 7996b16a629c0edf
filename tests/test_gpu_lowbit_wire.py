"""GPU: the 4-bit wire of the coalesced gather and reduce-scatter against the
oracle (``oracle.lowbit``), bit for bit: codes, scales, gathered values and
averages (every step is exact or one IEEE operation)."""

import numpy as np
import pytest

import oracle
import zero_sharded_state_amd as zs
from gpu_util import Buf16, note, require_gpu, sync
from oracle import lowbit as lb

pytestmark = pytest.mark.gpu
PACK, UNPACK, REDUCE = zs.ZS3_PACK, zs.ZS3_UNPACK, zs.ZS3_REDUCE
GUARD = 64


class Bytes:
    """`rows` chunks of `n` bytes at a pitch, between canaries."""

    def __init__(self, rows, n, gap=0, data=None):
        import torch
        self.rows, self.n, self.pitch = rows, n, n + gap
        self.base = torch.full((rows * self.pitch + 2 * GUARD,), 0xA5, dtype=torch.uint8, device="cuda")
        if data is not None:
            for r in range(rows):
                self.row(r).copy_(torch.from_numpy(np.ascontiguousarray(data[r])).cuda())

    def row(self, r):
        return self.base[GUARD + r * self.pitch:GUARD + r * self.pitch + self.n]

    def ptrs(self):
        return [self.row(r).data_ptr() for r in range(self.rows)]

    def host(self):
        return np.stack([self.row(r).cpu().numpy() for r in range(self.rows)])


class Set:
    def __init__(self, world, sizes, dtype, seed=0, threshold=0):
        self.rng = np.random.default_rng(seed)
        self.world, self.dtype = world, dtype
        self.ids = [int(i) for i in self.rng.permutation(1000)[:len(sizes)]]
        self.h = zs.zs3_layout_create(world, threshold, self.ids, sizes)
        self.L = oracle.make_layout(world, threshold, self.ids, sizes)
        self.wire_ids = [p.ds_id for p in self.L.params if not p.persistent]

    def values(self, n, scale=0.02):
        x = self.rng.standard_normal(n) * scale * np.exp(self.rng.uniform(-3, 3, n))
        return oracle.from_f32(x.astype(np.float32), self.dtype)

    def full(self, scale=0.02):
        return {p.ds_id: self.values(p.numel, scale) for p in self.L.params}

    def __enter__(self):
        return self

    def __exit__(self, *a):
        zs.zs3_layout_destroy(self.h)


SETS = [
    (1, [1]),
    (1, [31, 32, 33, 100]),
    (2, [1, 2, 65]),
    (3, [1, 7, 96, 97, 1000]),
    (4, [2048, 32, 512, 16]),
    (5, [4, 5, 6, 12345]),
    (8, [8 * 32, 8 * 32 + 1, 70000]),
    (64, [63, 64 * 33, 100001]),
    (300, [150, 60001]),
]


def _ids(s):
    return "N%d-%s" % (s[0], "+".join(map(str, s[1])))


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("case", SETS, ids=_ids)
@pytest.mark.parametrize("shift", [0, 3])
def test_gather(case, dtype, shift):
    """Pack and unpack in one launch and apart, at the first, a middle and the
    last rank, requests in any order, garbage in the shard's padding."""
    require_gpu()
    world, sizes = case
    with Set(world, sizes, dtype, seed=world) as st:
        full = st.full()
        request = st.wire_ids[::-1]
        _, _, blocks, size = lb.bucket_places(st.L, request)
        shards = {}
        for r in range(world):
            shards[r] = oracle.partition(st.L, r, full)
            for p in st.L.params:
                lo, hi = st.L.own_range(p, r)
                shards[r][p.shard_offset + hi - lo:p.shard_offset + p.partition_size] = 0x7BFF
        chunks = [lb.pack4(st.L, r, request, shards[r], dtype, fill=0xA5) for r in range(world)]
        ref = lb.unpack4(st.L, request, chunks, dtype)
        n = sum(sizes)
        for rank in sorted({0, world // 2, world - 1}):
            note(f"mx4 gather N={world} rank {rank} {sizes} {dtype} shift {shift}")
            shard = Buf16(st.L.shard_numel, shift, shards[rank])
            for fused in (True, False):
                wire = Bytes(world, size, gap=16 * (rank % 2))
                for v in range(world):
                    if v != rank:
                        wire.row(v).copy_(__import__("torch").from_numpy(chunks[v]).cuda())
                out = Buf16(n, shift)
                ptrs = wire.ptrs()
                if fused:
                    offs = zs.zs3_gather_coalesced_mx4(st.h, rank, dtype, PACK | UNPACK, request, shard.ptr(), ptrs[rank],
                                                       ptrs[:rank] + [None] + ptrs[rank + 1:], out.ptr())
                else:
                    zs.zs3_gather_coalesced_mx4(st.h, rank, dtype, PACK, request, shard.ptr(), ptrs[rank])
                    offs = zs.zs3_gather_coalesced_mx4(st.h, rank, dtype, UNPACK, request, rank_chunks=ptrs, full_flat=out.ptr())
                sync()
                assert np.array_equal(wire.host()[rank], chunks[rank]), "own chunk"
                assert np.array_equal(out.host(), ref), "gathered values"
                out.check_guards()
                shard.check_guards()
                assert np.array_equal(shard.host(), shards[rank])
                at = {}
                f = 0
                for p in sorted(st.L.params, key=lambda p: p.ds_id):
                    at[p.ds_id] = f
                    f += p.numel
                assert offs == [at[d] for d in request]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("case", SETS, ids=_ids)
@pytest.mark.parametrize("stochastic", [False, True])
def test_send(case, dtype, stochastic):
    require_gpu()
    world, sizes = case
    with Set(world, sizes, dtype, seed=world + 100) as st:
        note(f"mx4 send N={world} {sizes} {dtype} sr={stochastic}")
        full = st.full(1e-3)
        request = st.wire_ids[::-1]
        _, _, _, size = lb.bucket_places(st.L, request)
        grads = {d: Buf16(len(full[d]), 1 + i % 8, full[d]) for i, d in enumerate(request)}
        send = Bytes(1, world * size)
        zs.zs3_reduce_scatter_coalesced_mx4(st.h, 0, dtype, PACK, request, grads=[grads[d].ptr() for d in request], send=send.ptrs()[0],
                                            rounding=int(stochastic), seed=77)
        sync()
        ref = lb.send4(st.L, request, full, dtype, lb.keys(77, 0, 0) if stochastic else None, fill=0xA5)
        got = send.host().reshape(world, size)
        assert np.array_equal(got, ref), int((got != ref).sum())
        b = send.base.cpu().numpy()
        assert np.all(b[:GUARD] == 0xA5) and np.all(b[-GUARD:] == 0xA5)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("case", SETS, ids=_ids)
@pytest.mark.parametrize("shift", [0, 1])
def test_reduce(case, dtype, shift):
    """The averages and, with them, every norm slot of the parameters (filled
    with NaN before): sums within 1e-12 of the oracle's, no slot left."""
    require_gpu()
    import torch
    world, sizes = case
    with Set(world, sizes, dtype, seed=world + 200) as st:
        request = st.wire_ids[::-1]
        _, _, _, size = lb.bucket_places(st.L, request)
        sends = [lb.send4(st.L, request, st.full(1e-3), dtype, fill=0xA5) for _ in range(min(world, 6))]
        for rank in sorted({0, world - 1}):
            note(f"mx4 reduce N={world} rank {rank} {sizes} {dtype} shift {shift}")
            data = [sends[v % len(sends)][rank] for v in range(world)]
            recv = Bytes(world, size, data=data)
            ref = np.full(st.L.shard_numel, 0x5A5A, np.uint16)
            lb.reduce4(st.L, rank, request, data, dtype, ref)
            for norm in (False, True):
                flat = Buf16(st.L.shard_numel, shift)
                slots, part = zs.zs3_layout_norm_slots(st.h)
                partials = torch.full((slots,), float("nan"), dtype=torch.float64, device="cuda")
                zs.zs3_reduce_scatter_coalesced_mx4(st.h, rank, dtype, REDUCE, request, recv_chunks=recv.ptrs(), grad_flat=flat.ptr(),
                                                    partials=partials if norm else None)
                sync()
                assert np.array_equal(flat.host(), ref), int((flat.host() != ref).sum())
                flat.check_guards()
                if norm:
                    got = float(partials.sum())
                    want = float((oracle.to_f32(ref, dtype).astype(np.float64) ** 2).sum())
                    assert abs(got - want) <= 1e-12 * want
                else:
                    assert torch.isnan(partials).all()


@pytest.mark.parametrize("world", [1, 2, 3, 7, 15, 37])
def test_reduce_of_a_large_partition(world):
    """Own parts of 2.1M elements and more take a thread two groups of elements at
    a time, smaller ones one: both, with ranks that fill no batch of chunks."""
    require_gpu()
    import torch
    note(f"mx4 large reduce N={world}")
    own = 512 * 4096 + 4097
    with Set(world, [own * world - 1, 333], "bf16", seed=world) as st:
        ids = st.wire_ids
        _, _, blocks, size = lb.bucket_places(st.L, ids)
        # random codes and scales are as good as any
        data = [st.rng.integers(0, 256, size).astype(np.uint8) for _ in range(min(world, 4))]
        for d in data:
            d[16 * blocks:17 * blocks] = st.rng.integers(100, 125, blocks)
        data = [data[v % len(data)] for v in range(world)]
        recv = Bytes(world, size, data=data)
        ref = np.zeros(st.L.shard_numel, np.uint16)
        lb.reduce4(st.L, world - 1, ids, data, "bf16", ref)
        flat = Buf16(st.L.shard_numel)
        slots, _ = zs.zs3_layout_norm_slots(st.h)
        partials = torch.full((slots,), float("nan"), dtype=torch.float64, device="cuda")
        zs.zs3_reduce_scatter_coalesced_mx4(st.h, world - 1, "bf16", REDUCE, ids, recv_chunks=recv.ptrs(), grad_flat=flat.ptr(),
                                            partials=partials)
        sync()
        assert np.array_equal(flat.host(), ref)
        want = float((oracle.to_f32(ref, "bf16").astype(np.float64) ** 2).sum())
        assert abs(float(partials.sum()) - want) <= 1e-12 * want


def test_norm_slots_of_some_parameters_only():
    """A bucket's slots are its parameters' own: those of persistent and of other
    parameters stay as they were, and the norm from both wires' slots is the norm
    of the flat gradient."""
    require_gpu()
    import torch
    world, rank = 4, 1
    with Set(world, [140000, 40, 33000, 4 * 32768, 500, 4 * 32768 + 4], "bf16", seed=5, threshold=100) as st:
        note("mx4 norm slots")
        L, ids = st.L, st.wire_ids
        slots, n_part = zs.zs3_layout_norm_slots(st.h)
        partials = torch.full((slots,), float("nan"), dtype=torch.float64, device="cuda")
        flat = Buf16(L.shard_numel)
        ref = np.full(L.shard_numel, 0x5A5A, np.uint16)
        for bucket in (ids[1::2], ids[::2]):
            _, _, _, size = lb.bucket_places(L, bucket)
            sends = [lb.send4(L, bucket, st.full(1e-3), "bf16") for _ in range(world)]
            recv = Bytes(world, size, data=[s[rank] for s in sends])
            lb.reduce4(L, rank, bucket, [s[rank] for s in sends], "bf16", ref)
            zs.zs3_reduce_scatter_coalesced_mx4(st.h, rank, "bf16", REDUCE, bucket, recv_chunks=recv.ptrs(), grad_flat=flat.ptr(),
                                                partials=partials)
            sync()
            if bucket == ids[1::2]:
                assert int(torch.isnan(partials[:n_part]).sum()) > 0
        host = partials.cpu().numpy()
        assert not np.isnan(host[:n_part]).any() and np.isnan(host[n_part:]).all()
        pers = [p for p in L.params if p.persistent]
        assert pers and all(np.all(flat.host()[p.shard_offset:p.shard_offset + p.numel] == 0x5A5A) for p in pers)
        assert np.array_equal(flat.host(), ref)
        real = np.concatenate([ref[p.shard_offset:p.shard_offset + p.partition_size] for p in L.params if not p.persistent])
        want = float((oracle.to_f32(real, "bf16").astype(np.float64) ** 2).sum())
        partials[n_part:] = 0
        sumsq = torch.zeros(world + 1, dtype=torch.float64, device="cuda")
        zs.zs3_grad_norm_partials(st.h, rank, partials, sumsq, False)
        sync()
        assert abs(float(sumsq[rank]) - want) <= 1e-12 * want


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_range_ends_and_nonfinite_values(dtype):
    """The types' largest and smallest values, zeros of both signs, and blocks
    with NaN and infinities, through pack, unpack and reduce."""
    require_gpu()
    note(f"mx4 range ends {dtype}")
    world = 2
    with Set(world, [512], dtype) as st:
        d = st.ids[0]
        big = 0x7BFF if dtype == "fp16" else 0x7F7F
        inf, nan = (0x7C00, 0x7E01) if dtype == "fp16" else (0x7F80, 0x7FC1)
        x = st.values(512)
        x[0], x[1] = big, big | 0x8000
        x[32:64] = 0
        x[40] = 0x8000
        x[64:96] = 0
        x[64] = 1                                    # the smallest subnormal
        x[96:128] = np.arange(32) if dtype == "fp16" else 0x0080 + np.arange(32)
        x[130] = nan
        x[170] = inf | 0x8000
        full = {d: x}
        shards = [oracle.partition(st.L, r, full) for r in range(world)]
        chunks = [lb.pack4(st.L, r, [d], shards[r], dtype) for r in range(world)]
        wire = Bytes(world, len(chunks[0]), data=chunks)
        wire.row(0).zero_()
        shard, out = Buf16(256, 0, shards[0]), Buf16(512)
        zs.zs3_gather_coalesced_mx4(st.h, 0, dtype, PACK | UNPACK, [d], shard.ptr(), wire.ptrs()[0], wire.ptrs(), out.ptr())
        flat = Buf16(256)
        zs.zs3_reduce_scatter_coalesced_mx4(st.h, 0, dtype, REDUCE, [d], recv_chunks=wire.ptrs(), grad_flat=flat.ptr())
        sync()
        got, ref = wire.host()[0], chunks[0]
        if dtype == "bf16":                          # fp32 subnormals: codes of a block under 2^-126 are not pinned
            got, ref = got.copy(), ref.copy()
            got[16 * 2:16 * 3], ref[16 * 2:16 * 3] = 0, 0
        assert np.array_equal(got, ref)
        o, r = oracle.to_f32(out.host(), dtype), oracle.to_f32(lb.unpack4(st.L, [d], chunks, dtype), dtype)
        assert np.isfinite(o[:128]).all() and np.isnan(o[128:192]).all()
        keep = np.r_[0:64, 96:512]
        assert np.array_equal(o[keep], r[keep], equal_nan=True)
        assert np.abs(o[64:96]).max() <= 2.0 ** -126 if dtype == "bf16" else np.array_equal(o[64:96], r[64:96])
        mean = oracle.to_f32(flat.host(), dtype)
        assert np.isnan(mean[128:192]).all() and np.isfinite(np.delete(mean, np.r_[128:192])).all()


def test_chunks_anywhere_and_pack_with_reduce():
    """Received chunks in separate allocations, the own one inside the send
    buffer, pack and reduce in one call."""
    require_gpu()
    note("mx4 pack + reduce")
    world, rank = 5, 3
    with Set(world, [9999, 31, 640], "fp16", seed=11) as st:
        ids = st.wire_ids
        _, _, _, size = lb.bucket_places(st.L, ids)
        mine, others = st.full(1e-3), [st.full(1e-3) for _ in range(world)]
        grads = [Buf16(len(mine[d]), 0, mine[d]) for d in ids]
        send = Bytes(1, world * size)
        sends = [lb.send4(st.L, ids, g, "fp16", lb.keys(5, 0, 0)) for g in others]
        sends[rank] = lb.send4(st.L, ids, mine, "fp16", lb.keys(5, 0, 0))
        recv = [Bytes(1, size, data=[sends[v][rank]]) for v in range(world)]
        ptrs = [r.ptrs()[0] for r in recv]
        ptrs[rank] = send.ptrs()[0] + rank * size
        flat = Buf16(st.L.shard_numel)
        zs.zs3_reduce_scatter_coalesced_mx4(st.h, rank, "fp16", PACK | REDUCE, ids, [g.ptr() for g in grads], send.ptrs()[0], ptrs,
                                            flat.ptr(), None, zs.ZS3_ROUND_STOCHASTIC, 5)
        sync()
        ref = np.zeros(st.L.shard_numel, np.uint16)
        lb.reduce4(st.L, rank, ids, [s[rank] for s in sends], "fp16", ref)
        assert np.array_equal(flat.host(), ref)


def test_many_parameters_in_a_bucket():
    """70 parameters (a launch holds 24) on 3 ranks, all three directions."""
    require_gpu()
    note("mx4 70 parameters")
    rng = np.random.default_rng(3)
    with Set(3, [int(x) for x in rng.integers(1, 900, 70)], "bf16", seed=21) as st:
        ids = [int(i) for i in rng.permutation(st.wire_ids)]
        _, _, _, size = lb.bucket_places(st.L, ids)
        full = st.full()
        shards = [oracle.partition(st.L, r, full) for r in range(3)]
        chunks = [lb.pack4(st.L, r, ids, shards[r], "bf16", fill=0xA5) for r in range(3)]
        wire = Bytes(3, size, data=chunks)
        wire.row(1).fill_(0xA5)
        shard, out = Buf16(st.L.shard_numel, 0, shards[1]), Buf16(sum(p.numel for p in st.L.params))
        zs.zs3_gather_coalesced_mx4(st.h, 1, "bf16", PACK | UNPACK, ids, shard.ptr(), wire.ptrs()[1], wire.ptrs(), out.ptr())
        grads = {d: Buf16(len(full[d]), 0, full[d]) for d in ids}
        send = Bytes(1, 3 * size)
        zs.zs3_reduce_scatter_coalesced_mx4(st.h, 1, "bf16", PACK, ids, [grads[d].ptr() for d in ids], send.ptrs()[0],
                                            rounding=1, seed=1)
        sync()
        assert np.array_equal(wire.host()[1], chunks[1])
        assert np.array_equal(out.host(), lb.unpack4(st.L, ids, chunks, "bf16"))
        ref = lb.send4(st.L, ids, full, "bf16", lb.keys(1, 0, 0), fill=0xA5)
        assert np.array_equal(send.host().reshape(3, size), ref)
        flat = Buf16(st.L.shard_numel)
        got = [send.ptrs()[0] + size] * 3
        zs.zs3_reduce_scatter_coalesced_mx4(st.h, 1, "bf16", REDUCE, ids, recv_chunks=got, grad_flat=flat.ptr())
        sync()
        want = np.zeros(st.L.shard_numel, np.uint16)
        lb.reduce4(st.L, 1, ids, [ref[1]] * 3, "bf16", want)
        assert np.array_equal(flat.host(), want)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_gather_past_the_last_level_cache(dtype):
    """A bucket of more than 256 MB, which is cut into other tiles: the values,
    and the own chunk, of calls that take its parameters one at a time."""
    require_gpu()
    import torch
    note(f"mx4 gather of 2^27 + elements {dtype}")
    world, rank = 3, 1
    sizes = [(1 << 26) + 5, 1, 8193, 3 * 8192, 3 * 8192 - 31, (1 << 26) + 4099]
    t = getattr(torch, {"fp16": "float16", "bf16": "bfloat16"}[dtype])
    with Set(world, sizes, dtype, seed=51) as st:
        ids = st.wire_ids
        gen = torch.Generator("cuda").manual_seed(5)
        shards = [(torch.randn(st.L.shard_numel, device="cuda", generator=gen) * 0.02).to(t) for _ in range(world)]

        def chunks_of(some):
            _, size = zs.zs3_mx4_sizes(st.h, some)
            wire = torch.zeros(world * size, dtype=torch.uint8, device="cuda")
            ptrs = [wire.data_ptr() + v * size for v in range(world)]
            for v in range(world):
                zs.zs3_gather_coalesced_mx4(st.h, v, dtype, PACK, some, shards[v], ptrs[v])
            return wire, ptrs

        one = {}
        for p in st.L.params:
            wire, ptrs = chunks_of([p.ds_id])
            one[p.ds_id] = torch.empty(p.numel, dtype=t, device="cuda")
            zs.zs3_gather_coalesced_mx4(st.h, rank, dtype, UNPACK, [p.ds_id], rank_chunks=ptrs, full_flat=one[p.ds_id])
        wire, ptrs = chunks_of(ids)
        packed = wire.clone()
        for fused in (False, True):
            out = torch.full((sum(sizes) + 64,), 7.0, dtype=t, device="cuda")
            if fused:
                wire.view(world, -1)[rank].zero_()
                zs.zs3_gather_coalesced_mx4(st.h, rank, dtype, PACK | UNPACK, ids, shards[rank], ptrs[rank], ptrs, out)
            else:
                zs.zs3_gather_coalesced_mx4(st.h, rank, dtype, UNPACK, ids, rank_chunks=ptrs, full_flat=out)
            sync()
            assert torch.equal(wire, packed)
            at = 0
            for d in ids:
                n = one[d].numel()
                assert torch.equal(out[at:at + n].view(torch.int16), one[d].view(torch.int16)), (d, fused)
                at += n
            assert bool((out[at:] == 7.0).all())


def test_captured_and_replayed():
    """Pack, unpack, send and reduce captured at their first call; every replay,
    with eager work between, gives the eager result of its inputs."""
    require_gpu()
    import torch
    note("mx4 captured")
    world, rank = 4, 2
    with Set(world, [4097, 130, 77], "bf16", seed=31) as st:
        ids = st.wire_ids
        _, _, _, size = lb.bucket_places(st.L, ids)
        full = [st.full() for _ in range(3)]
        chunks = [[lb.pack4(st.L, r, ids, oracle.partition(st.L, r, f), "bf16") for r in range(world)] for f in full]
        wire, out = Bytes(world, size, data=chunks[0]), Buf16(sum(p.numel for p in st.L.params))
        shard, flat = Buf16(st.L.shard_numel), Buf16(st.L.shard_numel)
        grads = {d: Buf16(len(full[0][d])) for d in ids}
        send = Bytes(1, world * size)
        graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(graph, stream=side):
            s = torch.cuda.current_stream()
            zs.zs3_gather_coalesced_mx4(st.h, rank, "bf16", PACK | UNPACK, ids, shard.ptr(), wire.ptrs()[rank], wire.ptrs(), out.ptr(), stream=s)
            zs.zs3_reduce_scatter_coalesced_mx4(st.h, rank, "bf16", PACK | REDUCE, ids, [grads[d].ptr() for d in ids], send.ptrs()[0],
                                                [send.ptrs()[0] + rank * size] * world, flat.ptr(), None, 1, 3, stream=s)
        for k in range(3):
            shard.view.copy_(torch.from_numpy(oracle.partition(st.L, rank, full[k]).view(np.int16)).cuda())
            for d in ids:
                grads[d].view.copy_(torch.from_numpy(full[k][d].view(np.int16)).cuda())
            for v in range(world):
                if v != rank:
                    wire.row(v).copy_(torch.from_numpy(chunks[k][v]).cuda())
            sync()
            graph.replay()
            sync()
            assert np.array_equal(out.host(), lb.unpack4(st.L, ids, chunks[k], "bf16"))
            ref = lb.send4(st.L, ids, full[k], "bf16", lb.keys(3, 0, 0))
            want = np.zeros(st.L.shard_numel, np.uint16)
            lb.reduce4(st.L, rank, ids, [ref[rank]] * world, "bf16", want)
            assert np.array_equal(flat.host(), want)


def test_two_streams_at_once():
    require_gpu()
    import torch
    note("mx4 two streams")
    with Set(2, [300001, 5003], "fp16", seed=41) as st:
        full = st.full()
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        work = []
        for d in st.wire_ids:
            chunks = [lb.pack4(st.L, r, [d], oracle.partition(st.L, r, full), "fp16") for r in range(2)]
            work.append((d, chunks, Bytes(2, len(chunks[0]), data=chunks), Buf16(len(full[d]))))
        shard = Buf16(st.L.shard_numel, 0, oracle.partition(st.L, 0, full))
        sync()
        for (d, _, wire, out), s in zip(work, streams):
            zs.zs3_gather_coalesced_mx4(st.h, 0, "fp16", PACK | UNPACK, [d], shard.ptr(), wire.ptrs()[0], wire.ptrs(), out.ptr(), stream=s)
        sync()
        for d, chunks, _, out in work:
            assert np.array_equal(out.host(), lb.unpack4(st.L, [d], chunks, "fp16"))


def test_a_parameter_past_32_bit_offsets():
    """One parameter of 2^32 + 2^20 + 7 elements over 2 ranks: a view of more
    than 2^32 elements, values sampled on both sides of 2^31 and 2^32."""
    require_gpu()
    import torch
    note("mx4 2^32 + 2^20 + 7 elements")
    n = (1 << 32) + (1 << 20) + 7
    h = zs.zs3_layout_create(2, 0, [0], [n])
    try:
        ps = -(-n // 2)
        _, size = zs.zs3_mx4_sizes(h, [0])
        grad = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
        spots = [0, ps - 40, ps, (1 << 31) + 7, (1 << 32) - 33, (1 << 32) + 5, n - 64]
        rng = np.random.default_rng(2)
        for s in spots:
            x = oracle.from_f32((rng.standard_normal(64) * 1e-3).astype(np.float32), "bf16")
            grad[s:s + 64] = torch.from_numpy(x.view(np.int16)).cuda().view(torch.bfloat16)
        send = torch.zeros(2 * size, dtype=torch.uint8, device="cuda")
        full = torch.empty(n, dtype=torch.bfloat16, device="cuda")
        flat = torch.empty(ps, dtype=torch.bfloat16, device="cuda")
        zs.zs3_reduce_scatter_coalesced_mx4(h, 0, "bf16", PACK, [0], [grad], send, rounding=1, seed=4)
        ptr = send.data_ptr()
        zs.zs3_gather_coalesced_mx4(h, 0, "bf16", UNPACK, [0], rank_chunks=[ptr, ptr + size], full_flat=full)
        zs.zs3_reduce_scatter_coalesced_mx4(h, 1, "bf16", REDUCE, [0], recv_chunks=[ptr + size] * 2, grad_flat=flat)
        sync()
        blocks = -(-ps // 32)
        for s in spots:
            for d in range(2):
                lo, hi = max(s, d * ps), min(s + 64, min(n, (d + 1) * ps))
                if hi <= lo:
                    continue
                k0 = (lo - d * ps) // 32 * 32                       # whole blocks around [lo, hi)
                k1 = min(-(-(hi - d * ps) // 32) * 32, blocks * 32)
                a, b = d * ps + k0, min(d * ps + k1, min(n, (d + 1) * ps))
                x = np.zeros(k1 - k0, np.float32)
                x[:b - a] = grad[a:b].float().cpu().numpy()
                at = d * blocks * 32 + k0 + np.arange(k1 - k0)
                w = lb.words(lb.keys(4, 0, 0), at // 2)
                w = np.where(at % 2 == 0, w, (w << np.uint32(1)) | (w >> np.uint32(31)))
                ref = lb.decode4(*lb.encode4(x, "bf16", w))[:b - a]
                assert np.array_equal(full[a:b].float().cpu().numpy(), ref), (s, d)
                if d == 1:
                    assert np.array_equal(flat[k0:k0 + b - a].float().cpu().numpy(), ref)
    finally:
        zs.zs3_layout_destroy(h)


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("world,rank", [(257, 0), (300, 150), (300, 299), (520, 1)])
def test_reduce_of_many_ranks_with_the_own_chunk_apart(world, rank, norm):
    """More chunks than a launch has pointers: evenly spaced ones, and the own one
    in an allocation of its own (what stands in its place between the others
    is not read)."""
    require_gpu()
    import torch
    note(f"mx4 reduce N={world} rank {rank}, own chunk apart, norm {norm}")
    with Set(world, [world * 5 + 1, 60001, 33], "bf16", seed=world + rank) as st:
        ids = st.wire_ids[::-1]
        _, _, _, size = lb.bucket_places(st.L, ids)
        sends = [lb.send4(st.L, ids, st.full(1e-3), "bf16", fill=0xA5) for _ in range(3)]
        data = [sends[v % 3][rank] for v in range(world)]
        recv = Bytes(world, size, gap=16, data=data)
        own = Bytes(1, size, data=[data[rank]])
        recv.row(rank).fill_(0xFF)
        ptrs = recv.ptrs()
        ptrs[rank] = own.ptrs()[0]
        flat = Buf16(st.L.shard_numel, 1)
        ref = np.full(st.L.shard_numel, 0x5A5A, np.uint16)
        lb.reduce4(st.L, rank, ids, data, "bf16", ref)
        slots, _ = zs.zs3_layout_norm_slots(st.h)
        partials = torch.full((slots,), float("nan"), dtype=torch.float64, device="cuda")
        zs.zs3_reduce_scatter_coalesced_mx4(st.h, rank, "bf16", REDUCE, ids, recv_chunks=ptrs, grad_flat=flat.ptr(),
                                            partials=partials if norm else None)
        sync()
        assert np.array_equal(flat.host(), ref)
        flat.check_guards()
        if norm:
            want = float((oracle.to_f32(ref, "bf16").astype(np.float64) ** 2).sum())
            assert abs(float(partials.sum()) - want) <= 1e-12 * want


@pytest.mark.parametrize("rank", [0, 150, 299])
def test_gather_of_many_ranks_with_chunks_anywhere(rank):
    """More unevenly spaced chunks than a launch has pointers: several launches,
    the own rank in the first or a later one, both modes."""
    require_gpu()
    import torch
    note(f"mx4 gather N=300 rank {rank}, uneven chunks")
    world = 300
    with Set(world, [world * 7 + 3, 60001, 64], "fp16", seed=rank) as st:
        ids = st.wire_ids
        _, _, _, size = lb.bucket_places(st.L, ids)
        full = st.full()
        shards = {r: oracle.partition(st.L, r, full) for r in range(world)}
        chunks = [lb.pack4(st.L, r, ids, shards[r], "fp16", fill=0xA5) for r in range(world)]
        at, o = [], 0
        for v in range(world):
            at.append(o)
            o += size + 16 * int(st.rng.integers(0, 5))
        shard = Buf16(st.L.shard_numel, 1, shards[rank])
        host = np.full(o, 0xA5, np.uint8)
        for v in range(world):
            host[at[v]:at[v] + size] = chunks[v]
        ref = lb.unpack4(st.L, ids, chunks, "fp16")
        for fused in (True, False):
            wire = torch.from_numpy(host).cuda()
            ptrs = [wire.data_ptr() + a for a in at]
            out = Buf16(sum(p.numel for p in st.L.params), 3)
            if fused:
                wire[at[rank]:at[rank] + size] = 0xA5
                zs.zs3_gather_coalesced_mx4(st.h, rank, "fp16", PACK | UNPACK, ids, shard.ptr(), ptrs[rank], ptrs, out.ptr())
            else:
                zs.zs3_gather_coalesced_mx4(st.h, rank, "fp16", UNPACK, ids, rank_chunks=ptrs, full_flat=out.ptr())
            sync()
            assert np.array_equal(wire.cpu().numpy(), host)
            assert np.array_equal(out.host(), ref)
            out.check_guards()
