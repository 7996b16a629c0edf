"""The low-bit entry points without a GPU: sizes against the oracle, and every
refusal (arguments are checked before any device work, so the addresses here
are made up and never read)."""

import ctypes
import os
import re
import shutil
import subprocess

import numpy as np
import pytest

import oracle
import zero_sharded_state_amd as zs
from oracle import lowbit as lb

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BASE = 1 << 40
HP = {"lr": 1e-3, "beta1": 0.9, "beta2": 0.999, "eps": 1e-8, "step": 1}


def _refused(status, text, fn, *a, **k):
    with pytest.raises(zs.Zs3Error) as e:
        fn(*a, **k)
    assert e.value.status == status, e.value
    assert text in e.value.message, e.value.message


def _tensor(numel=100, at=BASE, bits=32, grad_bytes=2, **over):
    step = 1 << 20
    t = dict(numel=numel, id=0, master=at, grad=at + step, param=at + 2 * step, exp_avg=at + 3 * step,
             exp_avg_sq=at + 4 * step, lr_scale=1.0, weight_decay=0.0)
    t.update(over)
    return t


def _step(tensors, dtype="bf16", grad="bf16", bits=32, scale=None, flag=None, hp=HP, seed=0):
    zs.zs3_adamw_tensors(dtype, grad, bits, tensors, scale, flag, hp, seed, stream=0)


def test_library_exports_every_declared_symbol():
    text = open(os.path.join(ROOT, "include", "zs3_lowbit.h")).read()
    syms = sorted(set(re.findall(r"ZS3_API\s+[\w\s\*]*?\b(zs3_\w+)\s*\(", text)))
    assert syms == sorted(zs.EXPORTS_LOWBIT) and all(hasattr(zs.lib(), s) for s in syms)


@pytest.mark.skipif(shutil.which("gcc") is None, reason="no gcc")
@pytest.mark.parametrize("lang", ["c99", "c++17"])
def test_header_is_plain_c(tmp_path, lang):
    """It compiles with warnings as errors, and its structs are laid out as the
    binding has them."""
    src = tmp_path / "t.c"
    src.write_text('''#include <stddef.h>
#include <stdio.h>
#include "zs3_lowbit.h"
int main(void) {
    int64_t b = 0;
    printf("%d %d %d %d\\n", (int)sizeof(zs3_adamw_tensor), (int)offsetof(zs3_adamw_tensor, lr_scale),
           (int)sizeof(zs3_moment8), (int)offsetof(zs3_moment8, kind));
    if (zs3_moment8_bytes(33, &b) != ZS3_OK || b != 80) return 1;
    return zs3_adamw_tensors(ZS3_BF16, ZS3_FP32, 9, 0, NULL, NULL, NULL, NULL, 0, NULL) == ZS3_EINVAL ? 0 : 2;
}
''')
    exe, pkg = str(tmp_path / "t"), os.path.join(ROOT, "zero_sharded_state_amd")
    cmd = ["gcc", "-std=c99", "-pedantic"] if lang == "c99" else ["g++", "-std=c++17", "-x", "c++"]
    cmd += ["-Wall", "-Wextra", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-x", "none", "-L", pkg, "-lzs3",
            f"-Wl,-rpath,{pkg}", "-o", exe]
    b = subprocess.run(cmd, capture_output=True, text=True)
    assert b.returncode == 0, b.stdout + b.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    t, m = zs.zs3_adamw_tensor, zs.zs3_moment8
    assert r.returncode == 0
    assert r.stdout.split() == [str(x) for x in (ctypes.sizeof(t), t.lr_scale.offset, ctypes.sizeof(m), m.kind.offset)]


# ------------------------------------------------------------------- AdamW

@pytest.mark.parametrize("n", [0, 1, 31, 32, 33, 511, 512, 513, 4095, 1 << 33, (1 << 35) - 2048])
def test_moment_bytes(n):
    assert zs.zs3_moment8_bytes(n) == lb.moment_bytes(n)


def test_moment_bytes_refusals():
    _refused(zs.ZS3_EINVAL, "out of range", zs.zs3_moment8_bytes, -1)
    _refused(zs.ZS3_EINVAL, "out of range", zs.zs3_moment8_bytes, 1 << 36)
    assert zs.lib().zs3_moment8_bytes(1, None) == zs.ZS3_EINVAL


def test_empty_lists_do_nothing():
    _step([])
    _step([_tensor(numel=0, master=0, grad=0, param=0, exp_avg=0, exp_avg_sq=0)], bits=8)
    zs.zs3_moment8_read("bf16", [], stream=0)
    zs.zs3_moment8_read("fp32", [dict(numel=0, kind=1, moment=0, out=0)], stream=0)


@pytest.mark.parametrize("bits", [8, 32])
def test_adamw_refusals(bits):
    t = _tensor
    for d in (0, 3, 7):
        _refused(zs.ZS3_EDTYPE, "dtype", _step, [t()], dtype=d, bits=bits)
    for d in (0, 4):
        _refused(zs.ZS3_EDTYPE, "grad_dtype", _step, [t()], grad=d, bits=bits)
    for b in (0, 4, 16, 64):
        _refused(zs.ZS3_EINVAL, "state_bits", _step, [t()], bits=b)
    for k in ("master", "grad", "exp_avg", "exp_avg_sq"):
        _refused(zs.ZS3_EINVAL, "NULL", _step, [t(**{k: 0})], bits=bits)
    _refused(zs.ZS3_EINVAL, "numel", _step, [t(numel=-1)], bits=bits)
    _refused(zs.ZS3_EINVAL, "numel", _step, [t(numel=1 << 60)], bits=bits)
    # nothing of a list is launched where a later tensor is refused
    _refused(zs.ZS3_EINVAL, "tensor 1: numel", _step, [t(), t(at=BASE + (1 << 30), numel=1 << 36)], bits=bits)
    for k, off in (("master", 2), ("grad", 1), ("param", 1)):
        _refused(zs.ZS3_EINVAL, "aligned", _step, [t(**{k: t()[k] + off})], bits=bits)
    _refused(zs.ZS3_EINVAL, "aligned", _step, [t(grad=t()["grad"] + 2)], grad="fp32", bits=bits)
    for k in ("exp_avg", "exp_avg_sq"):
        off = 8 if bits == 8 else 2
        _refused(zs.ZS3_EINVAL, "%d-byte" % (16 if bits == 8 else 4), _step, [t(**{k: t()[k] + off})], bits=bits)
    for k in ("lr_scale", "weight_decay"):
        _refused(zs.ZS3_EINVAL, "not finite", _step, [t(**{k: float("nan")})], bits=bits)
    for bad in ({"step": 0}, {"beta1": 1.0}, {"beta2": -0.1}, {"beta2": float("nan")}, {"eps": -1.0},
                {"eps": float("inf")}, {"lr": float("inf")}):
        _refused(zs.ZS3_EINVAL, "", _step, [t()], hp=dict(HP, **bad), bits=bits)
    if bits == 8:
        _refused(zs.ZS3_EINVAL, "eps", _step, [t()], hp=dict(HP, eps=1e-13), bits=bits)
    _refused(zs.ZS3_EINVAL, "scale", _step, [t()], scale=BASE + 2, bits=bits)
    _refused(zs.ZS3_EINVAL, "scale", _step, [t()], flag=BASE + 2, bits=bits)
    f = zs.lib().zs3_adamw_tensors
    assert f(2, 2, bits, 1, None, None, None, ctypes.byref(zs._hp(HP)), 0, None) == zs.ZS3_EINVAL
    assert f(2, 2, bits, -1, None, None, None, ctypes.byref(zs._hp(HP)), 0, None) == zs.ZS3_EINVAL
    assert f(2, 2, bits, 0, None, None, None, None, 0, None) == zs.ZS3_EINVAL


@pytest.mark.parametrize("bits", [8, 32])
def test_adamw_refuses_overlaps(bits):
    far = BASE + (1 << 30)
    _refused(zs.ZS3_EALIAS, "overlap", _step, [_tensor(), _tensor()], bits=bits)            # the same tensor twice
    _refused(zs.ZS3_EALIAS, "overlap", _step, [_tensor(), _tensor(at=far, master=BASE + 396)], bits=bits)
    one = _tensor()
    _refused(zs.ZS3_EALIAS, "overlap", _step, [_tensor(param=one["grad"])], bits=bits)
    _refused(zs.ZS3_EALIAS, "overlap", _step, [_tensor(exp_avg=one["exp_avg_sq"])], bits=bits)
    _refused(zs.ZS3_EALIAS, "overlap", _step, [one], scale=one["master"] + 4, bits=bits)
    size = lb.moment_bytes(100) if bits == 8 else 400
    _refused(zs.ZS3_EALIAS, "overlap", _step, [_tensor(exp_avg_sq=one["exp_avg"] + size - 16)], bits=bits)


def test_moment_read_refusals():
    m = dict(numel=100, kind=zs.ZS3_EXP_AVG, moment=BASE, out=BASE + (1 << 20))
    read = lambda d, **k: zs.zs3_moment8_read(d, [dict(m, **k)], stream=0)     # noqa: E731
    _refused(zs.ZS3_EDTYPE, "out_dtype", read, "fp16")
    _refused(zs.ZS3_EINVAL, "kind", read, "bf16", kind=0)
    _refused(zs.ZS3_EINVAL, "NULL", read, "bf16", moment=0)
    _refused(zs.ZS3_EINVAL, "NULL", read, "bf16", out=0)
    _refused(zs.ZS3_EINVAL, "aligned", read, "bf16", moment=BASE + 8)
    _refused(zs.ZS3_EINVAL, "aligned", read, "fp32", out=m["out"] + 2)
    _refused(zs.ZS3_EINVAL, "out of range", read, "bf16", numel=-5)
    _refused(zs.ZS3_EALIAS, "overlap", read, "bf16", out=BASE + 96)


# --------------------------------------------------------------------- wire

@pytest.fixture
def layout():
    h = zs.zs3_layout_create(4, 50, [5, 1, 9, 7], [1000, 33, 130, 40])
    yield h
    zs.zs3_layout_destroy(h)


@pytest.mark.parametrize("world", [1, 3, 8, 64])
def test_chunk_sizes(world):
    rng = np.random.default_rng(world)
    for _ in range(20):
        n = int(rng.integers(1, 8))
        ids, sizes = list(range(n)), [int(x) for x in rng.integers(1, 5000, n)]
        h = zs.zs3_layout_create(world, 0, ids, sizes)
        try:
            L = oracle.make_layout(world, 0, ids, sizes)
            pick = [int(i) for i in rng.permutation(n)[:max(1, n // 2)]]
            _, _, blocks, size = lb.bucket_places(L, pick)
            assert zs.zs3_mx4_sizes(h, pick) == (blocks, size)
        finally:
            zs.zs3_layout_destroy(h)


def test_size_refusals(layout):
    _refused(zs.ZS3_ENOTFOUND, "ds_id", zs.zs3_mx4_sizes, layout, [2])
    _refused(zs.ZS3_EPERSIST, "persistent", zs.zs3_mx4_sizes, layout, [1])
    _refused(zs.ZS3_EDUPID, "twice", zs.zs3_mx4_sizes, layout, [5, 9, 5])
    assert zs.lib().zs3_mx4_sizes(None, 0, None, None, None) == zs.ZS3_EINVAL
    assert zs.lib().zs3_mx4_sizes(layout, -1, None, None, None) == zs.ZS3_EINVAL
    assert zs.zs3_mx4_sizes(layout, []) == (0, 0)


def _gather(h, rank=1, dtype="bf16", mode=3, ids=(5, 9), shard=BASE, own=BASE + (1 << 20), chunks=None, full=BASE + (8 << 20)):
    if chunks is None:
        chunks = [own if v == rank else BASE + (2 << 20) + (v << 16) for v in range(4)]
    zs.zs3_gather_coalesced_mx4(h, rank, dtype, mode, list(ids), shard, own, chunks, full, stream=0)


def test_gather_refusals(layout):
    g = _gather
    _refused(zs.ZS3_EINVAL, "rank", g, layout, rank=4, chunks=[BASE] * 4)
    _refused(zs.ZS3_EINVAL, "rank", g, layout, rank=-1, chunks=[BASE] * 4)
    _refused(zs.ZS3_EDTYPE, "dtype", g, layout, dtype="fp32")
    for m in (0, 4, 7, -1):
        _refused(zs.ZS3_EINVAL, "mode", g, layout, mode=m)
    _refused(zs.ZS3_EPERSIST, "persistent", g, layout, ids=(5, 1))
    _refused(zs.ZS3_EDUPID, "twice", g, layout, ids=(5, 5))
    _refused(zs.ZS3_EINVAL, "shard_flat", g, layout, shard=0)
    _refused(zs.ZS3_EINVAL, "shard_flat", g, layout, shard=BASE + 1)
    _refused(zs.ZS3_EINVAL, "own_chunk", g, layout, own=BASE + 8)
    _refused(zs.ZS3_EINVAL, "full_flat", g, layout, full=0)
    _refused(zs.ZS3_EINVAL, "rank_chunks[rank]", g, layout, chunks=[BASE + (2 << 20) + (v << 16) for v in range(4)])
    ok = [BASE + (1 << 20) if v == 1 else BASE + (2 << 20) + (v << 16) for v in range(4)]
    _refused(zs.ZS3_EINVAL, "rank_chunks[v]", g, layout, chunks=ok[:3] + [0])
    _refused(zs.ZS3_EINVAL, "rank_chunks[v]", g, layout, chunks=ok[:3] + [ok[3] + 8])
    _refused(zs.ZS3_EINVAL, "rank_chunks[v]", g, layout, mode=2, chunks=[ok[0], 0, ok[2], ok[3]])   # unpack alone reads it
    _refused(zs.ZS3_EALIAS, "overlaps", g, layout, full=BASE + (2 << 20))
    _refused(zs.ZS3_EALIAS, "overlaps", g, layout, chunks=[ok[1] + 16] + ok[1:])
    _refused(zs.ZS3_EALIAS, "overlaps", g, layout, shard=ok[1])
    _gather(layout, ids=())                                                        # nothing to do


def _scatter(h, rank=1, dtype="bf16", mode=5, ids=(5, 9), grads=None, send=BASE, recv=None, flat=BASE + (8 << 20),
             partials=None, rounding=0):
    grads = [BASE + (1 << 20), BASE + (2 << 20)] if grads is None else grads
    recv = [BASE + (3 << 20) + (v << 16) for v in range(4)] if recv is None else recv
    zs.zs3_reduce_scatter_coalesced_mx4(h, rank, dtype, mode, list(ids), grads, send, recv, flat, partials, rounding, 0,
                                        stream=0)


def test_scatter_refusals(layout):
    g = _scatter
    _refused(zs.ZS3_EINVAL, "rank", g, layout, rank=4)
    _refused(zs.ZS3_EDTYPE, "dtype", g, layout, dtype="fp32")
    for m in (0, 2, 3, 8):
        _refused(zs.ZS3_EINVAL, "mode", g, layout, mode=m)
    for r in (-1, 2):
        _refused(zs.ZS3_EINVAL, "rounding", g, layout, rounding=r)
    _refused(zs.ZS3_EPERSIST, "persistent", g, layout, ids=(5, 1))
    _refused(zs.ZS3_EINVAL, "grads", g, layout, grads=[BASE + (1 << 20), 0])
    _refused(zs.ZS3_EINVAL, "send", g, layout, send=BASE + 8)
    _refused(zs.ZS3_EINVAL, "grad_flat", g, layout, flat=BASE + (8 << 20) + 1)
    _refused(zs.ZS3_EINVAL, "recv_chunks", g, layout, recv=[BASE + (3 << 20)] * 3 + [0])
    _refused(zs.ZS3_EINVAL, "partials", g, layout, partials=BASE + (9 << 20) + 4)
    _refused(zs.ZS3_EALIAS, "send", g, layout, grads=[BASE + 64, BASE + (2 << 20)])
    _refused(zs.ZS3_EALIAS, "grad_flat", g, layout, recv=[BASE + (8 << 20)] * 4)
    _refused(zs.ZS3_EALIAS, "send overlaps", g, layout, send=BASE + (8 << 20) + 64)
    _refused(zs.ZS3_EALIAS, "grad_flat", g, layout, partials=BASE + (3 << 20))
    _refused(zs.ZS3_EALIAS, "send overlaps", g, layout, partials=BASE + 16)


def test_partitions_too_large_for_a_launch():
    h = zs.zs3_layout_create(2, 0, [0, 1], [64, 1 << 37])
    try:
        _refused(zs.ZS3_EINVAL, "too large", zs.zs3_mx4_sizes, h, [0, 1])
        _refused(zs.ZS3_EINVAL, "too large", zs.zs3_gather_coalesced_mx4, h, 0, "bf16", zs.ZS3_PACK, [0, 1], BASE, BASE + (1 << 39), stream=0)
    finally:
        zs.zs3_layout_destroy(h)


def test_more_ranks_than_pointers_need_even_spacing():
    world = 300
    h = zs.zs3_layout_create(world, 0, [0], [100000])
    try:
        recv = [BASE + (3 << 20) + (v << 12) for v in range(world)]
        recv[17] += 16
        with pytest.raises(zs.Zs3Error) as e:
            zs.zs3_reduce_scatter_coalesced_mx4(h, 0, "bf16", zs.ZS3_REDUCE, [0], recv_chunks=recv, grad_flat=BASE,
                                                stream=0)
        assert e.value.status == zs.ZS3_EINVAL and "evenly" in e.value.message
    finally:
        zs.zs3_layout_destroy(h)


def test_types_of_the_16_bit_calls_are_what_they_were():
    """fp32 names a type of gradients and read moments only."""
    assert zs.DTYPES == {"fp16": zs.ZS3_FP16, "bf16": zs.ZS3_BF16}
    h = zs.zs3_layout_create(2, 0, [0], [64])
    try:
        with pytest.raises(KeyError):
            zs.zs3_init_master(h, 0, "fp32", 0, 32, 4096, 8192, stream=0)
    finally:
        zs.zs3_layout_destroy(h)


def test_lists_made_without_the_helpers():
    """A plain array of the structures counts its own entries."""
    for arr, call in (((zs.zs3_adamw_tensor * 3)(), lambda a: zs.zs3_adamw_tensors("bf16", "fp32", 8, a, None, None,
                                                                                  dict(HP, step=1), stream=0)),
                      ((zs.zs3_moment8 * 3)(), lambda a: zs.zs3_moment8_read("fp32", a, stream=0))):
        if isinstance(arr[0], zs.zs3_moment8):
            for x in arr:
                x.kind = zs.ZS3_EXP_AVG
        call(arr)                      # numel 0: skipped
        arr[2].numel = 5
        _refused(zs.ZS3_EINVAL, " 2: ", call, arr)


def _host_step(**k):
    from zero_sharded_state_amd.shard_step import ShardStep
    return ShardStep(world_size=2, rank=0, threshold=0, ds_ids=[0, 1], numels=[64, 65], dtype="bf16", prefetch_bucket_size=1000,
                     reduce_bucket_size=1000, sub_group_size=1000, device="cpu", **k)


def test_shard_step_takes_no_decay_from_any_iterable():
    for names in ([1], (1,), {1}, (d for d in [1])):
        st = _host_step(no_decay=names)
        assert st.no_decay == {1} and st.listed
        st.destroy()
    with pytest.raises(ValueError, match="not there"):
        _host_step(no_decay=(d for d in [7]))


def test_a_refused_step_does_not_count():
    st = _host_step(gather_bits=4)
    with pytest.raises(ValueError, match="16-bit wire"):
        st.step(trace_pass=object())
    assert st.t == 0
    st.destroy()


def test_a_step_of_more_ranks_than_pointers_places_its_chunks():
    """``ShardStep``'s received chunks of the 4-bit wire past 256 ranks: evenly
    spaced but for the own one, which lies in the send buffer, so the call gets
    as far as its launch (made only where there is no GPU to launch on)."""
    import torch
    from zero_sharded_state_amd.shard_step import ShardStep
    if torch.cuda.is_available():
        pytest.skip("a GPU is visible: the buffers here are the host's")
    for world, rank in ((300, 0), (300, 150), (300, 299), (257, 1)):
        st = ShardStep(world_size=world, rank=rank, threshold=0, ds_ids=[0, 1, 2], numels=[5000, 40000, 640], dtype="bf16",
                       prefetch_bucket_size=100000, reduce_bucket_size=41000, sub_group_size=1000, device="cpu",
                       reduce_path="coalesced", reduce_bits=4)
        for bi, (part, _, C, send, _) in enumerate(st.coalesced):
            at = [st.recv_chunk_ptr(bi, v) for v in range(world)]
            assert at[rank] == st.send_ptr(bi) + rank * C and len(set(at)) == world
            others = [v for v in range(world) if v != rank]
            assert all(at[v] - at[others[0]] == (v - others[0]) * C for v in others)
            assert max(at) + C <= st.xbuf.data_ptr() + st.xbuf.numel()
        for n, ids, grads, send, recv in st._x:
            code = zs.lib().zs3_reduce_scatter_coalesced_mx4(st.h, rank, st.dcode, zs.ZS3_PACK | zs.ZS3_REDUCE, n, ids, grads, send, recv,
                                                             st.grad.data_ptr(), None, zs.ZS3_ROUND_STOCHASTIC, 1, None)
            assert code == zs.ZS3_EHIP, zs.zs3_last_error()
        st.destroy()


@pytest.mark.parametrize("bits", [8, 32])
def test_a_changed_decay_reaches_the_next_step(bits, monkeypatch):
    """``ShardStep.adam`` is read at every step, its weight decay with the rest:
    changed in place or replaced, the lists carry the new one, and none for
    parameters in no_decay."""
    import dataclasses
    seen = []

    class Recorder:
        @staticmethod
        def zs3_adamw_tensors(dtype, grad, state_bits, n, tensors, scale, flag, hp, seed, stream):
            seen.extend((hp._obj.lr, tensors[i].id, tensors[i].weight_decay) for i in range(n))
            return zs.ZS3_OK

    from zero_sharded_state_amd.shard_step import AdamConfig
    st = _host_step(state_bits=bits, no_decay=[1], adam=AdamConfig())
    try:
        with monkeypatch.context() as m:
            m.setattr(zs, "lib", lambda: Recorder)
            for lr, wd in ((1e-3, 0.1), (2e-3, 0.3), (2e-3, 0.0), (1e-3, 0.2)):
                if wd == 0.2:
                    st.adam = dataclasses.replace(st.adam, lr=lr, weight_decay=wd)
                else:
                    st.adam.lr, st.adam.weight_decay = lr, wd
                seen.clear()
                st.adam_step(1, stream=0)
                assert sorted(seen) == [(lr, 0, wd), (lr, 1, 0.0)]
    finally:
        st.destroy()


def test_pack_with_reduce_refuses_every_overlap(layout):
    """With both bits the gradients, too, may not lie under what the reduce
    writes; received chunks may lie in the send buffer, at any rank."""
    import torch
    flat, slots = BASE + (8 << 20), BASE + (9 << 20)
    p = zs.zs3_layout_param(layout, 9)
    first = flat + 2 * p["shard_offset"]            # of what the reduce writes for a parameter
    for g in (first, first + 10, first + 2 * p["partition_size"] - 2):
        for grads in ([g, BASE + (2 << 20)], [BASE + (1 << 20), g]):
            _refused(zs.ZS3_EALIAS, "gradient overlaps", _scatter, layout, grads=grads, flat=flat)
    _refused(zs.ZS3_EALIAS, "gradient overlaps", _scatter, layout, grads=[BASE + (1 << 20), slots + 8], partials=slots)
    _refused(zs.ZS3_EALIAS, "gradient overlaps", _scatter, layout, grads=[slots - 2, BASE + (1 << 20)], partials=slots)
    if not torch.cuda.is_available():       # taken: they get as far as their launch
        _, size = zs.zs3_mx4_sizes(layout, [5, 9])
        for recv in ([BASE + size] * 4, [BASE + v * size for v in range(4)]):
            _refused(zs.ZS3_EHIP, "", _scatter, layout, recv=recv)
        # two gradients may share memory: they are read only
        _refused(zs.ZS3_EHIP, "", _scatter, layout, grads=[BASE + (1 << 20)] * 2)


def test_wire_seeds_do_not_repeat():
    """``ShardStep.wire_seed``: another one for every seed, step, rank and bucket,
    also where steps times ranks pass 16 bits, buckets do, or the seed passes
    32; where all fit, the fields lie side by side."""
    seen = {}
    for seed in (0, 1, 2, 3, (1 << 32) - 1, 1 << 32, (1 << 32) + 1, (1 << 63) + 5, -1):
        st = _host_step(seed=seed)
        try:
            st.N = 64
            for t in (1, 2, 1023, 1024, 1025, 2047, 2048, 65536, 1 << 20, 1 << 40):
                for st.rank in (0, 1, 63):
                    st.t = t
                    for bucket in (0, 1, 65535, 65536, 65537, 1 << 20):
                        s = st.wire_seed(bucket)
                        assert 0 <= s < 1 << 64
                        assert seen.setdefault(s, (seed, t, st.rank, bucket)) == (seed, t, st.rank, bucket)
                        count = t * 64 + st.rank
                        if 0 <= seed < 1 << 32 and count < 1 << 16 and bucket < 1 << 16:
                            assert s == (seed << 32) + (count << 16) + bucket
        finally:
            st.destroy()


def test_gather_timers_are_refused_with_the_4_bit_wire():
    """The 4-bit calls record no events: a timer's pair would be left to the next
    other launch.  Refused before anything runs, and the step does not count."""
    st = _host_step(gather_bits=4)
    pairs = []
    timer = lambda: pairs.append(1) or (None, None)     # noqa: E731
    try:
        with pytest.raises(ValueError, match="4-bit"):
            st.step(gather_timer=timer)
        with pytest.raises(ValueError, match="4-bit"):
            st.gather_pass(timer=timer)
        assert st.t == 0 and not pairs
    finally:
        st.destroy()


def test_an_eps_that_8_bit_states_refuse_is_refused_at_once():
    """What the list step would refuse in the first step, after its gathers."""
    from zero_sharded_state_amd.shard_step import AdamConfig
    for eps in (0.0, 1e-13, float("nan")):
        with pytest.raises(ValueError, match="eps"):
            _host_step(state_bits=8, adam=AdamConfig(eps=eps))
    for bits, eps in ((8, 1e-12), (32, 0.0)):
        _host_step(state_bits=bits, no_decay=[1], adam=AdamConfig(eps=eps)).destroy()
