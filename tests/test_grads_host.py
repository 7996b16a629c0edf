"""The gradient-list entry points without a GPU: every refusal (arguments are checked
before any device work, so the addresses here are made up and never read)."""

import ctypes
import math
import os
import re
import shutil
import subprocess

import pytest

import zero_sharded_state_amd as zs

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BASE = 1 << 40
STEP = 1 << 24


def _refused(status, text, fn, *a, **k):
    with pytest.raises(zs.Zs3Error) as e:
        fn(*a, **k)
    assert e.value.status == status, e.value
    assert text in e.value.message, e.value.message


def _t(numel=100, at=BASE, dtype="bf16", **over):
    d = dict(numel=numel, grad=at, dtype=dtype, out=at + STEP, out_dtype="fp32")
    d.update(over)
    return d


def _args(**over):
    o = BASE << 2
    d = dict(kind=zs.ZS3_NORM_2, rank=0, world=2, sums=o, norm=o + 64, scale=o + 128, nonfinite=o + 132, tensor_norms=o + 4096,
             workspace=o + (1 << 20), workspace_bytes=1 << 20)
    d.update(over)
    return d


def _norm(tensors, **over):
    zs.zs3_grad_norm_tensors(tensors, _args(**over), stream=0)


def _clip(tensors, scale=BASE << 3, nonfinite=None):
    zs.zs3_clip_tensors(tensors, scale, nonfinite, stream=0)


def _acc(tensors, factor=1.0, first=False, norm=None):
    zs.zs3_accumulate_tensors(tensors, factor, first, norm=norm, stream=0)


def _fused(tensors, **over):
    _acc(tensors, norm=_args(**over))


def test_library_exports_every_declared_symbol():
    text = open(os.path.join(ROOT, "include", "zs3_grads.h")).read()
    syms = sorted(set(re.findall(r"ZS3_API\s+[\w\s\*]*?\b(zs3_\w+)\s*\(", text)))
    assert syms == sorted(zs.EXPORTS_GRADS) and all(hasattr(zs.lib(), s) for s in syms)


@pytest.mark.skipif(shutil.which("gcc") is None, reason="no gcc")
@pytest.mark.parametrize("lang", ["c99", "c++17"])
def test_header_is_plain_c(tmp_path, lang):
    """It compiles with warnings as errors, and its structs are laid out as the binding has them."""
    src = tmp_path / "t.c"
    src.write_text('''#include <stddef.h>
#include <stdio.h>
#include "zs3_grads.h"
int main(void) {
    int64_t b = 0;
    printf("%d %d %d %d\\n", (int)sizeof(zs3_grad_tensor), (int)offsetof(zs3_grad_tensor, shared),
           (int)sizeof(zs3_norm_args), (int)offsetof(zs3_norm_args, workspace_bytes));
    if (zs3_norm_workspace_bytes(0, NULL, &b) != ZS3_OK || b <= 0) return 1;
    return zs3_clip_tensors(0, NULL, NULL, NULL, NULL) == ZS3_EINVAL ? 0 : 2;
}
''')
    exe, pkg = str(tmp_path / "t"), os.path.join(ROOT, "zero_sharded_state_amd")
    cmd = ["gcc", "-std=c99", "-pedantic"] if lang == "c99" else ["g++", "-std=c++17", "-x", "c++"]
    cmd += ["-Wall", "-Wextra", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-x", "none", "-L", pkg, "-lzs3",
            f"-Wl,-rpath,{pkg}", "-o", exe]
    b = subprocess.run(cmd, capture_output=True, text=True)
    assert b.returncode == 0, b.stdout + b.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    t, a = zs.zs3_grad_tensor, zs.zs3_norm_args
    assert r.returncode == 0
    assert r.stdout.split() == [str(x) for x in (ctypes.sizeof(t), t.shared.offset, ctypes.sizeof(a), a.workspace_bytes.offset)]


def test_workspace_is_small():
    """About 50 KB for every 150 tensors, or 8 bytes for every 2048 elements."""
    one = zs.zs3_norm_workspace_bytes([_t()])
    assert 0 < one < 1 << 16 and one % 16 == 0 and zs.zs3_norm_workspace_bytes([]) <= one
    for n, numel in ((1000, 100), (1, 1 << 34), (4, 1 << 34), (300, 10**7)):
        got = zs.zs3_norm_workspace_bytes([_t(numel=numel)] * n)
        assert one < got < (n // 150 + 4) * (1 << 16) + n * (numel // 256 + 16)
    _refused(zs.ZS3_EINVAL, "numel", zs.zs3_norm_workspace_bytes, [_t(numel=-1)])
    assert zs.lib().zs3_norm_workspace_bytes(0, None, None) == zs.ZS3_EINVAL


@pytest.mark.parametrize("call", [_norm, _clip, _acc, _fused])
def test_list_refusals(call):
    for d in (0, 4, 7):
        _refused(zs.ZS3_EDTYPE, "dtype", call, [_t(dtype=d)])
    _refused(zs.ZS3_EINVAL, "numel", call, [_t(numel=-1)])
    _refused(zs.ZS3_EINVAL, "numel", call, [_t(numel=(1 << 34) + 1)])
    # nothing of a list is launched where a later tensor is refused
    _refused(zs.ZS3_EINVAL, "tensor 1: numel", call, [_t(), _t(at=2 * BASE, numel=1 << 36)])
    _refused(zs.ZS3_EINVAL, "grad is NULL", call, [_t(grad=0)])
    _refused(zs.ZS3_EINVAL, "grad is not aligned", call, [_t(grad=BASE + 1)])
    _refused(zs.ZS3_EINVAL, "grad is not aligned", call, [_t(grad=BASE + 2, dtype="fp32")])
    arr = zs.zs3_grad_tensor_list([_t()])
    arr[0].reserved = 1
    _refused(zs.ZS3_EINVAL, "reserved", call, arr)


@pytest.mark.parametrize("call", [_norm, _fused])
def test_norm_refusals(call):
    t = [_t()]
    for k in (0, 3):
        _refused(zs.ZS3_EINVAL, "kind", call, t, kind=k)
    _refused(zs.ZS3_EINVAL, "world", call, t, world=0)
    for r in (-1, 2):
        _refused(zs.ZS3_EINVAL, "rank", call, t, rank=r)
    for v in (0.0, -1.0, math.nan):
        _refused(zs.ZS3_EINVAL, "max_norm", call, t, max_norm=v)
    for v in (0.0, -1.0, math.nan, math.inf):
        _refused(zs.ZS3_EINVAL, "loss_scale", call, t, loss_scale=v)
    o = _args()
    for k, off in (("sums", 4), ("norm", 4), ("scale", 2), ("nonfinite", 2), ("tensor_norms", 4), ("workspace", 8)):
        _refused(zs.ZS3_EINVAL, k, call, t, **{k: o[k] + off})
        if k != "tensor_norms":
            _refused(zs.ZS3_EINVAL, "NULL", call, t, **{k: 0})
    need = zs.zs3_norm_workspace_bytes(t)
    _refused(zs.ZS3_EINVAL, "workspace has", call, t, workspace_bytes=need - 1)
    _refused(zs.ZS3_EINVAL, "workspace has", call, t, workspace_bytes=0)


@pytest.mark.parametrize("call", [_norm, _fused])
def test_norm_refuses_overlaps(call):
    t, o = [_t()], _args()
    outs = ("sums", "norm", "scale", "nonfinite", "tensor_norms", "workspace")
    for k in outs:
        _refused(zs.ZS3_EALIAS, "tensor 0", call, t, **{k: BASE + 192})         # the gradient's last 8 bytes
    _refused(zs.ZS3_EALIAS, "overlap", call, t, norm=o["sums"] + 16)            # world + 1 sums
    _refused(zs.ZS3_EALIAS, "overlap", call, t, scale=o["norm"] + 4)
    _refused(zs.ZS3_EALIAS, "overlap", call, t, nonfinite=o["scale"])
    _refused(zs.ZS3_EALIAS, "overlap", call, t, tensor_norms=o["sums"] + 8)
    _refused(zs.ZS3_EALIAS, "overlap", call, t, sums=o["workspace"] + 1024)


def test_norm_finalize_refusals():
    def call(**over):
        zs.zs3_norm_finalize(_args(**over), stream=0)
    for k, bad in (("kind", 0), ("world", 0), ("rank", 5), ("max_norm", 0.0), ("loss_scale", 0.0), ("sums", 0), ("norm", 0),
                   ("scale", 0), ("nonfinite", 0)):
        _refused(zs.ZS3_EINVAL, k if bad != 0 or k in ("kind", "world", "max_norm", "loss_scale") else "NULL", call, **{k: bad})
    _refused(zs.ZS3_EALIAS, "overlap", call, norm=_args()["sums"] + 8)
    assert zs.lib().zs3_norm_finalize(None, None) == zs.ZS3_EINVAL
    assert zs.lib().zs3_grad_norm_tensors(0, None, None, None) == zs.ZS3_EINVAL


def test_clip_refusals():
    far = BASE + (1 << 34)
    _refused(zs.ZS3_EDTYPE, "out_dtype", _clip, [_t(out_dtype=0)])
    _refused(zs.ZS3_EINVAL, "out is not aligned", _clip, [_t(out=BASE + STEP + 2)])
    _refused(zs.ZS3_EINVAL, "scale", _clip, [_t()], scale=0)
    _refused(zs.ZS3_EINVAL, "scale", _clip, [_t()], scale=BASE + 2)
    _refused(zs.ZS3_EINVAL, "nonfinite", _clip, [_t()], nonfinite=BASE + 2)
    _refused(zs.ZS3_EALIAS, "overlap", _clip, [_t(out=None), _t(out=None)])                    # the same tensor twice
    _refused(zs.ZS3_EALIAS, "overlap", _clip, [_t(out=BASE)])                                  # its own place in another type
    _refused(zs.ZS3_EALIAS, "overlap", _clip, [_t(out=BASE + 2, out_dtype="bf16")])            # its own place, shifted
    _refused(zs.ZS3_EALIAS, "overlap", _clip, [_t(), _t(at=far, out=BASE + 100, out_dtype="bf16")])
    _refused(zs.ZS3_EALIAS, "overlap", _clip, [_t(), _t(at=far, out=BASE + STEP + 396)])
    _refused(zs.ZS3_EALIAS, "scale", _clip, [_t(out=None)], scale=BASE + 196)
    _refused(zs.ZS3_EALIAS, "nonfinite", _clip, [_t(out=None)], nonfinite=BASE)
    f = zs.lib().zs3_clip_tensors
    assert f(1, None, BASE, None, None) == zs.ZS3_EINVAL
    assert f(-1, None, BASE, None, None) == zs.ZS3_EINVAL


def test_accumulate_refusals():
    for call in (_acc, _fused):
        for d in ("bf16", "fp16", 0):
            _refused(zs.ZS3_EDTYPE, "out_dtype", call, [_t(out_dtype=d)])
        _refused(zs.ZS3_EINVAL, "out is NULL", call, [_t(out=None)])
        _refused(zs.ZS3_EINVAL, "out is NULL or not", call, [_t(out=BASE + STEP + 2)])
        _refused(zs.ZS3_EALIAS, "overlap", call, [_t(), _t()])
        _refused(zs.ZS3_EALIAS, "overlap", call, [_t(dtype="fp32", out=BASE)])
        _refused(zs.ZS3_EALIAS, "overlap", call, [_t(out=BASE + 196)])
    for f in (math.inf, math.nan, 1e39):
        _refused(zs.ZS3_EINVAL, "factor", _acc, [_t()], factor=f)


def test_overlaps_are_found_in_any_order():
    """Random lists of apart ranges are taken, and refused once any two of them touch."""
    import random
    rng = random.Random(5)
    for _ in range(200):
        n = rng.randint(2, 12)
        sizes = [rng.randint(1, 50) for _ in range(n)]
        at, cells = BASE, []
        for s in sizes:                       # a gradient of 2 * s bytes and an accumulator of 4 * s, apart by a word or not at all
            cells.append([at, at + 2 * s + (2 * s) % 4])
            at = cells[-1][1] + 4 * s + rng.choice([0, 4, 64])
        order = list(range(n))
        rng.shuffle(order)
        i, j = rng.sample(range(n), 2)
        for a_of, b_of in ((0, 1), (1, 1), (1, 0)):       # make tensor i's one array reach into j's other
            moved = [list(c) for c in cells]
            moved[i][a_of] = cells[j][b_of] + (4 * sizes[j] - 4 if b_of else 2 * ((sizes[j] - 1) // 2) // 4 * 4)
            ts = [_t(numel=sizes[k], grad=moved[k][0], out=moved[k][1]) for k in order]
            _refused(zs.ZS3_EALIAS, "overlap", _acc, ts)


def test_tensors_have_to_fit_what_is_said_of_them():
    """Lists and arguments made of torch tensors (never read here)."""
    import torch
    g, a = torch.zeros(10, dtype=torch.bfloat16), torch.zeros(10)
    ok = zs.zs3_grad_tensor_list([dict(numel=10, grad=g, dtype="bf16", out=a, out_dtype="fp32"), dict(numel=9, grad=g, dtype="bf16")])
    assert (ok[0].grad, ok[0].out, ok[1].out, ok[1].out_dtype) == (g.data_ptr(), a.data_ptr(), None, zs.ZS3_BF16)
    for bad, text in ((dict(numel=10, grad=a, dtype="bf16"), "grad has 4-byte"), (dict(numel=11, grad=g, dtype="bf16"), "11 elements"),
                      (dict(numel=10, grad=g, dtype="bf16", out=a), "out has 4-byte"),
                      (dict(numel=5, grad=g[::2], dtype="bf16"), "one behind the other"),
                      (dict(numel=10, grad=g, dtype="bf16", out=a[:9], out_dtype="fp32"), "10 elements")):
        with pytest.raises(ValueError, match=text):
            zs.zs3_grad_tensor_list([bad])
    d, f, i = torch.zeros(4, dtype=torch.float64), torch.zeros(1), torch.zeros(1, dtype=torch.int32)
    args = dict(sums=d[:3], world=2, norm=d[3:], scale=f, nonfinite=i, workspace=torch.zeros(64, dtype=torch.uint8))
    assert zs.zs3_norm_args_of(**args).workspace_bytes == 64
    for k, bad in (("sums", d[:2]), ("sums", f), ("norm", f), ("scale", d), ("nonfinite", d), ("tensor_norms", f)):
        with pytest.raises(ValueError, match=k):
            zs.zs3_norm_args_of(**dict(args, **{k: bad}))


# --------------------------------------------------------------- ShardStep

def _host_step(**k):
    from zero_sharded_state_amd.shard_step import ShardStep
    return ShardStep(world_size=2, rank=1, threshold=0, ds_ids=[0, 1], numels=[64, 65], dtype="bf16", prefetch_bucket_size=1000,
                     reduce_bucket_size=1000, sub_group_size=1000, device="cpu", **k)


def test_shard_step_takes_micro_batches_in_order():
    st = _host_step(accumulate=3, gather_bits=4)
    assert st.listed and st.acc.numel() == st.S
    with pytest.raises(ValueError, match="0 of 2 micro-batches"):
        st.step()
    with pytest.raises(ValueError, match="16-bit wire"):
        st.micro_step(trace_pass=object())
    assert (st.t, st.micro) == (0, 0)
    st.micro = 2
    with pytest.raises(ValueError, match="micro-batch 3 of 3"):
        st.micro_step()
    with pytest.raises(ValueError, match="no events"):
        st.step(gather_timer=object())
    assert (st.t, st.micro) == (0, 2)
    st.destroy()
    one = _host_step()
    assert one.acc is None and not one.listed
    with pytest.raises(ValueError, match="micro-batch 1 of 1"):
        one.micro_step()
    with pytest.raises(ValueError, match="no accumulators"):
        one.accumulate_grads()
    one.destroy()


def test_shard_step_refuses_accumulation_it_cannot_do():
    for k in (0, -1):
        with pytest.raises(ValueError, match="accumulate"):
            _host_step(accumulate=k)
    with pytest.raises(TypeError):
        _host_step(accumulate=1.5)
    with pytest.raises(ValueError, match="16-bit gradients"):
        _host_step(accumulate=2, offload=True)


def test_shard_step_seeds_do_not_repeat_over_micro_batches():
    """One micro-batch a step has the seeds it had; several have one each."""
    seen = set()
    for rank in (0, 1):
        from zero_sharded_state_amd.shard_step import ShardStep
        st = ShardStep(world_size=2, rank=rank, threshold=0, ds_ids=[0], numels=[64], dtype="bf16", prefetch_bucket_size=1000,
                       reduce_bucket_size=1000, sub_group_size=1000, device="cpu", reduce_path="coalesced", reduce_bits=4, seed=7,
                       accumulate=3)
        for st.t in range(1, 6):
            for st.micro in range(3):
                for bucket in range(4):
                    seen.add(st.wire_seed(bucket))
        st.destroy()
    assert len(seen) == 2 * 5 * 3 * 4
    st = _host_step(seed=7)
    st.t = 9
    assert st.wire_seed(3) == 7 << 32 | (9 * 2 + 1) << 16 | 3
    st.destroy()


def test_shard_step_counts_the_bytes_of_every_micro_batch():
    one, four = _host_step(), _host_step(accumulate=4)
    a, b = one.algorithmic_bytes(), four.algorithmic_bytes()
    own = one.own_real
    assert b["unpack"] == 4 * a["unpack"] and b["reduce_scatter"] == 4 * a["reduce_scatter"]
    assert b["accumulate"] == 4 * (2 + 4) * own + 3 * 4 * own
    assert b["grad_norm"] == 4 * own and b["adam"] == a["adam"] + 2 * own
    one.destroy(), four.destroy()


class _Recorder:
    """Takes the library's place: what each call of a gradient list carries."""

    def __init__(self):
        self.calls, self.real = [], zs.lib()

    def __getattr__(self, name):
        if name.startswith("zs3_layout") or name in ("zs3_norm_workspace_bytes", "zs3_last_error"):
            return getattr(self.real, name)

        def call(*args):
            self.calls.append((name, args))
            return zs.ZS3_OK
        return call


@pytest.mark.parametrize("accumulate", [1, 3])
def test_single_norms_use_buffers_that_the_step_keeps(accumulate, monkeypatch):
    """Sums and workspace of ``grad_norms`` are the step's own from its start (a buffer made or
    dropped at the call belongs to another stream than the kernel's)."""
    import torch
    st = _host_step(accumulate=accumulate)
    held = [(t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()) for t in vars(st).values() if torch.is_tensor(t)]
    rec = _Recorder()
    with monkeypatch.context() as m:
        m.setattr(zs, "lib", lambda: rec)
        for inf in (False, True):
            each = st.grad_norms(inf=inf, stream=0)
    for name, (n, _, args, _) in rec.calls:
        a = args._obj
        assert name == "zs3_grad_norm_tensors" and n == each.numel() == 2
        for p, size in ((a.sums, 16), (a.workspace, a.workspace_bytes)):
            assert any(lo <= p and p + size <= hi for lo, hi in held)
    assert a.tensor_norms == each.data_ptr() and len(rec.calls) == 2
    assert a.sums != st.sumsq.data_ptr()
    st.destroy()


class _NoStream:
    """What the recorder's calls run on."""
    cuda_stream = 0


@pytest.mark.parametrize("path", ["phases", "micro_step", "mixed"])
def test_every_way_through_a_step_counts_its_micro_batches(path, monkeypatch):
    """Two steps without AdamW, by phases, by ``micro_step`` and ``gradient_step``, and
    by both in turn: the first micro-batch of each overwrites, the others add, the norm comes once, seeds
    of the 4-bit wire do not repeat, and what takes the whole sum waits for it."""
    from zero_sharded_state_amd.shard_step import ShardStep
    st = ShardStep(world_size=2, rank=1, threshold=0, ds_ids=[0, 1], numels=[64, 65], dtype="bf16", prefetch_bucket_size=1000,
                   reduce_bucket_size=1000, sub_group_size=1000, device="cpu", reduce_path="coalesced", reduce_bits=4, accumulate=3,
                   fuse_norm=True)
    on = _NoStream()
    rec = _Recorder()

    def by_phases(last):
        st.gather_pass(on)
        st.reduce_scatter(on)
        st.accumulate_grads(on, norm=last)
    with monkeypatch.context() as m:
        m.setattr(zs, "lib", lambda: rec)
        for t in (1, 2, 3, 4):
            for k in range(3):
                if path == "phases" or path == "mixed" and (t + k) % 2:
                    by_phases(k == 2)
                else:
                    (st.gradient_step if k == 2 else st.micro_step)(on)
                assert (st.t, st.micro) == (t, (k + 1) % 3)
                if k < 2:
                    for call in (st.clip_grads, lambda **a: st.adam_step(1, **a)):
                        with pytest.raises(ValueError, match=f"{k + 1} of 3 micro-batches"):
                            call(stream=0)
            st.clip_grads(stream=0)
        st.micro_step(on)
        with pytest.raises(ValueError, match="1 of 2 micro-batches before"):
            st.gradient_step(on)
        st.micro_step(on)
        with pytest.raises(ValueError, match="micro-batch 3 of 3"):
            st.micro_step(on)
        st.step(on)
        assert (st.t, st.micro) == (5, 0)
    acc = [a for name, a in rec.calls if name == "zs3_accumulate_tensors"]
    assert [a[3] for a in acc] == [1, 0, 0] * 5 and all(a[2] == 1 / 3 for a in acc)
    assert [a[4] is not None for a in acc] == [False, False, True] * 5
    seeds = [a[-2] for name, a in rec.calls if name == "zs3_reduce_scatter_coalesced_mx4"]
    assert len(seeds) == len(set(seeds)) == 15 * len(st._x)
    order = [name for name, _ in rec.calls if name in ("zs3_clip_tensors", "zs3_adamw_tensors")]
    assert order == ["zs3_clip_tensors"] * 4 + ["zs3_adamw_tensors"] * len(st._lists)
    st.destroy()


def test_a_step_without_accumulators_stops_before_adamw(monkeypatch):
    st, rec = _host_step(), _Recorder()
    phases = []
    with monkeypatch.context() as m:
        m.setattr(zs, "lib", lambda: rec)
        st.gradient_step(_NoStream(), on_phase=phases.append)
        st.clip_grads(stream=0)
        st.step(_NoStream())
    assert phases == ["gather_fwd", "gather_bwd", "reduce_scatter", "grad_norm", None] and st.t == 2
    names = [name for name, _ in rec.calls]
    assert names.count("zs3_grad_norm") == 2 and names.count("zs3_adam_step") == len(st.sub_groups)
    assert names.index("zs3_clip_tensors") < names.index("zs3_adam_step")
    st.destroy()


def test_what_a_norm_writes_has_to_hold_it(monkeypatch):
    """One place for each tensor's norm, and a workspace of the bytes it counts (the library is not reached)."""
    import torch
    rec = _Recorder()
    monkeypatch.setattr(zs, "lib", lambda: rec)
    each = torch.zeros(3, dtype=torch.float64)
    for made in (lambda d: d, lambda d: zs.zs3_norm_args_of(**d)):
        for call in (zs.zs3_grad_norm_tensors, lambda ts, a, stream: zs.zs3_accumulate_tensors(ts, norm=a, stream=stream)):
            for ts in ([_t()] * 4, zs.zs3_grad_tensor_list([_t()] * 4)):
                with pytest.raises(ValueError, match="tensor_norms has 3 elements, the list 4"):
                    call(ts, made(_args(tensor_norms=each)), stream=0)
            with pytest.raises(ValueError, match="tensor_norms has 0 elements"):
                call([_t()], made(_args(tensor_norms=each[:0])), stream=0)
    assert not rec.calls
    for call, a in ((lambda a: zs.zs3_grad_norm_tensors([_t()] * 3, a, stream=0), each), (lambda a: zs.zs3_norm_finalize(a, stream=0), each[:0])):
        with pytest.raises(ValueError, match="host memory"):        # long enough
            call(_args(tensor_norms=a))
    for bad in (torch.zeros(64, dtype=torch.uint8)[::2], torch.zeros(1, dtype=torch.uint8).expand(1 << 20)):
        with pytest.raises(ValueError, match="workspace"):
            zs.zs3_norm_args_of(**dict(_args(workspace=bad), workspace_bytes=None))


def test_tensors_have_to_be_of_the_type_that_is_said(monkeypatch):
    """A type of the same width is another one; 16-bit values may come as their bits."""
    import torch
    rec = _Recorder()
    monkeypatch.setattr(zs, "lib", lambda: rec)
    t = {d: torch.zeros(8, dtype=getattr(torch, d)) for d in ("float16", "bfloat16", "float32", "float64", "int16", "int32", "int64", "bool")}
    for said, good in (("fp16", ("float16", "int16")), ("bf16", ("bfloat16", "int16")), ("fp32", ("float32",))):
        for name, x in t.items():
            for d, what in ((dict(numel=8, grad=x, dtype=said), "tensor 1: grad"), (dict(_t(), out=x, numel=8, out_dtype=said), "tensor 1: out")):
                if name in good:
                    zs.zs3_grad_tensor_list([_t(), d])
                    continue
                with pytest.raises(ValueError, match=what):
                    zs.zs3_grad_tensor_list([_t(), d])
    for k, good in (("sums", "float64"), ("norm", "float64"), ("tensor_norms", "float64"), ("scale", "float32"), ("nonfinite", "int32")):
        for name, x in t.items():
            if name == good:
                zs.zs3_norm_args_of(**_args(**{k: x}))
                continue
            with pytest.raises(ValueError, match=k):
                zs.zs3_norm_args_of(**_args(**{k: x}))
    # a norm's own double as the scale, a flag of one byte, and neither
    for scale, flag, what in ((t["float64"], None, "scale"), (t["bfloat16"], None, "scale"), (BASE, t["bool"], "nonfinite"),
                              (BASE, t["float32"], "nonfinite"), (t["float32"][:0], None, "scale"), (BASE, t["int32"][:0], "nonfinite")):
        with pytest.raises(ValueError, match=what):
            zs.zs3_clip_tensors([_t()], scale, flag, stream=0)
    assert not rec.calls


class _On:
    """A tensor's face, on a device that is not there."""

    def __init__(self, device, dtype, pinned=False, n=16):
        import torch
        self.device, self.dtype, self.pinned, self.n = device, getattr(torch, dtype), pinned, n

    def get_device(self):
        return self.device

    def is_pinned(self):
        return self.pinned

    def is_contiguous(self):
        return True

    def numel(self):
        return self.n

    def element_size(self):
        return self.dtype.itemsize

    def data_ptr(self):
        return BASE + 64 * (self.device + 2) + (1 << 30) * id(self) % (1 << 36) // 64 * 64


def test_tensors_have_to_be_on_the_device_of_the_call(monkeypatch):
    """Host memory and another GPU's do not reach a launch; addresses and pinned memory are the caller's word."""
    rec = _Recorder()
    monkeypatch.setattr(zs, "lib", lambda: rec)
    monkeypatch.setattr(zs, "_device", lambda: 1, raising=False)
    calls = (lambda ts, **a: zs.zs3_grad_norm_tensors(ts, _args(**a), stream=0),
             lambda ts, **a: zs.zs3_accumulate_tensors(ts, norm=_args(**a), stream=0),
             lambda ts, scale=BASE, nonfinite=None, **a: zs.zs3_clip_tensors(ts, scale, nonfinite, stream=0))
    made = dict(sums="float64", norm="float64", scale="float32", nonfinite="int32", tensor_norms="float64", workspace="uint8")
    for device, text in ((-1, "host memory in a call on the GPU"), (0, "cuda:0 in a call on cuda:1")):
        g, a = _On(device, "bfloat16"), _On(device, "float32")
        for call in calls:
            for d in (dict(grad=g), dict(out=a)):
                for ts in ([_t(numel=16, **d)], zs.zs3_grad_tensor_list([_t(), _t(numel=16, **d)])):
                    with pytest.raises(ValueError, match=text):
                        call(ts)
            for k, dtype in made.items():
                if call is calls[2] and k not in ("scale", "nonfinite"):
                    continue
                with pytest.raises(ValueError, match=text):
                    call([_t()], **dict({k: _On(device, dtype)}, **({"workspace_bytes": 64} if k == "workspace" else {})))
        with pytest.raises(ValueError, match=text):
            zs.zs3_norm_finalize(_args(scale=_On(device, "float32")), stream=0)
    assert not rec.calls
    with pytest.raises(ValueError, match="more than one device: host memory, cuda:1"):
        zs.zs3_grad_tensor_list([_t(numel=16, grad=_On(1, "bfloat16")), _t(numel=16, grad=_On(-1, "bfloat16"))])
    with pytest.raises(ValueError, match="more than one device: cuda:0, cuda:1"):
        zs.zs3_norm_args_of(**_args(sums=_On(0, "float64"), scale=_On(1, "float32")))
    for call in calls:
        call([_t(numel=16, grad=_On(1, "bfloat16"), out=_On(-1, "float32", pinned=True))], scale=_On(1, "float32"), nonfinite=_On(-1, "int32", True))
        call([_t()])
    assert len(rec.calls) == 6


@pytest.mark.parametrize("call", [_norm, _fused, lambda t, **a: zs.zs3_norm_finalize(_args(**a), stream=0)])
def test_a_loss_scale_whose_reciprocal_is_infinite_is_refused(call):
    """The scale of finite gradients is finite wherever the flag is 0: 1 / loss_scale rounds to at most the largest float."""
    for v in (5e-324, 1e-300, 1e-40, 2.0 ** -128 * (1 - 2.0 ** -20)):
        assert 1.0 / v >= 2.0 ** 128
        _refused(zs.ZS3_EINVAL, "loss_scale", call, [_t()], loss_scale=v)
    # the next larger ones get as far as the argument that is wrong besides
    for v in (2.0 ** -128 * (1 + 2.0 ** -20), 1e-30):
        _refused(zs.ZS3_EINVAL, "sums", call, [_t()], loss_scale=v, sums=0)


def test_the_norm_of_the_sum_can_wait_for_the_other_ranks(monkeypatch):
    st, rec = _host_step(accumulate=2), _Recorder()
    with monkeypatch.context() as m:
        m.setattr(zs, "lib", lambda: rec)
        st.accumulate_grads(stream=0)
        st.accumulate_grads(stream=0, norm=True, finalize=False)
        st.finalize_norm(stream=0)
        st.accumulate_grads(stream=0, norm=True)
    acc = [a[4] for name, a in rec.calls if name == "zs3_accumulate_tensors"]
    assert acc[0] is None and [a._obj.finalize for a in acc[1:]] == [0, 1]
    (end,) = [a[0]._obj for name, a in rec.calls if name == "zs3_norm_finalize"]
    assert (end.sums, end.norm, end.rank, end.world) == (st.sumsq.data_ptr(), st.norm_ptr, 1, 2)
    st.destroy()
