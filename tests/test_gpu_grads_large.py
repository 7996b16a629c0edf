"""GPU: additions to accumulators of hundreds of millions of elements in one launch, and past
2^31 of them.  Small whole numbers: every product, sum and sum of squares is exact in
any order, and every element is compared."""

import gc
import math

import pytest

import zero_sharded_state_amd as zs
from gpu_util import note, require_gpu
from test_gpu_grads import Norm

pytestmark = pytest.mark.gpu
CHUNK = 1 << 28


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()
    yield
    import torch
    gc.collect()
    torch.cuda.empty_cache()


def _ints(n, seed, dtype, gap):
    """n whole numbers of -8 .. 8 between `gap` elements of 99 on either side."""
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.full((n + 2 * gap,), 99.0, dtype=dtype, device="cuda")
    for i in range(0, n, CHUNK):
        m = min(CHUNK, n - i)
        x[gap + i:gap + i + m] = torch.randint(-8, 9, (m,), dtype=torch.int8, device="cuda", generator=g)
    return x


@pytest.mark.parametrize("kind", [None, "2", "inf"])
@pytest.mark.parametrize("sizes", [(211_000_003,), (400_001,) * 530, (5, 190_000_001, 33, 45_000_002)], ids=["one", "many", "mixed"])
def test_large_additions(sizes, kind):
    _add(sizes, kind)


@pytest.mark.parametrize("kind", [None, "2"])
def test_additions_past_32_bits(kind):
    _add((7, (1 << 31) + 4099, 12), kind)


def _add(sizes, kind):
    import torch
    note(f"{len(sizes)} tensors, {sum(sizes)} elements added, norm {kind}")
    total, gap = sum(sizes), 129
    g, acc = _ints(total, 1, torch.bfloat16, gap), _ints(total, 2, torch.float32, gap)
    was = acc.clone()
    starts = [0]
    for n in sizes:
        starts.append(starts[-1] + n)
    entries = [dict(numel=n, grad=g.data_ptr() + 2 * (gap + s), dtype="bf16", out=acc.data_ptr() + 4 * (gap + s), out_dtype="fp32",
                    shared=i % 3 == 2) for i, (n, s) in enumerate(zip(sizes, starts))]
    norm = Norm(entries, kind=kind, max_norm=math.inf) if kind else None
    zs.zs3_accumulate_tensors(entries, 2.0, first=False, norm=norm.args if norm else None)
    torch.cuda.synchronize()
    assert bool((acc[:gap] == 99).all()) and bool((acc[gap + total:] == 99).all())
    for i in range(gap, gap + total, CHUNK):
        j = min(i + CHUNK, gap + total)
        assert torch.equal(acc[i:j], was[i:j] + 2.0 * g[i:j].float()), i
    if kind is None:
        return
    each = []
    for n, s in zip(sizes, starts):
        parts = [acc[gap + i:gap + min(i + CHUNK, s + n)] for i in range(s, s + n, CHUNK)]
        each.append(sum(int(p.double().square().sum()) for p in parts) if kind == "2" else max(float(p.abs().max()) for p in parts))
    join = sum if kind == "2" else (lambda v: max(v, default=0.0))
    want = [float(join([e for i, e in enumerate(each) if (i % 3 == 2) == second])) for second in (False, True)]
    got = norm.got()
    assert got["sums"].tolist() == want and got["flag"] == 0
    assert got["norm"] == (math.sqrt(want[0] + want[1]) if kind == "2" else max(want))
    for e, x in zip(each, got["each"]):
        assert abs(x - (math.sqrt(e) if kind == "2" else e)) <= (2.0 ** -52 * x if kind == "2" else 0.0)
