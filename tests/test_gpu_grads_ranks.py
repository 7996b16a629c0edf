"""GPU: ranks that hold the same sums end a norm with the same bits, whichever rank they are and
whichever kernel ends it: otherwise their clip scales, and with them the
parameters that every rank holds whole, would part."""

import math
import struct

import numpy as np
import pytest

import zero_sharded_state_amd as zs
from gpu_util import note, require_gpu
from test_gpu_grads import KINDS

pytestmark = pytest.mark.gpu


def _bits(x):
    return struct.pack("<d", x).hex()


# elements behind the one that counts: zeros, which add nothing to any sum.  One workgroup, several, joined
# by the accumulation's last kernel, and by its many
@pytest.mark.parametrize("zeros,fused", [(0, False), (300_000, False), (300_000, True), (40_000_000, True)])
@pytest.mark.parametrize("world", [2, 3, 8, 63, 64, 65, 200])
def test_every_rank_ends_with_the_same_bits(world, zeros, fused):
    import torch
    require_gpu()
    note(f"{world} ranks, {zeros} zeros, fused {fused}")
    rng = np.random.default_rng(world)
    # squares of fp32 values are exact; magnitudes apart, so that another order of additions rounds elsewhere
    x = (rng.standard_normal(world + 1) * 10.0 ** rng.uniform(-3, 3, world + 1)).astype(np.float32)
    x[np.abs(x) < 1e-20] = 1.0
    for kind in ("2", "inf"):
        s = x.astype(np.float64) ** 2 if kind == "2" else np.abs(x).astype(np.float64)
        data = torch.zeros(zeros + 66, device="cuda")
        acc = torch.zeros_like(data) if fused else None
        base = dict(numel=zeros + 1, grad=data[:zeros + 1], dtype="fp32", out_dtype="fp32", **({"out": acc[:zeros + 1]} if fused else {}))
        shared = dict(numel=1, grad=data[zeros + 65:], dtype="fp32", shared=True, out_dtype="fp32", **({"out": acc[zeros + 65:]} if fused else {}))
        arr = zs.zs3_grad_tensor_list([base, shared])
        ws = torch.zeros(zs.zs3_norm_workspace_bytes(arr), dtype=torch.uint8, device="cuda")
        sums, norm = torch.zeros(world + 1, dtype=torch.float64, device="cuda"), torch.zeros(1, dtype=torch.float64, device="cuda")
        scale, flag = torch.zeros(1, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        seen = set()
        for rank in sorted({0, 1, world // 2, world - 1}):
            a = zs.zs3_norm_args_of(kind=KINDS[kind], rank=rank, world=world, sums=sums, norm=norm, scale=scale, nonfinite=flag, workspace=ws)
            data[0], data[zeros + 65] = float(x[rank]), float(x[world])
            for alone in (False, True):
                want = torch.from_numpy(s).cuda()
                sums.copy_(want)
                if not alone:
                    sums[rank], sums[world] = -1.0, -1.0
                    if fused:
                        zs.zs3_accumulate_tensors(arr, 1.0, first=True, norm=a)
                    else:
                        zs.zs3_grad_norm_tensors(arr, a)
                else:
                    zs.zs3_norm_finalize(a)
                torch.cuda.synchronize()
                assert torch.equal(sums, want) and int(flag) == 0
                seen.add((_bits(float(norm)), _bits(float(scale))))
        assert len(seen) == 1, (kind, seen)
        got = struct.unpack("<d", bytes.fromhex(next(iter(seen))[0]))[0]
        exact = math.sqrt(math.fsum(s)) if kind == "2" else max(s)
        # world + 1 positive terms in binary64, then a root
        assert abs(got - exact) <= ((world + 2) * 2.0 ** -53 * exact if kind == "2" else 0.0)
