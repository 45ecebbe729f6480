"""GPU: the decoder-step operators at the ends of what their arguments may say: groups, windows and sizes near the end of 31 bits,
infinities in the steps of a cache, empty caches.  Definition and bounds as in test_gpu_llm.py."""
import math

import pytest
import torch

import llm_reference as ref
import test_gpu_llm as base

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    llm, KIND = base.llm, base.KIND


# ---------------------------------------------------------------- 4-bit linear


@pytest.mark.parametrize("kind", ["bf16", "f16", "i8", "f32"])
@pytest.mark.parametrize("rows,k", [(1, 4096), (5, 40), (33, 1024), (33, 1021)])
@pytest.mark.parametrize("group", [2**31 - 128, 1 << 30, 1 << 24])
def test_w4_group_longer_than_k(kind, rows, k, group):
    """One group, whatever its length: the same bits as with a group that ends where k does."""
    g = base.gen(group % 1000 + k)
    n = 48
    packed = torch.randint(0, 256, (n, (k + 31) // 32 * 16), generator=g, dtype=torch.uint8).cuda()
    scales, zeros = (0.5 + torch.rand(1, n, generator=g)).half().cuda(), torch.randint(0, 16, (1, n), generator=g, dtype=torch.uint8).cuda()
    x = torch.randint(-128, 128, (rows, k), generator=g, dtype=torch.int8).cuda() if kind == "i8" else base.normal(g, rows, k, kind=kind).cuda()
    step = torch.rand(rows, generator=g).cuda() if kind == "i8" else None
    out = []
    for length in (group, (k + 127) // 128 * 128):
        out.append(torch.full((rows, n), math.nan, device="cuda"))
        llm.cbs_w4_linear(llm.make_w4_desc(k, n, length, dtype=KIND[kind], out_dtype=llm.CBS_F32), x, packed, scales, out[-1], zeros=zeros, x_scale=step)
    assert torch.isfinite(out[0]).all() and torch.equal(*out)
