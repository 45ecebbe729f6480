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


# ---------------------------------------------------------------- attention


def deep(made):
    """The same with a table that has room for 2^18 tokens: enough work by its bounds that long chunks go in units of many rows."""
    made = list(made)
    table = torch.full((made[3].shape[0], (1 << 18) // made[4].shape[2]), -1, dtype=torch.int32)
    table[:, : made[3].shape[1]] = made[3]
    made[3] = table
    return tuple(made)


def check_made(made, heads, kv_heads, dim, kind, cache, causal=True, window=0, scale=None):
    q, q_start, kv_len, table, k, v, ks, vs = made
    scale = dim ** -0.5 if scale is None else scale
    attn = llm.cbs_attn_create(llm.make_attn_desc(heads, kv_heads, dim, k.shape[2], dtype=KIND[kind], cache_dtype=KIND[cache], causal=causal, window=window, scale=scale,
                                                  max_seqs=table.shape[0]))
    out = base.run_attn(made, heads, kv_heads, dim, k.shape[2], kind, cache, attn=attn)
    want, mags, tops = ref.attention(q, q_start, kv_len, table, k, v, scale, causal, window, ks, vs)
    base.close(out, want, base.attn_bound(want, mags, tops, kind, dim, max(1, int(kv_len.max()))), "attention")
    return out


@pytest.mark.parametrize("kind,cache", base.PAIRS)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window", [2**31 - 1, 2**31 - 5, 2**31 - 200])
@pytest.mark.parametrize("new,kv", [([10, 6, 1], [4, 6, 0]), ([300, 150], [41, 149])])
def test_attn_window_of_all_there_can_be(kind, cache, causal, window, new, kv):
    """More new tokens than keys, and a window near 2^31: places before the first key, and the rows beside them, keep theirs."""
    made = base.make_attn(new, kv, 4, 2, 64, 16, kind, cache)
    check_made(made if len(new) == 3 else deep(made), 4, 2, 64, kind, cache, causal, window)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("which", ["key", "value", "both"])
@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("key", [70, 200, 300])
@pytest.mark.parametrize("new", [1, 40, 130])
def test_attn_nonfinite_steps_seen(bad, which, kind, key, new):
    """A step that is infinite or NaN, in a tile that all rows see whole (70, 200) and in one that some of them see in part (300):
    rows that do not see it stay as they are, and those that do have what the formula says of a NaN, and of an infinite step of values."""
    heads, dim, page, kv = 4, 64, 16, 310
    made = deep(base.make_attn([new], [kv], heads, 2, dim, page, kind, "i8", q_by=0.3))
    q, q_start, kv_len, table, k, v, ks, vs = made
    pg, o = int(table[0, key // page]), key % page
    v[pg, :, ::3, o] = 0  # codes of zero, whose value is NaN
    v[pg, :, 1::3, o] = 5
    v[pg, :, 2::3, o] = -9
    clean, mags, tops = ref.attention(q, q_start, kv_len, table, k, v, dim ** -0.5, True, 0, ks, vs)
    if which != "value":
        ks[pg, :, o] = bad
    if which != "key":
        vs[pg, :, o] = bad
    out = base.run_attn(made, heads, 2, dim, page, kind, "i8").double().cpu()
    bound = base.attn_bound(clean, mags, tops, kind, dim, kv)
    sees = torch.arange(new) + kv - new >= key
    if not sees.all():
        base.close(out[~sees], clean[~sees], bound[~sees], "rows that do not see it")
    out, want = out[sees], clean[sees].clone()
    if which == "value":  # a weight times 0, 5 or -9 times it
        want[..., ::3], want[..., 1::3], want[..., 2::3] = math.nan, 5 * bad, -9 * bad
        assert torch.equal(torch.isnan(out), torch.isnan(want)) and torch.equal(out.nan_to_num(0.0), want.nan_to_num(0.0))
    elif math.isnan(bad):
        assert torch.isnan(out).all()
