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



@pytest.mark.parametrize("rows,k", [(1, 4096), (3, 250), (16, 512)])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("by", [2.0 ** 95, 2.0 ** 113])
def test_w4_large_bfloat16(rows, k, zeros, by):
    """Inputs near the type's end, whose weighted sum 32 bits hold, and rows of other sizes beside them."""
    g = base.gen(k)
    n, group = 50, 64
    packed = torch.randint(0, 256, (n, (k + 31) // 32 * 16), generator=g, dtype=torch.uint8)
    sc = (0.5 + torch.rand(-(-k // group), n, generator=g)) * 2.0 ** -12
    z = torch.randint(0, 16, sc.shape, generator=g, dtype=torch.uint8) if zeros else None
    x = base.normal(g, rows, k, kind="bf16", by=by)
    x[rows // 2] = base.normal(g, k, kind="bf16")
    x[0, k // 2] = 2.0 ** 126
    out = torch.full((rows, n), math.nan, device="cuda")
    llm.cbs_w4_linear(llm.make_w4_desc(k, n, group, out_dtype=llm.CBS_F32, scale_dtype=llm.CBS_F32), x.cuda(), packed.cuda(), sc.cuda(), out, zeros=z.cuda() if zeros else None)
    y, mag = ref.w4_linear(x, packed, sc, group, z)
    _, sums = ref.w4_linear(x.abs(), packed, sc, group, torch.zeros_like(sc, dtype=torch.uint8))
    base.close(out, y, (mag + 2 * sums) * (k + sc.shape[0] + 4) * base.U32 + y.abs() * base.U32, "large")


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
@pytest.mark.parametrize("window", [2**31 - 1, 2**31 - 200])
@pytest.mark.parametrize("new,kv", [([10, 6, 1], [4, 6, 0]), ([300, 150], [41, 149])])
def test_attn_window_of_all_there_can_be(kind, cache, causal, window, new, kv):
    """More new tokens than keys, and a window near 2^31: places before the first key, and the rows beside them, keep theirs."""
    made = base.make_attn(new, kv, 4, 2, 64, 16, kind, cache)
    check_made(made if len(new) == 3 else deep(made), 4, 2, 64, kind, cache, causal, window)


@pytest.mark.parametrize("bad,which", [(math.nan, "key"), (math.nan, "value"), (math.inf, "value"), (-math.inf, "both")])
@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("key", [200, 300])
@pytest.mark.parametrize("new", [1, 40, 130])
def test_attn_nonfinite_steps_seen(bad, which, kind, key, new):
    """A step that is infinite or NaN, in a tile that all rows see whole (200) and in one that some of them see in part (300):
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


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("new,max_kv", [(1, 1), (1, None), (20, 1), (150, None), (4800, 500)])
@pytest.mark.parametrize("drop,logn", [(26, 18), (22, 18), (29, 20)])
def test_attn_many_small_weights(kind, new, max_kv, drop, logn):
    """2^18 (2^20) keys of a weight that is 2^-26 (2^-22, 2^-29) of that of four keys before them, whose values are zero: all of the
    output comes from the small ones.  Each is off by its rounding to 16 bits: half a step, which of a float16 weight of 2^-29
    taken 2^7 times is 2^-25 of 2^-22.  max_kv: the keys in one range, or in many."""
    heads, dim, page, many = 2, 64, 64, 1 << logn
    q = torch.zeros(new, heads, dim, dtype=base.TYPES[kind])
    q[..., 0] = 8.0
    k, v = torch.zeros(2, 1, page, dim, dtype=base.TYPES[kind]), torch.ones(2, 1, dim, page, dtype=base.TYPES[kind])
    k[1, 0, :, 0], v[1] = -100.0, 0.0
    k[1, 0, 5, 0] = k[1, 0, 37, 0] = 4.0
    scale = drop * math.log(2) / (8 * 4)
    table = torch.zeros(1, 2 + many // page, dtype=torch.int32)  # one page for all of the small ones
    table[0, :2] = 1
    made = (q, torch.tensor([0, new], dtype=torch.int32), torch.tensor([many + 2 * page], dtype=torch.int32), table, k, v, None, None)
    attn = llm.cbs_attn_create(llm.make_attn_desc(heads, 1, dim, page, dtype=KIND[kind], cache_dtype=KIND[kind], causal=False, scale=scale))
    out = base.run_attn(made, heads, 1, dim, page, kind, kind, attn=attn, max_kv=max_kv)
    one = math.exp(-8 * 4 * scale)
    want = torch.full(out.shape, many * one / (4 + many * one), dtype=torch.float64)
    rel, _ = base.half_step(base.TYPES[kind])
    weight = rel if kind == "bf16" else max(rel, 2.0 ** -25 / 2.0 ** (7 - drop))
    # a weight's rounding, its score's (drop times 8 steps of 32 bits), the two sums' (all keys, one after the other, each addition half
    # a step: the terms are equal, so roundings may agree)
    base.close(out, want, want * (rel + weight + (8 * drop + many) * base.U32), "small weights")


def test_attn_most_rows_there_can_be():
    """2^31 - 32768 rows of one sequence (69 GB of outputs): the rows of a block past the last would begin beyond 31 bits."""
    heads, tokens, dim, page = 65535, 32768, 16, 16
    q = torch.ones(1, 1, dim, dtype=torch.bfloat16, device="cuda").expand(tokens, heads, dim)
    k, v, ks, vs = base.kv_buffers(1, 1, dim, page, "i8", fill=1)
    v[0, 0, :, 0] = torch.arange(1, dim + 1, dtype=torch.int8, device="cuda")
    vs.fill_(1.0)
    attn = llm.cbs_attn_create(llm.make_attn_desc(heads, 1, dim, page, causal=False))
    out = torch.full((tokens, heads, dim), 77, dtype=torch.bfloat16, device="cuda")
    starts, one, table = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, tokens], [1], [[0]]))
    llm.cbs_attn_run(attn, q, starts, one, table, k, v, out, ks, vs, max_new=1)
    want = v[0, 0, :, 0].to(out.dtype)
    for part in out.split(1024):
        assert (part == want).all()



@pytest.mark.parametrize("kind,cache", base.PAIRS)
@pytest.mark.parametrize("scale", [-0.125, 0.0, 3.0])
@pytest.mark.parametrize("new,kv,window", [([1, 40], [70, 300], 0), ([140, 9], [300, 77], 0), ([140, 9], [300, 77], 45)])
def test_attn_scales(kind, cache, scale, new, kv, window):
    """Negative scales turn the order of the keys; one of zero has all keys' mean."""
    check_made(deep(base.make_attn(new, kv, 4, 2, 64, 16, kind, cache, q_by=0.5)), 4, 2, 64, kind, cache, window=window, scale=scale)


@pytest.mark.parametrize("kind,cache", base.PAIRS)
@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("new", [[1, 1], [40, 3], [140, 9]])
def test_attn_nonfinite_queries(kind, cache, bad, new):
    """A query that holds a NaN, or an infinity that some key's feature lifts above all or meets as zero, has NaN; all others stay."""
    made = list(deep(base.make_attn(new, [300, 77], 4, 2, 64, 16, kind, cache)))
    clean = base.run_attn(made, 4, 2, 64, 16, kind, cache)
    made[0] = made[0].clone()
    rows = [(0, 1), (sum(new) - 1, 3), (sum(new) // 2, 0)]
    for t, h in rows:
        made[0][t, h, 5] = bad
    out = base.run_attn(made, 4, 2, 64, 16, kind, cache)
    hit = torch.zeros(out.shape[:2], dtype=torch.bool)
    for t, h in rows:
        hit[t, h] = True
    assert torch.isnan(out[hit]).all() and torch.equal(out[~hit], clean[~hit])


@pytest.mark.parametrize("kind,cache", [("bf16", "bf16"), ("f16", "f16")])
@pytest.mark.parametrize("new", [1, 40, 140])
def test_attn_scores_of_minus_infinity(kind, cache, new):
    """Keys of minus infinity weigh nothing, with others beside them and without."""
    made = list(deep(base.make_attn([new], [300], 2, 1, 64, 16, kind, cache)))
    q, q_start, kv_len, table, k, v, _, _ = made
    q[..., 3] = q[..., 3].abs() + 1
    lost = [j for j in range(300) if j % 3]
    beside = [t.clone() for t in made[4:6]]
    for j in lost:
        beside[0][int(table[0, j // 16]), :, j % 16, 3] = -math.inf
    out = base.run_attn((q, q_start, kv_len, table, *beside, None, None), 2, 1, 64, 16, kind, cache)
    _, _, tops = ref.attention(q, q_start, kv_len, table, k, v, 64 ** -0.5)  # of finite scores
    want, mags, _ = ref.attention(q, q_start, kv_len, table, *beside, 64 ** -0.5)
    base.close(out, want, base.attn_bound(want, mags, tops, kind, 64, 300), "beside others")
    for j in range(300):
        beside[0][int(table[0, j // 16]), :, j % 16, 3] = -math.inf
    assert (base.run_attn((q, q_start, kv_len, table, *beside, None, None), 2, 1, 64, 16, kind, cache) == 0).all()


@pytest.mark.parametrize("kind,cache", base.PAIRS)
@pytest.mark.parametrize("max_new", [None, 200, 1, 7])
def test_attn_chunk_beside_single_tokens(kind, cache, max_new):
    """One call of a chunk and of single tokens, on each of the kernels."""
    new, kv = [200, 1, 1, 7, 1, 0], [700, 1, 900, 7, 2000, 40]
    made = deep(base.make_attn(new, kv, 4, 1, 64, 16, kind, cache))
    out = base.run_attn(made, 4, 1, 64, 16, kind, cache, max_new=max_new)
    want, mags, tops = ref.attention(made[0], made[1], made[2], made[3], made[4], made[5], 64 ** -0.5, k_scale=made[6], v_scale=made[7])
    base.close(out, want, base.attn_bound(want, mags, tops, kind, 64, 2000), "mixed")


# ---------------------------------------------------------------- more than one launch takes


@pytest.mark.parametrize("out", ["same", "i8"])
def test_norm_rows_past_one_launch(out):
    """2^26 + 1029 rows of a wave each: 2^32 threads and more."""
    rows, dim, part = (1 << 26) + 1029, 8, 1 << 24
    g = torch.Generator(device="cuda").manual_seed(3)
    x, r = (torch.randn(rows, dim, generator=g, device="cuda").bfloat16() for _ in range(2))
    w = (1 + 0.2 * torch.randn(dim, generator=g, device="cuda")).bfloat16()
    y = torch.full((rows, dim), 77, dtype=torch.int8 if out == "i8" else torch.bfloat16, device="cuda")
    h, step = torch.full_like(x, 77), torch.full((rows,), 77.0, device="cuda") if out == "i8" else None
    desc = llm.make_rms_desc(dim, out_dtype=KIND[out if out == "i8" else "bf16"])
    llm.cbs_rms_norm(desc, x, w, y, residual=r, residual_out=h, out_scale=step)
    got = [torch.empty_like(t[:part]) if t is not None else None for t in (y, h, step)]
    for at in range(0, rows, part):  # parts of the same, of one launch each: the same bits
        n = min(part, rows - at)
        a, b, c = (None if t is None else t[:n] for t in got)
        llm.cbs_rms_norm(desc, x[at : at + n], w, a, residual=r[at : at + n], residual_out=b, out_scale=c)
        assert torch.equal(y[at : at + n], a) and torch.equal(h[at : at + n], b) and (c is None or torch.equal(step[at : at + n], c)), at


def test_kv_vectors_past_one_launch():
    """2^30 vectors and more (69 GB read back), of which all but a few tokens, at the ends of launches, have no slot."""
    heads, dim, page, tokens = 65535, 16, 16, 16400
    good = list(range(5)) + list(range(8186, 8198)) + list(range(16381, 16389)) + list(range(tokens - 4, tokens))
    slots = torch.full((tokens,), -1, dtype=torch.int64)
    slots[good] = torch.arange(len(good)) + 7
    slots = slots.cuda()
    g = base.gen(4)
    k, v = (base.normal(g, tokens, 1, dim, kind="bf16").cuda().expand(tokens, heads, dim) for _ in range(2))
    kc, vc, ks, vs = base.kv_buffers(3, heads, dim, page, "i8")
    desc = llm.make_kv_desc(heads, dim, page)
    llm.cbs_kv_write(desc, k, v, slots, kc, vc, ks, vs)
    want = base.kv_buffers(3, heads, dim, page, "i8")  # the same of the few tokens alone: one launch
    llm.cbs_kv_write(desc, k[good], v[good], slots[good], *want)
    for a, b in zip((kc, vc, ks, vs), want):
        assert torch.equal(a, b)
    out = [torch.full((tokens, heads, dim), 77, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    llm.cbs_kv_read(desc, slots, kc, vc, out[0], out[1], ks, vs)
    few = [torch.empty(len(good), heads, dim, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    llm.cbs_kv_read(desc, slots[good], kc, vc, few[0], few[1], ks, vs)
    for a, b in zip(out, few):
        assert torch.equal(a[good], b)
        a[good] = 0
        assert not any(part.any() for part in a.split(1024))


def many_sequences(seqs, heads, kv_heads, dim, kind, seed):
    """A new token each, over two pages that they share."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    page = 16
    q = torch.randn(seqs, heads, dim, generator=g, device="cuda").to(base.TYPES[kind])
    k, v = (torch.randint(-127, 128, shape, generator=g, device="cuda", dtype=torch.int8) for shape in ((2, kv_heads, page, dim), (2, kv_heads, dim, page)))
    ks, vs = ((0.5 + torch.rand(2, kv_heads, page, generator=g, device="cuda")) / 70 for _ in range(2))
    kv_len = torch.randint(0, 33, (seqs,), generator=g, device="cuda", dtype=torch.int32)
    table = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda").repeat(seqs, 1)
    return q, torch.arange(seqs + 1, dtype=torch.int32, device="cuda"), kv_len, table, k, v, ks, vs


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_attn_sequences_past_one_launch(kind):
    """65535 sequences over 512 heads of the cache: 2^25 units."""
    seqs, heads, dim, part = 65535, 512, 16, 8000
    q, q_start, kv_len, table, k, v, ks, vs = many_sequences(seqs, heads, heads, dim, kind, 6)
    attn = llm.cbs_attn_create(llm.make_attn_desc(heads, heads, dim, 16, dtype=KIND[kind], max_seqs=seqs))
    out = torch.full_like(q, 77)
    llm.cbs_attn_run(attn, q, q_start, kv_len, table, k, v, out, ks, vs, max_new=1)
    few = torch.empty_like(q[:part])
    for at in range(0, seqs, part):  # parts of the same, of one launch each: the same bits
        n = min(part, seqs - at)
        llm.cbs_attn_run(attn, q[at : at + n], q_start[: n + 1], kv_len[at : at + n], table[at : at + n], k, v, few[:n], ks, vs, max_new=1)
        assert torch.equal(out[at : at + n], few[:n]), at


@pytest.mark.parametrize("kind,heads,dim", [("bf16", 512, 64), ("f16", 512, 64), ("f32", 64, 64), ("bf16", 64, 48)])
def test_attn_bounds_past_one_launch(kind, heads, dim):
    """max_new as if all tokens were one sequence's: units of 2^32 threads and more, of many rows and of 16."""
    seqs = 2048
    q, q_start, kv_len, table, k, v, ks, vs = many_sequences(seqs, heads, 1, dim, kind, 7)
    attn = llm.cbs_attn_create(llm.make_attn_desc(heads, 1, dim, 16, dtype=KIND[kind], causal=False, max_seqs=seqs))
    out = torch.full_like(q, 77), torch.full_like(q, 78)
    for to, most in zip(out, (seqs, 1)):
        llm.cbs_attn_run(attn, q, q_start, kv_len, table, k, v, to, ks, vs, max_new=most)
    assert torch.equal(*out)
    want, mags, tops = ref.attention(*(t.cpu() for t in (q[:5], q_start[:6], kv_len[:5], table[:5], k, v)), dim ** -0.5, False, 0, ks.cpu(), vs.cpu())
    base.close(out[0][:5], want, base.attn_bound(want, mags, tops, kind, dim, 32), "of the first")


# ---------------------------------------------------------------- what the bindings pass


@pytest.fixture
def passed(monkeypatch):
    """Arguments of cbs_attn_run, from the extension module and from the checks in Python, in place of a run."""
    import ctypes
    from types import SimpleNamespace
    got = []

    def take(attn, args, stream):
        got.append(llm.cbs_attn_args.from_buffer_copy(ctypes.string_at(args, ctypes.sizeof(llm.cbs_attn_args))))
        return 0

    names = ("cbs_rms_norm", "cbs_w4_linear", "cbs_kv_write", "cbs_kv_read", "cbs_attn_run")
    addresses = [ctypes.cast(getattr(llm.lib, name), ctypes.c_void_p).value for name in names]
    called = ctypes.CFUNCTYPE(ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p)(take)
    llm._llm_bind.setup(*addresses[:4], ctypes.cast(called, ctypes.c_void_p).value)
    monkeypatch.setattr(llm, "lib", SimpleNamespace(cbs_attn_run=lambda attn, args, stream: take(attn, args, stream), cbs_attn_destroy=llm.lib.cbs_attn_destroy))
    yield got
    llm._llm_bind.setup(*addresses)


@pytest.mark.parametrize("tokens,seqs,most", [(32, 32, 1), (32, 1, 32), (543, 32, 543), (5, 9, 5), (1, 1, 1), (0, 3, 0)])
def test_attn_default_of_max_new(passed, tokens, seqs, most):
    """As many as there are, but for a batch of single tokens."""
    attn = llm.Attn(0, llm.make_attn_desc(2, 1, 16, 16, max_seqs=seqs))
    attn.handle = 1  # no run uses it
    try:
        q = torch.zeros(tokens, 2, 16, dtype=torch.bfloat16, device="cuda")
        caches = base.kv_buffers(2, 1, 16, 16, "i8")
        starts, lengths = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (seqs + 1, seqs))
        table = torch.zeros(seqs, 3, dtype=torch.int32, device="cuda")
        for stream in (None, torch.cuda.current_stream()):
            llm.cbs_attn_run(attn, q, starts, lengths, table, caches[0], caches[1], q, caches[2], caches[3], stream=stream)
            llm.cbs_attn_run(attn, q, starts, lengths, table, caches[0], caches[1], q, caches[2], caches[3], max_new=7, max_kv=9, stream=stream)
    finally:
        attn.handle = 0
    assert [(a.max_new, a.max_kv) for a in passed] == [(most, 48), (7, 9)] * 2


def test_attn_default_of_max_kv(passed):
    """A table with room for 2^31 tokens and more."""
    attn = llm.Attn(0, llm.make_attn_desc(1, 1, 16, 1024))
    attn.handle = 1  # no run uses it
    try:
        q = torch.zeros(2, 1, 16, dtype=torch.bfloat16, device="cuda")
        caches = base.kv_buffers(2, 1, 16, 1024, "i8")
        starts, lengths = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (2, 1))
        for columns, most in ((1 << 21, 2**31 - 1), ((1 << 21) - 1, 2**31 - 1024)):
            table = torch.zeros(1, columns, dtype=torch.int32, device="cuda")
            for stream in (None, torch.cuda.current_stream()):
                llm.cbs_attn_run(attn, q, starts, lengths, table, caches[0], caches[1], q, caches[2], caches[3], stream=stream)
                assert (passed[-1].max_new, passed[-1].max_kv) == (2, most)
    finally:
        attn.handle = 0
    assert len(passed) == 4


def test_attn_table_past_31_bits():
    """The run itself with such a table."""
    made = list(base.make_attn([1, 3], [40, 40], 2, 1, 16, 1024, "bf16", "i8"))
    want = base.run_attn(made, 2, 1, 16, 1024, "bf16", "i8")
    table = torch.full((2, (1 << 21) + 3), -1, dtype=torch.int32)
    table[:, :1] = made[3]
    made[3] = table
    assert torch.equal(base.run_attn(made, 2, 1, 16, 1024, "bf16", "i8"), want)


# ---------------------------------------------------------------- empty caches and tables


@pytest.mark.parametrize("kind,cache", base.PAIRS)
@pytest.mark.parametrize("new", [[1, 1], [150, 40]])
@pytest.mark.parametrize("pages,columns", [(0, 3), (2, 0), (0, 0)])
def test_attn_of_an_empty_cache(kind, cache, new, pages, columns):
    """No pages, no columns: no key is seen, whatever the lengths say."""
    made = list(base.make_attn(new, [200, 64], 4, 2, 64, 16, kind, cache))
    made[3] = torch.zeros(2, columns, dtype=torch.int32)
    made[4:] = [None if t is None else t[:pages] for t in made[4:]]
    for max_kv in (None, 1 << 18):
        assert (base.run_attn(made, 4, 2, 64, 16, kind, cache, max_kv=max_kv) == 0).all()


@pytest.mark.parametrize("kind,cache,read", [("bf16", "i8", "bf16"), ("f16", "f16", "f16"), ("f32", "i8", "f32")])
@pytest.mark.parametrize("heads", [1, 300])
def test_kv_of_an_empty_cache(kind, cache, read, heads):
    """All slots lie outside; reading gives zeros.  And no tokens of a transposed tensor."""
    kc, vc, ks, vs = base.kv_buffers(0, heads, 64, 16, cache)
    desc = llm.make_kv_desc(heads, 64, 16, dtype=KIND[kind], cache_dtype=KIND[cache], read_dtype=KIND[read])
    x, slots = base.normal(base.gen(1), 40, heads, 64, kind=kind).cuda(), torch.arange(-3, 37).cuda()
    llm.cbs_kv_write(desc, x, x, slots, kc, vc, ks, vs)
    k, v = (torch.full(x.shape, 77, dtype=base.TYPES[read], device="cuda") for _ in range(2))
    llm.cbs_kv_read(desc, slots, kc, vc, k, v, ks, vs)
    assert (k == 0).all() and (v == 0).all()
    kc, vc, ks, vs = base.kv_buffers(1, heads, 64, 16, cache)
    none = torch.empty(heads, 0, 64, dtype=base.TYPES[read], device="cuda").transpose(0, 1)
    llm.cbs_kv_read(desc, slots[:0], kc, vc, none, none, ks, vs)


@pytest.mark.parametrize("rows,dim", [(1, 512), (7, 512), (40, 1000)])
def test_norm_int8_rows_into_their_input(rows, dim):
    """Codes into the bytes of the row that they come from; the sum into the residual."""
    g = base.gen(rows)
    x, r = (base.normal(g, rows, dim, kind="bf16").cuda() for _ in range(2))
    w = torch.ones(dim, dtype=torch.bfloat16, device="cuda")
    desc = llm.make_rms_desc(dim, out_dtype=llm.CBS_I8)
    step = [torch.empty(rows, device="cuda") for _ in range(2)]
    want, h = torch.empty(rows, dim, dtype=torch.int8, device="cuda"), torch.empty_like(x)
    llm.cbs_rms_norm(desc, x, w, want, residual=r, residual_out=h, out_scale=step[0])
    codes = x.view(torch.int8)[:, :dim]
    llm.cbs_rms_norm(desc, x, w, codes, residual=r, residual_out=r, out_scale=step[1])
    assert torch.equal(codes, want) and torch.equal(*step) and torch.equal(r, h)
    if rows > 1:
        with pytest.raises(llm.CbsError, match="begins at"):
            llm.cbs_rms_norm(desc, r, w, r.view(torch.int8).flatten()[: rows * dim].view(rows, dim), out_scale=step[0])


# ---------------------------------------------------------------- the example's decoder


def test_decoder_past_its_pages():
    """Single tokens go on where a sequence has no room: what is cached stays, the other's goes on as it would."""
    from convolution_implicit_gemm_02_amd import decoder_step as ds
    small = dict(hidden=256, heads=4, kv_heads=2, head_dim=64, ffn=640, layers=2, group=64, page=16)
    x = torch.randn(2, 30, 256, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda").bfloat16()
    got = []
    for long in (29, 20):
        decoder = ds.Decoder(ds.Config(**small), 2, 32, 32, seed=5)
        assert decoder.table.shape == (2, 2)
        rows = torch.stack([decoder.prompt(0, x[0, :long]), decoder.prompt(1, x[1, :10])])
        for step in range(8):
            decoder.single(rows)
            if long + step + 1 == 32:
                full = [t.clone() for layer in range(2) for t in decoder.cached(layer, 0)]
        got.append((rows[1].clone(), [t for layer in range(2) for t in decoder.cached(layer, 1)]))
        assert decoder.kv_len.tolist() == [min(long + 8, 32), 18] and rows.isfinite().all()
        if long == 29:
            assert all(torch.equal(a, b) for a, b in zip(full, [t for layer in range(2) for t in decoder.cached(layer, 0)]))
    assert torch.equal(got[0][0], got[1][0]) and all(torch.equal(a, b) for a, b in zip(got[0][1], got[1][1]))
    with pytest.raises(ValueError, match="room"):
        decoder.prompt(1, x[1, :15])
