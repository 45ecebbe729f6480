"""CPU-tier checks of the decoder-step operators: the library exports what include/cbs_llm.h declares, the binding's
structures follow the header, and bad descriptors and arguments are refused before a device is touched."""
import ctypes
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "cbs_llm.h")


@pytest.fixture(scope="module")
def llm():
    from convolution_implicit_gemm_02_amd import llm as mod
    return mod


def header():
    return re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)


def test_header_symbols_exported(llm):
    names = sorted(set(re.findall(r"\b(cbs_[a-z0-9_]+)\s*\(", header())))
    assert len(names) >= 7
    assert not [n for n in names if not hasattr(ctypes.CDLL(llm.lib._name), n)]
    assert set(names) == set(llm._SIGNATURES)


@pytest.mark.parametrize("name", ["rms_desc", "rms_args", "w4_desc", "w4_args", "kv_desc", "kv_args", "attn_desc", "attn_args"])
def test_structures_follow_header(llm, name):
    body = re.search(r"typedef struct cbs_%s \{(.*?)\}" % name, header(), re.S).group(1)
    fields = []
    for line in body.split(";"):
        line = " ".join(line.split())
        if line:
            kind, rest = re.match(r"((?:const )?\w+)\s*(.*)", line).groups()
            for f in rest.split(","):
                fields.append((f.strip().lstrip("* "), 8 if "*" in f or kind == "int64_t" else 4))
    cls = getattr(llm, "cbs_" + name)
    assert [f for f, _ in fields] == [f for f, _ in cls._fields_]
    assert [s for _, s in fields] == [ctypes.sizeof(t) for _, t in cls._fields_]
    pack = getattr(llm, "_pack_" + name.split("_")[0], None)
    if name.endswith("_args"):
        assert pack.__self__.size == ctypes.sizeof(cls)


def test_header_compiles_as_c(tmp_path):
    import shutil
    import subprocess
    cc = shutil.which("gcc")
    if cc is None:
        pytest.skip("no host compiler")
    src = tmp_path / "use.c"
    src.write_text('#include "cbs_llm.h"\nint main(void) { cbs_rms_desc d; cbs_attn_args a; return sizeof d + sizeof a > 0 ? 0 : 1; }\n')
    subprocess.run([cc, "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic", "-fsyntax-only", "-I", os.path.dirname(HEADER), str(src)], check=True)


A = 1 << 20  # an address: none of these calls gets as far as using it
RMS = dict(dim=64, dtype=4, out_dtype=4, weight_dtype=4, eps=1e-6)
RMS_ARGS = dict(x=A, weight=A, out=A, rows=4, x_stride=64, out_stride=64)
W4 = dict(k=64, n=32, group=32, dtype=4, out_dtype=4, scale_dtype=3)
W4_ARGS = dict(x=A, codes=A, scales=A, out=A, rows=2, x_stride=64, out_stride=32)
KV = dict(heads=2, head_dim=64, page_size=16, dtype=4, cache_dtype=1, read_dtype=4)
KV_ARGS = dict(k=A, v=A, slots=A, k_cache=A, v_cache=A, k_scale=A, v_scale=A, tokens=3, pages=4, k_token_stride=128, k_head_stride=64, v_token_stride=128,
               v_head_stride=64)
ATTN = dict(heads=4, kv_heads=2, head_dim=64, page_size=16, dtype=4, cache_dtype=1, causal=1, window=0, scale=0.125, max_seqs=2)


def status(llm, fn, name, desc, args):
    d = getattr(llm, "cbs_%s_desc" % name)(**desc)
    a = getattr(llm, "cbs_%s_args" % name)(**args)
    return getattr(llm.lib, fn)(d, bytes(a), None)


@pytest.mark.parametrize("desc,args,want", [
    (dict(dim=0), {}, "EINVAL"), (dict(dim=65537), {}, "EUNSUPPORTED"), (dict(dtype=1), {}, "EINVAL"), (dict(dtype=9), {}, "EINVAL"),
    (dict(weight_dtype=1), {}, "EINVAL"), (dict(out_dtype=0), {}, "EUNSUPPORTED"), (dict(eps=-1.0), {}, "EINVAL"), (dict(eps=float("nan")), {}, "EINVAL"),
    ({}, dict(rows=-1), "EINVAL"), ({}, dict(rows=1 << 40), "EUNSUPPORTED"), ({}, dict(x=None), "EINVAL"), ({}, dict(weight=None), "EINVAL"),
    ({}, dict(out=None), "EINVAL"), ({}, dict(residual_out=A, residual_out_stride=64), "EINVAL"), ({}, dict(out_scale=A), "EINVAL"),
    (dict(out_dtype=1), {}, "EINVAL"), ({}, dict(x_stride=-64), "EINVAL"), ({}, dict(out_stride=63), "EINVAL"), ({}, dict(x_stride=1 << 60), "EUNSUPPORTED"),
    ({}, dict(residual=A, residual_stride=64, residual_out=A, residual_out_stride=0), "EINVAL"),
    ({}, dict(rows=0), "OK"), (dict(out_dtype=1), dict(rows=0, x=None, out=None), "OK"),
])
def test_rms_norm_refusals(llm, desc, args, want):
    assert status(llm, "cbs_rms_norm", "rms", {**RMS, **desc}, {**RMS_ARGS, **args}) == getattr(llm, "CBS_" + want)


B = A + (1 << 19)


@pytest.mark.parametrize("desc,args", [
    (dict(out_dtype=1), dict(out=A, out_scale=B)),                                          # int8 rows closer together than x's
    ({}, dict(out=A, out_stride=80)),
    ({}, dict(x_stride=0)),                                                                 # one row for all, and written
    ({}, dict(x=B, residual=A, residual_stride=72)),
    ({}, dict(out=B, residual=B + 1024, residual_stride=64, residual_out=A, residual_out_stride=65)),
    ({}, dict(x=B, out=B, residual=A, residual_stride=0, residual_out=A, residual_out_stride=64)),
    ({}, dict(x=B, residual=B, residual_stride=64, residual_out=A, residual_out_stride=64)),  # both outputs
])
def test_rms_norm_into_its_input(llm, desc, args):
    """An output where an input lies, whose rows lie elsewhere: a row would be written before others are read."""
    assert status(llm, "cbs_rms_norm", "rms", {**RMS, **desc}, {**RMS_ARGS, **args}) == llm.CBS_EINVAL
    assert "begins at" in llm.lib.cbs_last_error().decode() or "out is residual_out" in llm.lib.cbs_last_error().decode()


@pytest.mark.parametrize("desc,args,want", [
    (dict(k=0), {}, "EINVAL"), (dict(n=-1), {}, "EINVAL"), (dict(k=(1 << 24) + 1), {}, "EUNSUPPORTED"), (dict(group=0), {}, "EINVAL"),
    (dict(group=16), {}, "EUNSUPPORTED"), (dict(group=96), {}, "EUNSUPPORTED"), (dict(group=192), {}, "EUNSUPPORTED"), (dict(dtype=2), {}, "EINVAL"),
    (dict(out_dtype=1), {}, "EINVAL"), (dict(scale_dtype=1), {}, "EINVAL"), ({}, dict(codes=None), "EINVAL"), ({}, dict(codes=A + 8), "EINVAL"),
    ({}, dict(scales=None), "EINVAL"), ({}, dict(x_scale=A), "EINVAL"), (dict(dtype=1), {}, "EINVAL"), ({}, dict(rows=-2), "EINVAL"),
    ({}, dict(out_stride=31), "EINVAL"), ({}, dict(x=None), "EINVAL"), ({}, dict(rows=0), "OK"),
])
def test_w4_refusals(llm, desc, args, want):
    assert status(llm, "cbs_w4_linear", "w4", {**W4, **desc}, {**W4_ARGS, **args}) == getattr(llm, "CBS_" + want)


@pytest.mark.parametrize("fn", ["cbs_kv_write", "cbs_kv_read"])
@pytest.mark.parametrize("desc,args,want", [
    (dict(heads=0), {}, "EINVAL"), (dict(head_dim=72), {}, "EUNSUPPORTED"), (dict(head_dim=272), {}, "EUNSUPPORTED"), (dict(head_dim=-16), {}, "EINVAL"),
    (dict(page_size=8), {}, "EUNSUPPORTED"), (dict(page_size=0), {}, "EINVAL"), (dict(page_size=2048), {}, "EUNSUPPORTED"), (dict(dtype=1), {}, "EINVAL"),
    (dict(cache_dtype=3), {}, "EUNSUPPORTED"), (dict(cache_dtype=4, read_dtype=3), {}, "EUNSUPPORTED"), (dict(cache_dtype=0, dtype=0, read_dtype=0), {}, "EUNSUPPORTED"),
    (dict(cache_dtype=4), {}, "EINVAL"),  # scales with a 16-bit cache
    ({}, dict(k_scale=None), "EINVAL"), ({}, dict(k_cache=None), "EINVAL"), ({}, dict(v_cache=A + 4), "EINVAL"), ({}, dict(slots=None), "EINVAL"),
    ({}, dict(tokens=-1), "EINVAL"), ({}, dict(pages=-1), "EINVAL"), ({}, dict(k_token_stride=-1), "EINVAL"), ({}, dict(pages=1 << 42), "EUNSUPPORTED"),
    ({}, dict(tokens=0, k=None, v=None, slots=None), "OK"),
])
def test_kv_refusals(llm, fn, desc, args, want):
    assert status(llm, fn, "kv", {**KV, **desc}, {**KV_ARGS, **args}) == getattr(llm, "CBS_" + want)


@pytest.mark.parametrize("args", [dict(k_token_stride=0), dict(v_head_stride=0), dict(k_token_stride=64, k_head_stride=64), dict(v_token_stride=100)])
def test_kv_read_into_overlapping_vectors(llm, args):
    assert status(llm, "cbs_kv_read", "kv", KV, {**KV_ARGS, **args}) == llm.CBS_EINVAL


@pytest.mark.parametrize("fn", ["cbs_kv_write", "cbs_kv_read"])
@pytest.mark.parametrize("args", [
    dict(k_token_stride=64, k_head_stride=64), dict(v_token_stride=0, v_head_stride=0), dict(pages=0, k_cache=None, v_cache=None, k_scale=None, v_scale=None)])
def test_kv_of_nothing(llm, fn, args):
    """No tokens, whatever their strides (those of a transposed empty tensor among them), and a cache of no pages."""
    assert status(llm, fn, "kv", KV, {**KV_ARGS, "tokens": 0, "k": None, "v": None, "slots": None, **args}) == llm.CBS_OK


@pytest.mark.parametrize("desc,want", [
    (dict(heads=3), "EINVAL"), (dict(kv_heads=0), "EINVAL"), (dict(heads=0), "EINVAL"), (dict(head_dim=40), "EUNSUPPORTED"), (dict(page_size=24), "EUNSUPPORTED"),
    (dict(dtype=1), "EINVAL"), (dict(cache_dtype=3), "EUNSUPPORTED"), (dict(cache_dtype=0, dtype=0), "EUNSUPPORTED"), (dict(causal=2), "EINVAL"),
    (dict(window=-1), "EINVAL"), (dict(scale=float("inf")), "EINVAL"), (dict(max_seqs=0), "EINVAL"), (dict(max_seqs=70000), "EINVAL"),
])
def test_attn_create_refusals(llm, desc, want):
    h = ctypes.c_void_p(7)
    assert llm.lib.cbs_attn_create(llm.cbs_attn_desc(**{**ATTN, **desc}), ctypes.byref(h)) == getattr(llm, "CBS_" + want)
    assert h.value is None
    assert "attn_create" in llm.lib.cbs_last_error().decode()


def test_null_arguments(llm):
    for fn in (llm.lib.cbs_rms_norm, llm.lib.cbs_w4_linear, llm.lib.cbs_kv_write, llm.lib.cbs_kv_read, llm.lib.cbs_attn_run):
        assert fn(None, None, None) == llm.CBS_EINVAL
    assert llm.lib.cbs_attn_create(None, None) == llm.CBS_EINVAL
    llm.lib.cbs_attn_destroy(None)


def test_host_tensors_refused(llm):
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="not on a GPU"):
        llm.cbs_rms_norm(llm.make_rms_desc(64), x, x[0], x)


def test_bind_hands_back_what_is_not_in_order(llm):
    """The extension module never refuses: it returns -1, and the checks in Python say what is wrong."""
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    w, d = torch.ones(64, dtype=torch.bfloat16), llm.make_rms_desc(64)
    bind = llm._llm_bind
    assert bind.rms_norm(d, x, w, x, None, None, None) == -1  # not on a GPU
    assert bind.rms_norm(d, None, w, x, None, None, None) == -1 and bind.rms_norm(d, x) == -1 and bind.rms_norm(None, x, w, x, None, None, None) == -1
    assert bind.rms_norm(llm.make_w4_desc(64, 64), x, w, x, None, None, None) == -1  # another operator's descriptor
    assert bind.w4_linear(llm.make_w4_desc(64, 32), x, x, x, x, None, None) == -1
    assert bind.kv_write(llm.make_kv_desc(1, 16, 16), x, x, x, x, x, None, None) == -1 and bind.kv_read(3) == -1
    assert bind.attn_run(0, llm.make_attn_desc(1, 1, 16, 16), x, x, x, x, x, x, x, None, None, None, "many") == -1
    with pytest.raises(ValueError, match="not on a GPU"):
        llm.cbs_rms_norm(d, x, w, x)


def test_decoder_slots_past_its_pages():
    """Places that the decoder has no pages for have no slot."""
    from types import SimpleNamespace

    from convolution_implicit_gemm_02_amd.decoder_step import Config, Decoder
    d = SimpleNamespace(cfg=Config(page=16), table=torch.tensor([[4, 1], [0, 3]], dtype=torch.int32))
    seq, place = torch.tensor([0, 0, 1, 1, 1, 0]), torch.tensor([0, 31, 16, 32, 1 << 40, 17])
    assert Decoder.slots(d, seq, place).tolist() == [64, 31, 48, -1, -1, 17]


def test_decoder_prompt_past_its_pages():
    from types import SimpleNamespace

    from convolution_implicit_gemm_02_amd.decoder_step import Config, Decoder
    d = SimpleNamespace(cfg=Config(page=16), table=torch.tensor([[4, 1]], dtype=torch.int32), kv_len=torch.tensor([20], dtype=torch.int32))
    with pytest.raises(ValueError, match="room for 32"):
        Decoder.prompt(d, 0, torch.zeros(13, 8))
