"""CPU-tier checks of the build script."""
import os
import sys

import pytest

from convolution_implicit_gemm_02_amd import build


@pytest.mark.parametrize("torch_is_there", [True, False])
def test_library_builds_without_torch(monkeypatch, tmp_path, torch_is_there):
    """hipcc alone is enough for libcbs.so; the extension module is built where torch is there."""
    ran, moved = [], []
    monkeypatch.setattr(build, "BUILD_DIR", str(tmp_path))
    monkeypatch.setattr(build, "LIB_PATH", str(tmp_path / "libcbs.so"))
    monkeypatch.setattr(build, "BIND_PATH", str(tmp_path / "_llm_bind.so"))
    for name in [n for n in vars(build) if n.startswith("check_")]:
        monkeypatch.setattr(build, name, lambda hipcc: None)
    monkeypatch.setattr(build, "_run", ran.append)
    monkeypatch.setattr(build.os, "replace", lambda a, b: moved.append(os.path.basename(b)))
    if not torch_is_there:
        for name in [n for n in sys.modules if n == "torch" or n.startswith("torch.")]:
            monkeypatch.setitem(sys.modules, name, None)
    build.build()
    assert sorted(moved) == (["_llm_bind.so", "libcbs.so"] if torch_is_there else ["libcbs.so"])
    text = [" ".join(c) for c in ran]
    assert sum("llm_bind.cpp" in c for c in text) == torch_is_there
    assert all(any(src in c for c in text) for src in ("cbs_host.cpp", "llm_host.cpp", "llm_attn.hip", "llm_w4.hip", "llm_kv.hip", "llm_norm.hip"))


RING = """
_ZN3cbs12_GLOBAL__N_114w4_ring_kernelILi4ELi2ELi2ELb1EEEvNS_8W4ParamsE: ; @name
	global_load_lds_dwordx4 v[4:5], off
.LBB0_1:                                ; =>This Loop
%s	s_waitcnt vmcnt(10) lgkmcnt(0)
	;;#ASMSTART
	;;#ASMEND
	s_barrier
	global_load_lds_dwordx4 v[4:5], off
	s_cbranch_vccnz .LBB0_2
.LBB0_2:
%s	s_waitcnt vmcnt(10) lgkmcnt(0)
	s_barrier
	s_waitcnt vmcnt(0) lgkmcnt(0)
	s_barrier
.Lfunc_end0:
"""
CHUNK = """
_ZN3cbs12_GLOBAL__N_117attn_chunk_kernelILi4ELi4ELi4ELi2EEEvNS_10AttnParamsE: ; @name
	global_load_dword v1, v[4:5], off
	s_waitcnt vmcnt(0)
%s	s_waitcnt vmcnt(4) lgkmcnt(0)
	s_barrier
.LBB0_1:
	s_waitcnt vmcnt(2) lgkmcnt(0)
	s_barrier
	global_load_lds_dwordx4 v[4:5], off
	global_load_lds_dwordx4 v[4:5], off
	s_cbranch_vccnz .LBB0_1
	s_waitcnt vmcnt(0) lgkmcnt(0)
	s_barrier
.Lfunc_end0:
"""


def test_wait_counts_check():
    """The build's check flags a load that is missing, one that is on one way only, and one more than is counted."""
    load, lds = "\tglobal_load_dword v1, v[2:3], off\n", "\tglobal_load_lds_dwordx4 v[4:5], off\n"
    assert build.miscounted_waits(RING % (load * 10, load * 10)) == ([], 1)
    for first, second in ((load * 9, load * 10), (load * 10, load * 11), (load * 10, load + "\ts_cbranch_scc0 .LBB0_3\n" + load * 9),
                          (load + ".LBB0_4:\n" + load * 9, load * 10), (load * 2 + lds + load * 8, load * 10)):
        bad, found = build.miscounted_waits(RING % (first, second))
        assert found == 1 and len(bad) == 1
    assert build.miscounted_waits(CHUNK % (lds * 6)) == ([], 1)
    for n in (0, 4, 5, 7):
        bad, found = build.miscounted_waits(CHUNK % (lds * n))
        assert found == 1 and len(bad) == 1, n
