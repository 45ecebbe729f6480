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
