"""The native binding of the paged-cache calls is built against the installed PyTorch; what
does not need it, does not depend on it."""
import subprocess
import sys
import textwrap

import pytest

from exact_attention_55_gb300 import build
from tests.conftest import ROOT


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


def run(code):
    r = subprocess.run([sys.executable, "-c", textwrap.dedent(code)], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr


@pytest.mark.parametrize("content", [None, b"not a library"])
def test_without_the_binding_only_its_own_calls_raise(tmp_path, content):
    """Missing, or there and not loadable."""
    path = tmp_path / "binding.so"
    if content is not None:
        path.write_bytes(content)
        (tmp_path / "binding.so.abi").write_text(build._abi())
    run(f"""
        import torch
        from exact_attention_55_gb300 import build
        build.BINDING_PATH = {str(path)!r}
        import exact_attention_55_gb300 as fa
        assert fa.load_library().attn_fwd_bf16(*[None] * 5, 1, 1, 1, 64, 0.1, 0, 0, None) == 1
        assert fa.attn_status_string(0) and fa.attn_fp8_qk_block_rows(128) > 0
        i = torch.zeros(2, dtype=torch.int32)
        for _ in range(2):
            try:
                fa.attn_paged_plan(i, i, i[None], i, i[:1], 16, 4)
            except (RuntimeError, ImportError) as e:
                assert {str(path)!r} in str(e), e
            else:
                raise AssertionError("no binding, no error")
    """)


def test_the_binding_is_loaded_by_the_first_call_that_needs_it():
    run("""
        import torch
        import exact_attention_55_gb300 as fa
        fa.load_library()
        assert fa._binding is None
        i = torch.zeros(2, dtype=torch.int32)
        try:
            fa.attn_paged_plan(i, i, i[None], i, i[:1], 16, 4)
        except TypeError as e:
            assert "CUDA" in str(e), e
        assert fa._binding is not None
    """)


def test_the_library_is_linked_before_the_binding_may_fail(monkeypatch, tmp_path):
    """A binding that does not compile is an error of build(), behind a library that is there."""
    lib = tmp_path / "lib.so"
    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    monkeypatch.setattr(build, "LIB_PATH", str(lib))
    monkeypatch.setattr(build, "BINDING_PATH", str(tmp_path / "binding.so"))
    monkeypatch.setattr(build, "UNITS", [("schedule", "quant_fp8.cu", [])])

    def fails():
        raise RuntimeError("g++ failed for binding.cpp")
    monkeypatch.setattr(build, "_compile_binding", fails)
    with pytest.raises(RuntimeError, match="binding"):
        build.build()
    assert lib.exists()


def test_a_binding_for_another_pytorch_is_stale(monkeypatch, tmp_path):
    """build() compiles the binding again, and only it; loading it before that says why not."""
    lib, path = tmp_path / "lib.so", tmp_path / "binding.so"
    lib.write_bytes(b"")
    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    monkeypatch.setattr(build, "LIB_PATH", str(lib))
    monkeypatch.setattr(build, "BINDING_PATH", str(path))
    real, calls = subprocess.run, []

    def compiler(cmd, **kw):
        if cmd[0] != "g++":
            return real(cmd, **kw)
        calls.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "wb") as f:
            f.write(b"")
        return subprocess.CompletedProcess(cmd, 0, "", "")
    monkeypatch.setattr(build.subprocess, "run", compiler)
    monkeypatch.setattr(build, "_nvcc", lambda: "/usr/local/cuda/bin/nvcc")
    build.build()
    build.build()
    assert len(calls) == 1                               # built once, then up to date
    import torch
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", "99.0.1+cu990")
        with pytest.raises(RuntimeError, match="built against torch .*99.0.1"):
            build.load_binding()
        build.build()
        build.build()
    assert len(calls) == 2
    build.build()                                        # and back
    assert len(calls) == 3
