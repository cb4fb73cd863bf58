"""What the build needs: the CUDA library needs nvcc alone, the compiled binding torch's headers.  No compiler runs
here."""
import builtins

import pytest

from output_head_kl_b200 import build as B


@pytest.fixture
def steps(monkeypatch, tmp_path):
    """A build into an empty folder whose compiler calls are recorded instead of made."""
    done = []
    for name in ("LIB", "DEBUG_LIB", "PROFILE_LIB", "BINDING"):
        monkeypatch.setattr(B, name, str(tmp_path / (name.lower() + ".so")))
    monkeypatch.setattr(B, "OUT_DIR", str(tmp_path))
    monkeypatch.setattr(B, "_build_one", lambda lib, *a: done.append(lib) or [])
    monkeypatch.setattr(B, "_build_binding", lambda: done.append(B.BINDING))
    return done


def _no_torch(monkeypatch):
    real = builtins.__import__

    def imp(name, *a, **kw):
        if name == "torch" or name.startswith("torch."):
            raise ModuleNotFoundError("No module named 'torch'")
        return real(name, *a, **kw)
    monkeypatch.setattr(builtins, "__import__", imp)


def test_the_library_comes_first(steps):
    B.build()
    assert steps == [B.LIB, B.DEBUG_LIB, B.PROFILE_LIB, B.BINDING]


def test_a_failing_binding_leaves_the_libraries_built(steps, monkeypatch):
    def fails():
        raise RuntimeError("g++ failed on binding.cpp")
    monkeypatch.setattr(B, "_build_binding", fails)
    with pytest.raises(RuntimeError, match="binding.cpp"):
        B.build()
    assert steps == [B.LIB, B.DEBUG_LIB, B.PROFILE_LIB]


def test_without_torch_the_library_is_built_alone(steps, monkeypatch, capsys):
    """No torch, no binding to build: C callers need the library only."""
    _no_torch(monkeypatch)
    assert B.build(debug=False, profile=False) == B.LIB
    assert steps == [B.LIB] and "binding" in capsys.readouterr().err


def test_another_torch_rebuilds_the_binding(steps, monkeypatch, tmp_path):
    import torch
    for lib in (B.LIB, B.BINDING):
        with open(lib, "w"):
            pass
    monkeypatch.setattr(B, "_stale", lambda lib: False)
    stamp = B.BINDING + ".torch"
    with open(stamp, "w") as f:
        f.write(torch.__version__)
    B.build(debug=False, profile=False)
    assert steps == []
    with open(stamp, "w") as f:
        f.write("0.0.1")
    B.build(debug=False, profile=False)
    assert steps == [B.BINDING]


def test_a_binding_of_another_torch_is_not_loaded(monkeypatch, tmp_path):
    import torch

    import output_head_kl_b200 as K
    path = tmp_path / "kdkl_binding.so"
    path.write_bytes(b"")
    monkeypatch.setattr(K, "_binding", None)
    monkeypatch.setattr(K, "BINDING_PATH", str(path))
    x = torch.zeros(4, 16, dtype=torch.bfloat16)
    for stamp in (None, "0.0.1"):
        if stamp:
            (tmp_path / "kdkl_binding.so.torch").write_text(stamp)
        with pytest.raises(RuntimeError, match="built against torch"):
            K.kdkl_rmsnorm_forward(x, x[0], x)
