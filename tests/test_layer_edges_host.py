"""The layer operators' torch binding and build, without a GPU: devices, what the
package needs to be imported, and when the binding is built."""
import pytest

import dense_fp32_matrix_sgemm_gb300 as sg
from dense_fp32_matrix_sgemm_gb300 import _build


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()
    return sg.load_library()


# ------------------------------------------------------------------ devices


def test_tensors_of_different_devices_are_refused():
    # the comparison that every entry makes of its tensors, on devices that
    # exist everywhere
    torch = pytest.importorskip("torch")
    from dense_fp32_matrix_sgemm_gb300.layers import _layers
    a, b = torch.zeros(2, 2), torch.zeros(2, 2, device="meta")
    assert _layers.check_device(a, a.t()) is None
    with pytest.raises(ValueError, match="t is on meta.*first tensor on cpu"):
        _layers.check_device(b, a)
    with pytest.raises(TypeError):
        _layers.check_device(None, a)


def test_a_stream_of_another_device_is_refused():
    torch = pytest.importorskip("torch")

    class Stream:
        cuda_stream, device = 0, torch.device("cuda", 1)

    class Tensor:
        device = torch.device("cuda", 0)

    with pytest.raises(ValueError, match="stream is of cuda:1"):
        sg.quantize_rows(Tensor(), stream=Stream())


# ------------------------------------------------------------------ rows of no elements


def test_rows_of_no_elements_are_checked_like_others():
    fake = 0x100000
    assert sg.sgemm_quantize_rows(0, 4, 0, 0, 1, 0, 1, 0, check=False) == 3          # scale
    assert sg.sgemm_quantize_rows(0, 4, 0, 0, 1, 0, 1, fake + 2, check=False) == 3
    assert sg.sgemm_add_rmsnorm(0, 4, 0, 0, 1, 0, 1, 0, 1e-6, 0, 1, 0, 1, q_scale=fake + 1,
                                check=False) == 3
    assert sg.sgemm_add_rmsnorm(0, 4, 0, 0, 1, 0, 1, 0, 1e-6, 0, 1, 0, 1, rstd=fake + 1,
                                check=False) == 3
    assert sg.sgemm_add_rmsnorm(0, 4, 0, 0, 1, 0, 1, 0, 1e-6, 0, 1, 0, 1, check=False) == 0


# ------------------------------------------------------------------ imports


def test_star_import_needs_no_torch():
    # torch hidden, and the binding's module with it
    import os
    import subprocess
    import sys
    code = ("import sys\n"
            "sys.modules['torch'] = None\n"
            "from dense_fp32_matrix_sgemm_gb300 import *\n"
            "import dense_fp32_matrix_sgemm_gb300 as sg\n"
            "assert all(hasattr(sg, n) for n in sg.__all__)\n"
            "assert sgemm_linear and matmul and load_library\n"
            "try:\n"
            "    sg.linear\n"
            "except ImportError:\n"
            "    print('fine')\n")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.stdout == "fine\n", r.stderr


def test_the_torch_functions_are_attributes():
    pytest.importorskip("torch")
    for name in ("linear", "linear_backward", "add_rmsnorm", "add_rmsnorm_backward", "quantize_rows"):
        assert callable(getattr(sg, name))
    with pytest.raises(AttributeError):
        sg.no_such_operator


# ------------------------------------------------------------------ build


@pytest.fixture
def scratch_build(tmp_path, monkeypatch):
    """_build on a copy of the binding's source, with a compiler that records its
    calls: `state` holds its exit status and the commands it got."""
    import shutil
    import types
    pytest.importorskip("torch")
    shutil.copy(_build.PKG + "/_layers.cpp", tmp_path)
    monkeypatch.setattr(_build, "PKG", str(tmp_path))
    monkeypatch.setattr(_build, "BUILD", str(tmp_path / "build"))
    (tmp_path / "build").mkdir()
    state = types.SimpleNamespace(status=0, commands=[], dir=tmp_path)

    def run(cmd, **kw):
        if state.status is None:
            raise FileNotFoundError("no compiler")
        state.commands.append(cmd)
        if state.status == 0:
            with open(cmd[cmd.index("-o") + 1], "w") as f:
                f.write("built")
        return types.SimpleNamespace(returncode=state.status, stdout="", stderr="cannot find -ltorch_cuda")

    monkeypatch.setattr(_build.subprocess, "run", run)
    return state


@pytest.mark.parametrize("status", [1, None])
def test_a_binding_that_cannot_be_built_is_a_note(scratch_build, capsys, status):
    # a torch without CUDA libraries, or no C++ compiler
    built = _build._build_layers()
    assert built is not None
    scratch_build.status = status
    _touch(scratch_build.dir / "_layers.cpp")
    assert _build._build_layers() is None
    assert "does not build" in capsys.readouterr().err
    import os
    assert not os.path.exists(built)     # what was built from the older source is gone


def test_the_binding_is_rebuilt_for_another_torch(scratch_build, tmp_path, monkeypatch):
    import importlib.util
    import types
    torch_dir = tmp_path / "torch"
    torch_dir.mkdir()
    (torch_dir / "version.py").write_text("__version__ = '1'\n")
    monkeypatch.setattr(importlib.util, "find_spec",
                        lambda name: types.SimpleNamespace(origin=str(torch_dir / "__init__.py")))
    built = _build._build_layers()
    assert len(scratch_build.commands) == 1
    assert _build._build_layers() == built and len(scratch_build.commands) == 1
    (torch_dir / "version.py").write_text("__version__ = '2'\n")
    import os
    os.utime(torch_dir / "version.py", (0, 0))      # an archive's old file times
    assert _build._build_layers() == built and len(scratch_build.commands) == 2
    assert _build._build_layers() == built and len(scratch_build.commands) == 2


def _touch(path):
    import os
    import time
    os.utime(path, (time.time() + 100,) * 2)
