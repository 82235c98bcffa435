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
