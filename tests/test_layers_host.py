"""Host-side checks of the layer operators' C ABI (no GPU): every refusal has
its status and detail and happens before a device is touched, empty problems
succeed, workspace sizes follow from sizes and alignment alone, and both
marshalling routes agree."""
import pytest

import dense_fp32_matrix_sgemm_gb300 as sg
from dense_fp32_matrix_sgemm_gb300 import _build

FAKE = 0x100000   # aligned, never dereferenced by these calls
F32, BF16, F16, E4M3 = 0, 1, 2, 3


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()
    return sg.load_library()


def linear(**kw):
    p = dict(dtype=BF16, M=32, N=16, K=8, X=FAKE, ldx=8, x_scale=0, W=FAKE, ldw=8, transW=1,
             w_scale=0, bias=0, activation=0, residual=0, ldr=0, out_dtype=BF16, Y=2 * FAKE, ldy=16)
    p.update(kw)
    return sg.sgemm_linear(**p, check=False)


@pytest.mark.parametrize("args,code", [
    (dict(dtype=4), 9), (dict(dtype=-1), 9), (dict(out_dtype=F16), 9), (dict(activation=5), 9),
    (dict(dtype=E4M3, out_dtype=F32, x_scale=FAKE, w_scale=FAKE), 9),
    (dict(transW=2), 4), (dict(dtype=E4M3, transW=0, ldw=16, x_scale=FAKE, w_scale=FAKE), 4),
    (dict(M=-1), 1), (dict(N=1 << 31), 1), (dict(K=-3), 1),
    (dict(ldx=7), 2), (dict(ldw=7), 2), (dict(transW=0, ldw=15), 2), (dict(ldy=15), 2),
    (dict(residual=FAKE, ldr=15), 2), (dict(preact=FAKE, ldp=15), 2), (dict(ldx=1 << 40), 2),
    (dict(residual=2 * FAKE, ldr=17), 2),
    (dict(X=0), 3), (dict(W=0), 3), (dict(Y=0), 3), (dict(X=FAKE + 1), 3), (dict(bias=FAKE + 1), 3),
    (dict(x_scale=FAKE), 3), (dict(dtype=E4M3), 3), (dict(dtype=E4M3, x_scale=FAKE), 3),
    (dict(dtype=E4M3, x_scale=FAKE, w_scale=FAKE + 2), 3),
    (dict(X=FAKE + 2), 8),                                   # needs a copy with aligned rows
    (dict(dtype=F32, out_dtype=F32), 8),                     # needs the split planes
    (dict(X=FAKE + 2, workspace=FAKE + 16, workspace_bytes=1 << 20), 8),
])
def test_linear_refusals(args, code):
    assert linear(**args) == code, sg.last_error()
    assert sg.last_error() != ""


def test_linear_workspace_follows_alignment():
    size = sg.linear_workspace_size
    assert size(BF16, 32, 16, 8, FAKE, 8, FAKE, 8, 1) == 0
    assert size(BF16, 32, 16, 8, FAKE + 2, 8, FAKE, 8, 1) == 32 * 128
    assert size(BF16, 32, 16, 7, FAKE, 7, FAKE, 7, 1) == 32 * 128 + 16 * 128
    assert size(BF16, 32, 15, 8, FAKE, 8, FAKE, 15, 0) == 8 * 128     # a K x N weight
    assert size(E4M3, 32, 16, 129, FAKE, 129, FAKE, 144, 1) == 32 * 256
    assert size(BF16, 2, 16, 7, FAKE, 7, FAKE, 7, 1) == 0             # few rows: any alignment
    assert size(F32, 16, 64, 64, FAKE, 64, FAKE, 64, 1) == 0
    # f32: three bf16 planes of both operands, rows padded to 64 elements
    assert size(F32, 32, 64, 65, FAKE, 65, FAKE, 65, 1) == 3 * 2 * 128 * (32 + 64)
    assert size(F32, 32, 64, 65, FAKE, 65, FAKE, 64, 0) == 3 * 2 * 128 * 32 + \
        (3 * 2 * 64 * 65 + 255) // 256 * 256
    for empty in ((0, 16, 8), (32, 0, 8), (32, 16, 0), (-1, 16, 8)):
        assert size(BF16, *empty, FAKE, 8, FAKE, 8, 1) == 0


def backward(**kw):
    p = dict(dtype=F16, M=32, N=16, K=8, dY=FAKE, lddy=16, Z=FAKE, ldz=16, activation=2, X=FAKE,
             ldx=8, W=FAKE, ldw=8, transW=1, dX=2 * FAKE, lddx=8, dW=3 * FAKE, lddw=8, db=4 * FAKE,
             workspace=5 * FAKE, workspace_bytes=1 << 30)
    p.update(kw)
    return sg.sgemm_linear_backward(**p, check=False)


@pytest.mark.parametrize("args,code", [
    (dict(dtype=E4M3), 9), (dict(activation=-1), 9), (dict(transW=3), 4), (dict(M=-1), 1),
    (dict(lddy=15), 2), (dict(ldz=15), 2), (dict(ldx=7), 2), (dict(ldw=7), 2), (dict(lddx=7), 2),
    (dict(lddw=7), 2), (dict(transW=0, ldw=16, lddw=15), 2),
    (dict(dY=0), 3), (dict(Z=0), 3), (dict(X=0), 3), (dict(W=0), 3), (dict(dX=FAKE + 1), 3),
    (dict(db=FAKE + 1), 3), (dict(workspace=0), 8), (dict(workspace_bytes=64), 8),
    (dict(workspace=FAKE + 8), 8),
])
def test_linear_backward_refusals(args, code):
    assert backward(**args) == code, sg.last_error()


def test_linear_backward_asks_only_for_what_it_reads():
    # nothing to compute is a no-op; K = 0 leaves db only
    assert backward(dX=0, dW=0, db=0) == 0
    assert backward(M=0, N=0, K=0) == 0
    assert sg.linear_backward_workspace_size(F16, 0, 16, 8, 0, 16, 2, 0, 8, 0, 8, 1) == 0


def norm(**kw):
    p = dict(dtype=BF16, rows=4, D=64, X=FAKE, ldx=64, residual=FAKE, ldr=64, weight=FAKE, eps=1e-6,
             S=2 * FAKE, lds=64, Y=3 * FAKE, ldy=64)
    p.update(kw)
    return sg.sgemm_add_rmsnorm(**p, check=False)


@pytest.mark.parametrize("args,code", [
    (dict(dtype=E4M3), 9), (dict(rows=-1), 1), (dict(D=1 << 31), 1), (dict(ldx=63), 2),
    (dict(ldr=63), 2), (dict(lds=63), 2), (dict(ldy=63), 2), (dict(X=0), 3), (dict(Y=0), 3),
    (dict(weight=0), 3), (dict(Y=3 * FAKE + 1), 3), (dict(q_scale=FAKE + 2), 3),
    (dict(rstd=FAKE + 1), 3),
])
def test_add_rmsnorm_refusals(args, code):
    assert norm(**args) == code, sg.last_error()


@pytest.mark.parametrize("args,code", [
    (dict(dtype=7), 9), (dict(rows=-2), 1), (dict(dY=0), 3), (dict(S=0), 3), (dict(rstd=0), 3),
    (dict(weight=0), 3), (dict(dX=0), 3), (dict(lddx=3), 2), (dict(dS=FAKE, ldds=3), 2),
    (dict(workspace=0), 8), (dict(workspace_bytes=100), 8),
])
def test_add_rmsnorm_backward_refusals(args, code):
    p = dict(dtype=F32, rows=4, D=64, dY=FAKE, lddy=64, S=FAKE, lds=64, rstd=FAKE, weight=FAKE, dS=0,
             ldds=0, dX=2 * FAKE, lddx=64, dweight=3 * FAKE, workspace=4 * FAKE,
             workspace_bytes=1 << 20)
    p.update(args)
    assert sg.sgemm_add_rmsnorm_backward(**p, check=False) == code, sg.last_error()


@pytest.mark.parametrize("args,code", [
    (dict(dtype=E4M3), 9), (dict(rows=-2), 1), (dict(X=0), 3), (dict(Q=0), 3), (dict(scale=0), 3),
    (dict(ldx=3), 2), (dict(ldq=3), 2),
])
def test_quantize_rows_refusals(args, code):
    p = dict(dtype=F32, rows=4, D=64, X=FAKE, ldx=64, Q=FAKE, ldq=64, scale=FAKE)
    p.update(args)
    assert sg.sgemm_quantize_rows(**p, check=False) == code, sg.last_error()


def test_empty_problems_need_no_device():
    assert linear(M=0) == 0 and linear(N=0, X=0, W=0, Y=0) == 0
    assert norm(rows=0) == 0 and norm(D=0) == 0
    assert sg.sgemm_quantize_rows(F32, 0, 8, 0, 8, 0, 8, 0) == 0
    assert sg.sgemm_add_rmsnorm_backward(F32, 0, 8, 0, 8, 0, 8, 0, 0, 0, 0, 0, 8, 0) == 0
    assert sg.add_rmsnorm_backward_workspace_size(F32, 0, 8) == 0


def test_status_nine_has_a_name():
    assert sg.status_string(9).startswith(sg.STATUS_NAMES[9])


def test_extension_marshalling_matches_ctypes(lib):
    if sg.marshalling() != "extension":
        pytest.skip("the _calls extension was not built here")
    from dense_fp32_matrix_sgemm_gb300 import _calls
    # every argument but the last differs, so a swapped pair changes the answer
    cases = {
        "sgemm_linear": (BF16, 5, 6, 7, FAKE, 6, 0, FAKE, 9, 1, 0, 0, 0, 0, 0, BF16, FAKE, 6, 0, 0, 0,
                         0, 0),
        "sgemm_linear_workspace_size": (BF16, 32, 16, 7, FAKE, 9, FAKE, 11, 1),
        "sgemm_linear_backward": (F16, 5, 6, 7, FAKE, 6, FAKE, 5, 2, FAKE, 7, FAKE, 7, 1, FAKE, 7,
                                  FAKE, 7, FAKE, FAKE, 1, 0),
        "sgemm_linear_backward_workspace_size": (F16, 32, 16, 7, FAKE, 17, 0, FAKE, 9, FAKE, 11, 1),
        "sgemm_add_rmsnorm": (F32, 5, 6, FAKE, 6, 0, 0, FAKE, 1e-6, FAKE, 5, FAKE, 6, 0, 0, 0),
        "sgemm_add_rmsnorm_backward": (F32, 5, 6, FAKE, 6, FAKE, 6, FAKE, FAKE, 0, 0, FAKE, 6, FAKE,
                                       FAKE, 1, 0),
        "sgemm_add_rmsnorm_backward_workspace_size": (F32, 5, 6),
        "sgemm_quantize_rows": (F32, 5, 6, FAKE, 6, FAKE, 5, FAKE, 0),
    }
    assert sorted(cases) == sorted(sg.LAYER_ENTRIES)
    for name, args in cases.items():
        via_ctypes = getattr(lib, name)(*args)
        detail = sg.last_error()
        assert via_ctypes != 0, name
        assert getattr(_calls, name)(*args) == via_ctypes, name
        assert sg.last_error() == detail, name


def test_torch_level_refusals():
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 8)
    with pytest.raises(TypeError):
        sg.linear(x, torch.zeros(3, 8))                       # not on a GPU
    with pytest.raises(TypeError):
        sg.linear(x.double(), torch.zeros(3, 8))
    with pytest.raises(TypeError):
        sg.quantize_rows(x.to(torch.int32))
    with pytest.raises(TypeError):
        sg.add_rmsnorm(x, torch.ones(8))
