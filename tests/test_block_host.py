"""Host-side checks of the gated block's C ABI and torch functions (no GPU): every refusal has
its status and detail and happens before a device is touched, empty problems succeed, and
workspace sizes follow from sizes and alignment alone."""
import pytest

import dense_fp32_matrix_sgemm_gb300 as sg
from dense_fp32_matrix_sgemm_gb300 import _build

FAKE = 0x100000   # aligned, never dereferenced by these calls
F32, BF16, F16, E4M3 = 0, 1, 2, 3


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()
    return sg.load_library()


def gated(**kw):
    p = dict(dtype=BF16, M=32, N=16, K=8, X=FAKE, ldx=8, x_scale=0, Wg=FAKE, ldwg=8, gate_scale=0,
             Wu=FAKE, ldwu=8, up_scale=0, transW=1, bias_gate=0, bias_up=0, activation=4,
             out_dtype=BF16, H=2 * FAKE, ldh=16)
    p.update(kw)
    return sg.sgemm_gated_linear(**p, check=False)


SCALES = dict(x_scale=FAKE, gate_scale=FAKE, up_scale=FAKE)


@pytest.mark.parametrize("args,code", [
    (dict(dtype=4), 9), (dict(dtype=-1), 9), (dict(out_dtype=F16), 9), (dict(activation=5), 9),
    (dict(dtype=E4M3, out_dtype=F32, **SCALES), 9), (dict(transW=2), 4),
    (dict(dtype=E4M3, transW=0, ldwg=16, ldwu=16, **SCALES), 4),
    (dict(M=-1), 1), (dict(N=(1 << 29) + 1), 1), (dict(K=-3), 1), (dict(K=1 << 31), 1),
    (dict(ldx=7), 2), (dict(ldwg=7), 2), (dict(ldwu=7), 2), (dict(transW=0, ldwg=16, ldwu=15), 2),
    (dict(ldh=15), 2), (dict(preact_gate=FAKE, ldpg=15), 2), (dict(preact_up=FAKE, ldpu=15), 2),
    (dict(X=0), 3), (dict(Wg=0), 3), (dict(Wu=0), 3), (dict(H=0), 3), (dict(H=FAKE + 1), 3),
    (dict(bias_gate=FAKE + 1), 3), (dict(bias_up=FAKE + 1), 3), (dict(x_scale=FAKE), 3),
    (dict(up_scale=FAKE), 3), (dict(dtype=E4M3), 3), (dict(dtype=E4M3, x_scale=FAKE, gate_scale=FAKE), 3),
    (dict(dtype=E4M3, x_scale=FAKE, gate_scale=FAKE + 2, up_scale=FAKE), 3),
    (dict(X=FAKE + 2), 8), (dict(Wu=FAKE + 2), 8), (dict(dtype=F32, out_dtype=F32), 8),
    (dict(X=FAKE + 2, workspace=FAKE + 16, workspace_bytes=1 << 20), 8),
])
def test_gated_linear_refusals(args, code):
    assert gated(**args) == code, sg.last_error()
    assert sg.last_error() != ""


def test_gated_linear_workspace_follows_alignment():
    size = sg.gated_linear_workspace_size
    assert size(BF16, 32, 16, 8, FAKE, 8, FAKE, 8, FAKE, 8, 1) == 0
    assert size(BF16, 32, 16, 8, FAKE + 2, 8, FAKE, 8, FAKE, 8, 1) == 32 * 128
    assert size(BF16, 32, 16, 7, FAKE, 7, FAKE, 7, FAKE, 8, 1) == 32 * 128 + 16 * 128
    assert size(BF16, 1, 16, 7, FAKE, 7, FAKE, 7, FAKE, 7, 1) == 0     # few rows: any alignment
    assert size(BF16, 1, 15, 8, FAKE, 8, FAKE, 15, FAKE, 15, 0) == 2 * 8 * 128   # K x N: never few
    # f32: three bf16 planes of all three matrices
    assert size(F32, 32, 64, 65, FAKE, 65, FAKE, 65, FAKE, 65, 1) == 3 * 2 * 128 * (32 + 64 + 64)
    assert size(F32, 16, 64, 64, FAKE, 64, FAKE, 64, FAKE, 64, 1) == 0
    for empty in ((0, 16, 8), (32, 0, 8), (32, 16, 0), (-1, 16, 8)):
        assert size(BF16, *empty, FAKE, 8, FAKE, 8, FAKE, 8, 1) == 0


def backward(**kw):
    p = dict(dtype=F16, M=32, N=16, K=8, dH=FAKE, lddh=16, Zg=FAKE, ldzg=16, Zu=FAKE, ldzu=16,
             activation=2, X=FAKE, ldx=8, Wg=FAKE, ldwg=8, Wu=FAKE, ldwu=8, transW=1, dX=2 * FAKE,
             lddx=8, dWg=3 * FAKE, lddwg=8, dWu=4 * FAKE, lddwu=8, db_gate=5 * FAKE, db_up=6 * FAKE,
             workspace=7 * FAKE, workspace_bytes=1 << 30)
    p.update(kw)
    return sg.sgemm_gated_linear_backward(**p, check=False)


@pytest.mark.parametrize("args,code", [
    (dict(dtype=E4M3), 9), (dict(activation=-1), 9), (dict(transW=3), 4), (dict(M=-1), 1),
    (dict(N=1 << 30), 1), (dict(lddh=15), 2), (dict(ldzg=15), 2), (dict(ldzu=15), 2),
    (dict(ldx=7), 2), (dict(ldwg=7), 2), (dict(ldwu=7), 2), (dict(lddx=7), 2), (dict(lddwg=7), 2),
    (dict(lddwu=7), 2), (dict(dH=0), 3), (dict(Zg=0), 3), (dict(Zu=0), 3), (dict(X=0), 3),
    (dict(Wg=0), 3), (dict(Wu=0), 3), (dict(dX=FAKE + 1), 3), (dict(db_up=FAKE + 1), 3),
    (dict(workspace=0), 8), (dict(workspace_bytes=64), 8), (dict(workspace=FAKE + 8), 8),
    (dict(activation=0, Zg=0), 3),
])
def test_gated_linear_backward_refusals(args, code):
    assert backward(**args) == code, sg.last_error()


def test_gated_linear_backward_asks_only_for_what_it_reads():
    assert backward(dX=0, dWg=0, dWu=0, db_gate=0, db_up=0) == 0
    assert backward(M=0, N=0, K=0) == 0
    assert sg.gated_linear_backward_workspace_size(F16, 0, 16, 8, 0, 8, 0, 8, 0, 8, 1) == 0
    assert backward(dX=0, Wg=0, Wu=0, workspace_bytes=64) == 8      # no weights without dX
    assert backward(dWg=0, dWu=0, X=0, workspace_bytes=64) == 8


@pytest.mark.parametrize("args,code", [
    (dict(dtype=E4M3), 9), (dict(rows=-1), 1), (dict(D=1 << 31), 1), (dict(ldx=63), 2),
    (dict(ldr=63), 2), (dict(lds=63), 2), (dict(ldy=63), 2), (dict(X=0), 3), (dict(Y=0), 3),
    (dict(weight=0), 3), (dict(bias=FAKE + 1), 3), (dict(q_scale=FAKE + 2), 3),
    (dict(mean=FAKE + 1), 3), (dict(rstd=FAKE + 1), 3),
])
def test_add_layernorm_refusals(args, code):
    p = dict(dtype=BF16, rows=4, D=64, X=FAKE, ldx=64, residual=FAKE, ldr=64, weight=FAKE, bias=FAKE,
             eps=1e-6, S=2 * FAKE, lds=64, Y=3 * FAKE, ldy=64)
    p.update(args)
    assert sg.sgemm_add_layernorm(**p, check=False) == code, sg.last_error()


@pytest.mark.parametrize("args,code", [
    (dict(dtype=7), 9), (dict(rows=-2), 1), (dict(dY=0), 3), (dict(S=0), 3), (dict(mean=0), 3),
    (dict(rstd=0), 3), (dict(weight=0), 3), (dict(dX=0), 3), (dict(dbias=FAKE + 2), 3),
    (dict(lddx=3), 2), (dict(dS=FAKE, ldds=3), 2), (dict(workspace=0), 8),
    (dict(workspace_bytes=100), 8), (dict(dweight=0, workspace_bytes=100), 8),
])
def test_add_layernorm_backward_refusals(args, code):
    p = dict(dtype=F32, rows=4, D=64, dY=FAKE, lddy=64, S=FAKE, lds=64, mean=FAKE, rstd=FAKE,
             weight=FAKE, dS=0, ldds=0, dX=2 * FAKE, lddx=64, dweight=3 * FAKE, dbias=4 * FAKE,
             workspace=5 * FAKE, workspace_bytes=1 << 20)
    p.update(args)
    assert sg.sgemm_add_layernorm_backward(**p, check=False) == code, sg.last_error()


def clip(dtypes=(F32, BF16), sizes=(10, 20), X=(FAKE, 2 * FAKE), Y=(FAKE, 2 * FAKE), max_norm=1.0,
         eps=1e-6, norm=4 * FAKE, **kw):
    return sg.sgemm_clip_grad_norm(dtypes, sizes, X, Y, max_norm, eps, norm, check=False, **kw)


NAN = float("nan")


@pytest.mark.parametrize("args,code", [
    (dict(dtypes=(F32, E4M3)), 9), (dict(sizes=(10, -1)), 1), (dict(sizes=((1 << 40) + 1, 1)), 1),
    (dict(X=(FAKE, 0)), 3), (dict(Y=(FAKE, 0)), 3), (dict(X=(FAKE + 2, 2 * FAKE)), 3),
    (dict(Y=(FAKE, 2 * FAKE + 1)), 3), (dict(norm=FAKE + 2), 3),
    (dict(max_norm=-1.0), 1), (dict(max_norm=NAN), 1), (dict(eps=-1e-3), 1), (dict(eps=NAN), 1),
    # the same tensor twice, results that overlap one another or another tensor
    (dict(dtypes=(F32, F32), X=(FAKE, FAKE), Y=(FAKE, FAKE)), 3),
    (dict(X=(FAKE, FAKE + 32), Y=(FAKE, FAKE + 32)), 3),
    (dict(Y=(3 * FAKE, 3 * FAKE + 36)), 3), (dict(Y=(2 * FAKE + 36, 5 * FAKE)), 3),
    (dict(Y=(FAKE + 4, 5 * FAKE)), 3),
    # neighbours are not overlaps, nor are inputs that share memory
    (dict(X=(FAKE, FAKE + 40), Y=(FAKE, FAKE + 40)), 8), (dict(Y=(2 * FAKE + 40, 5 * FAKE)), 8),
    (dict(dtypes=(F32, F32), X=(FAKE, FAKE), Y=(3 * FAKE, 5 * FAKE)), 8),
    (dict(Y=None), 8), (dict(workspace=FAKE + 8, workspace_bytes=1 << 20), 8),
])
def test_clip_grad_norm_refusals(args, code):
    assert clip(**args) == code, sg.last_error()


def test_clip_grad_norm_workspace_and_empty():
    size = sg.clip_grad_norm_workspace_size
    assert size([F32], [5]) == size([F32] * 1000, [5] * 1000) > 0
    assert size([F32] * 1001, [5] * 1001) == 2 * size([F32], [5])
    assert size([F32] * 1001, [5] * 1000 + [0]) == size([F32], [5])
    assert size([E4M3], [5]) == 0
    assert clip(Y=None, norm=0) == 0                    # nothing to compute
    with pytest.raises(ValueError):
        sg.sgemm_clip_grad_norm([F32], [1, 2], [FAKE], None, 1.0, 0.0, FAKE)


def test_empty_problems_need_no_device():
    assert gated(M=0) == 0 and gated(N=0, X=0, Wg=0, Wu=0, H=0) == 0
    assert sg.sgemm_add_layernorm(F32, 0, 8, 0, 8, 0, 0, 0, 0, 1e-5, 0, 0, 0, 8) == 0
    assert sg.sgemm_add_layernorm_backward(F32, 0, 8, 0, 8, 0, 8, 0, 0, 0, 0, 0, 0, 8, 0, 0) == 0
    assert sg.add_layernorm_backward_workspace_size(F32, 0, 8) == 0


def test_torch_level_refusals():
    torch = pytest.importorskip("torch")
    x, w = torch.zeros(4, 8), torch.zeros(3, 8)
    with pytest.raises(TypeError):
        sg.gated_linear(x, w, w)                              # not on a GPU
    with pytest.raises(ValueError):
        sg.gated_linear(x, w, w, activation="tanh")
    with pytest.raises(TypeError):
        sg.gated_linear(x, w, w, out_dtype=torch.float16)
    with pytest.raises(TypeError):
        sg.add_layernorm(x, torch.ones(8))
    with pytest.raises(TypeError):
        sg.add_layernorm_backward(x, x, torch.ones(4), torch.ones(4), torch.ones(8))
    with pytest.raises(TypeError):
        sg.clip_grad_norm([x], 1.0)
    with pytest.raises(TypeError):
        sg.grad_norm([x.double()])
    with pytest.raises(TypeError):
        sg.grad_norm([3.0])
    with pytest.raises(ValueError):
        sg.grad_norm([])
    with pytest.raises(TypeError):
        sg.clip_grad_norm([x], 1.0, out=5)
    with pytest.raises(TypeError):
        sg.clip_grad_norm([x], "much")
