"""The gated block's operators on the GPU against plain formulas in 64 bits.

Tolerances are derived as in test_layers_gpu.py (its helpers are used), with EPS = 2^-23, u the
output's unit roundoff and, for a product, t its bound (product_tol and 4 EPS of the absolute
sum):
  * gated: h = act(zg) zu errs by (1.2 tg + 16 EPS |zg|) (|zu| + tu) + |act(zg)| tu and u |h|;
  * its gradients: act' and act are evaluated to 32 EPS (1 + |zg|) of what they multiply, and
    dZ is rounded once (u) for the 16-bit types;
  * layer norm: a sum of d terms errs by r = (d / 32 + 72) EPS of the absolute sum.  The first
    mean errs by r mean|s|; the second sum, of what is left, by r of a mean|c| that is larger
    by no more than that; s itself by EPS |s| / 2;
  * clipping: a thread's fp32 sum of up to 64 squares in two chains errs by 33 EPS / 2 of it,
    which halves in the square root; the sums of those are in 64 bits.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import dense_fp32_matrix_sgemm_gb300 as sg  # noqa: E402
from test_layers_gpu import (EPS, TINY, TYPES, UNIT, act, act_grad, check, codes_ok, gen,  # noqa: E402
                             normal, product_tol, strided)


@pytest.fixture(scope="module", autouse=True)
def no_pipeline_errors():
    sg.device_status(reset=True)
    yield
    assert sg.device_status(reset=True) == 0


# ------------------------------------------------------------------ gated_linear


def run_gated(m, n, k, t, name="silu", bias=False, preact=False, w_kn=False, pad=0, offset=0,
              out_dtype=None):
    g = gen(7 * m + 11 * n + 13 * k)
    e4m3 = t == "e4m3"
    dtype = (out_dtype or torch.bfloat16) if e4m3 else TYPES[t]
    x = normal(g, m, k)
    ws = [normal(g, n, k, std=max(k, 1) ** -0.5) for _ in range(2)]
    kw = {}
    if e4m3:
        x, kw["x_scale"] = sg.quantize_rows(x)
        ws[0], kw["gate_scale"] = sg.quantize_rows(ws[0])
        ws[1], kw["up_scale"] = sg.quantize_rows(ws[1])
    else:
        x, ws = x.to(dtype), [w.to(dtype) for w in ws]
    bs = [normal(g, n, dtype=dtype) if bias else None for _ in range(2)]
    stored = [strided(w.t().contiguous(), pad, offset).t() if w_kn else strided(w, pad, offset)
              for w in ws]
    buf = torch.full((m * (n + pad) + offset + 64,), float("nan"), dtype=dtype, device="cuda")
    out = buf[offset:offset + m * (n + pad)].view(m, n + pad)[:, :n]
    got = sg.gated_linear(strided(x, pad, offset), *stored, *bs, activation=name,
                          save_preact=preact, out=out, out_dtype=dtype if e4m3 else None, **kw)
    torch.cuda.synchronize()
    h = got[0] if preact else got
    xd = x.double()
    if e4m3:
        xd = xd * kw["x_scale"].double()[:, None]
    z, tol = [], []
    for w, b, s in zip(ws, bs, ("gate_scale", "up_scale")):
        wd = w.double() * kw[s].double()[:, None] if e4m3 else w.double()
        zd, S = xd @ wd.t(), xd.abs() @ wd.abs().t()
        if bias:
            zd, S = zd + b.double(), S + b.double().abs()
        z.append(zd)
        tol.append(product_tol(S, k, torch.float32 if t == "f32" else dtype) + 4 * EPS * S)
    a = act(z[0], name)
    hd = a * z[1]
    htol = ((1.2 * tol[0] + 16 * EPS * z[0].abs()) * (z[1].abs() + tol[1]) + a.abs() * tol[1] +
            (UNIT[dtype] + 4 * EPS) * hd.abs() + TINY[dtype])
    what = f"{m}x{n}x{k} {t} {name} bias={bias} preact={preact} w_kn={w_kn} pad={pad}+{offset}"
    check(h, hd, htol, what)
    if preact:
        for i in range(2):
            check(got[1 + i], z[i], tol[i] + UNIT[dtype] * z[i].abs() + TINY[dtype], what + f" z{i}")
    if pad:
        full = buf[offset:offset + m * (n + pad)].view(m, n + pad)
        assert torch.isnan(full[:, n:]).all(), "padding columns were written"
    assert torch.isnan(buf[offset + m * (n + pad):]).all() and torch.isnan(buf[:offset]).all()


# one row and few rows (CUDA cores), ragged tiles, split K over clusters (few tiles), one wave
# and several waves of each tile width
SIZES = [(1, 1, 1), (1, 300, 257), (1, 2048, 1024), (2, 77, 640), (3, 1000, 8), (4, 129, 4096),
         (5, 64, 64), (16, 520, 200), (17, 96, 1000), (33, 500, 520), (64, 512, 2048),
         (127, 255, 129), (128, 64, 64), (129, 129, 4104), (300, 1, 72), (513, 320, 16),
         (1290, 515, 136), (2300, 1020, 200), (4610, 2052, 40)]


@pytest.mark.parametrize("t", ["f32", "bf16", "f16", "e4m3"])
@pytest.mark.parametrize("m,n,k", SIZES)
def test_gated_sizes(m, n, k, t):
    run_gated(m, n, k, t, "silu", bias=True, preact=True)


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("m,n,k", SIZES)
def test_gated_weights_stored_by_columns(m, n, k, t):
    run_gated(m, n, k, t, "gelu", w_kn=True)


@pytest.mark.parametrize("t", ["f32", "bf16", "f16", "e4m3"])
@pytest.mark.parametrize("name", ["none", "relu", "gelu", "gelu_erf", "silu"])
@pytest.mark.parametrize("m", [1, 70, 1300])
def test_gated_activations(m, name, t):
    run_gated(m, 520, 320, t, name, bias=True, preact=True)
    run_gated(m, 519, 320, t, name)


@pytest.mark.parametrize("t", ["f32", "bf16", "f16", "e4m3"])
@pytest.mark.parametrize("pad,offset", [(8, 0), (3, 0), (0, 1), (5, 3), (16, 16)])
@pytest.mark.parametrize("m", [1, 3, 70, 700])
def test_gated_strides_and_offsets(m, pad, offset, t):
    run_gated(m, 344, 200, t, "relu", bias=True, preact=True, pad=pad, offset=offset)
    run_gated(m, 171, 201, t, "none", pad=pad, offset=offset)
    if t != "e4m3":
        run_gated(m, 171, 201, t, "none", pad=pad, offset=offset, w_kn=True)


# few rows: f32 weights by columns, and both sides of the rows that go to the CUDA cores
@pytest.mark.parametrize("m", [1, 2, 3, 4, 5, 8, 9, 16, 17])
@pytest.mark.parametrize("n,k", [(1, 1), (7, 300), (132, 64), (256, 512), (1000, 257), (4100, 129),
                                 (2052, 2000)])
def test_gated_few_rows_by_columns(m, n, k):
    run_gated(m, n, k, "f32", "silu", bias=True, preact=True, w_kn=True)
    run_gated(m, n, k, "f32", "gelu", w_kn=True, pad=8)
    run_gated(m, n, k, "f32", "relu", preact=True, w_kn=True, pad=3, offset=1)


@pytest.mark.parametrize("t", ["bf16", "f16", "e4m3"])
@pytest.mark.parametrize("m", [1, 2, 3, 4, 5, 7, 8, 9])
@pytest.mark.parametrize("n,k", [(40, 1000), (2048, 1024), (2048, 2048), (2050, 1031), (4104, 2048)])
def test_gated_few_rows(m, n, k, t):
    run_gated(m, n, k, t, "silu", bias=True, preact=True)
    run_gated(m, n, k, t, "gelu_erf", pad=3, offset=1)


# tiles of every width that the rounds of SMs call for, whole and in parts of K, of few and many rows
@pytest.mark.parametrize("t", ["bf16", "e4m3"])
@pytest.mark.parametrize("m,n,k", [(64, 8192, 264), (9, 11264, 136), (100, 300, 4096), (8, 4096, 2208),
                                   (130, 1369, 1001), (33, 16000, 72), (40, 1216, 200), (70, 2432, 129),
                                   (128, 24, 2048), (2000, 600, 264), (120, 19000, 64)])
def test_gated_tile_widths(m, n, k, t):
    run_gated(m, n, k, t, "silu", bias=True, preact=True)
    run_gated(m, n, k, t, "gelu")
    run_gated(m, n, k, t, "none", preact=True, pad=8)


# long sums: tiles with K split over clusters, whole waves followed by a split rest
@pytest.mark.parametrize("m,n,k,t", [(1024, 1024, 8192, "f32"), (1000, 1025, 8200, "bf16"),
                                     (1020, 1020, 16400, "e4m3"), (2560, 1280, 2600, "f32"),
                                     (2500, 1270, 8008, "f16")])
def test_gated_long_sums(m, n, k, t):
    run_gated(m, n, k, t, "gelu", bias=True, preact=True)
    if t != "e4m3":
        run_gated(m, n, k, t, "relu", w_kn=True)


@pytest.mark.parametrize("t", ["bf16", "e4m3"])
@pytest.mark.parametrize("m", [1, 2, 3, 4, 5])
@pytest.mark.parametrize("n,k", [(1024, 2048), (1028, 2064), (1025, 2051)])
def test_gated_few_rows_of_either_kernel(n, k, m, t):
    run_gated(m, n, k, t, "silu", bias=True, preact=True)


def test_gated_e4m3_to_f16():
    run_gated(2, 96, 256, "e4m3", out_dtype=torch.float16)
    run_gated(200, 500, 256, "e4m3", bias=True, preact=True, out_dtype=torch.float16)


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("m", [1, 200])
@pytest.mark.parametrize("w_kn", [False, True])
def test_gated_halves_of_one_matrix(w_kn, m, t):
    # a merged weight's halves: by rows, or (K x N storage) interleaved in the leading dimension
    g, dtype, n, k = gen(3), TYPES[t], 136, 72
    both = normal(g, 2 * n, k, dtype=dtype, std=k ** -0.5)
    x = normal(g, m, k, dtype=dtype)
    stored = both.t().contiguous().t() if w_kn else both
    h = sg.gated_linear(x, stored[:n], stored[n:])
    gate, up = both[:n].t().contiguous().t() if w_kn else both[:n].clone(), both[n:].clone()
    if w_kn:
        up = up.t().contiguous().t()
    assert torch.equal(h, sg.gated_linear(x, gate, up))


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("m", [1, 9, 300])
def test_gated_without_inputs(m, t):
    dtype, g = TYPES[t], gen(3)
    bg, bu = normal(g, 130, dtype=dtype), normal(g, 130, dtype=dtype)
    x, w = torch.empty(m, 0, dtype=dtype, device="cuda"), torch.empty(130, 0, dtype=dtype, device="cuda")
    h = sg.gated_linear(x, w, w, bg, bu, activation="relu")
    want = (bg.double().clamp(min=0) * bu.double()).expand(m, 130)
    check(h, want, 2 * UNIT[dtype] * want.abs() + TINY[dtype], "K = 0")
    assert not sg.gated_linear(x, w, w, bg).any()          # no bias of the factor: a factor of 0
    assert sg.gated_linear(x[:0], w, w, bg).shape == (0, 130)
    assert sg.gated_linear(x, w[:0], w[:0]).shape == (m, 0)


@pytest.mark.parametrize("t", ["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("m", [2, 100, 1500])
def test_gated_nan_and_infinity_stay_in_their_row(m, t):
    g = gen(4)
    x, wg, wu = normal(g, m, 256), normal(g, 150, 256, std=1 / 16), normal(g, 150, 256, std=1 / 16)
    kw = {}
    if t == "e4m3":
        x, kw["x_scale"] = sg.quantize_rows(x)
        wg, kw["gate_scale"] = sg.quantize_rows(wg)
        wu, kw["up_scale"] = sg.quantize_rows(wu)
        clean = sg.gated_linear(x, wg, wu, **kw)
        x.view(torch.uint8)[m // 2, 17] = 0x7f
    else:
        x, wg, wu = (v.to(TYPES[t]) for v in (x, wg, wu))
        clean = sg.gated_linear(x, wg, wu)
        x[m // 2, 17] = float("nan")
    h = sg.gated_linear(x, wg, wu, **kw)
    assert torch.isnan(h[m // 2]).all()
    keep = torch.arange(m, device="cuda") != m // 2
    assert torch.equal(h[keep], clean[keep])
    if t != "e4m3":
        # a weight's NaN stays in its feature
        x[m // 2, 17] = 0
        clean = sg.gated_linear(x, wg, wu)
        wu[7, 3] = float("nan")
        h = sg.gated_linear(x, wg, wu)
        assert torch.isnan(h[:, 7]).all()
        keep = torch.arange(150, device="cuda") != 7
        assert torch.equal(h[:, keep], clean[:, keep])


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("m", [1, 200])
def test_gated_streams_graph_and_workspace(m, t):
    g, dtype = gen(1), TYPES[t]
    x, wg, wu = (normal(g, *s, dtype=dtype, std=0.1) for s in ((m, 1000), (640, 1000), (640, 1000)))
    first = sg.gated_linear(x, wg, wu)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = sg.gated_linear(x, wg, wu, stream=side)
    raw = sg.gated_linear(x, wg, wu, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(first, other) and torch.equal(first, raw)
    need = sg.gated_linear_workspace_size(0 if t == "f32" else 1, m, 640, 1000, x.data_ptr(), 1000,
                                          wg.data_ptr(), 1000, wu.data_ptr(), 1000, 1)
    ws = torch.full((need + 256,), 7, dtype=torch.uint8, device="cuda")
    assert torch.equal(sg.gated_linear(x, wg, wu, workspace=ws[:need]), first)
    assert (ws[need:] == 7).all()
    graph, out = torch.cuda.CUDAGraph(), torch.empty_like(first)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        sg.gated_linear(x, wg, wu, out=out)
    x.mul_(0.5)
    want = sg.gated_linear(x, wg, wu)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


# ------------------------------------------------------------------ gated_linear_backward


def run_gated_backward(m, n, k, t, name="silu", w_kn=False, pad=0, offset=0):
    dtype = TYPES[t]
    g = gen(3 * m + 5 * n + 17 * k)
    x, wg, wu, zg, zu, dh = (normal(g, *s, dtype=dtype, std=std) for s, std in
                             (((m, k), 1), ((n, k), max(k, 1) ** -0.5), ((n, k), max(k, 1) ** -0.5),
                              ((m, n), 1.5), ((m, n), 1), ((m, n), 1)))
    stored = [strided(w.t().contiguous(), pad, offset).t() if w_kn else strided(w, pad, offset)
              for w in (wg, wu)]
    dx, dwg, dwu, dbg, dbu = sg.gated_linear_backward(
        strided(dh, pad, offset), strided(x, pad, offset), *stored, strided(zg, pad, offset),
        strided(zu, pad, offset), activation=name)
    torch.cuda.synchronize()
    G, U, D = zg.double(), zu.double(), dh.double()
    dz = [D * U * act_grad(G, name), D * act(G, name)]
    err = [32 * EPS * (D * U).abs() * (1 + G.abs()), 32 * EPS * D.abs() * (1 + G.abs())]
    u = UNIT[dtype]
    sums = [e.sum(0) for e in err]
    if t != "f32":
        err = [e + u * z.abs() + TINY[dtype] for e, z in zip(err, dz)]
    what = f"{m}x{n}x{k} {t} {name} w_kn={w_kn} pad={pad}+{offset}"
    X, W = x.double(), [wg.double(), wu.double()]
    want = dz[0] @ W[0] + dz[1] @ W[1]
    S = dz[0].abs() @ W[0].abs() + dz[1].abs() @ W[1].abs()
    e = err[0] @ W[0].abs() + err[1] @ W[1].abs()
    assert dx.shape == want.shape
    check(dx, want, product_tol(S, 2 * n, dtype) + e + u * want.abs() + TINY[dtype] + 1e-30,
          what + " dx")
    for i, got in enumerate((dwg, dwu)):
        want, S = dz[i].t() @ X, dz[i].t().abs() @ X.abs()
        assert got.shape == want.shape and (not w_kn or n == 1 or k == 1 or got.stride(0) == 1)
        check(got, want, product_tol(S, m, dtype) + err[i].t() @ X.abs() + u * want.abs() +
              TINY[dtype] + 1e-30, what + f" dw{i}")
    for i, got in enumerate((dbg, dbu)):
        want = dz[i].sum(0)
        check(got, want, (m + 8) * EPS / 2 * dz[i].abs().sum(0) + sums[i] + u * want.abs() +
              TINY[dtype], what + f" db{i}")


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("w_kn", [False, True])
@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (1, 300, 200), (3, 64, 520), (4, 1000, 72), (17, 96, 128),
                                   (64, 256, 512), (129, 257, 131), (500, 777, 301), (1000, 128, 1024),
                                   (4096, 264, 136), (2300, 1020, 264)])
def test_gated_backward_sizes(m, n, k, w_kn, t):
    run_gated_backward(m, n, k, t, "silu", w_kn)


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("name", ["none", "relu", "gelu", "gelu_erf", "silu"])
@pytest.mark.parametrize("m,pad,offset", [(2, 0, 0), (2, 3, 1), (200, 8, 0), (200, 0, 1), (200, 5, 2)])
def test_gated_backward_activations_and_strides(m, pad, offset, name, t):
    run_gated_backward(m, 136, 208, t, name, False, pad, offset)
    run_gated_backward(m, 135, 207, t, name, True, pad, offset)


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("m,n,k", [(9, 77, 130), (96, 64, 80), (301, 259, 130)])
def test_gated_backward_parts_give_the_same_bits(m, n, k, t):
    g = gen(23)
    dh, x, wg, wu, zg, zu = (normal(g, *s, dtype=TYPES[t]) for s in
                             ((m, n), (m, k), (n, k), (n, k), (m, n), (m, n)))
    full = sg.gated_linear_backward(dh, x, wg, wu, zg, zu)
    for need in range(1, 8):
        some = sg.gated_linear_backward(dh, x, wg, wu, zg, zu, need_dx=bool(need & 1),
                                        need_dw=bool(need & 2), need_db=bool(need & 4))
        for i, bit in enumerate((1, 2, 2, 4, 4)):
            if need & bit:
                assert torch.equal(some[i], full[i]), (need, i)
            else:
                assert some[i] is None


@pytest.mark.parametrize("t", ["f32", "bf16"])
def test_gated_backward_empty(t):
    d = TYPES[t]
    e = lambda *s: torch.ones(*s, dtype=d, device="cuda")  # noqa: E731
    back = lambda m, n, k: sg.gated_linear_backward(e(m, n), e(m, k), e(n, k), e(n, k), e(m, n),  # noqa: E731
                                                    e(m, n), activation="none")
    dx, dwg, dwu, dbg, dbu = back(0, 6, 5)
    assert dx.shape == (0, 5) and dwg.shape == dwu.shape == (6, 5)
    assert not dwg.any() and not dwu.any() and not dbg.any() and not dbu.any()
    dx, dwg, *_ = back(4, 0, 5)
    assert not dx.any() and dx.shape == (4, 5) and dwg.shape == (0, 5)
    dx, dwg, dwu, dbg, dbu = back(4, 6, 0)
    assert dx.shape == (4, 0) and torch.equal(dbg, 4 * e(6)) and torch.equal(dbu, 4 * e(6))


@pytest.mark.parametrize("m,n,k,t", [(500, 777, 301, "f32"), (1024, 520, 776, "bf16")])
def test_gated_backward_back_to_back_in_a_graph_and_on_another_stream(m, n, k, t):
    g, dtype = gen(37), TYPES[t]
    x, wg, wu, zg, zu, dh = (normal(g, *s, dtype=dtype) for s in
                             ((m, k), (n, k), (n, k), (m, n), (m, n), (m, n)))
    call = lambda **kw: sg.gated_linear_backward(dh, x, wg, wu, zg, zu, **kw)  # noqa: E731
    first = call()
    torch.cuda.synchronize()
    again = [call() for _ in range(4)]     # launches of one call behind another's
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again.append(call(stream=side))
    torch.cuda.synchronize()
    for got in again:
        assert all(torch.equal(a, b) for a, b in zip(first, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = [call() for _ in range(3)]
    dh.mul_(0.5)
    x.mul_(2)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    want = call()
    for got in out:
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("name", ["none", "gelu", "gelu_erf", "silu"])
def test_gated_gradient_against_differences(name):
    """As test_linear_gradient_against_differences: L = <dh, h> in 64 bits along each
    argument, 1e-5 of the norms' product."""
    g, step = gen(8), 1e-4
    m, n, k = 40, 72, 56
    x, wg, wu, bg, bu, dh = (normal(g, *s, std=std) for s, std in
                             (((m, k), 1), ((n, k), k ** -0.5), ((n, k), k ** -0.5), ((n,), 1), ((n,), 1),
                              ((m, n), 1)))
    _, zg, zu = sg.gated_linear(x, wg, wu, bg, bu, activation=name, save_preact=True)
    grads = sg.gated_linear_backward(dh, x, wg, wu, zg, zu, activation=name)

    def loss(x, wg, wu, bg, bu):
        return (dh.double() * act(x @ wg.t() + bg, name) * (x @ wu.t() + bu)).sum()

    p = [t.double() for t in (x, wg, wu, bg, bu)]
    for i, grad in enumerate(grads):
        v = torch.randn(p[i].shape, generator=g, device="cuda", dtype=torch.float64)
        plus, minus = list(p), list(p)
        plus[i], minus[i] = p[i] + step * v, p[i] - step * v
        diff = (loss(*plus) - loss(*minus)) / (2 * step)
        along = (grad.double() * v).sum()
        assert abs(float(diff - along)) <= 1e-5 * float(grad.double().norm() * v.norm()) + 1e-6, (name, i)


# ------------------------------------------------------------------ add_layernorm


NORM_SIZES = [(1, 1), (1, 4096), (3, 7), (5, 64), (9, 200), (33, 256), (40, 1001), (700, 4096),
              (2, 8192), (310, 8192), (2, 16384), (311, 16000), (2, 40000), (3, 9001), (5000, 72)]


def run_layernorm(rows, d, t, residual=True, bias=True, quantize=False, pad=0, offset=0, mean=0.0,
                  call=sg.add_layernorm):
    dtype = TYPES[t]
    g = gen(rows + 31 * d)
    x, r = normal(g, rows, d), normal(g, rows, d, dtype=dtype)
    x = (x + mean).to(dtype)
    w = (1 + normal(g, d, std=0.2)).to(dtype)
    b = normal(g, d, std=0.3, dtype=dtype) if bias else None
    got = call(strided(x, pad, offset), w, b, strided(r, pad, offset) if residual else None, eps=1e-5,
               quantize=quantize)
    torch.cuda.synchronize()
    s = x.double() + (r.double() if residual else 0)
    m = s.mean(1, keepdim=True)
    c = s - m
    rstd = 1 / torch.sqrt(c.square().mean(1, keepdim=True) + 1e-5)
    B = b.double() if bias else torch.zeros(d, dtype=torch.float64, device="cuda")
    y = c * rstd * w.double() + B
    rel = (d / 32 + 72) * EPS
    size, spread = s.abs().mean(1, keepdim=True), c.abs().mean(1, keepdim=True)
    mtol = 2 * EPS * m.abs() + EPS * size + rel * (spread + rel * size)
    rtol = rstd * (rel + 8 * EPS + EPS * (s * c).abs().mean(1, keepdim=True) * rstd ** 2 +
                   rel * (rel * size * rstd) ** 2)
    what = f"{rows}x{d} {t} residual={residual} bias={bias} quantize={quantize} pad={pad}+{offset} mean={mean}"
    check(got[-1], rstd[:, 0], rtol[:, 0], what + " rstd")
    check(got[-2], m[:, 0], mtol[:, 0] + TINY[torch.float32], what + " mean")
    check(got[-3], s, UNIT[dtype] * s.abs() + TINY[dtype], what + " s")
    ytol = (w.double().abs() * ((mtol + EPS * s.abs()) * rstd + c.abs() * rtol) +
            4 * EPS * (y.abs() + B.abs() + (c * rstd * w.double()).abs()))
    if quantize:
        q, scale = got[:2]
        want = y.abs().amax(1).clamp(min=1e-30) / 448
        stol = ytol.amax(1) / 448 + 8 * EPS * want
        check(scale, want, stol, what + " scale")
        # half a step of the code, and what y's own error moves it by
        exact = y / scale.double()[:, None]
        v = exact.abs().clamp(max=448.0)
        e = torch.floor(torch.log2(v.clamp(min=2.0 ** -6)))
        check(q, exact, 0.5 * 2.0 ** (e - 3) * (1 + 2.0 ** -20) + 2.0 ** -17 * v +
              ytol / scale.double()[:, None], what + " codes")
    else:
        check(got[0], y, ytol + UNIT[dtype] * y.abs() + TINY[dtype], what + " y")


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("quantize", [False, True])
@pytest.mark.parametrize("rows,d", NORM_SIZES)
def test_add_layernorm_sizes(rows, d, quantize, t):
    run_layernorm(rows, d, t, True, True, quantize)
    run_layernorm(rows, d, t, False, False, quantize)


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("quantize", [False, True])
@pytest.mark.parametrize("pad,offset", [(8, 0), (3, 0), (0, 1), (5, 3)])
def test_add_layernorm_strides(pad, offset, quantize, t):
    run_layernorm(20, 512, t, True, True, quantize, pad, offset)
    run_layernorm(400, 520, t, False, True, quantize, pad, offset)


# accesses of 8 and 4 bytes and of one element, groups of every width
@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,d", [(3, 12), (40, 1002), (320, 1004), (330, 6428), (500, 6426), (310, 6427),
                                    (2, 12004), (2, 12002), (3, 12001), (1, 16386)])
def test_add_layernorm_accesses(rows, d, t):
    run_layernorm(rows, d, t, True, True, False)
    run_layernorm(rows, d, t, True, True, True)
    run_layernorm_backward(rows, d, t, True)


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("pad,offset", [(4, 0), (2, 0), (0, 2), (0, 4), (6, 2)])
def test_add_layernorm_accesses_by_alignment(pad, offset, t):
    run_layernorm(20, 512, t, True, True, False, pad, offset)
    run_layernorm(20, 512, t, True, True, True, pad, offset)
    run_layernorm_backward(400, 520, t, True, pad, offset)


@pytest.mark.parametrize("rows,d", [(4, 64), (9, 1001), (3, 4096), (400, 4096), (2, 40000)])
@pytest.mark.parametrize("mean", [1e2, -1e4])
def test_add_layernorm_keeps_a_large_mean_out_of_the_variance(rows, d, mean):
    run_layernorm(rows, d, "f32", False, True, mean=mean)


@pytest.mark.parametrize("d", [1, 41, 47, 61, 1001, 4096, 40000])
def test_add_layernorm_of_equal_values(d):
    # The first mean is off by r |v|, the corrected one by r of that: below half an ulp, so it
    # is v again.  What the variance is off by, r (r v)^2, halves in rstd.
    rel = (d / 32 + 72) * EPS
    for value in (0.1, -3.7, 12345.678):
        x = torch.full((3, d), value, device="cuda")
        b = normal(gen(d), d)
        y, _, mean, rstd = sg.add_layernorm(x, torch.ones(d, device="cuda"), b, eps=1e-5)
        assert torch.equal(mean, x[:, 0]), value
        want = b.double().expand(3, d)
        check(y, want, rel * rel * abs(value) * 320 + EPS * want.abs(), "y")
        root = torch.full((3,), 1e-5 ** -0.5, dtype=torch.float64, device="cuda")
        check(rstd, root, root * (rel * (rel * value) ** 2 / 1e-5 + 4 * EPS), "rstd")


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("d", [256, 40000])
def test_add_layernorm_special_rows(d, t):
    dtype = TYPES[t]
    x = normal(gen(0), 6, d, dtype=dtype)
    w, b = torch.ones(d, dtype=dtype, device="cuda"), torch.zeros(d, dtype=dtype, device="cuda")
    clean = sg.add_layernorm(x, w, b)[0]
    x[1] = 0
    x[2, 5] = float("nan")
    x[3, 7] = float("inf")
    y, s, mean, rstd = sg.add_layernorm(x, w, b)
    q, scale, _, _, _ = sg.add_layernorm(x, w, b, quantize=True)
    assert not y[1].any() and mean[1] == 0 and torch.isfinite(rstd[1])
    for i in (2, 3):
        assert torch.isnan(y[i]).all() and torch.isnan(rstd[i]) and torch.isnan(q[i].float()).all()
    assert torch.isnan(mean[2]) and torch.isinf(mean[3])
    for i in (0, 4, 5):
        assert torch.equal(y[i], clean[i])
    assert not q[1].float().any() and float(scale[1]) == pytest.approx(1e-30 / 448, rel=1e-6)
    assert torch.isfinite(q[4].float()).all()


def test_add_layernorm_empty():
    x, w = torch.empty(3, 0, device="cuda"), torch.empty(0, device="cuda")
    y, s, mean, rstd = sg.add_layernorm(x, w, w, eps=1e-4)
    assert y.shape == (3, 0) and not mean.any()
    assert torch.allclose(rstd, torch.full_like(rstd, 100.0))
    _, scale, *_ = sg.add_layernorm(x, w, quantize=True)
    assert torch.allclose(scale, torch.full_like(scale, 1e-30 / 448))
    y, *_ = sg.add_layernorm(torch.empty(0, 8, device="cuda"), torch.ones(8, device="cuda"))
    assert y.shape == (0, 8)


def run_layernorm_backward(rows, d, t, stream=True, pad=0, offset=0, call=sg.add_layernorm_backward):
    dtype = TYPES[t]
    g = gen(rows + 37 * d)
    s, dy, ds = (normal(g, rows, d, dtype=dtype) for _ in range(3))
    w = (1 + normal(g, d, std=0.2)).to(dtype)
    mean = s.double().mean(1).float()
    rstd = torch.rsqrt((s.double() - mean.double()[:, None]).square().mean(1) + 1e-5).float()
    dx, dw, db = call(strided(dy, pad, offset), strided(s, pad, offset), mean, rstd, w,
                      strided(ds, pad, offset) if stream else None)
    torch.cuda.synchronize()
    R = rstd.double()[:, None]
    n, DY = (s.double() - mean.double()[:, None]) * R, dy.double()
    gg = DY * w.double()
    kg, kn = gg.mean(1, keepdim=True), (gg * n).mean(1, keepdim=True)
    want = R * (gg - kg - n * kn) + (ds.double() if stream else 0)
    rel = (d / 32 + 72) * EPS
    tol = (R * rel * (gg.abs().mean(1, keepdim=True) + n.abs() * (gg * n).abs().mean(1, keepdim=True)) +
           16 * EPS * (R * (gg.abs() + kg.abs() + (n * kn).abs()) + want.abs()) +
           UNIT[dtype] * want.abs() + TINY[dtype])
    what = f"{rows}x{d} {t} ds={stream} pad={pad}+{offset}"
    check(dx, want, tol, what + " dx")
    for got, terms, label in ((dw, DY * n, " dw"), (db, DY, " db")):
        want = terms.sum(0)
        check(got, want, UNIT[dtype] * want.abs() + (rows + 16) * EPS / 2 * terms.abs().sum(0) +
              TINY[dtype], what + label)


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,d", NORM_SIZES)
def test_add_layernorm_backward_sizes(rows, d, t):
    run_layernorm_backward(rows, d, t, True)
    run_layernorm_backward(rows, d, t, False)


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("pad,offset", [(8, 0), (3, 0), (0, 1), (5, 3)])
def test_add_layernorm_backward_strides(pad, offset, t):
    run_layernorm_backward(20, 512, t, True, pad, offset)
    run_layernorm_backward(400, 520, t, True, pad, offset)


# rows long and many enough for the ring: whole and ragged turns, groups that do not fill the CTA
@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,d", [(9801, 520), (2501, 4096), (1300, 8192), (48700, 520), (24321, 1024),
                                    (6081, 4096), (12163, 2008), (3041, 8192), (6200, 3000)])
def test_add_layernorm_backward_of_many_rows(rows, d, t):
    run_layernorm_backward(rows, d, t, True)
    run_layernorm_backward(rows, d, t, False, pad=8)


# 16-bit rows of 32 columns a thread: two and three rows in the ring, every number of turns
@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,d", [(1, 8200), (2, 16384), (151, 9008), (153, 12288), (306, 10240),
                                    (458, 16376), (700, 8264), (1000, 12296)])
def test_add_layernorm_backward_of_wide_rows(rows, d, t):
    run_layernorm_backward(rows, d, t, True)
    run_layernorm_backward(rows, d, t, False, pad=8)


@pytest.mark.parametrize("t", ["f32", "bf16"])
def test_add_layernorm_backward_in_place(t):
    # dX may be dY or dS itself: through the C ABI, one and many rows
    dtype, code = TYPES[t], 0 if t == "f32" else 1
    for rows, d in ((3, 264), (1300, 4096), (6100, 4096), (700, 9001), (2100, 1001), (900, 12288)):
        g = gen(rows)
        dy, s, ds = (normal(g, rows, d, dtype=dtype) for _ in range(3))
        mean, rstd, w = normal(g, rows), normal(g, rows).abs() + 0.5, normal(g, d, dtype=dtype)
        dx, dw, db = sg.add_layernorm_backward(dy, s, mean, rstd, w, ds)
        need = sg.add_layernorm_backward_workspace_size(code, rows, d)
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        for over in (0, 1):
            a, b = dy.clone(), ds.clone()
            out, dw2, db2 = (a, b)[over], torch.empty_like(dw), torch.empty_like(db)
            sg.sgemm_add_layernorm_backward(code, rows, d, a.data_ptr(), d, s.data_ptr(), d,
                                            mean.data_ptr(), rstd.data_ptr(), w.data_ptr(),
                                            b.data_ptr(), d, out.data_ptr(), d, dw2.data_ptr(),
                                            db2.data_ptr(), ws.data_ptr(), need,
                                            torch.cuda.current_stream().cuda_stream)
            assert torch.equal(out, dx) and torch.equal(dw2, dw) and torch.equal(db2, db)


def test_add_layernorm_backward_empty_and_parts():
    e = lambda *s: torch.ones(*s, device="cuda")  # noqa: E731
    dx, dw, db = sg.add_layernorm_backward(e(0, 8), e(0, 8), e(0), e(0), e(8))
    assert dx.shape == (0, 8) and not dw.any() and not db.any()
    dy, s = normal(gen(1), 30, 64), normal(gen(2), 30, 64)
    args = (dy, s, e(30), e(30), e(64))
    dx, dw, db = sg.add_layernorm_backward(*args)
    for w, b in ((True, False), (False, True), (False, False)):
        a = sg.add_layernorm_backward(*args, need_dweight=w, need_dbias=b)
        assert torch.equal(a[0], dx)
        assert torch.equal(a[1], dw) if w else a[1] is None
        assert torch.equal(a[2], db) if b else a[2] is None


# Rows that start off a 16-byte boundary: in torch's layout those of an odd width, and by the C ABI
# with every matrix as far off it.
@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,d", [(305, 513), (400, 519), (1000, 1001), (500, 2050), (306, 8191),
                                    (2000, 257), (310, 32001), (20, 2049), (304, 9001), (313, 515)])
def test_add_layernorm_rows_off_the_boundary(rows, d, t):
    for quantize in (False, True):
        run_layernorm(rows, d, t, True, True, quantize)
        run_layernorm(rows, d, t, False, False, quantize)


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,d", [(4100, 513), (2100, 1001), (1100, 2047), (530, 4095), (300, 8191),
                                    (17001, 257), (1025, 2049), (4091, 517)])
def test_add_layernorm_backward_rows_off_the_boundary(rows, d, t):
    run_layernorm_backward(rows, d, t, True)
    run_layernorm_backward(rows, d, t, False)


def off_by(rows, d, ld, offset, dtype, fill=None):
    """(rows, d) of leading dimension ld, `offset` elements past an allocation's start; what lies
    around it is 77, which no call may write."""
    buffer = torch.full((offset + rows * ld + 16,), 77.0, device="cuda").to(dtype)
    at = buffer[offset:offset + rows * ld].view(rows, ld)[:, :d]
    if fill is not None:
        at.copy_(fill)
    return buffer, at


def assert_untouched(buffer, at):
    around = buffer.clone()
    around[at.storage_offset():at.storage_offset() + at.shape[0] * at.stride(0)].view(
        at.shape[0], at.stride(0))[:, :at.shape[1]] = torch.full((), 77.0, device="cuda").to(at.dtype)
    assert (around.float() == torch.full((), 77.0, device="cuda").to(at.dtype).float()).all()


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("rows,d,ld", [(310, 1024, 1027), (320, 1003, 1003), (309, 515, 520), (340, 2061, 2065)])
def test_add_layernorm_alike_off_the_boundary(rows, d, ld, t):
    dtype, code = TYPES[t], 0 if t == "f32" else 1

    def forward(offset, in_place):
        def call(x, w, b, r, eps, quantize):
            _, X = off_by(rows, d, ld, offset, dtype, x)
            R = off_by(rows, d, ld, offset, dtype, r)[1] if r is not None else None
            kept, S = (None, R) if in_place and r is not None else off_by(rows, d, ld, offset, dtype)
            out = torch.float8_e4m3fn if quantize else dtype
            buffer, Y = off_by(rows, d, ld, offset, out)
            scale, mean, rstd = (torch.empty(rows, device="cuda") for _ in range(3))
            sg.sgemm_add_layernorm(code, rows, d, X.data_ptr(), ld, R.data_ptr() if r is not None else 0,
                                   ld, w.data_ptr(), b.data_ptr() if b is not None else 0, eps,
                                   S.data_ptr(), ld, Y.data_ptr(), ld,
                                   scale.data_ptr() if quantize else 0, mean.data_ptr(),
                                   rstd.data_ptr(), torch.cuda.current_stream().cuda_stream)
            assert_untouched(buffer, Y)
            if kept is not None:
                assert_untouched(kept, S)
            return ((Y, scale) if quantize else (Y,)) + (S, mean, rstd)
        return call

    for offset in range(0, 9, 1 if t == "bf16" else 2):
        for quantize in (False, True):
            run_layernorm(rows, d, t, True, True, quantize, call=forward(offset, False))
        run_layernorm(rows, d, t, True, False, False, call=forward(offset + 1, True))
        run_layernorm(rows, d, t, False, False, True, call=forward(offset, False))


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("rows,d,ld", [(2100, 1024, 1027), (1100, 2043, 2043), (4200, 515, 520)])
def test_add_layernorm_backward_alike_off_the_boundary(rows, d, ld, t):
    dtype, code = TYPES[t], 0 if t == "f32" else 1

    def backward(offset, in_place):
        def call(dy, s, mean, rstd, w, ds):
            (kept, DY), (_, S) = (off_by(rows, d, ld, offset, dtype, v) for v in (dy, s))
            DS = off_by(rows, d, ld, offset, dtype, ds)[1] if ds is not None else None
            buffer, DX = (kept, DY) if in_place else off_by(rows, d, ld, offset, dtype)
            dw, db = (torch.empty(d, dtype=dtype, device="cuda") for _ in range(2))
            need = sg.add_layernorm_backward_workspace_size(code, rows, d)
            ws = torch.empty(need, dtype=torch.uint8, device="cuda")
            sg.sgemm_add_layernorm_backward(code, rows, d, DY.data_ptr(), ld, S.data_ptr(), ld,
                                            mean.data_ptr(), rstd.data_ptr(), w.data_ptr(),
                                            DS.data_ptr() if ds is not None else 0, ld, DX.data_ptr(),
                                            ld, dw.data_ptr(), db.data_ptr(), ws.data_ptr(), need,
                                            torch.cuda.current_stream().cuda_stream)
            assert_untouched(buffer, DX)
            return DX, dw, db
        return call

    for offset in range(0, 9, 1 if t == "bf16" else 2):
        run_layernorm_backward(rows, d, t, True, call=backward(offset, False))
        run_layernorm_backward(rows, d, t, offset % 4 == 0, call=backward(offset + 1, True))


def test_add_layernorm_gradient_against_differences():
    """L = <dy, y> + <ds, s> in 64 bits along x, the residual, the weight and the bias."""
    g, h = gen(6), 1e-4
    rows, d = 24, 136
    x, r, dy, ds = (normal(g, rows, d) for _ in range(4))
    w, b = 1 + normal(g, d, std=0.2), normal(g, d)
    _, s, mean, rstd = sg.add_layernorm(x, w, b, r, eps=1e-3)
    dx, dw, db = sg.add_layernorm_backward(dy, s, mean, rstd, w, ds)

    def loss(x, r, w, b):
        s = x + r
        c = s - s.mean(1, keepdim=True)
        y = c / torch.sqrt(c.square().mean(1, keepdim=True) + 1e-3) * w + b
        return (dy.double() * y).sum() + (ds.double() * s).sum()

    p = [t.double() for t in (x, r, w, b)]
    for i, grad in enumerate((dx, dx, dw, db)):
        v = torch.randn(p[i].shape, generator=g, device="cuda", dtype=torch.float64)
        plus, minus = list(p), list(p)
        plus[i], minus[i] = p[i] + h * v, p[i] - h * v
        diff = (loss(*plus) - loss(*minus)) / (2 * h)
        along = (grad.double() * v).sum()
        assert abs(float(diff - along)) <= 1e-5 * float(grad.double().norm() * v.norm()) + 1e-6, i


# ------------------------------------------------------------------ clip_grad_norm


def exact_norm(tensors):
    return sum(float(t.double().square().sum()) for t in tensors) ** 0.5


def check_clip(tensors, max_norm, apart=None, eps=1e-6):
    """In place on copies, and (apart: the results' misalignment in elements) elsewhere."""
    norm = exact_norm(tensors)
    want = [t.double() * min(1.0, max_norm / (norm + eps)) for t in tensors]
    if apart is None:
        got = tensors
        buffers = []
    else:
        buffers = [torch.full((t.numel() + apart + 9,), float("nan"), dtype=t.dtype, device="cuda")
                   for t in tensors]
        got = [b[apart:apart + t.numel()].view(t.shape) for b, t in zip(buffers, tensors)]
        before = [t.clone() for t in tensors]
    result = sg.clip_grad_norm(tensors, max_norm, eps=eps, out=None if apart is None else got)
    torch.cuda.synchronize()
    assert result.shape == () and result.dtype == torch.float32
    assert abs(float(result) - norm) <= 10 * EPS * norm, (float(result), norm)
    for g, w in zip(got, want):
        check(g, w, (UNIT[g.dtype] + 12 * EPS) * w.abs() + TINY[g.dtype], "scaled")
    for b, t in zip(buffers, tensors):
        assert torch.isnan(b[:apart]).all() and torch.isnan(b[apart + t.numel():]).all()
    if apart is not None:
        assert all(torch.equal(a, b) for a, b in zip(before, tensors))


SHAPES = [(1,), (7,), (64, 64), (), (3, 0, 5), (1001,), (255, 33), (8192,), (8193,), (70000,), (300, 1000)]


def some(types, shapes=SHAPES, seed=0, std=1.0):
    g = gen(seed)
    return [normal(g, int(np.prod(s)), std=std).view(s).to(TYPES[types[i % len(types)]])
            for i, s in enumerate(shapes)]


@pytest.mark.parametrize("types", [("f32",), ("bf16",), ("f16",), ("bf16", "f32", "f16")])
@pytest.mark.parametrize("max_norm", [0.0, 1.0, 1e6, float("inf")])
def test_clip_types_and_factors(types, max_norm):
    check_clip(some(types), max_norm)
    check_clip(some(types), max_norm, apart=0)


@pytest.mark.parametrize("types", [("f32",), ("bf16", "f32")])
@pytest.mark.parametrize("offset", [1, 2, 3, 5, 7])
@pytest.mark.parametrize("apart", [None, 0, 1, 3])
def test_clip_any_alignment(types, offset, apart):
    tensors = []
    for t in some(types, [(1,), (6,), (9,), (1000,), (20000,), (8192 * 3,)]):
        buf = torch.full((t.numel() + offset + 8,), float("nan"), dtype=t.dtype, device="cuda")
        buf[offset:offset + t.numel()] = t
        tensors.append(buf[offset:offset + t.numel()])
    check_clip(tensors, 0.5, apart=apart)
    for t in tensors:     # nothing around a tensor is read or written
        whole = t._base if t._base is not None else t
        assert torch.isnan(whole[:offset]).all() and torch.isnan(whole[offset + t.numel():]).all()


@pytest.mark.parametrize("count", [1, 32, 33, 256, 257, 1000, 1001, 2300])
def test_clip_many_tensors(count):
    # every table of a launch's arguments, and several launches
    g = gen(count)
    sizes = torch.randint(0, 700, (count,), generator=g, device="cuda").tolist()
    sizes[-1] = 12345
    check_clip([normal(g, n) for n in sizes], 1.0)
    check_clip([normal(g, n, dtype=torch.bfloat16) for n in sizes], 1.0, apart=2)


@pytest.mark.parametrize("t,elements", [("bf16", 40_000_003), ("f32", 25_000_001)])
def test_clip_large(t, elements):
    check_clip([normal(gen(5), elements, dtype=TYPES[t], std=1e-3), normal(gen(6), 77, dtype=TYPES[t])], 1.0)


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("size", [1e-30, 1e-20, 3e-13, 1e12, 1e17, 1e25])
def test_clip_of_very_small_and_large_elements(t, size):
    # their squares leave fp32's range; the norm's bound does not change
    tensors = some((t,), [(1000,), (77, 40)], std=size)
    tensors[0][::2] = 0
    check_clip(tensors, size, eps=0.0)
    mixed = some((t,), [(5000,)], std=1.0) + tensors
    check_clip(mixed, 1.0, eps=0.0)


def test_clip_subnormal_elements():
    t = torch.full((4099,), 2.0 ** -140, device="cuda")
    assert float(sg.grad_norm([t])) == pytest.approx(2.0 ** -140 * 4099 ** 0.5, rel=1e-2)   # (subnormal result)
    big = torch.full((100,), 3e38, device="cuda")
    assert torch.isinf(sg.grad_norm([big]))          # the norm itself is beyond fp32
    sg.clip_grad_norm([big], 1.0)                    # its factor is not
    assert float(big.double().norm()) == pytest.approx(1.0, rel=1e-6)


def test_clip_zeros_nan_and_infinity():
    zeros = [torch.zeros(5000, device="cuda"), torch.zeros(3, device="cuda", dtype=torch.float16)]
    assert float(sg.clip_grad_norm(zeros, 1.0)) == 0 and not zeros[0].any() and not zeros[1].any()
    for t in ("f32", "bf16", "f16"):
        a = some((t,))
        a[5][17] = float("nan")
        assert torch.isnan(sg.clip_grad_norm(a, 1.0))
        assert all(torch.isnan(x).all() for x in a)
        a = some((t,))
        a[5][17] = float("-inf")
        assert torch.isinf(sg.clip_grad_norm(a, 1.0))
        assert torch.isnan(a[5][17]) and torch.isnan(a[5]).sum() == 1
        a[5][17] = 0
        assert not any(x.any() for x in a)


def test_clip_of_nothing_but_zeros_without_eps():
    # norm + eps is 0: the factor is 1, not 0 / 0
    a = torch.zeros(100, device="cuda")
    for max_norm in (0.0, 1.0, float("inf")):
        assert float(sg.clip_grad_norm([a], max_norm, eps=0.0)) == 0 and not a.any()


def test_clip_without_a_bound_scales_nothing():
    for value in (2.0, float("inf")):
        a = normal(gen(3), 4000)
        a[7] = value
        kept, out = a.clone(), torch.empty_like(a)
        assert float(sg.clip_grad_norm([a], float("inf"), out=[out])) == float(sg.grad_norm([a]))
        assert torch.equal(out, kept)
        sg.clip_grad_norm([a], float("inf"))
        assert torch.equal(a, kept)
    a[8] = float("nan")
    sg.clip_grad_norm([a], float("inf"))
    assert torch.isnan(a).all()


def test_clip_takes_one_tensor_and_any_iterable():
    a, b = normal(gen(1), 50, 7), normal(gen(2), 33)
    want = exact_norm([a])
    assert abs(float(sg.grad_norm(a)) - want) <= 10 * EPS * want
    out = torch.empty_like(a)
    sg.clip_grad_norm(a, 1.0, out=out)
    kept = a.clone()
    sg.clip_grad_norm(a, 1.0)
    assert torch.equal(a, out) and not torch.equal(a, kept)
    want = exact_norm([a, b])
    norm = sg.clip_grad_norm((t for t in (a, b)), 0.5, out=iter([a, b]))
    assert abs(float(norm) - want) <= 10 * EPS * want
    assert exact_norm([a, b]) == pytest.approx(0.5, rel=1e-5)


def test_clip_leaves_tensors_below_the_norm_as_they_are():
    a = some(("bf16", "f32"))
    a[3].fill_(float(2.0 ** -130))
    before = [t.clone() for t in a]
    norm = sg.clip_grad_norm(a, 1e5)
    assert float(norm) > 1 and all(torch.equal(x, y) for x, y in zip(a, before))


def test_grad_norm_alone_and_strides():
    a = some(("f32", "bf16"))
    a.append(normal(gen(4), 300, 77).t())                       # any dense order of strides
    a.append(normal(gen(5), 4, 5, 6, 7).permute(2, 0, 3, 1))
    before = [t.clone() for t in a]
    norm = exact_norm(a)
    assert abs(float(sg.grad_norm(a)) - norm) <= 10 * EPS * norm
    assert all(torch.equal(x, y) for x, y in zip(a, before))
    check_clip(a, 1.0)
    with pytest.raises(ValueError):
        sg.grad_norm([normal(gen(1), 8, 8)[:, :5]])
    with pytest.raises(ValueError):
        sg.clip_grad_norm(a[:2], 1.0, out=a[:1])
    with pytest.raises(ValueError):
        sg.clip_grad_norm([normal(gen(1), 4, 6)], 1.0, out=[normal(gen(1), 6, 4).t()])
    with pytest.raises(sg.SgemmError):
        sg.clip_grad_norm([a[5], a[5]], 1.0)                    # the same tensor twice
    twice = [a[5], a[5]]
    assert abs(float(sg.grad_norm(twice)) - exact_norm(twice)) <= 10 * EPS * exact_norm(twice)


def test_clip_counts_as_changed_in_place():
    a, b = torch.ones(8, device="cuda"), torch.empty(8, device="cuda")
    v = a._version, b._version
    sg.grad_norm([a])
    sg.clip_grad_norm([a], 1.0, out=[b])
    assert a._version == v[0] and b._version > v[1]
    sg.clip_grad_norm([a], 1.0)
    assert a._version > v[0]


def test_clip_streams_graph_and_the_same_bits():
    a = some(("bf16", "f32"), SHAPES * 12, seed=3)
    out = [torch.empty_like(t) for t in a]
    first = sg.clip_grad_norm(a, 1.0, out=out)
    kept = [t.clone() for t in out]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        norm = sg.clip_grad_norm(a, 1.0, out=out, stream=side)
    side.synchronize()
    assert torch.equal(norm, first) and all(torch.equal(x, y) for x, y in zip(out, kept))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        norm = sg.clip_grad_norm(a, 1.0, out=out)
    for t in a:
        t.mul_(3)
    graph.replay()
    torch.cuda.synchronize()
    want = sg.clip_grad_norm(a, 1.0)
    assert torch.equal(norm, want) and all(torch.equal(x, y) for x, y in zip(out, a))


# ------------------------------------------------------------------ together


@pytest.mark.parametrize("t", ["f32", "bf16"])
def test_gated_block_trains_as_its_formula_says(t):
    """norm -> gated projections -> down-projection + residual, its gradients and their
    clipping, against autograd in 64 bits.  bf16: about six roundings of 2^-8 on the way to a
    gradient, averaged by the sums: 2 % in the 2-norm; f32: 2e-5."""
    g, dtype = gen(12), TYPES[t]
    rows, d, f = 70, 256, 520
    x, res, dout = (normal(g, rows, d, dtype=dtype) for _ in range(3))
    p = [(1 + normal(g, d, std=0.1)), normal(g, d, std=0.1), normal(g, f, d, std=d ** -0.5),
         normal(g, f, d, std=d ** -0.5), normal(g, f, std=0.1), normal(g, f, std=0.1),
         normal(g, d, f, std=f ** -0.5)]
    w, b, wg, wu, bg, bu, wd = p = [v.to(dtype) for v in p]
    y, s, mean, rstd = sg.add_layernorm(x, w, b, res)
    h, zg, zu = sg.gated_linear(y, wg, wu, bg, bu, save_preact=True)
    out = sg.linear(h, wd, residual=s)
    dh, dwd, _ = sg.linear_backward(dout, h, wd, need_db=False)
    dy, dwg, dwu, dbg, dbu = sg.gated_linear_backward(dh, y, wg, wu, zg, zu)
    dx, dw, db = sg.add_layernorm_backward(dy, s, mean, rstd, w, dout)
    grads = [dw, db, dwg, dwu, dbg, dbu, dwd]
    q = [v.double().requires_grad_(True) for v in [x, *p]]
    S = q[0] + res.double()
    Y = torch.nn.functional.layer_norm(S, (d,), q[1], q[2], 1e-5)
    H = torch.nn.functional.silu(Y @ q[3].t() + q[5]) * (Y @ q[4].t() + q[6])
    O = H @ q[7].t() + S
    want = torch.autograd.grad((O * dout.double()).sum(), q)
    rel = 2e-5 if t == "f32" else 0.02
    for got, ref in zip([out, dx, *grads], [O.detach(), *want]):
        assert float((got.double() - ref).norm() / ref.norm()) < rel
    norm = sg.clip_grad_norm(grads, 1.0)
    total = sum(float(v.square().sum()) for v in want[1:]) ** 0.5
    assert float(norm) == pytest.approx(total, rel=rel)
    assert exact_norm(grads) == pytest.approx(1.0, rel=rel)


def test_gated_block_in_8_bits():
    """The block served in 8 bits against 64 bits: three roundings of 2^-4 relative to 8 bits
    on each way, averaged by the sums: 8 % in the 2-norm."""
    g = gen(13)
    rows, d, f = 70, 512, 1024
    x, res = normal(g, rows, d, dtype=torch.bfloat16), normal(g, rows, d, dtype=torch.bfloat16)
    w, b = (1 + normal(g, d, std=0.1)).to(torch.bfloat16), normal(g, d, std=0.1, dtype=torch.bfloat16)
    wg, wu, wd = (normal(g, *s, dtype=torch.bfloat16, std=s[1] ** -0.5) for s in ((f, d), (f, d), (d, f)))
    S = x.double() + res.double()
    Y = torch.nn.functional.layer_norm(S, (d,), w.double(), b.double(), 1e-5)
    want = (torch.nn.functional.silu(Y @ wg.double().t()) * (Y @ wu.double().t())) @ wd.double().t() + S
    (qg, sgate), (qu, sup), (qd, sdown) = (sg.quantize_rows(v) for v in (wg, wu, wd))
    for rows_used in (70, 1):
        q, qs, s, _, _ = sg.add_layernorm(x[:rows_used], w, b, res[:rows_used], quantize=True)
        h = sg.gated_linear(q, qg, qu, x_scale=qs, gate_scale=sgate, up_scale=sup)
        hq, hs = sg.quantize_rows(h)
        got = sg.linear(hq, qd, residual=s, x_scale=hs, w_scale=sdown)
        ref = want[:rows_used]
        assert float((got.double() - ref).norm() / ref.norm()) < 0.08


def example(name):
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        name + ".py")
    spec = importlib.util.spec_from_file_location(name + "_example", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("t", ["bf16", "f16"])
def test_gated_example(t):
    """It runs, and its gradients are the formula's: against autograd in 64 bits, 2 % in the
    2-norm (as test_gated_block_trains_as_its_formula_says); the served output is within 8 %."""
    module, dtype = example("gated_feed_forward"), TYPES[t]
    losses, norms, off = module.run(130, 256, 520, 3, dtype)
    assert all(np.isfinite(losses)) and all(np.isfinite(norms)) and off < 0.08
    block = module.GatedFeedForward(256, 520, dtype)
    g = gen(3)
    x, r, dout = (normal(g, 40, 256, dtype=dtype) for _ in range(3))
    out, saved = block.forward(x, r)
    dx, grads = block.backward(dout, saved)
    p = [v.double().requires_grad_(True) for v in (x, block.g, block.c, block.wg, block.wu, block.wd)]
    S = p[0] + r.double()
    Y = torch.nn.functional.layer_norm(S, (256,), p[1], p[2], 1e-5)
    O = (torch.nn.functional.silu(Y @ p[3].t()) * (Y @ p[4].t())) @ p[5].t() + S
    want = torch.autograd.grad((O * dout.double()).sum(), p)
    for got, ref in zip([out, dx, *grads], [O.detach(), *want]):
        assert float((got.double() - ref).norm() / ref.norm()) < 0.02
    before = [getattr(block, n).clone() for n in block.PARAMETERS]
    norm = block.step(grads, 0.5, 1e-2)
    assert exact_norm(grads) <= 1e-2 * (1 + UNIT[dtype] + 12 * EPS) and float(norm) > 1e-2
    # p + d alpha is rounded once more where it is stored
    for old, n, d in zip(before, block.PARAMETERS, grads):
        want = old.double() - 0.5 * d.double()
        check(getattr(block, n), want, (UNIT[dtype] + 4 * EPS) * (want.abs() + d.double().abs()) +
              TINY[dtype], n)


def test_feed_forward_example_clips():
    module = example("feed_forward")
    losses, _ = module.run(70, 128, 256, 3, torch.bfloat16, max_norm=1e-3)
    assert all(np.isfinite(losses))
    block = module.FeedForward(128, 256, torch.float32)
    g = gen(4)
    x, r, dout = (normal(g, 30, 128) for _ in range(3))
    _, saved = block.forward(x, r)
    _, grads = block.backward(dout, saved)
    before, want = block.w1.clone(), exact_norm(grads.values())
    block.step(grads, 1.0, max_norm=0.25 * want)
    assert exact_norm(grads.values()) == pytest.approx(0.25 * want, rel=1e-5)
    check(block.w1, before.double() - grads["w1"].double(),
          2 * EPS * (before.double().abs() + grads["w1"].double().abs()) + 1e-30, "w1")
