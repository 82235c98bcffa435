"""The layer operators on the GPU against plain formulas in 64 bits.

Tolerances are derived from the arithmetic, with u the output's unit roundoff
(2^-24 f32, 2^-8 bf16, 2^-11 f16; e4m3 codes: half a spacing):
  * one rounding of the result: u |y|;
  * sums in fp32: every update of a running sum errs by at most one unit
    (2^-23) of the largest partial sum, which the sum S of absolute terms
    bounds.  Tensor cores update once per 16 terms (32 for 8 bits) and drop low
    bits when they align the terms, so (K / 8 + 8) 2^-23 S covers them; f32
    products drop terms of 2^-20 S besides and round lo to 2^-21;
  * an activation's slope is below 1.2 and its own evaluation errs by a few
    units of |z| (16 2^-23);
  * dZ enters the 16-bit products rounded once: u S.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import dense_fp32_matrix_sgemm_gb300 as sg  # noqa: E402

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
UNIT = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 1e-37, torch.bfloat16: 1e-37, torch.float16: 2.0 ** -25}
EPS = 2.0 ** -23


@pytest.fixture(scope="module", autouse=True)
def no_pipeline_errors():
    sg.device_status(reset=True)
    yield
    assert sg.device_status(reset=True) == 0


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, *shape, dtype=torch.float32, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def strided(t, pad, offset=0):
    """The same matrix with rows `pad` elements longer, starting `offset`
    elements into its buffer; the rest is NaN."""
    r, c = t.shape
    if t.dtype == torch.float8_e4m3fn:
        buf = torch.full((r * (c + pad) + offset,), 0x7f, dtype=torch.uint8, device="cuda").view(t.dtype)
        view = buf[offset:].view(r, c + pad)[:, :c]
        view.view(torch.uint8).copy_(t.view(torch.uint8))
        return view
    buf = torch.full((r * (c + pad) + offset,), float("nan"), dtype=t.dtype, device="cuda")
    view = buf[offset:].view(r, c + pad)[:, :c]
    view.copy_(t)
    return view


def act(z, name):
    if name == "relu":
        return z.clamp(min=0)
    if name == "gelu":
        return 0.5 * z * (1 + torch.tanh((2 / np.pi) ** 0.5 * (z + 0.044715 * z ** 3)))
    if name == "gelu_erf":
        return 0.5 * z * (1 + torch.erf(z / 2 ** 0.5))
    if name == "silu":
        return z * torch.sigmoid(z)
    return z


def act_grad(z, name):
    if name == "none":
        return torch.ones_like(z)
    if name == "relu":
        return (z > 0).double()
    z = z.detach().requires_grad_(True)
    return torch.autograd.grad(act(z, name).sum(), z)[0].detach()


def check(got, want, tol, what):
    err = (got.double() - want).abs()
    bad = ~(err <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst "
                           f"{float((err / tol).max()):.3g} of the tolerance at "
                           f"{np.unravel_index(int((err / tol).argmax()), bad.shape)}")


def product_tol(S, K, dtype):
    if dtype == torch.float32:
        return (2.0 ** -19 + (64 + K / 8) * EPS / 4) * S
    return (K / 8 + 8) * EPS * S


# ------------------------------------------------------------------ linear


def run_linear(m, n, k, t, name="none", bias=False, residual=False, preact=False, w_kn=False, pad=0,
               offset=0, seed=0, out_dtype=None):
    g = gen(seed + 7 * m + 11 * n + 13 * k)
    e4m3 = t == "e4m3"
    dtype = (out_dtype or torch.bfloat16) if e4m3 else TYPES[t]
    x, w = normal(g, m, k), normal(g, n, k, std=max(k, 1) ** -0.5)
    kw = {}
    if e4m3:
        x, kw["x_scale"] = sg.quantize_rows(x)
        w, kw["w_scale"] = sg.quantize_rows(w)
    else:
        x, w = x.to(dtype), w.to(dtype)
    b = normal(g, n, dtype=dtype) if bias else None
    r = normal(g, m, n, dtype=dtype) if residual else None
    xs = strided(x, pad, offset)
    ws = strided(w.t().contiguous(), pad, offset).t() if w_kn else strided(w, pad, offset)
    rs = strided(r, pad, offset) if residual else None
    buf = torch.full((m * (n + pad) + offset + 64,), float("nan"), dtype=dtype, device="cuda")
    out = buf[offset:offset + m * (n + pad)].view(m, n + pad)[:, :n]
    got = sg.linear(xs, ws, b, activation=name, residual=rs, save_preact=preact, out=out,
                    out_dtype=dtype if e4m3 else None, **kw)
    y, z = got if preact else (got, None)
    torch.cuda.synchronize()
    xd, wd = x.double(), w.double()
    if e4m3:
        xd, wd = xd * kw["x_scale"].double()[:, None], wd * kw["w_scale"].double()[:, None]
    zd = xd @ wd.t()
    S = xd.abs() @ wd.abs().t()
    if bias:
        zd, S = zd + b.double(), S + b.double().abs()
    yd = act(zd, name) + (r.double() if residual else 0)
    ztol = product_tol(S, k, torch.float32 if t == "f32" else dtype) + 4 * EPS * S
    tol = 1.2 * ztol + 16 * EPS * (zd.abs() + yd.abs()) + UNIT[dtype] * yd.abs() + TINY[dtype]
    what = f"{m}x{n}x{k} {t} {name} bias={bias} residual={residual} w_kn={w_kn} pad={pad}+{offset}"
    check(y, yd, tol, what)
    if preact:
        check(z, zd, ztol + UNIT[dtype] * zd.abs() + TINY[dtype], what + " preact")
    if pad:
        full = buf[offset:offset + m * (n + pad)].view(m, n + pad)
        assert torch.isnan(full[:, n:]).all(), "padding columns were written"
    assert torch.isnan(buf[offset + m * (n + pad):]).all() and torch.isnan(buf[:offset]).all()


# one row and few rows (CUDA cores, either storage), ragged tiles, split K over
# clusters (few tiles), one wave and several waves of either tile width
SIZES = [(1, 1, 1), (1, 300, 257), (1, 4096, 1024), (2, 77, 640), (3, 1000, 8), (4, 129, 4096),
         (5, 64, 64), (16, 520, 200), (17, 96, 1000), (33, 1000, 520), (64, 512, 2048),
         (127, 255, 129), (128, 128, 64), (129, 257, 4104), (300, 1, 72), (513, 640, 16),
         (1290, 1030, 136), (2300, 2040, 200), (4610, 4100, 40)]


@pytest.mark.parametrize("t", ["f32", "bf16", "f16", "e4m3"])
@pytest.mark.parametrize("m,n,k", SIZES)
def test_linear_sizes(m, n, k, t):
    run_linear(m, n, k, t, "gelu", bias=True, residual=True)


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("m,n,k", SIZES)
def test_linear_weight_stored_by_columns(m, n, k, t):
    run_linear(m, n, k, t, "silu", bias=True, w_kn=True)


@pytest.mark.parametrize("t", ["f32", "bf16", "f16", "e4m3"])
@pytest.mark.parametrize("name", ["none", "relu", "gelu", "gelu_erf", "silu"])
@pytest.mark.parametrize("m", [1, 70, 1300])
def test_linear_epilogues(m, name, t):
    run_linear(m, 1032, 320, t, name, bias=True, residual=True, preact=True)
    run_linear(m, 1032, 320, t, name, preact=True)
    run_linear(m, 1031, 320, t, name, residual=True)


@pytest.mark.parametrize("t", ["f32", "bf16", "f16", "e4m3"])
@pytest.mark.parametrize("pad,offset", [(8, 0), (3, 0), (0, 1), (5, 3), (16, 16)])
@pytest.mark.parametrize("m", [1, 3, 70, 700])
def test_linear_strides_and_offsets(m, pad, offset, t):
    run_linear(m, 344, 200, t, "relu", bias=True, residual=True, preact=True, pad=pad, offset=offset)
    run_linear(m, 345, 201, t, "none", pad=pad, offset=offset)
    if t != "e4m3":
        run_linear(m, 345, 201, t, "none", pad=pad, offset=offset, w_kn=True)


# long sums: pairs' tiles with K split over two pairs, and whole waves of pairs'
# tiles followed by a second launch that splits the rest
@pytest.mark.parametrize("m,n,k,t", [(1024, 2048, 8192, "f32"), (1000, 2050, 8200, "bf16"),
                                     (1024, 2048, 8192, "f16"), (1020, 2040, 16400, "e4m3"),
                                     (2560, 2560, 2600, "f32"), (2500, 2540, 8008, "bf16"),
                                     (2560, 2560, 16000, "e4m3")])
def test_linear_long_sums(m, n, k, t):
    run_linear(m, n, k, t, "gelu", bias=True, residual=True, preact=True)
    if t != "e4m3":
        run_linear(m, n, k, t, "relu", bias=True, residual=True, w_kn=True)


@pytest.mark.parametrize("t", ["bf16", "e4m3"])
@pytest.mark.parametrize("m", [1, 2, 3, 4, 5])
@pytest.mark.parametrize("n,k", [(2048, 2048), (2056, 2064), (2050, 2051)])
def test_linear_few_rows_of_either_kernel(n, k, m, t):
    run_linear(m, n, k, t, "silu", bias=True, residual=True, preact=True)


def test_linear_e4m3_to_f16():
    run_linear(2, 96, 256, "e4m3", "silu", bias=True, out_dtype=torch.float16)
    run_linear(200, 500, 256, "e4m3", "silu", bias=True, residual=True, out_dtype=torch.float16)


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("m", [1, 9, 300])
def test_linear_without_inputs(m, t):
    # K = 0: act(bias) + residual
    dtype = TYPES[t]
    g = gen(3)
    b, r = normal(g, 130, dtype=dtype), normal(g, m, 130, dtype=dtype)
    x, w = torch.empty(m, 0, dtype=dtype, device="cuda"), torch.empty(130, 0, dtype=dtype, device="cuda")
    y = sg.linear(x, w, b, activation="relu", residual=r)
    want = b.double().clamp(min=0) + r.double()
    check(y, want, 2 * UNIT[dtype] * want.abs() + TINY[dtype], "K = 0")
    assert sg.linear(x[:0], w, b).shape == (0, 130)
    assert sg.linear(x, w[:0]).shape == (m, 0)


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("m", [1, 40, 600])
def test_linear_residual_in_place(m, t):
    g, dtype = gen(5), TYPES[t]
    x, w, r = (normal(g, *s, dtype=dtype) for s in ((m, 256), (520, 256), (m, 520)))
    apart = sg.linear(x, w, residual=r)
    inplace = r.clone()
    assert sg.linear(x, w, residual=inplace, out=inplace) is inplace
    assert torch.equal(apart, inplace)


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("m", [1, 50, 700])
def test_linear_small_integers_exact(m, t):
    # products and sums are exact, so any order gives the same bits
    g, dtype = gen(9), TYPES[t]
    x = torch.randint(-2, 3, (m, 128), generator=g, device="cuda").to(dtype)
    w = torch.randint(-1, 2, (264, 128), generator=g, device="cuda").to(dtype)
    assert torch.equal(sg.linear(x, w).double(), (x.double() @ w.double().t()).to(dtype).double())


@pytest.mark.parametrize("t", ["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("m", [2, 100, 1500])
def test_linear_nan_and_infinity_stay_in_their_row(m, t):
    g = gen(4)
    x, w = normal(g, m, 256), normal(g, 300, 256, std=1 / 16)
    kw = {}
    if t == "e4m3":
        x, kw["x_scale"] = sg.quantize_rows(x)
        w, kw["w_scale"] = sg.quantize_rows(w)
        clean = sg.linear(x, w, **kw)
        x.view(torch.uint8)[m // 2, 17] = 0x7f
    else:
        x, w = x.to(TYPES[t]), w.to(TYPES[t])
        clean = sg.linear(x, w)
        x[m // 2, 17] = float("nan")
        x[0, 3] = float("inf")
    y = sg.linear(x, w, **kw)
    assert torch.isnan(y[m // 2]).all()
    keep = torch.ones(m, dtype=torch.bool, device="cuda")
    keep[m // 2] = False
    if t != "e4m3":
        keep[0] = False
        if m // 2 != 0:
            assert not torch.isfinite(y[0]).any()
    assert torch.equal(y[keep], clean[keep])


def test_linear_deterministic_streams_and_graph():
    g = gen(1)
    x, w, r = (normal(g, *s, dtype=torch.bfloat16) for s in ((200, 2048), (640, 2048), (200, 640)))
    first = sg.linear(x, w, residual=r, activation="gelu")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = sg.linear(x, w, residual=r, activation="gelu", stream=side)
    side.synchronize()
    assert torch.equal(first, other)
    raw = sg.linear(x, w, residual=r, activation="gelu", stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(first, raw)
    graph, out = torch.cuda.CUDAGraph(), torch.empty_like(first)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        sg.linear(x, w, residual=r, activation="gelu", out=out)
    x.mul_(0.5)
    want = sg.linear(x, w, residual=r, activation="gelu")
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


# ------------------------------------------------------------------ linear_backward


def run_backward(m, n, k, t, name="gelu", w_kn=False, pad=0, offset=0, seed=0):
    dtype = TYPES[t]
    g = gen(seed + 3 * m + 5 * n + 17 * k)
    x, w, z, dy = (normal(g, *s, dtype=dtype, std=std) for s, std in
                   (((m, k), 1), ((n, k), max(k, 1) ** -0.5), ((m, n), 1.5), ((m, n), 1)))
    ws = strided(w.t().contiguous(), pad, offset).t() if w_kn else strided(w, pad, offset)
    dx, dw, db = sg.linear_backward(strided(dy, pad, offset), strided(x, pad, offset), ws,
                                    strided(z, pad, offset) if name != "none" else None,
                                    activation=name)
    torch.cuda.synchronize()
    slope = act_grad(z.double(), name)
    dz = dy.double() * slope
    u = UNIT[dtype]
    # dZ: the slope's evaluation, and one rounding for the 16-bit types
    dz_err = 32 * EPS * dy.double().abs() * (1 + z.double().abs()) if name != "none" else 0 * dz
    if t != "f32" and name != "none":
        dz_err = dz_err + u * dz.abs() + TINY[dtype]
    what = f"{m}x{n}x{k} {t} {name} w_kn={w_kn} pad={pad}+{offset}"
    wd, xd = w.double(), x.double()
    for got, a, e, b, red, label in ((dx, dz, dz_err, wd, n, "dx"),
                                     (dw, dz.t(), dz_err.t(), xd, m, "dw")):
        want, S = a @ b, a.abs() @ b.abs()
        tol = product_tol(S, red, dtype) + e @ b.abs() + u * want.abs() + TINY[dtype]
        assert got.shape == want.shape
        check(got, want, tol + 1e-30, what + " " + label)
    want = dz.sum(0)
    tol = (m + 8) * EPS / 2 * dz.abs().sum(0) + (32 * EPS * dy.double().abs() *
                                                (1 + z.double().abs())).sum(0) + u * want.abs()
    check(db, want, tol + TINY[dtype], what + " db")


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("w_kn", [False, True])
@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (1, 300, 200), (3, 64, 520), (4, 1000, 72), (17, 96, 128),
                                   (64, 256, 512), (129, 257, 131), (500, 777, 301), (1000, 128, 1024),
                                   (4096, 264, 136), (2300, 2040, 264)])
def test_linear_backward_sizes(m, n, k, w_kn, t):
    run_backward(m, n, k, t, "gelu", w_kn)


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("name", ["none", "relu", "gelu", "gelu_erf", "silu"])
@pytest.mark.parametrize("m,pad,offset", [(2, 0, 0), (2, 3, 1), (200, 8, 0), (200, 0, 1), (200, 5, 2)])
def test_linear_backward_activations_and_strides(m, pad, offset, name, t):
    run_backward(m, 136, 208, t, name, False, pad, offset)
    run_backward(m, 135, 207, t, name, True, pad, offset)


def test_linear_backward_parts():
    g = gen(2)
    dy, x, w, z = (normal(g, *s, dtype=torch.bfloat16) for s in ((96, 64), (96, 80), (64, 80), (96, 64)))
    dx, dw, db = sg.linear_backward(dy, x, w, z, activation="silu")
    a = sg.linear_backward(dy, x, w, z, activation="silu", need_dw=False, need_db=False)
    b = sg.linear_backward(dy, x, w, z, activation="silu", need_dx=False, need_db=False)
    c = sg.linear_backward(dy, x, w, z, activation="silu", need_dx=False, need_dw=False)
    assert torch.equal(a[0], dx) and a[1] is None and a[2] is None
    assert torch.equal(b[1], dw) and b[0] is None
    assert torch.equal(c[2], db) and c[1] is None


@pytest.mark.parametrize("t", ["f32", "f16"])
@pytest.mark.parametrize("name", ["none", "silu"])
@pytest.mark.parametrize("m,n,k", [(9, 77, 130), (96, 64, 80), (301, 259, 130)])
def test_linear_backward_parts_give_the_same_bits(m, n, k, name, t):
    # what dZ is written as, and by which pass, follows from what is asked for
    g = gen(23)
    dy, x, w, z = (normal(g, *s, dtype=TYPES[t]) for s in ((m, n), (m, k), (n, k), (m, n)))
    z = z if name != "none" else None
    full = sg.linear_backward(dy, x, w, z, activation=name)
    for need in range(1, 8):
        some = sg.linear_backward(dy, x, w, z, activation=name, need_dx=bool(need & 1),
                                  need_dw=bool(need & 2), need_db=bool(need & 4))
        for i in range(3):
            if need >> i & 1:
                assert torch.equal(some[i], full[i]), (need, i)
            else:
                assert some[i] is None


@pytest.mark.parametrize("m,n,k,t", [(500, 777, 301, "f32"), (300, 264, 520, "bf16"), (1030, 520, 777, "f16"),
                                     (2560, 2560, 2600, "f32"), (2500, 2540, 8008, "bf16")])
def test_products_back_to_back_give_the_same_bits(m, n, k, t):
    # launches that overlap one another's ends: every call reads what the one
    # before it wrote, in the same memory, without waiting on the host
    g, dtype = gen(31), TYPES[t]
    x, w, z, dy = (normal(g, *s, dtype=dtype, std=std) for s, std in
                   (((m, k), 1), ((n, k), k ** -0.5), ((m, n), 1), ((m, n), 0.05)))

    def chain(wait):
        a, b, d, out = x.clone(), w.clone(), dy.clone(), []
        for _ in range(6):
            da, db, dbias = sg.linear_backward(d, a, b, z, activation="gelu")
            wait()
            y = sg.linear(da, b, residual=d, out=d)
            wait()
            d = sg.linear(a, db, activation="silu").mul_(1e-3).add_(y, alpha=0.1)
            wait()
            out += [da, db, dbias, y.clone(), d.clone()]
        return out
    apart = chain(torch.cuda.synchronize)
    for _ in range(3):
        for i, (p, q) in enumerate(zip(chain(lambda: None), apart)):
            assert torch.equal(p, q), i


@pytest.mark.parametrize("m,n,k,t", [(500, 777, 301, "f32"), (1024, 520, 776, "bf16")])
def test_linear_backward_in_a_graph_and_on_another_stream(m, n, k, t):
    g, dtype = gen(37), TYPES[t]
    x, w, z, dy = (normal(g, *s, dtype=dtype) for s in ((m, k), (n, k), (m, n), (m, n)))
    call = lambda **kw: sg.linear_backward(dy, x, w, z, activation="silu", **kw)  # noqa: E731
    first = call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = call(stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, other))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = [call() for _ in range(3)]      # launches of one call behind another's
        back = sg.linear(out[-1][0], out[-1][1])
    dy.mul_(0.5)
    x.mul_(2)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    want = call()
    for got in out:
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert torch.equal(back, sg.linear(want[0], want[1]))


@pytest.mark.parametrize("t", ["f32", "bf16"])
def test_linear_backward_empty(t):
    d = TYPES[t]
    e = lambda *s: torch.ones(*s, dtype=d, device="cuda")  # noqa: E731
    dx, dw, db = sg.linear_backward(e(0, 6), e(0, 5), e(6, 5))
    assert dx.shape == (0, 5) and not dw.any() and dw.shape == (6, 5) and not db.any()
    dx, dw, db = sg.linear_backward(e(4, 0), e(4, 5), e(0, 5))
    assert not dx.any() and dx.shape == (4, 5) and dw.shape == (0, 5)
    dx, dw, db = sg.linear_backward(e(4, 6), e(4, 0), e(6, 0))
    assert dx.shape == (4, 0) and torch.equal(db, 4 * e(6))


@pytest.mark.parametrize("name", ["none", "gelu", "gelu_erf", "silu"])
def test_linear_gradient_against_differences(name):
    """<dL/dp, v> against the central difference of L = <dy, y> in 64 bits
    along v.  The difference errs by h^2 / 6 times a third derivative (below
    4 |v|^3 terms here), far under the gradient's own fp32 error, which is held
    to 1e-5 of the norms' product."""
    g, h = gen(8), 1e-4
    m, n, k = 40, 72, 56
    x, w, b, dy = normal(g, m, k), normal(g, n, k, std=k ** -0.5), normal(g, n), normal(g, m, n)
    _, z = sg.linear(x, w, b, activation=name, save_preact=True)
    dx, dw, db = sg.linear_backward(dy, x, w, z, activation=name)

    def loss(x, w, b):
        return (dy.double() * act(x @ w.t() + b, name)).sum()

    p = [t.double() for t in (x, w, b)]
    for i, grad in enumerate((dx, dw, db)):
        v = torch.randn(p[i].shape, generator=g, device="cuda", dtype=torch.float64)
        plus, minus = list(p), list(p)
        plus[i], minus[i] = p[i] + h * v, p[i] - h * v
        diff = (loss(*plus) - loss(*minus)) / (2 * h)
        along = (grad.double() * v).sum()
        scale = grad.double().norm() * v.norm()
        assert abs(float(diff - along)) <= 1e-5 * float(scale) + 1e-6, (name, i)


# ------------------------------------------------------------------ norm and quantiser


def codes_ok(q, exact, what):
    """q is `exact` rounded to e4m3: off by at most half the spacing there
    (the spacing is 2^(e-3) for 2^e <= |v| < 2^(e+1), 2^-9 below 2^-6), plus
    what 32-bit arithmetic moves the value before rounding (2^-17)."""
    v = exact.abs().clamp(max=448.0)
    e = torch.floor(torch.log2(v.clamp(min=2.0 ** -6)))
    check(q, exact, 0.5 * 2.0 ** (e - 3) * (1 + 2.0 ** -20) + 2.0 ** -17 * v, what)


NORM_SIZES = [(1, 1), (1, 4096), (3, 7), (5, 64), (9, 200), (33, 256), (40, 1001), (700, 4096),
              (2, 8192), (310, 8192), (2, 16384), (311, 16000), (2, 40000), (3, 9001), (5000, 72)]


def run_norm(rows, d, t, residual=True, quantize=False, pad=0, offset=0):
    dtype = TYPES[t]
    g = gen(rows + 31 * d)
    x, r = normal(g, rows, d, dtype=dtype), normal(g, rows, d, dtype=dtype)
    w = (1 + normal(g, d, std=0.2)).to(dtype)
    got = sg.add_rmsnorm(strided(x, pad, offset), w, strided(r, pad, offset) if residual else None,
                         eps=1e-5, quantize=quantize)
    torch.cuda.synchronize()
    s = x.double() + (r.double() if residual else 0)
    rstd = 1 / torch.sqrt(s.square().mean(1) + 1e-5)
    y = s * rstd[:, None] * w.double()
    # a sum of d positive terms, at most d / 32 + 64 of them one after another
    rel = (d / 32 + 72) * EPS
    what = f"{rows}x{d} {t} residual={residual} quantize={quantize} pad={pad}+{offset}"
    check(got[-1], rstd, rel * rstd, what + " rstd")
    check(got[-2], s, UNIT[dtype] * s.abs() + TINY[dtype], what + " s")
    if quantize:
        q, scale = got[:2]
        want = y.abs().amax(1) / 448
        check(scale, want, (rel + 8 * EPS) * want, what + " scale")
        codes_ok(q, y / scale.double()[:, None], what + " codes")
    else:
        check(got[0], y, (UNIT[dtype] + rel + 4 * EPS) * y.abs() + TINY[dtype], what + " y")


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("quantize", [False, True])
@pytest.mark.parametrize("rows,d", NORM_SIZES)
def test_add_rmsnorm_sizes(rows, d, quantize, t):
    run_norm(rows, d, t, True, quantize)
    run_norm(rows, d, t, False, quantize)


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("quantize", [False, True])
@pytest.mark.parametrize("pad,offset", [(8, 0), (3, 0), (0, 1), (5, 3)])
def test_add_rmsnorm_strides(pad, offset, quantize, t):
    run_norm(20, 512, t, True, quantize, pad, offset)
    run_norm(400, 520, t, False, quantize, pad, offset)


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
def test_add_rmsnorm_special_rows(t):
    dtype = TYPES[t]
    x = normal(gen(0), 6, 256, dtype=dtype)
    w = torch.ones(256, dtype=dtype, device="cuda")
    clean = sg.add_rmsnorm(x, w)[0]
    x[1] = 0
    x[2, 5] = float("nan")
    x[3, 7] = float("inf")
    y, s, rstd = sg.add_rmsnorm(x, w, eps=1e-6)
    q, scale, _, _ = sg.add_rmsnorm(x, w, eps=1e-6, quantize=True)
    assert not y[1].any() and torch.isfinite(rstd[1])
    assert torch.isnan(y[2]).all() and torch.isnan(rstd[2])
    assert torch.isnan(y[3, 7]) and rstd[3] == 0
    for i in (0, 4, 5):
        assert torch.equal(y[i], clean[i])
    assert not q[1].float().any() and float(scale[1]) == pytest.approx(1e-30 / 448, rel=1e-6)
    assert torch.isnan(q[2].float()).all() and torch.isnan(scale[2])
    assert torch.isfinite(q[4].float()).all()


def run_norm_backward(rows, d, t, stream=True, pad=0, offset=0):
    dtype = TYPES[t]
    g = gen(rows + 37 * d)
    s, dy, ds = (normal(g, rows, d, dtype=dtype) for _ in range(3))
    w = (1 + normal(g, d, std=0.2)).to(dtype)
    rstd = torch.rsqrt(s.float().square().mean(1) + 1e-6)
    dx, dw = sg.add_rmsnorm_backward(strided(dy, pad, offset), strided(s, pad, offset), rstd, w,
                                     strided(ds, pad, offset) if stream else None)
    torch.cuda.synchronize()
    S, DY, W, R = s.double(), dy.double(), w.double(), rstd.double()[:, None]
    gg = DY * W
    mean = (gg * S).mean(1, keepdim=True)
    want = R * (gg - S * R * R * mean) + (ds.double() if stream else 0)
    rel = (d / 32 + 72) * EPS
    tol = (UNIT[dtype] * want.abs() + rel * (R ** 3 * S.abs() * (gg * S).abs().mean(1, keepdim=True)) +
           16 * EPS * (R * gg.abs() + want.abs()) + TINY[dtype])
    what = f"{rows}x{d} {t} ds={stream} pad={pad}+{offset}"
    check(dx, want, tol, what + " dx")
    want = (DY * S * R).sum(0)
    tol = UNIT[dtype] * want.abs() + (rows + 8) * EPS / 2 * (DY * S * R).abs().sum(0) + TINY[dtype]
    check(dw, want, tol, what + " dw")


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,d", NORM_SIZES)
def test_add_rmsnorm_backward_sizes(rows, d, t):
    run_norm_backward(rows, d, t, True)
    run_norm_backward(rows, d, t, False)


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("pad,offset", [(8, 0), (3, 0), (0, 1), (5, 3)])
def test_add_rmsnorm_backward_strides(pad, offset, t):
    run_norm_backward(20, 512, t, True, pad, offset)
    run_norm_backward(400, 520, t, True, pad, offset)


def test_add_rmsnorm_backward_empty_and_parts():
    e = lambda *s: torch.ones(*s, device="cuda")  # noqa: E731
    dx, dw = sg.add_rmsnorm_backward(e(0, 8), e(0, 8), e(0), e(8))
    assert dx.shape == (0, 8) and not dw.any()
    dy, s = normal(gen(1), 30, 64), normal(gen(2), 30, 64)
    both = sg.add_rmsnorm_backward(dy, s, e(30), e(64))
    only = sg.add_rmsnorm_backward(dy, s, e(30), e(64), need_dweight=False)
    assert torch.equal(both[0], only[0]) and only[1] is None


def test_add_rmsnorm_gradient_against_differences():
    """As the linear layer's: L = <dy, y> + <ds, s> in 64 bits, along x, the
    residual and the weight."""
    g, h = gen(6), 1e-4
    rows, d = 24, 136
    x, r, dy, ds = (normal(g, rows, d) for _ in range(4))
    w = 1 + normal(g, d, std=0.2)
    _, s, rstd = sg.add_rmsnorm(x, w, r, eps=1e-3)
    dx, dw = sg.add_rmsnorm_backward(dy, s, rstd, w, ds)

    def loss(x, r, w):
        s = x + r
        y = s / torch.sqrt(s.square().mean(1, keepdim=True) + 1e-3) * w
        return (dy.double() * y).sum() + (ds.double() * s).sum()

    p = [t.double() for t in (x, r, w)]
    for i, grad in enumerate((dx, dx, dw)):
        v = torch.randn(p[i].shape, generator=g, device="cuda", dtype=torch.float64)
        plus, minus = list(p), list(p)
        plus[i], minus[i] = p[i] + h * v, p[i] - h * v
        diff = (loss(*plus) - loss(*minus)) / (2 * h)
        along = (grad.double() * v).sum()
        assert abs(float(diff - along)) <= 1e-5 * float(grad.double().norm() * v.norm()) + 1e-6, i


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,d", NORM_SIZES)
def test_quantize_rows(rows, d, t):
    for pad, offset in ((0, 0), (3, 1)):
        x = normal(gen(rows + d), rows, d, dtype=TYPES[t])
        x[0] = 0
        q, scale = sg.quantize_rows(strided(x, pad, offset))
        want = x.double().abs().amax(1).clamp(min=1e-30) / 448
        check(scale, want, 4 * EPS * want, "scale")
        codes_ok(q, x.double() / scale.double()[:, None], f"{rows}x{d} {t}")
        assert not q[0].float().any()


@pytest.mark.parametrize("rows,cols", [(64, 256), (7, 1001)])
def test_quantize_rows_matches_the_definition_bit_for_bit(rows, cols):
    # torch's own conversion of x * (448 / a), formed in fp32; the scale by
    # numpy's division (torch divides by a Python number through its reciprocal)
    x = normal(gen(3), rows, cols)
    q, scale = sg.quantize_rows(x)
    a = x.abs().amax(1)
    want = (x * (448.0 / a)[:, None]).to(torch.float8_e4m3fn)
    assert torch.equal(q.view(torch.uint8), want.view(torch.uint8))
    assert np.array_equal(scale.cpu().numpy(), a.cpu().numpy() / np.float32(448))


def test_feed_forward_block():
    """norm -> up-projection -> down-projection + residual, in bf16 and with
    8-bit rows, against the block in 64 bits.  bf16: three roundings on the way
    (y, the hidden activation, the result) of 2^-8 each, averaged by the sums;
    e4m3: two roundings of 2^-4 relative.  Held in the 2-norm: 1 % and 8 %."""
    g = gen(12)
    t, d, f = 70, 512, 1024
    x, res = normal(g, t, d, dtype=torch.bfloat16), normal(g, t, d, dtype=torch.bfloat16)
    w = (1 + normal(g, d, std=0.1)).to(torch.bfloat16)
    w1, w2 = (normal(g, *s, dtype=torch.bfloat16, std=s[1] ** -0.5) for s in ((f, d), (d, f)))
    b1 = normal(g, f, dtype=torch.bfloat16, std=0.1)
    S = x.double() + res.double()
    Y = S / torch.sqrt(S.square().mean(1, keepdim=True) + 1e-6) * w.double()
    want = act(Y @ w1.double().t() + b1.double(), "gelu") @ w2.double().t() + S
    y, s, _ = sg.add_rmsnorm(x, w, res)
    got = sg.linear(sg.linear(y, w1, b1, activation="gelu"), w2, residual=s)
    assert float((got.double() - want).norm() / want.norm()) < 0.01
    q1, s1 = sg.quantize_rows(w1)
    q2, s2 = sg.quantize_rows(w2)
    q, qs, s, _ = sg.add_rmsnorm(x, w, res, quantize=True)
    hidden = sg.linear(q, q1, b1, activation="gelu", x_scale=qs, w_scale=s1)
    hq, hs = sg.quantize_rows(hidden)
    got = sg.linear(hq, q2, residual=s, x_scale=hs, w_scale=s2)
    assert float((got.double() - want).norm() / want.norm()) < 0.08


@pytest.mark.parametrize("t", ["bf16", "f16"])
def test_feed_forward_example(t):
    """The example block learns (a gradient step along the exact gradient lowers
    this smooth loss), and its 8-bit form stays near it: two roundings of 2^-4
    relative to 8 bits on the way, averaged by the sums, under 8 %."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "feed_forward.py")
    spec = importlib.util.spec_from_file_location("feed_forward_example", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    losses, off = example.run(130, 256, 512, 12, TYPES[t])
    assert all(b < a for a, b in zip(losses, losses[1:])), losses
    assert losses[-1] < 0.9 * losses[0]
    assert off < 0.08
