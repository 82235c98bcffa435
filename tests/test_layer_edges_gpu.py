"""The layer operators on the GPU where they can go wrong: empty rows, the
activations' tails and limits, special values, devices, overlapping launches."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import dense_fp32_matrix_sgemm_gb300 as sg  # noqa: E402

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def no_pipeline_errors():
    sg.device_status(reset=True)
    yield
    assert sg.device_status(reset=True) == 0


# ------------------------------------------------------------------ devices


def test_operands_on_the_host_are_refused():
    # (of two GPUs' tensors: the host tests' comparison, which every operand goes through)
    x, w = torch.ones(4, 8, device="cuda"), torch.ones(16, 8, device="cuda")
    v, rstd = torch.ones(8, device="cuda"), torch.ones(4, device="cuda")
    host = lambda t: t.cpu()  # noqa: E731
    for call in (lambda: sg.linear(x, host(w)), lambda: sg.linear(x, w, host(v.repeat(2))),
                 lambda: sg.linear(x, w, residual=host(x @ w.t())),
                 lambda: sg.linear(x, w, out=host(x @ w.t())),
                 lambda: sg.linear(torch.ones(32, 8, device="cuda"), w,
                                   workspace=torch.zeros(1 << 20, dtype=torch.uint8)),
                 lambda: sg.linear_backward(x @ w.t(), host(x), w),
                 lambda: sg.add_rmsnorm(x, host(v)), lambda: sg.add_rmsnorm(x, v, host(x)),
                 lambda: sg.add_rmsnorm_backward(x, x, host(rstd), v),
                 lambda: sg.add_rmsnorm_backward(x, host(x), rstd, v)):
        with pytest.raises((TypeError, ValueError)):
            call()
    torch.cuda.synchronize()


def test_calls_leave_the_current_device():
    at = torch.cuda.current_device()
    sg.quantize_rows(torch.ones(4, 8, device="cuda"))
    assert torch.cuda.current_device() == at


# ------------------------------------------------------------------ rows of no elements


def poisoned(*shape):
    """The allocator's next block of this size holds NaN."""
    t = torch.full(shape, float("nan"), device="cuda")
    del t


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("rows", [1, 4, 700])
def test_rows_of_no_elements_have_scales(rows, t):
    # 1e-30 / 448 and eps^(-1/2), each formed in fp32 with two roundings at most
    x = torch.empty(rows, 0, dtype=TYPES[t], device="cuda")
    w = torch.empty(0, dtype=TYPES[t], device="cuda")
    ones = torch.ones(rows, dtype=torch.float64)
    poisoned(rows)
    q, scale = sg.quantize_rows(x)
    assert q.shape == (rows, 0) and q.dtype == torch.float8_e4m3fn
    torch.testing.assert_close(scale.cpu().double(), ones * (1e-30 / 448), rtol=2.0 ** -22, atol=0)
    for residual in (None, x.clone()):
        poisoned(rows)
        y, s, rstd = sg.add_rmsnorm(x, w, residual, eps=0.25)
        assert y.shape == s.shape == (rows, 0)
        assert torch.equal(rstd.cpu().double(), 2 * ones)
        poisoned(rows)
        q, scale, s, rstd = sg.add_rmsnorm(x, w, residual, eps=0.25, quantize=True)
        torch.testing.assert_close(scale.cpu().double(), ones * (1e-30 / 448), rtol=2.0 ** -22, atol=0)
        assert torch.equal(rstd.cpu().double(), 2 * ones)


@pytest.mark.parametrize("out", ["bf16", "f16"])
@pytest.mark.parametrize("m", [1, 9, 300])
def test_linear_e4m3_without_inputs(m, out):
    # K = 0: act(bias) + residual, two exact terms and one rounding, whatever the scales hold
    d = TYPES[out]
    x, w = (torch.empty(r, 0, dtype=torch.float8_e4m3fn, device="cuda") for r in (m, 130))
    b = torch.linspace(-3, 3, 130, device="cuda").to(d)
    r = torch.linspace(-1, 1, m * 130, device="cuda").view(m, 130).to(d)
    want = (b.double().clamp(min=0) + r.double()).float().to(d)
    for value in (float("nan"), float("inf"), 1.0):
        xs, ws = (torch.full((n,), value, device="cuda") for n in (m, 130))
        assert torch.equal(sg.linear(x, w, b, activation="relu", residual=r, x_scale=xs, w_scale=ws,
                                     out_dtype=d), want)
    xs = sg.quantize_rows(torch.empty(m, 0, device="cuda"))[1]
    ws = sg.quantize_rows(torch.empty(130, 0, device="cuda"))[1]
    assert torch.equal(sg.linear(x, w, b, activation="relu", residual=r, x_scale=xs, w_scale=ws,
                                 out_dtype=d), want)


# ------------------------------------------------------------------ activations


def slopes(z, name):
    """act'(z) by the bias gradient of one row with dY = 1."""
    z = z.view(1, -1)
    x, w = (torch.zeros(n, 1, dtype=z.dtype, device="cuda") for n in (1, z.shape[1]))
    return sg.linear_backward(torch.ones_like(z), x, w, z, activation=name, need_dx=False,
                              need_dw=False)[2]


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("name", ["relu", "gelu", "gelu_erf", "silu"])
def test_slopes_at_large_and_infinite_z(name, t):
    # exactly 0 or 1: the exponentials in them are below 2^-149 or their complements
    big = [300.0, 65504.0, float("inf")] + ([] if t == "f16" else [1e13, 1e14, 2e19, 1e30, 3e38])
    for n in (len(big), 8 * len(big), 8 * len(big) + 1):     # single elements, 16-byte accesses
        z = torch.tensor(big * 9, device="cuda")[:n].to(TYPES[t])
        assert torch.equal(slopes(z, name).float(), torch.ones(n, device="cuda"))
        assert torch.equal(slopes(-z, name).float().abs(), torch.zeros(n, device="cuda"))
    if name != "relu":
        assert torch.isnan(slopes(torch.full((17,), float("nan"), device="cuda", dtype=TYPES[t]),
                                  name)).all()


@pytest.mark.parametrize("t", TYPES)
def test_gradients_where_the_stored_z_has_overflowed(t):
    # an infinite z in one place changes nothing but that place's slope
    d, inf = TYPES[t], float("inf")
    g = torch.Generator(device="cuda").manual_seed(5)
    dy, z, x, w = (torch.randn(*s, generator=g, device="cuda").to(d)
                   for s in ((40, 64), (40, 64), (40, 72), (64, 72)))
    z[3, 5], z[7, 9] = inf, -inf
    for name in ("gelu", "gelu_erf", "silu"):
        got = sg.linear_backward(dy, x, w, z, activation=name)
        near = z.clone()
        near[3, 5], near[7, 9] = 300.0, -300.0    # slopes 1 and 0 to the last bit
        for a, b in zip(got, sg.linear_backward(dy, x, w, near, activation=name)):
            assert torch.equal(a, b)


UNIT = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
STEP = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}   # smallest


def values(z, name, m):
    """act(z) in m rows, z coming in as the bias (m > 16: on the tensor cores)."""
    x, w = (torch.zeros(n, 64, dtype=z.dtype, device="cuda") for n in (m, z.numel()))
    return sg.linear(x, w, z, activation=name)


def within(got, want, rel, what):
    """rel of the value and half a step of the type's smallest values (rounding
    there is absolute), both of them per element."""
    err = (got.double() - want).abs()
    tol = rel * want.abs() + 0.75 * STEP[got.dtype]
    assert (err <= tol).all(), (what, float((err / tol).max()), int((err / tol).argmax()))


@pytest.mark.parametrize("t", TYPES)
def test_erf_gelu_keeps_its_relative_accuracy(t):
    """z Phi(z) and Phi(z) + z phi(z) for z in [-12, 12] against erfc in 64 bits.
    Phi's argument z / sqrt 2, or z^2 / 2 in an exponent, carries 1.5 roundings of
    2^-24, which the tail magnifies by at most z^2 + 2; the functions called err by 4
    units of 2^-23 at most, the products and sums by 2^-24 each: 16 2^-24 together;
    the 16-bit types' own form adds the fit's 1.3e-6 and two hardware functions of
    2^-22 each: 32 2^-24.  The slope's two terms have either sign: their sizes
    count."""
    d = TYPES[t]
    z = torch.linspace(-12, 12, 4001, dtype=torch.float64).to(d)
    z = z[: 4000 if t == "f32" else 4001].cuda()
    zd = z.double()
    phi = torch.exp(-0.5 * zd * zd) * 0.3989422804014326779
    Phi = 0.5 * torch.special.erfc(-zd * 0.70710678118654752440)
    rel = (1.5 * (zd * zd + 2) + 16 + (0 if t == "f32" else 32)) * 2.0 ** -24
    for m in (1, 200):
        y = values(z, "gelu_erf", m)
        within(y, (zd * Phi).expand(m, -1), (rel + UNIT[d]).expand(m, -1), f"value, {m} rows")
    want, size = Phi + zd * phi, Phi + zd.abs() * phi
    err = (slopes(z, "gelu_erf").double() - want).abs()
    assert (err <= rel * size + UNIT[d] * want.abs() + 0.75 * STEP[d]).all(), float(err.max())


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("name,low", [("silu", -104.0), ("gelu", -12.0)])
def test_activations_in_the_far_tail(name, low, t):
    """z p(z) and its slope, p = 1 / (1 + exp(-v)), where p is near or below the
    smallest normal number (2^-126), against 64 bits.  v = z, or 2 sqrt(2/pi) (z +
    0.044715 z^3) with 5 roundings, enters an exponential: (6 |v| + 16) 2^-24 relative.
    A p below 2^-126 has an absolute error of up to 2^-149 in fp32, which z, or the
    slope's factor f, multiplies."""
    d = TYPES[t]
    z = torch.linspace(low, 0.75 * low, 801, dtype=torch.float64).to(d)
    z = z[: 800 if t == "f32" else 801].cuda()
    zd = z.double()
    if name == "silu":
        v, dv = zd, torch.ones_like(zd)
    else:
        c = (8 / torch.pi) ** 0.5
        v, dv = c * (zd + 0.044715 * zd ** 3), c * (1 + 3 * 0.044715 * zd ** 2)
    p = torch.exp(v) / (1 + torch.exp(v))
    f = 1 + zd * dv * (1 - p)
    rel = (6 * v.abs() + 16) * 2.0 ** -24 + UNIT[d]
    for m in (1, 200):
        y = values(z, name, m)
        err, tol = (y.double() - zd * p).abs(), rel * (zd * p).abs() + 2.0 ** -149 * zd.abs()
        assert (err <= tol + 0.75 * STEP[d]).all(), (m, float((err / tol).max()))
    err = (slopes(z, name).double() - p * f).abs()
    tol = rel * p * (1 + (zd * dv).abs()) + 2.0 ** -149 * f.abs()
    assert (err <= tol + 0.75 * STEP[d]).all(), float((err / tol).max())


# ------------------------------------------------------------------ norm gradient


@pytest.mark.parametrize("t", TYPES)
def test_norm_gradient_of_constant_rows_is_zero(t):
    """dY = s = w = rstd = 1: dX = 1 - mean(1).  Sums of D ones are exact in any
    order up to 2^24, so is D / D; D times a rounded 1 / D is not always 1 (here for
    several of the widths, both kernels)."""
    for d in (1, 3, 41, 47, 49, 61, 82, 83, 98, 97, 103, 328, 1001, 1312, 2048, 4099, 6150, 9001, 40000):
        one = torch.ones(5, d, dtype=TYPES[t], device="cuda")
        dx, dw = sg.add_rmsnorm_backward(one, one, torch.ones(5, device="cuda"), one[0].contiguous())
        assert not dx.any(), d
        assert torch.equal(dw, 5 * one[0]), d


# ------------------------------------------------------------------ torch


def test_out_counts_as_changed_in_place():
    x, w = torch.ones(4, 8, device="cuda"), torch.ones(16, 8, device="cuda")
    r = torch.ones(4, 16, device="cuda")
    before = r._version
    sg.linear(x, w, residual=r, out=r)
    assert r._version == before + 1
    # so a product's backward that saved it is refused, as after any change in place
    p = torch.ones(16, 4, device="cuda", requires_grad=True)
    y = (r @ p).sum()
    sg.linear(x, w, out=r)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
    with torch.inference_mode():
        o = torch.empty(4, 16, device="cuda")
        assert torch.equal(sg.linear(x, w, out=o), torch.full((4, 16), 8.0, device="cuda"))


def test_results_record_no_gradient():
    x = torch.ones(4, 8, device="cuda", requires_grad=True)
    w = torch.ones(16, 8, device="cuda", requires_grad=True)
    assert not sg.linear(x, w).requires_grad
    assert not any(t.requires_grad for t in sg.add_rmsnorm(x, w[0].detach(), x))


def test_memory_running_out_is_torchs_error():
    # (refused by torch's allocator at the limit set here, before the device is asked)
    x, w = (torch.ones(1 << 15, 1, device="cuda") for _ in range(2))
    torch.cuda.empty_cache()
    torch.cuda.set_per_process_memory_fraction(0.01)
    try:
        with pytest.raises(torch.OutOfMemoryError):
            sg.linear(x, w)      # 4 GB
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    assert torch.equal(sg.linear(x[:4], w[:8]), torch.ones(4, 8, device="cuda"))


def test_an_argument_without_a_truth_value_is_its_own_error():
    x, w = torch.ones(4, 8, device="cuda"), torch.ones(16, 8, device="cuda")

    class Undecided:
        def __bool__(self):
            raise ValueError("neither")

    for call in (lambda u: sg.linear(x, w, save_preact=u), lambda u: sg.add_rmsnorm(x, w[0], quantize=u),
                 lambda u: sg.linear_backward(x @ w.t(), x, w, need_db=u),
                 lambda u: sg.add_rmsnorm_backward(x, x, x[:, 0].contiguous(), w[0], need_dweight=u)):
        with pytest.raises(ValueError, match="neither"):
            call(Undecided())
    assert sg.linear(x, w, save_preact=1)[1].shape == (4, 16)


# ------------------------------------------------------------------ special values


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("d", [256, 257, 40000])
def test_quantize_rows_special_rows(d, t):
    # a = max |x|: a NaN makes scale and codes NaN; an infinity makes the scale
    # infinite, 448 / a 0, its own code NaN (inf 0) and the others 0
    x = torch.randn(6, d, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").to(TYPES[t])
    clean_q, clean_scale = sg.quantize_rows(x)
    x[1, d - 1], x[2, 0], x[3, 5] = float("nan"), float("inf"), -float("inf")
    q, scale = sg.quantize_rows(x)
    f = q.float()
    assert torch.isnan(scale[1]) and torch.isnan(f[1]).all()
    for row, col in ((2, 0), (3, 5)):
        assert torch.isinf(scale[row]) and scale[row] > 0
        assert torch.isnan(f[row, col])
        f[row, col] = 0
        assert not f[row].any()
    for row in (0, 4, 5):
        assert torch.equal(q[row].view(torch.uint8), clean_q[row].view(torch.uint8))
        assert torch.equal(scale[row], clean_scale[row])


@pytest.mark.parametrize("w_kn", [False, True])
@pytest.mark.parametrize("m", [1, 8, 16, 17, 200])
def test_linear_f32_infinities(m, w_kn):
    """An infinity in X reaches its own row, one in W its own feature, all of their
    values non-finite and nobody else's changed; up to 16 rows (FP32 FMAs) they are
    the formula's infinities, above (differences of infinities) they may be NaN."""
    g = torch.Generator(device="cuda").manual_seed(2)
    x, w = torch.randn(m, 96, generator=g, device="cuda"), torch.randn(130, 96, generator=g, device="cuda")
    make = (lambda w: w.t().contiguous().t()) if w_kn else (lambda w: w)
    clean = sg.linear(x, make(w))
    bad = x.clone()
    bad[m // 2, 7] = float("inf")
    y = sg.linear(bad, make(w))
    rest = torch.arange(m, device="cuda") != m // 2
    assert torch.equal(y[rest], clean[rest]) and not torch.isfinite(y[m // 2]).any()
    if m <= 16:
        assert torch.equal(y[m // 2], torch.where(w[:, 7] > 0, float("inf"), -float("inf")))
    bad = w.clone()
    bad[50, 3] = -float("inf")
    y = sg.linear(x, make(bad))
    rest = torch.arange(130, device="cuda") != 50
    assert torch.equal(y[:, rest], clean[:, rest]) and not torch.isfinite(y[:, 50]).any()
    if m <= 16:
        assert torch.equal(y[:, 50], torch.where(x[:, 3] > 0, -float("inf"), float("inf")))


@pytest.mark.parametrize("m", [1, 2, 3, 40, 300])
@pytest.mark.parametrize("k", [200, 201, 208])
@pytest.mark.parametrize("pad,offset", [(0, 0), (3, 1), (8, 0), (16, 8)])
def test_linear_e4m3_to_f16_of_any_alignment(pad, offset, k, m):
    """Codes and scales whose products and sums are exact in fp32 (codes of -2 .. 2,
    scales of powers of two): one rounding to f16, the same bits as torch's."""
    g = torch.Generator(device="cuda").manual_seed(k + m)
    n = 131

    def strided(t):
        buf = torch.full((t.shape[0] * (t.shape[1] + pad) + offset,), 0x7f if t.element_size() == 1 else 0,
                         dtype=torch.uint8 if t.element_size() == 1 else t.dtype, device="cuda")
        v = buf[offset:].view(t.shape[0], t.shape[1] + pad)[:, :t.shape[1]]
        v.copy_(t.view(torch.uint8) if t.element_size() == 1 else t)
        return v.view(t.dtype)

    x, w = (torch.randint(-2, 3, s, generator=g, device="cuda").float().to(torch.float8_e4m3fn)
            for s in ((m, k), (n, k)))
    xs, ws = (2.0 ** torch.randint(-3, 2, (s,), generator=g, device="cuda").float() for s in (m, n))
    r = strided(torch.randint(-8, 9, (m, n), generator=g, device="cuda").half())
    out = strided(torch.zeros(m, n, dtype=torch.float16, device="cuda"))
    y = sg.linear(strided(x), strided(w), activation="relu", residual=r, x_scale=xs, w_scale=ws,
                  out_dtype=torch.float16, out=out)
    z = (x.double() @ w.double().t()) * xs.double()[:, None] * ws.double()
    assert torch.equal(y, (z.clamp(min=0) + r.double()).float().half())


@pytest.mark.parametrize("e", [-108, -113, -119, -125])
@pytest.mark.parametrize("m", [16, 64])
def test_linear_f32_of_tiny_elements(m, e):
    """Elements of 2^e, normal f32 numbers.  By FP32 FMAs, K = 256 updates of half a
    unit of the sum of sizes S; on the tensor cores 64 2^-23 / 4 + 2^-19 of S as for
    any f32 product, and every tiny element to 2^-134."""
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(m, 256, generator=g, device="cuda").clamp(-4, 4)
    w = torch.randn(130, 256, generator=g, device="cuda")
    tiny = torch.ldexp(x, torch.tensor(e, device="cuda"))
    want, S = tiny.double() @ w.double().t(), tiny.double().abs() @ w.double().abs().t()
    tol = (256 * 2.0 ** -24 if m <= 16 else 2.0 ** -19 + (64 + 32) * 2.0 ** -25) * S
    if m > 16:
        tol = tol + 2.0 ** -134 * w.double().abs().sum(1)
    assert ((sg.linear(tiny, w).double() - want).abs() <= tol + 2.0 ** -149 * 256).all()
    if m > 16:      # the same of a weight
        y = sg.linear(w, tiny).double()
        assert ((y - want.t()).abs() <= tol.t() + 2.0 ** -149 * 256).all()
