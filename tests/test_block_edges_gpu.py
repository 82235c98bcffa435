"""The gated block's operators on the GPU where they can go wrong, against 64 bits.

EPS = 2^-23, u the output's unit roundoff, 2^-150 half of fp32's smallest step.
"""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import dense_fp32_matrix_sgemm_gb300 as sg  # noqa: E402
from test_layers_gpu import EPS, TYPES, UNIT, check, gen, normal  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def no_pipeline_errors():
    sg.device_status(reset=True)
    yield
    assert sg.device_status(reset=True) == 0


# ------------------------------------------------------------------ clip_grad_norm

# Roundings on the way to a sum of squares: a thread's FMAs of 16 (f32: 8) squares in each of two
# chains, their join, five additions across the warp; from there on 64 bits hold the sum.  Each
# errs by EPS / 2 of a sum of positive terms, and the square root halves that.
NORM_TOL = {t: (n + 6) / 4 * EPS for t, n in ((torch.float32, 8), (torch.bfloat16, 16), (torch.float16, 16))}


def check_clipped(tensors, max_norm, how, eps=1e-6):
    """Clips copies of `tensors` in place or into `out`, or takes the norm alone (`how`)."""
    norm = math.sqrt(sum(float(t.double().square().sum()) for t in tensors if t.numel()))
    factor = min(1.0, max_norm / (norm + eps))
    tol = max(NORM_TOL[t.dtype] for t in tensors)
    given = [t.clone() for t in tensors]
    if how == "norm":
        result, got, factor = sg.grad_norm(given), given, 1.0
    elif how == "in place":
        result, got = sg.clip_grad_norm(given, max_norm, eps=eps), given
    else:
        got = [torch.full_like(t, float("nan")) for t in tensors]
        result = sg.clip_grad_norm(given, max_norm, eps=eps, out=got)
    # (the norm is rounded once; a bound for the second order of all that)
    assert abs(float(result) - norm) <= 1.001 * (tol + EPS / 2) * norm, (float(result), norm)
    flat = lambda ts: torch.cat([t.double().flatten() for t in ts])  # noqa: E731
    want = flat(tensors) * factor
    # the factor and the product are rounded in fp32, the result to its type
    each = lambda f: torch.cat([torch.full((t.numel(),), f(t.dtype), dtype=torch.float64, device="cuda")  # noqa: E731
                                for t in tensors])
    step = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}   # half of the smallest
    check(flat(got), want, (1.001 * (tol + EPS) + each(UNIT.get)) * want.abs() + each(step.get) +
          1.01 * 2.0 ** -150, how)
    if how == "out":
        assert all(torch.equal(a, b) for a, b in zip(given, tensors))


HOW = ("in place", "out", "norm")


@pytest.mark.parametrize("how", HOW)
@pytest.mark.parametrize("empty", [0, 1, 2, 1000])
@pytest.mark.parametrize("full", [31, 32, 33, 255, 256, 257, 999, 1000, 1001, 2000])
def test_clip_lists_with_empty_tensors(full, empty, how):
    # behind as many tensors as a launch's table holds, before them and among them
    g = gen(full)
    flat = normal(g, full * 5)
    some, none = list(flat.view(full, 5)), [flat[:0]] * empty
    check_clipped(some + none, 1.0, how)
    if empty > 0:
        check_clipped(none + some, 1.0, how)
        check_clipped(none + some[:full // 2] + none + some[full // 2:] + none, 1.0, how)


@pytest.mark.parametrize("how", HOW)
def test_clip_lists_of_empty_tensors(how):
    for count in (1, 33, 257, 1000, 1001, 2300):
        check_clipped([torch.empty(0, device="cuda")] * count, 1.0, how)


@pytest.mark.parametrize("how", HOW)
@pytest.mark.parametrize("types", [("f32",), ("bf16",), ("f16",), ("bf16", "f32", "f16")])
def test_clip_errs_by_its_roundings(types, how):
    # the largest errors are those of whole chunks of equal elements, whose roundings agree
    for value in (1.0 / 3, 1.1, 0.7):
        check_clipped([torch.full((n,), value, device="cuda").to(TYPES[types[i % len(types)]])
                       for i, n in enumerate((50000, 16384, 8192, 777))], 0.3, how)
    g = gen(11)
    check_clipped([normal(g, n).to(TYPES[types[i % len(types)]]) for i, n in enumerate((100000, 8193, 7))],
                  0.3, how)


@pytest.mark.parametrize("how", ["in place", "out"])
@pytest.mark.parametrize("types", [("f32",), ("bf16",), ("f32", "bf16")])
@pytest.mark.parametrize("bits", [-20, -50, -57, -60, -66, -70, -90, -100, -120, -126, -140, -149])
def test_clip_to_a_norm_far_below(bits, types, how):
    # factors from 2^-146 down to 2^-275, far beyond what fp32 holds; the results are fp32 numbers
    g = gen(13)
    tensors = [normal(g, n, std=2.0 ** 121).to(TYPES[types[i % len(types)]]) for i, n in enumerate((900, 61))]
    check_clipped(tensors, 2.0 ** bits, how)
    if bits > -149:   # (an fp32 number)
        check_clipped(tensors, 1.5 * 2.0 ** bits, how)


# ------------------------------------------------------------------ activations in f32

# Where the sigmoid is at fp32's lower end.  z exact in few bits, so that any order of the product's
# sums gives it exactly.  The sigmoid errs by 2^-22 (the power of two), 2 EPS (reciprocal, products) and,
# in the tanh form, by 4 EPS of its argument, a product of seven rounded factors; the result is
# rounded once, at the lower end to half of fp32's smallest step.
def sigmoid_argument(z, name):
    if name == "silu":
        return z, torch.ones_like(z)
    c = 2 * (2 / math.pi) ** 0.5
    return c * (z + 0.044715 * z ** 3), c * (1 + 3 * 0.044715 * z ** 2)


def tails(name):
    if name == "silu":
        z = torch.arange(-112, -84, 1 / 8, device="cuda")
    else:
        z = torch.arange(-11, -9, 1 / 128, device="cuda")
    t, slope = sigmoid_argument(z.double(), name)
    p = torch.sigmoid(t)
    rel = 8 * EPS + (4 * EPS * t.abs() if name == "gelu" else 0.0)
    return z, z.double() * p, p + z.double() * p * (1 - p) * slope, rel


@pytest.mark.parametrize("name", ["silu", "gelu"])
@pytest.mark.parametrize("w_kn", [False, True])
@pytest.mark.parametrize("m", [1, 3, 16, 17, 300])
def test_gated_f32_activations_reach_the_smallest_numbers(m, w_kn, name):
    z, want, _, rel = tails(name)
    one, zero = torch.ones_like(z), torch.zeros_like(z)
    ws = [torch.stack(w) if w_kn else torch.stack(w, 1) for w in ((z, zero), (zero, one))]
    h, zg, zu = sg.gated_linear(torch.ones(m, 2, device="cuda"), *[w.t() if w_kn else w for w in ws],
                                activation=name, save_preact=True)
    assert torch.equal(zg, z.expand(m, -1)) and torch.equal(zu, one.expand(m, -1))
    check(h, want.expand(m, -1), (rel * want.abs() + 1.01 * 2.0 ** -150).expand(m, -1), name)


@pytest.mark.parametrize("name", ["silu", "gelu"])
def test_gated_f32_slopes_reach_the_smallest_numbers(name):
    # the biases' gradients of one row are dZ itself, unrounded
    z, value, slope, rel = tails(name)
    one, k = torch.ones(1, z.numel(), device="cuda"), torch.zeros(z.numel(), 1, device="cuda")
    got = sg.gated_linear_backward(one, torch.zeros(1, 1, device="cuda"), k, k, z[None], one, activation=name,
                                   need_dx=False, need_dw=False)
    check(got[3], slope, (rel + 8 * EPS) * slope.abs() + 1.01 * 2.0 ** -150, name)
    check(got[4], value, rel * value.abs() + 1.01 * 2.0 ** -150, name)


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("name", ["relu", "gelu", "gelu_erf", "silu"])
def test_gated_gradients_at_an_infinite_gate(name, t):
    # a stored pre-activation may have left its type's range: act and act' are then their limits,
    # as at any z so far down (both 0) or up
    g = gen(17)
    m, n, k = 70, 136, 64
    x, wg, wu, zg, zu, dh = (normal(g, *s, dtype=TYPES[t]) for s in
                             ((m, k), (n, k), (n, k), (m, n), (m, n), (m, n)))
    grads = lambda: sg.gated_linear_backward(dh, x, wg, wu, zg, zu, activation=name)  # noqa: E731
    zg[5, 7] = zg[69, 135] = -60000.0
    want = grads()
    zg[5, 7] = zg[69, 135] = float("-inf")
    got = grads()
    assert all(torch.isfinite(v).all() and torch.equal(v, w) for v, w in zip(got, want))
    zg[5, 7] = float("inf")   # dZu is infinite there, dZg as for any large z
    zg[69, 135] = -60000.0
    dx, dwg, dwu, dbg, dbu = grads()
    zg[5, 7] = 60000.0
    want = grads()
    assert torch.equal(dwg, want[1]) and torch.equal(dbg, want[3])
    keep = torch.arange(n, device="cuda") != 7
    assert torch.equal(dwu[keep], want[2][keep]) and torch.equal(dbu[keep], want[4][keep])
    assert torch.isinf(dbu[7]) and not torch.isfinite(dx[5]).any()
