"""Products on decoded weights against 64-bit evaluations of their formulas.

Bounds.  eps(t) = finfo(t).eps.  Rounding a result to type t costs at most
eps(t) / 2 of it, or half the smallest subnormal.  A 32-bit sum of n products,
in any order and with additions that may be truncated instead of rounded
(2^-23 each), is within (n + 8) 2^-23 of S, the sum of the products'
magnitudes.  The activations (ex2, rcp and a fitted tail in fp32) are within 2^-19 of
their value plus 2^-19 of their argument's share; their slopes are at most
1.13 in size and change by at most 1.2 per unit of the argument.
"""
import ctypes
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

ACTS = ["silu", "gelu", "gelu_tanh", "relu"]
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
U = 2.0 ** -23


@pytest.fixture(scope="module")
def tcq():
    assert torch.cuda.is_available(), "GPU test"
    from trellis_coded_weight_bitshift_b200.build import build
    build()
    import trellis_coded_weight_bitshift_b200 as t
    return t


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, device="cuda", generator=g)


def _act_id(tcq, act):
    return {"silu": tcq.ACT_SILU, "gelu": tcq.ACT_GELU, "gelu_tanh": tcq.ACT_GELU_TANH, "relu": tcq.ACT_RELU}[act]


def _gate(v, act):
    """The activation in 64 bits, by torch's functions (differentiable)."""
    f = torch.nn.functional
    return {"silu": f.silu, "gelu": f.gelu, "gelu_tanh": lambda t: f.gelu(t, approximate="tanh"),
            "relu": f.relu}[act](v)


def _slope(v, act):
    v = v.detach().clone().requires_grad_()
    return torch.autograd.grad(_gate(v, act).sum(), v)[0]


def _half_step(y, dtype):
    fi = torch.finfo(dtype)
    return y.abs() * (fi.eps / 2) + fi.smallest_normal * fi.eps / 2


def _within(got, want, bound):
    # a value past the type's largest (plus half its step) rounds to infinity: in fp16 that is 65520
    assert got.shape == want.shape
    got, fi = got.double(), torch.finfo(got.dtype)
    edge = fi.max * (1 + fi.eps / 4)
    inf = torch.isinf(got)
    assert not bool(torch.isnan(got).any())
    assert bool((got[inf].sign() == want[inf].sign()).all()) and bool((want.abs() + bound >= edge)[inf].all())
    off = torch.where(inf, 0.0, (got - want).abs() / (bound + 1e-300))
    assert float(off.max()) <= 1.0, (float(off.max()), int(off.argmax()))


# ------------------------------------------------------------ quantisation

def _quantize_ref(x):
    amax = x.double().abs().amax(dim=1)
    scale = (amax / 127).float()
    by = torch.where(scale > 0, scale, torch.ones_like(scale)).double()[:, None]
    return torch.round(x.double() / by).to(torch.int8), scale


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 2), (5, 31), (4, 32), (7, 255), (2, 256), (9, 1000), (3, 1024),
                                       (2, 1032), (5, 2047), (3, 4096), (2, 8191), (300, 8192), (2, 8200),
                                       (1, 20000), (2, 33333),
                                       (7, 2049), (5, 8185), (9, 4101), (40, 8190), (3, 2056), (2, 8193)])
def test_quantize_equals_the_definition(tcq, dtype, rows, cols):
    x = (_randn(_gen(rows * 7 + cols), rows, cols) * 3).to(dtype)
    q, s = tcq.quantize_int8(x)
    rq, rs = _quantize_ref(x)
    assert torch.equal(s, rs) and torch.equal(q, rq)
    assert int(q.abs().max()) == 127


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
def test_quantize_ties_go_to_even(tcq, dtype):
    # a row whose largest value is 127 has scale 1: halves are exact ties
    half = torch.arange(-126.5, 127, 1.0, device="cuda")
    for unit in (1.0, 2.0 ** -6, 2.0 ** 7):
        x = (torch.cat([torch.tensor([127.0], device="cuda"), half]) * unit).to(dtype)[None]
        q, s = tcq.quantize_int8(x)
        rq, rs = _quantize_ref(x)
        assert float(s) == unit and torch.equal(q, rq) and torch.equal(s, rs)
        if dtype == F32:
            assert bool((q[0, 1:].int() % 2 == 0).all())


def test_quantize_values_next_to_a_border(tcq):
    # the neighbours of every border between two integers, for many scales
    g = _gen(3)
    amax = (torch.rand(64, device="cuda", generator=g) + 0.5) * torch.exp2(
        torch.randint(-100, 100, (64,), device="cuda", generator=g).float())
    scale = (amax.double() / 127).float()
    border = (torch.arange(-127, 127, device="cuda").double() + 0.5)[None] * scale.double()[:, None]
    mid = border.float()
    x = torch.cat([amax[:, None], mid, torch.nextafter(mid, mid * 2), torch.nextafter(mid, mid * 0)], 1)
    q, s = tcq.quantize_int8(x.contiguous())
    rq, rs = _quantize_ref(x)
    assert torch.equal(s, rs) and torch.equal(q, rq)


def test_quantize_special_rows(tcq):
    tiny = torch.finfo(F32).tiny
    x = torch.zeros(9, 40, device="cuda")
    x[1, 3] = 2.0 ** -149                        # its scale rounds to zero
    x[2, :] = torch.linspace(-1, 1, 40) * 200 * 2.0 ** -149
    x[3, :] = torch.linspace(-1, 1, 40) * tiny * 5
    x[4, 5] = float("inf")
    x[5, 6] = float("nan")
    x[6, :] = torch.linspace(-1, 1, 40) * 3.4e38
    x[7, 0] = -1.0
    x[8, 1], x[8, 2] = float("-inf"), float("nan")
    q, s = tcq.quantize_int8(x)
    for r in (4, 5, 8):
        assert bool(torch.isnan(s[r])) and not bool(q[r].any())
    keep = [0, 1, 2, 3, 6, 7]
    rq, rs = _quantize_ref(x[keep])
    assert torch.equal(q[keep], rq) and torch.equal(s[keep], rs)
    assert int(q[7, 0]) == -127 and float(s[0]) == 0.0


@pytest.mark.parametrize("cols", [40, 2047, 2048, 2500, 5001, 8191, 9001])
def test_quantize_special_rows_of_every_length(tcq, cols):
    # the first and last places of rows that start anywhere; a row's neighbours do not reach it
    x = _randn(_gen(cols), 9, cols)
    x[1, 0], x[2, cols - 1], x[3, cols // 2] = float("inf"), float("nan"), float("-inf")
    x[4] *= 2.0 ** -130
    x[5] = 0
    x[6, 0], x[7, cols - 1] = 900.0, -900.0
    q, s = tcq.quantize_int8(x)
    assert bool(torch.isnan(s[1:4]).all()) and not bool(q[1:4].any())
    keep = [0, 4, 5, 6, 7, 8]
    rq, rs = _quantize_ref(x[keep])
    assert torch.equal(q[keep], rq) and torch.equal(s[keep], rs)
    assert int(q[6, 0]) == 127 and int(q[7, cols - 1]) == -127


# ------------------------------------------------------------ int8 decode

@pytest.mark.parametrize("L", [8, 12, 16])
@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("n,T", [(3, 256), (5, 16), (1, 240), (7, 37), (2, 1), (300, 255), (9, 32)])
def test_decode_int8_sequences(tcq, L, layout, n, T):
    if layout == 0 and (2 * T % 32 or 2 * T < L):
        pytest.skip("no tail-biting stream of this length")
    W = tcq.stream_words(L, T, layout)
    bits = torch.randint(-2 ** 31, 2 ** 31, (n, W), device="cuda", generator=_gen(T + L)).to(torch.int32).view(
        torch.uint32)
    got = tcq.decode_int8(bits, L, T, layout)
    # tcq.decode is pinned bit for bit to the oracle: its fp16 code times 147.8 is the numerator to within 0.25
    k = torch.round(tcq.decode(bits, L, T, layout).double() * 147.8)
    assert torch.equal(got, torch.round(k / 4).to(torch.int8))


@pytest.mark.parametrize("L", [8, 12, 16])
@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("rows,cols", [(16, 16), (48, 32), (16, 2064), (1040, 16), (256, 512)])
def test_decode_int8_tiles(tcq, L, layout, rows, cols):
    n = rows * cols // 256
    W = tcq.stream_words(L, 256, layout)
    bits = torch.randint(-2 ** 31, 2 ** 31, (n, W), device="cuda", generator=_gen(rows + L)).to(torch.int32).view(
        torch.uint32)
    out = torch.full((rows, cols), 77, dtype=torch.int8, device="cuda")
    got = tcq.decode_int8(bits, L, 256, layout, tcq.OUT_TILE16, rows, cols, out=out)
    assert got is out
    k = torch.round(tcq.decode(bits, L, 256, layout, tcq.OUT_TILE16, rows, cols).double() * 147.8)
    assert torch.equal(got, torch.round(k / 4).to(torch.int8))


def test_decode_int8_refuses_shapes_that_are_not_the_tiles(tcq):
    bits = torch.zeros(4, 16, dtype=torch.int32, device="cuda").view(torch.uint32)
    for rows, cols, error in ((32, 48, tcq.TcqError), (30, 32, tcq.TcqError), (0, 0, tcq.TcqError),
                              (-32, -32, ValueError)):
        with pytest.raises(error):
            tcq.decode_int8(bits, 16, 256, tcq.TAILBITING, tcq.OUT_TILE16, rows, cols)


# ------------------------------------------------------------ int8 product

SIZES = [(1, 1, 1), (1, 8, 16), (1, 256, 4096), (2, 17, 16), (3, 100, 33), (15, 129, 128), (16, 128, 256),
         (17, 127, 1000), (33, 64, 1024), (48, 520, 48), (64, 300, 2048), (65, 257, 160), (100, 1000, 127),
         (127, 128, 64), (128, 256, 128), (129, 256, 144), (200, 96, 8192), (255, 513, 96), (256, 1024, 1024),
         (257, 240, 31), (300, 511, 272), (777, 1041, 640), (129, 250, 8192), (300, 96, 5000), (1000, 2100, 1500),
         (1, 20000, 65)]


def _int8(g, *shape):
    return torch.randint(-127, 128, shape, device="cuda", generator=g).to(torch.int8)


def _pos(g, n):
    return torch.exp(_randn(g, n))


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("dtype,bias", [(F16, True), (BF16, False), (F32, True)])
def test_int8_matmul(tcq, M, N, K, dtype, bias):
    g = _gen(M + 3 * N + 7 * K)
    a, w, sa, sw = _int8(g, M, K), _int8(g, N, K), _pos(g, M) * 1e-3, _pos(g, N) * 1e-2
    b = _randn(g, N) if bias else None
    got = tcq.int8_matmul(a, sa, w, sw, bias=b, out_dtype=dtype)
    p = (a.double() @ w.double().t()) * sa.double()[:, None] * sw.double()
    y = p if b is None else p + b.double()
    # the sum, two products (and the bias): three or four roundings of fp32, one of the output
    _within(got, y, p.abs() * 3.01 * 2.0 ** -24 + y.abs() * 2.0 ** -24 + _half_step(y, dtype) * 1.01)
    assert got.dtype == dtype


def test_int8_matmul_largest_sums(tcq):
    # every value at its largest, n_in at its limit: the sums come within 2^-17 of 2^31
    K = 131071
    a = torch.full((3, K), -128, dtype=torch.int8, device="cuda")
    w = torch.full((5, K), -128, dtype=torch.int8, device="cuda")
    a[1] = 127
    got = tcq.int8_matmul(a, torch.ones(3, device="cuda"), w, torch.ones(5, device="cuda"), out_dtype=F32)
    want = (a.double() @ w.double().t()).float()
    assert torch.equal(got, want)


def test_int8_matmul_scales_of_any_size(tcq):
    # a NaN scale (a row that held one) stays in its row, a zero scale gives zeros
    g = _gen(5)
    a, w, sa, sw = _int8(g, 20, 64), _int8(g, 40, 64), _pos(g, 20), _pos(g, 40)
    sa[3], sa[4], sw[7] = float("nan"), 0.0, float("inf")
    got = tcq.int8_matmul(a, sa, w, sw, out_dtype=F32)
    assert bool(torch.isnan(got[3]).all()) and not bool(got[4, :7].any())
    rest = [i for i in range(20) if i not in (3, 4)]
    cols = [j for j in range(40) if j != 7]
    want = tcq.int8_matmul(a[rest].contiguous(), sa[rest].contiguous(), w[cols].contiguous(), sw[cols].contiguous(),
                           out_dtype=F32)
    assert torch.equal(got[rest][:, cols], want)


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("act,dtype", [("silu", F16), ("gelu", BF16), ("gelu_tanh", F32), ("relu", F16)])
def test_int8_gated_ffn(tcq, M, N, K, act, dtype):
    g = _gen(M + 5 * N + 11 * K)
    a, wg, wu = _int8(g, M, K), _int8(g, N, K), _int8(g, N, K)
    sa, sg, su = _pos(g, M) / 73, _pos(g, N) / (73 * math.sqrt(K)), _pos(g, N) / (73 * math.sqrt(K))
    got = tcq.int8_gated_ffn(a, sa, wg, sg, wu, su, act=_act_id(tcq, act), out_dtype=dtype)
    gate = (a.double() @ wg.double().t()) * sa.double()[:, None] * sg.double()
    up = (a.double() @ wu.double().t()) * sa.double()[:, None] * su.double()
    val = _gate(gate, act)
    y = val * up
    # gate and up carry three roundings each; the activation 2^-19 of its value and of its argument's share
    dv = 1.13 * gate.abs() * 3.01 * 2.0 ** -24 + 2.0 ** -19 * (val.abs() + gate.abs() * (val - gate).abs().clamp(max=1) * 2.0 ** -4)
    _within(got, y, dv * up.abs() * 1.01 + val.abs() * up.abs() * 4.01 * 2.0 ** -24 + _half_step(y, dtype) * 1.01)


# ------------------------------------------------------------ gated block

# after these: one token, a very long and a very wide matrix; few tiles and a long sum (split over
# clusters) of the block, of grad_x and of the weights' gradients; half tiles in the last round
FFN_SIZES = SIZES + [(1, 1000, 2048), (5, 8192, 64), (512, 384, 520), (3, 20, 100000), (70, 260, 4100),
                     (140, 4100, 264), (129, 8200, 40), (5000, 200, 136), (700, 2500, 130), (2, 30000, 24),
                     (70000, 9, 24), (40000, 130, 7)]


def _ffn_inputs(seed, M, N, K, dtype):
    g = _gen(seed)
    return (_randn(g, M, K).to(dtype), (_randn(g, N, K) / math.sqrt(K)).to(dtype),
            (_randn(g, N, K) / math.sqrt(K)).to(dtype), (_randn(g, M, N) * 0.25).to(dtype))


def _forward_ref(x, wg, wu, act):
    """Projections, output, and the bounds of all three before the output's rounding."""
    K = x.shape[1]
    x, wg, wu = x.double(), wg.double(), wu.double()
    gate, up = x @ wg.t(), x @ wu.t()
    dg, du = ((K + 8) * U * (x.abs() @ w.abs().t()) for w in (wg, wu))
    val = _gate(gate, act)
    dv = 1.13 * dg + 2.0 ** -19 * (val.abs() + gate.abs() * 2.0 ** -4)
    return gate, up, val * up, dg, du, dv * (up.abs() + du) + val.abs() * du + (val * up).abs() * 2.0 ** -22


@pytest.mark.parametrize("M,N,K", FFN_SIZES)
@pytest.mark.parametrize("act,dtype", [("silu", F16), ("gelu", BF16), ("gelu_tanh", F16), ("relu", BF16)])
def test_gated_ffn_forward(tcq, M, N, K, act, dtype):
    x, wg, wu, _ = _ffn_inputs(M + 3 * N + 5 * K, M, N, K, dtype)
    h = tcq.gated_ffn(x, wg, wu, act=_act_id(tcq, act))
    h2, gate, up = tcq.gated_ffn(x, wg, wu, act=_act_id(tcq, act), save=True)
    rg, ru, rh, dg, du, dh = _forward_ref(x, wg, wu, act)
    _within(h, rh, dh * 1.01 + _half_step(rh, dtype) * 1.01)
    _within(h2, rh, dh * 1.01 + _half_step(rh, dtype) * 1.01)
    _within(gate, rg, dg)
    _within(up, ru, du)
    assert gate.dtype == F32 and h.dtype == dtype


def _backward_ref(x, wg, wu, gate, up, grad, act, dtype):
    """Gradients in 64 bits from the given projections, and their bounds: dg and
    du are formed in fp32 and rounded to 16 bits, the sums are fp32."""
    M, K = x.shape
    N = wg.shape[0]
    x, wg, wu, gate, up, grad = (t.double() for t in (x, wg, wu, gate, up, grad))
    val, slope = _gate(gate, act), _slope(gate, act)
    dg, du = grad * up * slope, grad * val
    f = 2.0 ** -19
    eg = (_half_step(dg, dtype) + f * (grad * up).abs() * (slope.abs() + gate.abs() * 2.0 ** -3 + 2.0 ** -3)) * 1.01
    eu = (_half_step(du, dtype) + f * grad.abs() * (val.abs() + gate.abs() * 2.0 ** -4)) * 1.01
    ag, au = dg.abs() + eg, du.abs() + eu
    out = []
    for want, slack, mass, n in (
            (dg @ wg + du @ wu, eg @ wg.abs() + eu @ wu.abs(), ag @ wg.abs() + au @ wu.abs(), 2 * N),
            (dg.t() @ x, eg.t() @ x.abs(), ag.t() @ x.abs(), M),
            (du.t() @ x, eu.t() @ x.abs(), au.t() @ x.abs(), M)):
        out.append((want, slack + (n + 8) * U * mass + _half_step(want, dtype) * 1.01))
    return out


@pytest.mark.parametrize("M,N,K", FFN_SIZES)
@pytest.mark.parametrize("act,dtype", [("silu", BF16), ("gelu", F16), ("gelu_tanh", BF16), ("relu", F16)])
def test_gated_ffn_backward(tcq, M, N, K, act, dtype):
    x, wg, wu, grad = _ffn_inputs(M + 7 * N + 9 * K, M, N, K, dtype)
    gate, up = (x.double() @ wg.double().t()).float(), (x.double() @ wu.double().t()).float()
    got = tcq.gated_ffn_backward(x, wg, wu, gate, up, grad, act=_act_id(tcq, act))
    for g, (want, bound) in zip(got, _backward_ref(x, wg, wu, gate, up, grad, act, dtype)):
        _within(g, want, bound)
        assert g.dtype == dtype


@pytest.mark.parametrize("need", [(True, False, False), (False, True, False), (False, False, True),
                                  (True, True, False), (False, True, True), (False, False, False)])
def test_gated_ffn_backward_of_some_inputs(tcq, need):
    x, wg, wu, grad = _ffn_inputs(1, 70, 136, 200, BF16)
    _, gate, up = tcq.gated_ffn(x, wg, wu, save=True)
    every = tcq.gated_ffn_backward(x, wg, wu, gate, up, grad)
    some = tcq.gated_ffn_backward(x, wg, wu, gate, up, grad, need=need)
    for a, b, n in zip(every, some, need):
        assert (b is None) if not n else torch.equal(a, b)


@pytest.mark.parametrize("act", ACTS)
def test_autograd_against_differences(tcq, act):
    # central differences of the 64-bit block along random directions; a bf16
    # gradient's inner product with a direction is off by at most the bounds' sum
    M, N, K, dtype = 40, 72, 48, BF16
    x, wg, wu, grad = _ffn_inputs(5, M, N, K, dtype)
    leaves = [t.clone().requires_grad_() for t in (x, wg, wu)]
    h = tcq.GatedFfn.apply(*leaves, _act_id(tcq, act))
    grads = torch.autograd.grad(h, leaves, grad)
    rg, ru, _, dg, du, _ = _forward_ref(x, wg, wu, act)
    ref = _backward_ref(x, wg, wu, rg, ru, grad, act, dtype)
    # the projections are off by dg and du when the gradients are formed
    eg = (grad.double().abs() * (1.13 * du + ru.abs() * 1.2 * dg)) * 1.01
    eu = grad.double().abs() * 1.13 * dg * 1.01
    more = [eg @ wg.double().abs() + eu @ wu.double().abs(), eg.t() @ x.double().abs(), eu.t() @ x.double().abs()]
    base = [t.double() for t in (x, wg, wu)]

    def loss(p):
        return float(((_gate(p[0] @ p[1].t(), act) * (p[0] @ p[2].t())) * grad.double()).sum())

    for i in range(3):
        d = _randn(_gen(60 + i), *base[i].shape).double()
        if act == "relu":
            continue                              # kinks between the two points would count; the formula test stands
        step = 1e-5
        plus, minus = list(base), list(base)
        plus[i], minus[i] = base[i] + step * d, base[i] - step * d
        diff = (loss(plus) - loss(minus)) / (2 * step)
        assert abs(diff - float((ref[i][0] * d).sum())) <= 1e-5 * float((ref[i][0] * d).abs().sum())
        assert abs(float((grads[i].double() * d).sum()) - diff) <= float(((ref[i][1] + more[i]) * d.abs()).sum()) + 1e-6
    for g, (want, bound), m in zip(grads, ref, more):
        if act != "relu":                         # a projection within its bound of 0 may take either slope
            _within(g, want, bound + m)


def test_autograd_takes_any_gradient_layout(tcq):
    # a broadcast gradient (of a sum), a slice that starts off a 16-byte boundary, a frozen weight, a shared weight
    x, wg, wu, grad = _ffn_inputs(2, 33, 45, 24, F16)
    xr, wr = x.clone().requires_grad_(), wg.clone().requires_grad_()
    tcq.GatedFfn.apply(xr, wr, wu).sum().backward()
    ones = torch.ones(33, 45, dtype=F16, device="cuda")
    _, gate, up = tcq.gated_ffn(x, wg, wu, save=True)
    want = tcq.gated_ffn_backward(x, wg, wu, gate, up, ones)
    assert torch.equal(xr.grad, want[0]) and torch.equal(wr.grad, want[1])
    a, b = x.clone().requires_grad_(), x.clone().requires_grad_()
    big = torch.cat([tcq.GatedFfn.apply(a, wg, wu), tcq.GatedFfn.apply(b, wg, wu)])
    big.backward(torch.cat([grad, grad]))
    assert torch.equal(a.grad, b.grad)
    shared = wg.clone().requires_grad_()
    tcq.GatedFfn.apply(x, shared, shared).backward(grad)
    _, gate, up = tcq.gated_ffn(x, wg, wg, save=True)
    _, g1, g2 = tcq.gated_ffn_backward(x, wg, wg, gate, up, grad)
    assert torch.equal(shared.grad, g1 + g2)
    assert not tcq.GatedFfn.apply(x, wg, wu).requires_grad
    with torch.no_grad():
        plain = tcq.GatedFfn.apply(xr, wr, wu)
    assert not plain.requires_grad and torch.equal(plain, tcq.gated_ffn(x, wg, wu))
    none = x[:0].clone().requires_grad_()
    wr.grad = None
    tcq.GatedFfn.apply(none, wr, wu).sum().backward()
    assert none.grad.shape == (0, 24) and not bool(wr.grad.any())
    y = tcq.GatedFfn.apply(xr, wg, wu)
    (g,) = torch.autograd.grad(y.sum(), xr, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()


def test_a_long_sum_of_equal_signs(tcq):
    # nothing cancels: an accumulator that lost low bits would show at once
    x = torch.full((4, 60000), 0.5, dtype=F16, device="cuda")
    w = torch.full((24, 60000), 2.0 ** -11, dtype=F16, device="cuda")
    h, gate, up = tcq.gated_ffn(x, w, w, act=tcq.ACT_RELU, save=True)
    want = 60000 * 0.5 * 2.0 ** -11
    assert bool((gate == want).all()) and bool((up == want).all())         # exact in fp32
    assert bool((h.double() - want * want).abs().max() <= want * want * 2.0 ** -11)


@pytest.mark.parametrize("N,K", [(200, 136), (77, 61)])
def test_int8_results_do_not_depend_on_the_batch(tcq, N, K):
    g = _gen(8)
    a, sa, w, sw, b = _int8(g, 400, K), _pos(g, 400), _int8(g, N, K), _pos(g, N), _randn(g, N)
    every = tcq.int8_matmul(a, sa, w, sw, bias=b, out_dtype=F32)
    for lo, hi in ((0, 1), (7, 20), (100, 160), (3, 130), (0, 257)):
        part = tcq.int8_matmul(a[lo:hi].clone(), sa[lo:hi].clone(), w, sw, bias=b, out_dtype=F32)
        assert torch.equal(part, every[lo:hi])


def test_offsets_past_32_bits(tcq):
    # more than 2^31 values in and out; the last rows, and some in between, against the definition
    rows, cols = 262200, 8200
    x = torch.empty(rows, cols, dtype=F16, device="cuda")
    pick = torch.tensor([0, 1, 130000, 261900, rows - 2, rows - 1], device="cuda")
    x[:] = torch.randn(cols, device="cuda", generator=_gen(1)).half()
    x[pick] = _randn(_gen(2), 6, cols).half()
    q, s = tcq.quantize_int8(x)
    rq, rs = _quantize_ref(x[pick])
    assert torch.equal(q[pick], rq) and torch.equal(s[pick], rs)
    del x
    w, sw = _int8(_gen(3), 48, cols), _pos(_gen(4), 48)
    y = tcq.int8_matmul(q, s, w, sw, out_dtype=F32)
    p = (rq.double() @ w.double().t()) * rs.double()[:, None] * sw.double()
    _within(y[pick], p, p.abs() * 4.01 * 2.0 ** -24)
    del q, y
    # results past 2^31: 65,700 tokens by 32,800 channels
    M, N, K = 65700, 32800, 64
    a, sa, w, sw = _int8(_gen(5), M, K), _pos(_gen(6), M), _int8(_gen(7), N, K), _pos(_gen(8), N)
    y = tcq.int8_matmul(a, sa, w, sw, out_dtype=BF16)
    r = torch.tensor([0, 255, 40000, M - 1], device="cuda")
    p = (a[r].double() @ w.double().t()) * sa[r].double()[:, None] * sw.double()
    _within(y[r], p, p.abs() * 4.01 * 2.0 ** -24 + _half_step(p, BF16) * 1.01)
    del y
    n = (1 << 23) + 40                               # streams of 256 weights
    bits = torch.randint(0, 2 ** 31, (n, 16), device="cuda", generator=_gen(9), dtype=torch.int32).view(torch.uint32)
    out = tcq.decode_int8(bits, 16)
    assert out.numel() > 2 ** 31
    assert torch.equal(out[-300:], tcq.decode_int8(bits[-300:].clone(), 16))
    assert torch.equal(out[:300], tcq.decode_int8(bits[:300].clone(), 16))


def test_training_step_captured_into_a_graph(tcq):
    x, wg, wu, grad = _ffn_inputs(4, 140, 264, 96, BF16)
    leaves = [t.clone().requires_grad_() for t in (x, wg, wu)]

    def step():
        h = tcq.GatedFfn.apply(*leaves, tcq.ACT_GELU)
        return (h.detach(), *torch.autograd.grad(h, leaves, grad))
    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got = step()
    torch.cuda.current_stream().wait_stream(side)
    for _ in range(2):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_empty_batches(tcq):
    x, w = torch.zeros(0, 32, dtype=F16, device="cuda"), torch.ones(24, 32, dtype=F16, device="cuda")
    assert tcq.gated_ffn(x, w, w).shape == (0, 24)
    gate = torch.zeros(0, 24, device="cuda")
    gx, g1, g2 = tcq.gated_ffn_backward(x, w, w, gate, gate, gate.half())
    assert gx.shape == (0, 32) and not bool(g1.any()) and not bool(g2.any()) and g1.shape == w.shape
    q, s = tcq.quantize_int8(x)
    assert q.shape == (0, 32) and s.shape == (0,)
    wq, ws = tcq.quantize_int8(w)
    assert tcq.int8_matmul(q, s, wq, ws).shape == (0, 24)
    assert tcq.int8_gated_ffn(q, s, wq, ws, wq, ws).shape == (0, 24)


@pytest.mark.parametrize("M", [1, 20, 300])
def test_values_that_are_not_finite_stay_in_their_row_or_channel(tcq, M):
    x, wg, wu, _ = _ffn_inputs(9, M, 200, 136, F16)
    clean = tcq.gated_ffn(x, wg, wu)
    r, c = M // 2, 77
    bad = x.clone()
    bad[r, 5] = float("nan")
    h = tcq.gated_ffn(bad, wg, wu)
    keep = torch.arange(M, device="cuda") != r
    assert bool(torch.isnan(h[r]).all()) and torch.equal(h[keep], clean[keep])
    bw = wu.clone()
    bw[c, 100] = float("inf")
    h = tcq.gated_ffn(x, wg, bw)
    ch = torch.arange(200, device="cuda") != c
    assert not bool(torch.isfinite(h[:, c]).any()) and torch.equal(h[:, ch], clean[:, ch])


# ------------------------------------------------------------ use

GUARD, FILL = 4096, 0xA5


class Guarded:
    def __init__(self, nbytes):
        self.n = int(nbytes)
        self.buf = torch.full((2 * GUARD + (self.n + 255) // 256 * 256,), FILL, dtype=torch.uint8, device="cuda")
        self.ptr = ctypes.c_void_p(self.buf.data_ptr() + GUARD)

    def intact(self):
        torch.cuda.synchronize()
        return bool((self.buf[:GUARD] == FILL).all()) and bool((self.buf[GUARD + self.n:] == FILL).all())


def _p(t):
    return ctypes.c_void_p(t.data_ptr())


@pytest.mark.parametrize("M,N,K", [(1, 3, 5), (1, 136, 64), (17, 129, 33), (40, 77, 80), (70, 300, 128),
                                   (257, 130, 45), (300, 264, 192), (5, 20, 3001), (3, 33, 8191)])
def test_writes_stay_inside(tcq, M, N, K):
    lib, st = tcq.lib(), ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    x, wg, wu, grad = _ffn_inputs(1, M, N, K, F16)
    h, gate, up = Guarded(M * N * 2), Guarded(M * N * 4), Guarded(M * N * 4)
    need = lib.tcq_gated_ffn_workspace_size(M, N, K)
    ws = Guarded(need)
    assert lib.tcq_gated_ffn(_p(x), _p(wg), _p(wu), 0, M, N, K, 0, h.ptr, gate.ptr, up.ptr, ws.ptr, need, st) == 0
    assert all(t.intact() for t in (h, gate, up, ws))
    need = lib.tcq_gated_ffn_backward_workspace_size(M, N, K)
    ws, gx, g1, g2 = Guarded(need), Guarded(M * K * 2), Guarded(N * K * 2), Guarded(N * K * 2)
    assert lib.tcq_gated_ffn_backward(_p(x), _p(wg), _p(wu), gate.ptr, up.ptr, _p(grad), 0, M, N, K, 0, gx.ptr,
                                      g1.ptr, g2.ptr, ws.ptr, need, st) == 0
    assert all(t.intact() for t in (ws, gx, g1, g2, gate, up))
    g = _gen(2)
    q, s = Guarded(M * K), Guarded(M * 4)
    assert lib.tcq_quantize_int8(_p(x), 0, M, K, q.ptr, s.ptr, st) == 0
    assert q.intact() and s.intact()
    w, sw, b = _int8(g, N, K), _pos(g, N), _randn(g, N)
    for dt, size in ((0, 2), (2, 4)):
        y = Guarded(M * N * size)
        need = lib.tcq_int8_matmul_workspace_size(M, N, K)
        ws = Guarded(need)
        assert lib.tcq_int8_matmul(q.ptr, s.ptr, _p(w), _p(sw), _p(b), M, N, K, y.ptr, dt, ws.ptr, need, st) == 0
        assert y.intact() and ws.intact()
        need = lib.tcq_int8_gated_ffn_workspace_size(M, N, K)
        ws = Guarded(need)
        assert lib.tcq_int8_gated_ffn(q.ptr, s.ptr, _p(w), _p(sw), _p(w), _p(sw), M, N, K, 0, y.ptr, dt, ws.ptr,
                                      need, st) == 0
        assert y.intact() and ws.intact()
    for L, T, lay in ((8, 37, 1), (16, 256, 0), (12, 48, 0)):
        n = 5
        bits = torch.randint(0, 2 ** 31, (n, tcq.stream_words(L, T, lay)), device="cuda", generator=g).to(torch.int32)
        o = Guarded(n * T)
        assert lib.tcq_decode_int8(ctypes.byref(tcq.trellis(L, T)), _p(bits), n, lay, 0, 0, 0, o.ptr, st) == 0
        assert o.intact()


def _block(tcq, x, bits, M):
    """A quantised feed-forward block as it is served: 2-bit streams -> int8 weights; tokens -> int8."""
    K, F = 256, 512
    ws = torch.full((F,), tcq.DECODE_INT8_SCALE / 16, device="cuda")
    wd = torch.full((K,), tcq.DECODE_INT8_SCALE / 22, device="cuda")
    wg, wu = (tcq.decode_int8(b, 16, 256, tcq.TAILBITING, tcq.OUT_TILE16, F, K) for b in bits[:2])
    dn = tcq.decode_int8(bits[2], 16, 256, tcq.TAILBITING, tcq.OUT_TILE16, K, F)
    q, s = tcq.quantize_int8(x)
    h = tcq.int8_gated_ffn(q, s, wg, ws, wu, ws, out_dtype=F16)
    q2, s2 = tcq.quantize_int8(h)
    return (q, s, wg, wu, ws, h, q2, s2, dn, wd), tcq.int8_matmul(q2, s2, dn, wd, out_dtype=F16)


def _streams(seed):
    g = _gen(seed)
    return [torch.randint(-2 ** 31, 2 ** 31, (512, 16), device="cuda", generator=g).to(torch.int32).view(torch.uint32)
            for _ in range(3)]


@pytest.mark.parametrize("M", [1, 24, 150])
def test_a_served_block_of_streams(tcq, M):
    x = _randn(_gen(M), M, 256).half()
    bits = _streams(3)
    (q, s, wg, wu, ws, h, q2, s2, dn, wd), y = _block(tcq, x, bits, M)
    # every step against its definition on the operands it was given, then the whole against fp16 weights
    a = q.double() * s.double()[:, None]
    gate, up = (a @ (w.double() * ws.double()[:, None]).t() for w in (wg, wu))
    rh = _gate(gate, "silu") * up
    _within(h, rh, rh.abs() * 2.0 ** -17 + up.abs() * gate.abs() * 2.0 ** -21 + _half_step(rh, F16) * 1.01)
    rq, rs = _quantize_ref(h)
    assert torch.equal(q2, rq) and torch.equal(s2, rs)
    ry = (q2.double() * s2.double()[:, None]) @ (dn.double() * wd.double()[:, None]).t()
    _within(y, ry, ry.abs() * 2.0 ** -21 + _half_step(ry, F16) * 1.01)
    wf = [tcq.decode(b, 16, 256, tcq.TAILBITING, tcq.OUT_TILE16, *sh).double()
          for b, sh in zip(bits, ((512, 256), (512, 256), (256, 512)))]
    full = (_gate(x.double() @ wf[0].t() / 16, "silu") * (x.double() @ wf[1].t() / 16)) @ wf[2].t() / 22
    assert float((y.double() - full).norm() / full.norm()) < 0.05      # 8-bit tokens and weights: about 1% a product


def test_captured_and_replayed_on_a_side_stream(tcq):
    x1, x2 = (_randn(_gen(i), 24, 256).half() for i in (1, 2))
    bits = _streams(4)
    want = [_block(tcq, x, bits, 24)[1] for x in (x1, x2)]
    gx, gwg, gwu, grad = _ffn_inputs(3, 50, 90, 61, BF16)
    ref = tcq.gated_ffn(gx, gwg, gwu, save=True)
    ref_g = tcq.gated_ffn_backward(gx, gwg, gwu, ref[1], ref[2], grad)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):                    # eager on another stream, then captured there
        assert torch.equal(_block(tcq, x1, bits, 24)[1], want[0])
        inp = x1.clone()
        graphs = []
        for _ in range(2):                           # two graphs of the same calls
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                y = _block(tcq, inp, bits, 24)[1]
                h, gate, up = tcq.gated_ffn(gx, gwg, gwu, save=True)
                grads = tcq.gated_ffn_backward(gx, gwg, gwu, gate, up, grad)
            graphs.append((graph, y, h, grads))
    torch.cuda.current_stream().wait_stream(side)
    for x, w in ((x2, want[1]), (x1, want[0]), (x2, want[1])):
        inp.copy_(x)
        for graph, _, _, _ in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for _, y, h, grads in graphs:
            assert torch.equal(y, w) and torch.equal(h, ref[0])
            assert all(torch.equal(a, b) for a, b in zip(grads, ref_g))


def test_calls_on_two_streams_at_once(tcq):
    data = [_ffn_inputs(20 + i, 300 - 100 * i, 520, 136 + i, BF16) for i in range(2)]
    want = [tcq.gated_ffn(d[0], d[1], d[2]) for d in data]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(tcq.gated_ffn(data[i][0], data[i][1], data[i][2]))
    torch.cuda.synchronize()
    assert all(torch.equal(g, want[i]) for i in range(2) for g in got[i])


def test_results_repeat_bit_for_bit(tcq):
    x, wg, wu, grad = _ffn_inputs(8, 333, 777, 1000, BF16)
    h, gate, up = tcq.gated_ffn(x, wg, wu, save=True)
    first = tcq.gated_ffn_backward(x, wg, wu, gate, up, grad)
    for _ in range(3):
        again = tcq.gated_ffn(x, wg, wu, save=True)
        assert torch.equal(again[0], h) and torch.equal(again[1], gate) and torch.equal(again[2], up)
        for a, b in zip(first, tcq.gated_ffn_backward(x, wg, wu, gate, up, grad)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("M,N,K", [(20, 72, 40), (300, 72, 40), (300, 77, 41), (130, 72, 9000)])
def test_caller_owned_outputs_and_workspaces(tcq, M, N, K):
    x, wg, wu, grad = _ffn_inputs(M, M, N, K, BF16)
    h, gate, up = tcq.gated_ffn(x, wg, wu, save=True)
    grads = tcq.gated_ffn_backward(x, wg, wu, gate, up, grad)
    g = _gen(1)
    a, sa, w, sw = _int8(g, M, K), _pos(g, M), _int8(g, N, K), _pos(g, N)
    y, z = tcq.int8_matmul(a, sa, w, sw), tcq.int8_gated_ffn(a, sa, w, sw, w, sw, out_dtype=F32)
    for extra in (0, 4096, -1):                      # exactly enough, more, too little (then one of its own)
        def ws(need):
            # filled with values that would show if a call relied on what it finds there
            return torch.full((max(need + extra, 0),), 0x7F, dtype=torch.uint8, device="cuda")
        out = torch.full((M, N), 9.0, dtype=BF16, device="cuda")
        assert tcq.gated_ffn(x, wg, wu, out=out, workspace=ws(tcq.gated_ffn_workspace_size(M, N, K))) is out
        assert torch.equal(out, h)
        got = tcq.gated_ffn_backward(x, wg, wu, gate, up, grad,
                                     workspace=ws(tcq.gated_ffn_backward_workspace_size(M, N, K)))
        assert all(torch.equal(p, q) for p, q in zip(got, grads))
        o16, o32 = torch.empty(M, N, dtype=F16, device="cuda"), torch.empty(M, N, device="cuda")
        assert tcq.int8_matmul(a, sa, w, sw, out=o16, workspace=ws(tcq.int8_matmul_workspace_size(M, N, K))) is o16
        assert torch.equal(o16, y)
        tcq.int8_gated_ffn(a, sa, w, sw, w, sw, out_dtype=F32, out=o32,
                           workspace=ws(tcq.int8_gated_ffn_workspace_size(M, N, K)))
        assert torch.equal(o32, z)
    if tcq.gated_ffn_backward_workspace_size(M, N, K):
        odd = torch.empty(tcq.gated_ffn_backward_workspace_size(M, N, K) + 16, dtype=torch.uint8, device="cuda")[16:]
        with pytest.raises(tcq.TcqError):
            tcq.gated_ffn_backward(x, wg, wu, gate, up, grad, workspace=odd)
    flat = torch.zeros(M * max(N, K), dtype=BF16, device="cuda")
    onto = flat[:M * K].view(M, K)
    with pytest.raises(tcq.TcqError):                # an output on top of an operand
        tcq.gated_ffn(onto, wg, wu, out=flat[:M * N].view(M, N))


def test_binding_refuses_misaligned_and_strided_operands(tcq):
    x, wg, wu, _ = _ffn_inputs(1, 8, 16, 32, F16)
    with pytest.raises(ValueError, match="contiguous"):
        tcq.gated_ffn(x.t().contiguous().t(), wg, wu)
    with pytest.raises(ValueError, match="contiguous"):
        tcq.gated_ffn(x[:, :16], wg[:, :16].contiguous(), wu[:, :16].contiguous())
    off = torch.zeros(8 * 32 + 1, dtype=F16, device="cuda")[1:].view(8, 32)
    with pytest.raises(tcq.TcqError):
        tcq.gated_ffn(off, wg, wu)
    with pytest.raises(ValueError):
        tcq.gated_ffn(x, wg.cpu(), wu)


def test_no_wait_ever_ran_out(tcq):
    x, wg, wu, _ = _ffn_inputs(1, 300, 300, 300, F16)
    tcq.gated_ffn(x, wg, wu)
    assert tcq.products_gave_up() == 0
