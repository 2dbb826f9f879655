"""Edges of the products on decoded weights: the smallest rows, the tails of the
activations, early starts, reports of waits that ran out."""
import ctypes
import math

import pytest
import torch

import test_gpu_products as products

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


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


# ------------------------------------------------------------ quantisation

# every way a row is read: by warps and by blocks, in registers or twice, whole units or from anywhere, single values
@pytest.mark.parametrize("cols", [3, 33, 40, 300, 1024, 2048, 2047, 2501, 5001, 5000, 9001])
def test_quantize_rows_of_the_smallest_values(tcq, cols):
    # values are whole numbers of 2^-149, the scale too: max / 127 to the nearest, ties to even; a scale of few
    # units leaves quotients past 127, which are held there
    tops = list(range(63, 202)) + [317, 318, 444, 5524, 5525, 8000, 16129, 16130, 20000, 40000]
    g = torch.Generator().manual_seed(cols)
    n = torch.stack([torch.randint(-t, t + 1, (cols,), generator=g) for t in tops]).double()
    top = torch.tensor(tops).double()
    n[:, 0], n[:, cols - 1] = top, -top
    unit = torch.round(top / 127)
    want = torch.where(unit[:, None] > 0, torch.round(n / unit.clamp(min=1)[:, None]), 0.0).clamp(-127, 127)
    assert float((n.abs() / unit.clamp(min=1)[:, None]).max()) > 189          # the ranges hold what they are for
    q, s = tcq.quantize_int8((n * 2.0 ** -149).float().cuda())
    assert torch.equal(s.cpu().double(), unit * 2.0 ** -149)
    assert torch.equal(q.cpu().double(), want)


# ------------------------------------------------------------ waits that run out

def test_the_count_of_waits_covers_every_stream(tcq):
    # torch's side streams do not block the default one: the count has to wait for them itself
    side = torch.cuda.Stream()
    done = torch.cuda.Event()
    tcq.products_gave_up()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)                   # about 0.1 s
        done.record()
    assert not done.query()
    assert tcq.products_gave_up() == 0
    assert done.query()


def test_a_wait_that_nothing_meets_ends(tcq, tmp_path):
    from native import compiled
    out = torch.zeros(8, dtype=torch.int64, device="cuda")
    lib = compiled("waits", tmp_path)
    assert lib.wait_runs_out(ctypes.c_ulonglong(20_000_000), ctypes.c_void_p(out.data_ptr())) == 0
    met0, t0, met1, t1, met2, t2, stop, _ = out.tolist()
    # the limit ends the first wait (looked at every 32 tries, of a millisecond each at most), its flag the second;
    # one that is met is met
    assert (met0, met1, met2, stop) == (0, 0, 1, 1)
    assert 20e6 <= t0 < 150e6 and t1 < 300e6 and t2 < 5e6
    assert lib.drain_ends(ctypes.c_void_p(out.data_ptr())) == 0
    assert 125e6 <= int(out[0]) < 300e6


def test_a_wait_that_ran_out_is_reported_once(tcq, tmp_path):
    from native import compiled
    lib = compiled("waits", tmp_path)
    count, first, second = ctypes.c_uint(), ctypes.c_int(), ctypes.c_int()
    for i in (1, 2):
        assert lib.report(ctypes.byref(count), ctypes.byref(first), ctypes.byref(second)) == 0
        assert (count.value, first.value, second.value) == (i, 1, 0)


def test_the_first_product_of_a_process_may_be_a_captured_one(tcq):
    # its word of host memory is pinned within the call
    import subprocess
    import sys
    code = """
import torch, trellis_coded_weight_bitshift_b200 as tcq
x, w = (torch.randn(s, 64, device="cuda").half() for s in (5, 40))
out, side, graph = torch.empty(5, 40, device="cuda").half(), torch.cuda.Stream(), torch.cuda.CUDAGraph()
side.wait_stream(torch.cuda.current_stream())
with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
    tcq.gated_ffn(x, w, w, out=out)
graph.replay()
torch.cuda.synchronize()
assert torch.equal(out, tcq.gated_ffn(x, w, w)) and tcq.products_gave_up() == 0
"""
    subprocess.run([sys.executable, "-c", code], check=True, timeout=300)


# ------------------------------------------------------------ pairs of blocks

@pytest.mark.parametrize("M,N,K", [(4096, 8192, 2048), (700, 2500, 264)])
def test_thousands_of_training_steps(tcq, M, N, K):
    # the gradients' pairs of blocks start behind the elementwise kernel, whose blocks delay one of the two: every one
    # of many thousands has to find the other
    import time
    g = _gen(3)
    x, wg, wu = _randn(g, M, K).bfloat16(), _randn(g, N, K).bfloat16() / K ** 0.5, _randn(g, N, K).bfloat16() / K ** 0.5
    grad = _randn(g, M, N).bfloat16()
    leaves = [t.requires_grad_() for t in (x, wg, wu)]

    def step():
        h = tcq.GatedFfn.apply(*leaves, tcq.ACT_GELU)
        return (h.detach(), *torch.autograd.grad(h, leaves, grad))
    want = step()
    side, graph, done = torch.cuda.Stream(), torch.cuda.CUDAGraph(), torch.cuda.Event()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        with torch.cuda.graph(graph, stream=side):
            for _ in range(10):
                got = step()
    torch.cuda.synchronize()
    for _ in range(10):                                  # a minute's worth of patience for each thousand steps
        for _ in range(60):
            graph.replay()
        done.record()
        end = time.monotonic() + 60
        while not done.query():
            assert time.monotonic() < end, "a step does not end"
            time.sleep(0.002)
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and tcq.products_gave_up() == 0


# ------------------------------------------------------------ activations

ACTS = ["silu", "gelu", "gelu_tanh", "relu"]


def _act_id(tcq, act):
    return getattr(tcq, "ACT_" + act.upper())


def _activation(v, act):
    """The activation in 64 bits by functions that keep its tail's digits, and the bound on its fp32 form:
    (8 + e) 2^-23 of the value, e the weight of the roundings of the exponential's argument: one and a constant's
    for silu, two and a constant's for gelu, three and a constant's for the tanh form."""
    z = 2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)
    y, e = {"silu": lambda: (v * torch.sigmoid(v), v.abs()),
            "gelu": lambda: (v * 0.5 * torch.special.erfc(-v / math.sqrt(2)), 0.75 * v * v),
            "gelu_tanh": lambda: (v * torch.sigmoid(z), 2 * z.abs()),
            "relu": lambda: (v.clamp(min=0), torch.zeros_like(v) - 8)}[act]()
    return y, y.abs() * (8 + e) * 2.0 ** -23 + 2.0 ** -110


def _half_step(y, dtype):
    fi = torch.finfo(dtype)
    return y.abs() * (fi.eps / 2) + fi.smallest_normal * fi.eps / 2


def _within(got, want, bound):
    off = (got.double() - want).abs() / bound
    assert float(off.max()) <= 1, (float(off.max()), int(off.argmax()))


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("M,N", [(16001, 3), (16001, 16), (60, 5)])
def test_activations_keep_their_tails_digits(tcq, act, dtype, M, N):
    # gates that are exact (multiples of 2^-9 from -15.6 to 15.6) against an up projection of exactly 1, by both kernels
    n = torch.randint(-8000, 8001, (M,), generator=_gen(M + N), device="cuda") if M < 100 else torch.arange(
        -8000, 8001, device="cuda")
    hi = torch.div(n, 64, rounding_mode="floor")
    a = torch.zeros(M, 16, dtype=torch.int8, device="cuda")
    a[:, 0], a[:, 1], a[:, 2] = hi, n - 64 * hi, 1
    wg, wu = torch.zeros(N, 16, dtype=torch.int8, device="cuda"), torch.zeros(N, 16, dtype=torch.int8, device="cuda")
    wg[:, 0], wg[:, 1], wu[:, 2] = 64, 1, 1
    one = torch.ones(N, device="cuda")
    h = tcq.int8_gated_ffn(a, torch.full((M,), 2.0 ** -9, device="cuda"), wg, one, wu, 512 * one, act=_act_id(tcq, act),
                           out_dtype=dtype)
    y, bound = _activation(n.double() * 2.0 ** -9, act)
    y, bound = y[:, None].expand(M, N), bound[:, None].expand(M, N)
    _within(h, y, bound + y.abs() * 2.0 ** -24 + _half_step(y, dtype) * 1.01)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("M", [4000, 64])
def test_activations_of_16_bit_projections_keep_their_tails_digits(tcq, act, dtype, M):
    v = torch.linspace(-8, 8, M, device="cuda").to(dtype)
    x, one = torch.stack([v, torch.ones_like(v)], 1), torch.tensor([[0, 1]] * 9, dtype=dtype, device="cuda")
    h, gate, up = tcq.gated_ffn(x, one.flip(1).contiguous(), one, act=_act_id(tcq, act), save=True)
    assert torch.equal(gate, v.float()[:, None].expand(M, 9)) and bool((up == 1).all())
    y, bound = _activation(gate.double(), act)
    _within(h, y, bound + y.abs() * 2.0 ** -24 + _half_step(y, dtype) * 1.01)


# ------------------------------------------------------------ errors

def test_a_failed_call_leaves_no_error_behind(tcq):
    # the count waits for the device, which a captured stream refuses; the next call is not to answer for it
    bits = torch.zeros(4, 16, dtype=torch.int32, device="cuda").view(torch.uint32)
    want = tcq.decode(bits, 16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        graph.capture_begin()
        with pytest.raises(tcq.TcqError):
            tcq.products_gave_up()
        with pytest.raises(RuntimeError):
            graph.capture_end()
    torch.cuda.synchronize()
    assert torch.equal(tcq.decode(bits, 16), want)
    assert tcq.products_gave_up() == 0


# ------------------------------------------------------------ what no test held before

def test_relu_gradients_against_the_formula_and_differences(tcq):
    # a projection within its bound of zero may take either slope: the output's gradient is zero there, and where the
    # differences' two points could lie on both sides
    M, N, K, dtype, step = 40, 72, 48, BF16, 1e-5
    x, wg, wu, grad = products._ffn_inputs(5, M, N, K, dtype)
    rg, ru, _, dg, du, _ = products._forward_ref(x, wg, wu, "relu")
    base = [t.double() for t in (x, wg, wu)]
    dirs = [_randn(_gen(60 + i), *t.shape).double() for i, t in enumerate(base)]
    near = dg + 2 * step * (dirs[0].abs() @ base[1].abs().t() + base[0].abs() @ dirs[1].abs().t())
    grad = torch.where(rg.abs() > near, grad, torch.zeros_like(grad))
    assert 0 < int((grad != 0).sum()) and int((grad == 0).sum()) < M * N // 50
    leaves = [t.clone().requires_grad_() for t in (x, wg, wu)]
    grads = torch.autograd.grad(tcq.GatedFfn.apply(*leaves, tcq.ACT_RELU), leaves, grad)
    ref = products._backward_ref(x, wg, wu, rg, ru, grad, "relu", dtype)
    # the projections are off by dg and du when the gradients are formed; relu's slope is 0 or 1, and does not change
    eg, eu = grad.double().abs() * du * 1.01, grad.double().abs() * dg * 1.01
    more = [eg @ base[1].abs() + eu @ base[2].abs(), eg.t() @ base[0].abs(), eu.t() @ base[0].abs()]
    for g, (want, bound), m in zip(grads, ref, more):
        products._within(g, want, bound + m)

    def loss(p):
        return float(((p[0] @ p[1].t()).clamp(min=0) * (p[0] @ p[2].t()) * grad.double()).sum())
    for i in range(3):
        plus, minus = list(base), list(base)
        plus[i], minus[i] = base[i] + step * dirs[i], base[i] - step * dirs[i]
        diff = (loss(plus) - loss(minus)) / (2 * step)
        bound = float(((ref[i][1] + more[i]) * dirs[i].abs()).sum())
        # the loss is at most quadratic in one operand, so the difference is exact but for 64-bit cancellation
        assert abs(float((grads[i].double() * dirs[i]).sum()) - diff) <= bound + 1e-6


@pytest.mark.parametrize("N,K", [(200, 4096), (77, 8191), (520, 8192), (2048, 2048), (1000, 130)])
def test_int8_results_do_not_depend_on_the_batch_or_its_split(tcq, N, K):
    # long sums: split over a cluster, over clusters and joined, or not at all, as the number of tokens decides
    g = _gen(N + K)
    a, w, wu = (products._int8(g, m, K) for m in (600, N, N))
    sa, sw, su, b = (_randn(g, n).exp() * c for n, c in ((600, 1 / 73), (N, 1 / (73 * math.sqrt(K))), (N, 0.01), (N, 1.0)))
    for dtype in (F32, F16):
        whole = tcq.int8_matmul(a, sa, w, sw, bias=b, out_dtype=dtype)
        gated = {act: tcq.int8_gated_ffn(a, sa, w, sw, wu, su, act=_act_id(tcq, act), out_dtype=dtype) for act in ACTS}
        for lo, hi in ((0, 1), (5, 20), (100, 130), (3, 67), (3, 68), (0, 129), (0, 256), (0, 257), (17, 417)):
            part, s = a[lo:hi].clone(), sa[lo:hi].clone()
            assert torch.equal(tcq.int8_matmul(part, s, w, sw, bias=b, out_dtype=dtype), whole[lo:hi]), (lo, hi)
            for act in ACTS:
                h = tcq.int8_gated_ffn(part, s, w, sw, wu, su, act=_act_id(tcq, act), out_dtype=dtype)
                assert torch.equal(h, gated[act][lo:hi]), (lo, hi, act)


@pytest.mark.parametrize("shape", [(1,), (7,), (3, 5), (0, 4), (4, 0), (0, 0), (1, 1), (5, 8192)])
def test_both_ways_to_allocate_give_the_same_tensors(tcq, monkeypatch, shape):
    for dtype in (torch.int8, torch.uint8, F16, BF16, F32):
        quick = tcq._empty(shape, dtype)
        with monkeypatch.context() as m:
            m.setattr(tcq, "_empty_strided", None)
            plain = tcq._empty(shape, dtype)
        for what in ("shape", "dtype", "device", "requires_grad"):
            assert getattr(quick, what) == getattr(plain, what)
        assert quick.stride() == plain.stride() and quick.is_contiguous()
        assert quick.untyped_storage().nbytes() == plain.untyped_storage().nbytes()


def test_calls_without_the_quick_allocation(tcq, monkeypatch):
    x, wg, wu, grad = products._ffn_inputs(3, 20, 72, 41, F16)

    def calls():
        h, gate, up = tcq.gated_ffn(x, wg, wu, save=True)
        q, s = tcq.quantize_int8(x)
        wq, ws = tcq.quantize_int8(wg)
        return [h, gate, up, q, s, *tcq.gated_ffn_backward(x, wg, wu, gate, up, grad), tcq.int8_matmul(q, s, wq, ws),
                tcq.int8_gated_ffn(q, s, wq, ws, wq, ws), tcq.gated_ffn(x[:0], wg, wu)]
    want = calls()
    monkeypatch.setattr(tcq, "_empty_strided", None)
    assert all(torch.equal(a, b) for a, b in zip(calls(), want))


def test_pairs_of_blocks_start_behind_anything(tcq):
    # products of pairs, products of clusters, elementwise kernels and the gradients' chain on four streams at once
    import time
    a = products._ffn_inputs(1, 1500, 2048, 512, BF16)
    b = products._ffn_inputs(2, 40, 2048, 512, F16)
    c = products._ffn_inputs(3, 300, 1000, 130, BF16)
    _, gate, up = tcq.gated_ffn(*c[:3], save=True)
    z = torch.zeros(1 << 22, device="cuda")
    work = [lambda: (tcq.gated_ffn(*a[:3]),), lambda: (tcq.gated_ffn(*b[:3]),), lambda: (z.mul_(1.0),),
            lambda: tcq.gated_ffn_backward(*c[:3], gate, up, c[3])]
    want = [w() for w in work]
    streams, done = [torch.cuda.Stream() for _ in work], [torch.cuda.Event() for _ in work]
    torch.cuda.synchronize()
    got = [None] * len(work)
    for _ in range(2000):
        for i, (stream, call) in enumerate(zip(streams, work)):
            with torch.cuda.stream(stream):
                got[i] = call()
                done[i].record()
    end = time.monotonic() + 60
    while not all(e.query() for e in done):
        assert time.monotonic() < end, "a call does not end"
        time.sleep(0.002)
    assert all(torch.equal(p, q) for g, w in zip(got, want) for p, q in zip(g, w)) and tcq.products_gave_up() == 0


@pytest.mark.parametrize("N", [40, 4096, 4097])
@pytest.mark.parametrize("K", [512, 513, 1536, 1537])
def test_int8_results_on_both_sides_of_the_kernels_borders(tcq, N, K):
    # up to 32 tokens one kernel works, beyond them sums, channels and tokens decide
    g = _gen(N + K)
    a, w, wu = (products._int8(g, m, K) for m in (257, N, N))
    sa, sw, su = (_randn(g, n).exp() * c for n, c in ((257, 1 / 73), (N, 1 / (73 * math.sqrt(K))), (N, 0.01)))

    def both(lo, hi):
        part, s = a[lo:hi].clone(), sa[lo:hi].clone()
        return torch.cat([tcq.int8_matmul(part, s, w, sw, out_dtype=F32),
                          tcq.int8_gated_ffn(part, s, w, sw, wu, su, out_dtype=F32)], 1)
    want = torch.cat([both(i, min(i + 32, 257)) for i in range(0, 257, 32)])
    p = (a.double() @ w.double().t()) * sa.double()[:, None] * sw.double()
    products._within(want[:, :N], p, p.abs() * 4.01 * 2.0 ** -24)
    for M in (33, 64, 65, 128, 129, 256, 257):
        assert torch.equal(both(0, M), want[:M]), M
        assert torch.equal(both(257 - M, 257), want[257 - M:]), M
