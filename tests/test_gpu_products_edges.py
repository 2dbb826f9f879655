"""Edges of the products on decoded weights: the smallest rows, the tails of the
activations, early starts, reports of waits that ran out."""
import ctypes
import math

import pytest
import torch

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
