"""Products on decoded weights: the refusals of the C ABI and of the binding,
and the host-side facts that the kernels rely on (no GPU needed)."""
import ctypes

import numpy as np
import pytest
import torch

import trellis_coded_weight_bitshift_b200 as tcq
from trellis_coded_weight_bitshift_b200 import _abi

P = ctypes.c_void_p(256)                   # never dereferenced: every call below is refused or empty
BIG = 1 << 40
INV, UNS, WSP, OK = _abi.TCQ_ERR_INVALID_ARG, _abi.TCQ_ERR_UNSUPPORTED, _abi.TCQ_ERR_WORKSPACE, _abi.TCQ_OK


@pytest.fixture(scope="module")
def L():
    from trellis_coded_weight_bitshift_b200.build import build
    build()
    return _abi.lib()


def _calls(L):
    """name -> (call(pointers, sizes, **codes), number of pointers that must not be NULL)."""
    return {
        "int8_matmul": (lambda p, m, n, k, dt=0, act=0, ws=P, wb=BIG: L.tcq_int8_matmul(
            p[0], p[1], p[2], p[3], None, m, n, k, p[4], dt, ws, wb, None), 5),
        "int8_gated_ffn": (lambda p, m, n, k, dt=0, act=0, ws=P, wb=BIG: L.tcq_int8_gated_ffn(
            p[0], p[1], p[2], p[3], p[4], p[5], m, n, k, act, p[6], dt, ws, wb, None), 7),
        "gated_ffn": (lambda p, m, n, k, dt=0, act=0, ws=P, wb=BIG: L.tcq_gated_ffn(
            p[0], p[1], p[2], dt, m, n, k, act, p[3], None, None, ws, wb, None), 4),
        "gated_ffn_backward": (lambda p, m, n, k, dt=0, act=0, ws=P, wb=BIG: L.tcq_gated_ffn_backward(
            p[0], p[1], p[2], p[3], p[4], p[5], dt, m, n, k, act, P, P, P, ws, wb, None), 6),
    }


NAMES = ["int8_matmul", "int8_gated_ffn", "gated_ffn", "gated_ffn_backward"]


@pytest.mark.parametrize("name", NAMES)
def test_products_refuse_bad_arguments(L, name):
    call, n_ptr = _calls(L)[name]
    good = [P] * n_ptr
    for sizes in ((-1, 8, 8), (4, 0, 8), (4, 8, 0), (4, -8, 8), (4, 8, -8)):
        assert call(good, *sizes) == INV, sizes
    for sizes in ((1 << 30, 8, 8), (4, 1 << 30, 8), (4, 8, 1 << 30)):
        assert call(good, *sizes) == UNS, sizes
    for dt in (-1, 3):
        assert call(good, 4, 8, 8, dt=dt) == INV
    if name.startswith("gated"):
        assert call(good, 4, 8, 8, dt=_abi.F32) == INV
    else:
        assert call(good, 4, 8, 131072) == UNS                 # 32-bit sums could overflow
    if name != "int8_matmul":
        for act in (-1, 4):
            assert call(good, 4, 8, 8, act=act) == INV
    for i in range(n_ptr):
        for bad in (None, ctypes.c_void_p(256 + 8)):
            p = list(good)
            p[i] = bad
            assert call(p, 4, 8, 8) == INV, (i, bad)


@pytest.mark.parametrize("name", NAMES)
def test_products_check_the_workspace(L, name):
    call, n_ptr = _calls(L)[name]
    good = [P] * n_ptr
    need = getattr(L, f"tcq_{name}_workspace_size")(5, 9, 7)   # rows of 7: operands are copied
    if name == "gated_ffn_backward":
        assert need >= 2 * 5 * 9 * 2
    if need:
        assert call(good, 5, 9, 7, wb=need - 1) == WSP
        assert call(good, 5, 9, 7, ws=None) == WSP
        assert call(good, 5, 9, 7, ws=ctypes.c_void_p(128)) == WSP


@pytest.mark.parametrize("name", ["int8_matmul", "int8_gated_ffn", "gated_ffn"])
def test_empty_batch_reads_no_pointer(L, name):
    call, n_ptr = _calls(L)[name]
    assert call([None] * n_ptr, 0, 8, 8, ws=None, wb=0) == OK


def test_backward_argument_combinations(L):
    f = L.tcq_gated_ffn_backward
    # a misaligned gradient; no gradient wanted at all
    assert f(P, P, P, P, P, P, 0, 4, 8, 8, 0, ctypes.c_void_p(264), None, None, P, BIG, None) == INV
    assert f(P, P, P, P, P, P, 0, 4, 8, 8, 0, None, None, None, None, 0, None) == OK
    # saved projections come in pairs
    g = L.tcq_gated_ffn
    assert g(P, P, P, 0, 4, 8, 8, 0, P, P, None, P, BIG, None) == INV
    assert g(P, P, P, 0, 4, 8, 8, 0, P, None, P, P, BIG, None) == INV
    assert g(P, P, P, 0, 4, 8, 8, 0, P, ctypes.c_void_p(260), P, P, BIG, None) == INV
    # a misaligned bias
    assert L.tcq_int8_matmul(P, P, P, P, ctypes.c_void_p(260), 4, 8, 8, P, 0, P, BIG, None) == INV


def test_outputs_may_not_overlap(L):
    # every operand in its own megabyte, then the output moved onto each of them, and onto the workspace
    def at(i, off=0):
        return ctypes.c_void_p((i + 1) << 20 | off)
    m, n, k = 200, 24, 40                                      # rows of 40 bytes: the workspace is in use
    ws = at(20)
    for onto in [at(i) for i in range(5)] + [at(0, m * k - 16), at(20), at(20, 256)]:
        assert L.tcq_int8_matmul(at(0), at(1), at(2), at(3), at(4), m, n, k, onto, 0, ws, BIG, None) == INV, onto
    for onto in [at(i) for i in range(6)] + [at(20)]:
        assert L.tcq_int8_gated_ffn(at(0), at(1), at(2), at(3), at(4), at(5), m, n, k, 0, onto, 0, ws, BIG,
                                    None) == INV
    for h, g, u in ((at(0), None, None), (at(2), None, None), (at(5), at(5), at(6)), (at(5), at(6), at(6, 16)),
                    (at(5), at(1), at(6))):
        assert L.tcq_gated_ffn(at(0), at(1), at(2), 0, m, n, 41, 0, h, g, u, ws, BIG, None) == INV
    for gx, g1, g2 in ((at(0), None, None), (None, at(1), None), (None, None, at(5)), (at(7), at(7), None),
                       (None, at(8), at(8, 16)), (at(20), None, None)):
        assert L.tcq_gated_ffn_backward(at(0), at(1), at(2), at(3), at(4), at(5), 0, m, n, k, 0, gx, g1, g2, ws, BIG,
                                        None) == INV
    assert L.tcq_quantize_int8(at(0), 0, m, k, at(0), at(1), None) == INV
    assert L.tcq_quantize_int8(at(0), 0, m, k, at(1), at(1, m * k - 16), None) == INV
    tr = ctypes.byref(_abi.trellis(16, 256))
    assert L.tcq_decode_int8(tr, at(0), 4, 0, 0, 0, 0, at(0, 64), None) == INV


def test_sizes_whose_tiles_pass_32_bits_are_refused(L):
    big = 1 << 29
    assert L.tcq_int8_matmul(P, P, P, P, None, big, big, 64, P, 0, P, BIG, None) == UNS
    assert L.tcq_gated_ffn(P, P, P, 0, 64, big, big, 0, P, None, None, P, BIG, None) == UNS
    assert L.tcq_gated_ffn_backward_workspace_size(big, 64, big) == 0


def test_workspace_sizes_of_impossible_products_are_zero(L):
    for name in NAMES:
        size = getattr(L, f"tcq_{name}_workspace_size")
        for bad in ((-1, 8, 8), (4, 0, 8), (4, 8, -1), (1 << 31, 8, 8)):
            assert size(*bad) == 0


def test_quantize_and_decode_refuse_bad_arguments(L):
    q = L.tcq_quantize_int8
    assert q(None, 0, 0, 8, None, None, None) == OK            # empty batch
    for dt, rows, cols, want in ((3, 4, 8, INV), (0, -1, 8, INV), (0, 4, 0, INV), (0, 1 << 30, 8, UNS),
                                 (0, 4, 1 << 30, UNS)):
        assert q(P, dt, rows, cols, P, P, None) == want
    for i in range(3):
        for bad in (None, ctypes.c_void_p(258)):
            p = [P, P, P]
            p[i] = bad
            assert q(p[0], 0, 4, 8, p[1], p[2], None) == INV
    d = L.tcq_decode_int8
    tr = ctypes.byref(_abi.trellis(16, 256))
    assert d(tr, None, 0, 0, 0, 0, 0, None, None) == OK
    for n, lay, out, r, c, want in ((-1, 0, 0, 0, 0, INV), (4, 2, 0, 0, 0, INV), (4, 0, 2, 0, 0, INV),
                                    (4, 0, 1, 32, 48, INV), (4, 0, 1, 32, 30, INV), (0, 0, 1, 0, 16, INV)):
        assert d(tr, P, n, lay, out, r, c, P, None) == want, (n, lay, out, r, c)
    assert d(tr, None, 4, 0, 0, 0, 0, P, None) == INV
    assert d(tr, P, 4, 0, 0, 0, 0, ctypes.c_void_p(264), None) == INV
    assert d(ctypes.byref(_abi.trellis(16, 128)), P, 4, 0, 1, 32, 32, P, None) == UNS
    assert d(ctypes.byref(_abi.trellis(10, 256)), P, 4, 0, 0, 0, 0, P, None) == UNS
    assert d(ctypes.byref(_abi.trellis(16, 7)), P, 4, 0, 0, 0, 0, P, None) == UNS


def test_quarter_of_the_code_numerator_fits_eight_bits():
    # decode_int8 does not clamp: no state of a supported trellis comes near 127
    for Lb in (8, 12, 16):
        x = (np.arange(1 << Lb, dtype=np.uint64) * 34038481 + 76625530) & 0xFFFFFFFF
        k = sum((x >> s) & 255 for s in (0, 8, 16, 24)).astype(np.int64) - 510
        assert np.abs(k).max() <= 483 and np.abs(np.rint(k / 4)).max() <= 121
        # the mean squared error the header quotes: k mod 4 spread evenly leaves (0 + 1 + 4 + 1) / 4 = 1.5 in
        # units of 1 / 147.8^2, a single state's error has a standard deviation of 1.5 of them
        err = (np.rint(k / 4) * tcq.DECODE_INT8_SCALE - k / 147.8) ** 2 * 147.8 ** 2
        assert abs(err.mean() - 1.5) < 4 * 1.5 / 2 ** (Lb / 2)


# ------------------------------------------------------------------ binding

class _NoLaunch:
    def __getattr__(self, name):
        raise AssertionError(f"{name} was reached")


@pytest.fixture
def no_launch(monkeypatch):
    monkeypatch.setattr(tcq, "lib", lambda: _NoLaunch())


def test_binding_refuses_host_tensors(no_launch):
    x = torch.zeros(4, 32, dtype=torch.float16)
    w = torch.zeros(8, 32, dtype=torch.float16)
    q, s = torch.zeros(4, 32, dtype=torch.int8), torch.ones(4)
    qw, sw = torch.zeros(8, 32, dtype=torch.int8), torch.ones(8)
    g = torch.zeros(4, 8)
    bits = torch.zeros(4, 16, dtype=torch.int32).view(torch.uint32)
    for call in (lambda: tcq.quantize_int8(x), lambda: tcq.decode_int8(bits, 16),
                 lambda: tcq.int8_matmul(q, s, qw, sw), lambda: tcq.gated_ffn(x, w, w),
                 lambda: tcq.int8_gated_ffn(q, s, qw, sw, qw, sw),
                 lambda: tcq.gated_ffn_backward(x, w, w, g, g, g.half()),
                 lambda: tcq.GatedFfn.apply(x, w.requires_grad_(), w, tcq.ACT_SILU)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_binding_checks_shapes_and_types(no_launch, monkeypatch):
    # past the device check, so that the host tensors stand for device ones
    monkeypatch.setattr(tcq, "_require_cuda", lambda *t: None)
    f16 = dict(dtype=torch.float16)
    x, w = torch.zeros(4, 32, **f16), torch.zeros(8, 32, **f16)
    q, s = torch.zeros(4, 32, dtype=torch.int8), torch.ones(4)
    qw, sw = torch.zeros(8, 32, dtype=torch.int8), torch.ones(8)
    g, h = torch.zeros(4, 8), torch.zeros(4, 8, **f16)
    bad = [
        lambda: tcq.quantize_int8(torch.zeros(4)),
        lambda: tcq.quantize_int8(torch.zeros(4, 4, dtype=torch.float64)),
        lambda: tcq.int8_matmul(x, s, qw, sw), lambda: tcq.int8_matmul(q, s[:3], qw, sw),
        lambda: tcq.int8_matmul(q, s.double(), qw, sw), lambda: tcq.int8_matmul(q, s, qw[:, :16], sw),
        lambda: tcq.int8_matmul(q, s, sw.to(torch.int8), sw), lambda: tcq.int8_matmul(q, s, sw[0].to(torch.int8), sw),
        lambda: tcq.int8_matmul(q, s, w, sw), lambda: tcq.int8_matmul(q, s, qw, sw[:7]),
        lambda: tcq.int8_matmul(q, s, qw, sw, bias=torch.zeros(7)),
        lambda: tcq.int8_matmul(q, s, qw, sw, bias=torch.zeros(8, **f16)),
        lambda: tcq.int8_matmul(q, s, qw, sw, out_dtype=torch.float64),
        lambda: tcq.int8_matmul(q, s, qw, sw, out=torch.zeros(4, 7, **f16)),
        lambda: tcq.int8_gated_ffn(q, s, qw, sw, qw[:4], sw),
        lambda: tcq.int8_gated_ffn(q, s, qw, sw, qw, sw[:4]),
        lambda: tcq.gated_ffn(x.float(), w.float(), w.float()), lambda: tcq.gated_ffn(x[0], w, w),
        lambda: tcq.gated_ffn(x, w, w[:4]), lambda: tcq.gated_ffn(x, w.bfloat16(), w.bfloat16()),
        lambda: tcq.gated_ffn(x, w[:, :16], w[:, :16]),
        lambda: tcq.gated_ffn(x, w, w, out=torch.zeros(4, 8)),
        lambda: tcq.gated_ffn_backward(x, w, w, g.half(), g, h),
        lambda: tcq.gated_ffn_backward(x, w, w, g, g[:, :4], h),
        lambda: tcq.gated_ffn_backward(x, w, w, g, g, g),
        lambda: tcq.gated_ffn_backward(x, w, w, g, g, h[:2]),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(str(i))
