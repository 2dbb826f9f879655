"""Bitshift-trellis coded quantisation on NVIDIA B200 (sm_100a).

Thin PyTorch binding of ``libtcq.so`` (C ABI in ``include/tcq.h``).  Every
step of the computation runs in the library's CUDA kernels; this module only
checks tensor shapes, allocates outputs and workspaces with torch's caching
allocator and passes device pointers and the current CUDA stream.  There is
no CPU fallback: without the built library or a CUDA device every call raises.

Functions (QTIP blog "The trellis: a stateful codebook" / "The codebook is
computed" / "Tail-biting is worth its complexity"; BCJR-QAT abstract):
  viterbi_encode(s, L)                   -> (states uint16 [n,T], mse f32 [n])
  viterbi_encode_tailbiting(s, L)        -> tail-biting walks (2 bits per weight)
  bcjr_soft(s, L, temp)                  -> (soft f32 [n,T], log_z f32 [n])
  bcjr_soft_backward(s, L, temp, soft, g)-> grad_s f32 [n,T]
  bcjr_soft_and_grad(s, L, temp, g)      -> (soft, log_z, grad_s) in one sweep
  BcjrSoft.apply(s, L, temp)             -> soft (autograd through the VJP)
  pack_states(states, L, layout)         -> bits uint32 [n, words]
  decode(bits, L, T, layout, ...)        -> fp16 weights
  rht(W, sign_rows, sign_cols)           -> random-sign Hadamard rotation of W
Products on decoded weights:
  quantize_int8(x)                       -> (int8 rows, fp32 scale a row)
  decode_int8(bits, L, T, layout, ...)   -> int8 weights (scale DECODE_INT8_SCALE)
  int8_matmul(a, a_scale, w, w_scale)    -> a w^T with token and channel scales
  gated_ffn(x, w_gate, w_up, act)        -> act(x w_gate^T) * (x w_up^T)
  gated_ffn_backward(...)                -> its three gradients
  GatedFfn.apply(x, w_gate, w_up, act)   -> the block under autograd
  int8_gated_ffn(a, a_scale, ...)        -> the block on int8 tokens and weights
"""
from __future__ import annotations

import ctypes
from functools import lru_cache

import torch
from torch.autograd.forward_ad import unpack_dual

from . import _abi
from ._abi import (ACT_GELU, ACT_GELU_TANH, ACT_RELU, ACT_SILU, FREE_START, OUT_SEQ, OUT_TILE16,
                   TAILBITING, TcqError, check, lib, status_string, trellis)

__all__ = [
    "viterbi_encode", "viterbi_encode_tailbiting", "bcjr_soft", "bcjr_soft_and_grad", "bcjr_soft_backward", "BcjrSoft", "pack_states", "decode",
    "stream_words", "viterbi_workspace_size", "bcjr_workspace_size", "TcqError", "rht",
    "decode_gemv",
    "TAILBITING", "FREE_START", "OUT_SEQ", "OUT_TILE16", "lib", "status_string",
    "quantize_int8", "decode_int8", "int8_matmul", "gated_ffn", "gated_ffn_backward", "GatedFfn",
    "int8_gated_ffn", "DECODE_INT8_SCALE", "int8_matmul_workspace_size", "gated_ffn_workspace_size",
    "gated_ffn_backward_workspace_size", "int8_gated_ffn_workspace_size",
    "ACT_SILU", "ACT_GELU", "ACT_GELU_TANH", "ACT_RELU", "products_gave_up",
]

# one step of decode_int8 in units of the 1MAD code: (bytesum - 510) / 147.8 = 4 q / 147.8
DECODE_INT8_SCALE = 4 / 147.8

_DTYPE = {torch.float16: _abi.F16, torch.bfloat16: _abi.BF16, torch.float32: _abi.F32}


def _require_cuda(*tensors: "torch.Tensor | None") -> None:
    """Every tensor a call hands to the library (None entries skipped) is
    contiguous and on the current CUDA device, the one the library launches
    on: a host pointer, or another device's, would reach the kernels."""
    dev = None
    for t in tensors:
        if t is None:
            continue
        at = t.get_device() if t.is_cuda else -1
        if at < 0:
            raise ValueError("tensors must be CUDA tensors (no CPU fallback)")
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous")
        if dev is None:
            dev = at
        elif at != dev:
            raise ValueError(f"tensors must all be on one device (cuda:{dev} and cuda:{at})")
    if dev is not None and dev != torch.cuda.current_device():
        raise ValueError(f"tensors are on cuda:{dev} but the current device is "
                         f"cuda:{torch.cuda.current_device()} (select it with torch.cuda.device)")


def _out(out: torch.Tensor, shape, dtype, *like: torch.Tensor) -> torch.Tensor:
    """A caller's output tensor, checked before any launch: the kernels
    write all of ``shape`` in ``dtype`` through its pointer."""
    if tuple(out.shape) != tuple(shape) or out.dtype != dtype:
        raise ValueError(f"out must be a {dtype} tensor of shape {tuple(shape)}, "
                         f"not {out.dtype} {tuple(out.shape)}")
    _require_cuda(out, *like)
    return out


def _nbytes(t: torch.Tensor) -> int:
    return t.numel() * t.element_size()


# Plain integers for the void* parameters: ctypes converts them by the declared
# argument types, and building a c_void_p and a Stream object for each call
# costs a small call more than its kernel runs (14 against 7 us for one row).
def _stream() -> int:
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


def _ptr(t: "torch.Tensor | None") -> int:
    return t.data_ptr() if t is not None else 0


def _workspace(nbytes: int, device) -> torch.Tensor:
    # 256-byte aligned: the caching allocator hands out 512-byte aligned blocks
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


# torch.empty spends most of its 1.6 us on parsing its arguments; the entry point
# that torch's own generated code allocates with takes 0.8 (a call of the products
# below runs for 2 to 13 us on the GPU).  Both use the caching allocator.
_empty_strided = getattr(getattr(getattr(torch._C, "_dynamo", None), "guards", None),
                         "_empty_strided_cuda", None)


def _empty(shape: tuple, dtype: torch.dtype) -> torch.Tensor:
    """An uninitialised contiguous 1-D or 2-D tensor on the current device (the
    one every operand was checked to be on)."""
    if _empty_strided is None:
        return torch.empty(shape, dtype=dtype, device="cuda")
    return _empty_strided(shape, (1,) if len(shape) == 1 else (shape[1] or 1, 1), dtype)


def _scratch(workspace: "torch.Tensor | None", need: int, like: torch.Tensor) -> torch.Tensor:
    """As _use_workspace, for the products."""
    return _empty((need or 256,), torch.uint8) if workspace is None else _use_workspace(workspace, need, like)


def _use_workspace(workspace: "torch.Tensor | None", need: int, like: torch.Tensor) -> torch.Tensor:
    """The caller's workspace (any dtype, counted in bytes) when it holds
    ``need`` bytes, else a fresh one on ``like``'s device."""
    if workspace is not None:
        _require_cuda(workspace, like)
        if _nbytes(workspace) >= need:
            return workspace
    return _workspace(need, like.device)


def stream_words(L: int, seq_len: int, layout: int) -> int:
    return int(lib().tcq_stream_words(ctypes.byref(trellis(L, seq_len)), int(layout)))


def viterbi_workspace_size(L: int, seq_len: int, n_seq: int) -> int:
    return int(lib().tcq_viterbi_workspace_size(ctypes.byref(trellis(L, seq_len)), int(n_seq)))


def bcjr_workspace_size(L: int, seq_len: int, n_seq: int, with_grad: bool = False) -> int:
    return int(lib().tcq_bcjr_workspace_size(ctypes.byref(trellis(L, seq_len)), int(n_seq),
                                             int(bool(with_grad))))


def _weights(D: torch.Tensor | None, s: torch.Tensor) -> torch.Tensor | None:
    if D is None:
        return None
    _require_cuda(D, s)
    if D.shape != s.shape or D.dtype != torch.float32:
        raise ValueError("D must be a float32 tensor shaped like s")
    return D


def viterbi_encode(s: torch.Tensor, L: int, workspace: torch.Tensor | None = None,
                   D: torch.Tensor | None = None, margin: bool = False):
    """Min-MSE walk of every row of ``s`` [n, T] (fp32) on the (L, 2, 1)
    bitshift trellis with the 1MAD code; returns (states uint16, mse fp32),
    and with ``margin=True`` also the smallest relative decision margin along
    each walk (fp32 [n]; a second forward pass).  ``D`` (optional, same
    shape) weights each step's squared error."""
    _require_cuda(s)
    D = _weights(D, s)
    if s.dtype != torch.float32 or s.dim() != 2:
        raise ValueError("s must be a 2-D float32 tensor [n_seq, seq_len]")
    n, T = s.shape
    tr = trellis(L, T)
    states = torch.empty((n, T), dtype=torch.uint16, device=s.device)
    mse = torch.empty((n,), dtype=torch.float32, device=s.device)
    mrg = torch.empty((n,), dtype=torch.float32, device=s.device) if margin else None
    need = int(lib().tcq_viterbi_workspace_size(ctypes.byref(tr), n))
    ws = _use_workspace(workspace, need, s)
    check(lib().tcq_viterbi_encode(ctypes.byref(tr), _ptr(s), _ptr(D), n, _ptr(states), _ptr(mse),
                                   _ptr(mrg), _ptr(ws), _nbytes(ws), _stream()), "tcq_viterbi_encode")
    return (states, mse, mrg) if margin else (states, mse)


def viterbi_encode_tailbiting(s: torch.Tensor, L: int, workspace: torch.Tensor | None = None,
                              D: torch.Tensor | None = None):
    """Tail-biting walk of every row (two-run search: rotated free run, then a
    run with both ends pinned to the overlap read at the seam); returns
    (states uint16, mse fp32).  Pack the walk with layout TAILBITING."""
    _require_cuda(s)
    D = _weights(D, s)
    if s.dtype != torch.float32 or s.dim() != 2:
        raise ValueError("s must be a 2-D float32 tensor [n_seq, seq_len]")
    n, T = s.shape
    tr = trellis(L, T)
    states = torch.empty((n, T), dtype=torch.uint16, device=s.device)
    mse = torch.empty((n,), dtype=torch.float32, device=s.device)
    need = int(lib().tcq_viterbi_workspace_size(ctypes.byref(tr), n))
    ws = _use_workspace(workspace, need, s)
    check(lib().tcq_viterbi_encode_tailbiting(ctypes.byref(tr), _ptr(s), _ptr(D), n, _ptr(states),
                                              _ptr(mse), _ptr(ws), _nbytes(ws), _stream()),
          "tcq_viterbi_encode_tailbiting")
    return states, mse


def bcjr_soft(s: torch.Tensor, L: int, temp: float, workspace: torch.Tensor | None = None,
              D: torch.Tensor | None = None):
    """Soft codeword (Boltzmann expectation of the code at temperature
    ``temp``) of every row of ``s``; returns (soft fp32 [n,T], log_z fp32 [n])."""
    _require_cuda(s)
    D = _weights(D, s)
    if s.dtype != torch.float32 or s.dim() != 2:
        raise ValueError("s must be a 2-D float32 tensor [n_seq, seq_len]")
    n, T = s.shape
    tr = trellis(L, T)
    soft = torch.empty_like(s)
    logz = torch.empty((n,), dtype=torch.float32, device=s.device)
    need = int(lib().tcq_bcjr_workspace_size(ctypes.byref(tr), n, 0))
    ws = _use_workspace(workspace, need, s)
    check(lib().tcq_bcjr_soft(ctypes.byref(tr), _ptr(s), _ptr(D), n, float(temp), _ptr(soft),
                              _ptr(logz), _ptr(ws), _nbytes(ws), _stream()), "tcq_bcjr_soft")
    return soft, logz


def bcjr_soft_backward(s: torch.Tensor, L: int, temp: float, soft: torch.Tensor,
                       grad_soft: torch.Tensor, workspace: torch.Tensor | None = None,
                       D: torch.Tensor | None = None):
    """Vector-Jacobian product: grad_s[u] = sum_t grad_soft[t] d soft[t] / d s[u]."""
    _require_cuda(s, soft, grad_soft)
    D = _weights(D, s)
    if (s.dim() != 2 or s.shape != soft.shape or s.shape != grad_soft.shape
            or any(t.dtype != torch.float32 for t in (s, soft, grad_soft))):
        raise ValueError("s, soft and grad_soft must be float32 tensors of one shape [n_seq, seq_len]")
    n, T = s.shape
    tr = trellis(L, T)
    grad = torch.empty_like(s)
    need = int(lib().tcq_bcjr_workspace_size(ctypes.byref(tr), n, 1))
    ws = _use_workspace(workspace, need, s)
    check(lib().tcq_bcjr_soft_backward(ctypes.byref(tr), _ptr(s), _ptr(D), n, float(temp),
                                       _ptr(soft), _ptr(grad_soft), _ptr(grad), _ptr(ws),
                                       _nbytes(ws), _stream()), "tcq_bcjr_soft_backward")
    return grad


def bcjr_soft_and_grad(s: torch.Tensor, L: int, temp: float, grad_soft: torch.Tensor,
                       workspace: torch.Tensor | None = None, D: torch.Tensor | None = None):
    """Soft codeword, log Z and the vector-Jacobian product for a known
    cotangent ``grad_soft``, in one forward-backward sweep; returns
    (soft, log_z, grad_s)."""
    _require_cuda(s, grad_soft)
    D = _weights(D, s)
    if (s.dim() != 2 or s.shape != grad_soft.shape or s.dtype != torch.float32
            or grad_soft.dtype != torch.float32):
        raise ValueError("s and grad_soft must be float32 tensors of one shape [n_seq, seq_len]")
    n, T = s.shape
    tr = trellis(L, T)
    soft = torch.empty_like(s)
    logz = torch.empty((n,), dtype=torch.float32, device=s.device)
    grad = torch.empty_like(s)
    need = int(lib().tcq_bcjr_workspace_size(ctypes.byref(tr), n, 1))
    ws = _use_workspace(workspace, need, s)
    check(lib().tcq_bcjr_soft_and_grad(ctypes.byref(tr), _ptr(s), _ptr(D), n, float(temp),
                                       _ptr(grad_soft), _ptr(soft), _ptr(logz), _ptr(grad),
                                       _ptr(ws), _nbytes(ws), _stream()), "tcq_bcjr_soft_and_grad")
    return soft, logz, grad


class BcjrSoft(torch.autograd.Function):
    """soft = BcjrSoft.apply(s, L, temp[, D]): differentiable soft codeword."""

    @staticmethod
    def forward(ctx, s, L, temp, D=None):
        soft, _ = bcjr_soft(s, L, temp, D=D)
        ctx.save_for_backward(s, soft, D)
        ctx.L, ctx.temp = L, temp
        return soft

    @staticmethod
    def backward(ctx, g):
        s, soft, D = ctx.saved_tensors
        return bcjr_soft_backward(s, ctx.L, ctx.temp, soft, g.contiguous(), D=D), None, None, None


def pack_states(states: torch.Tensor, L: int, layout: int = FREE_START) -> torch.Tensor:
    """Pack walks [n, T] (uint16) into MSB-first bitstreams [n, words] (uint32)."""
    _require_cuda(states)
    if states.dtype != torch.uint16 or states.dim() != 2:
        raise ValueError("states must be a 2-D uint16 tensor")
    n, T = states.shape
    tr = trellis(L, T)
    words = int(lib().tcq_stream_words(ctypes.byref(tr), int(layout)))
    if words == 0:
        raise TcqError(_abi.TCQ_ERR_UNSUPPORTED, "tcq_stream_words")
    bits = torch.empty((n, words), dtype=torch.uint32, device=states.device)
    check(lib().tcq_pack_states(ctypes.byref(tr), _ptr(states), n, int(layout), _ptr(bits),
                                _stream()), "tcq_pack_states")
    return bits


def decode(bits: torch.Tensor, L: int, seq_len: int = 256, layout: int = TAILBITING,
           out_layout: int = OUT_SEQ, rows: int = 0, cols: int = 0,
           out: torch.Tensor | None = None) -> torch.Tensor:
    """Decode bitstreams [n, words] (uint32) into fp16 weights: [n, seq_len]
    (OUT_SEQ) or a [rows, cols] matrix of 16x16 tiles (OUT_TILE16)."""
    _require_cuda(bits)
    if bits.dtype != torch.uint32 or bits.dim() != 2:
        raise ValueError("bits must be a 2-D uint32 tensor")
    n = bits.shape[0]
    tr = trellis(L, seq_len)
    words = int(lib().tcq_stream_words(ctypes.byref(tr), int(layout)))
    if words == 0:
        raise TcqError(_abi.TCQ_ERR_UNSUPPORTED, "tcq_stream_words")
    if bits.shape[1] != words:
        raise ValueError(f"bits must have {words} words per sequence for this trellis and layout")
    shape = (rows, cols) if out_layout == OUT_TILE16 else (n, seq_len)
    if out is None:
        out = torch.empty(shape, dtype=torch.float16, device=bits.device)
    else:
        _out(out, shape, torch.float16, bits)
    check(lib().tcq_decode(ctypes.byref(tr), _ptr(bits), n, int(layout), int(out_layout), int(rows),
                           int(cols), _ptr(out), _stream()), "tcq_decode")
    return out


def rht(W: torch.Tensor, sign_rows: torch.Tensor, sign_cols: torch.Tensor,
        out: torch.Tensor | None = None) -> torch.Tensor:
    """Random-sign Hadamard rotation (H_R/sqrt R) diag(sign_rows) W
    diag(sign_cols) (H_C/sqrt C) of a fp32 matrix (``out`` may be ``W``)."""
    _require_cuda(W, sign_rows, sign_cols)
    if W.dim() != 2 or W.dtype != torch.float32:
        raise ValueError("W must be a 2-D float32 tensor")
    R, C = W.shape
    if sign_rows.shape != (R,) or sign_cols.shape != (C,):
        raise ValueError("sign vectors must match W's rows and columns")
    out = torch.empty_like(W) if out is None else _out(out, (R, C), torch.float32, W)
    # named: an address does not keep a converted copy alive, and the second could take the first's memory
    sign_rows, sign_cols = sign_rows.float().contiguous(), sign_cols.float().contiguous()
    check(lib().tcq_rht(_ptr(W), R, C, _ptr(sign_rows), _ptr(sign_cols), _ptr(out), _stream()), "tcq_rht")
    return out


def decode_gemv(bits: torch.Tensor, x: torch.Tensor, rows: int, cols: int, L: int = 16,
                layout: int = TAILBITING, out: torch.Tensor | None = None) -> torch.Tensor:
    """y = W x with W the fp16 matrix decoded from 16x16-tile streams ``bits``,
    decoded in registers (never materialised); fp32 products and sums."""
    _require_cuda(bits, x)
    if bits.dtype != torch.uint32 or x.dtype != torch.float32 or x.shape != (cols,):
        raise ValueError("bits must be uint32 [tiles, words] and x float32 [cols]")
    tr = trellis(L, 256)
    words = int(lib().tcq_stream_words(ctypes.byref(tr), int(layout)))
    if bits.shape != ((rows // 16) * (cols // 16), words):
        raise ValueError("bits must hold one stream per 16x16 tile")
    y = (torch.empty((rows,), dtype=torch.float32, device=x.device) if out is None
         else _out(out, (rows,), torch.float32, x))
    check(lib().tcq_decode_gemv(ctypes.byref(tr), _ptr(bits), int(layout), int(rows), int(cols),
                                _ptr(x), _ptr(y), _stream()), "tcq_decode_gemv")
    return y


def products_gave_up() -> int:
    """How often a product's kernel on the current device gave up a wait of
    its own (0 unless something is wrong); waits for the device.  The next
    product after such a one raises TcqError, with status -5."""
    count = ctypes.c_uint()
    check(lib().tcq_products_gave_up(ctypes.byref(count)), "tcq_products_gave_up")
    return count.value


def int8_matmul_workspace_size(n_tok: int, n_out: int, n_in: int) -> int:
    return int(lib().tcq_int8_matmul_workspace_size(int(n_tok), int(n_out), int(n_in)))


def gated_ffn_workspace_size(n_tok: int, n_out: int, n_in: int) -> int:
    return int(lib().tcq_gated_ffn_workspace_size(int(n_tok), int(n_out), int(n_in)))


def gated_ffn_backward_workspace_size(n_tok: int, n_out: int, n_in: int) -> int:
    return int(lib().tcq_gated_ffn_backward_workspace_size(int(n_tok), int(n_out), int(n_in)))


def int8_gated_ffn_workspace_size(n_tok: int, n_out: int, n_in: int) -> int:
    return int(lib().tcq_int8_gated_ffn_workspace_size(int(n_tok), int(n_out), int(n_in)))


def quantize_int8(x: torch.Tensor):
    """Row-wise symmetric int8 quantisation of ``x`` [rows, cols] (fp16, bf16
    or fp32); returns (q int8 [rows, cols], scale fp32 [rows]) with x ~ q *
    scale: scale = max|row| / 127, q = x / scale rounded to nearest, ties to
    even, at most 127 in size.  A zero row gives scale 0, a row with an
    infinity or NaN scale NaN."""
    _require_cuda(x)
    if x.dim() != 2 or x.dtype not in _DTYPE:
        raise ValueError("x must be a 2-D float16, bfloat16 or float32 tensor")
    rows, cols = x.shape
    q, scale = _empty((rows, cols), torch.int8), _empty((rows,), torch.float32)
    check(lib().tcq_quantize_int8(_ptr(x), _DTYPE[x.dtype], rows, cols, _ptr(q), _ptr(scale),
                                  _stream()), "tcq_quantize_int8")
    return q, scale


@lru_cache(maxsize=256)
def _stream_shape(L: int, seq_len: int, layout: int):
    """The trellis as the library takes it, and the words of a stream."""
    tr = trellis(L, seq_len)
    return tr, stream_words(L, seq_len, layout)


def decode_int8(bits: torch.Tensor, L: int, seq_len: int = 256, layout: int = TAILBITING,
                out_layout: int = OUT_SEQ, rows: int = 0, cols: int = 0,
                out: torch.Tensor | None = None) -> torch.Tensor:
    """Decode bitstreams as ``decode`` does, but to int8: the code is
    DECODE_INT8_SCALE times the result to within half a step."""
    _require_cuda(bits)
    if bits.dtype != torch.uint32 or bits.dim() != 2:
        raise ValueError("bits must be a 2-D uint32 tensor")
    n = bits.shape[0]
    tr, words = _stream_shape(int(L), int(seq_len), int(layout))
    if words == 0:
        raise TcqError(_abi.TCQ_ERR_UNSUPPORTED, "tcq_stream_words")
    if bits.shape[1] != words:
        raise ValueError(f"bits must have {words} words per sequence for this trellis and layout")
    shape = (int(rows), int(cols)) if out_layout == OUT_TILE16 else (n, int(seq_len))
    if min(shape) < 0:
        raise ValueError("rows and cols must not be negative")
    if out is None:
        out = _empty(shape, torch.int8)
    else:
        _out(out, shape, torch.int8, bits)
    check(lib().tcq_decode_int8(ctypes.byref(tr), _ptr(bits), n, int(layout), int(out_layout),
                                int(rows), int(cols), _ptr(out), _stream()), "tcq_decode_int8")
    return out


def _int8_operands(a, a_scale, weights, bias=None):
    """Shapes and types of an int8 product's operands; returns (n_tok, n_out, n_in)."""
    _require_cuda(a, a_scale, bias, *weights)
    if a.dim() != 2 or a.dtype != torch.int8:
        raise ValueError("a must be a 2-D int8 tensor [n_tok, n_in]")
    n_tok, n_in = a.shape
    n_out = weights[0].shape[0] if weights[0].dim() == 2 else -1
    for w, ws in zip(weights[::2], weights[1::2]):
        if w.dtype != torch.int8 or w.shape != (n_out, n_in):
            raise ValueError(f"weights must be int8 tensors of one shape [n_out, {n_in}]")
        if ws.dtype != torch.float32 or ws.shape != (n_out,):
            raise ValueError(f"a weight's scale must be a float32 tensor [{n_out}]")
    if a_scale.dtype != torch.float32 or a_scale.shape != (n_tok,):
        raise ValueError(f"a_scale must be a float32 tensor [{n_tok}]")
    if bias is not None and (bias.dtype != torch.float32 or bias.shape != (n_out,)):
        raise ValueError(f"bias must be a float32 tensor [{n_out}]")
    return n_tok, n_out, n_in


def _result(out, shape, dtype, like):
    if dtype not in _DTYPE:
        raise ValueError("the output type must be float16, bfloat16 or float32")
    return _empty(shape, dtype) if out is None else _out(out, shape, dtype, like)


def int8_matmul(a: torch.Tensor, a_scale: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor,
                bias: torch.Tensor | None = None, out_dtype: torch.dtype = torch.float16,
                out: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """out[m, n] = a_scale[m] w_scale[n] (a w^T)[m, n] + bias[n] for int8
    tokens ``a`` [n_tok, n_in] and weights ``w`` [n_out, n_in] with fp32
    scales; the product is exact in 32-bit integers."""
    n_tok, n_out, n_in = _int8_operands(a, a_scale, (w, w_scale), bias)
    out = _result(out, (n_tok, n_out), out_dtype, a)
    need = int(lib().tcq_int8_matmul_workspace_size(n_tok, n_out, n_in))
    ws = _scratch(workspace, need, a) if need else None
    check(lib().tcq_int8_matmul(_ptr(a), _ptr(a_scale), _ptr(w), _ptr(w_scale), _ptr(bias), n_tok,
                                n_out, n_in, _ptr(out), _DTYPE[out_dtype], _ptr(ws),
                                _nbytes(ws) if need else 0, _stream()), "tcq_int8_matmul")
    return out


def int8_gated_ffn(a: torch.Tensor, a_scale: torch.Tensor, w_gate: torch.Tensor,
                   w_gate_scale: torch.Tensor, w_up: torch.Tensor, w_up_scale: torch.Tensor,
                   act: int = ACT_SILU, out_dtype: torch.dtype = torch.float16,
                   out: torch.Tensor | None = None,
                   workspace: torch.Tensor | None = None) -> torch.Tensor:
    """The gated feed-forward block on int8 operands: act(g) * u with g and u
    the scaled int8 products of ``a`` with ``w_gate`` and ``w_up``."""
    n_tok, n_out, n_in = _int8_operands(a, a_scale, (w_gate, w_gate_scale, w_up, w_up_scale))
    out = _result(out, (n_tok, n_out), out_dtype, a)
    need = int(lib().tcq_int8_gated_ffn_workspace_size(n_tok, n_out, n_in))
    ws = _scratch(workspace, need, a) if need else None
    check(lib().tcq_int8_gated_ffn(_ptr(a), _ptr(a_scale), _ptr(w_gate), _ptr(w_gate_scale),
                                   _ptr(w_up), _ptr(w_up_scale), n_tok, n_out, n_in, int(act),
                                   _ptr(out), _DTYPE[out_dtype], _ptr(ws),
                                   _nbytes(ws) if need else 0, _stream()), "tcq_int8_gated_ffn")
    return out


def _ffn_operands(x, w_gate, w_up):
    _require_cuda(x, w_gate, w_up)
    if x.dim() != 2 or x.dtype not in (torch.float16, torch.bfloat16):
        raise ValueError("x must be a 2-D float16 or bfloat16 tensor [n_tok, n_in]")
    n_tok, n_in = x.shape
    if w_gate.dim() != 2 or w_gate.shape[1] != n_in or w_up.shape != w_gate.shape:
        raise ValueError(f"w_gate and w_up must be tensors of one shape [n_out, {n_in}]")
    if w_gate.dtype != x.dtype or w_up.dtype != x.dtype:
        raise ValueError(f"w_gate and w_up must be {x.dtype} like x")
    return n_tok, w_gate.shape[0], n_in


def _launch_ffn(x, w_gate, w_up, act, sizes, out, gate, up, workspace):
    """gated_ffn on checked operands; gate and up: addresses, 0 for none."""
    need = int(lib().tcq_gated_ffn_workspace_size(*sizes))
    ws = _scratch(workspace, need, x) if need else None
    check(lib().tcq_gated_ffn(_ptr(x), _ptr(w_gate), _ptr(w_up), _DTYPE[x.dtype], *sizes, int(act),
                              _ptr(out), gate, up, _ptr(ws), _nbytes(ws) if need else 0, _stream()),
          "tcq_gated_ffn")


def _launch_ffn_backward(x, w_gate, w_up, gate, up, grad_out, act, sizes, need, workspace):
    """gated_ffn_backward on checked operands; gate and up: addresses."""
    grads = [_empty(tuple(t.shape), t.dtype) if n else None for t, n in zip((x, w_gate, w_up), need)]
    size = int(lib().tcq_gated_ffn_backward_workspace_size(*sizes))
    ws = _scratch(workspace, size, x)
    check(lib().tcq_gated_ffn_backward(_ptr(x), _ptr(w_gate), _ptr(w_up), gate, up, _ptr(grad_out),
                                       _DTYPE[x.dtype], *sizes, int(act), _ptr(grads[0]),
                                       _ptr(grads[1]), _ptr(grads[2]), _ptr(ws), _nbytes(ws),
                                       _stream()), "tcq_gated_ffn_backward")
    return tuple(grads)


def gated_ffn(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, act: int = ACT_SILU,
              out: torch.Tensor | None = None, save: bool = False,
              workspace: torch.Tensor | None = None):
    """h = act(x w_gate^T) * (x w_up^T) for fp16 or bf16 tokens ``x`` [n_tok,
    n_in] and weights [n_out, n_in], sums and activation in fp32.  With
    ``save=True`` returns (h, gate, up), the fp32 projections that
    ``gated_ffn_backward`` takes."""
    sizes = _ffn_operands(x, w_gate, w_up)
    out = _result(out, sizes[:2], x.dtype, x)
    gate = up = None
    if save:
        gate, up = _empty(sizes[:2], torch.float32), _empty(sizes[:2], torch.float32)
    _launch_ffn(x, w_gate, w_up, act, sizes, out, _ptr(gate), _ptr(up), workspace)
    return (out, gate, up) if save else out


def gated_ffn_backward(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor,
                       gate: torch.Tensor, up: torch.Tensor, grad_out: torch.Tensor,
                       act: int = ACT_SILU, need: "tuple[bool, bool, bool]" = (True, True, True),
                       workspace: torch.Tensor | None = None):
    """Gradients of ``gated_ffn`` for the output gradient ``grad_out`` and the
    saved ``gate`` and ``up``; returns (grad_x, grad_w_gate, grad_w_up), None
    where ``need`` is false."""
    sizes = _ffn_operands(x, w_gate, w_up)
    _require_cuda(x, gate, up, grad_out)
    if any(t.shape != sizes[:2] or t.dtype != torch.float32 for t in (gate, up)):
        raise ValueError(f"gate and up must be float32 tensors {list(sizes[:2])}")
    if grad_out.shape != sizes[:2] or grad_out.dtype != x.dtype:
        raise ValueError(f"grad_out must be a {x.dtype} tensor {list(sizes[:2])}")
    return _launch_ffn_backward(x, w_gate, w_up, _ptr(gate), _ptr(up), grad_out, act, sizes, need,
                                workspace)


class GatedFfn(torch.autograd.Function):
    """h = GatedFfn.apply(x, w_gate, w_up, act): ``gated_ffn`` with its
    gradients.  It keeps the two projections in fp32 for the backward pass (8
    bytes a hidden value; rounded to 16 bits they would cost the gradients
    more than the rounding of their own operands); without gradients to
    compute, or under ``torch.no_grad()``, it is ``gated_ffn``.  Twice
    differentiable it is not: a second derivative raises.  A step may be
    captured into a CUDA graph once eager graphs of the same leaves are gone
    (torch's own rule for captured backward passes)."""

    @classmethod
    def apply(cls, x, w_gate, w_up, act=ACT_SILU):
        # inside forward() the grad mode is always off, so it is asked here; a tangent of forward mode,
        # which no_grad() leaves on, goes to the Function, which refuses it
        if not torch.is_grad_enabled() and all(unpack_dual(t).tangent is None for t in (x, w_gate, w_up)):
            return gated_ffn(x, w_gate, w_up, act)
        return super().apply(x, w_gate, w_up, act)

    @staticmethod
    def forward(ctx, x, w_gate, w_up, act):
        if not any(ctx.needs_input_grad[:3]):
            return gated_ffn(x, w_gate, w_up, act)
        sizes = _ffn_operands(x, w_gate, w_up)
        out = _result(None, sizes[:2], x.dtype, x)
        # both projections in one buffer, the second on a 16-byte boundary
        half = (sizes[0] * sizes[1] + 3) // 4 * 4
        saved = _empty((2 * half,), torch.float32)
        _launch_ffn(x, w_gate, w_up, act, sizes, out, _ptr(saved), _ptr(saved) + 4 * half, None)
        ctx.save_for_backward(x, w_gate, w_up, saved)
        ctx.act, ctx.sizes = act, sizes
        return out

    @staticmethod
    def _gradients(ctx, grad_out):
        x, w_gate, w_up, saved = ctx.saved_tensors
        # hooks on saved tensors, or a parameter whose data was exchanged, may bring back others
        half = (ctx.sizes[0] * ctx.sizes[1] + 3) // 4 * 4
        if _ffn_operands(x, w_gate, w_up) != ctx.sizes or saved.dtype != torch.float32 or saved.shape != (2 * half,):
            raise ValueError("the operands of the backward pass are not those of the forward pass")
        grad_out = grad_out.contiguous()
        if grad_out.data_ptr() % 16:                 # a slice of a larger gradient may start anywhere
            grad_out = grad_out.clone()
        _require_cuda(x, saved, grad_out)
        return (*_launch_ffn_backward(x, w_gate, w_up, _ptr(saved), _ptr(saved) + 2 * saved.numel(),
                                      grad_out, ctx.act, ctx.sizes, ctx.needs_input_grad[:3], None),
                None)

    _once = staticmethod(torch.autograd.function.once_differentiable(_gradients.__func__))

    @staticmethod
    def backward(ctx, grad_out):
        # only a backward pass that builds a graph needs the guard against a second derivative
        return (GatedFfn._once if torch.is_grad_enabled() else GatedFfn._gradients)(ctx, grad_out)
