"""Python binding of the 8-bit feed-forward path of include/lsh.h: the norm
before a sublayer, e4m3 matrices with a scale per block of 128, their
products and the feed-forward made of them (argument marshalling only).

An 8-bit matrix is a pair (codes, scales): codes ``torch.float8_e4m3fn``
[rows, cols], scales fp32 [rows, ceil(cols / 128)] (1 x 128 blocks) or
[ceil(rows / 128), ceil(cols / 128)] (128 x 128 blocks).

Calls run on the tensors' device, on its current stream or on ``stream`` (what
a call allocates then belongs to that stream).
"""

from __future__ import annotations

import contextlib
from typing import Optional, Tuple

import torch

from . import lsh as _lsh
from .lsh import LSH_BF16, LSH_F32, LshError, _validate, load_library

LSH_E4M3 = 2
F8 = torch.float8_e4m3fn
_CODES = {torch.float32: LSH_F32, torch.bfloat16: LSH_BF16, F8: LSH_E4M3}
_FLOATS = (torch.float32, torch.bfloat16)
_HERE = contextlib.nullcontext()


def _up(n: int, to: int) -> int:
    return -(-n // to) * to


def _fits(t, shape, dtype, index: int) -> bool:
    """Whether t is a dense tensor of that shape and type on that device."""
    return (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape
            and t.get_device() == index and t.is_contiguous())


def _fits_if_given(t, shape, dtype, index: int) -> bool:
    return t is None or _fits(t, shape, dtype, index)


def _refuse(*specs, optional=()):
    """Reports what is wrong with (name, tensor, shape, dtype) entries, of
    which one at least does not fit (those of ``optional`` may be None)."""
    for name, t, _, _ in specs:
        if t is None:
            raise TypeError(f"{name} must be a torch.Tensor")
    _validate([(n, t, s, d, True) for n, t, s, d in (*specs, *optional)])
    raise ValueError("tensors must be on one CUDA device")


def _device(t, name: str) -> int:
    """The index of a tensor's CUDA device, -1 on the host."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    return t.get_device()


def _matrix(name: str, t, dtypes) -> Tuple[int, int]:
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError(f"{name} must be a [rows, cols] tensor")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} has dtype {t.dtype}, expected one of "
                         f"{', '.join(str(d) for d in dtypes)}")
    return t.shape


def _on(index: int, stream):
    """The context in which a call allocates and runs: the tensors' device and
    the stream asked for."""
    if stream is not None:
        if stream.device.index != index:
            raise ValueError(f"stream is on {stream.device}, expected cuda:{index}")
        return torch.cuda.stream(stream)
    return _HERE if index == _current_device() else torch.cuda.device(index)


_current_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") \
    else torch.cuda.current_device
_raw_stream = torch._C._cuda_getCurrentRawStream \
    if hasattr(torch._C, "_cuda_getCurrentRawStream") \
    else lambda index: torch.cuda.current_stream(index).cuda_stream


def _lib():
    return _lsh._lib or load_library()


def _done(name: str, rc: int) -> None:
    if rc != 0:
        raise LshError(name, rc)


def _p(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _scratch(name: str, sizes, ws, index: int):
    """(workspace, pointer, bytes): the caller's, or one of the size the library asks for."""
    if ws is None:
        n = getattr(_lib(), name)(*sizes)
        if n == 0:
            return None, None, 0
        ws = torch.empty(n, dtype=torch.uint8, device=index)
    elif not isinstance(ws, torch.Tensor) or ws.get_device() != index or not ws.is_contiguous():
        raise ValueError(f"ws must be a contiguous tensor on cuda:{index}")
    return ws, ws.data_ptr(), ws.numel() * ws.element_size()


def lsh_rmsnorm_forward(X, w, *, R=None, eps: float = 1e-6, out_dtype=None, H=None, Y=None,
                        scales=None, rstd=None, want_rstd: bool = False, stream=None):
    """H = X + R (X's type; X itself without R) and Y = H rsqrt(mean(H^2) + eps) w of every row
    of X [..., cols].  Returns (H, Y, scales, rstd): Y in ``out_dtype`` (X's type by default;
    ``torch.float8_e4m3fn`` gives 8 bits with 1 x 128 ``scales`` [rows, ceil(cols / 128)], else
    None), rstd fp32 [rows] where ``rstd`` is given or ``want_rstd`` (the backward needs it)."""
    if not isinstance(X, torch.Tensor) or X.dim() < 2 or X.dtype not in _FLOATS:
        raise ValueError("X must be a [..., cols] tensor of float32 or bfloat16")
    if not isinstance(w, torch.Tensor) or w.dtype not in _FLOATS:
        raise ValueError("w must be a [cols] tensor of float32 or bfloat16")
    shape, cols = X.shape, X.shape[-1]
    rows = X.numel() // cols if cols else 0
    yt = out_dtype or X.dtype
    if yt not in _CODES:
        raise ValueError(f"out_dtype {yt} is not float32, bfloat16 or float8_e4m3fn")
    rt = X.dtype
    if R is not None and isinstance(R, torch.Tensor) and R.dtype is torch.bfloat16:
        rt = torch.bfloat16
    if R is None and H is not None:
        raise ValueError("H is written only where R is given")
    f32 = torch.float32
    if yt is not F8:
        scales = None
    dev = _device(X, "X")
    try:  # spelt out: a call of one token costs little more than its checks
        fits = (dev >= 0
                and X.is_contiguous()
                and w.shape == (cols,) and w.get_device() == dev and w.is_contiguous()
                and (R is None or R.shape == shape and R.dtype is rt and R.get_device() == dev
                    and R.is_contiguous())
                and (H is None or H.shape == shape and H.dtype is X.dtype
                    and H.get_device() == dev and H.is_contiguous())
                and (Y is None or Y.shape == shape and Y.dtype is yt and Y.get_device() == dev
                    and Y.is_contiguous())
                and (scales is None or scales.shape == (rows, _up(cols, 128) // 128)
                    and scales.dtype is f32 and scales.get_device() == dev
                    and scales.is_contiguous())
                and (rstd is None or rstd.shape == (rows,) and rstd.dtype is f32
                    and rstd.get_device() == dev and rstd.is_contiguous()))
    except AttributeError:  # not a tensor
        fits = False
    if not fits:
        _refuse(("X", X, shape, X.dtype),
                ("w", w, (cols,), w.dtype),
                optional=(("R", R, shape, rt),
                          ("H", H, shape, X.dtype),
                          ("Y", Y, shape, yt),
                          ("scales", scales, (rows, _up(cols, 128) // 128), f32),
                          ("rstd", rstd, (rows,), f32)))
    with _on(dev, stream):
        if R is not None and H is None:
            H = torch.empty_like(X)
        if Y is None:
            Y = torch.empty_like(X, dtype=yt)
        if yt is F8 and scales is None:
            scales = X.new_empty((rows, _up(cols, 128) // 128), dtype=f32)
        if rstd is None and want_rstd:
            rstd = X.new_empty((rows,), dtype=f32)
        _done("lsh_rmsnorm_forward", _lib().lsh_rmsnorm_forward(
            rows, cols, _CODES[X.dtype], _CODES[rt], _CODES[w.dtype], _CODES[yt],
            X.data_ptr(), _p(R), w.data_ptr(), eps, _p(H), Y.data_ptr(), _p(scales),
            _p(rstd), _raw_stream(dev)))
    return X if R is None else H, Y, scales, rstd


def lsh_rmsnorm_backward(dY, H, w, rstd, *, dH=None, dX=None, dw=None, ws=None, stream=None):
    """Gradients of lsh_rmsnorm_forward: (dX in H's type, dw fp32).  H is the sum as normalised,
    dH the gradient that reaches it past the norm; dX is the gradient of X and of R alike."""
    if not isinstance(H, torch.Tensor) or H.dim() < 2 or H.dtype not in _FLOATS:
        raise ValueError("H must be a [..., cols] tensor of float32 or bfloat16")
    for name, t in (("w", w), ("dY", dY)):
        if not isinstance(t, torch.Tensor) or t.dtype not in _FLOATS:
            raise ValueError(f"{name} must be a tensor of float32 or bfloat16")
    shape, cols, f32 = H.shape, H.shape[-1], torch.float32
    rows = H.numel() // cols if cols else 0
    dev = _device(dY, "dY")
    if dev < 0 or not (
            _fits(dY, shape, dY.dtype, dev)
            and _fits(H, shape, H.dtype, dev)
            and _fits(w, (cols,), w.dtype, dev)
            and _fits(rstd, (rows,), f32, dev)
            and _fits_if_given(dH, shape, H.dtype, dev)
            and _fits_if_given(dX, shape, H.dtype, dev)
            and _fits_if_given(dw, (cols,), f32, dev)):
        _refuse(("dY", dY, shape, dY.dtype),
                ("H", H, shape, H.dtype),
                ("w", w, (cols,), w.dtype),
                ("rstd", rstd, (rows,), f32),
                optional=(("dH", dH, shape, H.dtype),
                          ("dX", dX, shape, H.dtype),
                          ("dw", dw, (cols,), f32)))
    with _on(dev, stream):
        if dX is None:
            dX = torch.empty_like(H)
        if dw is None:
            dw = H.new_empty((cols,), dtype=f32)
        ws, wp, wn = _scratch("lsh_rmsnorm_bwd_ws_size", (rows, cols), ws, dev)
        _done("lsh_rmsnorm_backward", _lib().lsh_rmsnorm_backward(
            rows, cols, _CODES[H.dtype], _CODES[dY.dtype], _CODES[w.dtype],
            dY.data_ptr(), H.data_ptr(), w.data_ptr(), rstd.data_ptr(), _p(dH),
            dX.data_ptr(), dw.data_ptr(), wp, wn, _raw_stream(dev)))
    return dX, dw


def lsh_quantize_fp8(X, *, block_rows: int = 1, transposed: bool = False, Y=None, scales=None,
                     Yt=None, scales_t=None, stream=None):
    """X [rows, cols] (fp32 or bf16) in 8 bits: (Y, scales), blocks of ``block_rows`` (1 or 128) x
    128; with ``transposed`` also (Yt, scales_t), the 8-bit form of X's transpose [cols, rows
    rounded up to a multiple of 16], its added columns zero."""
    rows, cols = _matrix("X", X, _FLOATS)
    if block_rows not in (1, 128):
        raise ValueError("block_rows must be 1 or 128")
    br, f32 = block_rows, torch.float32
    s_shape = (_up(rows, br) // br, _up(cols, 128) // 128)
    t_shape = (_up(cols, br) // br, _up(rows, 128) // 128)
    yt_shape = (cols, _up(rows, 16))
    if not transposed and (Yt is not None or scales_t is not None):
        raise ValueError("Yt and scales_t are written only with transposed=True")
    dev = _device(X, "X")
    if dev < 0 or not (
            _fits(X, (rows, cols), X.dtype, dev)
            and _fits_if_given(Y, (rows, cols), F8, dev)
            and _fits_if_given(scales, s_shape, f32, dev)
            and _fits_if_given(Yt, yt_shape, F8, dev)
            and _fits_if_given(scales_t, t_shape, f32, dev)):
        _refuse(("X", X, (rows, cols), X.dtype),
                optional=(("Y", Y, (rows, cols), F8),
                          ("scales", scales, s_shape, f32),
                          ("Yt", Yt, yt_shape, F8),
                          ("scales_t", scales_t, t_shape, f32)))
    with _on(dev, stream):
        if Y is None:
            Y = torch.empty_like(X, dtype=F8)
        if scales is None:
            scales = X.new_empty(s_shape, dtype=f32)
        if transposed:
            if Yt is None:
                Yt = X.new_empty(yt_shape, dtype=F8)
            if scales_t is None:
                scales_t = X.new_empty(t_shape, dtype=f32)
        _done("lsh_quantize_fp8", _lib().lsh_quantize_fp8(
            rows, cols, _CODES[X.dtype], br, X.data_ptr(), Y.data_ptr(),
            scales.data_ptr(), _p(Yt), _p(scales_t), _raw_stream(dev)))
    return (Y, scales, Yt, scales_t) if transposed else (Y, scales)


def lsh_matmul_fp8(A, a_scales, B, b_scales, *, bias=None, relu: bool = False,
                   out_dtype=torch.bfloat16, C=None, stream=None):
    """C [M, N] = A B^T (+ bias) (max(0, .) if ``relu``) of 8-bit matrices A [M, K] (1 x 128
    blocks) and B [N, K] (1 x 128 or 128 x 128 blocks, told by b_scales' shape), in fp32 or bf16."""
    M, K = _matrix("A", A, (F8,))
    N, Kb = _matrix("B", B, (F8,))
    if out_dtype not in _FLOATS:
        raise ValueError(f"out_dtype {out_dtype} is not float32 or bfloat16")
    kb, f32 = _up(K, 128) // 128, torch.float32
    rowwise = isinstance(b_scales, torch.Tensor) and N >= 16 and b_scales.shape == (N, kb)
    sb_shape = (N if rowwise else _up(N, 128) // 128, kb)
    dev = _device(A, "A")
    try:  # spelt out: a call of one token costs little more than its checks
        fits = (dev >= 0
                and A.shape == (M, K) and A.dtype is F8 and A.get_device() == dev
                and A.is_contiguous()
                and a_scales.shape == (M, kb) and a_scales.dtype is f32
                and a_scales.get_device() == dev and a_scales.is_contiguous()
                and B.shape == (N, K) and B.dtype is F8 and B.get_device() == dev
                and B.is_contiguous()
                and b_scales.shape == sb_shape and b_scales.dtype is f32
                and b_scales.get_device() == dev and b_scales.is_contiguous()
                and (bias is None or bias.shape == (N,) and bias.dtype is torch.bfloat16
                    and bias.get_device() == dev and bias.is_contiguous())
                and (C is None or C.shape == (M, N) and C.dtype is out_dtype
                    and C.get_device() == dev and C.is_contiguous()))
    except AttributeError:  # not a tensor
        fits = False
    if not fits:
        _refuse(("A", A, (M, K), F8),
                ("a_scales", a_scales, (M, kb), f32),
                ("B", B, (N, K), F8),
                ("b_scales", b_scales, sb_shape, f32),
                optional=(("bias", bias, (N,), torch.bfloat16),
                          ("C", C, (M, N), out_dtype)))
    with _on(dev, stream):
        if C is None:
            C = A.new_empty((M, N), dtype=out_dtype)
        _done("lsh_matmul_fp8", _lib().lsh_matmul_fp8(
            M, N, K, A.data_ptr(), a_scales.data_ptr(), B.data_ptr(),
            b_scales.data_ptr(), 1 if rowwise else 128, _p(bias), int(relu),
            _CODES[out_dtype], C.data_ptr(), _raw_stream(dev)))
    return C


def lsh_matmul_fp8_backward(dC, A, Bt, bt_scales, *, out_dtype=torch.bfloat16, dA=None, dB=None,
                            db=None, ws=None, stream=None):
    """Gradients of C = A B^T + bias (without relu), every product in 8 bits: (dA [M, K] in
    ``out_dtype``, dB [N, K] fp32, db [N] fp32).  dC and A (before quantisation) bf16; Bt [K, N]
    and bt_scales are B's transpose in 128 x 128 blocks, as lsh_quantize_fp8 gives it."""
    bf, f32 = torch.bfloat16, torch.float32
    M, N = _matrix("dC", dC, (bf,))
    K = _matrix("A", A, (bf,))[1]
    if out_dtype not in _FLOATS:
        raise ValueError(f"out_dtype {out_dtype} is not float32 or bfloat16")
    dev = _device(dC, "dC")
    if dev < 0 or not (
            _fits(dC, (M, N), bf, dev)
            and _fits(A, (M, K), bf, dev)
            and _fits(Bt, (K, N), F8, dev)
            and _fits(bt_scales, (_up(K, 128) // 128, _up(N, 128) // 128), f32, dev)
            and _fits_if_given(dA, (M, K), out_dtype, dev)
            and _fits_if_given(dB, (N, K), f32, dev)
            and _fits_if_given(db, (N,), f32, dev)):
        _refuse(("dC", dC, (M, N), bf),
                ("A", A, (M, K), bf),
                ("Bt", Bt, (K, N), F8),
                ("bt_scales", bt_scales, (_up(K, 128) // 128, _up(N, 128) // 128), f32),
                optional=(("dA", dA, (M, K), out_dtype),
                          ("dB", dB, (N, K), f32),
                          ("db", db, (N,), f32)))
    with _on(dev, stream):
        if dA is None:
            dA = torch.empty_like(A, dtype=out_dtype)
        if dB is None:
            dB = A.new_empty((N, K), dtype=f32)
        if db is None:
            db = A.new_empty((N,), dtype=f32)
        ws, wp, wn = _scratch("lsh_matmul_fp8_bwd_ws_size", (M, N, K), ws, dev)
        _done("lsh_matmul_fp8_backward", _lib().lsh_matmul_fp8_backward(
            M, N, K, dC.data_ptr(), A.data_ptr(), Bt.data_ptr(), bt_scales.data_ptr(),
            _CODES[out_dtype], dA.data_ptr(), dB.data_ptr(), db.data_ptr(), wp, wn,
            _raw_stream(dev)))
    return dA, dB, db


def ffn_fp8_workspace(tokens: int, d_model: int, d_ff: int, chunk: int, device) -> torch.Tensor:
    """Device scratch for lsh_ffn_forward_fp8: the hidden activation of two times ``chunk``
    positions, or of as many as take 32 MB each where that is more (and no more than there are)."""
    n = load_library().lsh_ffn_fp8_ws_size(tokens, d_model, d_ff, chunk)
    return torch.empty(max(n, 16), dtype=torch.uint8, device=device)


def lsh_ffn_forward_fp8(X, x_scales, W1, w1_scales, b1, W2, w2_scales, b2, chunk: int, *, Y=None,
                        ws=None, stream=None):
    """Chunked feed-forward in 8 bits: Y = W2 q(max(0, W1 x + b1)) + b2 (bf16) per position of X
    [..., d_model] (1 x 128 blocks, x_scales [tokens, ceil(d_model / 128)]; W1 [d_ff, d_model] and
    W2 [d_model, d_ff] in 128 x 128 blocks), `chunk` positions at a time, or as many as have a
    hidden activation of 32 MB."""
    if not isinstance(X, torch.Tensor) or X.dim() < 2:
        raise ValueError("X must be a [..., d_model] tensor")
    d_model, bf, f32 = X.shape[-1], torch.bfloat16, torch.float32
    tokens = X.numel() // d_model if d_model else 0
    d_ff = W1.shape[0] if isinstance(W1, torch.Tensor) and W1.dim() == 2 else -1
    mb, fb = _up(d_model, 128) // 128, _up(d_ff, 128) // 128
    dev = _device(X, "X")
    try:  # spelt out: a call of one token costs little more than its checks
        fits = (dev >= 0
                and X.dtype is F8 and X.is_contiguous()
                and x_scales.shape == (tokens, mb) and x_scales.dtype is f32
                and x_scales.get_device() == dev and x_scales.is_contiguous()
                and W1.shape == (d_ff, d_model) and W1.dtype is F8 and W1.get_device() == dev
                and W1.is_contiguous()
                and w1_scales.shape == (fb, mb) and w1_scales.dtype is f32
                and w1_scales.get_device() == dev and w1_scales.is_contiguous()
                and b1.shape == (d_ff,) and b1.dtype is bf and b1.get_device() == dev
                and b1.is_contiguous()
                and W2.shape == (d_model, d_ff) and W2.dtype is F8 and W2.get_device() == dev
                and W2.is_contiguous()
                and w2_scales.shape == (mb, fb) and w2_scales.dtype is f32
                and w2_scales.get_device() == dev and w2_scales.is_contiguous()
                and b2.shape == (d_model,) and b2.dtype is bf and b2.get_device() == dev
                and b2.is_contiguous()
                and (Y is None or Y.shape == X.shape and Y.dtype is bf
                    and Y.get_device() == dev and Y.is_contiguous()))
    except AttributeError:  # not a tensor
        fits = False
    if not fits:
        _refuse(("X", X, X.shape, F8),
                ("x_scales", x_scales, (tokens, mb), f32),
                ("W1", W1, (d_ff, d_model), F8),
                ("w1_scales", w1_scales, (fb, mb), f32),
                ("b1", b1, (d_ff,), bf),
                ("W2", W2, (d_model, d_ff), F8),
                ("w2_scales", w2_scales, (mb, fb), f32),
                ("b2", b2, (d_model,), bf),
                optional=(("Y", Y, X.shape, bf),))
    with _on(dev, stream):
        if Y is None:
            Y = torch.empty_like(X, dtype=bf)
        ws, wp, wn = _scratch("lsh_ffn_fp8_ws_size", (tokens, d_model, d_ff, chunk), ws, dev)
        _done("lsh_ffn_forward_fp8", _lib().lsh_ffn_forward_fp8(
            tokens, d_model, d_ff, chunk, X.data_ptr(), x_scales.data_ptr(),
            W1.data_ptr(), w1_scales.data_ptr(), b1.data_ptr(), W2.data_ptr(),
            w2_scales.data_ptr(), b2.data_ptr(), Y.data_ptr(), wp, wn,
            _raw_stream(dev)))
    return Y
