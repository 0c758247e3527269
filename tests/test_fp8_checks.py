"""What the 8-bit feed-forward path refuses, before any launch: the binding (tensors of the wrong
shape, type or memory) and the C ABI (sizes, pointers, workspaces).  These run on the CPU."""
import ctypes

import pytest
import torch

import lsh_attention_long_b200 as L
from lsh_attention_long_b200 import build as B

F8, BF, F32 = torch.float8_e4m3fn, torch.bfloat16, torch.float32
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 4


def z(*shape, t=F32):
    return torch.zeros(*shape, dtype=t)


def test_norm_binding():
    X, w = z(4, 64), z(64)
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        L.lsh_rmsnorm_forward(X, w)
    for bad, msg in ((dict(R=z(4, 32)), "R has shape"), (dict(R=z(4, 64, t=torch.float16)), "R has dtype"),
                     (dict(out_dtype=torch.float16), "out_dtype"), (dict(H=z(4, 64)), "H is written"),
                     (dict(out_dtype=F8, scales=z(4, 2)), "scales has shape"),
                     (dict(Y=z(4, 64, t=BF)), "Y has dtype"), (dict(rstd=z(5)), "rstd has shape")):
        with pytest.raises(ValueError, match=msg):
            L.lsh_rmsnorm_forward(X, w, **bad)
    with pytest.raises(ValueError, match="X must be"):
        L.lsh_rmsnorm_forward(X.half(), w)
    with pytest.raises(ValueError, match="w has shape"):
        L.lsh_rmsnorm_forward(X, z(63))
    with pytest.raises(ValueError, match="contiguous"):
        L.lsh_rmsnorm_forward(z(64, 4).t(), w)
    with pytest.raises(ValueError, match="dH has dtype"):
        L.lsh_rmsnorm_backward(X, X, w, z(4), dH=X.bfloat16())
    with pytest.raises(ValueError, match="rstd has shape"):
        L.lsh_rmsnorm_backward(X, X, w, z(4, 1))


def test_quantizer_and_product_binding():
    X = z(32, 64)
    with pytest.raises(ValueError, match="block_rows"):
        L.lsh_quantize_fp8(X, block_rows=64)
    with pytest.raises(ValueError, match="written only with"):
        L.lsh_quantize_fp8(X, Yt=z(64, 32, t=F8))
    with pytest.raises(ValueError, match="X has dtype"):
        L.lsh_quantize_fp8(X.half())
    with pytest.raises(ValueError, match="must be a .rows, cols."):
        L.lsh_quantize_fp8(z(2, 3, 64))
    A, Bm, s = z(4, 256, t=F8), z(32, 256, t=F8), z(4, 2)
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        L.lsh_matmul_fp8(A, s, Bm, z(1, 2))
    for args, kw, msg in (((A, z(4, 1), Bm, z(1, 2)), {}, "a_scales has shape"),
                          ((A, s, Bm, z(2, 2)), {}, "b_scales has shape"),
                          ((A, s, z(32, 128, t=F8), z(1, 2)), {}, "B has shape"),
                          ((A, s, z(32, 256), z(1, 2)), {}, "B has dtype"),
                          ((A, s, Bm, z(1, 2)), {"bias": z(32)}, "bias has dtype"),
                          ((A, s, Bm, z(1, 2)), {"C": z(4, 32)}, "C has dtype"),
                          ((A, s, Bm, z(1, 2)), {"out_dtype": F8}, "out_dtype")):
        with pytest.raises(ValueError, match=msg):
            L.lsh_matmul_fp8(*args, **kw)
    with pytest.raises(ValueError, match="bt_scales has shape"):
        L.lsh_matmul_fp8_backward(z(4, 32, t=BF), z(4, 256, t=BF), z(256, 32, t=F8), z(1, 2))
    with pytest.raises(ValueError, match="dC has dtype"):
        L.lsh_matmul_fp8_backward(z(4, 32), z(4, 256, t=BF), z(256, 32, t=F8), z(2, 1))


def test_feed_forward_binding():
    X, s, W1, W2 = z(4, 64, t=F8), z(4, 1), z(128, 64, t=F8), z(64, 128, t=F8)
    b1, b2, one = z(128, t=BF), z(64, t=BF), z(1, 1)
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        L.lsh_ffn_forward_fp8(X, s, W1, one, b1, W2, one, b2, 128)
    with pytest.raises(ValueError, match="W2 has shape"):
        L.lsh_ffn_forward_fp8(X, s, W1, one, b1, W1, one, b2, 128)
    with pytest.raises(ValueError, match="x_scales has shape"):
        L.lsh_ffn_forward_fp8(X, z(3, 1), W1, one, b1, W2, one, b2, 128)
    with pytest.raises(ValueError, match="b1 has dtype"):
        L.lsh_ffn_forward_fp8(X, s, W1, one, b1.float(), W2, one, b2, 128)


def test_a_missing_tensor_is_named():
    """None where a tensor is needed (the norm gives no rstd unless asked) is refused by name."""
    X, w, A, Bm, s = z(4, 64), z(64), z(4, 256, t=F8), z(32, 256, t=F8), z(4, 2)
    dC, Ab, Bt = z(4, 32, t=BF), z(4, 256, t=BF), z(256, 32, t=F8)
    X8, W1, W2 = z(4, 64, t=F8), z(128, 64, t=F8), z(64, 128, t=F8)
    one, b1, b2 = z(1, 1), z(128, t=BF), z(64, t=BF)
    layer = [X8, z(4, 1), W1, one, b1, W2, one, b2]
    calls = [("rstd", lambda: L.lsh_rmsnorm_backward(X, X, w, None)),
             ("a_scales", lambda: L.lsh_matmul_fp8(A, None, Bm, z(1, 2))),
             ("b_scales", lambda: L.lsh_matmul_fp8(A, s, Bm, None)),
             ("Bt", lambda: L.lsh_matmul_fp8_backward(dC, Ab, None, z(2, 1))),
             ("bt_scales", lambda: L.lsh_matmul_fp8_backward(dC, Ab, Bt, None))]
    for i, name in enumerate(("x_scales", "W1", "w1_scales", "b1", "W2", "w2_scales", "b2"), 1):
        args = layer[:i] + [None] + layer[i + 1:]
        calls.append((name, lambda a=args: L.lsh_ffn_forward_fp8(*a, 128)))
    for name, call in calls:
        with pytest.raises(TypeError, match=f"^{name} must be a torch.Tensor"):
            call()
    for name, call in (("X", lambda: L.lsh_rmsnorm_forward(None, w)),
                       ("w", lambda: L.lsh_rmsnorm_forward(X, None)),
                       ("dY", lambda: L.lsh_rmsnorm_backward(None, X, w, z(4))),
                       ("H", lambda: L.lsh_rmsnorm_backward(X, None, w, z(4))),
                       ("X", lambda: L.lsh_quantize_fp8(None)),
                       ("B", lambda: L.lsh_matmul_fp8(A, s, None, s)),
                       ("X", lambda: L.lsh_ffn_forward_fp8(None, *layer[1:], 128))):
        with pytest.raises(ValueError, match=f"^{name} must be"):
            call()


def test_a_missing_tensor_is_named_on_the_device_too(monkeypatch):
    """The same where everything else fits: the library is not reached."""
    from lsh_attention_long_b200 import fp8

    class OnDevice(torch.Tensor):
        get_device = lambda self: 0  # noqa: E731
        is_cuda = property(lambda self: True)

    d = lambda *sh, t=F32: z(*sh, t=t).as_subclass(OnDevice)  # noqa: E731
    monkeypatch.setattr(fp8, "_lib", lambda: pytest.fail("reached the library"))
    for name, call in (("rstd", lambda: L.lsh_rmsnorm_backward(d(4, 64), d(4, 64), d(64), None)),
                       ("Bt", lambda: L.lsh_matmul_fp8_backward(d(4, 32, t=BF), d(4, 256, t=BF),
                                                                None, d(2, 1))),
                       ("bt_scales", lambda: L.lsh_matmul_fp8_backward(
                           d(4, 32, t=BF), d(4, 256, t=BF), d(256, 32, t=F8), None))):
        with pytest.raises(TypeError, match=f"^{name} must be a torch.Tensor"):
            call()


@pytest.fixture(scope="module")
def lib():
    B.build()
    return L.load_library()


P = ctypes.c_void_p(4096)  # never read: every call below ends before a launch


def test_norm_abi(lib):
    def fwd(rows=4, cols=64, x=0, r=1, w=0, y=2, X=P, R=P, W=P, eps=1e-6, H=P, Y=P, s=P):
        return lib.lsh_rmsnorm_forward(rows, cols, x, r, w, y, X, R, W, eps, H, Y, s, None, None)
    for kw in (dict(rows=-1), dict(cols=0), dict(x=2), dict(w=2), dict(y=3), dict(x=1, r=0),
               dict(X=None), dict(W=None), dict(Y=None), dict(H=None), dict(R=None), dict(s=None),
               dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
               dict(X=ctypes.c_void_p(4100)), dict(s=ctypes.c_void_p(4100))):
        assert fwd(**kw) == INVALID, kw
    assert fwd(cols=24) == UNSUPPORTED and fwd(cols=16400) == UNSUPPORTED
    assert fwd(rows=0, X=None) == OK

    def bwd(rows=4, cols=64, x=0, dy=1, w=0, dY=P, H=P, W=P, rstd=P, dX=P, dw=P, ws=P, n=1 << 30):
        return lib.lsh_rmsnorm_backward(rows, cols, x, dy, w, dY, H, W, rstd, None, dX, dw, ws, n,
                                        None)
    for kw in (dict(rows=-1), dict(x=2), dict(dy=2), dict(dY=None), dict(H=None), dict(rstd=None),
               dict(dX=None), dict(dw=None), dict(W=ctypes.c_void_p(4098))):
        assert bwd(**kw) == INVALID, kw
    assert bwd(cols=8) == UNSUPPORTED
    assert lib.lsh_rmsnorm_bwd_ws_size(4, 64) == 0          # one block: no partial sums
    need = lib.lsh_rmsnorm_bwd_ws_size(4096, 64)
    assert need > 0 and bwd(rows=4096, n=need - 1) == WORKSPACE
    assert bwd(rows=4096, ws=None) == WORKSPACE


def test_quantizer_abi(lib):
    def q(rows=4, cols=64, x=0, br=1, X=P, Y=P, s=P, Yt=None, st=None):
        return lib.lsh_quantize_fp8(rows, cols, x, br, X, Y, s, Yt, st, None)
    for kw in (dict(rows=-1), dict(cols=0), dict(x=2), dict(br=2), dict(X=None), dict(Y=None),
               dict(s=None), dict(Yt=P), dict(Y=ctypes.c_void_p(4104))):
        assert q(**kw) == INVALID, kw
    assert q(cols=40) == UNSUPPORTED
    assert q(rows=0, X=None, Y=None) == OK


def test_product_abi(lib):
    def mm(M=4, N=32, K=64, A=P, sa=P, Bm=P, sb=P, br=128, bias=None, c=1, C=P):
        return lib.lsh_matmul_fp8(M, N, K, A, sa, Bm, sb, br, bias, 0, c, C, None)
    for kw in (dict(M=-1), dict(N=0), dict(K=0), dict(br=64), dict(c=2), dict(A=None),
               dict(sa=None), dict(Bm=None), dict(sb=None), dict(C=None),
               dict(bias=ctypes.c_void_p(4098)), dict(A=ctypes.c_void_p(4104))):
        assert mm(**kw) == INVALID, kw
    assert mm(N=24) == UNSUPPORTED and mm(K=24) == UNSUPPORTED
    assert mm(M=0, A=None, C=None) == OK

    def bwd(M=4, N=32, K=64, dC=P, A=P, Bt=P, st=P, t=1, dA=P, dB=P, db=P, ws=P, n=1 << 40):
        return lib.lsh_matmul_fp8_backward(M, N, K, dC, A, Bt, st, t, dA, dB, db, ws, n, None)
    for kw in (dict(M=-1), dict(t=2), dict(dC=None), dict(Bt=None), dict(st=None), dict(A=None),
               dict(dA=None, dB=None, db=None), dict(dB=ctypes.c_void_p(4104))):
        assert bwd(**kw) == INVALID, kw
    assert bwd(N=8) == UNSUPPORTED
    need = lib.lsh_matmul_fp8_bwd_ws_size(4, 32, 64)
    assert bwd(n=need - 1) == WORKSPACE and bwd(ws=None) == WORKSPACE


def test_feed_forward_abi(lib):
    def ffn(T=4, D=64, F=128, chunk=128, X=P, Y=P, ws=P, n=1 << 40):
        return lib.lsh_ffn_forward_fp8(T, D, F, chunk, X, P, P, P, P, P, P, P, Y, ws, n, None)
    for kw in (dict(T=-1), dict(D=0), dict(F=0), dict(chunk=0), dict(X=None), dict(Y=None),
               dict(ws=ctypes.c_void_p(4104))):
        assert ffn(**kw) == INVALID, kw
    for kw in (dict(D=24), dict(F=24), dict(chunk=100)):
        assert ffn(**kw) == UNSUPPORTED, kw
    need = lib.lsh_ffn_fp8_ws_size(4, 64, 128, 128)
    assert need > 0 and ffn(n=need - 1) == WORKSPACE and ffn(ws=None) == WORKSPACE
    assert ffn(T=0, X=None, ws=None) == OK and lib.lsh_ffn_fp8_ws_size(0, 64, 128, 128) == 0
    # the hidden activation of two chunks of 32 MB, however many there are
    size = lib.lsh_ffn_fp8_ws_size
    assert size(128, 64, 128, 128) < 32768
    assert size(1 << 24, 64, 128, 128) == size(1 << 25, 64, 128, 128) <= 70 << 20
    # a longer chunk asked for: two of it, and no more than the positions there are
    assert size(1 << 25, 64, 128, 1 << 20) >= 2 * 128 << 20
    assert size(1000, 64, 128, 1 << 20) < 1 << 18


def test_sizes_beyond_whole_tiles_of_32_bits(lib):
    """Sizes whose tiles end past 2^31 are refused, not wrapped round."""
    for n in (2 ** 31 - 16, 2 ** 31 - 240):
        for M, N, K in ((n, 16, 16), (1, n, 16), (1, 16, n)):
            assert lib.lsh_matmul_fp8(M, N, K, P, P, P, P, 128, None, 0, 1, P, None) == UNSUPPORTED
            assert lib.lsh_matmul_fp8_bwd_ws_size(M, N, K) == 0
            assert lib.lsh_matmul_fp8_backward(M, N, K, P, P, P, P, 1, P, P, P, P, 1 << 62,
                                               None) == UNSUPPORTED
        assert lib.lsh_quantize_fp8(1, n, 1, 1, P, P, P, None, None, None) == UNSUPPORTED
        for T, D, F in ((n, 16, 16), (1, n, 16), (1, 16, n)):
            assert lib.lsh_ffn_fp8_ws_size(T, D, F, 128) == 0
            assert lib.lsh_ffn_forward_fp8(T, D, F, 128, *[P] * 10, 1 << 62, None) == UNSUPPORTED
    n = 2 ** 31 - 256
    assert lib.lsh_matmul_fp8_bwd_ws_size(n, 16, 16) > 4 * n
    assert lib.lsh_ffn_fp8_ws_size(n, 16, 16, 128) >= 32 << 20
