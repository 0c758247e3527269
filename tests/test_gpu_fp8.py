"""The 8-bit feed-forward path on the GPU against its definitions in 64 bits.

Tolerances count roundings: half a step is 2^-24 (fp32), 2^-8 (bf16), 2^-4 (e4m3) of the value.
"""
import pytest
import torch

import fp8_reference as ref
import lsh_attention_long_b200 as L

pytestmark = pytest.mark.gpu

F32, BF, F8 = torch.float32, torch.bfloat16, torch.float8_e4m3fn
HALF = {F32: 2.0 ** -24, BF: 2.0 ** -8}
EPS = 1e-6
# rstd: at most 64 squares added in one thread, then 5 + 8 partial sums, the
# division, the addition of eps (fp32 each, halved by the root), and the root's
# own error of two units
RSTD = (64 + 13 + 2) * 2.0 ** -25 + 2.0 ** -22


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from lsh_attention_long_b200 import build
    build.build()
    L.load_library()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rnd(g, *shape, t=F32):
    return torch.randn(*shape, generator=g, device="cuda").to(t)


def ok():
    torch.cuda.synchronize()
    assert L.lsh_device_status() == 0


def close(got, want, tol, what=""):
    """|got - want| <= tol elementwise (tol a tensor or number), in 64 bits."""
    d = (got.double() - want).abs()
    bad = ~(d <= tol)
    assert not bad.any(), (what, int(bad.sum()), float(d[bad].max()))


def guarded(shape, t, fill=77):
    """A tensor with 256 bytes of `fill` on both sides, and a check that they are still there."""
    n = torch.empty(shape, dtype=t, device="meta").numel() * torch.empty((), dtype=t).element_size()
    raw = torch.full((n + 512,), fill, dtype=torch.uint8, device="cuda")
    def intact():
        assert bool((raw[:256] == fill).all()) and bool((raw[256 + n:] == fill).all())
    return raw[256:256 + n].view(t).view(shape), intact


# ------------------------------------------------------------------ norm

COLS = [16, 128, 144, 256, 272, 1008, 1024, 1040, 2048, 4112, 8208, 16384]


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("xt,rt,wt,yt", [(F32, BF, F32, F8), (BF, BF, BF, BF), (F32, None, BF, F32),
                                         (BF, None, F32, F8), (F32, F32, F32, BF)])
def test_norm(cols, xt, rt, wt, yt):
    g = gen(cols)
    for rows in (1, 37):
        X, w = rnd(g, rows, cols, t=xt), (1 + 0.2 * rnd(g, cols)).to(wt)
        X[rows // 2] = 0
        R = rnd(g, rows, cols, t=rt) if rt else None
        (Y, y_ok), (rstd, r_ok) = guarded((rows, cols), yt), guarded((rows,), F32)
        H, h_ok = guarded((rows, cols), xt)
        S, s_ok = guarded((rows, ref.up(cols, 128) // 128), F32)
        H, Y, S, rstd = L.lsh_rmsnorm_forward(X, w, R=R, eps=EPS, out_dtype=yt, Y=Y, rstd=rstd,
                                              H=None if R is None else H, scales=S)
        ok()
        for f in (y_ok, r_ok, h_ok, s_ok):
            f()
        h = X if R is None else (X.float() + R.float()).to(xt)
        assert torch.equal(H, h)
        y, r = ref.norm(h.double(), w.double(), EPS)
        close(rstd, r, RSTD * r, "rstd")
        rel = RSTD + 2 * 2.0 ** -24  # two products
        if yt is not F8:
            close(Y, y, (rel + HALF[yt] * (1 + rel)) * y.abs() + 1e-40, "Y")
            continue
        _, s = ref.blocks(y, 1)
        close(S, s, (rel + 2 * 2.0 ** -24) * s, "scales")
        got = ref.values(Y, S)
        # half a step of e4m3: 2^-4 of the value, or 2^-10 scales below 2^-6
        step = torch.maximum(y.abs() * 2.0 ** -4, ref.expand(s, 1, *y.shape) * 2.0 ** -10)
        close(got, y, step + 4 * rel * y.abs(), "Y")


def test_norm_in_place_and_three_dimensions():
    g = gen(1)
    X, R, w = rnd(g, 2, 9, 512), rnd(g, 2, 9, 512, t=BF), rnd(g, 512)
    H0, Y0, S0, r0 = L.lsh_rmsnorm_forward(X, w, R=R, out_dtype=F8, want_rstd=True)
    assert Y0.shape == X.shape and S0.shape == (18, 4) and r0.shape == (18,)
    H1, Y1, S1, _ = L.lsh_rmsnorm_forward(X, w, R=R, out_dtype=F8, H=X)
    ok()
    assert H1 is X and torch.equal(X, H0) and torch.equal(S0, S1)
    assert torch.equal(Y0.view(torch.uint8), Y1.view(torch.uint8))


def test_norm_of_what_is_not_finite_stays_in_its_row():
    X = rnd(gen(2), 4, 256)
    X[1, 3], X[2, 200] = float("nan"), float("inf")
    w = torch.ones(256, device="cuda")
    _, Y, _, rstd = L.lsh_rmsnorm_forward(X, w, want_rstd=True)
    _, Y8, S, _ = L.lsh_rmsnorm_forward(X, w, out_dtype=F8)
    ok()
    assert Y[1].isnan().all() and Y[2, 200].isnan() and not Y[0].isnan().any()
    v = ref.values(Y8, S)
    assert v[1].isnan().all() and v[2, 128:].isnan().all()
    assert not v[0].isnan().any() and not v[3].isnan().any()


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("xt,dyt,wt,with_dh", [(F32, BF, F32, True), (BF, BF, BF, False),
                                               (F32, F32, F32, False), (BF, F32, F32, True)])
def test_norm_gradients(cols, xt, dyt, wt, with_dh):
    for rows in (1, 8, 9, 700 if cols > 1024 else 5000):
        g = gen(cols + rows)
        h, dY = rnd(g, rows, cols, t=xt), rnd(g, rows, cols, t=dyt)
        w = (1 + 0.2 * rnd(g, cols)).to(wt)
        dH = rnd(g, rows, cols, t=xt) if with_dh else None
        rstd = torch.rsqrt(h.float().square().mean(1) + EPS)
        (dX, x_ok), (dw, w_ok) = guarded((rows, cols), xt), guarded((cols,), F32)
        L.lsh_rmsnorm_backward(dY, h, w, rstd, dH=dH, dX=dX, dw=dw)
        ok()
        x_ok(), w_ok()
        r = rstd.double()[:, None]
        n, gg = h.double() * r, dY.double() * w.double()
        want = r * (gg - n * (gg * n).mean(1, keepdim=True))
        # the mean adds up to 64 products in a thread and 13 partial sums; each
        # product has three roundings; then four more on the way to dX
        size = (r * (gg.abs() + n.abs() * (gg * n).abs().mean(1, keepdim=True)))
        tol = (64 + 13 + 3 + 5) * 2.0 ** -24 * size
        if dH is not None:
            want = want + dH.double()
            tol = tol + 2.0 ** -24 * (dH.double().abs() + size)
        close(dX, want, tol + HALF[xt] * (want.abs() + tol), "dX")
        # dw: a thread adds its rows in order (at most ceil(rows / blocks)), then warps, blocks
        parts = (dY.double() * n)
        close(dw, parts.sum(0), (rows / 100 + 100) * 2.0 ** -24 * parts.abs().sum(0) + 1e-30, "dw")


def test_norm_gradients_against_autograd_and_differences():
    """The closed form against autograd of the definition, and along a line against a central
    difference of it (64 bits, step 1e-5: error of the order 1e-10)."""
    g = gen(3)
    h, w, R = rnd(g, 5, 272), rnd(g, 272), rnd(g, 5, 272)
    f = lambda a, b: (ref.norm(a, b, EPS)[0] * R.double()).sum()  # noqa: E731
    a, b = h.double().requires_grad_(), w.double().requires_grad_()
    f(a, b).backward()
    _, _, _, rstd = L.lsh_rmsnorm_forward(h, w, eps=EPS, want_rstd=True)
    dX, dw = L.lsh_rmsnorm_backward(R, h, w, rstd)
    ok()
    close(dX, a.grad, 1e-5 * a.grad.abs().max(), "dX")   # 85 roundings of 2^-24: 5e-6
    close(dw, b.grad, 1e-5 * b.grad.abs().max(), "dw")
    da, db = rnd(g, 5, 272).double(), rnd(g, 272).double()
    t = 1e-5
    with torch.no_grad():
        slope = (f(a + t * da, b + t * db) - f(a - t * da, b - t * db)) / (2 * t)
    got = (dX.double() * da).sum() + (dw.double() * db).sum()
    size = (dX.double() * da).abs().sum() + (dw.double() * db).abs().sum()
    assert abs(float(got - slope)) <= 1e-5 * float(size)


# ------------------------------------------------------------------ quantiser

@pytest.mark.parametrize("rows,cols", [(1, 16), (5, 128), (127, 144), (128, 256), (129, 272),
                                       (333, 1040), (2000, 64)])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("t", [F32, BF])
def test_quantize(rows, cols, block_rows, t):
    g = gen(rows + cols)
    X = rnd(g, rows, cols) * torch.exp(2 * rnd(g, rows, 1))
    X[rows // 3] = 0
    X = X.to(t)
    rp = ref.up(rows, 16)
    (Y, a), (Yt, b) = guarded((rows, cols), F8), guarded((cols, rp), F8)
    s_shape = (ref.up(rows, block_rows) // block_rows, ref.up(cols, 128) // 128)
    t_shape = (ref.up(cols, block_rows) // block_rows, ref.up(rows, 128) // 128)
    (S, c), (St, d) = guarded(s_shape, F32), guarded(t_shape, F32)
    L.lsh_quantize_fp8(X, block_rows=block_rows, transposed=True, Y=Y, scales=S, Yt=Yt,
                       scales_t=St)
    Y1, S1 = L.lsh_quantize_fp8(X, block_rows=block_rows)
    ok()
    for f in (a, b, c, d):
        f()
    assert torch.equal(Y.view(torch.uint8), Y1.view(torch.uint8)) and torch.equal(S, S1)
    for got, s, (q, w) in ((Y, S, ref.quantize(X.double(), block_rows)),
                           (Yt, St, ref.transposed(X.double(), block_rows))):
        close(s, w, 2.0 ** -24 * w, "scales")  # one division
        if t is BF:
            assert torch.equal(got.double(), q)  # borders included
        else:  # the quotient in fp32: one code beside it where that near a border
            x = X.double()
            if got is Yt:
                x = torch.nn.functional.pad(x.t(), (0, rp - rows))
            quot, _ = ref.blocks(x, block_rows)
            lo = ref.round_e4m3(quot * (1 - 2.0 ** -21))
            hi = ref.round_e4m3(quot * (1 + 2.0 ** -21))
            assert bool(((got.double() == lo) | (got.double() == hi)).all())


def test_quantize_extremes():
    """Blocks of zeros, of the smallest numbers and of the largest, and blocks with an infinity or a
    NaN, which stand for NaN throughout and leave the others alone."""
    X = torch.zeros(8, 256, device="cuda")
    X[1, :128] = 1e-45
    X[2, :128] = 2.0 ** -96
    X[3] = 3.0e38
    X[4, 5], X[5, 130] = float("inf"), float("nan")
    X[6] = torch.linspace(-1, 1, 256, device="cuda")
    for t in (F32, BF):
        Y, S = L.lsh_quantize_fp8(X.to(t))
        Y2, S2, Yt2, St2 = L.lsh_quantize_fp8(X.to(t), block_rows=128, transposed=True)
        ok()
        v = ref.values(Y, S)
        assert (v[0] == 0).all() and (v[1] == 0).all()
        close(v[2, :128], torch.full((128,), 2.0 ** -96, dtype=torch.float64, device="cuda"),
              2.0 ** -96 * 2.0 ** -23)
        x3 = X.to(t)[3].double()
        close(v[3], x3, x3 * 2.0 ** -23)
        assert v[4, :128].isnan().all() and not v[4, 128:].isnan().any()
        assert v[5, 128:].isnan().all() and not v[5, :128].isnan().any()
        x6 = X.to(t)[6].double()
        close(v[6], x6, torch.maximum(x6.abs() * (2.0 ** -4 + 1e-6), S[6, 0].double() * 2.0 ** -10))
        assert ref.values(Y2, S2, 128).isnan().all()  # one block of 128 x 128 each
        assert ref.values(Yt2, St2, 128)[:, :8].isnan().all()


# ------------------------------------------------------------------ products

def codes(g, rows, cols, block_rows):
    x = rnd(g, rows, cols) * torch.exp(rnd(g, rows, 1))
    q, s = ref.quantize(x.double(), block_rows)
    return q.to(F8), s.float()


def product(a, b):
    """The product in 64 bits and the sum of the magnitudes of its terms."""
    return a @ b.t(), a.abs() @ b.abs().t()


def sum_tol(K):
    # 128 terms of a block and ceil(K / 128) blocks added in fp32, cut off
    # rather than rounded at worst (2^-23), and each block's two scales
    return (128 + ref.up(K, 128) // 128 + 4) * 2.0 ** -23


PRODUCTS = [(1, 16, 16), (1, 144, 272), (3, 512, 2048), (8, 4096, 128), (9, 256, 512), (16, 640, 1024),
            (17, 128, 400), (33, 2064, 144), (64, 512, 512), (100, 272, 656), (128, 256, 128),
            (129, 272, 1040), (200, 1024, 4096), (256, 512, 384), (1000, 656, 400),
            (2049, 528, 208),
            # pairs of CTAs on 256 x 256 tiles; K shared by 8, 4 and 2 CTAs; few rows, long K
            (2500, 1040, 400), (8200, 272, 128), (300, 640, 2064), (64, 4096, 3088),
            (256, 4096, 4112), (12, 512, 1040), (16, 272, 4096),
            # few rows, many blocks of 16 of B's
            (1, 9488, 656), (8, 4752, 400), (13, 4752, 1040), (16, 9488, 272)]


@pytest.mark.parametrize("M,N,K", PRODUCTS)
@pytest.mark.parametrize("b_rows", [1, 128])
def test_matmul(M, N, K, b_rows):
    g = gen(M + N + K)
    A, sa = codes(g, M, K, 1)
    B, sb = codes(g, N, K, b_rows)
    bias = rnd(g, N, t=BF)
    want, size = product(ref.values(A, sa), ref.values(B, sb, b_rows))
    for t, with_bias, relu in ((F32, False, False), (BF, True, True), (F32, True, True),
                               (BF, False, False)):
        C, intact = guarded((M, N), t)
        L.lsh_matmul_fp8(A, sa, B, sb, bias=bias if with_bias else None, relu=relu, out_dtype=t,
                         C=C)
        ok()
        intact()
        w, z = want, size
        if with_bias:
            w, z = w + bias.double(), z + bias.double().abs()
        if relu:
            w = w.clamp_min(0)
        tol = sum_tol(K) * z
        close(C, w, tol + HALF[t] * (w.abs() + tol), (t, with_bias, relu))


@pytest.mark.parametrize("M", [1, 40, 300])
def test_matmul_nan_stays_in_its_row_and_column(M):
    g = gen(4)
    A, sa = codes(g, M, 256, 1)
    B, sb = codes(g, 256, 256, 128)
    sa[0, 1] = float("nan")
    sb[1, 0] = float("nan")
    C = L.lsh_matmul_fp8(A, sa, B, sb, relu=True, bias=torch.zeros(256, dtype=BF, device="cuda"))
    ok()
    assert C[0].isnan().all() and C[:, 128:].isnan().all()
    assert not C[1:, :128].isnan().any()


@pytest.mark.parametrize("M,N,K", [(1, 16, 16), (40, 144, 272), (128, 256, 128), (1000, 656, 400),
                                   (4000, 512, 256)])
@pytest.mark.parametrize("t", [F32, BF])
def test_matmul_gradients(M, N, K, t):
    g = gen(M + N + K)
    dC, A = rnd(g, M, N, t=BF), rnd(g, M, K, t=BF)
    B = rnd(g, N, K)
    _, _, Bt, st = L.lsh_quantize_fp8(B, block_rows=128, transposed=True)
    (dA, a_ok), (dB, b_ok), (db, c_ok) = guarded((M, K), t), guarded((N, K), F32), guarded((N,), F32)
    L.lsh_matmul_fp8_backward(dC, A, Bt, st, out_dtype=t, dA=dA, dB=dB, db=db)
    ok()
    for f in (a_ok, b_ok, c_ok):
        f()
    # bf16 inputs: their codes are the definition's own; the scales one rounding off each
    q = lambda x: ref.values(*ref.quantize(x.double()))  # noqa: E731
    qt = lambda x: ref.values(*ref.transposed(x.double()))  # noqa: E731
    want, size = product(q(dC), ref.values(Bt, st, 128))
    tol = (sum_tol(N) + 2.0 ** -23) * size
    close(dA, want, tol + HALF[t] * (want.abs() + tol), "dA")
    want, size = product(qt(dC), qt(A))
    close(dB, want, (sum_tol(M) + 2.0 ** -23) * size, "dB")
    d = dC.double()
    close(db, d.sum(0), (128 + M / 128) * 2.0 ** -24 * d.abs().sum(0), "db")
    # against the gradient of the unquantised product: each operand is off by half a step,
    # 2^-4 of itself or, below 2^-6 of a scale, 2^-10 scales (entries are below 6)
    want, size = product(dC.double().t(), A.double().t())
    small = 2 * 2.0 ** -10 * (6 / 448) * 6 * M
    close(dB, want, 2.0 ** -3 * (1 + 2.0 ** -5) * size + 1.1 * small, "dB, unquantised")


# ------------------------------------------------------------------ feed-forward

def ffn_state(T, D, F, seed=0):
    g = gen(T + D + F + seed)
    s = {"X": rnd(g, T, D), "w": 1 + 0.1 * rnd(g, D), "b1": 0.3 * rnd(g, F), "b2": rnd(g, D)}
    s["b1"], s["b2"] = s["b1"].to(BF), s["b2"].to(BF)
    s["W1"], s["s1"] = L.lsh_quantize_fp8(rnd(g, F, D) / D ** 0.5, block_rows=128)
    s["W2"], s["s2"] = L.lsh_quantize_fp8(rnd(g, D, F) / F ** 0.5, block_rows=128)
    s["X8"], s["sx"] = L.lsh_quantize_fp8(s["X"])
    return s


def ffn(s, chunk, **kw):
    return L.lsh_ffn_forward_fp8(s["X8"], s["sx"], s["W1"], s["s1"], s["b1"], s["W2"], s["s2"],
                                 s["b2"], chunk, **kw)


@pytest.mark.parametrize("T,D,F,chunk", [(1, 16, 16, 128), (1, 512, 2048, 128), (4, 512, 2048, 128),
                                         (16, 272, 1040, 128), (17, 128, 400, 128),
                                         (129, 256, 512, 128), (300, 144, 656, 256),
                                         (1000, 512, 2048, 384), (2048, 768, 1024, 8192),
                                         (2500, 272, 1040, 8192), (12, 1040, 272, 128),
                                         (3, 272, 4752, 128), (16, 128, 9616, 128)])
def test_ffn(T, D, F, chunk):
    s = ffn_state(T, D, F)
    Y, intact = guarded((T, D), BF)
    ffn(s, chunk, Y=Y)
    ok()
    intact()
    W2 = ref.values(s["W2"], s["s2"], 128)
    h, size = product(ref.values(s["X8"], s["sx"]), ref.values(s["W1"], s["s1"], 128))
    h, size = h + s["b1"].double(), size + s["b1"].double().abs()
    rel1 = sum_tol(D)
    h = h.clamp_min(0)
    q = ref.values(*ref.quantize(h))
    want, size2 = product(q, W2)
    want, size2 = want + s["b2"].double(), size2 + s["b2"].double().abs()
    # the hidden sums are off by rel1 of their terms' magnitudes: by that much, over the
    # block's largest entry, relative to an entry's quotient; where a border between two
    # codes is that near, the code may be the next one
    quot, sc = ref.blocks(h, 1)
    off = rel1 * size / ref.expand(sc, 1, T, F)           # in units of the codes
    top = torch.nn.functional.pad(off, (0, ref.up(F, 128) - F)).view(T, -1, 128).amax(2)
    off = off + quot * ref.expand(top, 1, T, F) / 448     # the largest entry's own error
    move = (ref.round_e4m3(quot + off) - ref.round_e4m3(quot - off)).abs()
    move = (move + quot.abs() * ref.expand(top, 1, T, F) / 448) * ref.expand(sc, 1, T, F)
    tol = move @ W2.abs().t() + sum_tol(F) * size2
    close(Y, want, tol + HALF[BF] * (want.abs() + tol), "Y")


@pytest.mark.parametrize("T,D,F,chunk", [(9000, 64, 8208, 128), (20000, 128, 4112, 4096),
                                         (257, 64, 131088, 128)])  # the last chunk one position
def test_ffn_of_several_chunks(T, D, F, chunk):
    """Enough positions for three chunks and more, whose products overlap from launch to launch and
    take turns on two buffers: the same as each position's own row of one call on it alone, up to
    the order of fp32 sums, and the same bits on every run."""
    s = ffn_state(T, D, F)
    ws = L.ffn_fp8_workspace(T, D, F, chunk, torch.device("cuda"))
    assert T > 2 * max(chunk, (32 << 20) // F // 256 * 256)  # three chunks
    assert ws.numel() < 2.2 * (max(32 << 20, chunk * F) + (1 << 20))
    ws.fill_(0x7f)  # NaN wherever something is read before it is written
    first = ffn(s, chunk, ws=ws).clone()
    ok()
    assert not first.isnan().any()
    for _ in range(10):
        assert torch.equal(ffn(s, chunk, ws=ws), first)
    ok()
    rows = torch.cat([torch.arange(0, T, 97), torch.tensor([T - 1])]).cuda()
    part = dict(s, X8=s["X8"].view(torch.uint8)[rows].view(F8), sx=s["sx"][rows])
    alone = ffn(part, chunk).double()
    # a sum in another order may put a hidden entry on the next code: 2^-4 of it, one in
    # thousands; the outputs are of order one
    close(first[rows].double(), alone, 2 * HALF[BF] * alone.abs() + 2.0 ** -6, "rows alone")


# ------------------------------------------------------------------ together

def layer(s, buf):
    """One pre-norm feed-forward sublayer and the next norm, as a serving loop runs them."""
    H, Y8, S, _ = L.lsh_rmsnorm_forward(s["X"], s["w"], R=buf["R"], out_dtype=F8, H=buf["H"],
                                        Y=buf["Y8"], scales=buf["S"])
    Y = L.lsh_ffn_forward_fp8(Y8, S, s["W1"], s["s1"], s["b1"], s["W2"], s["s2"], s["b2"], 128,
                              Y=buf["Y"], ws=buf["ws"])
    return L.lsh_rmsnorm_forward(H, s["w"], R=Y, out_dtype=BF, H=buf["H2"], Y=buf["Z"])


def layer_buffers(T, D, F, seed):
    e = lambda *sh, t=F32: torch.empty(*sh, dtype=t, device="cuda")  # noqa: E731
    return {"R": rnd(gen(seed), T, D, t=BF), "H": e(T, D), "Y8": e(T, D, t=F8),
            "S": e(T, ref.up(D, 128) // 128), "Y": e(T, D, t=BF), "H2": e(T, D), "Z": e(T, D, t=BF),
            "ws": L.ffn_fp8_workspace(T, D, F, 128, torch.device("cuda"))}


@pytest.mark.parametrize("T", [1, 16, 200])
def test_layer_replays_from_two_graphs_that_share_a_workspace(T):
    """The sublayer captured twice with one workspace, the graphs replayed in turn on new inputs,
    against eager runs; and the same bits every time."""
    D, F = 512, 1040
    s, b1, b2 = ffn_state(T, D, F), layer_buffers(T, D, F, 5), layer_buffers(T, D, F, 6)
    b2["ws"] = b1["ws"]
    want = [layer(s, b)[1].clone() for b in (b1, b2)]
    ok()
    graphs = []
    for b in (b1, b2):
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            layer(s, b)
        torch.cuda.current_stream().wait_stream(side)
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            layer(s, b)
        graphs.append(gr)
    for _ in range(3):
        for gr, b, w in zip(graphs, (b1, b2), want):
            b["Z"].zero_()
            gr.replay()
            ok()
            assert torch.equal(b["Z"], w)
    s["X"].mul_(1.5)
    fresh = layer(s, layer_buffers(T, D, F, 5))[1].clone()
    graphs[0].replay()
    ok()
    assert torch.equal(b1["Z"], fresh)
    del graphs


@pytest.mark.parametrize("T", [2, 300])
def test_another_stream(T):
    """Calls on a given stream order with that stream alone, allocate on it, and leave the
    current one alone."""
    s = ffn_state(T, 256, 528)
    want = ffn(s, 128)
    g = gen(9)
    dC, A = rnd(g, T, 256, t=BF), rnd(g, T, 528, t=BF)
    _, _, Bt, st = L.lsh_quantize_fp8(rnd(g, 256, 528), block_rows=128, transposed=True)
    want_b = L.lsh_matmul_fp8_backward(dC, A, Bt, st)
    ok()
    side = torch.cuda.Stream()
    for _ in range(5):
        Y = ffn(s, 128, stream=side)
        b = L.lsh_matmul_fp8_backward(dC, A, Bt, st, stream=side)
        junk = [torch.full((1 << 20,), 3, dtype=torch.uint8, device="cuda") for _ in range(4)]
        side.synchronize()
        assert torch.equal(Y, want) and all(torch.equal(x, y) for x, y in zip(b, want_b))
        del junk
    ok()


def test_two_calls_at_once():
    """Feed-forwards of several chunks and products on two streams at the same time, each with its
    own workspace, give what they give alone."""
    T, D, F = 9000, 128, 4112
    states = [ffn_state(T, D, F, seed) for seed in (1, 2)]
    want = [ffn(s, 128) for s in states]
    few = [ffn(dict(s, X8=s["X8"][:3], sx=s["sx"][:3]), 128) for s in states]
    ok()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(5):
        for i, (s, st) in enumerate(zip(states, streams)):
            got[i].append((ffn(s, 128, stream=st),
                           ffn(dict(s, X8=s["X8"][:3], sx=s["sx"][:3]), 128, stream=st)))
    ok()
    for i in range(2):
        assert all(torch.equal(y, want[i]) and torch.equal(z, few[i]) for y, z in got[i])


@pytest.mark.parametrize("T", [1, 3, 16, 40, 300])
def test_inputs_written_just_before(T):
    """Every input put into 8 bits anew right before the call that reads it, without a pause
    between them: no product reads what was there before."""
    D, F = 256, 1040
    g = gen(T)
    b1, b2 = rnd(g, F, t=BF), rnd(g, D, t=BF)
    sets = [(rnd(g, T, D), rnd(g, F, D), rnd(g, D, F)) for _ in range(2)]
    e = lambda *sh, t=F32: torch.empty(*sh, dtype=t, device="cuda")  # noqa: E731
    x8, sx = e(T, D, t=F8), e(T, D // 128)
    w1, s1, w2, s2 = e(F, D, t=F8), e(9, 2), e(D, F, t=F8), e(2, 9)

    def run(X, W1, W2):
        L.lsh_quantize_fp8(X, Y=x8, scales=sx)
        L.lsh_quantize_fp8(W1, block_rows=128, Y=w1, scales=s1)
        L.lsh_quantize_fp8(W2, block_rows=128, Y=w2, scales=s2)
        Y = L.lsh_ffn_forward_fp8(x8, sx, w1, s1, b1, w2, s2, b2, 128)
        L.lsh_quantize_fp8(W1, block_rows=128, Y=w1, scales=s1)  # over what was just read
        return Y, L.lsh_matmul_fp8(x8, sx, w1, s1)

    want = []
    for t in sets:
        want.append([y.clone() for y in run(*t)])
        ok()
    assert not torch.equal(want[0][0], want[1][0])
    got = [run(*sets[i & 1]) for i in range(40)]
    ok()
    for i, ys in enumerate(got):
        assert all(torch.equal(y, w) for y, w in zip(ys, want[i & 1]))


def test_empty_calls():
    e = lambda *sh, t=F32: torch.empty(*sh, dtype=t, device="cuda")  # noqa: E731
    w = torch.ones(64, device="cuda")
    assert L.lsh_rmsnorm_forward(e(0, 64), w, R=e(0, 64))[1].shape == (0, 64)
    dX, dw = L.lsh_rmsnorm_backward(e(0, 64), e(0, 64), w, e(0))
    assert dX.shape == (0, 64) and bool((dw == 0).all())
    assert L.lsh_quantize_fp8(e(0, 64), transposed=True)[2].shape == (64, 0)
    B, sb = codes(gen(1), 64, 64, 128)
    assert L.lsh_matmul_fp8(e(0, 64, t=F8), e(0, 1), B, sb).shape == (0, 64)
    dA, dB, db = L.lsh_matmul_fp8_backward(e(0, 64, t=BF), e(0, 64, t=BF), B, sb)
    assert dA.shape == (0, 64) and bool((dB == 0).all()) and bool((db == 0).all())
    z = torch.zeros(64, dtype=BF, device="cuda")
    assert L.lsh_ffn_forward_fp8(e(0, 64, t=F8), e(0, 1), B, sb, z, B, sb, z, 128).shape == (0, 64)
    ok()


def test_repeated_calls_give_the_same_bits():
    s = ffn_state(777, 256, 528)
    g = gen(10)
    dC, A, h = rnd(g, 777, 256, t=BF), rnd(g, 777, 528, t=BF), rnd(g, 777, 256)
    _, _, Bt, st = L.lsh_quantize_fp8(rnd(g, 256, 528), block_rows=128, transposed=True)
    rstd = torch.rsqrt(h.square().mean(1) + EPS)
    first = None
    for _ in range(10):
        out = [ffn(s, 128), *L.lsh_matmul_fp8_backward(dC, A, Bt, st),
               *L.lsh_rmsnorm_backward(dC, h, s["w"], rstd)]
        first = first or out
        assert all(torch.equal(a, b) for a, b in zip(first, out))
    ok()


# ------------------------------------------------------------------ failure path, parts of calls

@pytest.mark.parametrize("M,N,K,b_rows", [(128, 256, 1040, 128),    # one CTA to a tile
                                          (300, 640, 2064, 1),      # a cluster sharing K
                                          (2500, 1040, 400, 128),   # a pair
                                          (2500, 1040, 400, 1)])
def test_product_waits_that_run_out_are_reported_and_recovered(M, N, K, b_rows):
    """With a limit of one cycle a wait that is not over at its first look gives up: the call reports
    it, unless none had to wait, and the next one is as before."""
    g = gen(M)
    A, sa = codes(g, M, K, 1)
    B, sb = codes(g, N, K, b_rows)
    want = L.lsh_matmul_fp8(A, sa, B, sb)
    ok()
    L.lsh_set_wait_test(-1, 1)
    try:
        got = L.lsh_matmul_fp8(A, sa, B, sb)
        status = L.lsh_device_status()
    finally:
        L.lsh_set_wait_test(-1, 0)
    assert status == 5 or (status == 0 and torch.equal(got, want))  # LSH_ERR_TIMEOUT
    assert torch.equal(L.lsh_matmul_fp8(A, sa, B, sb), want)
    ok()


def test_gradients_asked_for_one_by_one():
    """The library's own entry point leaves out what its caller does not ask for."""
    import ctypes
    lib = L.load_library()
    g = gen(11)
    M, N, K = 200, 144, 272
    dC, A = rnd(g, M, N, t=BF), rnd(g, M, K, t=BF)
    _, _, Bt, st = L.lsh_quantize_fp8(rnd(g, N, K), block_rows=128, transposed=True)
    want = L.lsh_matmul_fp8_backward(dC, A, Bt, st, out_dtype=F32)
    n = lib.lsh_matmul_fp8_bwd_ws_size(M, N, K)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    for which in (0, 1, 2):
        out = torch.full_like(want[which], float("nan"))
        p = [out.data_ptr() if i == which else None for i in range(3)]
        rc = lib.lsh_matmul_fp8_backward(
            M, N, K, dC.data_ptr(), A.data_ptr() if which == 1 else None,
            Bt.data_ptr() if which == 0 else None, st.data_ptr() if which == 0 else None, 0, *p,
            ws.data_ptr(), n, ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
        ok()
        assert rc == 0 and torch.equal(out, want[which])


@pytest.mark.parametrize("K", [16, 144, 400, 656])
@pytest.mark.parametrize("b_rows", [1, 128])
def test_pairs_of_ctas_that_leave_at_once(K, b_rows):
    """Products on pairs of CTAs whose last blocks of K are their only ones, again and again without
    a pause: a barrier's last arrival belongs to the grid that waits for it, not to the next one on
    the same SM."""
    g = gen(K)
    A, sa = codes(g, 2500, K, 1)
    B, sb = codes(g, 1040, K, b_rows)
    want, size = product(ref.values(A, sa), ref.values(B, sb, b_rows))
    first = L.lsh_matmul_fp8(A, sa, B, sb, out_dtype=F32)
    ok()
    close(first, want, sum_tol(K) * size + HALF[F32] * want.abs())
    outs = [torch.empty_like(first) for _ in range(4)]
    for _ in range(25):
        for C in outs:
            L.lsh_matmul_fp8(A, sa, B, sb, out_dtype=F32, C=C)
        ok()
        assert all(torch.equal(C, first) for C in outs)


@pytest.mark.parametrize("T,D,F,chunk", [(16000, 768, 8208, 128),   # pairs of CTAs throughout
                                         (16000, 64, 8208, 128),    # the output on single ones
                                         (645, 64, 131088, 128),    # the last step five positions
                                         (13, 256, 1040, 128)])     # one step, few rows
def test_feed_forward_of_what_was_written_just_before(T, D, F, chunk):
    """Five steps whose input, weights, scales and biases were all rewritten in place right before
    the call, by two sets in turn on the same buffers and workspace, eagerly and as a replayed
    graph: the same bits as with a synchronisation after every launch sequence."""
    g = gen(T + D)
    sets = [[rnd(g, T, D) * (1 + 3 * i), rnd(g, F, D) / D ** 0.5, rnd(g, D, F) / F ** 0.5,
             rnd(g, F, t=BF), rnd(g, D, t=BF)] for i in range(2)]
    now = [t.clone() for t in sets[0]]
    up128 = lambda n: ref.up(n, 128) // 128  # noqa: E731
    e = lambda *sh, t=F32: torch.empty(*sh, dtype=t, device="cuda")  # noqa: E731
    x8, sx = e(T, D, t=F8), e(T, up128(D))
    w1, s1, w2, s2 = e(F, D, t=F8), e(up128(F), up128(D)), e(D, F, t=F8), e(up128(D), up128(F))
    b1, b2 = e(F, t=BF), e(D, t=BF)
    Y = e(T, D, t=BF)
    ws = L.ffn_fp8_workspace(T, D, F, chunk, torch.device("cuda"))
    ws.fill_(0x7f)  # NaN wherever something is read before it is written

    def run(pause=lambda: None):
        b1.copy_(now[3])
        b2.copy_(now[4])
        L.lsh_quantize_fp8(now[0], Y=x8, scales=sx)
        L.lsh_quantize_fp8(now[1], block_rows=128, Y=w1, scales=s1)
        L.lsh_quantize_fp8(now[2], block_rows=128, Y=w2, scales=s2)
        pause()
        L.lsh_ffn_forward_fp8(x8, sx, w1, s1, b1, w2, s2, b2, chunk, Y=Y, ws=ws)
        pause()

    def use(i):
        for a, b in zip(now, sets[i]):
            a.copy_(b)

    want = []
    for i in range(2):
        use(i)
        ok()
        run(torch.cuda.synchronize)
        want.append(Y.clone())
    ok()
    assert not torch.equal(*want) and not want[0].isnan().any()
    got = []
    for i in range(12):
        use(i & 1)
        run()
        got.append(Y.clone())
    ok()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for i in range(12):
        use(i & 1)
        graph.replay()
        got.append(Y.clone())
    ok()
    assert all(torch.equal(y, want[i & 1]) for i, y in enumerate(got))
    del graph


def held(call, tile):
    """The device status after `call` with tile `tile` of each block withheld and a short limit, and
    the time until it was there."""
    import time
    L.lsh_set_wait_test(tile, 2_000_000)  # about 1 ms
    try:
        t0 = time.perf_counter()
        call()
        status = L.lsh_device_status()
        return status, time.perf_counter() - t0
    finally:
        L.lsh_set_wait_test(-1, 0)


@pytest.mark.parametrize("M,N,K,b_rows,tile", [
    (128, 256, 1040, 128, 0), (1000, 656, 400, 1, 0),       # one CTA to a tile
    (300, 640, 2064, 1, 0), (64, 512, 4096, 128, 0),        # clusters of 8 that share K
    (64, 4096, 3088, 128, 0), (256, 4096, 4112, 1, 0),      # of 4 and 2
    (2500, 1040, 400, 128, 0), (2500, 1040, 400, 1, 0),     # a pair
    (40, 19200, 128, 128, 1), (8200, 1040, 144, 128, 1),    # its second tile
    (8200, 1040, 2064, 1, 1)])
def test_product_whose_loads_stop_is_reported_and_recovered(M, N, K, b_rows, tile):
    g = gen(M + K)
    A, sa = codes(g, M, K, 1)
    B, sb = codes(g, N, K, b_rows)
    want = L.lsh_matmul_fp8(A, sa, B, sb)
    ok()
    for _ in range(2):
        status, seconds = held(lambda: L.lsh_matmul_fp8(A, sa, B, sb), tile)
        assert status == 5 and seconds < 1.0  # LSH_ERR_TIMEOUT, by the short limit
        assert torch.equal(L.lsh_matmul_fp8(A, sa, B, sb), want)
        ok()


@pytest.mark.parametrize("T,D,F,chunk", [(16000, 768, 8208, 128), (300, 144, 656, 256),
                                         (2048, 768, 1024, 8192)])
def test_feed_forward_whose_loads_stop_is_reported_and_recovered(T, D, F, chunk):
    s = ffn_state(T, D, F)
    want = ffn(s, chunk)
    ok()
    status, seconds = held(lambda: ffn(s, chunk), 0)
    assert status == 5 and seconds < 1.0
    assert torch.equal(ffn(s, chunk), want)
    ok()


def test_gradients_whose_loads_stop_are_reported_and_recovered():
    g = gen(12)
    dC, A = rnd(g, 1000, 656, t=BF), rnd(g, 1000, 400, t=BF)
    _, _, Bt, st = L.lsh_quantize_fp8(rnd(g, 656, 400), block_rows=128, transposed=True)
    want = L.lsh_matmul_fp8_backward(dC, A, Bt, st)
    ok()
    status, seconds = held(lambda: L.lsh_matmul_fp8_backward(dC, A, Bt, st), 0)
    assert status == 5 and seconds < 1.0
    assert all(torch.equal(a, b) for a, b in zip(L.lsh_matmul_fp8_backward(dC, A, Bt, st), want))
    ok()


@pytest.mark.parametrize("T,at_once", [(128, 1), (128, 7), (128, 16), (128, 128), (9600, 9600)])
def test_feed_forward_quantises_as_defined_where_quotients_are_borders(T, at_once):
    """Hidden entries M / 16 and M / 32, 128 <= M < 256, each such M being the largest of a block
    once: many quotients 448 v / m lie exactly between two codes, and have to go to the even one.
    W1 adds c and c' / 16 of two codes, which fp32 holds exactly; W2 hands the codes out."""
    eye = torch.eye(128, device="cuda")
    one = lambda *sh: torch.ones(*sh, device="cuda")  # noqa: E731
    W1 = torch.cat([eye, eye / 16], 1).to(F8)          # [128, 256], scales 1
    W2 = torch.cat([eye, torch.zeros_like(eye)]).to(F8)
    big = (torch.arange(T, device="cuda") % 128 + 128).double()
    M = (torch.arange(128, device="cuda") + 128).double().expand(T, 128).clone()
    half = torch.full_like(M, 0.5)
    M[:, 127], half[:, 127] = big, 1
    c = torch.div(M, 16, rounding_mode="floor")
    X = torch.cat([c * half, (M - 16 * c) * half], 1).to(F8)
    h = M / 16 * half
    q, s = ref.quantize(h)
    z = lambda n: torch.zeros(n, dtype=BF, device="cuda")  # noqa: E731
    for t in range(0, T, at_once):
        x = X.view(torch.uint8)[t:t + at_once].view(F8)
        Y = L.lsh_ffn_forward_fp8(x, one(len(x), 2), W1, one(1, 2), z(128), W2, one(2, 1), z(256),
                                  128)
        ok()
        # Y is a code times its scale within 2^-8 + 2^-22, codes are 2^-4 apart or more
        got = ref.round_e4m3(Y[:, :128].double() / s[t:t + at_once])
        assert torch.equal(got, q[t:t + at_once]) and not Y[:, 128:].any()


def near_borders(g, rows, cols):
    """fp32 entries whose quotients 448 v / m are a few units of their last place from a border
    between two codes, m being each 1 x 128 block's first entry and all of its column's."""
    m = (1 + torch.rand(cols // 128, generator=g)).repeat_interleave(128).expand(rows, cols)
    c = torch.randint(16, 32, (rows, cols), generator=g) | 1          # borders: odd, of five bits
    c = c * 2.0 ** torch.randint(-4, 4, (rows, cols), generator=g)    # 1 to 248
    v = (c.double() * m / 448).float()
    v = v.view(torch.int32) + torch.randint(-2, 3, (rows, cols), generator=g).int()
    v = v.view(torch.float32)
    v[:, ::128] = m[:, ::128]
    return torch.where(torch.rand(rows, cols, generator=g) < 0.5, v, -v).contiguous()


def off_by(quot, codes, d):
    """Codes that no quotient within d of the exact one (relative) has."""
    lo, hi = ref.round_e4m3(quot * (1 - d)), ref.round_e4m3(quot * (1 + d))
    return int(((codes != lo) & (codes != hi)).sum())


# the quotient to the last bit of an fp32: half a unit, and what the sum that is rounded once is
# off by itself, far below 2^-10 of that
ONCE = 2.0 ** -24 * (1 + 2.0 ** -10)


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("rows", [3, 640])
def test_quantize_fp32_next_to_borders(rows, block_rows):
    """Quotients are right to the last bit of an fp32; the product with a rounded inverse, the mistake
    planted in the oracle, is not."""
    cols = 1024
    host = near_borders(torch.Generator().manual_seed(rows), rows, cols)
    quot, s = ref.blocks(host.double(), block_rows)
    m = ref.expand(s, block_rows, rows, cols) * 448
    assert off_by(quot, ref.round_e4m3(quot.float().double()), ONCE) == 0
    assert off_by(quot, ref.round_e4m3((host * (448 / m.float())).double()), ONCE) > rows
    X = host.cuda()
    Y, S, Yt, St = L.lsh_quantize_fp8(X, block_rows=block_rows, transposed=True)
    Y1, S1 = L.lsh_quantize_fp8(X, block_rows=block_rows)
    ok()
    assert torch.equal(Y.view(torch.uint8), Y1.view(torch.uint8)) and torch.equal(S, S1)
    assert off_by(quot.cuda(), Y.double(), ONCE) == 0
    t = torch.nn.functional.pad(host.t().double(), (0, ref.up(rows, 16) - rows))
    assert off_by(ref.blocks(t, block_rows)[0].cuda(), Yt.double(), ONCE) == 0


@pytest.mark.parametrize("cols", [1024, 4096])
def test_norm_codes_next_to_borders(cols):
    """The norm's codes are those of its own fp32 output, quotients right to the last bit."""
    g = torch.Generator().manual_seed(cols)
    X = torch.randn(40, cols, generator=g).cuda()
    w = near_borders(g, 1, cols)[0].cuda() / X[0]
    _, y, _, _ = L.lsh_rmsnorm_forward(X, w)
    _, Y, S, _ = L.lsh_rmsnorm_forward(X, w, out_dtype=F8)
    ok()
    quot, s = ref.blocks(y.double(), 1)
    assert off_by(quot, Y.double(), ONCE) == 0
    close(S, s, 2.0 ** -24 * s)  # one division


@pytest.mark.parametrize("T,D,F", [(3, 256, 512), (16, 256, 512), (40, 256, 512), (2500, 256, 1040)])
def test_feed_forward_of_units_switched_off(T, D, F):
    """A bias of -inf switches a hidden unit off: max(0, -inf) is 0, whatever its block's largest
    entry.  The same bits as with a bias of -1e30, which does so as well."""
    s = ffn_state(T, D, F)
    off = torch.rand(F, generator=gen(1), device="cuda") < 0.3
    off[128:256] = True                                # a block of zeros
    s["b1"][:16] = torch.tensor([7, 14, 28, 1.75] * 4, device="cuda")  # blocks whose largest entry divides 448
    s["b1"][16:128] = 1
    s["W1"].view(torch.uint8)[:128] = 0
    off[:128:3] = True
    want = ffn(dict(s, b1=torch.where(off, -1e30, s["b1"].float()).to(BF)), 128)
    got = ffn(dict(s, b1=torch.where(off, -float("inf"), s["b1"].float()).to(BF)), 128)
    ok()
    assert not want.isnan().any() and torch.equal(got, want)
    # as numbers: what a 64-bit sum over the units that are left gives, within the codes' steps
    h = ref.values(s["X8"], s["sx"]) @ ref.values(s["W1"], s["s1"], 128).t() + s["b1"].double()
    h = h.clamp_min(0) * ~off
    W2 = ref.values(s["W2"], s["s2"], 128)
    exact = h @ W2.t() + s["b2"].double()
    top = torch.nn.functional.pad(h, (0, ref.up(F, 128) - F)).view(T, -1, 128).amax(2)
    # half a step of a code (2^-4 of the entry, or 2^-10 scales), the fp32 sums before it
    # moving an entry by far less than that again, and the output's rounding
    step = torch.maximum(h * 2.0 ** -4, ref.expand(top / 448, 1, T, F) * 2.0 ** -10)
    tol = 1.01 * (step @ W2.abs().t()) + 1e-3
    close(got, exact, tol + HALF[BF] * (exact.abs() + tol))
