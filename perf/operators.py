"""Cases, plain forms and exact values of the library's 8-bit feed-forward path.

Six operators, which a pre-norm Reformer layer runs around its LSH attention:

* ``norm``       h = x + r, y = w h / sqrt(mean(h^2) + eps), y rounded to f32, bf16 or e4m3 with a
                 scale for each 128 columns of a row;
* ``norm_grad``  its gradients;
* ``quantize``   a matrix in e4m3 with a scale for each 1 x 128 or 128 x 128 block, and the same
                 of its transpose;
* ``matmul``     C = A B^T + bias of two such matrices;
* ``matmul_grad``  its gradients, from the output's gradient in bf16;
* ``ffn``        residual addition, norm and feed-forward in 8 bits:
                 W2 q(max(0, W1 q(y) + b1)) + b2.

A block is scaled by s = m / 448, m its largest magnitude and 2^-96 at least, and holds
e4m3(448 v / m), rounded to nearest even; it stands for those values times s.

Where ``own`` is false, ``run`` computes the plain form in torch operations; where it is true, it
calls the library.
"""

import math

import torch

own = False

EPS = 1e-6
F8 = torch.float8_e4m3fn
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": F8}
BYTES = {"f32": 4, "bf16": 2, "e4m3": 1}


def up(n, to):
    return -(-n // to) * to


# --------------------------------------------------------------------------- cases

def listed():
    return [
        # one new token of a fp32 residual stream before an 8-bit product: latency
        {"name": "norm_one_token", "op": "norm", "rows": 1, "cols": 512, "x": "f32", "y": "e4m3",
         "residual": True},
        # a layer of the L = 65 536 workload (8 heads of 64)
        {"name": "norm_long", "op": "norm", "rows": 65536, "cols": 512, "x": "f32", "y": "e4m3",
         "residual": True},
        # a short fine-tuning batch, an odd number of positions
        {"name": "norm_grad_short", "op": "norm_grad", "rows": 333, "cols": 768, "x": "bf16",
         "y": "bf16", "residual": True},
        # a wide layer's gradients over a long sequence
        {"name": "norm_grad_long", "op": "norm_grad", "rows": 16384, "cols": 2048, "x": "f32",
         "y": "bf16", "residual": True},
        # a feed-forward weight after an optimiser step, for the forward and the backward product
        {"name": "quantize_weight", "op": "quantize", "rows": 2048, "cols": 512, "x": "f32",
         "block_rows": 128, "transposed": True},
        # an output gradient on its way into both gradient products
        {"name": "quantize_gradient", "op": "quantize", "rows": 16000, "cols": 2048, "x": "bf16",
         "block_rows": 1, "transposed": True},
        # single-token serving: the weight is read once
        {"name": "matmul_one_token", "op": "matmul", "M": 1, "N": 8192, "K": 2048, "y": "bf16",
         "bias": True},
        # a training batch, the last tile of positions ragged
        {"name": "matmul_batch", "op": "matmul", "M": 8000, "N": 4096, "K": 4096, "y": "bf16",
         "bias": True},
        # gradients of a small layer, ragged in all three sizes
        {"name": "matmul_grad_ragged", "op": "matmul_grad", "M": 1000, "N": 656, "K": 400,
         "y": "bf16"},
        # gradients of the 512 -> 2048 product over 16 384 positions
        {"name": "matmul_grad_long", "op": "matmul_grad", "M": 16384, "N": 2048, "K": 512,
         "y": "f32"},
        # the sublayer for a few sequences' newest tokens
        {"name": "ffn_four_tokens", "op": "ffn", "tokens": 4, "d_model": 512, "d_ff": 2048,
         "chunk": 128},
        # the benchmarked feed-forward workload: 65 536 positions in chunks of 8192
        {"name": "ffn_long", "op": "ffn", "tokens": 65536, "d_model": 512, "d_ff": 2048,
         "chunk": 8192},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _log16(rng, lo, hi):
    return max(16, _log(rng, lo, hi) // 16 * 16)


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "quantize", "matmul", "matmul_grad", "ffn"])
    if op in ("norm", "norm_grad"):
        cols = _log16(rng, 64, 8192)
        rows = _log(rng, 1, max(2, min(65536, (1 << 25) // cols)))
        x = rng.choice(["f32", "bf16"])
        y = rng.choice(["bf16", "e4m3", x]) if op == "norm" else rng.choice(["bf16", x])
        return {"op": op, "rows": rows, "cols": cols, "x": x, "y": y,
                "residual": rng.random() < 0.7}
    if op == "quantize":
        cols = _log16(rng, 64, 8192)
        rows = _log(rng, 1, max(2, min(65536, (1 << 25) // cols)))
        return {"op": op, "rows": rows, "cols": cols, "x": rng.choice(["f32", "bf16"]),
                "block_rows": rng.choice([1, 128]), "transposed": rng.random() < 0.6}
    if op == "matmul":
        n, k = _log16(rng, 64, 8192), _log16(rng, 64, 8192)
        m = _log(rng, 1, max(2, min(65536, 8000 * 4096 * 4096 // (n * k), (1 << 27) // max(n, k))))
        return {"op": op, "M": m, "N": n, "K": k, "y": rng.choice(["bf16", "f32"]),
                "bias": rng.random() < 0.5}
    if op == "matmul_grad":
        n, k = _log16(rng, 64, 8192), _log16(rng, 64, 8192)
        m = _log(rng, 1, max(2, min(32768, 8000 * 2048 * 2048 // (n * k), (1 << 26) // max(n, k))))
        return {"op": op, "M": m, "N": n, "K": k, "y": rng.choice(["bf16", "f32"])}
    d_model, d_ff = _log16(rng, 128, 2048), _log16(rng, 256, 8192)
    tokens = _log(rng, 1, max(2, min(65536, 65536 * 512 * 2048 // (d_model * d_ff),
                                     (1 << 27) // d_ff)))
    return {"op": op, "tokens": tokens, "d_model": d_model, "d_ff": d_ff,
            "chunk": rng.choice([128, 1024, 8192])}


# --------------------------------------------------------------------------- inputs

def _stream(g, rows, cols, dtype):
    """A residual stream: rows of differing size, a few columns far larger than the others, and
    now and then a row of padding that is all zero."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    x *= torch.exp(0.5 * torch.randn(cols, generator=g, device="cuda"))
    x *= 0.25 + 2 * torch.rand(rows, 1, generator=g, device="cuda")
    x *= (torch.rand(rows, 1, generator=g, device="cuda") > 0.01) | (rows < 8)
    return x.to(dtype)


def _scaled(x, block_rows=1):
    """The plain form of a matrix in e4m3: (codes, scales).  The quotient is taken in fp64: bf16
    values often fall on the border between two codes exactly, and fp32 would move them off it."""
    rows, cols = x.shape
    p = torch.nn.functional.pad(x.float(), (0, up(cols, 128) - cols, 0, up(rows, block_rows) - rows))
    p = p.view(p.shape[0] // block_rows, block_rows, p.shape[1] // 128, 128)
    m = p.abs().amax((1, 3)).clamp_min(2.0 ** -96)
    q = (p.double() * 448.0 / m.double()[:, None, :, None]).to(F8)
    return q.view(up(rows, block_rows), up(cols, 128))[:rows, :cols].contiguous(), m / 448.0


def _stands_for(q, s, block_rows=1):
    """The values of codes and their scales, fp32 (fp64 where the scales are)."""
    s = s.repeat_interleave(block_rows, 0)[:q.shape[0]]
    s = s.repeat_interleave(128, 1)[:, :q.shape[1]]
    return q.to(s.dtype) * s


def _plain_transposed(x, block_rows):
    """(codes, scales) of x^T, its rows filled up with zeros to a multiple of 16 columns."""
    t = torch.nn.functional.pad(x.t().float(), (0, up(x.shape[0], 16) - x.shape[0]))
    return _scaled(t, block_rows)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 13)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    new = lambda *s, t=torch.float32: torch.empty(*s, dtype=t, device="cuda")  # noqa: E731
    op, s = case["op"], {"case": dict(case), "buf": {}}
    if op in ("norm", "norm_grad"):
        rows, cols, xt, yt = case["rows"], case["cols"], TYPES[case["x"]], TYPES[case["y"]]
        s["X"] = _stream(g, rows, cols, xt)
        s["w"] = 1 + 0.2 * rnd(cols)
        if op == "norm":
            s["R"] = (0.5 * rnd(rows, cols)).bfloat16() if case["residual"] else None
            s["buf"] = {"Y": new(rows, cols, t=yt), "rstd": new(rows)}
            if case["residual"]:
                s["buf"]["H"] = new(rows, cols, t=xt)
            if yt == F8:
                s["buf"]["scales"] = new(rows, up(cols, 128) // 128)
        else:
            s["dY"] = rnd(rows, cols).to(yt)
            s["dH"] = rnd(rows, cols).to(xt) if case["residual"] else None
            s["rstd"] = torch.rsqrt(s["X"].float().square().mean(1) + EPS)
            s["buf"] = {"dX": new(rows, cols, t=xt), "dw": new(cols)}
    elif op == "quantize":
        s["X"] = _stream(g, case["rows"], case["cols"], TYPES[case["x"]])
    elif op == "matmul":
        M, N, K = case["M"], case["N"], case["K"]
        s["A"], s["sa"] = _scaled(_stream(g, M, K, torch.float32))
        s["B"], s["sb"] = _scaled(rnd(N, K) / math.sqrt(K), 128)
        s["bias"] = rnd(N).bfloat16() if case["bias"] else None
        s["buf"] = {"C": new(M, N, t=TYPES[case["y"]])}
    elif op == "matmul_grad":
        M, N, K = case["M"], case["N"], case["K"]
        s["A"] = _stream(g, M, K, torch.bfloat16)
        s["dC"] = (rnd(M, N) * (0.1 + torch.rand(M, 1, generator=g, device="cuda"))).bfloat16()
        s["Bt"], s["st"] = _scaled((rnd(N, K) / math.sqrt(K)).t(), 128)
    else:
        T, D, F = case["tokens"], case["d_model"], case["d_ff"]
        s["X"], s["R"] = _stream(g, T, D, torch.float32), (0.5 * rnd(T, D)).bfloat16()
        s["w"] = 1 + 0.2 * rnd(D)
        s["W1"], s["s1"] = _scaled(rnd(F, D) / math.sqrt(D), 128)
        s["W2"], s["s2"] = _scaled(rnd(D, F) / math.sqrt(F), 128)
        s["b1"], s["b2"] = rnd(F).bfloat16(), rnd(D).bfloat16()
        s["buf"] = {"H": new(T, D), "Y8": new(T, D, t=F8), "scales": new(T, up(D, 128) // 128),
                    "Y": new(T, D, t=torch.bfloat16)}
    return s


# --------------------------------------------------------------------------- one pass

def _plain_norm(X, R, w):
    H = X if R is None else (X.float() + R.float()).to(X.dtype)
    h = H.float()
    rstd = torch.rsqrt(h.square().mean(1) + EPS)
    return H, h * rstd[:, None] * w, rstd


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op == "norm":
        H, y, rstd = _plain_norm(s["X"], s["R"], s["w"])
        out = {"rstd": rstd}
        if s["R"] is not None:
            out["H"] = H
        if c["y"] == "e4m3":
            out["Y"], out["scales"] = _scaled(y)
        else:
            out["Y"] = y.to(TYPES[c["y"]])
        return out
    if op == "norm_grad":
        n, rstd = s["X"].float() * s["rstd"][:, None], s["rstd"][:, None]
        dy = s["dY"].float()
        g = dy * s["w"]
        dx = rstd * (g - n * (g * n).mean(1, keepdim=True))
        if s["dH"] is not None:
            dx = dx + s["dH"].float()
        return {"dX": dx.to(s["X"].dtype), "dw": (dy * n).sum(0)}
    if op == "quantize":
        out = dict(zip(("Y", "scales"), _scaled(s["X"], c["block_rows"])))
        if c["transposed"]:
            out |= zip(("Yt", "scales_t"), _plain_transposed(s["X"], c["block_rows"]))
        return out
    if op == "matmul":
        C = _stands_for(s["A"], s["sa"]) @ _stands_for(s["B"], s["sb"], 128).t()
        return {"C": (C if s["bias"] is None else C + s["bias"].float()).to(TYPES[c["y"]])}
    if op == "matmul_grad":
        dc = _stands_for(*_scaled(s["dC"]))
        dct = _stands_for(*_plain_transposed(s["dC"], 1))
        at = _stands_for(*_plain_transposed(s["A"], 1))
        dA = dc @ _stands_for(s["Bt"], s["st"], 128).t()
        return {"dA": dA.to(TYPES[c["y"]]), "dB": dct @ at.t(), "db": s["dC"].float().sum(0)}
    H, y, _ = _plain_norm(s["X"], s["R"], s["w"])
    h = _stands_for(*_scaled(y)) @ _stands_for(s["W1"], s["s1"], 128).t() + s["b1"].float()
    h = _stands_for(*_scaled(h.clamp_min(0.0)))
    return {"H": H, "Y": (h @ _stands_for(s["W2"], s["s2"], 128).t() + s["b2"].float()).bfloat16()}


def _framework(s):
    import lsh_attention_long_b200 as L
    c, b = s["case"], s["buf"]
    op = c["op"]
    if op == "norm":
        L.lsh_rmsnorm_forward(s["X"], s["w"], R=s["R"], eps=EPS, out_dtype=TYPES[c["y"]], **b)
        return b
    if op == "norm_grad":
        L.lsh_rmsnorm_backward(s["dY"], s["X"], s["w"], s["rstd"], dH=s["dH"], **b)
        return b
    if op == "quantize":
        out = L.lsh_quantize_fp8(s["X"], block_rows=c["block_rows"], transposed=c["transposed"])
        return dict(zip(("Y", "scales", "Yt", "scales_t"), out))
    if op == "matmul":
        L.lsh_matmul_fp8(s["A"], s["sa"], s["B"], s["sb"], bias=s["bias"],
                         out_dtype=TYPES[c["y"]], **b)
        return b
    if op == "matmul_grad":
        out = L.lsh_matmul_fp8_backward(s["dC"], s["A"], s["Bt"], s["st"],
                                        out_dtype=TYPES[c["y"]])
        return dict(zip(("dA", "dB", "db"), out))
    L.lsh_rmsnorm_forward(s["X"], s["w"], R=s["R"], eps=EPS, out_dtype=F8, H=b["H"], Y=b["Y8"],
                          scales=b["scales"])
    L.lsh_ffn_forward_fp8(b["Y8"], b["scales"], s["W1"], s["s1"], s["b1"], s["W2"], s["s2"],
                          s["b2"], c["chunk"], Y=b["Y"])
    return {"H": b["H"], "Y": b["Y"]}


def run(state):
    return _framework(state) if own else _plain(state)


# --------------------------------------------------------------------------- floors

def work(case):
    op = case["op"]
    if op in ("norm", "norm_grad"):
        n, x, y = case["rows"] * case["cols"], BYTES[case["x"]], BYTES[case["y"]]
        if op == "norm":
            b = n * (x + y + ((2 + x) if case["residual"] else 0)) + 4 * case["rows"]
            if case["y"] == "e4m3":
                b += 4 * case["rows"] * up(case["cols"], 128) // 128
            return {"bytes": b + 4 * case["cols"], "flops": 5 * n}
        b = n * (2 * x + y + (x if case["residual"] else 0)) + 4 * case["rows"] + 8 * case["cols"]
        return {"bytes": b, "flops": 9 * n}
    if op == "quantize":
        r, c, br = case["rows"], case["cols"], case["block_rows"]
        b = r * c * (BYTES[case["x"]] + 1) + 4 * (up(r, br) // br) * (up(c, 128) // 128)
        if case["transposed"]:
            b += up(r, 16) * c + 4 * (up(c, br) // br) * (up(r, 128) // 128)
        return {"bytes": b, "flops": 2 * r * c * (2 if case["transposed"] else 1)}
    if op in ("matmul", "matmul_grad"):
        M, N, K = case["M"], case["N"], case["K"]
        blocks = (up(N, 128) // 128) * (up(K, 128) // 128)
        if op == "matmul":
            return {"bytes": M * K + N * K + M * N * BYTES[case["y"]]
                    + 4 * M * (up(K, 128) // 128) + 4 * blocks + (2 * N if case["bias"] else 0),
                    "flops": 2 * M * N * K}
        return {"bytes": 2 * M * N + 2 * M * K + N * K + 4 * blocks + M * K * BYTES[case["y"]]
                + 4 * N * K + 4 * N, "flops": 4 * M * N * K}
    T, D, F = case["tokens"], case["d_model"], case["d_ff"]
    return {"bytes": T * D * (4 + 2 + 4 + 2) + 2 * D * F + 8 * (up(D, 128) * up(F, 128) // 16384)
            + 2 * (D + F) + 4 * D, "flops": 4 * T * D * F}


# --------------------------------------------------------------------------- in 64 bits

def _round_e4m3(v):
    """The nearest of the numbers k 2^(e-3), 8 <= k < 16, e >= -6 (or k < 8, e = -6), ties to even
    k, at most 448 in magnitude."""
    e = torch.frexp(v)[1].clamp_min(-5) - 4
    step = torch.ldexp(torch.ones_like(v), e)
    return (torch.round(v / step) * step).clamp(-448, 448)


def _exact_scaled(v, block_rows=1):
    """codes and scales in fp64, block by block through a gather of each entry's block."""
    r, c = v.shape
    rb, cb = up(r, block_rows) // block_rows, up(c, 128) // 128
    m = torch.full((rb, cb), 2.0 ** -96, dtype=torch.float64, device=v.device)
    block = (torch.arange(r, device=v.device) // block_rows)[:, None] * cb \
        + (torch.arange(c, device=v.device) // 128)[None, :]
    m = m.view(-1).scatter_reduce(0, block.reshape(-1), v.abs().reshape(-1), "amax")
    return _round_e4m3(v * 448 / m[block]), (m / 448).view(rb, cb), block


def _exact_values(v, block_rows=1):
    q, s, block = _exact_scaled(v, block_rows)
    return q * s.view(-1)[block]


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    d = lambda t: t.to(torch.float64)  # noqa: E731
    if op in ("norm", "ffn"):
        h = d(s["X"])
        if s["R"] is not None:  # the sum is kept in the stream's type, and normalised as kept
            h = d((h + d(s["R"])).to(s["X"].dtype))
        rstd = 1 / torch.sqrt((h * h).sum(1) / h.shape[1] + EPS)
        y = torch.einsum("rc,r,c->rc", h, rstd, d(s["w"]))
    if op == "norm":
        out = {"rstd": rstd, "Y": y}
        if s["R"] is not None:
            out["H"] = h
        if case["y"] == "e4m3":
            out["Y"], out["scales"], _ = _exact_scaled(y)
        return out
    if op == "norm_grad":
        h, dy, r = d(s["X"]), d(s["dY"]), d(s["rstd"])
        g = torch.einsum("rc,c->rc", dy, d(s["w"]))
        inner = torch.einsum("rc,rc->r", g, h) / h.shape[1]
        dx = g * r[:, None] - h * (inner * r ** 3)[:, None]
        if s["dH"] is not None:
            dx = dx + d(s["dH"])
        return {"dX": dx, "dw": torch.einsum("rc,rc,r->c", dy, h, r)}
    if op == "quantize":
        out = {}
        out["Y"], out["scales"], _ = _exact_scaled(d(s["X"]), case["block_rows"])
        if case["transposed"]:
            t = d(s["X"]).t()
            t = torch.cat([t, t.new_zeros(t.shape[0], up(t.shape[1], 16) - t.shape[1])], 1)
            out["Yt"], out["scales_t"], _ = _exact_scaled(t, case["block_rows"])
        return out
    if op == "matmul":
        C = torch.einsum("mk,nk->mn", _stands_for(s["A"], d(s["sa"])),
                         _stands_for(s["B"], d(s["sb"]), 128))
        return {"C": C if s["bias"] is None else C + d(s["bias"])}
    if op == "matmul_grad":
        dc, a = d(s["dC"]), d(s["A"])
        dA = torch.einsum("mn,kn->mk", _exact_values(dc), _stands_for(s["Bt"], d(s["st"]), 128))
        dB = torch.einsum("nm,km->nk", _exact_values(dc.t()), _exact_values(a.t()))
        return {"dA": dA, "dB": dB, "db": dc.sum(0)}
    x = _exact_values(y)
    x = torch.einsum("td,fd->tf", x, _stands_for(s["W1"], d(s["s1"]), 128)) + d(s["b1"])
    x = _exact_values(torch.relu(x))
    return {"H": h, "Y": torch.einsum("tf,df->td", x, _stands_for(s["W2"], d(s["s2"]), 128))
            + d(s["b2"])}
