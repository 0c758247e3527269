"""The 8-bit feed-forward path in 64 bits, from its definitions (no library code)."""
import torch

MIN = 2.0 ** -96


def up(n, to):
    return -(-n // to) * to


def round_e4m3(v):
    """Nearest e4m3 number (ties to the even one), saturated at 448."""
    e = torch.frexp(v)[1].clamp_min(-5) - 4
    step = torch.ldexp(torch.ones_like(v), e)
    return (torch.round(v / step) * step).clamp(-448, 448)


def expand(s, block_rows, rows, cols):
    return s.repeat_interleave(block_rows, 0)[:rows].repeat_interleave(128, 1)[:, :cols]


def blocks(v, block_rows):
    """(quotients 448 v / m, scales m / 448) of a 64-bit matrix."""
    r, c = v.shape
    p = torch.nn.functional.pad(v.abs(), (0, up(c, 128) - c, 0, up(r, block_rows) - r))
    m = p.view(p.shape[0] // block_rows, block_rows, -1, 128).amax((1, 3)).clamp_min(MIN)
    return v * 448 / expand(m, block_rows, r, c), m / 448


def quantize(v, block_rows=1):
    quot, s = blocks(v, block_rows)
    return round_e4m3(quot), s


def values(q, s, block_rows=1):
    return q.double() * expand(s.double(), block_rows, *q.shape)


def transposed(v, block_rows=1):
    t = v.t()
    t = torch.nn.functional.pad(t, (0, up(t.shape[1], 16) - t.shape[1]))
    return quantize(t, block_rows)


def norm(h, w, eps):
    rstd = 1 / torch.sqrt((h * h).mean(-1) + eps)
    return h * rstd[:, None] * w, rstd
