"""Plain numpy forms of the KV-cache and attention calls, in 64 bits, for their tests.

Tolerances are worst-case rounding bounds, derived here and not from any run: u is half a
step of f32 (2^-24), h half a step of the tensor type (2^-11 f16, 2^-8 bf16, u for f32).
  score    a sum of D products in f32 is off by at most (D + 8) u * scale * sum |q k| (the 8
           covers the scales, the split of f32 operands, the multiplication by `scale`).
  weights  e^x of a score off by e is off by a factor within 1 +- 1.01 e; exp itself and the
           running maximum's rescaling add 16 u; their rounding to the 16-bit type adds h.
  sums     a sum of n terms in f32 adds n u in numerator and in denominator.
The output is then off by at most (2 (e + n u + 16 u) + h) * sum p |v| + h |out|, plus half
the smallest subnormal of the type.
"""
import numpy as np

U = 2.0 ** -24
HALF_STEP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 2.0 ** -149, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}


def page_bytes(tokens, dim):
    return tokens * (dim + dim // 8)


def unpack_row(page, tokens, dim, slot, is_v):
    """(codes int [D], scales f16 [D / 32]) of one slot of one head's page (uint8 [page bytes])."""
    nb = dim // 32
    base = (tokens * (dim // 2 + dim // 16)) if is_v else 0
    row = page[base + slot * dim // 2: base + (slot + 1) * dim // 2]
    codes = np.zeros(dim, np.int64)
    for e in range(dim):
        b, g, j = e // 32, e % 32 // 8, e % 8
        n = j // 2 + 4 * (j % 2)
        byte = row[(g * nb + b) * 4 + n // 2]
        codes[e] = (byte >> (4 * (n % 2))) & 15
    sc = page[base + tokens * dim // 2 + slot * 2 * nb: base + tokens * dim // 2 + (slot + 1) * 2 * nb]
    return codes, np.frombuffer(sc.tobytes(), np.float16)


def unpack_pages(pages, tokens, dim):
    """f64 K and V [pages][heads][tokens][D] of uint8 [pages][heads][page bytes]."""
    nb, half = dim // 32, tokens * (dim // 2 + dim // 16)
    e = np.arange(dim)
    b, g, j = e // 32, e % 32 // 8, e % 8
    n = j // 2 + 4 * (j % 2)
    out = []
    for base in (0, half):
        rows = pages[:, :, base:base + tokens * dim // 2].reshape(*pages.shape[:2], tokens, dim // 2)
        code = (rows[..., (g * nb + b) * 4 + n // 2] >> (4 * (n % 2))) & 15
        sc = np.ascontiguousarray(pages[:, :, base + tokens * dim // 2:base + half]).view(np.float16)
        sc = sc.reshape(*pages.shape[:2], tokens, nb).astype(np.float64)
        with np.errstate(invalid="ignore"):
            out.append((code.astype(np.float64) - 8) * sc[..., b])
    return out


def rotate(x, cs, style):
    """x f32 [n][heads][D], cs f32 [n][n_rot / 2][2]: the pairwise rotation, every f32 operation rounded."""
    y = x.copy()
    half = cs.shape[1]
    i = np.arange(half)
    lo, hi = (i, i + half) if style == "halves" else (2 * i, 2 * i + 1)
    a, b = x[..., lo], x[..., hi]
    c, s = cs[:, None, :, 0], cs[:, None, :, 1]
    y[..., lo] = a * c - b * s
    y[..., hi] = a * s + b * c
    return y


def rope_table(rows, n_rot, base=10000.0):
    a = np.arange(rows)[:, None] * base ** (-2.0 * np.arange(n_rot // 2) / n_rot)
    return np.stack([np.cos(a), np.sin(a)], -1).astype(np.float32)


def attend(q, k, v, scale, seen):
    """One head: q [n][D], k and v [t][D], seen bool [n][t], all f64 -> (out, sum p |v|, largest scale * sum |q k|)."""
    with np.errstate(invalid="ignore"):
        s = np.where(seen, (q @ np.where(seen.any(0)[:, None], k, 0).T) * scale, -np.inf)
    size = np.where(seen, (np.abs(q) @ np.abs(np.where(seen.any(0)[:, None], k, 0)).T) * abs(scale), 0.0)
    v = np.where(seen.any(0)[:, None], v, 0)
    if s.shape[1] == 0:
        z = np.zeros((q.shape[0], v.shape[1]))
        return z, z, np.zeros(q.shape[0])
    m = s.max(1, keepdims=True)
    p = np.exp(s - np.where(np.isfinite(m), m, 0))
    t = p.sum(1, keepdims=True)
    p = p / np.where(t == 0, 1, t)
    return p @ v, p @ np.abs(v), size.max(1)


def tolerance(dtype, out, absv, size, n, dim):
    h = HALF_STEP[dtype]
    e = 1.01 * (dim + 8) * U * size[:, None]
    extra = h if dtype != "f32" else 0.0
    return (2 * (e + n * U + 16 * U) + extra) * absv + h * np.abs(out) + TINY[dtype]
