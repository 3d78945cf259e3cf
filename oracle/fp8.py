"""CPU oracle: FP8 rows and weights (E4M3 codes, one scale per block of 128),
their product, the expert FFN over them, and the router's balance loss -- in
numpy and 64 bits, from the definitions.

TEST INFRASTRUCTURE ONLY.  Nothing in the product path imports this module.

E4M3 (FN): sign, 4 exponent bits with bias 7, 3 mantissa bits; exponent 0 is
subnormal (steps of 2^-9); 0x7F and 0xFF are NaN; the largest value is 448.
Of a block with values x_i: m = max(max |x_i|, 2^-100) without NaN, scale
m / 448, code nearest to 448 x_i / m, ties to the even code.
"""
from __future__ import annotations

import numpy as np

BLOCK = 128
MAX = 448.0
FLOOR = 2.0 ** -100


def blocks(n: int) -> int:
    return -(-n // BLOCK)


def e4m3_value(code: int) -> float:
    mag = code & 0x7F
    if mag == 0x7F:
        return float("nan")
    e, f = mag >> 3, mag & 7
    v = f * 2.0 ** -9 if e == 0 else (8 + f) * 2.0 ** (e - 10)
    return -v if code & 0x80 else v


TABLE = np.array([e4m3_value(c) for c in range(256)])
_MAGS = TABLE[:127]                                    # 0 .. 448, ascending


def encode(v: np.ndarray) -> np.ndarray:
    """Nearest code of each value (ties to the even code, saturating), by search in the table of magnitudes."""
    a = np.minimum(np.abs(v), MAX)
    hi = np.clip(np.searchsorted(_MAGS, np.nan_to_num(a)), 0, 126)
    lo = np.maximum(hi - 1, 0)
    d_lo, d_hi = a - _MAGS[lo], _MAGS[hi] - a
    code = np.where((d_hi < d_lo) | ((d_hi == d_lo) & (hi % 2 == 0)), hi, lo)
    code = np.where(np.isnan(v), 0x7F, code)
    return (code | np.where(np.signbit(v) & ~np.isnan(v), 0x80, 0)).astype(np.uint8)


def decode(codes: np.ndarray) -> np.ndarray:
    return TABLE[np.asarray(codes, np.uint8)]


def _top(part: np.ndarray) -> float:
    a = np.abs(part[~np.isnan(part)])
    return max(float(a.max()) if a.size else 0.0, FLOOR)


def quant_rows(x: np.ndarray):
    """[M, K] -> (codes uint8 [M, K], scales fp64 [M, ceil(K/128)], quotients fp64 [M, K])."""
    x = np.asarray(x, np.float64)
    M, K = x.shape
    scales, q = np.empty((M, blocks(K))), np.empty((M, K))
    for b in range(blocks(K)):
        part = x[:, b * BLOCK:(b + 1) * BLOCK]
        top = np.array([_top(r) for r in part])
        with np.errstate(invalid="ignore"):
            q[:, b * BLOCK:(b + 1) * BLOCK] = MAX * part / top[:, None]
        scales[:, b] = top / MAX
    return encode(q), scales, q


def pack(w: np.ndarray):
    """[N, K] -> (codes uint8 [N, K], scales fp64 [ceil(N/128), ceil(K/128)])."""
    w = np.asarray(w, np.float64)
    N, K = w.shape
    codes, scales = np.empty((N, K), np.uint8), np.empty((blocks(N), blocks(K)))
    for i in range(blocks(N)):
        for j in range(blocks(K)):
            at = (slice(i * BLOCK, (i + 1) * BLOCK), slice(j * BLOCK, (j + 1) * BLOCK))
            top = _top(w[at].reshape(-1))
            codes[at], scales[i, j] = encode(MAX * w[at] / top), top / MAX
    return codes, scales


def rows_value(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    return decode(codes) * np.repeat(np.asarray(scales, np.float64), BLOCK, axis=1)[:, :codes.shape[1]]


def weight_value(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    N, K = codes.shape
    s = np.repeat(np.repeat(np.asarray(scales, np.float64), BLOCK, axis=0)[:N], BLOCK, axis=1)[:, :K]
    return decode(codes) * s


def gemm_bound(a: np.ndarray, b: np.ndarray) -> np.ndarray:
    """How far an fp32 evaluation may be from a b^T: every term passes at most
    128 additions inside its block and one for each block after it, two
    roundings of the scales' product and its application; each of these loses at
    most 2^-23 (a truncated addition, a step) of the sum of magnitudes."""
    nb = blocks(a.shape[1])
    return (BLOCK + 2 * nb + 4) * 2.0 ** -23 * (np.abs(a) @ np.abs(b).T)


def ffn_rows(x: np.ndarray, gate, up, down):
    """One expert's FFN on rows x [n, H] (values): gate, up, down are (codes, scales).  Returns (out, bound) in
    fp64: bound is how far fp32 sums may move the result, the codes of h that sit near a tie counted with the
    step to the code they may become."""
    cx, sx, _ = quant_rows(x)
    xv = rows_value(cx, sx)
    g_w, u_w, d_w = (weight_value(*t) for t in (gate, up, down))
    g, u = xv @ g_w.T, xv @ u_w.T
    bg, bu = gemm_bound(xv, g_w), gemm_bound(xv, u_w)
    silu = g / (1.0 + np.exp(-g))
    h = silu * u
    # |silu'| <= 1.1; the exponential and the quotient are a few fp32 steps
    bh = 1.1 * bg * (np.abs(u) + bu) + np.abs(silu) * bu + 2.0 ** -19 * np.abs(h)
    ch, sh, q = quant_rows(h)
    spread = lambda s: np.repeat(s, BLOCK, axis=1)[:, :h.shape[1]]  # noqa: E731
    bm = np.stack([bh[:, b * BLOCK:(b + 1) * BLOCK].max(1) for b in range(blocks(h.shape[1]))], 1)   # of the maximum
    rel = bm / (MAX * sh) + 2.0 ** -23
    dq = (bh / spread(sh)) + np.abs(q) * spread(rel)
    hv = rows_value(ch, sh)
    move = np.maximum(np.abs(decode(encode(q + dq)) - decode(ch)), np.abs(decode(encode(q - dq)) - decode(ch)))
    bhv = move * spread(sh) + np.abs(hv) * spread(rel)
    out = hv @ d_w.T
    return out, gemm_bound(hv, d_w) + bhv @ np.abs(d_w).T


def balance(logits: np.ndarray, ids: np.ndarray, valid: np.ndarray, coef: float):
    """(counts, loss, dlogits for dloss = 1) of the balance loss, fp64."""
    T, E = logits.shape
    k = ids.shape[1]
    live = np.flatnonzero(valid)
    counts = np.bincount(ids[live].reshape(-1), minlength=E)
    d = np.zeros((T, E))
    if live.size == 0:
        return counts, 0.0, d
    z = np.asarray(logits, np.float64)[live]
    with np.errstate(invalid="ignore"):
        p = np.exp(z - z.max(1, keepdims=True))
    p[np.isneginf(z).all(1)] = 0.0
    s = p.sum(1, keepdims=True)
    p = np.divide(p, s, out=np.zeros_like(p), where=s != 0)
    n = live.size
    f = coef * E / (n * n * k)
    d[live] = f * p * (counts - (p * counts).sum(1, keepdims=True))
    return counts, f * float((counts * p.sum(0)).sum()), d


def weights_grad(ids: np.ndarray, w: np.ndarray, dw: np.ndarray, E: int) -> np.ndarray:
    """dlogits of the router's weights w = softmax of the selected logits."""
    w, dw = np.asarray(w, np.float64), np.asarray(dw, np.float64)
    mine = w * (dw - (w * dw).sum(1, keepdims=True))
    d = np.zeros((ids.shape[0], E))
    np.add.at(d, (np.arange(ids.shape[0])[:, None], ids), mine)
    return d
