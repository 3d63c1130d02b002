"""Oracle of the expert-grouped path and of the 4-bit format (fp64 NumPy).

Rows are grouped by expert; every product is written from its definition, one
group at a time.  Gradients are the formulas, which the oracle's own tests pin
against central differences of the forward functions."""

import numpy as np


# ----------------------------------------------------------------------------- dispatch
def plan(idx, n_groups):
    """idx [R, k] -> offsets [G + 1], pairs [R k] (-1 past the last group), pos [R k] (-1 skipped, -2 no group)."""
    flat = np.asarray(idx).reshape(-1)
    pairs = np.full(flat.size, -1, np.int32)
    pos = np.where(flat == -1, -1, -2).astype(np.int32)
    offsets = np.zeros(n_groups + 1, np.int32)
    at = 0
    for g in range(n_groups):
        offsets[g] = at
        for p in np.flatnonzero(flat == g):
            pairs[at] = p
            pos[p] = at
            at += 1
    offsets[n_groups] = at
    return offsets, pairs, pos


def gathered(x, src, src_div):
    """Rows x[src // src_div]; entries that name no row give zeros.  src None: x itself."""
    x = np.asarray(x, np.float64)
    if src is None:
        return x
    src = np.asarray(src, np.int64)
    row = np.where(src >= 0, src // src_div, -1)
    ok = (row >= 0) & (row < len(x))
    return np.where(ok[:, None], x[np.where(ok, row, 0)], 0.0) if len(x) else np.zeros((len(src), x.shape[1]))


def groups_of(offsets, rows):
    """[(group, begin, end)] with the offsets clamped to [0, rows]."""
    o = np.clip(np.asarray(offsets, np.int64), 0, rows)
    return [(g, int(o[g]), max(int(o[g]), int(o[g + 1]))) for g in range(len(o) - 1)]


# ----------------------------------------------------------------------------- products
def matmul(x, offsets, w, rows):
    """y [rows, n] = x W_g^T; NaN in rows of no group (which a call leaves alone)."""
    y = np.full((rows, w.shape[1]), np.nan)
    for g, b, e in groups_of(offsets, rows):
        y[b:e] = x[b:e] @ np.asarray(w[g], np.float64).T
    return y


def matmul_t(dy, offsets, w, rows):
    dx = np.full((rows, w.shape[2]), np.nan)
    for g, b, e in groups_of(offsets, rows):
        dx[b:e] = dy[b:e] @ np.asarray(w[g], np.float64)
    return dx


def wgrad(dy, x, offsets, n_groups):
    dw = np.zeros((n_groups, dy.shape[1], x.shape[1]))
    for g, b, e in groups_of(offsets, len(dy)):
        dw[g] = np.asarray(dy[b:e], np.float64).T @ x[b:e]
    return dw


def sigmoid(v):
    e = np.exp(-np.abs(v))
    return np.where(v >= 0, 1.0, e) / (1.0 + e)


def swiglu(pre):
    g, u = np.split(pre, 2, axis=1)
    return g * sigmoid(g) * u


def swiglu_grad(dh, pre):
    """Gradient of swiglu at pre = (g | u) for the output gradient dh."""
    g, u = np.split(np.asarray(pre, np.float64), 2, axis=1)
    s = sigmoid(g)
    return np.concatenate([dh * u * (s + g * s * (1.0 - s)), dh * g * s], axis=1)


# ----------------------------------------------------------------------------- combine
def combine(o, pos, wts, rows, top_k):
    """y[r] = sum_j wts[r, j] o[pos[r, j]]; -1 adds nothing, another place outside o makes the row NaN."""
    o = np.asarray(o, np.float64)
    pos = np.arange(rows * top_k) if pos is None else np.asarray(pos)
    pos = pos.reshape(rows, top_k)
    w = np.ones((rows, top_k)) if wts is None else np.asarray(wts, np.float64)
    y = np.zeros((rows, o.shape[1]))
    for r in range(rows):
        for j in range(top_k):
            p = pos[r, j]
            if 0 <= p < len(o):
                y[r] += w[r, j] * o[p]
            elif p != -1:
                y[r] = np.nan
    return y


def combine_grad(dy, o, pos, wts, top_k):
    """(d_o, d_wts): NaN in the rows of d_o that no pair names."""
    dy = np.asarray(dy, np.float64)
    o = np.asarray(o, np.float64)
    rows = len(dy)
    pos = (np.arange(rows * top_k) if pos is None else np.asarray(pos)).reshape(rows, top_k)
    w = np.ones((rows, top_k)) if wts is None else np.asarray(wts, np.float64)
    d_o, d_w = np.full(o.shape, np.nan), np.zeros((rows, top_k))
    for r in range(rows):
        for j in range(top_k):
            p = pos[r, j]
            if 0 <= p < len(o):
                d_o[p] = w[r, j] * dy[r]
                d_w[r, j] = dy[r] @ o[p]
            elif p != -1:
                d_w[r, j] = np.nan
    return d_o, d_w


# ----------------------------------------------------------------------------- 4-bit weights
def q4_quantise(w, group, zeros):
    """(codes [n, k] 0..15, scales [n, k / group] float16, zeros [n, k / group] or None), round to nearest, in fp32."""
    w = np.asarray(w, np.float32)
    n, k = w.shape
    g = w.reshape(n, k // group, group)
    lo, hi = np.minimum(g.min(2), np.float32(0)), np.maximum(g.max(2), np.float32(0))
    step = (hi - lo) / np.float32(15) if zeros else np.maximum(-lo, hi) / np.float32(7)
    d = np.minimum(step, np.float32(65504)).astype(np.float16)
    df = d.astype(np.float32)
    safe = np.where(df > 0, df, np.float32(1))
    z = np.clip(np.rint(-lo / safe), 0, 15) if zeros else np.full_like(df, 8)
    z = np.where(df > 0, z, np.float32(0 if zeros else 8))
    c = np.clip(np.rint(g / safe[..., None]) + z[..., None], 0, 15)
    c = np.where(df[..., None] > 0, c, z[..., None])
    return c.reshape(n, k).astype(np.int64), d, z.astype(np.int64) if zeros else None


def q4_values(codes, scales, zeros, group):
    """fp64 weights of codes [n, k]."""
    z = 8.0 if zeros is None else np.repeat(zeros.astype(np.float64), group, axis=1)
    return (codes - z) * np.repeat(np.asarray(scales).astype(np.float64), group, axis=1)


def q4_layout(codes, scales, zeros, group):
    """The packed arrays (bytes) of codes [n, k], one element at a time from the layout's definition."""
    n, k = codes.shape
    tn, tk = -(-n // 16), -(-k // 128)
    ng = tk * 128 // group
    word = np.zeros((tn, tk, 4, 16, 4), np.uint32)
    if zeros is None:
        word[:] = 0x88888888
    sc = np.zeros((tn, ng, 16), np.float16)
    zr = np.zeros((tn, ng, 16), np.uint8)
    for r in range(n):
        for c in range(k):
            i, q, e = c % 128 // 32, c % 32 // 8, c % 8
            v = int(word[r // 16, c // 128, q, r % 16, i])
            word[r // 16, c // 128, q, r % 16, i] = v & ~(15 << 4 * e) & 0xFFFFFFFF | int(codes[r, c]) << 4 * e
        for g in range(k // group):
            sc[r // 16, g, r % 16] = scales[r, g]
            if zeros is not None:
                zr[r // 16, g, r % 16] = zeros[r, g]
    return (word.view(np.uint8).reshape(-1), sc.view(np.uint8).reshape(-1),
            None if zeros is None else zr.reshape(-1))
