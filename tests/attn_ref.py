"""Plain fp64 restatement of fm_qk_norm_rope, fm_csa_attn and fm_csa_attn_tree
(the formulas of include/fm_index.h), with the error bounds the GPU results are
held to."""
import numpy as np

PAGE, D = 64, 512
HALF_BF16 = 2.0 ** -8  # a rounding to bf16 is off by at most this much of the value


def bf16(a):
    """fp32 -> bf16 bit patterns, round to nearest even (finite values)."""
    u = np.ascontiguousarray(a, np.float32).view(np.uint32).astype(np.uint64)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


def f64(bits):
    return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def freqs(rope_dim, base=160000.0, factor=16.0, orig=65536.0, fast=32.0, slow=1.0):
    out = []
    for i in range(rope_dim // 2):
        theta = base ** (-2.0 * i / rope_dim)
        g = min(1.0, max(0.0, (orig * theta / (2 * np.pi) - slow) / (fast - slow)))
        out.append((1 - g) * theta / factor + g * theta)
    return np.array(out)


def norm_rope(x, gain, pos, rope_dim, eps, **yarn):
    """x [T,h,d] fp64 -> (y, bound on |got - y|).  The fp32 steps (a sum of
    squares of at most 44 sequential additions, a reciprocal root, three
    products, an angle good to 2^-23 and its sine) are off by less than 2^-18 of
    the pair's size; then comes one rounding to bf16."""
    T, h, d = x.shape
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * (1.0 if gain is None else gain)
    size = np.abs(y)
    if rope_dim:
        a, b = y[..., d - rope_dim::2].copy(), y[..., d - rope_dim + 1::2].copy()
        ang = pos.astype(np.float64)[:, None] * freqs(rope_dim, **yarn)[None, :]
        c, s = np.cos(ang)[:, None, :], np.sin(ang)[:, None, :]
        y[..., d - rope_dim::2], y[..., d - rope_dim + 1::2] = a * c - b * s, a * s + b * c
        size[..., d - rope_dim::2] = size[..., d - rope_dim + 1::2] = np.abs(a) + np.abs(b)
    return y, HALF_BF16 * np.abs(y) * (1 + 2.0 ** -8) + 2.0 ** -18 * size + 2.0 ** -133


def visible(pos, window, n_sink, end):
    """Cached tokens that a token at `pos` sees among those below `end`."""
    return [j for j in range(max(0, min(end, pos + 1))) if j < n_sink or j > pos - window]


def attend(q, keys, sink, scale):
    """q [H,D], keys [n,D] -> out, lse and their error bounds.

    Scores: 512 products of bf16 values, exact in fp32, summed in fp32 in some
    order with at most one rounding or truncation (2^-23 of the running size)
    per addition: ds.  Weights: each is rounded once to bf16, and exp2 and the
    sums are off by less than 2^-16 together.  Output: one more rounding."""
    H = q.shape[0]
    out, lse = np.zeros((H, D)), np.full(H, -np.inf)
    tol, ltol = np.zeros((H, D)), np.zeros(H)
    if len(keys) == 0:
        return out, lse, tol, ltol
    s = scale * (q @ keys.T)
    ds = (512 * 2.0 ** -23 * scale * (np.abs(q) @ np.abs(keys).T)).max(1)
    m = s.max(1)
    w = np.exp(s - m[:, None])
    lse = m + np.log(w.sum(1))
    z = lse if sink is None else np.logaddexp(lse, sink)
    p = np.exp(s - z[:, None])
    out = p @ keys
    tol = HALF_BF16 * np.abs(out) * (1 + 2.0 ** -8) + (HALF_BF16 + 2 * ds + 2.0 ** -16)[:, None] * (p @ np.abs(keys)) + 1e-30
    ltol = ds + 2.0 ** -18 * (1 + np.abs(m) + np.abs(lse))
    return out, lse, tol, ltol
