"""Plain fp64 restatement of fm_prompt_attn, fm_kv_append_fp8 and fm_kv_attn_fp8 (the
formulas of include/fm_index.h), with the error bounds the GPU results are held to."""
import numpy as np

import attn_ref as ref

PAGE, BLOCK, TOP = 64, 16, 448.0
HALF_BF16, HALF_FP16 = 2.0 ** -8, 2.0 ** -11


def e4m3_values():
    """Value of each of the 256 codes (OCP FP8 E4M3: bias 7, no infinities, S.1111.111 = NaN)."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    x = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    x[(c & 127) == 127] = np.nan
    return np.where(c >= 128, -x, x)


VALUES = e4m3_values()


def e4m3_codes(x):
    """Codes nearest to x (|x| <= 448), ties to even; NaN gives 0x7F."""
    grid = VALUES[:127]
    a = np.minimum(np.abs(np.nan_to_num(x)), TOP)
    i = np.minimum(np.searchsorted(grid, a, side="right") - 1, 125)
    down, up = a - grid[i], grid[i + 1] - a
    code = np.where((up < down) | ((up == down) & (i % 2 == 1)), i + 1, i)
    return np.where(np.isnan(x), 127, code | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def need_scale(amax):
    """The least power of two >= 2^-100 with amax <= 448 * need."""
    e = -100
    while amax > TOP * 2.0 ** e:
        e += 1
    return 2.0 ** e


def rotate(x, pos, rope_dim, **yarn):
    """x [T,h,d] fp64 turned by pos [T]."""
    y = x.copy()
    if rope_dim:
        s = x.shape[-1] - rope_dim
        ang = pos.astype(np.float64)[:, None] * ref.freqs(rope_dim, **yarn)[None, :]
        c, n = np.cos(ang)[:, None, :], np.sin(ang)[:, None, :]
        a, b = x[..., s::2], x[..., s + 1::2]
        y[..., s::2], y[..., s + 1::2] = a * c - b * n, a * n + b * c
    return y


def append(k, v, pools, scales, table, start, cu, rope_dim, **yarn):
    """pools (codes uint8), scales (fp32) of keys and values, changed in place.  Returns, for each of the
    two, a mask of the cells written and the fp64 values that the new ones are rounded from
    (x / scale, NaN where none)."""
    written, exact = [np.zeros(p.shape, bool) for p in pools], [np.full(p.shape, np.nan) for p in pools]
    for b in range(len(start)):
        n, s0 = int(cu[b + 1]) - int(cu[b]), int(start[b])
        if n <= 0 or s0 < 0:
            continue
        rows = slice(int(cu[b]), int(cu[b + 1]))
        pos = s0 + np.arange(n)
        for which, x in enumerate((rotate(k[rows], pos, rope_dim, **yarn), v[rows])):
            for j in range(s0 // BLOCK, (s0 + n - 1) // BLOCK + 1):
                at = j * BLOCK // PAGE
                if at >= table.shape[1] or table[b, at] < 0 or table[b, at] >= pools[0].shape[0]:
                    continue
                page, sub, r0 = table[b, at], j * BLOCK % PAGE // BLOCK, j * BLOCK % PAGE
                lo, hi = max(s0, j * BLOCK), min(s0 + n, (j + 1) * BLOCK)
                kept = lo - j * BLOCK
                for h in range(x.shape[1]):
                    y = x[lo - s0:hi - s0, h]
                    fin = np.abs(y[np.isfinite(y)])
                    need = need_scale(fin.max() if fin.size else 0.0)
                    if kept:
                        old = float(scales[which][page, h, sub])
                        if need > old:
                            c = pools[which][page, h, r0:r0 + kept]
                            pools[which][page, h, r0:r0 + kept] = e4m3_codes(VALUES[c] * (old / need))
                            written[which][page, h, r0:r0 + kept] = True
                        need = max(old, need)
                    scales[which][page, h, sub] = need
                    z = np.where(np.isfinite(y), y, np.nan) / need
                    pools[which][page, h, r0 + kept:r0 + kept + hi - lo] = e4m3_codes(z)
                    written[which][page, h, r0 + kept:r0 + kept + hi - lo] = True
                    exact[which][page, h, r0 + kept:r0 + kept + hi - lo] = z
    return written, exact


def attend(q, k, v, past, window, sink, scale, held=None, weight_step=HALF_BF16, codes=None):
    """q [n,H,d], k, v [m,K,d] fp64, query i at position past + i of the m keys -> out [n,H,d], lse [n,H] and
    the bounds on what a kernel's may be off.

    A score is a dot product of d terms in fp32 (off by at most (d + 8) 2^-24 sum|q||k| however it is summed)
    and goes through an exponential of its difference from the maximum (another 2^-22 of its
    size); sums of m weights in fp32 are off by m 2^-24.  A weight is rounded by weight_step, and the output to
    bf16.  codes (|v| / scale of block, and that scale): weights in fp16 have besides an absolute error
    of 2^-25 of the row's largest weight times scale."""
    n, H, d = q.shape
    m, K = k.shape[0], k.shape[1]
    G = H // K
    out, lse = np.zeros((n, H, d)), np.full((n, H), -np.inf)
    tol, ltol = np.zeros((n, H, d)), np.zeros((n, H))
    for i in range(n):
        p = past + i
        j = np.arange(max(0, p - window + 1), min(p + 1, m))
        if held is not None:
            j = j[held[j]]
        if not len(j):
            continue
        for h in range(H):
            kk, vv = k[j, h // G], v[j, h // G]
            s = kk @ q[i, h] * scale
            size = np.abs(kk) @ np.abs(q[i, h]) * scale
            top = s.max()
            w = np.exp(s - top)
            z = w.sum()
            lse[i, h] = top + np.log(z)
            zs = z + (np.exp(np.float64(sink[h]) - top) if sink is not None else 0.0)
            out[i, h] = (w / zs) @ vv
            # relative error of the weights that matter (a weight of e^-30 may be off by all of itself)
            some = s > top - 30
            rel = 2 * ((d + 8) * 2.0 ** -24 * size[some].max() + 2.0 ** -22 * np.abs(s[some]).max()) + 2.0 ** -20 + len(j) * 2.0 ** -24
            a = (w / zs) @ np.abs(vv)
            tol[i, h] = a * (2 * rel + weight_step) + HALF_BF16 * np.abs(out[i, h]) + 2.0 ** -120
            if codes is not None:
                size_j, scale_j = codes[0][j, h // G], codes[1][j, h // G]
                tol[i, h] += 2.0 ** -24 * (w / zs * scale_j).max() * size_j.sum(0)
            ltol[i, h] = 2 * rel + 2.0 ** -21 * (abs(lse[i, h]) + 1)
    return out, lse, tol, ltol
