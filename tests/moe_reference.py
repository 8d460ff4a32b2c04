"""64-bit references of the per-token weight choice, on the CPU, element by element of the
definitions, with the error bounds the tests hold the kernels to."""
import numpy as np

BLOCK = {"q4_K": 144, "q6_K": 210}


def dequantise(raw, fmt):
    """raw uint8 [..., K/256 * bytes] -> float64 [..., K]."""
    b = raw.reshape(*raw.shape[:-1], -1, BLOCK[fmt])
    k = np.arange(256)

    def half(x):
        return np.ascontiguousarray(x).view(np.float16).astype(np.float64)

    if fmt == "q4_K":
        j = k // 32
        q = (b[..., 16 + 32 * (j // 2) + k % 32] >> (4 * (j % 2))) & 15
        s, jj = b[..., 4:16].astype(np.int64), np.arange(8)
        low = s[..., jj % 4] & 63, s[..., 4 + jj % 4] & 63
        top = s[..., jj % 4] >> 6, s[..., 4 + jj % 4] >> 6
        last = s[..., 8 + jj % 4]
        sc = np.where(jj < 4, low[0], (last & 15) | (top[0] << 4))
        mn = np.where(jj < 4, low[1], (last >> 4) | (top[1] << 4))
        w = half(b[..., 0:2]) * (sc[..., j] * q) - half(b[..., 2:4]) * mn[..., j]
    else:
        h, r = k // 128, k % 128
        q = ((b[..., 64 * h + r % 64] >> (4 * (r // 64))) & 15).astype(np.int64)
        q |= ((b[..., 128 + 32 * h + r % 32] >> (2 * (r // 32))) & 3).astype(np.int64) << 4
        sc = b[..., 192:208].view(np.int8).astype(np.int64)[..., k // 16]
        w = half(b[..., 208:210]) * (sc * (q - 32))
    return w.reshape(*raw.shape[:-1], -1)


def route(logits, topk, renormalize):
    """(ids, weights) of float64 logits [N, E]."""
    N, E = logits.shape
    ids = np.full((N, topk), -1)
    weights = np.zeros((N, topk))
    for n, row in enumerate(logits):
        open_ = [e for e in range(E) if row[e] > -np.inf]
        best = sorted(open_, key=lambda e: (-row[e], e))[:topk]
        if not best:
            continue
        with np.errstate(invalid="ignore"):
            ex = np.exp(row[best] - row[best[0]])
            total = ex.sum() if renormalize else np.exp(row - row[best[0]]).sum()
            if np.isnan(row).any():
                total = np.nan
            ids[n, :len(best)] = best
            weights[n, :len(best)] = ex / total
    return ids, weights


def group(ids, groups):
    """(offsets, rows, pos) of ids [N, per_row]."""
    flat = ids.reshape(-1)
    key = np.where((flat < 0) | (flat >= groups), groups, flat)
    order = np.argsort(key, kind="stable")
    offsets = np.concatenate([[0], np.cumsum(np.bincount(key, minlength=groups + 1))])
    pos = np.empty(len(flat), np.int64)
    pos[order] = np.arange(len(flat))
    pos[key == groups] = -1
    return offsets, order // ids.shape[1], pos.reshape(ids.shape)


# Unit roundoff (8 and 11 significant bits): one rounding of a value, relative to it.
ROUND = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def experts(raw, fmt, X, ids, E, swiglu, gather, type):
    """(Y, bound) over the sorted items: raw uint8 [E, M, bytes], X float64, ids [N, per_row].

    The bound: one rounding of each weight to the type (a q4_K weight in binary16 as two terms
    that round: twice), f32 sums of K terms in any order (2^-24 of the sum of their sizes each
    for a chain of at most 256 + K / 256 of them), one rounding of the result; binary16 results
    and weights are also off by half of the smallest subnormal (weights are scaled by a power of
    two before, so for them it is 2^-37 of the row's largest possible weight)."""
    offsets, rows, _ = group(ids, E)
    items = ids.size
    M, K = raw.shape[1], X.shape[1]
    Y = np.zeros((items, M // 2 if swiglu else M))
    bound = np.zeros_like(Y)
    u = ROUND[type]
    per_weight = 2 * u + (256 + K / 256) * 2.0 ** -24
    tiny = 2.0 ** -25 if type == "f16" else 0.0
    for e in range(E):
        i = np.arange(offsets[e], offsets[e + 1])
        if not len(i):
            continue
        w = dequantise(raw[e], fmt)
        x = X[rows[i]] if gather else X[i]
        y, size = x @ w.T, np.abs(x) @ np.abs(w).T
        err = per_weight * size
        if fmt == "q4_K":     # the two terms of a weight cancel: their sizes count
            big = np.abs(x).sum(1, keepdims=True) * np.abs(w).max(1)
            err = err + per_weight * big
        if swiglu:
            h = M // 2
            g, up, eg, eu = y[:, :h], y[:, h:], err[:, :h], err[:, h:]
            with np.errstate(over="ignore"):
                silu = g / (1 + np.exp(-g))
            y = silu * up
            # silu's slope is below 1.1; its exponential and division add 2^-20
            err = 1.1 * eg * (np.abs(up) + eu) + np.abs(silu) * eu + 2.0 ** -20 * np.abs(y)
        Y[i] = y
        bound[i] = err * (1 + u) + u * np.abs(y) + tiny
    return Y, bound


def lora(Y, X, A, B, scale, ids):
    """(out, bound): all float64, ids [N] (-1: none). The bound: a remainder of 2^-21 lost from
    each of x and T, f32 sums (chains of at most 64 + K / 32 and r terms), one rounding of T's
    scaling and of the sum with Y."""
    out, bound = Y.copy(), np.zeros_like(Y)
    K, r = X.shape[1], A.shape[1]
    rel = 2 * 2.0 ** -21 + (64 + K / 32 + r + 8) * 2.0 ** -24
    for n, a in enumerate(ids):
        if a < 0 or a >= len(A):
            continue
        t = scale[a] * (A[a] @ X[n])
        size = np.abs(scale[a]) * (np.abs(A[a]) @ np.abs(X[n]))
        out[n] += B[a] @ t
        bound[n] = rel * (np.abs(B[a]) @ size) + 2.0 ** -23 * np.abs(out[n])
    return out, bound
