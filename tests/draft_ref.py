"""Plain 64-bit forms of the drafted block's operators: heads normalised and turned, a tree's visible rows, attention over
them, and the stored rows of an exported state."""
import numpy as np

from oracle import numerics as L

EPS_OF = {"f32": 2.0**-24, "f16": 2.0**-11, "bf16": 2.0**-8}  # half a step of the type


def turned(x, pos, base, neox, w=None, eps=1e-6):
    """x [T][heads][D] in 64 bits: (y, bound of a 32-bit computation's distance before its last rounding)."""
    x = np.asarray(x, np.float64)
    D = x.shape[-1]
    if w is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(w, np.float64)
    angle = np.asarray(pos, np.float64)[:, None, None] * np.power(np.float64(base), -2.0 * np.arange(D // 2) / D)
    c, s = np.cos(angle), np.sin(angle)
    y, size = np.empty_like(x), np.empty_like(x)
    i = np.arange(D // 2)
    a, b = (i, i + D // 2) if neox else (2 * i, 2 * i + 1)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., a] * s + x[..., b] * c
    size[..., a] = size[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    # The norm: 12 additions at most after the products, halved by the root, then a reciprocal root (two units in the last
    # place: 4 x 2^-24) and two products (each 2^-24): 13 x 2^-24.  Cosine and sine: the angle is off by 2^-25 of itself (at most pi) and the function by 2^-23
    # (two units in the last place of values of at most 1): 3.6 x 2^-23 = 7.2 x 2^-24.  The turn itself: 3 x 2^-24.  In 64
    # bits the angle of a position of 2^21 is off by 2^-31: nothing beside it.
    return y, size * 24 * 2.0**-24


def tree_sees(parent, n, T):
    """[T][n]: which of a sequence's n rows each token of the tree over the last T sees."""
    sees = np.zeros((T, n), bool)
    sees[:, :n - T] = True
    for t in range(T):
        u = t
        while u >= 0:
            sees[t, n - T + u] = True
            p = u - 1 if parent is None else int(parent[u])
            u = p if 0 <= p < u else -1
    return sees


def attend(q, K, V, scale, sees):
    """q [T][H][D], K, V [n][Hk][D], sees [T][n], all in 64 bits: (out, sum p |v|, the largest sum |q k| |scale| of a seen
    row), the last two for the bound of a computation's distance."""
    T, H, D = q.shape
    Hk = K.shape[1]
    r = H // Hk
    out, mag, size = np.zeros((T, H, D)), np.zeros((T, H, D)), np.zeros((T, H))
    for t in range(T):
        m = np.flatnonzero(sees[t])
        for g in range(Hk):
            hs = slice(g * r, (g + 1) * r)
            s = q[t, hs] @ K[m, g].T * scale
            e = np.exp(s - s.max(1, keepdims=True))
            p = e / e.sum(1, keepdims=True)
            out[t, hs], mag[t, hs] = p @ V[m, g], p @ np.abs(V[m, g])
            size[t, hs] = (np.abs(q[t, hs]) @ np.abs(K[m, g]).T * abs(scale)).max(1)
    return out, mag, size


def attend_bound(mag, size, n, D, act, exact=False):
    """A score is off by ds = size (2^-s + (D + 4) 2^-24) + 2^-22 (operands of s = 20 bits or more, 11 for K where the
    queries have 16 bits, unless fp16 holds K exactly; fp32 sums, a base-2 factor), a weight by 2 ds relatively, by 2^-22 for
    its exponential and by 2 (n / 8 + 8) 2^-24 for the two sums over rows (eight at a time at the least), and by 2^-11 for
    its rounding where the queries have 16 bits, 2^-20 else, V as much; the result by half a step of its type (twice, for
    the bound is on an unrounded mag)."""
    ds = size * (2.0 ** -(20 if act == "f32" or exact else 11) + (D + 4) * 2.0**-24) + 2.0**-22
    rel = 2 * ds + 2.0**-22 + 2 * (n / 8 + 8) * 2.0**-24 + 2 * (2.0**-20 if act == "f32" else 2.0**-11)
    return mag * (rel[..., None] + 2 * EPS_OF[act]) + 1e-30


def _section(blob, at, kind, Hk, n, D):
    def take(count, dtype):
        nonlocal at
        a = np.frombuffer(blob, dtype, count, at)
        at += -(-a.nbytes // 16) * 16
        return a

    if kind == L.F16:
        return take(Hk * n * D, np.float16).reshape(Hk, n, D).astype(np.float64), None, at
    if kind == L.Q8_0:
        code = take(Hk * n * D, np.int8).reshape(Hk, n, D // 32, 32).astype(np.float64)
    else:
        byte = take(Hk * n * D // 2, np.uint8).reshape(Hk, n, D // 32, 16)
        code = np.concatenate([byte & 15, byte >> 4], -1).astype(np.float64) - 8
    d = take(Hk * n * D // 32, np.float16).reshape(Hk, n, D // 32, 1).astype(np.float64)
    return (code * d).reshape(Hk, n, D), np.repeat(np.abs(d), 32, -1).reshape(Hk, n, D), at


def stored(blob, n_layer, Hk, D, tk, tv):
    """An exported state: (positions, [(K, K's steps, V, V's steps)] by layer), values [Hk][rows][D] in 64 bits, a
    code's step (None for f16) like them."""
    n = int(np.frombuffer(blob, np.uint32, 8)[7])
    pos = np.frombuffer(blob, np.int32, n, 64)
    at, layers = 64 + -(-4 * n // 16) * 16, []
    for _ in range(n_layer):
        k, ks, at = _section(blob, at, tk, Hk, n, D)
        v, vs, at = _section(blob, at, tv, Hk, n, D)
        layers.append((k, ks, v, vs))
    assert at == len(blob)
    return pos, layers
