"""Plain 64-bit forms of the block operators, over the rows that the oracle stored.

Tolerances are worked out from the inputs here: a product's operands are
rounded to `bits` significant bits (half a step each, 2^-bits), sums are fp32.
"""
import numpy as np

from oracle import numerics as L

ACT_EPS = {"f32": 2.0**-24, "f16": 2.0**-11, "bf16": 2.0**-8}  # half a step of the result's type


def values(t):
    """Stored rows [n][Hk][D] of an oracle tensor in 64 bits."""
    if t.type == L.F16:
        return np.ascontiguousarray(t.a).view(np.float16).astype(np.float64)
    if t.type == L.Q4_0:
        return L.q4_0_dequantize(t.a, t.s)
    return L.q8_0_dequantize(t.a, t.s)


def cross(q, K, V, scale, vis):
    """q [T][H][D], K, V [n][Hk][D] in 64 bits, vis [T]: (out [T][H][D], lse [T][H], bound_out, bound_lse): the
    bounds of the distance, by operand roundings of 2^-bits, as functions of bits."""
    T, H, D = q.shape
    n, Hk = K.shape[0], K.shape[1]
    r = H // Hk
    out, lse = np.zeros((T, H, D)), np.full((T, H), -np.inf)
    mag, size = np.zeros((T, H, D)), np.zeros((T, H))  # sum p |v|, and the largest sum |q k| scale of a seen row
    for t in range(T):
        m = int(min(max(vis[t], 0), n))
        if m == 0:
            continue
        for g in range(Hk):
            qq = q[t, g * r:(g + 1) * r]
            s = qq @ K[:m, g].T * scale
            big = s.max(1, keepdims=True)
            e = np.exp(s - big)
            z = e.sum(1, keepdims=True)
            hs = slice(g * r, (g + 1) * r)
            out[t, hs] = e / z @ V[:m, g]
            lse[t, hs] = (big + np.log(z))[:, 0]
            mag[t, hs] = e / z @ np.abs(V[:m, g])
            size[t, hs] = (np.abs(qq) @ np.abs(K[:m, g]).T * abs(scale)).max(1)
    return out, lse, mag, size


def cross_bound(mag, size, n, D, act, s_bits, v_bits):
    """Largest distance of out and lse.  A score is off by ds = size * (2^-s_bits + (D + 4) 2^-24): its operands'
    rounding, the products' sum and its scaling in fp32.  A weight exp(s - lse) is off by 2 ds relatively (its own score and the
    others'), by 2^-22 for the exponential and by the sum of up to n terms, (n / 8 + 8) 2^-24 (eight terms at a time); the
    probabilities and V values lose 2^-v_bits each, the products' sum again (n / 8 + 8) 2^-24, the result half a step."""
    ds = size * (2.0**-s_bits + (D + 4) * 2.0**-24) + 2.0**-22
    rest = 2.0**-22 + 2 * (n / 8 + 8) * 2.0**-24
    rel = 2 * ds + rest + 2 * 2.0**-v_bits
    return mag * (rel[..., None] + 2 * ACT_EPS[act]) + 1e-30, ds + rest + 2.0**-22 * (1 + size + np.log(max(n, 2)))


def exact_kv(rng, n, Hk, D, step=2.0**-5):
    """Values that q8_0 and f16 hold exactly: integers in [-127, 127] times a power of two, one of them +-127 in
    every block of 32."""
    x = rng.integers(-127, 128, (n, Hk, D // 32, 32))
    x[..., 0] = 127 * rng.choice([-1, 1], x.shape[:-1])
    return (x.reshape(n, Hk, D) * step).astype(np.float32)


def weight(q, K, scale, vis, lse):
    """(w [Hk][n] that the tokens add, a bound of its distance for 32-bit arithmetic): exp(s - lse) is off by the score's
    error (operands of 20 bits or more, fp32 sums), by those of s - lse in fp32 (2^-23 of the larger one, twice) and of the exponential
    (2^-21), the sum over the query rows by 2^-24 for each of them."""
    T, H, D = q.shape
    n, Hk = K.shape[0], K.shape[1]
    r = H // Hk
    w, bound = np.zeros((Hk, n)), np.zeros((Hk, n))
    for t in range(T):
        m = int(min(max(vis[t], 0), n))
        for g in range(Hk):
            for h in range(g * r, (g + 1) * r):
                s = K[:m, g] @ q[t, h] * scale
                e = np.exp(s - lse[t, h])
                size = np.abs(K[:m, g]) @ np.abs(q[t, h]) * abs(scale)
                ds = size * (2.0**-20 + (D + 4) * 2.0**-24) + 2.0**-21 * (1 + np.abs(s) + abs(lse[t, h]))
                w[g, :m] += e
                bound[g, :m] += e * (2 * ds + 2.0**-21)
    return w, bound + w * (T * r + 4) * 2.0**-24


def evict(weights, cand, n, n_remove):
    """Row order after an eviction: rows of smallest (weight, row) among `cand` go, the kept ones behind the new end
    take their places.  weights [Hk][n] fp32.  Returns (order, removed): row i of the result is row order[i]."""
    w = weights[0].astype(np.float32)
    with np.errstate(invalid="ignore"):
        for g in range(1, len(weights)):
            w = (w + weights[g]).astype(np.float32)
    key = [(1, 0.0, j) if np.isnan(w[j]) else (0, float(w[j]), j) for j in cand]
    gone = sorted(k[2] for k in sorted(key)[:n_remove])
    left = n - len(gone)
    order = list(range(left))
    movers = [j for j in range(left, n) if j not in set(gone)]
    for hole, j in zip([g for g in gone if g < left], movers):
        order[hole] = j
    return order, gone
