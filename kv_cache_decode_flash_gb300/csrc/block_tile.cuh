// block_tile.cuh - what the kernels over a block of query tokens share: a
// step's cached rows as fp16 in shared memory, the query rows, and their
// products.  Not part of the ABI.
//
// Codes are exact in fp16; block scales stay apart, in 32 bits.  A query row is
// normalised by a power of two (its largest magnitude comes to lie in
// [2^13, 2^14)): exact for f16 and bf16 queries, while 32-bit queries are split
// into two fp16 parts, 22 bits together.  A step's scores are then as exact as
// sums in 32 bits are: a block of 32 products is summed by the tensor cores,
// scaled in 32 bits and added.
#pragma once

#include "block_attn.h"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace kvc {

// What preceding kernels wrote may be read behind this (launches by launch_behind).
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

constexpr int BLOCK_THREADS = 128;
constexpr int TILE_PAD = 8; // halves behind a row: 16 bytes off a multiple of 128, so ldmatrix has no bank conflicts

__device__ __forceinline__ uint32_t smem_u32(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                 "{%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t h2(float a, float b) {
    __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<uint32_t *>(&h);
}
__device__ __forceinline__ float2 f2(uint32_t u) { return __half22float2(*reinterpret_cast<__half2 *>(&u)); }

// Four offset-binary codes (code + 128) to four halves: the byte becomes the
// low mantissa of 1024, from which 1152 is taken (exact).
__device__ __forceinline__ uint2 codes4(uint32_t w) {
    const uint32_t k = 0x64646464u;
    uint32_t lo = __byte_perm(w, k, 0x4140), hi = __byte_perm(w, k, 0x4342);
    const __half2 c = __half2half2(__ushort_as_half(0x6480)); // 1152
    __half2 a = __hsub2(*reinterpret_cast<__half2 *>(&lo), c), b = __hsub2(*reinterpret_cast<__half2 *>(&hi), c);
    return make_uint2(*reinterpret_cast<uint32_t *>(&a), *reinterpret_cast<uint32_t *>(&b));
}
// The low nibbles of four bytes to four halves code - 8.
__device__ __forceinline__ uint2 nibbles4(uint32_t w) {
    w &= 0x0f0f0f0fu;
    const uint32_t k = 0x64646464u;
    uint32_t lo = __byte_perm(w, k, 0x4140), hi = __byte_perm(w, k, 0x4342);
    const __half2 c = __half2half2(__ushort_as_half(0x6408)); // 1032
    __half2 a = __hsub2(*reinterpret_cast<__half2 *>(&lo), c), b = __hsub2(*reinterpret_cast<__half2 *>(&hi), c);
    return make_uint2(*reinterpret_cast<uint32_t *>(&a), *reinterpret_cast<uint32_t *>(&b));
}
// Whether either half of the pair is inf or NaN; those set to 0.
__device__ __forceinline__ bool drop_nonfinite(uint32_t &u) {
    const bool a = (u & 0x7c00u) == 0x7c00u, b = (u & 0x7c000000u) == 0x7c000000u;
    if (a) u &= 0xffff0000u;
    if (b) u &= 0x0000ffffu;
    return a || b;
}

template <int KT> __device__ __forceinline__ constexpr int row_bytes(int D) {
    return KT == KVC_F16 ? 2 * D : (KT == KVC_Q4_0 ? D / 2 : D);
}

// A step's rows of one tensor, as they are stored, to fp16 (codes without their scale), both in shared memory; returns
// whether a value of them is not finite (V only: such values are set to 0).
template <int D, int T, bool V>
__device__ __forceinline__ bool fill(__half (*dst)[D + TILE_PAD], const uint8_t *raw, uint8_t *badrow, int tid) {
    constexpr int RB = row_bytes<T>(D), PIECES = RB / 16;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < CROSS_TILE_N * PIECES / BLOCK_THREADS; ++i) {
        const int at = tid + i * BLOCK_THREADS, j = at / PIECES, c = at % PIECES;
        uint4 u = *reinterpret_cast<const uint4 *>(raw + at * 16);
        if constexpr (T == KVC_F16) {
            if constexpr (V) {
                bool b = drop_nonfinite(u.x);
                b |= drop_nonfinite(u.y);
                b |= drop_nonfinite(u.z);
                b |= drop_nonfinite(u.w);
                if (b) badrow[j] = 1;
                bad |= b;
            }
            *reinterpret_cast<uint4 *>(&dst[j][c * 8]) = u;
        } else if constexpr (T == KVC_Q8_0) {
            const uint2 a = codes4(u.x), b = codes4(u.y), e = codes4(u.z), f = codes4(u.w);
            *reinterpret_cast<uint4 *>(&dst[j][c * 16]) = make_uint4(a.x, a.y, b.x, b.y);
            *reinterpret_cast<uint4 *>(&dst[j][c * 16 + 8]) = make_uint4(e.x, e.y, f.x, f.y);
        } else {
            // byte i of a 32-value block holds the codes i (low) and i + 16 (high)
            uint2 a = nibbles4(u.x), b = nibbles4(u.y), e = nibbles4(u.z), f = nibbles4(u.w);
            *reinterpret_cast<uint4 *>(&dst[j][c * 32]) = make_uint4(a.x, a.y, b.x, b.y);
            *reinterpret_cast<uint4 *>(&dst[j][c * 32 + 8]) = make_uint4(e.x, e.y, f.x, f.y);
            a = nibbles4(u.x >> 4), b = nibbles4(u.y >> 4), e = nibbles4(u.z >> 4), f = nibbles4(u.w >> 4);
            *reinterpret_cast<uint4 *>(&dst[j][c * 32 + 16]) = make_uint4(a.x, a.y, b.x, b.y);
            *reinterpret_cast<uint4 *>(&dst[j][c * 32 + 24]) = make_uint4(e.x, e.y, f.x, f.y);
        }
    }
    return bad;
}


// Pool rows of the step's cached rows base .. base + CROSS_TILE_N - 1 of KV head g: -1 past the sequence's end, and for
// a page that the pool does not have (reported).
__device__ __forceinline__ int32_t pool_row(const BlockParams &p, const BlockSeq &q, int g, int j) {
    if (j >= q.n_rows) return -1;
    const uint32_t lr = (uint32_t)q.off + (uint32_t)j, pi = lr / (uint32_t)p.P;
    const int32_t page = pi < (uint32_t)p.max_pages ? p.pt[(int64_t)q.id * p.max_pages + pi] : -1;
    if (page < 0 || page >= p.n_pages) {
        atomicOr(p.err, ERR_BAD_PAGE);
        return -1;
    }
    return (page * p.Hk + g) * p.P + (int32_t)(lr - pi * p.P); // rows of a layer's pool are fewer than 2^31
}

// A row's way through the page table in two steps, so that nobody waits for the table: its entry is requested, and
// looked at a step later.
struct Lookup {
    int32_t page = -1;
    uint32_t cell = 0;
    bool in = false;
    __device__ __forceinline__ void ask(const BlockParams &p, const BlockSeq &q, int j, bool valid) {
        in = valid && j < q.n_rows;
        const uint32_t lr = (uint32_t)q.off + (uint32_t)j, pi = lr / (uint32_t)p.P;
        cell = lr - pi * (uint32_t)p.P;
        page = -1;
        if (in && pi < (uint32_t)p.max_pages) page = p.pt[(int64_t)q.id * p.max_pages + pi];
    }
    // the pool row, -1 for none (a page that the pool does not have is reported)
    __device__ __forceinline__ int32_t row(const BlockParams &p, int g) const {
        if (in && (page < 0 || page >= p.n_pages)) {
            atomicOr(p.err, ERR_BAD_PAGE);
            return -1;
        }
        return in ? (page * p.Hk + g) * p.P + (int32_t)cell : -1;
    }
};

// The launch's sequence that work item `item` belongs to: the last one whose
// first item is not behind it (sequences without items share a first item).
__device__ __forceinline__ int item_seq(const BlockParams &p, int item) {
    int lo = 0, hi = p.n_seq - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (p.seq[mid].item0 <= item) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// Item `local` of a sequence: the unit (KV head, query tile) and the part of the rows that it is.
__device__ __forceinline__ void item_unit(const BlockSeq &q, int local, int &unit, int &part, int &parts) {
    const bool whole = local < q.whole;
    unit = whole ? local : q.whole + (local - q.whole) / q.splits;
    part = whole ? 0 : (local - q.whole) % q.splits;
    parts = whole ? 1 : q.splits;
}

// m / r (r <= 8, m < 2^29).
__device__ __forceinline__ int token_of(const BlockParams &p, int m) {
    return p.r == 1 ? m : (int)__umulhi((uint32_t)m, p.r_magic);
}

// Lane l's values l * D / 32 .. of query row m of KV head g, one warp a row.  ask() only requests them and the rows that
// the token sees (of the last row, for a row that is not there), so that several rows can be under way; get() looks.
template <int D> struct Query {
    static constexpr int V = D / 32;
    uint32_t raw[V];
    int32_t see;
    bool in;
    __device__ __forceinline__ void ask(const BlockParams &p, const BlockSeq &q, int g, int m, int m_all, int lane) {
        in = m < m_all;
        m = min(m, m_all - 1);
        const int t = token_of(p, m), j = m - t * p.r;
        const int64_t tok = (int64_t)q.tok0 + t;
        const int64_t at = (tok * p.H + (int64_t)g * p.r + j) * D + lane * V;
        if (p.act == KVC_ACT_F32) {
            const uint32_t *src = reinterpret_cast<const uint32_t *>(p.q) + at;
            if constexpr (V == 4) {
                const uint4 u = *reinterpret_cast<const uint4 *>(src);
                raw[0] = u.x, raw[1] = u.y, raw[2] = u.z, raw[3] = u.w;
            } else {
                const uint2 u = *reinterpret_cast<const uint2 *>(src);
                raw[0] = u.x, raw[1] = u.y;
            }
        } else {
            const uint16_t *src = reinterpret_cast<const uint16_t *>(p.q) + at;
            if constexpr (V == 4) {
                const uint2 u = *reinterpret_cast<const uint2 *>(src);
                raw[0] = u.x, raw[1] = u.y;
            } else {
                raw[0] = *reinterpret_cast<const uint32_t *>(src);
            }
        }
        see = p.n_vis ? p.n_vis[tok] : q.n_rows;
    }
    // the rows that it sees: 0 for a row that is not there, whose values are 0
    __device__ __forceinline__ int get(const BlockParams &p, const BlockSeq &q, float (&x)[V]) const {
#pragma unroll
        for (int i = 0; i < V; i += 2) {
            float2 f;
            if (p.act == KVC_ACT_F32) {
                f = make_float2(__uint_as_float(raw[i]), __uint_as_float(raw[i + 1]));
            } else if (p.act == KVC_ACT_F16) {
                f = f2(raw[i / 2]);
            } else {
                f = make_float2(__uint_as_float(raw[i / 2] << 16), __uint_as_float(raw[i / 2] & 0xffff0000u));
            }
            x[i] = in ? f.x : 0.f;
            x[i + 1] = in ? f.y : 0.f;
        }
        return in ? min(max(see, 0), q.n_rows) : 0;
    }
};

// The warp normalises the row: a lane's values as pairs of halves hi (and lo, what hi leaves).  Returns the score per unit
// of the normalised product, in log2 units.
template <int D, bool LO>
__device__ __forceinline__ float query_pack(const BlockParams &p, const float (&x)[D / 32], uint32_t (&hi)[D / 64],
                                            uint32_t (&lo)[D / 64]) {
    constexpr int V = D / 32;
    uint32_t top = 0; // magnitudes as bits are ordered like the numbers
#pragma unroll
    for (int i = 0; i < V; ++i) top = max(top, __float_as_uint(x[i]) & 0x7fffffffu);
    top = __reduce_max_sync(0xffffffffu, top);
    // times 2^(140 - exponent): to [2^13, 2^14).  (Rows below 2^-114 become zero scores; one with infinities keeps them.)
    const uint32_t e = min(max(267 - (int)(top >> 23), 1), 254);
    const float up = __uint_as_float(e << 23), down = __uint_as_float((254 - e) << 23);
#pragma unroll
    for (int i = 0; i < V; i += 2) {
        const float a = x[i] * up, b = x[i + 1] * up;
        const uint32_t h = h2(a, b);
        hi[i / 2] = h;
        if (LO) {
            const float2 f = f2(h);
            lo[i / 2] = h2(isinf(f.x) ? 0.f : a - f.x, isinf(f.y) ? 0.f : b - f.y);
        }
    }
    return p.scale_log2 * down;
}

// A V value as stored (the rare path of values that are not finite).
template <int D, int T>
__device__ float stored_value(const uint8_t *data, const uint16_t *scales, int32_t R, int d) {
    if constexpr (T == KVC_F16) {
        return __half2float(reinterpret_cast<const __half *>(data)[(int64_t)R * D + d]);
    } else {
        const float s = __half2float(__ushort_as_half(scales[(int64_t)R * (D / QK) + d / QK]));
        if constexpr (T == KVC_Q8_0) return (float)((int)data[(int64_t)R * D + d] - 128) * s;
        const int b = d / QK, e = d % QK;
        const uint8_t byte = data[(int64_t)R * (D / 2) + b * (QK / 2) + (e & 15)];
        return (float)((int)(e < 16 ? byte & 15 : byte >> 4) - 8) * s;
    }
}

// The values of row R that are not finite, marked in the two-bit words of a query row that sees it.
template <int D, int T>
__device__ __forceinline__ void mark_poison(uint32_t *words, const uint8_t *data, const uint16_t *scales, int32_t R) {
    for (int d = 0; d < D; ++d) {
        const float x = stored_value<D, T>(data, scales, R, d);
        if (fabsf(x) <= 3.4e38f) continue;
        const uint32_t two = x > 0.f ? 1u : (x < 0.f ? 2u : 3u);
        atomicOr(&words[d / 16], two << (2 * (d % 16)));
    }
}

__device__ __forceinline__ float poisoned(float x, uint32_t two_bits) {
    if (two_bits == 3) return __int_as_float(0x7fffffff);
    if (two_bits == 0) return x;
    return x + (two_bits == 1 ? __int_as_float(0x7f800000) : __int_as_float(0xff800000));
}

// Two values as the pair of a 16-bit type.
__device__ __forceinline__ uint32_t pack16(int act, float a, float b) {
    if (act == KVC_ACT_F16) return h2(a, b);
    __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t *>(&h);
}
__device__ __forceinline__ void store2(void *out, int act, int64_t at, float a, float b) {
    if (act == KVC_ACT_F32)
        *reinterpret_cast<float2 *>(reinterpret_cast<float *>(out) + at) = make_float2(a, b);
    else
        *reinterpret_cast<uint32_t *>(reinterpret_cast<uint16_t *>(out) + at) = pack16(act, a, b);
}

// sc = the products of 16 query rows (addresses qa, ql of their fp16 parts) and NT * 8 cached rows (address ka),
// block scales d[b][col] applied: the accumulator layout of mma.m16n8k16.
template <int D, int KT, int NT, bool LO>
__device__ __forceinline__ void scores(float (&sc)[NT][4], uint32_t qa, uint32_t ql, uint32_t ka,
                                       const float (*d)[CROSS_TILE_N], int col) {
    constexpr int PITCH = (D + TILE_PAD) * 2;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int k = 0; k < 4; ++k) sc[n][k] = 0.f;
#pragma unroll
    for (int b = 0; b < D / QK; ++b) {
        float t[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int k = 0; k < 4; ++k) t[n][k] = 0.f;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            uint32_t a[4], al[4];
            ldsm4(a, qa + (b * 32 + k * 16) * 2);
            if (LO) ldsm4(al, ql + (b * 32 + k * 16) * 2);
#pragma unroll
            for (int n = 0; n < NT; n += 2) {
                uint32_t kb[4];
                ldsm4(kb, ka + n * 8 * PITCH + (b * 32 + k * 16) * 2);
                mma(t[n], a, kb[0], kb[1]);
                mma(t[n + 1], a, kb[2], kb[3]);
                if (LO) {
                    mma(t[n], al, kb[0], kb[1]);
                    mma(t[n + 1], al, kb[2], kb[3]);
                }
            }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            if constexpr (KT != KVC_F16) {
                const float2 f = *reinterpret_cast<const float2 *>(&d[b][col + n * 8]);
                sc[n][0] = fmaf(t[n][0], f.x, sc[n][0]);
                sc[n][1] = fmaf(t[n][1], f.y, sc[n][1]);
                sc[n][2] = fmaf(t[n][2], f.x, sc[n][2]);
                sc[n][3] = fmaf(t[n][3], f.y, sc[n][3]);
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k) sc[n][k] += t[n][k];
            }
        }
    }
}

} // namespace kvc
