// tc_tile.cuh - what the tcgen05 kernels share: barriers with bounded waits,
// TMEM access, operand descriptors, and cached rows turned into swizzled fp16
// tiles of 128 rows.  Not part of the ABI.
#pragma once

#include "block_tile.cuh"

namespace kvc {

constexpr int TC_M = 128;  // rows of a tile: cached rows of a step, and lanes of an accumulator
constexpr int GROUP = 128; // threads of a role
constexpr uint32_t TMEM_COLS = 512; // all of it: one CTA per SM
constexpr int E_MIN = -24; // exponent of the smallest fp16 scale
constexpr uint32_t WAIT_LIMIT = 1u << 26;
constexpr uint64_t WAIT_NS = 2000000000ull;

// ---------------------------------------------------------------- PTX ----
__device__ __forceinline__ void bar_init(uint64_t *b, unsigned n) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(b)), "r"(n) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint64_t *b) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(b)) : "memory");
}
__device__ __forceinline__ bool bar_try(uint64_t *b, unsigned parity) {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok)
                 : "r"(smem_u32(b)), "r"(parity)
                 : "memory");
    return ok != 0;
}
__device__ __forceinline__ uint64_t now_ns() {
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}
// Bounded: gives up after WAIT_NS (reported, and every other wait of the CTA gives up too).  Nothing is skipped then:
// the loops run on over whatever the tiles hold, inside their buffers, so that every barrier is met and the CTA ends.
__device__ __forceinline__ void bar_wait_slow(uint64_t *b, unsigned parity, uint32_t *err, volatile int32_t *abort) {
    const uint64_t t0 = now_ns();
    for (uint32_t i = 0; i < WAIT_LIMIT; ++i) {
        if (bar_try(b, parity) || *abort) return;
        if (now_ns() - t0 > WAIT_NS) break;
    }
    atomicOr(err, ERR_WAIT_TIMEOUT);
    *abort = 1;
}
__device__ __forceinline__ void bar_wait(uint64_t *b, unsigned parity, uint32_t *err, volatile int32_t *abort) {
    if (!bar_try(b, parity)) bar_wait_slow(b, parity, err, abort);
}
// The same for a whole warp that goes on to a warp-wide TMEM access.
__device__ __forceinline__ void bar_wait_warp(uint64_t *b, unsigned parity, uint32_t *err, volatile int32_t *abort) {
    bar_wait(b, parity, err, abort);
    __syncwarp();
}
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint64_t *b) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(b)) : "memory");
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
                 "l"(a), "l"(b), "r"(idesc), "r"(acc)
                 : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
                 "r"(a), "l"(b), "r"(idesc), "r"(acc)
                 : "memory");
}
__device__ __forceinline__ void tm_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// 32 columns of the warp's 32 lanes: a thread has its own row.  The values are there after tm_wait on them.
__device__ __forceinline__ void tm_ld(uint32_t (&r)[32], uint32_t a) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
                 : "=r"(r[0]),"=r"(r[1]),"=r"(r[2]),"=r"(r[3]),"=r"(r[4]),"=r"(r[5]),"=r"(r[6]),"=r"(r[7]),"=r"(r[8]),"=r"(r[9]),"=r"(r[10]),"=r"(r[11]),"=r"(r[12]),"=r"(r[13]),"=r"(r[14]),"=r"(r[15]),"=r"(r[16]),"=r"(r[17]),"=r"(r[18]),"=r"(r[19]),"=r"(r[20]),"=r"(r[21]),"=r"(r[22]),"=r"(r[23]),"=r"(r[24]),"=r"(r[25]),"=r"(r[26]),"=r"(r[27]),"=r"(r[28]),"=r"(r[29]),"=r"(r[30]),"=r"(r[31])
                 : "r"(a)
                 : "memory");
}
__device__ __forceinline__ void tm_wait(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]),"+r"(r[1]),"+r"(r[2]),"+r"(r[3]),"+r"(r[4]),"+r"(r[5]),"+r"(r[6]),"+r"(r[7]),"+r"(r[8]),"+r"(r[9]),"+r"(r[10]),"+r"(r[11]),"+r"(r[12]),"+r"(r[13]),"+r"(r[14]),"+r"(r[15]),"+r"(r[16]),"+r"(r[17]),"+r"(r[18]),"+r"(r[19]),"+r"(r[20]),"+r"(r[21]),"+r"(r[22]),"+r"(r[23]),"+r"(r[24]),"+r"(r[25]),"+r"(r[26]),"+r"(r[27]),"+r"(r[28]),"+r"(r[29]),"+r"(r[30]),"+r"(r[31])
                 :
                 : "memory");
}
__device__ __forceinline__ void tm_ld16(uint32_t (&r)[16], uint32_t a) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : "=r"(r[0]),"=r"(r[1]),"=r"(r[2]),"=r"(r[3]),"=r"(r[4]),"=r"(r[5]),"=r"(r[6]),"=r"(r[7]),"=r"(r[8]),"=r"(r[9]),"=r"(r[10]),"=r"(r[11]),"=r"(r[12]),"=r"(r[13]),"=r"(r[14]),"=r"(r[15])
                 : "r"(a)
                 : "memory");
}
__device__ __forceinline__ void tm_wait16(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]),"+r"(r[1]),"+r"(r[2]),"+r"(r[3]),"+r"(r[4]),"+r"(r[5]),"+r"(r[6]),"+r"(r[7]),"+r"(r[8]),"+r"(r[9]),"+r"(r[10]),"+r"(r[11]),"+r"(r[12]),"+r"(r[13]),"+r"(r[14]),"+r"(r[15])
                 :
                 : "memory");
}
__device__ __forceinline__ void tm_ld32(float (&v)[32], uint32_t a) {
    uint32_t r[32];
    tm_ld(r, a);
    tm_wait(r);
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tm_st32(uint32_t a, const float (&v)[32]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
                 "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(a),
                 "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])), "r"(__float_as_uint(v[3])),
                 "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])), "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7])),
                 "r"(__float_as_uint(v[8])), "r"(__float_as_uint(v[9])), "r"(__float_as_uint(v[10])), "r"(__float_as_uint(v[11])),
                 "r"(__float_as_uint(v[12])), "r"(__float_as_uint(v[13])), "r"(__float_as_uint(v[14])), "r"(__float_as_uint(v[15])),
                 "r"(__float_as_uint(v[16])), "r"(__float_as_uint(v[17])), "r"(__float_as_uint(v[18])), "r"(__float_as_uint(v[19])),
                 "r"(__float_as_uint(v[20])), "r"(__float_as_uint(v[21])), "r"(__float_as_uint(v[22])), "r"(__float_as_uint(v[23])),
                 "r"(__float_as_uint(v[24])), "r"(__float_as_uint(v[25])), "r"(__float_as_uint(v[26])), "r"(__float_as_uint(v[27])),
                 "r"(__float_as_uint(v[28])), "r"(__float_as_uint(v[29])), "r"(__float_as_uint(v[30])), "r"(__float_as_uint(v[31]))
                 : "memory");
}
__device__ __forceinline__ void tm_st16(uint32_t a, const uint32_t (&v)[16]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(a),
                 "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
                 "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
                 : "memory");
}

// Shared-memory operand descriptor: 128-byte swizzle; sbo: bytes between groups of 8 rows; lbo: bytes between 64-wide
// blocks of the strided dimension (used by V, whose rows are the products' inner dimension).
__device__ __forceinline__ uint64_t desc(uint32_t addr, uint32_t lbo) {
    return (uint64_t)((addr & 0x3ffffu) >> 4) | (uint64_t)((lbo >> 4) & 0x3fffu) << 16 | (uint64_t)(1024u >> 4) << 32 |
           (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
// fp16 x fp16 -> fp32, 128 x n; bit 16: the second operand's rows are the inner dimension.
__device__ __forceinline__ constexpr uint32_t inst(int n, bool b_mn) {
    return (1u << 4) | (b_mn ? 1u << 16 : 0u) | ((uint32_t)(n / 8) << 17) | ((uint32_t)(TC_M / 16) << 24);
}

// Byte of (row, column) of an fp16 tile of ROWS rows: regions of 64 columns, rows of 128 bytes, 16-byte pieces swizzled by row.
template <int ROWS = TC_M> __device__ __forceinline__ uint32_t at(int row, int col) {
    return (uint32_t)((col >> 6) * (ROWS * 128) + row * 128 + ((((col >> 3) & 7) ^ (row & 7)) << 4) + (col & 7) * 2);
}

template <int ID, int N> __device__ __forceinline__ void named_sync() { asm volatile("bar.sync %0, %1;" ::"n"(ID), "n"(N) : "memory"); }
template <int N> __device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N> __device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

// Two 32-bit operations in one instruction, and the largest of three.
__device__ __forceinline__ uint64_t pair(uint32_t a, uint32_t b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint64_t pair(float a, float b) { return pair(__float_as_uint(a), __float_as_uint(b)); }
__device__ __forceinline__ float2 unpair(uint64_t v) {
    uint32_t a, b;
    asm("mov.b64 {%0, %1}, %2;" : "=r"(a), "=r"(b) : "l"(v));
    return make_float2(__uint_as_float(a), __uint_as_float(b));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Codes of one tensor: of every ROWS-th row of a step one of NT loading threads has one 16-byte piece, MINE in all.
template <int D, int T, int NT = GROUP> struct Codes {
    static constexpr int RB = row_bytes<T>(D), PIECES = RB / 16, ROWS = NT / PIECES, MINE = TC_M / ROWS;
    static_assert(ROWS % 8 == 0, "a thread's rows share their swizzle");
    // volatile: a load is to be under way as long before its use as it stands here
    __device__ __forceinline__ static void load(uint4 &u, const uint8_t *at, int32_t R) {
        asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
                     : "l"(at + (int64_t)R * RB));
    }
    // a row's scales
    __device__ __forceinline__ static void load(uint32_t (&s)[D / 64], const uint16_t *scales, int32_t R) {
        if constexpr (D == 128)
            asm volatile("ld.global.nc.v2.u32 {%0, %1}, [%2];" : "=r"(s[0]), "=r"(s[D / 64 - 1]) : "l"(scales + (int64_t)R * 4));
        else
            asm volatile("ld.global.nc.u32 %0, [%1];" : "=r"(s[0]) : "l"(scales + (int64_t)R * 2));
    }
    // The two halves of a thread's values may go to memory in an order of its own (f = swap), so that the eight threads
    // of a quarter warp write to eight different 16-byte columns of the banks.
    __device__ __forceinline__ static bool swap(int c) { return T == KVC_Q4_0 ? c >> 1 : ((c ^ (c >> 2)) & 1); }
    // byte offsets of the 8-value pieces of codes c * CODES .. of row j, in that order
    __device__ __forceinline__ static void places(int j, int c, uint32_t (&a)[4], int f) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            a[k] = T == KVC_Q4_0 ? at(j, c * 32 + (k ^ (2 * f)) * 8) : at(j, c * 16 + ((k ^ f) & 1) * 8);
    }
    // what store() rounds away of values of 8-bit codes: exact in fp16, as the product of a code and d has 18 bits
    __device__ __forceinline__ static void store_rest(uint8_t *dst, const uint32_t (&a)[4], const uint4 &u, __half2 d, bool f) {
        static_assert(T == KVC_Q8_0, "codes of 8 bits");
        auto put = [&](uint32_t o, uint2 x, uint2 y) {
            const uint32_t in[4] = {x.x, x.y, y.x, y.y};
            uint32_t r[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __half2 c = *reinterpret_cast<const __half2 *>(&in[i]), z = __hfma2(c, d, __hneg2(__hmul2(c, d)));
                r[i] = *reinterpret_cast<const uint32_t *>(&z);
            }
            *reinterpret_cast<uint4 *>(dst + o) = make_uint4(r[0], r[1], r[2], r[3]);
        };
        put(a[0], codes4(f ? u.z : u.x), codes4(f ? u.w : u.y));
        put(a[1], codes4(f ? u.x : u.z), codes4(f ? u.y : u.w));
    }
    // values = codes * d, rounded once (d: the scale times a power of two); dst: the piece's row
    __device__ __forceinline__ static void store(uint8_t *dst, const uint32_t (&a)[4], const uint4 &u, __half2 d, bool f) {
        auto put = [&](uint32_t o, uint2 x, uint2 y) {
            uint4 v;
            *reinterpret_cast<__half2 *>(&v.x) = __hmul2(*reinterpret_cast<__half2 *>(&x.x), d);
            *reinterpret_cast<__half2 *>(&v.y) = __hmul2(*reinterpret_cast<__half2 *>(&x.y), d);
            *reinterpret_cast<__half2 *>(&v.z) = __hmul2(*reinterpret_cast<__half2 *>(&y.x), d);
            *reinterpret_cast<__half2 *>(&v.w) = __hmul2(*reinterpret_cast<__half2 *>(&y.y), d);
            *reinterpret_cast<uint4 *>(dst + o) = v;
        };
        if constexpr (T == KVC_Q8_0) {
            put(a[0], codes4(f ? u.z : u.x), codes4(f ? u.w : u.y));
            put(a[1], codes4(f ? u.x : u.z), codes4(f ? u.y : u.w));
        } else {
            const int n = f ? 4 : 0;
            put(a[0], nibbles4(u.x >> n), nibbles4(u.y >> n));
            put(a[1], nibbles4(u.z >> n), nibbles4(u.w >> n));
            put(a[2], nibbles4(u.x >> (4 - n)), nibbles4(u.y >> (4 - n)));
            put(a[3], nibbles4(u.z >> (4 - n)), nibbles4(u.w >> (4 - n)));
        }
    }
};

__device__ __forceinline__ __half2 scaled(uint16_t s, float up) {
    return __half2half2(__float2half_rn(__half2float(__ushort_as_half(s)) * up));
}

// f16 rows go straight to shared memory.
template <int D> __device__ __forceinline__ void copy_halves(uint8_t *tile, const uint8_t *data, const int32_t *row, int t) {
    constexpr int PIECES = D / 8;
    const int c = t % PIECES;
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
        const int j = t / PIECES + i * (GROUP / PIECES);
        const int32_t R = row[j];
        const uint8_t *src = data + (int64_t)max(R, 0) * (2 * D) + c * 16;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(tile) + at(j, c * 8)), "l"(src),
                     "r"(R >= 0 ? 16 : 0)
                     : "memory");
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
}
// The thread's own pieces of a V tile: values that are not finite become 0, their rows are reported.
template <int D> __device__ __forceinline__ void drop_halves(uint8_t *tile, uint32_t *badrow, int t) {
    constexpr int PIECES = D / 8;
    const int c = t % PIECES;
#pragma unroll 4
    for (int i = 0; i < PIECES; ++i) {
        const int j = t / PIECES + i * (GROUP / PIECES);
        uint4 *q = reinterpret_cast<uint4 *>(tile + at(j, c * 8));
        uint4 u = *q;
        bool b = drop_nonfinite(u.x);
        b |= drop_nonfinite(u.y);
        b |= drop_nonfinite(u.z);
        b |= drop_nonfinite(u.w);
        if (b) {
            *q = u;
            atomicOr(&badrow[j >> 5], 1u << (j & 31));
        }
    }
}

} // namespace kvc
