// tree_kernel.cuh - attention of a tree of drafted tokens over the cache
// (kvc_attn_tree): the block's T tokens are the sequence's last T rows, and token
// t sees every row before them, the rows of its ancestors and its own,
//   s_j = scale * q[t][h] . K_j,   out = sum_j exp(s_j) V_j / sum_j exp(s_j),
// query head h reading KV head h / r.  Instantiated by k_tree_*.cu.
//
// A work item is one KV head, a tile of 16, 32 or 64 query rows (tokens x query
// heads of the group) and a part of the cached rows.  A drafted block is few query
// rows over many cached ones, so the kernel is built like the single-token one:
// one loading warp keeps a ring of 64-row stages full by TMA (boxes of 16 rows,
// swizzled for ldmatrix; a page holds whole boxes) and eight warps take 16 cached
// rows each, straight from the stored bytes: codes become exact fp16 values in
// registers, on their way into the products, and are used for 16 * MQ query rows
// (MQ: 2, or 1 for tiles of 16).  Bringing them to fp16 in shared memory first, as the
// block attention's tcgen05 kernel must, costs more than the products do here.
//   S = Q K^T by mma.sync m16n8k16, query rows as its rows; a 32-value block of
//   codes has sums of its own, which the block's scale multiplies in 32 bits.
//   O += P V: P goes from the scores' registers into the products' operand as it
//   lies; V's block scale is put into P (P' = P * d * 2^-E, E the exponent of the
//   largest V scale a warp has met, its sums rescaled when that grows).
//   32-bit queries and P' are two fp16 parts, and every chain of products ends
//   with the 16 rows, so that 32-bit results keep 32-bit accuracy (the tensor
//   cores truncate as they accumulate).  With 16-bit results P' is one fp16 value
//   (half a step: 2^-12), which averages out over the rows, below the result's own.
// A row's reference maximum is raised only when a score passes it by more than
// 2^8; weights stand 2^6 above their value for it, so that they stay normal fp16
// numbers down to 2^-20 of the largest.
// What a token does not see never reaches it: scores and P' are selected, and
// where V is f16 a value that is not finite, of a group of rows that not all tokens
// see (of any, where P is two parts), is left out of the products and added for
// those that see it (0 x inf is NaN).
// Warps are joined in shared memory, in their order, and the parts of a tile by
// join_kernel in theirs: results are bitwise repeatable.
#pragma once

#include "tc_tile.cuh"

namespace kvc {
namespace {

// Two groups of four warps of products and a group of which one warp loads.  A launch gives every thread 168 registers;
// the loading group hands most of its own to the others, whose sums alone are 128.
constexpr int TREE_THREADS = 12 * 32, TREE_WORK = 256;
constexpr int TREE_REGS = 168, TREE_REGS_WORK = 232, TREE_REGS_LOAD = 40;
static_assert(2 * TREE_REGS_WORK + TREE_REGS_LOAD <= 3 * TREE_REGS, "the groups' registers come from the launch's");
constexpr int TN = TREE_STEP, SLABS = TN / 16;
constexpr float T_GROW = 8.f, T_LIFT = 6.f;

template <int D, int KT, int VT, int MQ, int QS, bool LO> struct TreeShape {
    static constexpr int M = 16 * MQ * QS;       // query rows of a tile
    static constexpr int GROUPS = QS == 1 ? 2 : 1; // of warps that take stages in turn
    static constexpr int KROW = row_bytes<KT>(D), VROW = row_bytes<VT>(D);
    static constexpr bool KC = KT != KVC_F16, VC = VT != KVC_F16; // codes
    static constexpr int NB = D / QK, SB = 2 * NB;
    static constexpr int KBYTES = TN * KROW, VBYTES = TN * VROW, STAGE = KBYTES + VBYTES;
    static_assert(STAGE % 1024 == 0 && KBYTES % 1024 == 0, "swizzled boxes");
    static constexpr int SCALES = (KC ? TN * SB : 0) + (VC ? TN * SB : 0);
    static constexpr int QF = MQ * QS * (D / 16) * 32 * 16; // bytes of the query fragments (one part)
    static constexpr int AUX = 8192;
    static constexpr int FIXED = 1024 + QF * (LO ? 2 : 1) + AUX;
    static constexpr int FIT = (232448 - FIXED) / (STAGE + SCALES);
    static constexpr int STAGES = (FIT > 16 ? 16 : FIT) & ~1; // even: a stage's phases all belong to one group of warps
    static_assert(STAGES >= 4, "stages");
    static constexpr int SMEM = FIXED + STAGES * (STAGE + SCALES);
    static constexpr int PITCH = D + 16; // floats of a row where the warps are joined
    static_assert(8 * 16 * MQ * PITCH * 4 <= STAGES * (STAGE + SCALES) + QF * (LO ? 2 : 1), "the join goes over stages and queries");
};

struct TreeAux {
    uint64_t full[16], empty[16];
    int32_t parent[TREE_MAX];
    uint32_t sees[64][TREE_MAX / 32]; // of the tile's tokens, which of the block's rows they see
    float qscale[64];
    int32_t slot[64];         // query row's token, counted from the tile's first
    float m[8][32], l[8][32]; // the warps' maxima and sums
    int32_t bytes[16];
    volatile int32_t abort;
};
static_assert(sizeof(TreeAux) <= 8192, "TreeShape::AUX");

__device__ __forceinline__ void tree_box(void *dst, const CUtensorMap *map, int x, int y, uint64_t *bar) {
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
                     smem_u32(dst)),
                 "l"(map), "r"(x), "r"(y), "r"(smem_u32(bar))
                 : "memory");
}
__device__ __forceinline__ void tree_bulk(void *dst, const void *src, unsigned bytes, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

// Byte offset of 16-byte piece c of row `row` of a tile of ROWB-byte rows as the TMA's swizzle lays it (256-byte rows
// are two tiles of 128-byte ones).
template <int ROWB> __device__ __forceinline__ int tree_at(int row, int c) {
    if constexpr (ROWB == 256)
        return (c >> 3) * (TN * 128) + row * 128 + (((c & 7) ^ (row & 7)) << 4);
    else if constexpr (ROWB == 128)
        return row * 128 + ((c ^ (row & 7)) << 4);
    else
        return row * 64 + ((c ^ ((row >> 1) & 3)) << 4);
}

// Words of transposed pairs of code bytes, (row 2t: dims 2g, 2g + 1), (row 2t + 1: the same), as pairs of rows of the even
// and of the odd dim.
__device__ __forceinline__ void row_pairs(uint32_t w, uint32_t &even, uint32_t &odd) {
    const uint32_t k = 0x64646464u;
    uint32_t a = __byte_perm(w, k, 0x4240), b = __byte_perm(w, k, 0x4341);
    const __half2 c = __half2half2(__ushort_as_half(0x6480)); // 1152
    __half2 x = __hsub2(*reinterpret_cast<__half2 *>(&a), c), y = __hsub2(*reinterpret_cast<__half2 *>(&b), c);
    even = *reinterpret_cast<uint32_t *>(&x);
    odd = *reinterpret_cast<uint32_t *>(&y);
}
// The same of q4_0 bytes: the low nibbles are dims 2g, 2g + 1, the high ones those 16 further.
__device__ __forceinline__ void row_nibbles(uint32_t w, uint32_t (&v)[4]) {
    const uint32_t k = 0x64006400u;
    const __half2 c = __half2half2(__ushort_as_half(0x6408)); // 1032
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t s = i == 0 ? w : (i == 1 ? w >> 8 : (i == 2 ? w >> 4 : w >> 12));
        uint32_t a = (s & 0x000f000fu) | k;
        __half2 x = __hsub2(*reinterpret_cast<__half2 *>(&a), c);
        v[i] = *reinterpret_cast<uint32_t *>(&x);
    }
}
__device__ __forceinline__ void ldsm2t(uint32_t &a, uint32_t &b, uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0,%1}, [%2];" : "=r"(a), "=r"(b) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma1(float (&c)[4], const uint4 &a, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                 "{%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}
// 2^e of e in [-126, 127].
__device__ __forceinline__ float two_to(int e) { return __int_as_float((e + 127) << 23); }
__device__ __forceinline__ float half_of(uint32_t w, int hi) {
    return __half2float(__ushort_as_half((uint16_t)(hi ? w >> 16 : w & 0xffffu)));
}

// The two rows' block scales that a thread's columns 2t, 2t + 1 need: [row][pair of blocks].
template <int NB> __device__ __forceinline__ void load_scales(uint32_t (&w)[2][NB / 2], const uint8_t *at) {
    if constexpr (NB == 4) {
        const uint4 u = *reinterpret_cast<const uint4 *>(at);
        w[0][0] = u.x, w[0][NB / 2 - 1] = u.y, w[1][0] = u.z, w[1][NB / 2 - 1] = u.w;
    } else {
        const uint2 u = *reinterpret_cast<const uint2 *>(at);
        w[0][0] = u.x, w[1][0] = u.y;
    }
}

template <int D, int KT, int VT, int MQ, int QS, bool LO>
__global__ void __launch_bounds__(TREE_THREADS, 1)
    tree_kernel(const __grid_constant__ BlockParams p, const __grid_constant__ CUtensorMap tmk,
                const __grid_constant__ CUtensorMap tmv) {
    using S = TreeShape<D, KT, VT, MQ, QS, LO>;
    constexpr int M = S::M, NB = S::NB, NST = S::STAGES, NT = D / 8;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t *scales = smem + NST * S::STAGE;
    uint4 *qf = reinterpret_cast<uint4 *>(scales + NST * S::SCALES); // [m tile][k step][lane], then the second part
    constexpr int QPART = S::QF / 16;
    TreeAux &x = *reinterpret_cast<TreeAux *>(reinterpret_cast<uint8_t *>(qf) + S::QF * (LO ? 2 : 1));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int gq = lane >> 2, tq = lane & 3;

    const BlockSeq q = p.seq[item_seq(p, (int)blockIdx.x)];
    const int local = (int)blockIdx.x - q.item0;
    int unit, part, parts;
    item_unit(q, local, unit, part, parts);
    const int g = unit / q.tiles, tile = q.tiles - 1 - unit % q.tiles; // (the order that join_kernel takes)
    const int m_all = q.n_tok * p.r, m0 = tile * M, mrows = min(M, m_all - m0);
    // Rows are counted from the 16-row boundary at or below the sequence's first one: boxes start on such boundaries.
    const int skip = q.off & 15, first = q.off - skip, end = skip + q.n_rows, base = end - q.n_tok;
    const int a0 = part * q.split_rows, a1 = parts == 1 ? end : min(a0 + q.split_rows, end);
    const int steps = a1 > a0 ? (a1 - a0 + TN - 1) / TN : 0;

    if (tid == 0) {
        for (int i = 0; i < NST; ++i) {
            bar_init(&x.full[i], 1);
            bar_init(&x.empty[i], 8 / S::GROUPS);
        }
        x.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();

    if (warp >= 8) {
        // ------------------------------------------------------- loading
        regs_dec<TREE_REGS_LOAD>();
        if (warp > 8) return;
        // Lane s brings 16-row group s of a stage; it looks up the next step's page ahead of it.
        auto look = [&](int k) {
            const int a = a0 + k * TN + lane * 16;
            if (lane >= SLABS || k >= steps || a >= a1) return -1;
            const uint32_t pi = (uint32_t)(first + a) / (uint32_t)p.P;
            return pi < (uint32_t)p.max_pages ? p.pt[(int64_t)q.id * p.max_pages + pi] : -2;
        };
        int page = look(0);
        for (int k = 0; k < steps; ++k) {
            const int s = k % NST;
            const int a = a0 + k * TN + lane * 16;
            int pg = page;
            page = look(k + 1);
            if (pg == -1 && lane < SLABS && a < a1) pg = -2;
            if (pg != -1 && (pg < 0 || pg >= p.n_pages)) { // reported, and page 0 in its place: memory that is there
                atomicOr(p.err, ERR_BAD_PAGE);
                pg = 0;
            }
            if (k >= NST) bar_wait(&x.empty[s], ((k / NST) - 1) & 1, p.err, &x.abort);
            const unsigned have = __ballot_sync(0xffffffffu, pg >= 0);
            if (lane == 0)
                asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(&x.full[s])),
                             "r"((unsigned)__popc(have) * (unsigned)((S::STAGE + S::SCALES) / SLABS))
                             : "memory");
            __syncwarp();
            if (pg >= 0) {
                const int row = (pg * p.Hk + g) * p.P + (first + a) % p.P;
                uint8_t *kd = smem + s * S::STAGE, *vd = kd + S::KBYTES;
                if constexpr (S::KROW == 256) {
                    tree_box(kd + lane * 2048, &tmk, 0, row, &x.full[s]);
                    tree_box(kd + TN * 128 + lane * 2048, &tmk, 64, row, &x.full[s]);
                    tree_box(vd + lane * 2048, &tmv, 0, row, &x.full[s]);
                    tree_box(vd + TN * 128 + lane * 2048, &tmv, 64, row, &x.full[s]);
                } else {
                    tree_box(kd + lane * 16 * S::KROW, &tmk, 0, row, &x.full[s]);
                    tree_box(vd + lane * 16 * S::VROW, &tmv, 0, row, &x.full[s]);
                }
                uint8_t *sd = scales + s * S::SCALES + lane * 16 * S::SB;
                if constexpr (S::KC)
                    tree_bulk(sd, reinterpret_cast<const uint8_t *>(p.ks) + (int64_t)row * S::SB, 16 * S::SB, &x.full[s]);
                if constexpr (S::VC)
                    tree_bulk(sd + (S::KC ? TN * S::SB : 0), reinterpret_cast<const uint8_t *>(p.vs) + (int64_t)row * S::SB,
                              16 * S::SB, &x.full[s]);
            }
            __syncwarp();
        }
        // nothing may be under way when the CTA gives its memory back
        for (int k = max(steps - NST, 0); k < steps; ++k) {
            const uint64_t t0 = now_ns();
            while (!bar_try(&x.full[k % NST], (k / NST) & 1) && now_ns() - t0 < WAIT_NS) {
            }
        }
        return;
    }
    regs_inc<TREE_REGS_WORK>();
    {
        // The block's tree, where this part holds rows of it: which of them each of the tile's tokens sees.
        const int t_first = token_of(p, m0), t_count = token_of(p, m0 + mrows - 1) - t_first + 1;
        const bool tree = a1 > base;
        if (tree && p.parent)
            for (int i = tid; i < q.n_tok; i += TREE_WORK) {
                const int up = p.parent[(int64_t)q.tok0 + i];
                x.parent[i] = up >= 0 && up < i ? up : -1;
            }
        // Query rows, a warp each, normalised by a power of two, as the products' operand.
        constexpr int QR = M >= 32 ? 4 : 2;
        for (int mb = warp; mb < M; mb += 8 * QR) {
            Query<D> y[QR];
#pragma unroll
            for (int k = 0; k < QR; ++k) y[k].ask(p, q, g, m0 + mb + k * 8, m_all, lane);
#pragma unroll
            for (int k = 0; k < QR; ++k) {
                const int m = mb + k * 8;
                float v[D / 32];
                uint32_t hi[D / 64], lo[D / 64];
                y[k].get(p, q, v);
                const float scale = query_pack<D, LO>(p, v, hi, lo);
                if (m < M) {
                    const int r = m & 15;
#pragma unroll
                    for (int i = 0; i < D / 64; ++i) {
                        const int pr = lane * (D / 64) + i, ks = pr >> 3, pi = pr & 7; // the pair's place in its 16 dims
                        const int t = S::KC ? pi >> 1 : pi & 3, h = S::KC ? pi & 1 : pi >> 2;
                        const int at = ((m >> 4) * (D / 16) + ks) * 32 + (r & 7) * 4 + t;
                        reinterpret_cast<uint32_t *>(&qf[at])[2 * h + (r >> 3)] = hi[i];
                        if (LO) reinterpret_cast<uint32_t *>(&qf[QPART + at])[2 * h + (r >> 3)] = lo[i];
                    }
                    if (lane == 0) {
                        x.qscale[m] = scale;
                        x.slot[m] = token_of(p, min(m0 + m, m_all - 1)) - t_first;
                    }
                }
            }
        }
        if (tree) {
            named_sync<1, TREE_WORK>(); // (the parents are there)
            for (int i = tid; i < t_count; i += TREE_WORK) {
                uint32_t w[TREE_MAX / 32];
                const int t = t_first + i;
#pragma unroll
                for (int k = 0; k < TREE_MAX / 32; ++k) {
                    const int n = t + 1 - k * 32; // without a tree: a chain
                    w[k] = p.parent ? 0u : (n >= 32 ? 0xffffffffu : (n > 0 ? (1u << n) - 1u : 0u));
                    x.sees[i][k] = w[k];
                }
                if (p.parent)
                    for (int u = t; u >= 0; u = x.parent[u]) x.sees[i][u >> 5] |= 1u << (u & 31); // (a parent is below its child)
            }
        }
        named_sync<1, TREE_WORK>();
    }

    float acc[MQ][NT][4];
    float mx[MQ][2], sum[MQ][2];
#pragma unroll
    for (int i = 0; i < MQ; ++i) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[i][n][c] = 0.f;
        mx[i][0] = mx[i][1] = -INFINITY;
        sum[i][0] = sum[i][1] = 0.f;
    }
    int E = E_MIN;
    const int half = QS == 1 ? 0 : warp >> 2; // of the tile's query rows
    const int mw = half * 16 * MQ;            // the warp's first query row
    if (mw < mrows) {
        float qs[MQ][2];
#pragma unroll
        for (int i = 0; i < MQ; ++i) {
            qs[i][0] = x.qscale[mw + 16 * i + gq];
            qs[i][1] = x.qscale[mw + 16 * i + gq + 8];
        }
        const int slab = warp & 3;
        const int lrow = slab * 16 + (lane & 7) + ((lane >> 3) & 1) * 8, lhi = lane >> 4; // ldmatrix: the lane's row and piece
        const uint4 *qa = qf + (mw >> 4) * (D / 16) * 32 + lane;
        for (int k = QS == 1 ? warp >> 2 : 0; k < steps; k += S::GROUPS) {
            const int s = k % NST, a = a0 + k * TN + slab * 16;
            bar_wait_warp(&x.full[s], (k / NST) & 1, p.err, &x.abort);
            if (a < a1) {
                const uint32_t kt = smem_u32(smem + s * S::STAGE), vt = kt + S::KBYTES;
                const uint8_t *ksc = scales + s * S::SCALES + slab * 16 * S::SB;
                const uint8_t *vsc = ksc + (S::KC ? TN * S::SB : 0);
                // ---- scores: [m tile][columns 0-7, 8-15]
                float sc[MQ][2][4];
#pragma unroll
                for (int i = 0; i < MQ; ++i)
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int c = 0; c < 4; ++c) sc[i][n][c] = 0.f;
                if constexpr (S::KC) {
                    uint32_t kw[2][2][NB / 2];
                    load_scales<NB>(kw[0], ksc + tq * 2 * S::SB);
                    load_scales<NB>(kw[1], ksc + (8 + tq * 2) * S::SB);
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        uint32_t w[4];
                        ldsm4(w, kt + tree_at<S::KROW>(lrow, 2 * b + lhi));
                        const uint2 b00 = codes4(w[0]), b10 = codes4(w[1]), b01 = codes4(w[2]), b11 = codes4(w[3]);
#pragma unroll
                        for (int i = 0; i < MQ; ++i) {
                            float t0[4] = {0.f, 0.f, 0.f, 0.f}, t1[4] = {0.f, 0.f, 0.f, 0.f};
                            const uint4 qx = qa[(i * (D / 16) + 2 * b) * 32], qy = qa[(i * (D / 16) + 2 * b + 1) * 32];
                            mma1(t0, qx, b00.x, b00.y);
                            mma1(t1, qx, b10.x, b10.y);
                            mma1(t0, qy, b01.x, b01.y);
                            mma1(t1, qy, b11.x, b11.y);
                            if constexpr (LO) {
                                const uint4 lx = qa[QPART + (i * (D / 16) + 2 * b) * 32];
                                const uint4 ly = qa[QPART + (i * (D / 16) + 2 * b + 1) * 32];
                                mma1(t0, lx, b00.x, b00.y);
                                mma1(t1, lx, b10.x, b10.y);
                                mma1(t0, ly, b01.x, b01.y);
                                mma1(t1, ly, b11.x, b11.y);
                            }
                            const float d00 = half_of(kw[0][0][b >> 1], b & 1), d01 = half_of(kw[0][1][b >> 1], b & 1);
                            const float d10 = half_of(kw[1][0][b >> 1], b & 1), d11 = half_of(kw[1][1][b >> 1], b & 1);
                            sc[i][0][0] = fmaf(t0[0], d00, sc[i][0][0]);
                            sc[i][0][1] = fmaf(t0[1], d01, sc[i][0][1]);
                            sc[i][0][2] = fmaf(t0[2], d00, sc[i][0][2]);
                            sc[i][0][3] = fmaf(t0[3], d01, sc[i][0][3]);
                            sc[i][1][0] = fmaf(t1[0], d10, sc[i][1][0]);
                            sc[i][1][1] = fmaf(t1[1], d11, sc[i][1][1]);
                            sc[i][1][2] = fmaf(t1[2], d10, sc[i][1][2]);
                            sc[i][1][3] = fmaf(t1[3], d11, sc[i][1][3]);
                        }
                    }
                } else {
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks) {
                        uint32_t w[4];
                        ldsm4(w, kt + tree_at<S::KROW>(lrow, 2 * ks + lhi));
#pragma unroll
                        for (int i = 0; i < MQ; ++i) {
                            const uint4 qx = qa[(i * (D / 16) + ks) * 32];
                            if constexpr (LO) {
                                float t0[4] = {0.f, 0.f, 0.f, 0.f}, t1[4] = {0.f, 0.f, 0.f, 0.f};
                                const uint4 lx = qa[QPART + (i * (D / 16) + ks) * 32];
                                mma1(t0, qx, w[0], w[2]);
                                mma1(t1, qx, w[1], w[3]);
                                mma1(t0, lx, w[0], w[2]);
                                mma1(t1, lx, w[1], w[3]);
#pragma unroll
                                for (int c = 0; c < 4; ++c) {
                                    sc[i][0][c] += t0[c];
                                    sc[i][1][c] += t1[c];
                                }
                            } else {
                                mma1(sc[i][0], qx, w[0], w[2]);
                                mma1(sc[i][1], qx, w[1], w[3]);
                            }
                        }
                    }
                }
                // ---- what the query rows see: bit 8 i + 4 n + c of score [i][n][c]
                const bool masked = a < skip || a + 16 > base;
                uint32_t see = 0xffffffffu;
                if (masked) {
                    see = 0;
#pragma unroll
                    for (int i = 0; i < MQ; ++i)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int slot = x.slot[mw + 16 * i + gq + 8 * h];
#pragma unroll
                            for (int n = 0; n < 2; ++n)
#pragma unroll
                                for (int c = 0; c < 2; ++c) {
                                    const int j = a + 8 * n + 2 * tq + c; // the cached row
                                    bool yes = j >= skip && j < base;
                                    if (j >= base && j < end) yes = x.sees[slot][(j - base) >> 5] >> ((j - base) & 31) & 1;
                                    see |= (yes ? 1u : 0u) << (8 * i + 4 * n + 2 * h + c);
                                }
                        }
                }
                // ---- softmax, in log2 units
                float top[MQ][2];
                bool raise = false;
#pragma unroll
                for (int i = 0; i < MQ; ++i) {
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            sc[i][n][c] *= qs[i][c >> 1];
                            if (masked && !(see >> (8 * i + 4 * n + c) & 1)) sc[i][n][c] = -INFINITY;
                        }
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        top[i][h] = fmaxf(fmaxf(sc[i][0][2 * h], sc[i][0][2 * h + 1]), fmaxf(sc[i][1][2 * h], sc[i][1][2 * h + 1]));
                        raise |= top[i][h] > mx[i][h] + T_GROW;
                    }
                }
                raise = __any_sync(0xffffffffu, raise);
                // ---- V's scales and their exponent
                uint32_t vw[2][2][NB / 2];
                int e = E;
                if constexpr (S::VC) {
                    load_scales<NB>(vw[0], vsc + tq * 2 * S::SB);
                    load_scales<NB>(vw[1], vsc + (8 + tq * 2) * S::SB);
                    uint32_t most = 0;
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const int j = a + 8 * n + 2 * tq + c;
                            const bool in = !masked || (j >= skip && j < end); // (rows of nobody have no say)
#pragma unroll
                            for (int b = 0; b < NB / 2; ++b) {
                                uint32_t u = vw[n][c][b] & 0x7fff7fffu;
                                // (scales that are not finite: no say either)
                                if ((u & 0x7c00u) == 0x7c00u) u &= 0xffff0000u;
                                if ((u & 0x7c000000u) == 0x7c000000u) u &= 0xffffu;
                                most = __vmaxu2(most, in ? u : 0u);
                            }
                        }
                    most = __vmaxu2(most, __shfl_xor_sync(0xffffffffu, most, 1));
                    most = __vmaxu2(most, __shfl_xor_sync(0xffffffffu, most, 2));
                    const uint32_t one = max(most & 0xffffu, most >> 16);
                    // (an fp16 number is a normal 32-bit one)
                    if (one) e = max(E, (int)(__float_as_uint(half_of(one, 0)) >> 23) - 127);
                }
                if (raise || (S::VC && e != E)) {
                    const float ve = S::VC ? two_to(max(E - e, -126)) : 1.f;
                    E = e;
#pragma unroll
                    for (int i = 0; i < MQ; ++i)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            float t = top[i][h];
                            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 1));
                            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 2));
                            const float nm = t > mx[i][h] + T_GROW ? t : mx[i][h];
                            const float al = nm == mx[i][h] ? 1.f : ex2(mx[i][h] - nm); // nothing yet: 0
                            mx[i][h] = nm;
                            sum[i][h] *= al;
                            const float f = al * ve;
#pragma unroll
                            for (int n = 0; n < NT; ++n) {
                                acc[i][n][2 * h] *= f;
                                acc[i][n][2 * h + 1] *= f;
                            }
                        }
                }
#pragma unroll
                for (int i = 0; i < MQ; ++i)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float use = mx[i][h] == -INFINITY ? 0.f : mx[i][h] - T_LIFT;
                        float add = 0.f;
#pragma unroll
                        for (int n = 0; n < 2; ++n)
#pragma unroll
                            for (int c = 0; c < 2; ++c) {
                                const float y = ex2(sc[i][n][2 * h + c] - use);
                                sc[i][n][2 * h + c] = y;
                                add += y;
                            }
                        sum[i][h] += add;
                    }
                // ---- O += P V
                auto pack = [&](const float (&y)[2][4], uint4 &hi, uint4 &lo) {
                    hi = make_uint4(h2(y[0][0], y[0][1]), h2(y[0][2], y[0][3]), h2(y[1][0], y[1][1]), h2(y[1][2], y[1][3]));
                    if constexpr (LO) {
                        auto rest = [](uint32_t h, float u, float v) { // (an infinite scale: nothing)
                            const float2 f = f2(h);
                            return h2(isinf(f.x) ? 0.f : u - f.x, isinf(f.y) ? 0.f : v - f.y);
                        };
                        lo = make_uint4(rest(hi.x, y[0][0], y[0][1]), rest(hi.y, y[0][2], y[0][3]), rest(hi.z, y[1][0], y[1][1]),
                                        rest(hi.w, y[1][2], y[1][3]));
                    }
                };
                auto product = [&](float (&o)[4], const uint4 &hi, const uint4 &lo, uint32_t b0, uint32_t b1) {
                    if constexpr (LO) {
                        float t[4] = {0.f, 0.f, 0.f, 0.f};
                        mma1(t, hi, b0, b1);
                        mma1(t, lo, b0, b1);
#pragma unroll
                        for (int c = 0; c < 4; ++c) o[c] += t[c];
                    } else {
                        mma1(o, hi, b0, b1);
                    }
                };
                if constexpr (S::VC) {
                    const float down = two_to(-E);
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        uint32_t v0[4], v1[4]; // rows 2t, 2t + 1 and those 8 further of four columns of dims
                        if constexpr (VT == KVC_Q4_0) {
                            uint32_t wa, wb;
                            ldsm2t(wa, wb, vt + tree_at<S::VROW>(lrow, b));
                            row_nibbles(wa, v0);
                            row_nibbles(wb, v1);
                        } else {
                            uint32_t w[4];
                            ldsm4t(w, vt + tree_at<S::VROW>(lrow, 2 * b + lhi));
                            row_pairs(w[0], v0[0], v0[1]);
                            row_pairs(w[1], v1[0], v1[1]);
                            row_pairs(w[2], v0[2], v0[3]);
                            row_pairs(w[3], v1[2], v1[3]);
                        }
                        float d[2][2];
#pragma unroll
                        for (int n = 0; n < 2; ++n)
#pragma unroll
                            for (int c = 0; c < 2; ++c) d[n][c] = half_of(vw[n][c][b >> 1], b & 1) * down;
#pragma unroll
                        for (int i = 0; i < MQ; ++i) {
                            float y[2][4];
#pragma unroll
                            for (int n = 0; n < 2; ++n)
#pragma unroll
                                for (int c = 0; c < 4; ++c) {
                                    y[n][c] = sc[i][n][c] * d[n][c & 1];
                                    if (masked && !(see >> (8 * i + 4 * n + c) & 1)) y[n][c] = 0.f; // (0 x inf)
                                }
                            uint4 hi, lo;
                            pack(y, hi, lo);
#pragma unroll
                            for (int n = 0; n < 4; ++n) product(acc[i][4 * b + n], hi, lo, v0[n], v1[n]);
                        }
                    }
                } else {
                    uint4 hi[MQ], lo[MQ];
                    bool bad = false;
#pragma unroll
                    for (int i = 0; i < MQ; ++i) pack(sc[i], hi[i], lo[i]);
#pragma unroll
                    for (int n = 0; n < NT; n += 2) {
                        uint32_t w[4];
                        ldsm4t(w, vt + tree_at<S::VROW>(lrow, n + lhi));
                        if (LO || masked) { // values that are not finite: left out where P is two parts or not all tokens see them
#pragma unroll
                            for (int u = 0; u < 4; ++u) bad |= drop_nonfinite(w[u]);
                        }
#pragma unroll
                        for (int i = 0; i < MQ; ++i) {
                            product(acc[i][n], hi[i], lo[i], w[0], w[1]);
                            product(acc[i][n + 1], hi[i], lo[i], w[2], w[3]);
                        }
                    }
                    if ((LO || masked) && __any_sync(0xffffffffu, bad)) { // and added one by one for those that do
                        const uint8_t *v = smem + s * S::STAGE + S::KBYTES;
#pragma unroll 1
                        for (int j = 0; j < 16; ++j) { // row j's weights are the quad's, at lane (j % 8) / 2 of it
                            const int src = (lane & ~3) | ((j & 7) >> 1);
                            const uint32_t sees = __shfl_sync(0xffffffffu, see, src);
#pragma unroll
                            for (int i = 0; i < MQ; ++i)
#pragma unroll
                                for (int h = 0; h < 2; ++h) {
                                    const float a_ = __shfl_sync(0xffffffffu, sc[i][0][2 * h], src);
                                    const float b_ = __shfl_sync(0xffffffffu, sc[i][0][2 * h + 1], src);
                                    const float c_ = __shfl_sync(0xffffffffu, sc[i][1][2 * h], src);
                                    const float d_ = __shfl_sync(0xffffffffu, sc[i][1][2 * h + 1], src);
                                    const float w = j < 8 ? (j & 1 ? b_ : a_) : (j & 1 ? d_ : c_);
                                    if (sees >> (8 * i + 4 * (j >> 3) + 2 * h + (j & 1)) & 1) {
#pragma unroll
                                        for (int n = 0; n < NT; ++n) {
                                            const float2 y = __half22float2(*reinterpret_cast<const __half2 *>(
                                                v + tree_at<S::VROW>(slab * 16 + j, n) + tq * 4));
                                            if (!(fabsf(y.x) <= 65504.f)) acc[i][n][2 * h] += w * y.x;
                                            if (!(fabsf(y.y) <= 65504.f)) acc[i][n][2 * h + 1] += w * y.y;
                                        }
                                    }
                                }
                        }
                    }
                }
            }
            __syncwarp();
            if (lane == 0) bar_arrive(&x.empty[s]);
        }
    } else { // query rows that are not there: the stages are given back
        for (int k = QS == 1 ? warp >> 2 : 0; k < steps; k += S::GROUPS) {
            bar_wait_warp(&x.full[k % NST], (k / NST) & 1, p.err, &x.abort);
            if (lane == 0) bar_arrive(&x.empty[k % NST]);
        }
    }

    // ------------------------------------------------------- joining the warps
    constexpr int RW = QS == 1 ? 8 : 4; // warps that share query rows
    const int w0 = QS == 1 ? 0 : half * 4;
    {
#pragma unroll
        for (int i = 0; i < MQ; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                sum[i][h] += __shfl_xor_sync(0xffffffffu, sum[i][h], 1);
                sum[i][h] += __shfl_xor_sync(0xffffffffu, sum[i][h], 2);
                if (tq == 0) {
                    x.m[warp][16 * i + gq + 8 * h] = mx[i][h];
                    x.l[warp][16 * i + gq + 8 * h] = sum[i][h];
                }
            }
    }
    named_sync<1, TREE_WORK>(); // every stage has landed (its group waited for it) and is done with
    float *buf = reinterpret_cast<float *>(smem); // [warp][16 MQ][PITCH]
    {
        const float back = S::VC ? two_to(E) : 1.f;
#pragma unroll
        for (int i = 0; i < MQ; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int m = 16 * i + gq + 8 * h;
                float top = -INFINITY;
#pragma unroll
                for (int w = 0; w < RW; ++w) top = fmaxf(top, x.m[w0 + w][m]);
                const float f = ex2(mx[i][h] - (top == -INFINITY ? 0.f : top)) * back;
                float *row = buf + (warp * 16 * MQ + m) * S::PITCH;
                if constexpr (S::VC) { // columns 4b .. 4b + 3: dims 32 b + 4 t + {0, 1}, + 16
#pragma unroll
                    for (int b = 0; b < NB; ++b)
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            const float(&ev)[4] = acc[i][4 * b + 2 * u], (&od)[4] = acc[i][4 * b + 2 * u + 1];
                            *reinterpret_cast<float4 *>(row + 32 * b + 16 * u + 4 * tq) =
                                make_float4(ev[2 * h] * f, od[2 * h] * f, ev[2 * h + 1] * f, od[2 * h + 1] * f);
                        }
                } else {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        *reinterpret_cast<float2 *>(row + 8 * n + 2 * tq) = make_float2(acc[i][n][2 * h] * f, acc[i][n][2 * h + 1] * f);
                }
            }
    }
    named_sync<1, TREE_WORK>();
    const bool whole = parts == 1;
    const int prow = q.part_row0 + (local - q.whole) * p.part_rows;
    for (int at = tid; at < mrows * (D / 4); at += TREE_WORK) {
        const int m = at / (D / 4), c = at % (D / 4) * 4, hm = m / (16 * MQ), mm = m % (16 * MQ);
        float top = -INFINITY, L = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < RW; ++w) top = fmaxf(top, x.m[hm * RW + w][mm]);
        const float use = top == -INFINITY ? 0.f : top;
#pragma unroll
        for (int w = 0; w < RW; ++w) {
            const float4 y = *reinterpret_cast<const float4 *>(buf + ((hm * RW + w) * 16 * MQ + mm) * S::PITCH + c);
            L = fmaf(x.l[hm * RW + w][mm], ex2(x.m[hm * RW + w][mm] - use), L);
            o.x += y.x;
            o.y += y.y;
            o.z += y.z;
            o.w += y.w;
        }
        if (whole) {
            const int t = token_of(p, m0 + m), j = m0 + m - t * p.r;
            const int64_t out = (((int64_t)q.tok0 + t) * p.H + (int64_t)g * p.r + j) * D + c;
            const float inv = L == 0.f ? 0.f : 1.f / L;
            store2(p.out, p.act, out, o.x * inv, o.y * inv);
            store2(p.out, p.act, out + 2, o.z * inv, o.w * inv);
        } else {
            *reinterpret_cast<float4 *>(p.part + (int64_t)(prow + m) * D + c) = o;
            if (c == 0) *reinterpret_cast<float2 *>(p.part + p.part_cap * D + 2 * (int64_t)(prow + m)) = make_float2(top - T_LIFT, L);
        }
    }
}

template <int D, int KT, int VT, int MQ, int QS, bool LO>
cudaError_t tree_go(const BlockParams &p, const CUtensorMap &tmk, const CUtensorMap &tmv, cudaStream_t st) {
    auto k = tree_kernel<D, KT, VT, MQ, QS, LO>;
    constexpr int bytes = TreeShape<D, KT, VT, MQ, QS, LO>::SMEM;
    static SharedMemory set;
    cudaError_t e = set.allow((const void *)k, bytes, TREE_REGS);
    if (e != cudaSuccess) return e;
    k<<<(unsigned)p.n_items, TREE_THREADS, bytes, st>>>(p, tmk, tmv);
    e = cudaGetLastError();
    return e == cudaSuccess ? launch_join(p, st) : e;
}
template <int D, int KT, int VT>
cudaError_t tree_pick(const BlockParams &p, const CUtensorMap &tmk, const CUtensorMap &tmv, cudaStream_t st) {
    const bool lo = p.act == KVC_ACT_F32;
    switch (p.tile_m) {
    case 16: return lo ? tree_go<D, KT, VT, 1, 1, true>(p, tmk, tmv, st) : tree_go<D, KT, VT, 1, 1, false>(p, tmk, tmv, st);
    case 32: return lo ? tree_go<D, KT, VT, 2, 1, true>(p, tmk, tmv, st) : tree_go<D, KT, VT, 2, 1, false>(p, tmk, tmv, st);
    default: return lo ? tree_go<D, KT, VT, 2, 2, true>(p, tmk, tmv, st) : tree_go<D, KT, VT, 2, 2, false>(p, tmk, tmv, st);
    }
}

} // namespace
} // namespace kvc
