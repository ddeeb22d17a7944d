// tree_kernel.cuh - attention of a tree of drafted tokens over the cache
// (kvc_attn_tree): the block's T tokens are the sequence's last T rows, and token
// t sees every row before them, the rows of its ancestors and its own,
//   s_j = scale * q[t][h] . K_j,   out = sum_j exp(s_j) V_j / sum_j exp(s_j),
// query head h reading KV head h / r.  Instantiated by k_tree_*.cu.
//
// A work item is one KV head, a tile of up to 32 query rows (tokens x query heads
// of the group) and a part of the cached rows.  A drafted block is few query
// rows over many cached ones, so the kernel is built like the single-token one: a
// loading group keeps a ring of 64-row stages full by TMA (boxes of 64 or 16 rows,
// swizzled for ldmatrix; a page holds whole ones of 16) and eight warps take 16
// cached rows (twice, of neighbouring stages) by 16 query rows each, straight from
// the stored bytes: codes become exact fp16 values in registers, on their way into
// the products.  Bringing them to fp16 in shared memory first, as the block
// attention's tcgen05 kernel must, costs more than the products of few query rows
// (block_attn.cu has the rule between the two, and both sides measured).
//   S = Q K^T by mma.sync m16n8k16, query rows as its rows; a 32-value block of
//   codes has sums of its own, which the block's scale multiplies in 32 bits.
//   O += P V: P goes from the scores' registers into the products' operand as it
//   lies, with V's block scale in it (P' = P * d * 2^-E, E the exponent of the
//   largest V scale a warp has met, its sums rescaled when that grows).  With 32-bit
//   queries Q and P' are two fp16 parts, and every chain of products ends with the
//   16 rows, so that 32-bit results keep 32-bit accuracy (the tensor cores truncate
//   as they accumulate).  With 16-bit ones P' is one fp16 value, whose rounding (2^-11
//   at most) is no larger than the result's.  (V's codes times their scale, rounded,
//   let P be packed once for all of V's blocks: 2 % of the time, one rounding more.)
// A row's reference maximum is raised only when a score passes it by more than
// 2^8; weights stand 2^6 above their value for it, so that they stay normal fp16
// numbers down to 2^-20 of the largest.
// What a token does not see never reaches it: scores and P' are selected, and
// where V is f16 a value that is not finite, of a group of rows that not all tokens
// see (of any, where P is two parts), is left out of the products (0 x inf is NaN)
// and put into the results of the query rows that see it.
// Warps are joined in shared memory, in their order, and the parts of a tile by
// join_kernel in theirs: results are bitwise repeatable.
// What bounds it: with up to 16 query rows a KV head memory (halves: 65536 rows of 8
// KV heads of D 128 in 49 us, 5.5 TB/s; 16 sequences of 4096 rows 46 us) or, of codes,
// the instructions between their bytes and the products (38 us, 3.7 TB/s); with more
// of both the latter, two thirds of mma.sync's rate at the most.  What it cost to find:
// copies of 16 rows issued by one warp, 100 cycles each whatever their size (62 us),
// sixteen warps of 96 registers, whose spilled ones have no cache beside this much
// shared memory (59 against 54 us of 4 tokens), the next rows' scores among the weights
// and products of these (76 against 68 us of 26 tokens over 16k, by the first build).
#pragma once

#include "tc_tile.cuh"

#include <type_traits>

namespace kvc {
namespace {

// Two groups of four warps of products and one that loads.  A launch gives every thread 168 registers; the loading group
// hands most of its own to the others.
constexpr int TREE_WARPS = 8, TREE_WORK = TREE_WARPS * 32, TREE_THREADS = TREE_WORK + 128;
constexpr int TREE_REGS = 168, TREE_REGS_WORK = 232, TREE_REGS_LOAD = 40;
static_assert(2 * TREE_REGS_WORK + TREE_REGS_LOAD <= 3 * TREE_REGS, "the groups' registers come from the launch's");
constexpr int TN = TREE_STEP, SLABS = TN / 16;
constexpr float T_GROW = 8.f, T_LIFT = 6.f;

template <int D, int KT, int VT, bool LO> struct TreeShape {
    static constexpr int KROW = row_bytes<KT>(D), VROW = row_bytes<VT>(D);
    static constexpr bool KC = KT != KVC_F16, VC = VT != KVC_F16; // codes
    static constexpr int NB = D / QK, SB = 2 * NB;
    static constexpr int KBYTES = TN * KROW, VBYTES = TN * VROW, STAGE = KBYTES + VBYTES;
    static_assert(STAGE % 1024 == 0 && KBYTES % 1024 == 0, "swizzled boxes");
    static constexpr int SCALES = (KC ? TN * SB : 0) + (VC ? TN * SB : 0);
    static constexpr int QF = TREE_TILE / 16 * (D / 16) * 32 * 16; // bytes of the query fragments (one part)
    static constexpr int AUX = 8192;
    static constexpr int FIXED = 1024 + QF * (LO ? 2 : 1) + AUX;
    static constexpr int FIT = (232448 - FIXED) / (STAGE + SCALES);
    static constexpr int STAGES = FIT > 12 ? 12 : FIT;
    static_assert(STAGES >= 4, "a stage for every group");
    static constexpr int SMEM = FIXED + STAGES * (STAGE + SCALES);
    static constexpr int PITCH = D + 16; // floats of a row where the warps are joined
    static_assert(TREE_WARPS * 16 * PITCH * 4 <= STAGES * (STAGE + SCALES) + QF * (LO ? 2 : 1), "the join goes over stages and queries");
};

struct TreeAux {
    uint64_t full[12], empty[12];
    int32_t parent[TREE_MAX];
    uint32_t sees[TREE_TILE][TREE_MAX / 32]; // of the tile's tokens, which of the block's rows they see
    float qscale[TREE_TILE];
    uint32_t poison[TREE_TILE][8]; // two bits a value: +inf, -inf (both: NaN) received
    int32_t bad_first, bad_last; // 16-row groups with values that were left out of the products
    int32_t slot[TREE_TILE];  // query row's token, counted from the tile's first
    float m[TREE_WARPS][16], l[TREE_WARPS][16]; // the warps' maxima and sums
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
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
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
// The same of one pair of blocks.
template <int NB> __device__ __forceinline__ void load_pair(uint32_t (&w)[2], const uint8_t *at, int pair) {
    w[0] = *reinterpret_cast<const volatile uint32_t *>(at + 4 * pair);
    w[1] = *reinterpret_cast<const volatile uint32_t *>(at + 2 * NB + 4 * pair);
}

template <int D, int KT, int VT, bool LO>
__global__ void __launch_bounds__(TREE_THREADS, 1)
    tree_kernel(const __grid_constant__ BlockParams p, const __grid_constant__ CUtensorMap tmk,
                const __grid_constant__ CUtensorMap tmv, const __grid_constant__ CUtensorMap tmk16,
                const __grid_constant__ CUtensorMap tmv16) {
    using S = TreeShape<D, KT, VT, LO>;
    constexpr int M = TREE_TILE, NB = S::NB, NT = D / 8;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t *scales = smem + S::STAGES * S::STAGE;
    uint4 *qf = reinterpret_cast<uint4 *>(scales + S::STAGES * S::SCALES); // [m tile][k step][lane], then the second part
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
    // More than 16 query rows: the two groups have 16 of them each, over all stages; else they take pairs of stages in turn.
    // A stage's phases all belong to the same warps (a wait tells a phase only from the one before), so that stages are as
    // many as fit in whole turns of pairs.
    const int shares = mrows > 16 ? 2 : 1, turns = 2 / shares;
    const int nst = S::STAGES / (2 * turns) * (2 * turns);
    // Rows are counted from the 16-row boundary at or below the sequence's first one: boxes start on such boundaries.
    const int skip = q.off & 15, first = q.off - skip, end = skip + q.n_rows, base = end - q.n_tok;
    const int a0 = part * q.split_rows, a1 = parts == 1 ? end : min(a0 + q.split_rows, end);
    const int steps = a1 > a0 ? (a1 - a0 + TN - 1) / TN : 0;

    if (tid == 0) {
        for (int i = 0; i < S::STAGES; ++i) {
            bar_init(&x.full[i], 1);
            bar_init(&x.empty[i], 4 * shares);
        }
        x.abort = 0;
        x.bad_first = 0x7fffffff;
        x.bad_last = -1;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    wait_for_previous();

    if (warp >= TREE_WARPS) {
        // ------------------------------------------------------- loading
        regs_dec<TREE_REGS_LOAD>();
        // A stage's 64 rows that lie in one page come as boxes of 64: K and V and the scales of either by a warp each.  Else
        // each warp brings one of the stage's 16-row groups (a copy costs a warp about 100 cycles, whatever its size: with
        // 16 of them from one warp they took longer than the memory).  A warp looks up 32 steps' pages at once, the next
        // ones while it issues.
        const int w = warp - TREE_WARPS;
        auto look = [&](int k, int group) { // the page of 16-row group `group` of step k; -1: no rows, -2: no page
            const int a = a0 + k * TN + group * 16;
            if (a >= a1) return -1;
            const uint32_t pi = (uint32_t)(first + a) / (uint32_t)p.P;
            const int page = pi < (uint32_t)p.max_pages ? p.pt[(int64_t)q.id * p.max_pages + pi] : -2;
            return page < 0 || page >= p.n_pages ? -2 : page;
        };
        int own = -1, own_next = look(lane, w), lead = -1, lead_next = look(lane, 0);
        int s = 0, round = 0; // the step's stage, and how often the ring has gone round
        for (int k = 0; k < steps; ++k) {
            if (k % 32 == 0) {
                own = own_next, lead = lead_next;
                if (own == -2 || lead == -2) { // reported, and page 0 in its place: memory that is there
                    atomicOr(p.err, ERR_BAD_PAGE);
                    own = max(own, -1) + (own == -2), lead = max(lead, -1) + (lead == -2);
                }
                own_next = look(k + 32 + lane, w), lead_next = look(k + 32 + lane, 0);
            }
            const int pg = __shfl_sync(0xffffffffu, own, k & 31), pg0 = __shfl_sync(0xffffffffu, lead, k & 31);
            const int a = a0 + k * TN, cell = (first + a) % p.P;
            const bool one = cell + TN <= p.P;
            if (round > 0) bar_wait(&x.empty[s], (round - 1) & 1, p.err, &x.abort);
            if (lane == 0) {
                const int groups = one ? SLABS : min(SLABS, (a1 - a + 15) / 16); // of 16 rows that come
                uint64_t *bar = &x.full[s];
                if (w == 0)
                    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)),
                                 "r"((unsigned)groups * (unsigned)((S::STAGE + S::SCALES) / SLABS))
                                 : "memory");
                uint8_t *kd = smem + s * S::STAGE, *vd = kd + S::KBYTES;
                uint8_t *sd = scales + s * S::SCALES;
                const uint8_t *ks = reinterpret_cast<const uint8_t *>(p.ks), *vs = reinterpret_cast<const uint8_t *>(p.vs);
                if (one) {
                    const int row = (pg0 * p.Hk + g) * p.P + cell;
                    if (w == 0) {
                        tree_box(kd, &tmk, 0, row, bar);
                        if (S::KROW == 256) tree_box(kd + TN * 128, &tmk, 64, row, bar);
                    } else if (w == 1) {
                        tree_box(vd, &tmv, 0, row, bar);
                        if (S::VROW == 256) tree_box(vd + TN * 128, &tmv, 64, row, bar);
                    } else if (w == 2) {
                        if (S::KC) tree_bulk(sd, ks + (int64_t)row * S::SB, TN * S::SB, bar);
                    } else {
                        if (S::VC) tree_bulk(sd + (S::KC ? TN * S::SB : 0), vs + (int64_t)row * S::SB, TN * S::SB, bar);
                    }
                } else if (w < groups) {
                    const int row = (pg * p.Hk + g) * p.P + (first + a + w * 16) % p.P;
                    constexpr int KT_ = S::KROW == 256 ? 128 : S::KROW, VT_ = S::VROW == 256 ? 128 : S::VROW;
                    tree_box(kd + w * 16 * KT_, &tmk16, 0, row, bar);
                    if (S::KROW == 256) tree_box(kd + TN * 128 + w * 2048, &tmk16, 64, row, bar);
                    tree_box(vd + w * 16 * VT_, &tmv16, 0, row, bar);
                    if (S::VROW == 256) tree_box(vd + TN * 128 + w * 2048, &tmv16, 64, row, bar);
                    sd += w * 16 * S::SB;
                    if (S::KC) tree_bulk(sd, ks + (int64_t)row * S::SB, 16 * S::SB, bar);
                    if (S::VC) tree_bulk(sd + (S::KC ? TN * S::SB : 0), vs + (int64_t)row * S::SB, 16 * S::SB, bar);
                }
            }
            __syncwarp();
            if (++s == nst) {
                s = 0;
                ++round;
            }
        }
        // nothing may be under way when the CTA gives its memory back
        for (int k = max(steps - nst, 0); k < steps; ++k) {
            const uint64_t t0 = now_ns();
            while (!bar_try(&x.full[k % nst], (k / nst) & 1) && now_ns() - t0 < WAIT_NS) {
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
        for (int i = tid; i < M * (D / 16); i += TREE_WORK) x.poison[i / (D / 16)][i % (D / 16)] = 0;
        // Query rows, a warp each, normalised by a power of two, as the products' operand.
        constexpr int QR = 2;
        for (int mb = warp; mb < 16 * shares; mb += TREE_WARPS * QR) {
            Query<D> y[QR];
#pragma unroll
            for (int k = 0; k < QR; ++k) y[k].ask(p, q, g, m0 + mb + k * TREE_WARPS, m_all, lane);
#pragma unroll
            for (int k = 0; k < QR; ++k) {
                const int m = mb + k * TREE_WARPS;
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

    float acc[NT][4], mx[2], sum[2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[n][c] = 0.f;
    mx[0] = mx[1] = -INFINITY;
    sum[0] = sum[1] = 0.f;
    int E = E_MIN;
    const int group = warp >> 2, slab = warp & 3;
    const int mw = group % shares * 16, turn = group / shares; // the warp's first query row; its set of groups
    {
        const float qs[2] = {x.qscale[mw + gq], x.qscale[mw + gq + 8]};
        const int lrow = slab * 16 + (lane & 7) + ((lane >> 3) & 1) * 8, lhi = lane >> 4; // ldmatrix: the lane's row and piece
        const uint4 *qa = qf + (mw >> 4) * (D / 16) * 32 + lane;
        // SL groups of 16 rows, a first at row a of stage s and the others a stage further: a warp's two chains of products
        // and softmax run beside each other where nothing is masked.  MASK: some of the rows are not seen by all (rows of
        // the block, or of nobody).
        auto rows = [&](int s, int a, auto sl_) {
            constexpr int SL = decltype(sl_)::value;
            constexpr bool MASK = SL == 1;
            // ---- scores of columns 0-7 and 8-15
            float sc[SL][2][4];
            auto k_tile = [&](int l) { return smem_u32(smem + (s + l) * S::STAGE); };
            auto scale_at = [&](int l) { return scales + (s + l) * S::SCALES + slab * 16 * S::SB + tq * 2 * S::SB; }; // of the lane's columns
            [[maybe_unused]] constexpr int VS = S::KC ? TN * S::SB : 0; // V's behind K's
            if constexpr (S::KC) {
                uint32_t kw[SL][2][2];
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    const uint4 qx = qa[2 * b * 32], qy = qa[(2 * b + 1) * 32];
                    uint4 lx, ly;
                    if (LO) lx = qa[QPART + 2 * b * 32], ly = qa[QPART + (2 * b + 1) * 32];
#pragma unroll
                    for (int l = 0; l < SL; ++l) {
                        if (b % 2 == 0) {
                            load_pair<NB>(kw[l][0], scale_at(l), b / 2);
                            load_pair<NB>(kw[l][1], scale_at(l) + 8 * S::SB, b / 2);
                        }
                        uint32_t w[4];
                        ldsm4(w, k_tile(l) + tree_at<S::KROW>(lrow, 2 * b + lhi));
                        uint2 c0 = codes4(w[0]), c1 = codes4(w[1]);
                        float t[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
                        mma1(t[0], qx, c0.x, c0.y);
                        mma1(t[1], qx, c1.x, c1.y);
                        if (LO) {
                            mma1(t[0], lx, c0.x, c0.y);
                            mma1(t[1], lx, c1.x, c1.y);
                        }
                        c0 = codes4(w[2]), c1 = codes4(w[3]);
                        mma1(t[0], qy, c0.x, c0.y);
                        mma1(t[1], qy, c1.x, c1.y);
                        if (LO) {
                            mma1(t[0], ly, c0.x, c0.y);
                            mma1(t[1], ly, c1.x, c1.y);
                        }
#pragma unroll
                        for (int n = 0; n < 2; ++n) {
                            const float d0 = half_of(kw[l][n][0], b & 1), d1 = half_of(kw[l][n][1], b & 1);
#pragma unroll
                            for (int c = 0; c < 4; ++c)
                                sc[l][n][c] = b ? fmaf(t[n][c], c & 1 ? d1 : d0, sc[l][n][c]) : t[n][c] * (c & 1 ? d1 : d0);
                        }
                    }
                }
            } else {
#pragma unroll
                for (int l = 0; l < SL; ++l)
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int c = 0; c < 4; ++c) sc[l][n][c] = 0.f;
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                    const uint4 qx = qa[ks * 32];
                    uint4 lx;
                    if (LO) lx = qa[QPART + ks * 32];
#pragma unroll
                    for (int l = 0; l < SL; ++l) {
                        uint32_t w[4];
                        ldsm4(w, k_tile(l) + tree_at<S::KROW>(lrow, 2 * ks + lhi));
                        if constexpr (LO) {
                            float t[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
                            mma1(t[0], qx, w[0], w[2]);
                            mma1(t[1], qx, w[1], w[3]);
                            mma1(t[0], lx, w[0], w[2]);
                            mma1(t[1], lx, w[1], w[3]);
#pragma unroll
                            for (int n = 0; n < 2; ++n)
#pragma unroll
                                for (int c = 0; c < 4; ++c) sc[l][n][c] += t[n][c];
                        } else {
                            mma1(sc[l][0], qx, w[0], w[2]);
                            mma1(sc[l][1], qx, w[1], w[3]);
                        }
                    }
                }
            }
            // ---- what the query rows see: bit 4 n + c of score [n][c]
            uint32_t see = 0;
            if constexpr (MASK) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int slot = x.slot[mw + gq + 8 * h];
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const int j = a + 8 * n + 2 * tq + c; // the cached row
                            bool yes = j >= skip && j < base;
                            if (j >= base && j < end) yes = x.sees[slot][(j - base) >> 5] >> ((j - base) & 31) & 1;
                            see |= (yes ? 1u : 0u) << (4 * n + 2 * h + c);
                        }
                }
            }
            auto unseen = [&](int n, int c) { return MASK && !(see >> (4 * n + c) & 1); };
            // ---- softmax, in log2 units
            float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int l = 0; l < SL; ++l)
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        sc[l][n][c] *= qs[c >> 1];
                        if (unseen(n, c)) sc[l][n][c] = -INFINITY;
                        top[c >> 1] = fmaxf(top[c >> 1], sc[l][n][c]);
                    }
            const bool raise = __any_sync(0xffffffffu, top[0] > mx[0] + T_GROW || top[1] > mx[1] + T_GROW);
            // ---- V's scales and their exponent
            int e = E;
            bool bad = false; // V values of the rows are not finite
            if constexpr (S::VC) {
                uint32_t vw[SL][2][2][NB / 2];
#pragma unroll
                for (int l = 0; l < SL; ++l) {
                    load_scales<NB>(vw[l][0], scale_at(l) + VS);
                    load_scales<NB>(vw[l][1], scale_at(l) + VS + 8 * S::SB);
                }
                // the rows' largest; not of rows of nobody, and not of scales that are not finite (which are looked for in
                // all rows, as their products would be formed)
                auto largest = [&](bool all) {
                    uint32_t most = 0;
#pragma unroll
                    for (int l = 0; l < SL; ++l)
#pragma unroll
                        for (int n = 0; n < 2; ++n)
#pragma unroll
                            for (int c = 0; c < 2; ++c) {
                                const int j = a + 8 * n + 2 * tq + c;
                                const bool in = all || !MASK || (j >= skip && j < end);
#pragma unroll
                                for (int b = 0; b < NB / 2; ++b) {
                                    uint32_t u = vw[l][n][c][b] & 0x7fff7fffu;
                                    if (!all) u &= ~__vcmpgeu2(u, 0x7c007c00u);
                                    most = __vmaxu2(most, in ? u : 0u);
                                }
                            }
                    most = __vmaxu2(most, __shfl_xor_sync(0xffffffffu, most, 1));
                    most = __vmaxu2(most, __shfl_xor_sync(0xffffffffu, most, 2));
                    return max(most & 0xffffu, most >> 16);
                };
                uint32_t one = largest(true);
                bad = __any_sync(0xffffffffu, one >= 0x7c00u);
                if (MASK || bad) one = largest(false);
                // (an fp16 number is a normal 32-bit one; a quad's lanes hold all rows)
                if (one) e = max(E, (int)(__float_as_uint(half_of(one, 0)) >> 23) - 127);
            }
            if (raise || (S::VC && e != E)) {
                const float ve = S::VC ? two_to(max(E - e, -126)) : 1.f;
                E = e;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float t = top[h];
                    t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 1));
                    t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 2));
                    const float nm = t > mx[h] + T_GROW ? t : mx[h];
                    const float al = nm == mx[h] ? 1.f : ex2(mx[h] - nm); // nothing yet: 0
                    mx[h] = nm;
                    sum[h] *= al;
                    const float f = al * ve;
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        acc[n][2 * h] *= f;
                        acc[n][2 * h + 1] *= f;
                    }
                }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float use = mx[h] == -INFINITY ? 0.f : mx[h] - T_LIFT;
                float add = 0.f;
#pragma unroll
                for (int l = 0; l < SL; ++l)
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const float y = ex2(sc[l][n][2 * h + c] - use);
                            sc[l][n][2 * h + c] = y;
                            add += y;
                        }
                sum[h] += add;
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
            // Values that are not finite (0 x inf is NaN): reported, seen to in the end, and 0 in the products.  (`bad`
            // has them found; another warp that shares the rows may be at the same.)
            auto leave_out = [&] {
                for (int l = 0; l < SL; ++l) {
                    if (lane == 0) {
                        atomicMin(&x.bad_first, a + l * TN);
                        atomicMax(&x.bad_last, a + l * TN);
                    }
                    uint8_t *v = smem + (s + l) * S::STAGE + S::KBYTES;
                    for (int i = lane; i < 16 * S::VROW / 4; i += 32) {
                        uint32_t *w = reinterpret_cast<uint32_t *>(
                            v + tree_at<S::VROW>(slab * 16 + i / (S::VROW / 4), i % (S::VROW / 4) / 4) + i % 4 * 4);
                        uint32_t u = *w;
                        if (drop_nonfinite(u)) *w = u;
                    }
                }
                fence_async(); // (before the copies of a later step)
                __syncwarp();
            };
            if constexpr (S::VC) {
                const float down = two_to(-E);
                uint32_t vw[SL][2][2]; // (read again: a pair of blocks at a time)
#pragma unroll
                for (int b = 0; b < NB; ++b) {
#pragma unroll
                    for (int l = 0; l < SL; ++l) {
                        const uint32_t vt = k_tile(l) + S::KBYTES;
                        if (b % 2 == 0) {
                            load_pair<NB>(vw[l][0], scale_at(l) + VS, b / 2);
                            load_pair<NB>(vw[l][1], scale_at(l) + VS + 8 * S::SB, b / 2);
                        }
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
                        float y[2][4];
#pragma unroll
                        for (int n = 0; n < 2; ++n) {
                            const float d0 = half_of(vw[l][n][0], b & 1) * down, d1 = half_of(vw[l][n][1], b & 1) * down;
#pragma unroll
                            for (int c = 0; c < 4; ++c) y[n][c] = unseen(n, c) ? 0.f : sc[l][n][c] * (c & 1 ? d1 : d0); // (0 x inf)
                        }
                        uint4 hi, lo;
                        pack(y, hi, lo);
#pragma unroll
                        for (int n = 0; n < 4; ++n) product(acc[4 * b + n], hi, lo, v0[n], v1[n]);
                    }
                }
            } else {
                if (LO || MASK) { // (of 16-bit queries that all see the rows, P x inf is what it should be)
                    __half2 f = __float2half2_rn(0.f);
#pragma unroll
                    for (int l = 0; l < SL; ++l)
#pragma unroll
                        for (int n = 0; n < NT; n += 2) {
                            uint32_t w[4];
                            ldsm4t(w, k_tile(l) + S::KBYTES + tree_at<S::VROW>(lrow, n + lhi));
#pragma unroll
                            for (int u = 0; u < 4; ++u) f = __hfma2(*reinterpret_cast<__half2 *>(&w[u]), __float2half2_rn(0.f), f);
                        }
                    bad = !(__low2float(f) == 0.f && __high2float(f) == 0.f);
                    if (__any_sync(0xffffffffu, bad)) leave_out();
                }
                uint4 hi[SL], lo[SL];
#pragma unroll
                for (int l = 0; l < SL; ++l) pack(sc[l], hi[l], lo[l]);
#pragma unroll
                for (int n = 0; n < NT; n += 2) {
#pragma unroll
                    for (int l = 0; l < SL; ++l) {
                        uint32_t w[4];
                        ldsm4t(w, k_tile(l) + S::KBYTES + tree_at<S::VROW>(lrow, n + lhi));
                        product(acc[n], hi[l], lo[l], w[0], w[1]);
                        product(acc[n + 1], hi[l], lo[l], w[2], w[3]);
                    }
                }
            }
        };
        int s = 2 * turn, phase = 0;
        for (int k = 2 * turn; k < steps; k += 2 * turns) {
            const int a = a0 + k * TN + slab * 16, a2 = a + TN;
            const bool two = k + 1 < steps;
            bar_wait_warp(&x.full[s], phase, p.err, &x.abort);
            if (two) bar_wait_warp(&x.full[s + 1], phase, p.err, &x.abort);
            if (two && a >= skip && a2 + 16 <= base && a2 < a1) {
                rows(s, a, std::integral_constant<int, 2>{});
            } else {
#pragma unroll 1
                for (int l = 0; l < 2; ++l)
                    if (a + l * TN < a1) rows(s + l, a + l * TN, std::integral_constant<int, 1>{});
            }
            __syncwarp();
            if (lane == 0) {
                bar_arrive(&x.empty[s]);
                if (two) bar_arrive(&x.empty[s + 1]);
            }
            s += 2 * turns;
            if (s >= nst) {
                s -= nst;
                phase ^= 1;
            }
        }
    }

    // ------------------------------------------------------- joining the warps
    // Those of query rows mw ..: groups share, share + shares, ..., in that order.
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        sum[h] += __shfl_xor_sync(0xffffffffu, sum[h], 1);
        sum[h] += __shfl_xor_sync(0xffffffffu, sum[h], 2);
        if (tq == 0) {
            x.m[warp][gq + 8 * h] = mx[h];
            x.l[warp][gq + 8 * h] = sum[h];
        }
    }
    named_sync<1, TREE_WORK>(); // every stage has landed (its groups waited for it) and is done with
    float *buf = reinterpret_cast<float *>(smem); // [warp][16][PITCH]
    const int rw = 4 * turns;                     // warps that share query rows
    auto warp_of = [&](int m, int i) { return ((m >> 4) + (i >> 2) * shares) * 4 + (i & 3); };
    {
        const float back = S::VC ? two_to(E) : 1.f;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int m = gq + 8 * h;
            float top = -INFINITY;
            for (int i = 0; i < rw; ++i) top = fmaxf(top, x.m[warp_of(mw, i)][m]);
            const float f = ex2(mx[h] - (top == -INFINITY ? 0.f : top)) * back;
            float *row = buf + (warp * 16 + m) * S::PITCH;
            if constexpr (S::VC) { // columns 4b .. 4b + 3: dims 32 b + 4 t + {0, 1}, + 16
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const float(&ev)[4] = acc[4 * b + 2 * u], (&od)[4] = acc[4 * b + 2 * u + 1];
                        *reinterpret_cast<float4 *>(row + 32 * b + 16 * u + 4 * tq) =
                            make_float4(ev[2 * h] * f, od[2 * h] * f, ev[2 * h + 1] * f, od[2 * h + 1] * f);
                    }
            } else {
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    *reinterpret_cast<float2 *>(row + 8 * n + 2 * tq) = make_float2(acc[n][2 * h] * f, acc[n][2 * h + 1] * f);
            }
        }
    }
    named_sync<1, TREE_WORK>();
    if (x.bad_last >= 0) { // (rare) what was left out reaches the query rows that see its row
        for (int i = tid; i < (x.bad_last + 16 - x.bad_first) * D; i += TREE_WORK) {
            const int a = x.bad_first + i / D, d = i % D, j = a - skip;
            const int32_t R = a >= skip && a < min(end, a1) ? pool_row(p, q, g, j) : -1;
            if (R < 0) continue;
            const float v = stored_value<D, VT>(p.vdata, p.vs, R, d);
            if (fabsf(v) <= 3.4e38f) continue;
            const uint32_t two = (v > 0.f ? 1u : (v < 0.f ? 2u : 3u)) << (2 * (d & 15));
            for (int m = 0; m < mrows; ++m)
                if (a < base || (x.sees[x.slot[m]][(a - base) >> 5] >> ((a - base) & 31) & 1)) atomicOr(&x.poison[m][d >> 4], two);
        }
        named_sync<1, TREE_WORK>();
    }
    const bool whole = parts == 1;
    const int prow = q.part_row0 + (local - q.whole) * p.part_rows;
    for (int at = tid; at < mrows * (D / 4); at += TREE_WORK) {
        const int m = at / (D / 4), c = at % (D / 4) * 4, mm = m & 15;
        float top = -INFINITY, L = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int i = 0; i < rw; ++i) top = fmaxf(top, x.m[warp_of(m, i)][mm]);
        const float use = top == -INFINITY ? 0.f : top;
#pragma unroll 4
        for (int i = 0; i < rw; ++i) {
            const int w = warp_of(m, i);
            const float4 y = *reinterpret_cast<const float4 *>(buf + (w * 16 + mm) * S::PITCH + c);
            L = fmaf(x.l[w][mm], ex2(x.m[w][mm] - use), L);
            o.x += y.x;
            o.y += y.y;
            o.z += y.z;
            o.w += y.w;
        }
        if (x.bad_last >= 0) {
            const uint32_t two = x.poison[m][c >> 4] >> (2 * (c & 15));
            o.x = poisoned(o.x, two & 3u);
            o.y = poisoned(o.y, two >> 2 & 3u);
            o.z = poisoned(o.z, two >> 4 & 3u);
            o.w = poisoned(o.w, two >> 6 & 3u);
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

static_assert(sizeof(BlockParams) + 4 * sizeof(CUtensorMap) <= 4096, "launch parameters stay within 4 KB");
template <int D, int KT, int VT, bool LO> cudaError_t tree_go(const BlockParams &p, const TreeMaps &t, cudaStream_t st) {
    auto k = tree_kernel<D, KT, VT, LO>;
    constexpr int bytes = TreeShape<D, KT, VT, LO>::SMEM;
    static SharedMemory set;
    cudaError_t e = set.allow((const void *)k, bytes, TREE_REGS);
    if (e != cudaSuccess) return e;
    e = launch_behind(k, (unsigned)p.n_items, TREE_THREADS, bytes, st, p, *t.k, *t.v, *t.k16, *t.v16);
    return e == cudaSuccess ? launch_join(p, st) : e;
}
template <int D, int KT, int VT> cudaError_t tree_pick(const BlockParams &p, const TreeMaps &t, cudaStream_t st) {
    return p.act == KVC_ACT_F32 ? tree_go<D, KT, VT, true>(p, t, st) : tree_go<D, KT, VT, false>(p, t, st);
}

} // namespace
} // namespace kvc
