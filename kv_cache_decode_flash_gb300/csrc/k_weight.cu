// k_weight.cu - the attention weight that cached rows receive from a block of
// query tokens (kvc_attn_weight): for every KV head g and cached row j
//   w[g][j] += sum over tokens t that see j, query heads h of g:
//              exp(scale * q[t][h] . K_j - lse[t][h]),
// lse the statistics that the attention of the same tokens left behind.
//
// The scores are formed transposed, S^T = K Q^T, on tcgen05: 128 cached rows of a
// step are the accumulator's lanes and the query rows (tokens x query heads of
// the group, up to 256) its columns, so that a thread owns a cached row and the
// sum over the query rows is its own: no exchange, no atomics, one fixed order.
// The query rows lie in shared memory for a work item's whole range of cached
// rows (a KV head's), and K is read once.
//   Sums of weights are 32-bit results, so operands lose nothing that matters:
// K = code * scale is taken as two fp16 parts, which hold its 18 bits exactly
// (halves are one part), a 16-bit query is exact in fp16 and a 32-bit one two
// parts, whose product with K's second part (2^-22 of the first's) is left out.
// A power of two brings a step's largest scale to [2^3, 2^4); it changes only
// when the scales have moved by 2^4, so that the factors per query row, in which
// it is undone, are seldom rewritten.
//   One CTA per SM, five groups of four warps: two softmax groups and two loading groups that
// take the steps in turn, and that of the issuing thread; the accumulators alternate in TMEM.
// What bounds it: with many query rows shared memory, which the products' operands
// (two parts of K, each against all query rows), the conversion's stores and the
// factors' loads share (32 tokens of 40 heads over 131072 rows: q8_0 91 us, of which
// the products alone 36; 32-bit queries 140 us; halves, 32 heads, 62 us); with few,
// the memory for halves (one token: 55 us, 4.9 TB/s) and the conversion for codes
// (57 us, 2.5 TB/s).  The register-operand tensor path, which takes codes as they
// are, reached 228 us on the first of these.
#include "tc_tile.cuh"

namespace kvc {
namespace {

constexpr int THREADS = 5 * GROUP; // roles: softmax of even and of odd steps, loading of even and odd steps, the issuing warp
constexpr int TN = TC_M;           // cached rows of a step
// Registers: a launch gives every thread 96; the summing groups take what the issuing warp's group hands back.
constexpr int R_LAUNCH = 96, R_SUM = 128, R_MMA = 24;
static_assert(2 * R_SUM + 2 * R_LAUNCH + R_MMA <= 5 * R_LAUNCH, "the roles' registers come from the launch's");
static_assert(WEIGHT_STEP == TN, "items are whole steps");

enum Bar { KF0, KF1, KE0, KE1, SF0, SF1, SE0, SE1, QF, DRAIN, N_BARS };

template <int D, bool CODES, bool LO> struct Lay {
    static constexpr int MG = LO ? 128 : 256;         // query rows at a time
    static constexpr int QT = D / 64 * MG * 128;      // bytes of one of their fp16 parts
    static constexpr int KT = D / 64 * TN * 128;      // bytes of one part of a step
    static constexpr int KS = (CODES ? 2 : 1) * KT;   // of a stage
    static constexpr int K = (LO ? 2 : 1) * QT, AUX = K + 2 * KS;
};

struct Aux {
    uint64_t bar[N_BARS];
    alignas(16) float2 fz[2][256];   // per softmax group and query row: score factor, log2 of its sum
    float2 fz0[256];                 // the same before a step's exponent
    alignas(16) int32_t vis[256];
    int32_t row[2][2][TN];           // per loading group: pool rows of its step and of its next one
    int32_t kexp[2][4];              // exponent of a step, by its group and place
    alignas(16) uint32_t red[2][2][GROUP / 32];
    uint16_t scale[2][2][TN * 4];
    uint32_t tmem;
    int32_t vis_max, vis_min;
    volatile int32_t abort;
};

template <int D, bool CODES, bool LO> constexpr int smem_bytes() {
    const int need = Lay<D, CODES, LO>::AUX + (int)sizeof(Aux) + 1024;
    return need > 120 * 1024 ? need : 120 * 1024; // TMEM is allocated whole: one CTA per SM
}

// codes * d as two fp16 parts, exactly
template <int D>
__device__ __forceinline__ void store_parts(uint8_t *hi, uint8_t *lo, const uint32_t (&a)[4], const uint4 &u, __half2 d, bool f) {
    const uint32_t in[4] = {f ? u.z : u.x, f ? u.w : u.y, f ? u.x : u.z, f ? u.y : u.w};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        uint32_t h[4], l[4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint2 c = codes4(in[2 * k + i]);
            const uint32_t cc[2] = {c.x, c.y};
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const __half2 x = *reinterpret_cast<const __half2 *>(&cc[e]);
                const __half2 y = __hmul2(x, d);
                const __half2 z = __hfma2(x, d, __hneg2(y)); // what the first part leaves (one rounding, exact here)
                h[2 * i + e] = *reinterpret_cast<const uint32_t *>(&y);
                l[2 * i + e] = *reinterpret_cast<const uint32_t *>(&z);
            }
        }
        *reinterpret_cast<uint4 *>(hi + a[k]) = make_uint4(h[0], h[1], h[2], h[3]);
        *reinterpret_cast<uint4 *>(lo + a[k]) = make_uint4(l[0], l[1], l[2], l[3]);
    }
}

// The sum of a cached row's weights over `cols` query rows; MASK: of those that see row j.
template <bool MASK>
__device__ __forceinline__ float row_sum(uint32_t S, int cols, const float2 *fz, const int32_t *vis, int j) {
    uint64_t a0 = 0, a1 = 0;
    uint32_t r[2][16];
    auto block = [&](int c, const uint32_t(&v)[16]) {
#pragma unroll
        for (int k = 0; k < 16; k += 4) {
            float y[4];
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
                const float4 f = *reinterpret_cast<const float4 *>(&fz[c + k + i]); // (a broadcast)
                y[i] = ex2(fmaf(__uint_as_float(v[k + i]), f.x, f.y));
                y[i + 1] = ex2(fmaf(__uint_as_float(v[k + i + 1]), f.z, f.w));
            }
            if (MASK) {
                const int4 s = *reinterpret_cast<const int4 *>(&vis[c + k]);
                y[0] = j < s.x ? y[0] : 0.f;
                y[1] = j < s.y ? y[1] : 0.f;
                y[2] = j < s.z ? y[2] : 0.f;
                y[3] = j < s.w ? y[3] : 0.f;
            }
            a0 = add2(a0, pair(y[0], y[1]));
            a1 = add2(a1, pair(y[2], y[3]));
        }
    };
    tm_ld16(r[0], S);
    for (int c = 0; c < cols; c += 32) {
        tm_wait16(r[0]);
        if (c + 16 < cols) tm_ld16(r[1], S + c + 16);
        block(c, r[0]);
        if (c + 16 < cols) {
            tm_wait16(r[1]);
            if (c + 32 < cols) tm_ld16(r[0], S + c + 32);
            block(c + 16, r[1]);
        }
    }
    const float2 s = unpair(add2(a0, a1));
    return s.x + s.y;
}

template <int D, int KT, bool LO>
__global__ void __launch_bounds__(THREADS, 1) weight_kernel(const __grid_constant__ BlockParams p) {
    constexpr bool CODES = KT != KVC_F16;
    using L = Lay<D, CODES, LO>;
    constexpr int MG = L::MG;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    Aux &x = *reinterpret_cast<Aux *>(smem + L::AUX);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    const BlockSeq q = p.seq[item_seq(p, (int)blockIdx.x)];
    int g, part, parts;
    item_unit(q, (int)blockIdx.x - q.item0, g, part, parts);
    const int m_all = q.n_tok * p.r, groups = (m_all + MG - 1) / MG;
    if (tid == 0) {
        for (int i = 0; i < N_BARS; ++i)
            bar_init(&x.bar[i], i == KF0 || i == KF1 || i == SE0 || i == SE1 ? GROUP : (i == QF ? 2 * GROUP : 1));
        x.vis_max = 0;
        x.vis_min = 0x7fffffff;
        x.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&x.tmem)), "r"(TMEM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    __syncthreads();
    for (int t = tid; t < q.n_tok; t += THREADS) {
        const int v = p.n_vis ? min(max(p.n_vis[(int64_t)q.tok0 + t], 0), q.n_rows) : q.n_rows;
        atomicMax(&x.vis_max, v);
        atomicMin(&x.vis_min, v);
    }
    tc_before();
    __syncthreads();
    tc_after();
    const uint32_t tm = x.tmem; // two accumulators of 256 columns
    const int r0 = part * q.split_rows, r1 = min(parts == 1 ? q.n_rows : r0 + q.split_rows, x.vis_max);
    const int steps = r1 > r0 ? (r1 - r0 + TN - 1) / TN : 0, jobs = groups * steps; // job: a step of a group of query rows
    const int vis_min = x.vis_min;

    if (warp < 8) {
        // -------------------------------------------------- sums, and the query rows
        regs_inc<R_SUM>();
        const int h = warp >> 2, t = tid & 127;
        const uint32_t S = tm + h * 256 + ((uint32_t)(warp & 3) << 21);
        float *w = p.w + ((int64_t)q.w_index * p.Hk + g) * p.w_stride;
        int done = 0; // jobs of this group
        for (int mg = 0; mg < groups && steps > 0; ++mg) {
            const int rows = min(MG, m_all - mg * MG), cols = (rows + 15) / 16 * 16;
            named_sync<2, 2 * GROUP>(); // every product with the rows before is done: both groups have its scores
            constexpr int QR = 4;
            for (int mb = warp; mb < cols; mb += 8 * QR) {
                Query<D> y[QR];
                float z[QR];
#pragma unroll
                for (int k = 0; k < QR; ++k) {
                    if (mb + k * 8 >= cols) break;
                    const int m = mg * MG + mb + k * 8;
                    y[k].ask(p, q, g, m, m_all, lane);
                    const int mm = min(m, m_all - 1), tok = token_of(p, mm), j = mm - tok * p.r;
                    z[k] = p.lse[((int64_t)q.tok0 + tok) * p.H + (int64_t)g * p.r + j];
                }
#pragma unroll
                for (int k = 0; k < QR; ++k) {
                    const int m = mb + k * 8;
                    if (m >= cols) break;
                    float v[D / 32];
                    uint32_t hi[D / 64], lo[D / 64];
                    const int vis = y[k].get(p, q, v); // (a row behind the group's last one is its own part's, or none)
                    const float scale = query_pack<D, LO>(p, v, hi, lo);
                    uint8_t *dst = smem + at<MG>(m, lane * (D / 32));
                    if constexpr (D == 128) {
                        *reinterpret_cast<uint2 *>(dst) = make_uint2(hi[0], hi[1]);
                        if (LO) *reinterpret_cast<uint2 *>(dst + L::QT) = make_uint2(lo[0], lo[1]);
                    } else {
                        *reinterpret_cast<uint32_t *>(dst) = hi[0];
                        if (LO) *reinterpret_cast<uint32_t *>(dst + L::QT) = lo[0];
                    }
                    if (lane == 0) {
                        // a row that is not there, or sees nothing: weight 0
                        x.fz0[m] = make_float2(vis > 0 ? scale : 0.f, vis > 0 ? z[k] * 1.44269504f : INFINITY);
                        x.vis[m] = vis;
                    }
                }
            }
            fence_async();
            named_sync<2, 2 * GROUP>(); // the rows' factors are there
            bar_arrive(&x.bar[QF]);
            int E = 0x7fffffff; // exponent that this group's factors hold
            for (int i = mg * steps + ((mg * steps + h) & 1); i < (mg + 1) * steps; i += 2, ++done) {
                const int base = r0 + (i - mg * steps) * TN, j = base + t;
                const bool in = j < r1;
                const float old = in ? w[j] : 0.f;
                bar_wait_warp(&x.bar[SF0 + h], done & 1, p.err, &x.abort);
                tc_after();
                const int e = CODES ? x.kexp[h][done & 3] : 3;
                if (e != E) {
                    if (h == 0) named_sync<5, GROUP>(); else named_sync<6, GROUP>(); // the old ones are read no more
                    const float f = ldexpf(1.f, e - 3);
                    for (int m = t; m < cols; m += GROUP) x.fz[h][m] = make_float2(x.fz0[m].x * f, -x.fz0[m].y);
                    if (h == 0) named_sync<5, GROUP>(); else named_sync<6, GROUP>();
                    E = e;
                }
                const float add = base + TN > vis_min ? row_sum<true>(S, cols, x.fz[h], x.vis, j) : row_sum<false>(S, cols, x.fz[h], x.vis, j);
                tc_before();
                bar_arrive(&x.bar[SE0 + h]);
                if (in) w[j] = old + add;
            }
        }
        tc_before();
        named_sync<2, 2 * GROUP>();
        if (warp == 0) {
            tc_after();
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tm), "r"(TMEM_COLS));
        }
    } else if (warp < 16) {
        // -------------------------------------------------- cached rows: this group's steps into its stage
        const int y = (warp >> 2) & 1, t = tid & 127;
        uint8_t *tile = smem + L::K + y * L::KS;
        int32_t(*row)[TN] = x.row[y];
        auto sync = [&] {
            if (y == 0) named_sync<3, GROUP>(); else named_sync<4, GROUP>();
        };
        Lookup next; // of the step whose rows the group gets next
        int rs = y % max(steps, 1); // that step's place in the range
        auto look_up = [&](int i) {
            next.ask(p, q, r0 + rs * TN + t, i < jobs);
            rs += 2;
            while (rs >= steps && steps > 0) rs -= steps;
        };
        auto resolve = [&] { return max(next.row(p, g), 0); };
        if (y < jobs) {
            look_up(y);
            row[0][t] = resolve();
            look_up(y + 2);
            row[1][t] = resolve();
            look_up(y + 4);
            sync();
            int k = 0; // steps of this group done
            if constexpr (!CODES) {
                for (int i = y; i < jobs; i += 2, ++k) {
                    if (k > 0) bar_wait(&x.bar[KE0 + y], (k - 1) & 1, p.err, &x.abort);
                    copy_halves<D>(tile, p.kdata, row[k & 1], t);
                    sync();
                    row[k & 1][t] = resolve(); // of this group's step after next
                    look_up(i + 6);
                    asm volatile("cp.async.wait_group 0;" ::: "memory");
                    fence_async();
                    bar_arrive(&x.bar[KF0 + y]);
                    sync();
                }
            } else {
                using C = Codes<D, KT>;
                const int c = t % C::PIECES, j0 = t / C::PIECES;
                const uint8_t *codes = p.kdata + c * 16;
                uint32_t a[4];
                const bool f = C::swap(c);
                C::places(j0, c, a, f);
                uint4 u[C::PIECES];
                uint32_t sc[D / 64];
                int E = 0x7fffffff;
                int ps = y % steps; // the step's place in the range
                auto exponent = [&](int n, int s) { // of this group's n-th step (place s), whose scales are sc
                    uint32_t m = 0;
                    const bool in = r0 + s * TN + t < r1; // (rows that nobody sees have no say in the exponent)
#pragma unroll
                    for (int b = 0; b < D / QK; ++b) {
                        uint32_t v = sc[b >> 1] >> (16 * (b & 1)) & 0xffffu;
                        if (!in) v = 0;
                        if ((v & 0x7fffu) < 0x7c00u) m = max(m, v & 0x7fffu);
                        x.scale[y][n & 1][t * (D / QK) + b] = (uint16_t)v;
                    }
                    m = __reduce_max_sync(0xffffffffu, m);
                    if ((t & 31) == 0) x.red[y][n & 1][t >> 5] = m;
                    sync();
                    const uint4 r = *reinterpret_cast<const uint4 *>(x.red[y][n & 1]);
                    const uint32_t top = max(max(r.x, r.y), max(r.z, r.w));
                    const int e = top ? ilogbf(__half2float(__ushort_as_half((uint16_t)top))) : E_MIN;
                    if (E == 0x7fffffff || e > E + 4 || e < E - 4) E = e;
                    if (t == 0) x.kexp[y][n & 3] = E;
                };
                C::load(sc, p.ks, row[0][t]);
#pragma unroll
                for (int b = 0; b < C::PIECES; ++b) C::load(u[b], codes, row[0][j0 + b * C::ROWS]);
                exponent(0, ps);
                C::load(sc, p.ks, row[1][t]);
                for (int i = y; i < jobs; i += 2, ++k) {
                    if (k > 0) bar_wait(&x.bar[KE0 + y], (k - 1) & 1, p.err, &x.abort);
                    const float up = ldexpf(1.f, 3 - E);
                    // (scales and rows first: a shared load would wait for the stores before it)
                    const uint16_t *d = &x.scale[y][k & 1][j0 * (D / QK) + c / 2];
                    __half2 ds[C::PIECES];
                    int32_t R[C::PIECES];
#pragma unroll
                    for (int b = 0; b < C::PIECES; ++b) {
                        ds[b] = scaled(d[b * C::ROWS * (D / QK)], up);
                        R[b] = row[(k + 1) & 1][j0 + b * C::ROWS];
                    }
#pragma unroll
                    for (int b = 0; b < C::PIECES; ++b) {
                        store_parts<D>(tile + b * C::ROWS * 128, tile + L::KT + b * C::ROWS * 128, a, u[b], ds[b], f);
                        C::load(u[b], codes, R[b]); // (behind the last step: a row that is there)
                    }
                    fence_async();
                    bar_arrive(&x.bar[KF0 + y]);
                    if (i + 2 < jobs) {
                        row[k & 1][t] = resolve();
                        look_up(i + 6);
                        ps += 2;
                        while (ps >= steps) ps -= steps;
                        exponent(k + 1, ps); // (its barrier: the rows are there too)
                        C::load(sc, p.ks, row[k & 1][t]);
                    }
                }
            }
        }
    } else {
        regs_dec<R_MMA>();
        if (warp > 16 || lane > 0) return;
        // -------------------------------------------------- products
        const uint32_t sq = smem_u32(smem), sk = smem_u32(smem + L::K);
        int i = 0;
        for (int mg = 0; mg < groups && steps > 0; ++mg) {
            const int cols = (min(MG, m_all - mg * MG) + 15) / 16 * 16;
            bar_wait(&x.bar[QF], mg & 1, p.err, &x.abort);
            for (int s = 0; s < steps; ++s, ++i) {
                const int h = i & 1, k = i >> 1;
                bar_wait(&x.bar[KF0 + h], k & 1, p.err, &x.abort);
                if (k > 0) bar_wait(&x.bar[SE0 + h], (k - 1) & 1, p.err, &x.abort);
                tc_after();
                const uint32_t tS = tm + h * 256, kt = sk + h * L::KS, id = inst(cols, false);
                for (int n = 0; n < 1 + (CODES ? 1 : 0) + (LO ? 1 : 0); ++n) { // the parts' products, the largest first
                    const uint32_t ka = kt + (CODES && n == 1 ? L::KT : 0);
                    const uint32_t qa = sq + (LO && n == (CODES ? 2 : 1) ? L::QT : 0);
#pragma unroll
                    for (int d = 0; d < D / 16; ++d)
                        mma_ss(tS, desc(ka + (d >> 2) * (TN * 128) + (d & 3) * 32, 16),
                               desc(qa + (d >> 2) * (MG * 128) + (d & 3) * 32, 16), id, n > 0 || d > 0);
                }
                tc_commit(&x.bar[SF0 + h]);
                tc_commit(&x.bar[KE0 + h]);
            }
        }
        // nothing may be in flight when the CTA gives its memory back
        tc_commit(&x.bar[DRAIN]);
        const uint64_t t0 = now_ns();
        while (!bar_try(&x.bar[DRAIN], 0) && now_ns() - t0 < WAIT_NS) {
        }
    }
}

template <int D, int KT, bool LO> cudaError_t go(const BlockParams &p, cudaStream_t st) {
    auto k = weight_kernel<D, KT, LO>;
    constexpr int bytes = smem_bytes<D, KT != KVC_F16, LO>();
    static_assert(bytes <= 227 * 1024, "shared memory of a CTA");
    static SharedMemory set;
    cudaError_t e = set.allow((const void *)k, bytes, R_LAUNCH);
    if (e != cudaSuccess) return e;
    k<<<(unsigned)p.n_items, THREADS, bytes, st>>>(p);
    return cudaGetLastError();
}
template <int D, int KT> cudaError_t pick(const BlockParams &p, cudaStream_t st) {
    return p.act == KVC_ACT_F32 ? go<D, KT, true>(p, st) : go<D, KT, false>(p, st);
}

} // namespace

cudaError_t launch_weight(int type_k, const BlockParams &p, cudaStream_t st) {
    if (p.n_items <= 0) return cudaSuccess;
    if (p.D == 64) return type_k == KVC_F16 ? pick<64, KVC_F16>(p, st) : pick<64, KVC_Q8_0>(p, st);
    return type_k == KVC_F16 ? pick<128, KVC_F16>(p, st) : pick<128, KVC_Q8_0>(p, st);
}

} // namespace kvc
