// k_cross.cu - attention of a block of query tokens over cached rows
// (kvc_attn_cross): every token t of a sequence attends over its leading
// N_t = min(max(n_vis[t], 0), rows) cached rows,
//   s_j = scale * q[t][h] . K_j,   lse = log sum_j exp(s_j),
//   out = sum_j exp(s_j - lse) V_j        (j < N_t; 0 and -inf where N_t = 0),
// query head h reading KV head h / r.
//
// A work item is one KV head, one tile of up to 64 query rows (tokens x query
// heads of the group) and a part of the cached rows, walked in steps of 64.
// A step's rows are turned into fp16 in shared memory once for all warps; the
// products run on the tensor cores with fp32 sums and the softmax is the
// online one, so no score leaves the registers.
//   q8_0 and q4_0 codes are exact in fp16.  The scale of a 32-value block of K
//   multiplies the block's own partial score in 32 bits; the scale of a block
//   of V goes into the probabilities, P' = p * d * 2^(12 - E), E the exponent
//   of the largest V scale met so far (the sums are rescaled when it grows),
//   which keeps P' in the normal range of fp16 for scales of any size.
//   With 32-bit queries P' is split into two fp16 parts (22 bits), so that
//   32-bit results keep 32-bit accuracy.  With 16-bit results P' is one fp16
//   value: its rounding (at most 2^-11) averages out over the rows, below the
//   result's own.
// Rows behind the sequence's last and rows that a token does not see take no
// part, whatever they hold: scores are selected, not added to, and a
// non-finite V value is kept out of the products (0 x inf is NaN) and put into
// the result only of rows that see it.
// Few query tiles: the cached rows are split over items, and a second kernel
// joins their partial sums in order, so a result does not depend on the order in
// which items finish.
// It runs 32-bit queries, and 16-bit ones where the tcgen05 kernel does not pay
// (block_attn.cu has the rule).  What bounds it: the register-operand tensor
// path with many query rows (257 tokens of 40 heads over 4999 rows, q8_0 / q4_0,
// 32-bit: two products each, 262 us, 100 TFLOP/s of results), its start and one
// chain of steps with few (one token of 8 heads over 512 rows: 8.6 us).
#include "block_tile.cuh"

namespace kvc {
namespace {

constexpr int THREADS = BLOCK_THREADS;
constexpr int TM = CROSS_TILE_M, TN = CROSS_TILE_N;
constexpr int E_MIN = -24; // exponent of the smallest fp16 scale

template <int D, int KT, int VT, bool LO> struct Smem {
    static constexpr int PITCH = D + TILE_PAD;
    __half qhi[TM][PITCH];
    __half qlo[LO ? TM : 1][PITCH];
    __half k[TN][PITCH];
    __half v[TN][PITCH];
    uint8_t rawk[TN * row_bytes<KT>(D)]; // the next step's rows and block scales, as they are stored
    uint8_t rawv[TN * row_bytes<VT>(D)];
    uint16_t rks[TN * (D / QK)], rvs[TN * (D / QK)];
    float ks[D / QK][TN]; // block scales, by block
    float vs[D / QK][TN];
    int32_t row[2][TN];       // pool row of each row of a step, -1 past the end
    float qscale[TM];         // score per unit of the normalised product, in log2
    int32_t vis[TM];          // rows that the query row sees
    float red[THREADS / 32];
    float m[4][TM], l[4][TM]; // merge of warps that share query rows
    uint32_t poison[TM][D / 16]; // two bits a value: +inf, -inf (both: NaN) received
    uint8_t badrow[2][TN];
    int32_t vis_max;
    int32_t bad[2], any_bad;
};

// Requests 16 (or a row's scales: 8 or 4) bytes for shared memory; nothing is read, and zeros are written, where there is no row.
__device__ __forceinline__ void copy16(void *dst, const void *src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(in ? 16 : 0) : "memory");
}
template <int N> __device__ __forceinline__ void copy_scales(void *dst, const void *src, bool in) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(smem_u32(dst)), "l"(src), "n"(N), "r"(in ? N : 0) : "memory");
}
template <int RB> __device__ __forceinline__ void copy_rows(uint8_t *dst, const uint8_t *data, const int32_t *row, int tid) {
    constexpr int PIECES = RB / 16;
#pragma unroll
    for (int i = 0; i < TN * PIECES / THREADS; ++i) {
        const int at = tid + i * THREADS;
        const int32_t R = row[at / PIECES];
        copy16(dst + at * 16, data + (int64_t)max(R, 0) * RB + at % PIECES * 16, R >= 0);
    }
}

// Of a step's rows j < n that a query row sees, those that the quad's lane qc looks after and whose values were left out.
// (Out of line: in place it costs the step's registers, 10 % of 32-bit queries over f16 rows.)
template <int D, int T>
__device__ __noinline__ void mark_rows(uint32_t *words, const uint8_t *data, const uint16_t *scales, const int32_t *row,
                                       const uint8_t *badrow, int qc, int n) {
    for (int j = qc; j < n; j += 4)
        if (badrow[j] && row[j] >= 0) mark_poison<D, T>(words, data, scales, row[j]);
}

// WM: warps along the query rows (16 each); the 4 / WM warps of a row block
// share a step's cached rows and are joined at the end.  LO: 32-bit queries.
template <int D, int KT, int VT, int WM, bool LO>
__global__ void __launch_bounds__(THREADS, 2) cross_kernel(const __grid_constant__ BlockParams p) {
    constexpr int WN = 4 / WM, NC = TN / WN, NT = NC / 8, NB = D / QK;
    constexpr int MROWS = 16 * WM;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    using Sm = Smem<D, KT, VT, LO>;
    Sm &s = *reinterpret_cast<Sm *>(smem_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int wm = warp % WM, wn = warp / WM, gid = lane >> 2, qc = lane & 3;

    // the item: sequence, KV head, query tile, part of the rows
    const BlockSeq q = p.seq[item_seq(p, (int)blockIdx.x)];
    const int local = (int)blockIdx.x - q.item0;
    int unit, part, parts;
    item_unit(q, local, unit, part, parts);
    const int g = unit / q.tiles, tile = q.tiles - 1 - unit % q.tiles; // later tokens see more: they begin first
    const int m_all = q.n_tok * p.r, m0 = tile * MROWS, mrows = min(MROWS, m_all - m0);

    if (tid == 0) {
        s.vis_max = 0;
        s.any_bad = 0;
        s.bad[0] = s.bad[1] = 0;
    }
    __syncthreads();
    constexpr int QR = WM == 4 ? 8 : 4; // of a warp's rows, under way together
    for (int mb = warp; mb < MROWS; mb += THREADS / 32 * QR) {
        Query<D> y[QR];
#pragma unroll
        for (int k = 0; k < QR; ++k) y[k].ask(p, q, g, m0 + mb + k * (THREADS / 32), m_all, lane);
#pragma unroll
        for (int k = 0; k < QR; ++k) {
            const int m = mb + k * (THREADS / 32);
            float x[D / 32];
            uint32_t hi[D / 64], lo[D / 64];
            const int vis = y[k].get(p, q, x);
            const float scale = query_pack<D, LO>(p, x, hi, lo);
#pragma unroll
            for (int i = 0; i < D / 64; ++i) {
                *reinterpret_cast<uint32_t *>(&s.qhi[m][lane * (D / 32) + 2 * i]) = hi[i];
                if (LO) *reinterpret_cast<uint32_t *>(&s.qlo[m][lane * (D / 32) + 2 * i]) = lo[i];
            }
            if (lane == 0) {
                s.qscale[m] = scale;
                s.vis[m] = vis;
                if (vis > 0) atomicMax(&s.vis_max, vis);
            }
        }
    }
    for (int i = tid; i < MROWS * (D / 16); i += THREADS) s.poison[i / (D / 16)][i % (D / 16)] = 0;
    __syncthreads();
    const int r0 = part * q.split_rows;
    const int r1 = parts == 1 ? s.vis_max : min(r0 + q.split_rows, s.vis_max);

    float o[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[i][k] = 0.f;
    float mx[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f};
    int E = VT == KVC_F16 ? 0 : E_MIN;
    const int mrow = wm * 16 + gid;
    const float qs[2] = {s.qscale[mrow], s.qscale[mrow + 8]};
    const int vis[2] = {s.vis[mrow], s.vis[mrow + 8]};

    // A step's rows come while the step before is computed (as they are stored: they are turned into fp16 once for all
    // warps), their places in the pool a step earlier still; a page that the pool does not have is reported, its rows are left out.
    Lookup next;
    auto request = [&](int i) {
        const int32_t *row = s.row[i & 1];
        copy_rows<row_bytes<KT>(D)>(s.rawk, p.kdata, row, tid);
        copy_rows<row_bytes<VT>(D)>(s.rawv, p.vdata, row, tid);
        const int j = tid & (TN - 1);
        const int32_t R = row[j];
        if (KT != KVC_F16 && tid < TN) copy_scales<NB * 2>(&s.rks[j * NB], p.ks + (int64_t)max(R, 0) * NB, R >= 0);
        if (VT != KVC_F16 && tid >= TN) copy_scales<NB * 2>(&s.rvs[j * NB], p.vs + (int64_t)max(R, 0) * NB, R >= 0);
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    if (r0 < r1) {
        if (tid < TN) {
            s.row[0][tid] = pool_row(p, q, g, r0 + tid);
            s.badrow[0][tid] = 0;
            next.ask(p, q, r0 + TN + tid, true);
        }
        __syncthreads();
        request(0);
    }
    for (int base = r0, step = 0; base < r1; base += TN, ++step) {
        const int cur = step & 1;
        const int32_t *row = s.row[cur];
        const uint8_t *badrow = s.badrow[cur];
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads(); // the step's rows are there, the tiles of the step before are done with
        if (tid < TN) {
            s.row[cur ^ 1][tid] = next.row(p, g);
            s.badrow[cur ^ 1][tid] = 0;
        }
        if (tid == 0) s.bad[cur ^ 1] = 0;
        fill<D, KT, false>(s.k, s.rawk, nullptr, tid);
        bool bad = fill<D, VT, true>(s.v, s.rawv, s.badrow[cur], tid);
        float top = 0.f;
        if constexpr (KT != KVC_F16 || VT != KVC_F16) {
            for (int i = tid; i < TN * NB; i += THREADS) {
                const int j = i / NB, b = i % NB;
                if constexpr (KT != KVC_F16) s.ks[b][j] = __half2float(__ushort_as_half(s.rks[i]));
                if constexpr (VT != KVC_F16) {
                    float d = base + j < r1 ? __half2float(__ushort_as_half(s.rvs[i])) : 0.f; // (nobody sees it: no say in E)
                    if (!(fabsf(d) <= 65504.f)) {
                        d = 0.f;
                        s.badrow[cur][j] = 1;
                        bad = true;
                    }
                    s.vs[b][j] = d;
                    top = fmaxf(top, fabsf(d));
                }
            }
#pragma unroll
            for (int x = 16; x; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
            if (lane == 0) s.red[warp] = top;
        }
        if (bad) s.bad[cur] = 1;
        __syncthreads();
        if (base + TN < r1) {
            request(step + 1);
            if (tid < TN) next.ask(p, q, base + 2 * TN + tid, true);
        }
        float grow = 1.f; // factor of the sums so far when the range exponent grows
        if constexpr (VT != KVC_F16) {
            top = fmaxf(fmaxf(s.red[0], s.red[1]), fmaxf(s.red[2], s.red[3]));
            int e = E_MIN;
            if (top > 0.f) e = max(E_MIN, ilogbf(top));
            if (e > E) {
                grow = ldexpf(1.f, max(E - e, -126));
                E = e;
            }
        }

        // scores of 16 query rows x NC cached rows
        float sc[NT][4];
        scores<D, KT, NT, LO>(sc, smem_u32(&s.qhi[wm * 16 + (lane & 15)][(lane >> 4) * 8]),
                              smem_u32(&s.qlo[wm * 16 + (lane & 15)][(lane >> 4) * 8]),
                              smem_u32(&s.k[wn * NC + (lane & 7) + ((lane >> 4) << 3)][((lane >> 3) & 1) * 8]), s.ks,
                              wn * NC + qc * 2);
        // scale, mask, online softmax
        float nm[2] = {mx[0], mx[1]};
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int jt = wn * NC + n * 8 + qc * 2 + (k & 1);
                const float x = sc[n][k] * qs[k >> 1];
                sc[n][k] = base + jt < vis[k >> 1] && row[jt] >= 0 ? x : -INFINITY;
                nm[k >> 1] = fmaxf(nm[k >> 1], sc[n][k]);
            }
        float al[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            nm[h] = fmaxf(nm[h], __shfl_xor_sync(0xffffffffu, nm[h], 1));
            nm[h] = fmaxf(nm[h], __shfl_xor_sync(0xffffffffu, nm[h], 2));
            const float use = nm[h] == -INFINITY ? 0.f : nm[h];
            al[h] = ex2(mx[h] - use); // nothing yet: ex2(-inf) = 0
            mx[h] = nm[h];
            float add = 0.f;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float e = ex2(sc[n][2 * h + k] - use);
                    sc[n][2 * h + k] = e;
                    add += e;
                }
            sum[h] = sum[h] * al[h] + add;
            al[h] *= grow;
        }
        if (s.bad[cur]) { // a V value of this step is not finite: it goes to the rows that see it, of whatever weight
            for (int h = 0; h < 2; ++h)
                mark_rows<D, VT>(s.poison[mrow + 8 * h], p.vdata, p.vs, row + wn * NC, badrow + wn * NC, qc,
                                 min(s.vis[mrow + 8 * h] - base - wn * NC, NC));
            s.any_bad = 1;
        }
        // P V, a 32-value block of V at a time.  The tensor cores truncate their sums, so a chain of products is no
        // longer than the step: its sum is added, with the old ones' rescaling, by a rounded 32-bit operation.
        const float fe = VT == KVC_F16 ? 4096.f : ldexpf(1.f, 12 - E);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int k = 0; k < 4; ++k) sc[n][k] *= fe;
        uint32_t pa[NC / 16][4], plo[LO ? NC / 16 : 1][4];
        auto split = [&](int ks, const float (&y)[8]) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                pa[ks][k] = h2(y[2 * k], y[2 * k + 1]);
                if constexpr (LO) {
                    const float2 f = f2(pa[ks][k]);
                    plo[ks][k] = h2(y[2 * k] - f.x, y[2 * k + 1] - f.y);
                }
            }
        };
        if constexpr (VT == KVC_F16) {
#pragma unroll
            for (int ks = 0; ks < NC / 16; ++ks) {
                const float y[8] = {sc[2 * ks][0], sc[2 * ks][1], sc[2 * ks][2], sc[2 * ks][3],
                                    sc[2 * ks + 1][0], sc[2 * ks + 1][1], sc[2 * ks + 1][2], sc[2 * ks + 1][3]};
                split(ks, y);
            }
        }
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            float t[4][4];
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int k = 0; k < 4; ++k) t[n][k] = 0.f;
#pragma unroll
            for (int ks = 0; ks < NC / 16; ++ks) {
                if constexpr (VT != KVC_F16) {
                    const int j = wn * NC + ks * 16 + qc * 2;
                    const float2 d0 = *reinterpret_cast<const float2 *>(&s.vs[b][j]);
                    const float2 d1 = *reinterpret_cast<const float2 *>(&s.vs[b][j + 8]);
                    const float y[8] = {sc[2 * ks][0] * d0.x, sc[2 * ks][1] * d0.y, sc[2 * ks][2] * d0.x,
                                        sc[2 * ks][3] * d0.y, sc[2 * ks + 1][0] * d1.x, sc[2 * ks + 1][1] * d1.y,
                                        sc[2 * ks + 1][2] * d1.x, sc[2 * ks + 1][3] * d1.y};
                    split(ks, y);
                }
                const uint32_t va = smem_u32(&s.v[wn * NC + ks * 16 + (lane & 15)][(lane >> 4) * 8]) + b * 64;
#pragma unroll
                for (int n = 0; n < 4; n += 2) {
                    uint32_t vb[4];
                    ldsm4t(vb, va + n * 16);
                    mma(t[n], pa[ks], vb[0], vb[1]);
                    mma(t[n + 1], pa[ks], vb[2], vb[3]);
                    if constexpr (LO) {
                        mma(t[n], plo[ks], vb[0], vb[1]);
                        mma(t[n + 1], plo[ks], vb[2], vb[3]);
                    }
                }
            }
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int k = 0; k < 4; ++k) o[b * 4 + n][k] = fmaf(o[b * 4 + n][k], al[k >> 1], t[n][k]);
        }
    }
    __syncthreads();

    // the quad's sums, then the values themselves
    const float back = VT == KVC_F16 ? 1.f / 4096.f : ldexpf(1.f, E - 12);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        sum[h] += __shfl_xor_sync(0xffffffffu, sum[h], 1);
        sum[h] += __shfl_xor_sync(0xffffffffu, sum[h], 2);
    }
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[i][k] *= back;
    if constexpr (WN > 1) {
        // warps that share query rows: joined in warp order by the first of them, through the tiles' memory
        __syncthreads();
        float *buf = reinterpret_cast<float *>(&s.k[0][0]); // [WN - 1][MROWS][D]
        static_assert(sizeof(float) * (WN - 1) * MROWS * D <= sizeof(__half) * 2 * TN * Sm::PITCH, "merge buffer");
        if (qc == 0) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                s.m[wn][mrow + 8 * h] = mx[h];
                s.l[wn][mrow + 8 * h] = sum[h];
            }
        }
        if (wn > 0) {
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    *reinterpret_cast<float2 *>(&buf[((wn - 1) * MROWS + mrow + 8 * h) * D + i * 8 + qc * 2]) =
                        make_float2(o[i][2 * h], o[i][2 * h + 1]);
        }
        __syncthreads();
        if (wn == 0) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int m = mrow + 8 * h;
                float M = mx[h];
#pragma unroll
                for (int w = 1; w < WN; ++w) M = fmaxf(M, s.m[w][m]);
                const float use = M == -INFINITY ? 0.f : M;
                const float f0 = ex2(mx[h] - use);
                float L = sum[h] * f0;
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    o[i][2 * h] *= f0;
                    o[i][2 * h + 1] *= f0;
                }
#pragma unroll
                for (int w = 1; w < WN; ++w) {
                    const float f = ex2(s.m[w][m] - use);
                    L += s.l[w][m] * f;
#pragma unroll
                    for (int i = 0; i < D / 8; ++i) {
                        const float2 x =
                            *reinterpret_cast<const float2 *>(&buf[((w - 1) * MROWS + m) * D + i * 8 + qc * 2]);
                        o[i][2 * h] = fmaf(x.x, f, o[i][2 * h]);
                        o[i][2 * h + 1] = fmaf(x.y, f, o[i][2 * h + 1]);
                    }
                }
                mx[h] = M;
                sum[h] = L;
            }
        }
    }
    const bool bad = s.any_bad != 0;
    const bool whole = parts == 1;
    const int prow = q.part_row0 + (local - q.whole) * p.part_rows; // the item's partial rows
    if (wn == 0) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int m = mrow + 8 * h;
            if (m >= mrows) continue;
            if (bad) {
#pragma unroll
                for (int i = 0; i < D / 8; ++i)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int d = i * 8 + qc * 2 + k;
                        o[i][2 * h + k] = poisoned(o[i][2 * h + k], (s.poison[m][d / 16] >> (2 * (d % 16))) & 3u);
                    }
            }
            if (whole) {
                const int t = token_of(p, m0 + m), j = m0 + m - t * p.r;
                const int64_t head = ((int64_t)q.tok0 + t) * p.H + (int64_t)g * p.r + j;
                const float inv = sum[h] == 0.f ? 0.f : 1.f / sum[h];
#pragma unroll
                for (int i = 0; i < D / 8; ++i)
                    store2(p.out, p.act, head * D + i * 8 + qc * 2, o[i][2 * h] * inv, o[i][2 * h + 1] * inv);
                if (p.lse && qc == 0)
                    p.lse[head] = sum[h] == 0.f ? -INFINITY : mx[h] * 0.6931471805599453f + logf(sum[h]);
            } else {
                float *dst = p.part + (int64_t)(prow + m) * D;
#pragma unroll
                for (int i = 0; i < D / 8; ++i)
                    *reinterpret_cast<float2 *>(dst + i * 8 + qc * 2) = make_float2(o[i][2 * h], o[i][2 * h + 1]);
                if (qc == 0)
                    *reinterpret_cast<float2 *>(p.part + p.part_cap * D + 2 * (int64_t)(prow + m)) =
                        make_float2(mx[h], sum[h]);
            }
        }
    }
}

template <int D, int KT, int VT, int WM, bool LO> cudaError_t go(const BlockParams &p, cudaStream_t st) {
    auto k = cross_kernel<D, KT, VT, WM, LO>;
    const int bytes = (int)sizeof(Smem<D, KT, VT, LO>);
    static SharedMemory set;
    cudaError_t e = set.allow((const void *)k, bytes);
    if (e != cudaSuccess) return e;
    k<<<(unsigned)p.n_items, THREADS, bytes, st>>>(p);
    e = cudaGetLastError();
    return e == cudaSuccess ? launch_join(p, st) : e;
}
template <int D, int KT, int VT> cudaError_t pick(const BlockParams &p, bool narrow, cudaStream_t st) {
    const bool lo = p.act == KVC_ACT_F32;
    if (narrow) return lo ? go<D, KT, VT, 1, true>(p, st) : go<D, KT, VT, 1, false>(p, st);
    return lo ? go<D, KT, VT, 4, true>(p, st) : go<D, KT, VT, 4, false>(p, st);
}

} // namespace

cudaError_t launch_cross(int type_k, int type_v, const BlockParams &p, bool narrow, cudaStream_t st) {
    if (p.n_items <= 0) return cudaSuccess;
    if (p.D == 64) {
        if (type_k == KVC_F16) return pick<64, KVC_F16, KVC_F16>(p, narrow, st);
        return pick<64, KVC_Q8_0, KVC_Q8_0>(p, narrow, st);
    }
    if (type_k == KVC_F16) return pick<128, KVC_F16, KVC_F16>(p, narrow, st);
    if (type_v == KVC_Q4_0) return pick<128, KVC_Q8_0, KVC_Q4_0>(p, narrow, st);
    return pick<128, KVC_Q8_0, KVC_Q8_0>(p, narrow, st);
}

} // namespace kvc
