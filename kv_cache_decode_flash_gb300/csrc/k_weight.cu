// k_weight.cu - the attention weight that cached rows receive from a block of
// query tokens (kvc_attn_weight): for every KV head g and cached row j
//   w[g][j] += sum over tokens t that see j, query heads h of g:
//              exp(scale * q[t][h] . K_j - lse[t][h]),
// lse the statistics that the attention of the same tokens left behind.
//
// One CTA owns 64 cached rows of a KV head: their K is turned into fp16 in
// shared memory once and all query rows (tokens x query heads of the group)
// pass over it in tiles of 64, so K is read once and no weight is added by two
// CTAs: the sum's order is fixed and needs no atomics.  Scores come from the
// tensor cores as exactly as 32-bit sums are (block_tile.cuh); the sums over
// query rows stay in registers until the end.
#include "block_tile.cuh"

namespace kvc {
namespace {

constexpr int THREADS = BLOCK_THREADS;
constexpr int TM = CROSS_TILE_M, TN = CROSS_TILE_N;

template <int D> struct Smem {
    __half qhi[TM][D + TILE_PAD];
    __half qlo[TM][D + TILE_PAD];
    __half k[TN][D + TILE_PAD];
    float ks[D / QK][TN];
    int32_t row[TN];
    float qscale[TM];
    float lse[TM]; // in log2 units
    int32_t vis[TM];
    float sum[4][TN];
    int32_t vis_max;
};

// WM: warps along the query rows; the 4 / WM warps of a row block share the cached rows.
template <int D, int KT, int WM, bool LO>
__global__ void __launch_bounds__(THREADS) weight_kernel(const __grid_constant__ BlockParams p) {
    constexpr int WN = 4 / WM, NC = TN / WN, NT = NC / 8, NB = D / QK, MROWS = 16 * WM;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    Smem<D> &s = *reinterpret_cast<Smem<D> *>(smem_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int wm = warp % WM, wn = warp / WM, gid = lane >> 2, qc = lane & 3;
    const BlockSeq q = p.seq[item_seq(p, (int)blockIdx.x)];
    const int local = (int)blockIdx.x - q.item0;
    const int g = local / q.splits, base = (local % q.splits) * TN;
    const int m_all = q.n_tok * p.r;

    if (tid < TN) s.row[tid] = pool_row(p, q, g, base + tid);
    __syncthreads();
    fill<D, KT, false>(s.k, p.kdata, s.row, nullptr, tid);
    if constexpr (KT != KVC_F16)
        for (int i = tid; i < TN * NB; i += THREADS) {
            const int32_t R = s.row[i / NB];
            s.ks[i % NB][i / NB] = R >= 0 ? __half2float(__ushort_as_half(p.ks[(int64_t)R * NB + i % NB])) : 0.f;
        }
    float acc[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[n][0] = acc[n][1] = 0.f;
    const int mrow = wm * 16 + gid;
    for (int m0 = 0; m0 < m_all; m0 += MROWS) {
        __syncthreads(); // the tile before is done with the query rows
        if (tid == 0) s.vis_max = 0;
        __syncthreads();
        for (int m = warp; m < MROWS; m += THREADS / 32) {
            float x[D / 32];
            uint32_t hi[D / 64], lo[D / 64];
            const int vis = query_load<D>(p, q, g, m0 + m, m_all, lane, x);
            const float scale = query_pack<D, LO>(p, x, hi, lo);
#pragma unroll
            for (int i = 0; i < D / 64; ++i) {
                *reinterpret_cast<uint32_t *>(&s.qhi[m][lane * (D / 32) + 2 * i]) = hi[i];
                if (LO) *reinterpret_cast<uint32_t *>(&s.qlo[m][lane * (D / 32) + 2 * i]) = lo[i];
            }
            if (lane == 0) {
                s.qscale[m] = scale;
                s.vis[m] = vis;
                float z = 0.f;
                if (vis > base) {
                    const int t = (m0 + m) / p.r, j = (m0 + m) % p.r;
                    z = p.lse[((int64_t)q.tok0 + t) * p.H + (int64_t)g * p.r + j] * 1.44269504f;
                    atomicMax(&s.vis_max, vis);
                }
                s.lse[m] = z;
            }
        }
        __syncthreads();
        if (s.vis_max <= base) continue; // none of these tokens sees the rows
        float sc[NT][4];
        scores<D, KT, NT, LO>(sc, smem_u32(&s.qhi[wm * 16 + (lane & 15)][(lane >> 4) * 8]),
                              smem_u32(&s.qlo[wm * 16 + (lane & 15)][(lane >> 4) * 8]),
                              smem_u32(&s.k[wn * NC + (lane & 7) + ((lane >> 4) << 3)][((lane >> 3) & 1) * 8]), s.ks,
                              wn * NC + qc * 2);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float qs = s.qscale[mrow + 8 * h], z = s.lse[mrow + 8 * h];
            const int vis = s.vis[mrow + 8 * h] - base;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int jt = wn * NC + n * 8 + qc * 2 + k;
                    const float e = ex2(fmaf(sc[n][2 * h + k], qs, -z));
                    acc[n][k] += jt < vis ? e : 0.f;
                }
        }
    }
    // over the query rows of a warp, then over the warps that share the cached rows
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) acc[n][k] += __shfl_xor_sync(0xffffffffu, acc[n][k], o);
            if (gid == 0) s.sum[wm][wn * NC + n * 8 + qc * 2 + k] = acc[n][k];
        }
    __syncthreads();
    if (tid < TN && s.row[tid] >= 0) {
        float add = s.sum[0][tid];
#pragma unroll
        for (int w = 1; w < WM; ++w) add += s.sum[w][tid];
        float *dst = p.w + ((int64_t)q.w_index * p.Hk + g) * p.w_stride + base + tid;
        *dst += add;
    }
}

template <int D, int KT, int WM, bool LO> cudaError_t go(const BlockParams &p, cudaStream_t st) {
    auto k = weight_kernel<D, KT, WM, LO>;
    const int bytes = (int)sizeof(Smem<D>);
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    k<<<(unsigned)p.n_items, THREADS, bytes, st>>>(p);
    return cudaGetLastError();
}
template <int D, int KT> cudaError_t pick(const BlockParams &p, bool narrow, cudaStream_t st) {
    const bool lo = p.act == KVC_ACT_F32;
    if (narrow) return lo ? go<D, KT, 1, true>(p, st) : go<D, KT, 1, false>(p, st);
    return lo ? go<D, KT, 4, true>(p, st) : go<D, KT, 4, false>(p, st);
}

} // namespace

cudaError_t launch_weight(int type_k, const BlockParams &p, bool narrow, cudaStream_t st) {
    if (p.n_items <= 0) return cudaSuccess;
    if (p.D == 64) return type_k == KVC_F16 ? pick<64, KVC_F16>(p, narrow, st) : pick<64, KVC_Q8_0>(p, narrow, st);
    return type_k == KVC_F16 ? pick<128, KVC_F16>(p, narrow, st) : pick<128, KVC_Q8_0>(p, narrow, st);
}

} // namespace kvc
