// k_weight.cu - the attention weight that cached rows receive from a block of
// query tokens (kvc_attn_weight): for every KV head g and cached row j
//   w[g][j] += sum over tokens t that see j, query heads h of g:
//              exp(scale * q[t][h] . K_j - lse[t][h]),
// lse the statistics that the attention of the same tokens left behind.
//
// A work item is a KV head and a range of cached rows; its query rows (tokens x
// query heads of the group) lie in shared memory as fp16, up to MG of them at a
// time, for the whole range.  A warp owns 32 cached rows of a step of 256: it
// loads them straight into the operand layout of mma.m16n8k16 and keeps them
// while all query rows pass, so K is read once, scores never leave the
// registers, and a row's sum is one warp's: its order is fixed without atomics.
//   The products' order within a block of 32 values is free, so a quad's thread
// takes 8 consecutive ones of both operands: codes come as 8-byte loads, query
// rows as 16-byte shared loads.  Codes are exact in fp16 and so is a 16-bit
// query (32-bit ones are two parts): a block's partial score comes from the
// tensor cores, its scale is applied in 32 bits.
// What bounds it: few query rows, the bytes of K; many, the products (the
// register-operand tensor path, about 600 TFLOP/s here; tcgen05 would have to
// take K as two fp16 parts, and pad 160 query rows to 256, for the same
// accuracy, which comes to the same time).
#include "block_tile.cuh"

namespace kvc {
namespace {

constexpr int THREADS = 256, WARPS = THREADS / 32;
constexpr int NR = 32;            // cached rows of a warp's step
constexpr int STEP = WEIGHT_STEP; // of the CTA's
static_assert(STEP == WARPS * NR, "a step is every warp's rows");

template <int D, bool LO> struct Shape {
    static constexpr int MG = LO ? 128 : 256; // query rows in shared memory
    static constexpr int PITCH = D + 32;      // halves: rows 64 bytes off a multiple of 128, so a quarter warp's loads do not collide
    struct Smem {
        __half q[LO ? 2 : 1][MG][PITCH];
        float scale[MG];
        float lse[MG]; // in log2 units
        int32_t vis[MG];
    };
};

template <int D, int KT, bool LO>
__global__ void __launch_bounds__(THREADS, 1) weight_kernel(const __grid_constant__ BlockParams p) {
    using Sh = Shape<D, LO>;
    constexpr int NB = D / QK, NT = NR / 8;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    typename Sh::Smem &s = *reinterpret_cast<typename Sh::Smem *>(smem_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, gid = lane >> 2, qc = lane & 3;
    const BlockSeq q = p.seq[item_seq(p, (int)blockIdx.x)];
    int g, part, parts;
    item_unit(q, (int)blockIdx.x - q.item0, g, part, parts);
    const int m_all = q.n_tok * p.r;
    const int r0 = part * q.split_rows, r1 = parts == 1 ? q.n_rows : min(r0 + q.split_rows, q.n_rows);
    float *w = p.w + ((int64_t)q.w_index * p.Hk + g) * p.w_stride;

    for (int mg = 0; mg < m_all; mg += Sh::MG) {
        const int rows = min(Sh::MG, m_all - mg), tiles = (rows + 15) / 16;
        __syncthreads(); // the query rows before are done with
        constexpr int QR = 4;
        for (int mb = warp; mb < tiles * 16; mb += WARPS * QR) {
            float x[QR][D / 32];
            int vis[QR];
            float z[QR];
#pragma unroll
            for (int k = 0; k < QR; ++k) {
                const int m = mb + k * WARPS;
                vis[k] = query_load<D>(p, q, g, m < rows ? mg + m : m_all, m_all, lane, x[k]);
                z[k] = 0.f;
                if (m < rows && vis[k] > 0) {
                    const int t = (mg + m) / p.r, j = (mg + m) % p.r;
                    z[k] = p.lse[((int64_t)q.tok0 + t) * p.H + (int64_t)g * p.r + j] * 1.44269504f;
                }
            }
#pragma unroll
            for (int k = 0; k < QR; ++k) {
                const int m = mb + k * WARPS;
                if (m >= tiles * 16) break;
                uint32_t hi[D / 64], lo[D / 64];
                const float scale = query_pack<D, LO>(p, x[k], hi, lo);
#pragma unroll
                for (int i = 0; i < D / 64; ++i) {
                    *reinterpret_cast<uint32_t *>(&s.q[0][m][lane * (D / 32) + 2 * i]) = hi[i];
                    if (LO) *reinterpret_cast<uint32_t *>(&s.q[LO][m][lane * (D / 32) + 2 * i]) = lo[i];
                }
                if (lane == 0) {
                    s.scale[m] = scale;
                    s.lse[m] = z[k];
                    s.vis[m] = vis[k];
                }
            }
        }
        __syncthreads();

        for (int base = r0 + warp * NR; base < r1; base += STEP) {
            // the warp's rows: lane l looks row l up
            const int32_t R = max(base + lane < r1 ? pool_row(p, q, g, base + lane) : 0, 0);
            uint32_t kb[NT][NB][4]; // [8 rows][block of 32 values][operand registers of two products]
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const int64_t Rn = __shfl_sync(0xffffffffu, R, n * 8 + gid);
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    if constexpr (KT == KVC_F16) {
                        const uint4 u = __ldg(reinterpret_cast<const uint4 *>(p.kdata + Rn * (2 * D)) + b * 4 + qc);
                        kb[n][b][0] = u.x, kb[n][b][1] = u.y, kb[n][b][2] = u.z, kb[n][b][3] = u.w;
                    } else {
                        const uint2 u = __ldg(reinterpret_cast<const uint2 *>(p.kdata + Rn * D) + b * 4 + qc);
                        const uint2 lo = codes4(u.x), hi = codes4(u.y);
                        kb[n][b][0] = lo.x, kb[n][b][1] = lo.y, kb[n][b][2] = hi.x, kb[n][b][3] = hi.y;
                    }
                }
            }
            uint32_t ds[NT][NB]; // scales of the rows 2 qc and 2 qc + 1 of each eight, a half each
            if constexpr (KT != KVC_F16) {
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const int64_t Ra = __shfl_sync(0xffffffffu, R, n * 8 + qc * 2), Rb = __shfl_sync(0xffffffffu, R, n * 8 + qc * 2 + 1);
                    uint32_t a[NB / 2], c[NB / 2];
#pragma unroll
                    for (int b = 0; b < NB / 2; ++b) {
                        a[b] = __ldg(reinterpret_cast<const uint32_t *>(p.ks + Ra * NB) + b);
                        c[b] = __ldg(reinterpret_cast<const uint32_t *>(p.ks + Rb * NB) + b);
                    }
#pragma unroll
                    for (int b = 0; b < NB; ++b) ds[n][b] = __byte_perm(a[b / 2], c[b / 2], b & 1 ? 0x7632 : 0x5410);
                }
            }
            float acc[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n) acc[n][0] = acc[n][1] = 0.f;
#pragma unroll 1
            for (int mt = 0; mt < tiles; ++mt) {
                const int ma = mt * 16 + gid;
                const int va = s.vis[ma] - base, vb = s.vis[ma + 8] - base;
                if (!__any_sync(0xffffffffu, va > 0 || vb > 0)) continue; // none of these tokens sees the rows
                float sc[NT][4];
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int k = 0; k < 4; ++k) sc[n][k] = 0.f;
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    float t[NT][4];
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int k = 0; k < 4; ++k) t[n][k] = 0.f;
#pragma unroll
                    for (int l = 0; l < (LO ? 2 : 1); ++l) {
                        const uint4 x = *reinterpret_cast<const uint4 *>(&s.q[l][ma][b * 32 + qc * 8]);
                        const uint4 y = *reinterpret_cast<const uint4 *>(&s.q[l][ma + 8][b * 32 + qc * 8]);
                        const uint32_t a0[4] = {x.x, y.x, x.y, y.y}, a1[4] = {x.z, y.z, x.w, y.w};
#pragma unroll
                        for (int n = 0; n < NT; ++n) mma(t[n], a0, kb[n][b][0], kb[n][b][1]);
#pragma unroll
                        for (int n = 0; n < NT; ++n) mma(t[n], a1, kb[n][b][2], kb[n][b][3]);
                    }
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        if constexpr (KT != KVC_F16) {
                            const float2 d = f2(ds[n][b]);
                            sc[n][0] = fmaf(t[n][0], d.x, sc[n][0]);
                            sc[n][1] = fmaf(t[n][1], d.y, sc[n][1]);
                            sc[n][2] = fmaf(t[n][2], d.x, sc[n][2]);
                            sc[n][3] = fmaf(t[n][3], d.y, sc[n][3]);
                        } else {
#pragma unroll
                            for (int k = 0; k < 4; ++k) sc[n][k] += t[n][k];
                        }
                    }
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float f = s.scale[ma + 8 * h], z = s.lse[ma + 8 * h];
                    const int v = h ? vb : va;
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const float e = ex2(fmaf(sc[n][2 * h + k], f, -z));
                            acc[n][k] += n * 8 + qc * 2 + k < v ? e : 0.f;
                        }
                }
            }
            // over the eight row groups; then lane l has cached row l's sum
            float mine = 0.f;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) acc[n][k] += __shfl_xor_sync(0xffffffffu, acc[n][k], o);
                    const float x = __shfl_sync(0xffffffffu, acc[n][k], (lane & 7) >> 1);
                    if ((lane >> 3) == n && (lane & 1) == k) mine = x;
                }
            if (base + lane < r1) w[base + lane] += mine;
        }
    }
}

template <int D, int KT, bool LO> cudaError_t go(const BlockParams &p, cudaStream_t st) {
    auto k = weight_kernel<D, KT, LO>;
    const int bytes = (int)sizeof(typename Shape<D, LO>::Smem);
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
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
