// k_join.cu - the block attention's second kernel where cached rows were split
// over work items: joins the parts' sums of every query row, in their order:
//   M = max m_i,  L = sum l_i 2^(m_i - M),  out = sum o_i 2^(m_i - M) / L.
// One warp a query row, a lane D / 32 columns.  The partial sums were just
// written and are in L2; what bounds this is the latency of its loads, so all SMs
// take part and a warp has those of eight parts under way together.  (Joining in
// the part that arrived last left one SM per unit to read all of it: 16384 rows,
// 50 tokens of 40 heads, 19 parts took 120 us that way.)
#include "block_tile.cuh"

namespace kvc {
namespace {

constexpr int JOIN_THREADS = 128, JOIN_ROWS = JOIN_THREADS / 32, AHEAD = 8;

template <int D> __global__ void __launch_bounds__(JOIN_THREADS) join_kernel(const __grid_constant__ BlockParams p, int chunks) {
    constexpr int V = D / 32;
    const int cut = (int)blockIdx.x / chunks, lane = threadIdx.x & 31;
    int lo = 0, hi = p.n_seq - 1;
    while (lo < hi) { // the last sequence whose first cut unit is not behind ours
        const int mid = (lo + hi + 1) / 2;
        if (p.seq[mid].cut0 <= cut) lo = mid; else hi = mid - 1;
    }
    const BlockSeq q = p.seq[lo];
    const int unit = q.whole + cut - q.cut0, parts = q.splits;
    const int g = unit / q.tiles, m0 = (q.tiles - 1 - unit % q.tiles) * p.tile_m;
    const int m = (int)blockIdx.x % chunks * JOIN_ROWS + (threadIdx.x >> 5);
    if (m >= min(p.tile_m, q.n_tok * p.r - m0)) return;
    const int64_t row0 = (int64_t)q.part_row0 + (int64_t)(cut - q.cut0) * parts * p.part_rows + m;
    const float2 *ml = reinterpret_cast<const float2 *>(p.part + p.part_cap * D);
    float M = -INFINITY, L = 0.f, o[V];
#pragma unroll
    for (int e = 0; e < V; ++e) o[e] = 0.f;
    for (int i = lane; i < parts; i += 32) M = fmaxf(M, ml[row0 + (int64_t)i * p.part_rows].x);
#pragma unroll
    for (int x = 16; x; x >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
    if (M == -INFINITY) M = 0.f;
    for (int i0 = 0; i0 < parts; i0 += AHEAD) {
        float2 c[AHEAD];
        float v[AHEAD][V];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int64_t row = row0 + (int64_t)min(i0 + i, parts - 1) * p.part_rows;
            c[i] = ml[row];
            if constexpr (V == 4) {
                const float4 f = reinterpret_cast<const float4 *>(p.part + row * D)[lane];
                v[i][0] = f.x, v[i][1] = f.y, v[i][2] = f.z, v[i][3] = f.w;
            } else {
                const float2 f = reinterpret_cast<const float2 *>(p.part + row * D)[lane];
                v[i][0] = f.x, v[i][1] = f.y;
            }
        }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const float f = ex2(c[i].x - M);
            // nothing seen there, or nothing left of it (its sums may be anything)
            const bool skip = i0 + i >= parts || c[i].y == 0.f || (f == 0.f && c[i].y == c[i].y);
            if (skip) continue;
            L = fmaf(c[i].y, f, L);
#pragma unroll
            for (int e = 0; e < V; ++e) o[e] = fmaf(v[i][e], f, o[e]);
        }
    }
    const int t = token_of(p, m0 + m), j = m0 + m - t * p.r;
    const int64_t head = ((int64_t)q.tok0 + t) * p.H + (int64_t)g * p.r + j;
    const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
    for (int e = 0; e < V; e += 2) store2(p.out, p.act, head * D + lane * V + e, o[e] * inv, o[e + 1] * inv);
    if (p.lse && lane == 0) p.lse[head] = L == 0.f ? -INFINITY : M * 0.6931471805599453f + logf(L);
}

} // namespace

cudaError_t launch_join(const BlockParams &p, cudaStream_t st) {
    if (p.n_cut <= 0) return cudaSuccess;
    const int chunks = (p.part_rows + JOIN_ROWS - 1) / JOIN_ROWS;
    const unsigned grid = (unsigned)p.n_cut * (unsigned)chunks;
    if (p.D == 64)
        join_kernel<64><<<grid, JOIN_THREADS, 0, st>>>(p, chunks);
    else
        join_kernel<128><<<grid, JOIN_THREADS, 0, st>>>(p, chunks);
    return cudaGetLastError();
}

} // namespace kvc
