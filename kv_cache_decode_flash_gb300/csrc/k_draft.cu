// k_draft.cu - the two kernels around the attention over a drafted block.
//
// rope_append (kvc_append_rope): a token's head-rows come as the projections
// leave them, n = x * w / sqrt(mean(x^2) + eps) where a norm's weights are given, and
//   (a, b) -> (a cos - b sin, a sin + b cos),  angle = pos * base^(-2i/D),
// of its queries and keys; queries are handed back in their own type, keys and
// values become the sequence's next row, quantised by the steps of quant_row.cuh.
// Everything is fp32 from the load to the one rounding at the end.
//  A warp takes 2 (D 128) or 4 (D 64) head-rows at a time: a lane has four
// values of a row's first half and the four that are D/2 further, so that the pairs of
// either pairing and the halves of a quantisation block of 8 lanes are its
// own.  The angles are a lane's for all rows of a token that the warp takes.
//  An angle is formed in turns, as the fraction of pos * f in 64-bit fixed point
// (f = base^(-2i/D) / 2 pi): one integer product is exact for positions of any
// size, where a 32-bit product would be off by 2^-24 of the whole angle.
//
//  What bounds it: the launch for few tokens (1 token of 56 head-rows 2.2 us, 32
//  sequences 2.3), instructions for many (2048 tokens 17 us, 3.2 TB/s of projections
//  read and rows written; 248 a pass, issued in 64 % of the cycles), of which the
//  quantiser's are most: eight passes of 28 bring keys and values.
//
// keep (kvc_seq_keep): rows of the accepted path move down over the others.  A
// warp has one (layer, KV head) of a sequence, a lane a piece of 16 bytes (a row's
// scales: one of 8 or 4) of every row; it goes through the moves in order, eight
// loads and then their eight stores.  A row moves down or stays where it is, and the
// rows are ascending, so that no store reaches a row that is still to be read.
#include "draft.h"
#include "quant_row.cuh"

#include <cuda_bf16.h>

namespace kvc {
namespace {

constexpr int ROPE_THREADS = 128, BATCH = 4;

template <int ACT> struct Four; // four values of an activation type
template <> struct Four<KVC_ACT_F32> {
    using T = float;
    uint4 u;
    __device__ __forceinline__ void load(const T *p) { u = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ void get(float *x) const {
        x[0] = __uint_as_float(u.x), x[1] = __uint_as_float(u.y), x[2] = __uint_as_float(u.z), x[3] = __uint_as_float(u.w);
    }
    __device__ __forceinline__ static void store(T *p, const float *x) {
        *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
    }
};
template <> struct Four<KVC_ACT_F16> {
    using T = __half;
    uint2 u;
    __device__ __forceinline__ void load(const T *p) { u = *reinterpret_cast<const uint2 *>(p); }
    __device__ __forceinline__ void get(float *x) const {
        const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&u.x));
        const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&u.y));
        x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y;
    }
    __device__ __forceinline__ static void store(T *p, const float *x) {
        const __half2 a = __floats2half2_rn(x[0], x[1]), b = __floats2half2_rn(x[2], x[3]);
        *reinterpret_cast<uint2 *>(p) =
            make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
    }
};
template <> struct Four<KVC_ACT_BF16> {
    using T = __nv_bfloat16;
    uint2 u;
    __device__ __forceinline__ void load(const T *p) { u = *reinterpret_cast<const uint2 *>(p); }
    __device__ __forceinline__ void get(float *x) const {
        x[0] = __uint_as_float(u.x << 16), x[1] = __uint_as_float(u.x & 0xffff0000u);
        x[2] = __uint_as_float(u.y << 16), x[3] = __uint_as_float(u.y & 0xffff0000u);
    }
    __device__ __forceinline__ static void store(T *p, const float *x) {
        const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
        *reinterpret_cast<uint2 *>(p) =
            make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
    }
};

// A lane's eight values of a head-row, dims d .. d + 3 and those D/2 further, of two blocks that eight lanes hold, into pool
// row R (in: whether it is to be written).  The steps, and so the bytes, are quant_row.cuh's.
template <int D>
__device__ __forceinline__ void store_eight(int type, const TensorView &tv, int64_t R, int d, int lane, const float (&x)[8], bool in) {
    if (type == KVC_Q8_0) {
        // Each half of the eight lanes runs one block's two divisions; halves away from zero as the truncation of
        // y + copysign(0.49999997, y) (exact for |y| < 2^22).
        float top[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            top[h] = fmaxf(fmaxf(fabsf(x[4 * h]), fabsf(x[4 * h + 1])), fmaxf(fabsf(x[4 * h + 2]), fabsf(x[4 * h + 3])));
#pragma unroll
            for (int m = 1; m < 8; m <<= 1) top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], m));
        }
        const bool second = lane & 4;
        const float s = __fdiv_rn(second ? top[1] : top[0], 127.0f);
        const float inv = s != 0.0f ? __fdiv_rn(1.0f, s) : 0.0f, other = __shfl_xor_sync(0xffffffffu, inv, 4);
        const float by[2] = {second ? other : inv, second ? inv : other};
        uint32_t w[2] = {0, 0};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float y = __fmul_rn(x[i], by[i / 4]);
            const int c = __float2int_rz(__fadd_rn(y, copysignf(0.49999997f, y)));
            w[i / 4] |= ((uint32_t)c & 0xffu) << (8 * (i & 3));
        }
        if (!in) return;
        uint8_t *row = reinterpret_cast<uint8_t *>(tv.data) + R * D + d;
        *reinterpret_cast<uint32_t *>(row) = w[0] ^ CODE_FLIP;
        *reinterpret_cast<uint32_t *>(row + D / 2) = w[1] ^ CODE_FLIP;
        if ((lane & 3) == 0) // lanes 0 and 4 of the eight: the first block's scale, the second's
            tv.scales[R * (D / QK) + d / QK + (second ? D / QK / 2 : 0)] = __half_as_ushort(__float2half_rn(s));
    } else if (type == KVC_Q4_0) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float y[4] = {x[4 * h], x[4 * h + 1], x[4 * h + 2], x[4 * h + 3]};
            const int at = d + h * (D / 2);
            int c[4];
            float s;
            quantise_q4<4, 8>(y, lane, c, s);
            const uint32_t mine = (uint32_t)c[0] | (uint32_t)c[1] << 8 | (uint32_t)c[2] << 16 | (uint32_t)c[3] << 24;
            const uint32_t high = __shfl_xor_sync(0xffffffffu, mine, 4);
            if (!in) continue;
            if (d % QK < QK / 2)
                *reinterpret_cast<uint32_t *>(reinterpret_cast<uint8_t *>(tv.data) + R * (D / 2) + at / QK * (QK / 2) + at % QK) =
                    mine | high << 4;
            if (d % QK == 0) tv.scales[R * (D / QK) + at / QK] = __half_as_ushort(__float2half_rn(s));
        }
    } else if (in) {
        __half *row = reinterpret_cast<__half *>(tv.data) + R * D + d;
        Four<KVC_ACT_F16>::store(row, x);
        Four<KVC_ACT_F16>::store(row + D / 2, x + 4);
    }
}

template <int D, int ACT> __global__ void __launch_bounds__(ROPE_THREADS) rope_append_kernel(const __grid_constant__ RopeArgs a) {
    constexpr int LANES = D / 8, ROWS = 32 / LANES; // of a head-row; head-rows at a time
    using F = Four<ACT>;
    using T = typename F::T;
    // The next kernel may be scheduled now (see the append kernel: what it reads before its own wait is not written here);
    // inputs may come from the one before, so they are read behind the wait.
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x & 31, li = lane % LANES, sub = lane / LANES;
    const int64_t w = (int64_t)blockIdx.x * (ROPE_THREADS / 32) + (threadIdx.x >> 5);
    if (w >= (int64_t)a.n_tok * a.warps) return;
    const int t = (int)(w / a.warps), w0 = (int)(w % a.warps);
    int lo = 0, hi = a.n_pieces - 1;
    while (lo < hi) { // the last piece whose first token is not behind ours
        const int mid = (lo + hi + 1) / 2;
        if (a.piece[mid].first <= t) lo = mid; else hi = mid - 1;
    }
    const RopePiece &pc = a.piece[lo];
    const int at = t - pc.first;
    const int64_t tok = (int64_t)pc.tok0 + at;
    const int pos = pc.listed >= 0 ? a.pos[pc.listed + at] : pc.pos + at;

    // the lane's pairs: j, j + D/2 for four j (NEOX), or two neighbours twice in each half (NORM)
    float cs[4], sn[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int pr = a.neox ? 4 * li + i : (i < 2 ? 2 * li + i : D / 4 + 2 * li + i - 2);
        // the fraction of a turn in [-1/2, 1/2): its upper 32 bits are off by 2^-33 at most, as fp32 by 2^-26 more
        const int32_t f = (int32_t)((((uint64_t)(uint32_t)pos * a.turn[pr]) + 0x80000000ull) >> 32);
        sincospif((float)f * 0x1p-31f, &sn[i], &cs[i]);
    }
    const int nq = a.q ? (a.H + ROWS - 1) / ROWS : 0, nk = (a.Hk + ROWS - 1) / ROWS;
    const int64_t lr = (int64_t)pc.off + pc.row0 + at, pi = lr / a.P;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    int page = pi < a.max_pages ? a.pt[(int64_t)pc.id * a.max_pages + pi] : -1;
    const bool there = page >= 0 && page < a.n_pages;
    if (!there && lane == 0) atomicOr(a.err, ERR_BAD_PAGE);

    // Pass i: query rows, then keys', then values'.  A warp has those of BATCH passes under way together: with one pass ahead
    // 2048 tokens took 17.4 us, the memory waiting for requests.
    auto kind = [&](int i) { return i < nq ? 0 : (i < nq + nk ? 1 : 2); };
    auto head = [&](int i) { return (i - (i < nq ? 0 : (i < nq + nk ? nq : nq + nk))) * ROWS + sub; };
    for (int i0 = w0; i0 < a.passes; i0 += a.warps * BATCH) {
        F in[BATCH][2];
#pragma unroll
        for (int b = 0; b < BATCH; ++b) {
            const int i = i0 + b * a.warps, which = kind(i);
            if (i >= a.passes) break;
            const int64_t stride = which == 0 ? a.q_stride : (which == 1 ? a.k_stride : a.v_stride);
            const T *src = reinterpret_cast<const T *>(which == 0 ? a.q : (which == 1 ? a.k : a.v)) + tok * stride +
                           (int64_t)min(head(i), (which == 0 ? a.H : a.Hk) - 1) * D + 4 * li;
            in[b][0].load(src);
            in[b][1].load(src + D / 2);
        }
#pragma unroll
        for (int b = 0; b < BATCH; ++b) {
            const int i = i0 + b * a.warps, which = kind(i), h = head(i);
            if (i >= a.passes) break;
            float x[8];
            in[b][0].get(x);
            in[b][1].get(x + 4);
            const float *wt = which == 0 ? a.q_norm : (which == 1 ? a.k_norm : nullptr);
            if (wt) {
                const float4 w4 = *reinterpret_cast<const float4 *>(wt + 4 * li);
                const float4 w5 = *reinterpret_cast<const float4 *>(wt + D / 2 + 4 * li);
                float s = 0.f;
#pragma unroll
                for (int j = 0; j < 8; ++j) s = fmaf(x[j], x[j], s);
#pragma unroll
                for (int m = 1; m < LANES; m <<= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
                const float inv = rsqrtf(s * (1.0f / D) + a.eps);
                x[0] *= inv * w4.x, x[1] *= inv * w4.y, x[2] *= inv * w4.z, x[3] *= inv * w4.w;
                x[4] *= inv * w5.x, x[5] *= inv * w5.y, x[6] *= inv * w5.z, x[7] *= inv * w5.w;
            }
            if (which < 2) {
                if (a.neox) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float y = x[j], z = x[j + 4];
                        x[j] = y * cs[j] - z * sn[j];
                        x[j + 4] = y * sn[j] + z * cs[j];
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float y = x[2 * j], z = x[2 * j + 1];
                        x[2 * j] = y * cs[j] - z * sn[j];
                        x[2 * j + 1] = y * sn[j] + z * cs[j];
                    }
                }
            }
            if (which == 0) {
                if (h < a.H) {
                    T *dst = reinterpret_cast<T *>(a.q_out) + (tok * a.H + h) * D + 4 * li;
                    F::store(dst, x);
                    F::store(dst + D / 2, x + 4);
                }
            } else {
                const int64_t R = ((int64_t)page * a.Hk + h) * a.P + (int)(lr - pi * a.P);
                const bool is_in = there && h < a.Hk;
                store_eight<D>(which == 1 ? a.type_k : a.type_v, which == 1 ? a.lv.k : a.lv.v, R, 4 * li, lane, x, is_in);
            }
        }
    }
}

constexpr int KEEP_THREADS = 128;

__global__ void __launch_bounds__(KEEP_THREADS) keep_kernel(const __grid_constant__ KeepArgs a) {
    const int lane = threadIdx.x & 31;
    const int64_t w = (int64_t)blockIdx.x * (KEEP_THREADS / 32) + (threadIdx.x >> 5);
    if (w >= (int64_t)a.L * a.Hk * a.n_entries) return;
    const int e = (int)(w % a.n_entries), g = (int)(w / a.n_entries % a.Hk), l = (int)(w / a.n_entries / a.Hk);
    // the lane's piece: 16 bytes of a row's K or V, or the row's scales of one of them
    const int uk = a.rowb[0] / 16, uv = a.rowb[1] / 16;
    const int which = lane < uk ? 0 : (lane < uk + uv ? 1 : (lane == uk + uv ? 2 : (lane == uk + uv + 1 ? 3 : 4)));
    if (which == 4 || !a.base[which]) return;
    const int rb = a.rowb[which], wide = which < 2 ? 16 : rb;
    uint8_t *pool = a.base[which] + ((int64_t)l * a.pool_rows + (int64_t)g * a.P) * rb +
                    (which == 0 ? lane * 16 : (which == 1 ? (lane - uk) * 16 : 0));
    constexpr int AHEAD = 8;
    for (int i0 = a.first[e]; i0 < a.first[e + 1]; i0 += AHEAD) {
        uint4 v[AHEAD];
        const int n = min(AHEAD, a.first[e + 1] - i0);
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            if (i >= n) break;
            const uint8_t *src = pool + (int64_t)a.move[i0 + i].x * rb;
            if (wide == 16)
                v[i] = *reinterpret_cast<const uint4 *>(src);
            else if (wide == 8)
                *reinterpret_cast<uint2 *>(&v[i]) = *reinterpret_cast<const uint2 *>(src);
            else
                v[i].x = *reinterpret_cast<const uint32_t *>(src);
        }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            if (i >= n) break;
            uint8_t *dst = pool + (int64_t)a.move[i0 + i].y * rb;
            if (wide == 16)
                *reinterpret_cast<uint4 *>(dst) = v[i];
            else if (wide == 8)
                *reinterpret_cast<uint2 *>(dst) = *reinterpret_cast<const uint2 *>(&v[i]);
            else
                *reinterpret_cast<uint32_t *>(dst) = v[i].x;
        }
    }
}

template <int D> cudaError_t rope_pick(int act, const RopeArgs &a, const cudaLaunchConfig_t &cfg) {
    switch (act) {
    case KVC_ACT_F32: return cudaLaunchKernelEx(&cfg, rope_append_kernel<D, KVC_ACT_F32>, a);
    case KVC_ACT_F16: return cudaLaunchKernelEx(&cfg, rope_append_kernel<D, KVC_ACT_F16>, a);
    default: return cudaLaunchKernelEx(&cfg, rope_append_kernel<D, KVC_ACT_BF16>, a);
    }
}

} // namespace

cudaError_t launch_rope_append(int D, int act, const RopeArgs &a, cudaStream_t st) {
    const int64_t warps = (int64_t)a.n_tok * a.warps;
    if (warps <= 0) return cudaSuccess;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((warps + ROPE_THREADS / 32 - 1) / (ROPE_THREADS / 32)));
    cfg.blockDim = dim3(ROPE_THREADS);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return D == 64 ? rope_pick<64>(act, a, cfg) : rope_pick<128>(act, a, cfg);
}

cudaError_t launch_keep(const KeepArgs &a, cudaStream_t st) {
    const int64_t warps = (int64_t)a.L * a.Hk * a.n_entries;
    if (warps <= 0) return cudaSuccess;
    keep_kernel<<<(unsigned)((warps + KEEP_THREADS / 32 - 1) / (KEEP_THREADS / 32)), KEEP_THREADS, 0, st>>>(a);
    return cudaGetLastError();
}

} // namespace kvc
