// k_evict.cu - eviction of the rows that received the least attention weight
// (kvc_seq_evict_weight).
//
//   W_j = (w[0][j] + w[1][j]) + ... over the KV heads, in 32 bits and in that
//   order; the n_remove candidates of smallest (W_j, j) go.
//
// A candidate's weights are summed into an unsigned key of the same order (a NaN
// after everything else).  evict_select finds the n_remove-th smallest
// key digit by digit (four passes of 8 bits over the keys, which stay in L2) and
// lists the removed rows in ascending order: a warp owns a contiguous range of
// candidates, counts its smaller and its equal keys, and after one scan over
// the warps knows where its own go.  Then the sequence's last n_remove rows
// [n', n) give the places: the kept ones among them move, in order, into the
// removed places below n' (as many, by counting), so at most n_remove rows are
// read and written in every layer, whatever the sequence's length.  A mover's
// place is found by a binary search in the list; nothing of the cache has
// changed by then.  evict_move, the last kernel, moves the weights and the K and V
// rows of all layers and heads, unless the device's error word is set (by a page
// that the pool does not have, or by a kernel before): the call fails then, and
// weights, rows and positions are as they were.
// What bounds it: the chain of launches, barriers and two waits for the device with
// few rows (64 of 512 rows: 43 us for the call); the one CTA's passes over the keys
// with many (1024 of 32768: 117 us; 16 layers more move in 14 us).
#include "evict.h"

namespace kvc {
namespace {

constexpr int SEL = 1024; // threads of the selecting CTA
constexpr int WARPS = SEL / 32;

// Candidate i's weight as an unsigned key of the same order.
__device__ __forceinline__ void key_of(const EvictArgs &a, int64_t i) {
    const int64_t j = a.rows ? a.rows[i] : a.first + i;
    float s = a.w[j];
    for (int g = 1; g < a.Hk; ++g) s = __fadd_rn(s, a.w[g * a.w_stride + j]);
    s = __fadd_rn(s, 0.f); // -0 becomes +0
    uint32_t u = __float_as_uint(s);
    u = (u & 0x80000000u) ? ~u : u | 0x80000000u;
    if (s != s) u = 0xffffffffu;
    a.keys[i] = u;
}
__global__ void __launch_bounds__(256) evict_keys(const __grid_constant__ EvictArgs a) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i < a.n_cand) key_of(a, i);
}

__device__ __forceinline__ int64_t pool_row0(const EvictArgs &a, int32_t j) {
    const int64_t lr = (int64_t)a.off + j, pi = lr / a.P;
    const int32_t page = pi < a.pt_len ? a.pt[pi] : -1;
    if (page < 0 || page >= a.n_pages) {
        atomicOr(a.err, ERR_BAD_PAGE);
        return -1;
    }
    return (int64_t)page * a.Hk * a.P + (lr - pi * a.P);
}

// Row x of the last n_remove ones: its place among the holes, if it stays.
__device__ __forceinline__ void pair_of(const EvictArgs &a, int x) {
    const int32_t left = a.n - a.n_remove, j = left + x;
    int lo = 0, hi = a.n_remove; // removed rows before j
    while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (a.gone[mid] < j) lo = mid + 1; else hi = mid;
    }
    int4 pr = make_int4(-1, -1, -1, 0);
    if (lo >= a.n_remove || a.gone[lo] != j) {
        // kept: of the x rows before it in the tail, those removed are the removed ones below j that are not holes;
        // with h holes, lo - h of them, so it is mover x - (lo - h); holes are the first h of the list
        int hl = 0, hh = a.n_remove;
        while (hl < hh) {
            const int mid = (hl + hh) / 2;
            if (a.gone[mid] < left) hl = mid + 1; else hh = mid;
        }
        const int32_t hole = a.gone[x - (lo - hl)];
        const int64_t to = pool_row0(a, hole), from = pool_row0(a, j);
        if (to >= 0 && from >= 0) pr = make_int4((int)to, (int)from, hole, 0);
    }
    a.pairs[x] = pr;
}
__global__ void __launch_bounds__(128) evict_pairs(const __grid_constant__ EvictArgs a) {
    const int x = (int)blockIdx.x * 128 + threadIdx.x;
    if (x < a.n_remove) pair_of(a, x);
}

// ALL: few candidates, whose keys and pairs the one CTA sees to as well.
template <bool ALL> __global__ void __launch_bounds__(SEL) evict_select(const __grid_constant__ EvictArgs a) {
    constexpr int COPIES = 8; // of the counts: lanes that share a digit meet on few addresses
    __shared__ uint32_t hist[COPIES][256];
    constexpr int AHEAD = 8;  // a thread's keys that are under way together
    __shared__ uint32_t prefix, left;
    __shared__ int32_t below[WARPS], equal[WARPS];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n = a.n_cand;
    if (ALL)
        for (int i = tid; i < n; i += SEL) key_of(a, i); // (seen by the CTA after the barriers below)
    if (tid == 0) {
        prefix = 0;
        left = (uint32_t)a.n_remove; // rank of the wanted key among those that share the prefix, from 1
    }
    for (int shift = 24; shift >= 0; shift -= 8) {
        for (int i = tid; i < COPIES * 256; i += SEL) hist[i >> 8][i & 255] = 0;
        __syncthreads();
        const uint32_t pre = prefix;
        const uint32_t mask = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
        for (int i0 = tid; i0 < n; i0 += SEL * AHEAD) {
            uint32_t k[AHEAD];
#pragma unroll
            for (int j = 0; j < AHEAD; ++j) k[j] = i0 + j * SEL < n ? a.keys[i0 + j * SEL] : ~pre;
#pragma unroll
            for (int j = 0; j < AHEAD; ++j)
                if (i0 + j * SEL < n && (k[j] & mask) == pre) atomicAdd(&hist[lane % COPIES][(k[j] >> shift) & 255u], 1u);
        }
        __syncthreads();
        if (tid < 256) {
            uint32_t c = 0;
#pragma unroll
            for (int k = 0; k < COPIES; ++k) c += hist[k][tid];
            hist[0][tid] = c;
        }
        __syncthreads();
        if (warp == 0) {
            // eight digits a lane; the first digit whose cumulative count reaches the rank
            uint32_t c[8], sum = 0;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                c[k] = hist[0][lane * 8 + k];
                sum += c[k];
            }
            uint32_t inc = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t x = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += x;
            }
            const uint32_t rank = left;
            uint32_t before = inc - sum;
            __syncwarp();
            if (before < rank && rank <= inc) {
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    if (before < rank && rank <= before + c[k]) {
                        prefix = pre | ((uint32_t)(lane * 8 + k) << shift);
                        left = rank - before;
                    }
                    before += c[k];
                }
            }
        }
        __syncthreads();
    }
    const uint32_t key = prefix;
    const int ties = (int)left; // of the keys equal to it, the first `ties` go
    const int per = (n + WARPS * 32 - 1) / (WARPS * 32) * 32;
    const int lo = min(n, warp * per), hi = min(n, lo + per);
    int nb = 0, ne = 0;
    for (int i = lo + lane; i < hi; i += 32 * AHEAD) {
        uint32_t k[AHEAD];
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) k[j] = i + j * 32 < hi ? a.keys[i + j * 32] : 0u;
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
            nb += i + j * 32 < hi && k[j] < key;
            ne += i + j * 32 < hi && k[j] == key;
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        nb += __shfl_xor_sync(0xffffffffu, nb, o);
        ne += __shfl_xor_sync(0xffffffffu, ne, o);
    }
    if (lane == 0) {
        below[warp] = nb;
        equal[warp] = ne;
    }
    __syncthreads();
    int b0 = 0, e0 = 0;
    for (int w = 0; w < warp; ++w) {
        b0 += below[w];
        e0 += equal[w];
    }
    for (int i0 = lo; i0 < hi; i0 += 32 * AHEAD) {
        uint32_t k[AHEAD];
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) k[j] = i0 + j * 32 + lane < hi ? a.keys[i0 + j * 32 + lane] : 0xffffffffu;
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
            const int i = i0 + j * 32 + lane;
            const bool lt = i < hi && k[j] < key, eq = i < hi && k[j] == key;
            const uint32_t ml = __ballot_sync(0xffffffffu, lt), me = __ballot_sync(0xffffffffu, eq);
            const uint32_t under = (1u << lane) - 1u;
            const int er = e0 + __popc(me & under); // equal keys before this one
            if (lt || (eq && er < ties)) a.gone[b0 + __popc(ml & under) + min(er, ties)] = a.rows ? a.rows[i] : a.first + i;
            b0 += __popc(ml);
            e0 += __popc(me);
        }
    }
    if (ALL) {
        __syncthreads();
        for (int x = tid; x < a.n_remove; x += SEL) pair_of(a, x);
    }
}

// One warp a (pair, layer): every head's row of the four tensors, in the widest words that its rows allow; the first
// layer's sees to the pair's weights too.
template <class W>
__device__ __forceinline__ void move_rows(uint8_t *base, int rowb, int64_t to, int64_t from, int64_t head, int Hk, int lane) {
    const int words = rowb / (int)sizeof(W), all = words * Hk;
    for (int i = lane; i < all; i += 32) {
        const int g = i / words, c = i % words;
        const W v = reinterpret_cast<const W *>(base + (from + g * head) * rowb)[c];
        reinterpret_cast<W *>(base + (to + g * head) * rowb)[c] = v;
    }
}
__global__ void __launch_bounds__(256) evict_move(const __grid_constant__ EvictArgs a) {
    const int lane = threadIdx.x & 31;
    const int64_t i = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (i >= a.n_remove || *a.err != 0) return;
    const int4 pr = a.pairs[i];
    if (blockIdx.y == 0) {
        for (int g = lane; g < a.Hk; g += 32) {
            float *w = a.w + g * a.w_stride, *tail = w + (a.n - a.n_remove + i);
            if (pr.z >= 0) w[pr.z] = *tail;
            *tail = 0.f;
        }
    }
    if (pr.x < 0) return;
    const int64_t lo = (int64_t)blockIdx.y * a.pool_rows, to = lo + pr.x, from = lo + pr.y;
    move_rows<uint4>(a.base[0], a.rowb[0], to, from, a.P, a.Hk, lane);
    move_rows<uint4>(a.base[1], a.rowb[1], to, from, a.P, a.Hk, lane);
    if (a.base[2]) move_rows<uint32_t>(a.base[2], a.rowb[2], to, from, a.P, a.Hk, lane);
    if (a.base[3]) move_rows<uint32_t>(a.base[3], a.rowb[3], to, from, a.P, a.Hk, lane);
}

} // namespace

cudaError_t launch_evict(const EvictArgs &a, cudaStream_t st) {
    if (a.L > 65535) return cudaErrorInvalidValue;
    // Up to FEW candidates one CTA does it all, more are summed and paired by as many CTAs as there are.  The whole call,
    // 8 heads, 64 rows to go: 4096 rows 58.8 us by one CTA, 61.0 by many; 8128 rows 63.4 and 66.6; 32768 rows 134 and 113.
    constexpr int FEW = 8192;
    if (a.n_cand <= FEW) {
        evict_select<true><<<1, SEL, 0, st>>>(a);
    } else {
        evict_keys<<<(unsigned)((a.n_cand + 255) / 256), 256, 0, st>>>(a);
        evict_select<false><<<1, SEL, 0, st>>>(a);
        evict_pairs<<<(unsigned)((a.n_remove + 127) / 128), 128, 0, st>>>(a);
    }
    evict_move<<<dim3((unsigned)((a.n_remove + 7) / 8), (unsigned)a.L), 256, 0, st>>>(a);
    return cudaGetLastError();
}

} // namespace kvc
