// block_attn.h - shared by the operators over a block of query tokens: the
// block attention (kvc_attn_cross) and the rows' weights (kvc_attn_weight).
// Not part of the ABI.
#pragma once

#include "kvc_internal.h"

#include <atomic>

namespace kvc {

// One sequence of a launch.  Its query rows are the pairs (token t, query head
// j of the KV head's group), row m = t * r + j, cut into tiles of tile_m rows;
// a unit is (KV head, tile), a work item a unit or a part of its cached rows.
struct BlockSeq {
    int32_t id;         // sequence id (row of the page table)
    int32_t off;        // offset of logical row 0 in the first page
    int32_t n_rows;     // cached rows
    int32_t tok0;       // its first token in q / out / lse / n_vis
    int32_t n_tok;      // its tokens
    int32_t tiles;      // query tiles of a KV head
    int32_t item0;      // first work item of the launch that is this sequence's
    int32_t whole;      // leading units (KV head, query tile) that are one item each; the others are `splits` items
    int32_t splits;     // parts that the cached rows of a unit are cut into (>= 1)
    int32_t split_rows; // rows of a part (the last one may have fewer)
    int32_t part_row0;  // first partial row of its items (splits > 1)
    int32_t cut0;       // cut units of the launch before its own
    int32_t w_index;    // its accumulators (kvc_attn_weight)
};

struct BlockParams {
    int32_t H, Hk, D, r, P;
    int32_t n_pages, max_pages; // pages of a layer, entries of a page-table row
    int32_t n_seq, n_items;
    int32_t n_cut;        // units that are cut into parts
    uint32_t r_magic;     // ceil(2^32 / r), r > 1: m / r is the product's upper half
    int32_t act;          // kvc_act of q and out
    int32_t part_rows;    // partial rows of an item at most (min(tile_m, longest block * r))
    int32_t tile_m;
    float scale_log2;     // kq_scale * log2(e)
    const int32_t *pt;    // page tables
    const uint8_t *kdata; // this layer's pools
    const uint8_t *vdata;
    const uint16_t *ks;
    const uint16_t *vs;
    const void *q;
    void *out;
    float *lse;           // cross: written (may be null); weight: read
    const int32_t *n_vis; // null: every token sees all rows
    float *w;             // weight: accumulators [..][Hk][w_stride]
    int64_t w_stride;
    float *part;          // partials: [row][D] sums, then [row] (max, sum) pairs
    int64_t part_cap;     // partial rows
    uint32_t *err;
    BlockSeq seq[MAX_SEQ_PER_LAUNCH];
};
static_assert(sizeof(BlockParams) <= 4000, "launch parameters stay within 4 KB");

constexpr int CROSS_TILE_M = 64;     // query rows of a tile
constexpr int CROSS_TILE_N = 64;     // cached rows of a step
constexpr int CROSS_TC_TILE_M = 256; // the same of the tcgen05 kernel
constexpr int CROSS_TC_TILE_N = 128;

// A kernel's dynamic shared memory, allowed once in every CUDA context (one
// of these per kernel; threads may come at once: the worst is a second call).
// regs: registers that its roles share out, 0 for none: with fewer at launch
// they would wait for them forever, so that such a build is refused.
struct SharedMemory {
    std::atomic<uint64_t> ctx{0};
    cudaError_t allow(const void *kernel, int bytes, int regs = 0) {
        const uint64_t id = current_context_id();
        if (id && ctx.load(std::memory_order_acquire) == id) return cudaSuccess;
        cudaFuncAttributes a;
        cudaError_t e = cudaFuncGetAttributes(&a, kernel);
        if (e == cudaSuccess && a.numRegs < regs) e = cudaErrorInvalidConfiguration;
        if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e == cudaSuccess) ctx.store(id, std::memory_order_release);
        return e;
    }
};

// The block attention.  narrow: every sequence's query rows of a KV head fit
// 16 (one tensor-core row block), so the warps share the cached rows instead.
cudaError_t launch_cross(int type_k, int type_v, const BlockParams &p, bool narrow, cudaStream_t st);
// The same for 16-bit queries, by tcgen05 (tiles of CROSS_TC_TILE_M query rows).
cudaError_t launch_cross_tc(int type_k, int type_v, const BlockParams &p, cudaStream_t st);

// Joins the parts of the launch's cut units (k_join.cu; the two above end with it).
cudaError_t launch_join(const BlockParams &p, cudaStream_t st);

// The rows' weights: a unit is a KV head (one tile), a step WEIGHT_STEP rows.
constexpr int WEIGHT_STEP = 128;
cudaError_t launch_weight(int type_k, const BlockParams &p, cudaStream_t st);

} // namespace kvc
