// block_attn.cu - host side of the operators over a block of query tokens
// (kvc_attn_cross, kvc_attn_weight, kvc_attn_tree): checks, the split of the
// cached rows over work items, the work space and the launches.
#include "block_attn.h"
#include "ctx.h"

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstring>

namespace kvc {

int cuda_fail(Ctx *c, cudaError_t e, const char *what);
int dev_alloc(Ctx *c, void **p, int64_t bytes, const char *what);

#define KVC_CU(c, call)                                                                                            \
    do {                                                                                                           \
        cudaError_t e_ = (call);                                                                                   \
        if (e_ != cudaSuccess) return cuda_fail((c), e_, #call);                                                   \
    } while (0)

// Partial rows of the work space: every SM four items of a whole query tile.
static int64_t part_rows_cap(int sms) { return (int64_t)4 * sms * CROSS_TILE_M; }

// The work space of split rows: partial sums [rows][D] and (max, sum) pairs
// [rows].  Allocated once, with one size: a captured launch keeps its address.
static int ensure_block_space(Ctx *c, cudaStream_t st) {
    if (c->block_part) return KVC_OK;
    cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
    KVC_CU(c, cudaStreamIsCapturing(st, &cap));
    if (cap != cudaStreamCaptureStatusNone)
        return c->fail(KVC_EINVAL, "the first block attention of a context allocates its work space: call it once before a capture");
    return dev_alloc(c, (void **)&c->block_part, part_rows_cap(c->sms) * (c->D + 2) * 4, "block attention work space");
}

// Cut the cached rows of the launch's units into parts.  `want`: items that run
// at once; a part has `least` rows at least, and the partial rows of all parts
// fit the work space.  An item costs `fixed` steps beside its own, joining
// a sequence's `join` (one sequence).  tree: the launch's sequences may change
// places, and four waves of items are enough (32 sequences of 1024 to 8000 rows,
// 16 tokens each: 276 us with up to nine, 262 so; f16 190 and 177).  weighted: a
// step of a unit that fills half a tile at most costs 5/8 of another's, and an
// item six of them beside its own (4 to 16 tokens of 32 f16 sequences of 1024 to
// 8000 rows: 167 us with four, 147 so).
//  One sequence: its units are alike, so the schedule is whole waves; those of
// the last one or two are cut into the parts that shorten it most.
//  Several: all rows are cut into parts of at most one length, the one for
// which a schedule ends first that ends half the longest item after the mean
// (or, in one wave, with the longest item).
static void plan_splits(BlockParams &p, int64_t want, int64_t step, int64_t least, int64_t part_cap, int64_t join = 1,
                        bool tree = false, bool weighted = false) {
    const int64_t fixed = 4;
    auto half = [&](const BlockSeq &s) { return (int64_t)s.n_tok * p.r - (int64_t)s.tile0 * p.tile_m <= p.tile_m / 2; };
    const bool alike = !weighted || std::all_of(p.seq, p.seq + p.n_seq, half);
    auto eighths = [&](const BlockSeq &s) { return !alike && half(s) ? 5 : 8; };
    auto parts = [&](const BlockSeq &s, int64_t len) {
        return (int32_t)std::max<int64_t>(1, ((int64_t)s.n_rows * eighths(s) / 8 + len - 1) / len);
    };
    int64_t longest = step;
    for (int i = 0; i < p.n_seq; ++i)
        if (p.seq[i].tiles) longest = std::max<int64_t>(longest, (p.seq[i].n_rows + step - 1) / step * step);
    if (p.n_seq == 1) {
        BlockSeq &s = p.seq[0];
        const int64_t units = (int64_t)s.tiles * p.Hk, steps = (s.n_rows + step - 1) / step;
        const int64_t most = std::max<int64_t>(1, s.n_rows / least);
        int64_t best_cost = INT64_MAX;
        for (int64_t full = units / want * want; full >= 0; full = full > 0 ? full - want : -1) {
            const int64_t rest = units - full;
            if (rest > 2 * want) break;
            for (int64_t k = 1; k <= std::min<int64_t>(most, rest ? std::max<int64_t>(8, want / rest) : 1); ++k) {
                if (k > 1 && rest * k * p.part_rows > part_cap) break;
                const int64_t cost = full / want * (steps + fixed) +
                                     (rest * k + want - 1) / want * ((steps + k - 1) / k + fixed + (k > 1 ? join : 0));
                if (cost < best_cost) {
                    best_cost = cost;
                    s.splits = (int32_t)k;
                    s.whole = (int32_t)(k > 1 ? full : units);
                }
            }
        }
    } else {
        double best = 0;
        int64_t best_len = longest;
        const int64_t own = weighted ? 6 : fixed;
        int64_t cuts = 1; // of few sequences every length counts
        for (int64_t len = longest;;) {
            int64_t items = 0, slots = 0, most = 0;
            double total = 0;
            for (int i = 0; i < p.n_seq; ++i) {
                const BlockSeq &s = p.seq[i];
                const int64_t k = parts(s, len), n = (int64_t)s.tiles * p.Hk * k;
                if (!n) continue;
                const int64_t cost = own + (((s.n_rows + k - 1) / k + step - 1) / step * eighths(s) + 7) / 8;
                items += n;
                if (k > 1) slots += n;
                total += (double)n * (double)cost;
                most = std::max(most, cost);
            }
            if (slots * p.part_rows > part_cap) break;
            const double est = items <= want ? (double)most : total / (double)want + 0.5 * (double)most;
            if (len == longest || est < best) {
                best = est;
                best_len = len;
            }
            if (len <= least || (tree && items > 4 * want)) break;
            if (weighted && p.n_seq <= 4)
                len = std::max(least, (longest / ++cuts + step - 1) / step * step);
            else
                len = std::max(least, len * 3 / 4 / step * step);
        }
        for (int i = 0; i < p.n_seq; ++i) {
            BlockSeq &s = p.seq[i];
            s.splits = parts(s, best_len);
            s.whole = s.splits > 1 ? 0 : s.tiles * p.Hk;
        }
    }
    int64_t items = 0;
    for (int i = 0; i < p.n_seq; ++i) {
        const BlockSeq &s = p.seq[i];
        items += s.whole + ((int64_t)s.tiles * p.Hk - s.whole) * s.splits;
    }
    // The longest items begin first, so that none of them begins late (q8_0, 8 heads of 128, as given and sorted: 6 tokens of
    // 32 sequences of 64 to 400 rows 21.0 and 18.1 us, of 16 of 300 to 3000 rows 35.2 and 33.1; 20 to 80 tokens of 32 of 1024
    // to 8000 rows 412 and 370).  Not in more than two waves of items of alike steps, which the memory bounds: there the order
    // as given is no worse (1 token of 32 sequences of 1024 to 8000 rows: 99 as given, 103 sorted; f16 111 and 120).
    if (tree && (weighted || items <= 2 * want))
        std::stable_sort(p.seq, p.seq + p.n_seq, [&](const BlockSeq &a, const BlockSeq &b) {
            return (int64_t)a.n_rows * eighths(a) * b.splits > (int64_t)b.n_rows * eighths(b) * a.splits;
        });
    int32_t item = 0, row = 0;
    p.n_cut = 0;
    for (int i = 0; i < p.n_seq; ++i) {
        BlockSeq &s = p.seq[i];
        // equal parts, in whole steps
        const int64_t even = ((int64_t)s.n_rows + s.splits - 1) / s.splits;
        s.split_rows = (int32_t)std::min<int64_t>(INT32_MAX / 2 / step * step,
                                                  std::max<int64_t>(1, (even + step - 1) / step) * step);
        s.item0 = item;
        s.part_row0 = row;
        s.cut0 = p.n_cut;
        const int32_t cut = s.tiles * p.Hk - s.whole;
        item += s.whole + cut * s.splits;
        row += cut * s.splits * p.part_rows;
        p.n_cut += cut;
    }
    p.n_items = item;
}

// The query tiles and items of a launch over p.n_seq sequences (p.Hk, p.r and
// each one's n_rows and n_tok set), for the tcgen05 kernel or the other one.
// Returns whether the tiles are narrow.
static bool plan_block(BlockParams &p, int sms, bool tc) {
    int32_t most = 0;
    for (int i = 0; i < p.n_seq; ++i) most = std::max(most, p.seq[i].n_tok);
    const bool narrow = !tc && (int64_t)most * p.r <= 16;
    p.tile_m = tc ? CROSS_TC_TILE_M : (narrow ? 16 : CROSS_TILE_M);
    p.part_rows = (int32_t)std::max<int64_t>(1, std::min<int64_t>(p.tile_m, (int64_t)most * p.r));
    for (int i = 0; i < p.n_seq; ++i) {
        BlockSeq &s = p.seq[i];
        s.tiles = (int32_t)(((int64_t)s.n_tok * p.r + p.tile_m - 1) / p.tile_m);
    }
    const int step = tc ? CROSS_TC_TILE_N : CROSS_TILE_N;
    plan_splits(p, tc ? sms : 2 * sms, step, 2 * step, part_rows_cap(sms));
    return narrow;
}

// The query tiles and items of a tree attention: tiles of 32 query rows (or what there are: the kernel shares the work of
// fewer over all its warps too), one item at a time on an SM.  The kernel counts cached rows from the 16-row boundary at or
// below the sequence's first.
static void plan_tree(BlockParams &p, int sms) {
    constexpr int64_t JOIN = 4;
    int64_t most = 0;
    for (int i = 0; i < p.n_seq; ++i) most = std::max<int64_t>(most, (int64_t)p.seq[i].n_tok * p.r);
    p.tile_m = TREE_TILE;
    p.part_rows = (int32_t)std::max<int64_t>(1, std::min<int64_t>(p.tile_m, most));
    for (int i = 0; i < p.n_seq; ++i) {
        BlockSeq &s = p.seq[i];
        s.tiles = (int32_t)(((int64_t)s.n_tok * p.r + p.tile_m - 1) / p.tile_m);
        s.n_rows += s.off % 16;
    }
    plan_splits(p, sms, TREE_STEP, 2 * TREE_STEP, part_rows_cap(sms), JOIN, true);
    for (int i = 0; i < p.n_seq; ++i) p.seq[i].n_rows -= p.seq[i].off % 16;
}

// The same for the tcgen05 kernel.  A last tile whose query rows fill half of it at most costs less a step (65536 q8_0 rows of
// 8 KV heads: 125 rows 80 us, 255 rows 116), so it is an entry of its own, with longer parts, where the launch has room (64
// tokens of 5 heads over 32768 rows 111 us as one entry, 99 as two; 32 sequences of 20 to 80 tokens over 1024 to 8000 rows 388
// and 370).
static void plan_tree_tc(BlockParams &p, int sms) {
    int32_t most = 0;
    for (int i = 0; i < p.n_seq; ++i) most = std::max(most, p.seq[i].n_tok);
    p.tile_m = CROSS_TC_TILE_M;
    p.part_rows = (int32_t)std::max<int64_t>(1, std::min<int64_t>(p.tile_m, (int64_t)most * p.r));
    for (int i = 0, n = p.n_seq; i < n; ++i) {
        BlockSeq &s = p.seq[i];
        const int64_t m = (int64_t)s.n_tok * p.r;
        s.tiles = (int32_t)((m + p.tile_m - 1) / p.tile_m);
        s.tile0 = 0;
        if (s.tiles < 2 || m - (int64_t)(s.tiles - 1) * p.tile_m > p.tile_m / 2 || p.n_seq == MAX_SEQ_PER_LAUNCH) continue;
        BlockSeq &last = p.seq[p.n_seq++];
        last = s;
        last.tile0 = --s.tiles;
        last.tiles = 1;
    }
    plan_splits(p, sms, CROSS_TC_TILE_N, 2 * CROSS_TC_TILE_N, part_rows_cap(sms), 1, true, true);
}

// Which kernel attends a sequence of 16-bit queries (both hold scores to 32 bits).  The tcgen05 kernel pays where a call
// has enough to do, by its cached values (rows x KV heads x D) or its products (times query rows of a KV head); and in
// such a call for the sequences that have TC_MIN_ROWS rows or enough products of their own: an item of few tokens over
// fewer rows is all start.  Measured in us, mma.sync against tcgen05, q8_0, bf16 queries, heads/KV heads/D:
//   8/2/64,  1024 rows:   1 token   8.8 / 11.3,  256 tokens 14.0 / 19.4    (2^17 values, 2^27 products)
//   8/2/64,  16384 rows:  1 token  20.4 / 17.9                             (2^21 values)
//   40/8/128, 256 rows:  64 tokens 14.4 / 20.2,  256 tokens 21.5 / 20.3    (2^18 values; 2^26, 2^28 products)
//   40/8/128, 4096 rows:  1 token  17.1 / 17.5,  256 tokens 173 / 53       (2^22 values)
//   32/8/128, 64 sequences of 100 rows, 1 token each 19.2 / 58.3,  32 of 200 rows, 4 tokens each 15.1 / 36.7
//   40/8/128, 200 rows:  64 tokens 16.3 / 21.6,  512 tokens 41.2 / 24.3    (2^26, 2^29 products)
constexpr int TC_MIN_ROWS = 256;
constexpr double TC_VALUES = 1 << 21, TC_PRODUCTS = 1 << 28;
static bool tc_pays(double values, double products) { return values >= TC_VALUES || products >= TC_PRODUCTS; }
static bool use_tc(int rows, double products) { return rows >= TC_MIN_ROWS || products >= TC_PRODUCTS; }

// Which kernel runs a tree attention of 16-bit queries: the tcgen05 one where the sequences bring more than 32 query rows a
// KV head (on the mean over the cached rows) and there is enough to do, by the cached values and the products.  One kernel
// runs the whole call: two one after the other would each leave the machine to its last items (32 sequences of 1024 to 32768
// f16 rows, 4 to 16 tokens: 509 us by two, 394 by the tcgen05 one).  f16 queries over codes stay with the other: the tcgen05
// one rounds both P and the scaled V to 11 bits, which results of 11 bits would show (3.6e-4 rms against 2.9e-4, and 2.1e-4
// for the result's own rounding).  Measured in us, bf16 queries, mma.sync against tcgen05, heads/KV heads/D, rows: tokens
//   40/8/128 q8_0   512:  16 11.6 / 19.5,  64 14.1 / 25.3          4096:  8 16.6 / 21.1,  32 26.4 / 26.1,  64 48.3 / 30.4
//                 16384:  4 22.7 / 31.3,   8 32.7 / 32.4,  32 73.1 / 40.8      65536:  4 55.2 / 76.0,  8 98.1 / 76.5
//   32/8/128 f16   4096:  16 14.5 / 18.4,  64 25.4 / 26.3         65536:  8 51.4 / 59.1,  16 66.3 / 58.7,  64 229 / 83.8
//   8/2/64 q8_0   16384:  64 24.2 / 24.0                          65536:  16 26.5 / 29.3,  64 70.4 / 35.3
static bool tree_tc_pays(double values, double rows_m, double rows) {
    const double m = rows > 0 ? rows_m / rows : 0;
    return m > 32 && values >= 1 << 22 && m * values >= 1 << 28;
}

// Checks that the block operators share; *total: tokens of the block.
static int block_check(Ctx *c, int layer, int n_seq, const int32_t *seq_ids, const int32_t *n_q, int act, const void *q,
                       float kq_scale, int64_t *total) {
    if (c->host) return c->fail(KVC_EINVAL, "block operators need a device-resident context");
    if (layer < 0 || layer >= c->L) return c->fail(KVC_EINVAL, "layer out of range");
    if (n_seq < 1 || !seq_ids || !n_q) return c->fail(KVC_EINVAL, "n_seq >= 1, seq_ids and n_q required");
    if (act != KVC_ACT_F32 && act != KVC_ACT_F16 && act != KVC_ACT_BF16)
        return c->fail(KVC_EINVAL, "act must be KVC_ACT_F32, KVC_ACT_F16 or KVC_ACT_BF16");
    if (!std::isfinite(kq_scale)) return c->fail(KVC_EINVAL, "kq_scale must be finite");
    int64_t t = 0;
    for (int i = 0; i < n_seq; ++i) {
        if (seq_ids[i] < 0 || seq_ids[i] >= (int)c->seqs.size())
            return c->fail(KVC_EINVAL, "sequence id out of range");
        if (n_q[i] < 0) return c->fail(KVC_EINVAL, "n_q must not be negative");
        t += n_q[i];
    }
    if (t * c->r > INT32_MAX / 4 / c->Hk) return c->fail(KVC_EINVAL, "too many tokens in one block");
    *total = t;
    if (t == 0) return KVC_OK;
    if (!q) return c->fail(KVC_EINVAL, "q must be non-null");
    if ((uintptr_t)q & 15) return c->fail(KVC_EINVAL, "q must be 16-byte aligned");
    return KVC_OK;
}

static void block_params(const Ctx *c, int layer, float kq_scale, int act, BlockParams &p) {
    std::memset(&p, 0, sizeof(p));
    p.H = c->H;
    p.Hk = c->Hk;
    p.D = c->D;
    p.r = c->r;
    p.r_magic = c->r > 1 ? (uint32_t)((((uint64_t)1 << 32) + c->r - 1) / c->r) : 0;
    p.P = c->P;
    p.n_pages = c->n_pages;
    p.max_pages = c->max_pages;
    p.act = act;
    p.scale_log2 = (float)((double)kq_scale * 1.4426950408889634);
    p.pt = c->pt_dev;
    const int64_t lo = (int64_t)layer * c->pool_rows;
    p.kdata = c->kdata + lo * c->krow;
    p.vdata = c->vdata + lo * c->vrow;
    p.ks = c->ksb ? reinterpret_cast<const uint16_t *>(c->kscales + lo * c->ksb) : nullptr;
    p.vs = c->vsb ? reinterpret_cast<const uint16_t *>(c->vscales + lo * c->vsb) : nullptr;
    p.err = c->err_dev;
}

static bool overlap(const void *a, const void *b, int64_t bytes) {
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return x < y + (uintptr_t)bytes && y < x + (uintptr_t)bytes;
}

} // namespace kvc

using namespace kvc;

extern "C" int kvc_attn_cross(kvc_ctx *cc, int layer, int n_seq, const int32_t *seq_ids, const int32_t *n_q, int act,
                              const void *q, void *out, float *lse, const int32_t *n_vis, float kq_scale,
                              void *stream) {
    if (!cc) return KVC_EINVAL;
    Ctx *c = reinterpret_cast<Ctx *>(cc);
    int64_t total = 0;
    int rc = block_check(c, layer, n_seq, seq_ids, n_q, act, q, kq_scale, &total);
    if (rc) return rc;
    if (total == 0) return KVC_OK;
    if (!out) return c->fail(KVC_EINVAL, "out must be non-null");
    if ((uintptr_t)out & 15) return c->fail(KVC_EINVAL, "out must be 16-byte aligned");
    if (((uintptr_t)lse | (uintptr_t)n_vis) & 3) return c->fail(KVC_EINVAL, "lse and n_vis must be 4-byte aligned");
    if (overlap(q, out, total * c->H * c->D * (act == KVC_ACT_F32 ? 4 : 2)))
        return c->fail(KVC_EINVAL, "out may not overlap q");
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    KVC_CU(c, cudaSetDevice(c->dev));
    if ((rc = ensure_block_space(c, st))) return rc;
    const int64_t cap = part_rows_cap(c->sms);
    auto products_of = [&](int i) {
        return (double)c->seqs[(size_t)seq_ids[i]].lfill[(size_t)layer] * c->Hk * c->D * c->r * n_q[i];
    };
    double values = 0, products = 0;
    for (int i = 0; i < n_seq; ++i) {
        if (n_q[i] == 0) continue;
        values += (double)c->seqs[(size_t)seq_ids[i]].lfill[(size_t)layer] * c->Hk * c->D;
        products += products_of(i);
    }
    const bool pays = act != KVC_ACT_F32 && (c->block_kernel ? c->block_kernel == 2 : tc_pays(values, products));
    for (int tc = 0; tc < 2; ++tc) { // the sequences of either kernel, as many a launch as it carries
        BlockParams p;
        block_params(c, layer, kq_scale, act, p);
        p.q = q;
        p.out = out;
        p.lse = lse;
        p.n_vis = n_vis;
        p.part = c->block_part;
        p.part_cap = cap;
        int64_t tok0 = 0;
        for (int i = 0; i < n_seq; ++i) {
            const Seq &sq = c->seqs[(size_t)seq_ids[i]];
            const int32_t rows = sq.lfill[(size_t)layer];
            if (n_q[i] > 0 && (pays && (c->block_kernel || use_tc(rows, products_of(i)))) == (tc != 0)) {
                BlockSeq &s = p.seq[p.n_seq++];
                s.id = seq_ids[i];
                s.off = sq.off;
                s.n_rows = rows;
                s.tok0 = (int32_t)tok0;
                s.n_tok = n_q[i];
            }
            tok0 += n_q[i];
            if (p.n_seq == 0 || (p.n_seq < MAX_SEQ_PER_LAUNCH && i + 1 < n_seq)) continue;
            const bool narrow = plan_block(p, c->sms, tc != 0);
            cudaError_t e = tc ? launch_cross_tc(c->tk, c->tv, p, st) : launch_cross(c->tk, c->tv, p, narrow, st);
            if (e != cudaSuccess) return cuda_fail(c, e, "block attention kernel");
            p.n_seq = 0;
        }
    }
    return KVC_OK;
}

extern "C" int kvc_attn_tree(kvc_ctx *cc, int layer, int n_seq, const int32_t *seq_ids, const int32_t *n_q, int act,
                             const void *q, void *out, const int32_t *parent, float kq_scale, void *stream) {
    if (!cc) return KVC_EINVAL;
    Ctx *c = reinterpret_cast<Ctx *>(cc);
    int64_t total = 0;
    int rc = block_check(c, layer, n_seq, seq_ids, n_q, act, q, kq_scale, &total);
    if (rc) return rc;
    for (int i = 0; i < n_seq; ++i) {
        if (n_q[i] > TREE_MAX) return c->fail(KVC_EINVAL, "a tree has at most 256 tokens");
        if (n_q[i] > c->seqs[(size_t)seq_ids[i]].lfill[(size_t)layer])
            return c->fail(KVC_EINVAL, "a sequence has fewer rows than its tree has tokens");
    }
    if (total == 0) return KVC_OK;
    if (!out) return c->fail(KVC_EINVAL, "out must be non-null");
    if ((uintptr_t)out & 15) return c->fail(KVC_EINVAL, "out must be 16-byte aligned");
    if ((uintptr_t)parent & 3) return c->fail(KVC_EINVAL, "parent must be 4-byte aligned");
    if (overlap(q, out, total * c->H * c->D * (act == KVC_ACT_F32 ? 4 : 2)))
        return c->fail(KVC_EINVAL, "out may not overlap q");
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    KVC_CU(c, cudaSetDevice(c->dev));
    if ((rc = ensure_block_space(c, st))) return rc;
    auto *by_warps = c->tk == KVC_F16 ? launch_tree_f16 : (c->tv == KVC_Q4_0 ? launch_tree_q4 : launch_tree_q8);
    const size_t l = (size_t)layer;
    const TreeMaps maps = {&c->tmk64[l], &c->tmv64[l], &c->tmk[2 * l], &c->tmv[2 * l]};
    double values = 0, rows_m = 0, all_rows = 0;
    for (int i = 0; i < n_seq; ++i) {
        if (n_q[i] == 0) continue;
        const double rows = c->seqs[(size_t)seq_ids[i]].lfill[l];
        values += rows * c->Hk * c->D;
        rows_m += rows * n_q[i] * c->r;
        all_rows += rows;
    }
    const bool sixteen = act == KVC_ACT_BF16 || (act == KVC_ACT_F16 && c->tv == KVC_F16);
    const bool tc = act != KVC_ACT_F32 && (c->block_kernel ? c->block_kernel == 2 : sixteen && tree_tc_pays(values, rows_m, all_rows));
    BlockParams p;
    block_params(c, layer, kq_scale, act, p);
    p.q = q;
    p.out = out;
    p.parent = parent;
    p.part = c->block_part;
    p.part_cap = part_rows_cap(c->sms);
    int64_t tok0 = 0;
    for (int i = 0; i < n_seq; ++i) {
        if (n_q[i] > 0) {
            const Seq &sq = c->seqs[(size_t)seq_ids[i]];
            BlockSeq &s = p.seq[p.n_seq++];
            s.id = seq_ids[i];
            s.off = sq.off;
            s.n_rows = sq.lfill[l];
            s.tok0 = (int32_t)tok0;
            s.n_tok = n_q[i];
        }
        tok0 += n_q[i];
        if (p.n_seq == 0 || (p.n_seq < MAX_SEQ_PER_LAUNCH && i + 1 < n_seq)) continue;
        cudaError_t e;
        if (tc) {
            plan_tree_tc(p, c->sms);
            e = launch_tree_tc(c->tk, c->tv, p, st);
        } else {
            plan_tree(p, c->sms);
            e = by_warps(p, maps, st);
        }
        if (e != cudaSuccess) return cuda_fail(c, e, "tree attention kernel");
        p.n_seq = 0;
    }
    // Kernels after these start only once they have waited for all before them (captured ones wait at their replays).
    cudaStreamCaptureStatus status = cudaStreamCaptureStatusActive;
    KVC_CU(c, cudaStreamIsCapturing(st, &status));
    if (status == cudaStreamCaptureStatusNone) c->clear_recent();
    return KVC_OK;
}

extern "C" int kvc_attn_weight(kvc_ctx *cc, int layer, int n_seq, const int32_t *seq_ids, const int32_t *n_q, int act,
                               const void *q, const float *lse, const int32_t *n_vis, float kq_scale, float *w,
                               int64_t w_stride, void *stream) {
    if (!cc) return KVC_EINVAL;
    Ctx *c = reinterpret_cast<Ctx *>(cc);
    int64_t total = 0;
    int rc = block_check(c, layer, n_seq, seq_ids, n_q, act, q, kq_scale, &total);
    if (rc) return rc;
    for (int i = 0; i < n_seq; ++i)
        if (w_stride < c->seqs[(size_t)seq_ids[i]].lfill[(size_t)layer])
            return c->fail(KVC_EINVAL, "w_stride is below the rows of a sequence");
    if (total == 0) return KVC_OK;
    if (!lse || !w) return c->fail(KVC_EINVAL, "lse and w must be non-null");
    if (((uintptr_t)lse | (uintptr_t)n_vis | (uintptr_t)w) & 3)
        return c->fail(KVC_EINVAL, "lse, n_vis and w must be 4-byte aligned");
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    KVC_CU(c, cudaSetDevice(c->dev));
    int64_t tok0 = 0;
    for (int base = 0; base < n_seq; base += MAX_SEQ_PER_LAUNCH) {
        BlockParams p;
        block_params(c, layer, kq_scale, act, p);
        p.q = q;
        p.lse = const_cast<float *>(lse); // only read
        p.n_vis = n_vis;
        p.w = w;
        p.w_stride = w_stride;
        p.n_seq = std::min(MAX_SEQ_PER_LAUNCH, n_seq - base);
        p.part_rows = 1;
        for (int i = 0; i < p.n_seq; ++i) {
            BlockSeq &s = p.seq[i];
            const Seq &sq = c->seqs[(size_t)seq_ids[base + i]];
            s.id = seq_ids[base + i];
            s.off = sq.off;
            s.n_rows = sq.lfill[(size_t)layer];
            s.tok0 = (int32_t)tok0;
            s.n_tok = n_q[base + i];
            s.w_index = base + i;
            s.tiles = s.n_tok > 0 && s.n_rows > 0 ? 1 : 0;
            tok0 += s.n_tok;
        }
        plan_splits(p, c->sms, WEIGHT_STEP, WEIGHT_STEP, INT32_MAX); // (no partial rows: a cached row's sum is one item's)
        cudaError_t e = launch_weight(c->tk, p, st);
        if (e != cudaSuccess) return cuda_fail(c, e, "row weight kernel");
    }
    return KVC_OK;
}

extern "C" int kvc_debug_block_kernel(kvc_ctx *cc, int which) {
    if (!cc) return KVC_EINVAL;
    Ctx *c = reinterpret_cast<Ctx *>(cc);
    if (which < 0 || which > 2) return c->fail(KVC_EINVAL, "which must be 0, 1 or 2");
    c->block_kernel = which;
    return KVC_OK;
}

extern "C" int kvc_debug_block_plan(int n_head, int n_head_kv, int head_dim, int act, int sms, int n_seq,
                                    const int32_t *rows, const int32_t *n_q, int32_t *tile_m, int32_t *whole,
                                    int32_t *splits, int32_t *split_rows, int64_t *items, int64_t *part_rows,
                                    int64_t *part_cap) {
    if (n_head_kv < 1 || n_head < n_head_kv || n_head % n_head_kv || n_head / n_head_kv > MAX_GROUP ||
        (head_dim != 64 && head_dim != 128) || act < KVC_ACT_F32 || act > KVC_ACT_BF16 || sms < 1 || n_seq < 1 ||
        n_seq > MAX_SEQ_PER_LAUNCH || !rows || !n_q || !tile_m || !whole || !splits || !split_rows || !items || !part_rows ||
        !part_cap)
        return KVC_EINVAL;
    BlockParams p;
    std::memset(&p, 0, sizeof(p));
    p.H = n_head;
    p.Hk = n_head_kv;
    p.D = head_dim;
    p.r = n_head / n_head_kv;
    p.act = act;
    p.n_seq = n_seq;
    int64_t total = 0;
    for (int i = 0; i < n_seq; ++i) {
        if (rows[i] < 0 || n_q[i] < 0) return KVC_EINVAL;
        total += n_q[i];
        p.seq[i].n_rows = rows[i];
        p.seq[i].n_tok = n_q[i];
    }
    if (total * p.r > INT32_MAX / 4 / p.Hk) return KVC_EINVAL;
    plan_block(p, sms, act != KVC_ACT_F32);
    *tile_m = p.tile_m;
    *items = p.n_items;
    *part_rows = 0;
    *part_cap = part_rows_cap(sms);
    for (int i = 0; i < n_seq; ++i) {
        const BlockSeq &s = p.seq[i];
        whole[i] = s.whole;
        splits[i] = s.splits;
        split_rows[i] = s.split_rows;
        const int64_t cut = (int64_t)s.tiles * p.Hk - s.whole;
        *part_rows = std::max<int64_t>(*part_rows, s.part_row0 + cut * s.splits * p.part_rows);
    }
    return KVC_OK;
}

extern "C" int kvc_debug_recent_rows(kvc_ctx *cc, int layer, int seq, int32_t *rows) {
    if (!cc || !rows) return KVC_EINVAL;
    Ctx *c = reinterpret_cast<Ctx *>(cc);
    if (layer < 0 || layer >= c->L || seq < 0 || seq >= (int)c->recent.size()) return c->fail(KVC_EINVAL, "ids out of range");
    *rows = c->recent[(size_t)seq][(size_t)layer];
    return KVC_OK;
}

// The launch of a tree attention test hook, checked.
static bool tree_launch(int n_head, int n_head_kv, int sms, int n_seq, const int32_t *rows, const int32_t *off, const int32_t *n_q,
                        BlockParams &p) {
    if (n_head_kv < 1 || n_head < n_head_kv || n_head % n_head_kv || n_head / n_head_kv > MAX_GROUP || sms < 1 || n_seq < 1 ||
        n_seq > MAX_SEQ_PER_LAUNCH || !rows || !n_q)
        return false;
    std::memset(&p, 0, sizeof(p));
    p.H = n_head;
    p.Hk = n_head_kv;
    p.r = n_head / n_head_kv;
    p.n_seq = n_seq;
    for (int i = 0; i < n_seq; ++i) {
        if (n_q[i] < 1 || n_q[i] > TREE_MAX || rows[i] < n_q[i] || (off && off[i] < 0)) return false;
        p.seq[i].n_rows = rows[i];
        p.seq[i].off = off ? off[i] : 0;
        p.seq[i].n_tok = n_q[i];
        p.seq[i].id = i;
    }
    return true;
}

// Partial rows that the launch's parts take up.
static int64_t part_rows_of(const BlockParams &p) {
    int64_t most = 0;
    for (int i = 0; i < p.n_seq; ++i) {
        const BlockSeq &s = p.seq[i];
        const int64_t cut = (int64_t)s.tiles * p.Hk - s.whole;
        most = std::max<int64_t>(most, s.part_row0 + cut * s.splits * p.part_rows);
    }
    return most;
}

extern "C" int kvc_debug_tree_plan(int n_head, int n_head_kv, int sms, int n_seq, const int32_t *rows, const int32_t *off,
                                   const int32_t *n_q, int32_t *tile_m, int32_t *whole, int32_t *splits, int32_t *split_rows,
                                   int64_t *items, int64_t *part_rows, int64_t *part_cap) {
    BlockParams p;
    if (!off || !tile_m || !whole || !splits || !split_rows || !items || !part_rows || !part_cap ||
        !tree_launch(n_head, n_head_kv, sms, n_seq, rows, off, n_q, p))
        return KVC_EINVAL;
    plan_tree(p, sms);
    *tile_m = p.tile_m;
    *items = p.n_items;
    *part_rows = part_rows_of(p);
    *part_cap = part_rows_cap(sms);
    for (int i = 0; i < n_seq; ++i) {
        const BlockSeq &s = p.seq[i];
        whole[s.id] = s.whole;
        splits[s.id] = s.splits;
        split_rows[s.id] = s.split_rows;
    }
    return KVC_OK;
}

extern "C" int kvc_debug_tree_plan_tc(int n_head, int n_head_kv, int sms, int n_seq, const int32_t *rows, const int32_t *n_q,
                                      int32_t *tile_m, int32_t *n_entries, kvc_debug_entry *entries, int64_t *items,
                                      int64_t *part_rows, int64_t *part_cap) {
    BlockParams p;
    if (!tile_m || !n_entries || !entries || !items || !part_rows || !part_cap ||
        !tree_launch(n_head, n_head_kv, sms, n_seq, rows, nullptr, n_q, p))
        return KVC_EINVAL;
    plan_tree_tc(p, sms);
    *tile_m = p.tile_m;
    *items = p.n_items;
    *part_rows = part_rows_of(p);
    *part_cap = part_rows_cap(sms);
    *n_entries = p.n_seq;
    for (int i = 0; i < p.n_seq; ++i) {
        const BlockSeq &s = p.seq[i];
        const int64_t cut = (int64_t)s.tiles * p.Hk - s.whole;
        entries[i] = {s.id, s.tile0, s.tiles, s.whole, s.splits, s.split_rows, s.item0, s.part_row0, (int32_t)(cut * s.splits * p.part_rows),
                      s.cut0};
    }
    return KVC_OK;
}
