// head_api.cu -- the C entry points of the output layer's losses
// (gemm_ce_*, gemm_distill_*): argument checks, the layout of the caller's
// workspace and the order of launches.  The kernels are in
// head.cu and head_gemm.cu.

#include <algorithm>
#include <cmath>
#include <cstdio>
#include <cstring>
#include <limits>

#include "../../include/gb300gemm.h"
#include "cstore.cuh"
#include "head.h"
#include "head_gemm.h"
#include "internal.h"

using namespace gb300;

namespace {

#define GB_TRY(call)                                  \
    do {                                              \
        const gemm_status_t st_ = (call);             \
        if (st_ != GEMM_OK) return st_;               \
    } while (0)

// Tiles past the last row or column still have 32-bit coordinates.
constexpr int64_t kMostSize = (1ll << 31) - 1024;
// Elements of a matrix: 2^12 times what the memory holds.  The workspace, at
// most 64 FP32 parts and two copies of such matrices, stays far inside 64 bits.
constexpr int64_t kMostElements = 1ll << 50;

int64_t round_up(int64_t a, int64_t m) { return (a + m - 1) / m * m; }

struct Span {
    uintptr_t lo, hi;
};

// Rows of `cols` elements of `esize` bytes, `ld` apart.
Span span_of(const void* p, int64_t rows, int64_t cols, int64_t ld, int64_t esize) {
    if (!p || rows <= 0 || cols <= 0) return Span{0, 0};
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return Span{lo, lo + static_cast<uintptr_t>(((rows - 1) * ld + cols) * esize)};
}

bool meet(const Span& a, const Span& b) { return a.lo < b.hi && b.lo < a.hi; }

bool off(const void* p, uintptr_t align) { return (reinterpret_cast<uintptr_t>(p) & (align - 1)) != 0; }

// (rows - 1) * ld stays far inside 64 bits once multiplied by an element size.
bool far(int64_t rows, int64_t ld) { return rows > 1 && ld > (std::numeric_limits<int64_t>::max() / 64) / (rows - 1); }

gemm_status_t check_head(const gemm_head_t* h, int distill) {
    if (!h) return lib_invalid("head is NULL");
    if (h->dtype < 0 || h->dtype > 1) return lib_invalid("dtype is neither FP16 nor BF16");
    if (h->grad_dtype < 0 || h->grad_dtype > 1) return lib_invalid("grad_dtype");
    if (h->tokens < 0 || h->vocab < 0 || h->dim < 0 || h->tokens > kMostSize || h->vocab > kMostSize ||
        h->dim > kMostSize)
        return lib_invalid("tokens, vocab and dim must be in [0, 2^31 - 1024]");
    if (h->tokens * h->vocab > kMostElements || h->tokens * h->dim > kMostElements ||
        h->vocab * h->dim > kMostElements)
        return lib_invalid("no two of tokens, vocab and dim may have a product above 2^50");
    if (h->ldh < h->dim || h->ldw < h->dim || far(h->tokens, h->ldh) || far(h->vocab, h->ldw))
        return lib_invalid("row stride of hidden or weight");
    if (!(h->logit_scale > 0.0f) || !std::isfinite(h->logit_scale)) return lib_invalid("logit_scale");
    if (h->piece_bytes < 0) return lib_invalid("piece_bytes");
    if (off(h->hidden, 2) || off(h->weight, 2)) return lib_invalid("hidden or weight off its type's alignment");
    if (distill) {
        if (!(h->temperature > 0.0f) || !std::isfinite(h->temperature)) return lib_invalid("temperature");
        if (h->top_k < 1 || h->top_k > GEMM_DISTILL_MAX_TOP_K) return lib_invalid("top_k");
        if (h->teacher_dtype < 0 || h->teacher_dtype > 2) return lib_invalid("teacher_dtype");
        if (h->ld_index < 0 || h->ld_logits < 0 || (h->ld_index < h->top_k && h->ld_index != 0) ||
            (h->ld_logits < h->top_k && h->ld_logits != 0) || far(h->tokens, h->ld_index) ||
            far(h->tokens, h->ld_logits))
            return lib_invalid("row stride of teacher_index or teacher_logits");
        if (off(h->teacher_index, 8) || off(h->teacher_logits, h->teacher_dtype == 0 ? 4 : 2))
            return lib_invalid("teacher_index or teacher_logits off its type's alignment");
    } else {
        if (!(h->label_smoothing >= 0.0f && h->label_smoothing <= 1.0f)) return lib_invalid("label_smoothing");
        if (!(h->z_loss >= 0.0f) || !std::isfinite(h->z_loss)) return lib_invalid("z_loss");
        if (h->target_stride < 0 || far(h->tokens, h->target_stride)) return lib_invalid("target_stride");
        if (off(h->target, 8)) return lib_invalid("target off its type's alignment");
    }
    if (h->tokens > 0) {
        if (h->vocab < 1) return lib_invalid("vocab is 0");
        if (h->dim > 0 && (!h->hidden || !h->weight)) return lib_invalid("hidden or weight is NULL");
        if (distill ? (!h->teacher_index || !h->teacher_logits) : !h->target)
            return lib_invalid(distill ? "teacher_index or teacher_logits is NULL" : "target is NULL");
    }
    return GEMM_OK;
}

// The stride of a single row is never taken, whatever it is, but a tensor map
// holds strides below 2^40 bytes only: one that suits the copies stands for it.
gemm_head_t with_strides(const gemm_head_t& head) {
    gemm_head_t h = head;
    if (h.tokens <= 1) h.ldh = round_up(h.dim, 8);
    if (h.vocab <= 1) h.ldw = round_up(h.dim, 8);
    return h;
}

constexpr int kClusters = 76;   // CTA pairs of the 152 SMs; the workspace's size goes by it

// Whether the two gradient products go in one launch, whose clusters share the
// units of both.  With few tokens and a weight past L2 each product has a bound
// of its own (dhidden reads the weight, dweight is written), and a launch and a
// ring of its own pay: the backward call took, together and apart,
//     tokens x words x channels     16 x 65536 x 4096    383   307 us
//                                  128 x 65536 x 2048    214   187
//                                  512 x 131072 x 4096  1375  1289
//                                 1024 x 131072 x 4096  2236  2315
//                                   16 x 65536 x 1024    114   114
//                                   64 x 32768 x 1024     66    75
bool products_together(const gemm_head_t& h) {
    return !(h.tokens <= 512 && 2 * h.vocab * h.dim >= (1 << 27));
}

// How many slices the K of both gradient products is cut into: the least
// time, counted in K steps of one cluster.  A step of 256 x 256 x 128 takes
// about 0.55 us; one cluster's share of the memory bandwidth (6.8 TB/s / 76)
// moves an FP32 tile in 2.9 us, 5.3 steps, once when a slice is written and
// once when the slices are summed, by a launch of its own (4 us, 7 steps); a
// single slice is written in its final form, 2.6 steps, unless dhidden has
// more than one piece to sum (h_parts).  Products in one launch share the
// clusters evenly, but no unit ends before its own K does; a product alone
// takes whole rounds of its units.
struct Slices {
    int h, w;
};

Slices slices(bool together, int64_t h_tiles, int64_t h_steps, bool h_parts, int64_t w_tiles, int64_t w_steps) {
    Slices best{1, 1};
    double least = 0.0;
    for (int h = 1; h <= 64 && (h == 1 || h_steps >= 4 * h); ++h) {
        for (int w = 1; w <= 64 && (w == 1 || w_steps >= 4 * w); ++w) {
            const bool hp = h_parts || h > 1, wp = w > 1;
            const double h_unit = static_cast<double>(ceil_div(h_steps, h)) + (hp ? 5.3 : 2.6);
            const double w_unit = static_cast<double>(ceil_div(w_steps, w)) + (wp ? 5.3 : 2.6);
            const double even = (h_tiles * h * h_unit + w_tiles * w * w_unit) / kClusters;
            const double rounds = static_cast<double>(ceil_div(h_tiles * h, kClusters)) * h_unit +
                                  static_cast<double>(ceil_div(w_tiles * w, kClusters)) * w_unit;
            const double sums = (hp ? 7.0 + 5.3 * static_cast<double>(h_tiles * h) / kClusters : 0.0) +
                                (wp ? 7.0 + 5.3 * static_cast<double>(w_tiles * w) / kClusters : 0.0);
            const double cost = (together ? std::max({even, h_unit, w_unit}) : rounds) + sums;
            if ((h == 1 && w == 1) || cost < least) {
                least = cost;
                best = Slices{h, w};
            }
        }
    }
    return best;
}

// The workspace: regions on 256-byte boundaries, one after the other.
struct Layout {
    int64_t bytes = 0;
    int64_t dp, piece, np, tiles;   // padded dim, words of a piece, padded tokens
    int64_t count, factor, perm, rank, target_c, words, logq, active, lse2, gain, boost, z_at, stats, zsum;
    int64_t undo_row, ratio, spread;
    int64_t hidden = 0, weight, grad, by_row, dh, dw;
    int h_slices, w_slices;
    bool h_direct;      // dhidden needs no sum of parts: one piece, one slice
    bool pack_weight;
    bool in_place;      // forward: hidden is read where it is
};

Layout layout_of(const gemm_head_t& h, int distill, int backward) {
    Layout l;
    const int64_t n = h.tokens;
    auto take = [&](int64_t bytes) {
        const int64_t at = l.bytes;
        l.bytes += round_up(std::max<int64_t>(bytes, 1), 256);
        return at;
    };
    l.dp = std::max<int64_t>(64, round_up(h.dim, 64));   // rows on 128-byte lines
    l.np = round_up(n, kHeadTileM);
    l.tiles = ceil_div(h.vocab, kHeadTile);
    const int64_t limit = h.piece_bytes > 0 ? h.piece_bytes : GEMM_HEAD_PIECE_BYTES;
    const int64_t most = std::max<int64_t>(1, limit / (2 * std::max<int64_t>(n, 1)) / kHeadTileN) * kHeadTileN;
    const int64_t pieces = std::max<int64_t>(1, ceil_div(h.vocab, most));
    l.piece = round_up(ceil_div(std::max<int64_t>(h.vocab, 1), pieces), kHeadTileN);
    l.pack_weight = h.dim > 0 && (off(h.weight, 16) || (h.ldw & 7));

    l.count = take(4);
    l.factor = take(4);
    l.perm = take(4 * n);
    l.rank = take(4 * n);
    l.target_c = l.words = l.logq = l.active = 0;
    l.lse2 = l.gain = l.boost = l.z_at = l.stats = l.zsum = l.grad = l.by_row = l.dh = l.dw = l.weight = 0;
    l.undo_row = l.ratio = l.spread = 0;
    l.h_slices = l.w_slices = 1;
    l.h_direct = false;
    // A forward call of up to one tile of tokens saves no product by leaving
    // some out, and a token's row of logits is its own whatever the others
    // hold: the rows are read in place (16 x 1000 x 256: one launch of 4 us
    // less), where the tensor unit can take them.
    l.in_place = !backward && n <= kHeadTileM && h.dim > 0 && !off(h.hidden, 16) && (h.ldh & 7) == 0;
    if (distill) {
        l.words = take(4 * n * h.top_k);
        l.logq = take(4 * n * h.top_k);
        l.active = take(n);
    } else {
        l.target_c = take(4 * n);
    }
    if (!l.in_place) l.hidden = take(2 * n * l.dp);
    if (l.pack_weight) l.weight = take(2 * h.vocab * l.dp);
    if (!backward) {
        l.z_at = take(4 * n * (distill ? h.top_k : 1));
        l.stats = take(8 * l.tiles * l.np);
        if (!distill && h.label_smoothing > 0.0f) l.zsum = take(4 * l.tiles * l.np);
    } else {
        l.lse2 = take(4 * n);
        l.gain = take(4 * n);
        l.boost = take(4 * n);
        l.undo_row = take(4 * n);
        l.ratio = take(4 * n);
        l.spread = take(4);
        l.grad = take(2 * n * l.piece);
        // FP16: the copy with a scale for each row, written where weights differ much
        if (h.dtype == 0) l.by_row = take(2 * n * l.piece);
        const int64_t dim_tiles = ceil_div(h.dim, kHeadTileN);
        const Slices both = slices(products_together(h), ceil_div(n, kHeadTileM) * dim_tiles,
                                   l.piece / kHeadStepK, l.piece < h.vocab, l.piece / kHeadTileM * dim_tiles,
                                   ceil_div(n, kHeadStepK));
        l.h_slices = both.h;
        l.w_slices = both.w;
        l.h_direct = l.piece >= h.vocab && l.h_slices == 1;
        if (!l.h_direct) l.dh = take(4 * l.h_slices * l.np * l.dp);
        if (l.w_slices > 1) l.dw = take(4 * l.w_slices * l.piece * l.dp);
    }
    return l;
}

template <class T>
T* at(void* ws, int64_t offset) {
    return reinterpret_cast<T*>(static_cast<char*>(ws) + offset);
}

HeadRows rows_of(const gemm_head_t& h, int distill, const Layout& l, void* ws) {
    HeadRows r;
    memset(&r, 0, sizeof(r));
    r.tokens = h.tokens;
    r.vocab = h.vocab;
    r.dim = h.dim;
    r.distill = distill;
    if (!l.in_place) {
        r.count = at<int32_t>(ws, l.count);
        r.perm = at<int32_t>(ws, l.perm);
        r.rank = at<int32_t>(ws, l.rank);
    }
    if (distill) {
        r.top_k = h.top_k;
        r.words = at<int32_t>(ws, l.words);
        r.logq = at<float>(ws, l.logq);
        r.active = at<uint8_t>(ws, l.active);
    } else {
        r.target = h.target;
        r.target_stride = h.target_stride;
        r.ignore_index = h.ignore_index;
        r.target_c = at<int32_t>(ws, l.target_c);
    }
    return r;
}

gemm_status_t check_workspace(const void* ws, int64_t have, const Layout& l) {
    if (!ws || off(ws, 256)) return lib_invalid("workspace is NULL or off a 256-byte boundary");
    if (have < l.bytes) {
        char text[96];
        snprintf(text, sizeof(text), "workspace of %lld bytes, %lld needed", static_cast<long long>(have),
                 static_cast<long long>(l.bytes));
        return lib_invalid(text);
    }
    return GEMM_OK;
}

// What the call reads, and whether anything in `outs` meets it or another output.
gemm_status_t check_overlap(const gemm_head_t& h, int distill, const Span* more, int nmore, const Span* outs,
                            int nouts) {
    Span ins[8];
    int n = 0;
    ins[n++] = span_of(h.hidden, h.tokens, h.dim, h.ldh, 2);
    ins[n++] = span_of(h.weight, h.vocab, h.dim, h.ldw, 2);
    if (distill) {
        ins[n++] = span_of(h.teacher_index, h.tokens, h.top_k, h.ld_index, 8);
        ins[n++] = span_of(h.teacher_logits, h.tokens, h.top_k, h.ld_logits, h.teacher_dtype == 0 ? 4 : 2);
    } else {
        ins[n++] = span_of(h.target, h.tokens, 1, h.target_stride, 8);
    }
    for (int i = 0; i < nmore; ++i) ins[n++] = more[i];
    for (int i = 0; i < nouts; ++i) {
        for (int j = 0; j < n; ++j)
            if (meet(outs[i], ins[j])) return GEMM_ERR_OVERLAP;
        for (int j = 0; j < i; ++j)
            if (meet(outs[i], outs[j])) return GEMM_ERR_OVERLAP;
    }
    return GEMM_OK;
}

// The steps that forward and backward share: the teacher's list, the weight
// as the products can take it, and the compact rows.
gemm_status_t begin(const gemm_head_t& h, int distill, const Layout& l, void* ws, GatherArgs& g, int sms,
                    cudaStream_t stream, const uint16_t** weight, int64_t* ldw) {
    const HeadRows r = rows_of(h, distill, l, ws);
    if (distill) {
        TeacherArgs t;
        t.index = h.teacher_index;
        t.ld_index = h.ld_index;
        t.logits = h.teacher_logits;
        t.ld_logits = h.ld_logits;
        t.dtype = h.teacher_dtype;
        t.tokens = h.tokens;
        t.vocab = h.vocab;
        t.top_k = h.top_k;
        t.temperature = h.temperature;
        t.words = r.words;
        t.logq = r.logq;
        t.active = r.active;
        GB_TRY(lib_launch_status(teacher_launch(t, stream), "teacher"));
    }
    g.rows = r;
    g.hidden = static_cast<const uint16_t*>(h.hidden);
    g.ldh = h.ldh;
    g.out = at<uint16_t>(ws, l.hidden);
    g.ldc = l.dp;
    if (!l.in_place) GB_TRY(lib_launch_status(gather_launch(g, sms, stream), "gather"));
    *weight = static_cast<const uint16_t*>(h.weight);
    *ldw = h.ldw;
    if (l.pack_weight) {
        uint16_t* packed = at<uint16_t>(ws, l.weight);
        GB_TRY(lib_launch_status(pack_rows_launch(*weight, h.ldw, h.vocab, h.dim, packed, l.dp, sms, stream),
                                 "pack_rows"));
        *weight = packed;
        *ldw = l.dp;
    }
    return GEMM_OK;
}

HeadOperand operand(const void* base, int64_t inner, int64_t outer, int64_t ld, int kmajor) {
    HeadOperand o;
    o.base = base;
    o.inner = inner;
    o.outer = outer;
    o.ld = ld;
    o.kmajor = kmajor;
    return o;
}

// The product of compact hidden rows and words w0 .. w0 + cols, K = dim.
void logits_of(const gemm_head_t& h, const Layout& l, const GatherArgs& g, const uint16_t* weight, int64_t ldw,
               int64_t w0, int64_t cols, HeadGemm* p) {
    p->m = h.tokens;
    p->n = cols;
    p->k = h.dim;
    p->count_is = l.in_place ? 0 : 1;
    p->splits = 1;
    p->p = l.in_place ? operand(h.hidden, h.dim, h.tokens, h.ldh, 1) : operand(g.out, l.dp, h.tokens, l.dp, 1);
    // without channels there is no weight to read: any operand does, K is 0
    p->q = h.dim > 0 ? operand(weight + w0 * ldw, h.dim, cols, ldw, 1) : p->p;
    p->w0 = w0;
}

// pairs resident at once; more than that would only wait their turn
int clusters_at_once() {
    const int clusters = lib_pair_clusters();
    return clusters > 0 ? clusters : kClusters;
}

gemm_status_t run_gemm(const HeadGemm& p, const HeadGemm* and_then, cudaStream_t stream) {
    EncodeTiledFn encode = lib_encode_fn();
    if (!encode) {
        lib_invalid("cuTensorMapEncodeTiled entry point unavailable");
        return GEMM_ERR_CUDA;
    }
    return lib_launch_status(head_gemm_launch(p, and_then, clusters_at_once(), encode, stream), "head_gemm");
}

float scale_of(const gemm_head_t& h, int distill) {
    return distill ? h.logit_scale / h.temperature : h.logit_scale;
}

constexpr float kLog2e = 1.4426950408889634f;
// Stages of 128 K summed in tensor memory before they are added in registers.
// Statistics: at 8192 x 131072 x 4096, chunks of 1, 2, 3, 4 and 8 stages took
// 6289, 5234, 5133, 5156 and 5174 us, with lse off by 0.9, 1.4, 2.1, 2.8 and
// 5.8e-7 (an FP32 product on the CUDA cores: 3.4e-7).  The logits' gradient is
// rounded to 16 bits anyway; its products sum up to 2^17 terms.  Where the
// weight's read is the bound (up to 64 tokens), chunks of 2 cost no more than
// of 3 (16 x 131072 x 4096: 178 and 177 us; of 1: 191).
constexpr int kFewStatsChunk = 2, kStatsChunk = 3, kChunk = 8;

// A self-test of the tensor-core kernel's bounded waits (gemm_ce_stall_selftest).
struct HeadStall {
    uint64_t limit_ns;
    int32_t cluster, fill;
};

gemm_status_t forward(const gemm_head_t* head, int distill, float* loss, float* lse, void* ws,
                      int64_t ws_bytes, gemm_stream_t stream_, const HeadStall* stall = nullptr) {
    GB_TRY(check_head(head, distill));
    const gemm_head_t h = with_strides(*head);
    if (h.tokens == 0) return GEMM_OK;
    if (!loss || !lse || off(loss, 4) || off(lse, 4)) return lib_invalid("loss or lse is NULL or misaligned");
    const Layout l = layout_of(h, distill, 0);
    GB_TRY(check_workspace(ws, ws_bytes, l));
    const Span outs[] = {span_of(loss, 1, h.tokens, h.tokens, 4), span_of(lse, 1, h.tokens, h.tokens, 4),
                         span_of(ws, 1, l.bytes, l.bytes, 1)};
    GB_TRY(check_overlap(h, distill, nullptr, 0, outs, 3));
    int dev, sms;
    GB_TRY(lib_device(&dev, &sms));
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);

    HeadGemm p;
    memset(&p, 0, sizeof(p));
    if (stall) {
        p.m = h.tokens;
        p.n = h.vocab;
        p.splits = 1;
        if (stall->cluster < 0 || stall->cluster >= head_gemm_clusters(p, nullptr, clusters_at_once()) || stall->fill < 0)
            return lib_invalid("stall self-test: stall_cluster or stall_fill");
        p.wait_limit_ns = stall->limit_ns;
        p.stall_cluster = stall->cluster;
        p.stall_fill = stall->fill + 1;
    }
    GatherArgs g;
    memset(&g, 0, sizeof(g));
    g.pad_rows = kHeadStepK;
    const uint16_t* weight;
    int64_t ldw;
    GB_TRY(begin(h, distill, l, ws, g, sms, stream, &weight, &ldw));

    p.mode = distill ? kHeadStatsKd : kHeadStatsCe;
    p.bf16 = h.dtype;
    p.rows = g.rows;
    p.chunk = h.tokens <= 64 ? kFewStatsChunk : kStatsChunk;
    p.scale2 = scale_of(h, distill) * kLog2e;
    p.stats = at<float2>(ws, l.stats);
    p.zsum = l.zsum ? at<float>(ws, l.zsum) : nullptr;
    p.ld_stats = l.np;
    p.z_at = at<float>(ws, l.z_at);
    logits_of(h, l, g, weight, ldw, 0, h.vocab, &p);
    GB_TRY(run_gemm(p, nullptr, stream));
    JoinArgs j;
    j.rows = g.rows;
    j.stats = p.stats;
    j.zsum = p.zsum;
    j.ld_stats = l.np;
    j.tiles = static_cast<int>(l.tiles);
    j.z_at = p.z_at;
    j.scale = scale_of(h, distill);
    j.scale2 = p.scale2;
    j.label_smoothing = distill ? 0.0f : h.label_smoothing;
    j.z_loss = distill ? 0.0f : h.z_loss;
    j.temperature = distill ? h.temperature : 1.0f;
    j.loss = loss;
    j.lse = lse;
    return lib_launch_status(join_launch(j, stream), "join");
}

gemm_status_t backward(const gemm_head_t* head, int distill, const float* lse, const float* grad_loss,
                       int64_t grad_stride, void* dhidden, int64_t lddh, void* dweight, int64_t lddw,
                       void* ws, int64_t ws_bytes, gemm_stream_t stream_) {
    GB_TRY(check_head(head, distill));
    const gemm_head_t h = with_strides(*head);
    const int ct = h.grad_dtype == 1 ? kCF32 : h.dtype == 1 ? kCBF16 : kCF16;
    const int64_t ge = c_elem_bytes(ct);
    if (dhidden && (lddh < h.dim || far(h.tokens, lddh) || off(dhidden, ge))) return lib_invalid("dhidden");
    if (dweight && (lddw < h.dim || far(h.vocab, lddw) || off(dweight, ge))) return lib_invalid("dweight");
    if (h.vocab <= 1) lddw = h.dim;
    if (h.tokens <= 1) lddh = h.dim;
    if (grad_stride < 0 || far(h.tokens, grad_stride)) return lib_invalid("grad_stride");
    const bool want_h = dhidden && h.tokens > 0 && h.dim > 0, want_w = dweight && h.vocab > 0 && h.dim > 0;
    if (!want_h && !want_w) return GEMM_OK;
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    int dev, sms;
    if (h.tokens == 0) {   // no token: the weight's gradient is the empty sum
        if (meet(span_of(dweight, h.vocab, h.dim, lddw, ge), span_of(h.weight, h.vocab, h.dim, h.ldw, 2)))
            return GEMM_ERR_OVERLAP;
        GB_TRY(lib_device(&dev, &sms));
        return lib_launch_status(fill_scale_launch(dweight, ct, h.vocab, h.dim, lddw, 0.0f, stream), "fill");
    }
    if (!lse || !grad_loss || off(lse, 4) || off(grad_loss, 4))
        return lib_invalid("lse or grad_loss is NULL or misaligned");
    const Layout l = layout_of(h, distill, 1);
    GB_TRY(check_workspace(ws, ws_bytes, l));
    const Span more[] = {span_of(lse, 1, h.tokens, h.tokens, 4), span_of(grad_loss, h.tokens, 1, grad_stride, 4)};
    const Span outs[] = {span_of(dhidden, h.tokens, h.dim, lddh, ge), span_of(dweight, h.vocab, h.dim, lddw, ge),
                         span_of(ws, 1, l.bytes, l.bytes, 1)};
    GB_TRY(check_overlap(h, distill, more, 2, outs, 3));
    GB_TRY(lib_device(&dev, &sms));

    // The gather scales the logits' gradient to at most 1 in size; FP16 holds
    // it times 2^14, so that probabilities down to 2^-28 of the largest stay
    // normal numbers.  BF16 has FP32's range and needs no unit.
    const float unit = h.dtype == 1 ? 1.0f : 16384.0f;
    GatherArgs g;
    memset(&g, 0, sizeof(g));
    g.pad_rows = kHeadStepK;
    g.lse = lse;
    g.grad_loss = grad_loss;
    g.grad_stride = grad_stride;
    g.z_loss = distill ? 0.0f : h.z_loss;
    g.unit = unit;
    // d logits / d z, and the loss's own factor
    g.undo = (distill ? h.temperature * h.logit_scale : h.logit_scale) / unit;
    g.lse2 = at<float>(ws, l.lse2);
    g.gain = at<float>(ws, l.gain);
    g.boost = at<float>(ws, l.boost);
    g.factor = at<float>(ws, l.factor);
    g.undo_row = at<float>(ws, l.undo_row);
    g.ratio = at<float>(ws, l.ratio);
    g.spread = at<int32_t>(ws, l.spread);
    g.by_row = h.dtype == 0 && want_h;
    if (want_h && l.h_direct) {
        g.zero_rows = dhidden;
        g.ld_zero = lddh;
        g.zero_ct = ct;
    }
    const uint16_t* weight;
    int64_t ldw;
    GB_TRY(begin(h, distill, l, ws, g, sms, stream, &weight, &ldw));

    HeadGemm d;   // the logits' gradient
    memset(&d, 0, sizeof(d));
    d.mode = distill ? kHeadGradKd : kHeadGradCe;
    d.bf16 = h.dtype;
    d.rows = g.rows;
    d.chunk = kChunk;
    d.scale2 = scale_of(h, distill) * kLog2e;
    d.label_smoothing = distill ? 0.0f : h.label_smoothing;
    d.lse2 = g.lse2;
    d.gain = g.gain;
    d.boost = g.boost;
    d.out = at<uint16_t>(ws, l.grad);
    d.ct = h.dtype == 1 ? kCBF16 : kCF16;
    d.out_inner = d.ldo = l.piece;
    d.out_outer = h.tokens;
    // without dweight the only copy is the one by rows
    if (g.by_row && want_w) {
        d.mode = distill ? kHeadGradKdRows : kHeadGradCeRows;
        d.spread = g.spread;
        d.by_row = at<uint16_t>(ws, l.by_row);
        d.ratio = g.ratio;
    }

    HeadGemm ph;   // dhidden = gradient weight, summed over the pieces
    memset(&ph, 0, sizeof(ph));
    ph.mode = kHeadProduct;
    ph.bf16 = h.dtype;
    ph.rows = g.rows;
    ph.count_is = 1;
    ph.m = h.tokens;
    ph.n = h.dim;
    ph.splits = l.h_slices;
    ph.chunk = kChunk;
    ph.p.kmajor = 1;
    ph.spread = d.spread;
    ph.by_row = d.by_row;
    if (l.h_direct) {   // straight to the tokens' rows
        ph.out = dhidden;
        ph.ct = ct;
        ph.out_inner = h.dim;
        ph.ldo = lddh;
        ph.out_outer = h.tokens;
        ph.out_perm = g.rows.perm;
        ph.factor = g.factor;
        ph.row_factor = g.by_row ? g.undo_row : nullptr;
    } else {
        ph.out = at<float>(ws, l.dh);
        ph.ct = kCF32;
        ph.out_inner = ph.ldo = l.dp;
        ph.split_rows = l.np;
        ph.out_outer = l.np * l.h_slices;
    }

    HeadGemm pw;   // dweight = gradient^T hidden, a piece of its rows at a time
    memset(&pw, 0, sizeof(pw));
    pw.mode = kHeadProduct;
    pw.bf16 = h.dtype;
    pw.rows = g.rows;
    pw.count_is = 2;
    pw.n = h.dim;
    pw.k = h.tokens;
    pw.splits = l.w_slices;
    pw.chunk = kChunk;
    pw.q = operand(g.out, l.dp, h.tokens, l.dp, 0);

    SumRowsArgs s;
    memset(&s, 0, sizeof(s));
    s.ct = ct;
    s.cols = h.dim;
    s.ld = l.dp;
    s.factor = g.factor;
    for (int64_t w0 = 0; w0 < h.vocab; w0 += l.piece) {
        const int64_t cols = std::min(l.piece, h.vocab - w0);
        logits_of(h, l, g, weight, ldw, w0, cols, &d);
        GB_TRY(run_gemm(d, nullptr, stream));
        if (want_h) {
            ph.k = cols;
            ph.p = operand(d.out, l.piece, h.tokens, l.piece, 1);
            ph.q = operand(weight + w0 * ldw, h.dim, cols, ldw, 0);
            ph.add = w0 > 0;
        }
        void* to = want_w ? static_cast<char*>(dweight) + w0 * lddw * ge : nullptr;
        if (want_w) {
            pw.m = cols;
            pw.p = operand(d.out, l.piece, h.tokens, l.piece, 0);
            if (l.w_slices > 1) {
                pw.out = at<float>(ws, l.dw);
                pw.ct = kCF32;
                pw.out_inner = pw.ldo = l.dp;
                pw.split_rows = l.piece;
                pw.out_outer = l.piece * l.w_slices;
            } else {
                pw.out = to;
                pw.ct = ct;
                pw.out_inner = h.dim;
                pw.ldo = lddw;
                pw.out_outer = cols;
                pw.factor = g.factor;
            }
        }
        // both products in one launch: the one with the longer K first
        const bool together = want_h && want_w && products_together(h);
        if (together) {
            const bool h_first = ph.k * pw.splits >= pw.k * ph.splits;
            GB_TRY(run_gemm(h_first ? ph : pw, h_first ? &pw : &ph, stream));
        } else {
            if (want_h) GB_TRY(run_gemm(ph, nullptr, stream));
            if (want_w) GB_TRY(run_gemm(pw, nullptr, stream));
        }
        if (want_w) {
            if (l.w_slices > 1) {
                s.out = to;
                s.rows = cols;
                s.ldo = lddw;
                s.parts = at<float>(ws, l.dw);
                s.nparts = l.w_slices;
                s.part_stride = l.piece * l.dp;
                GB_TRY(lib_launch_status(sum_rows_launch(s, sms, stream), "sum_rows"));
            }
        }
    }
    if (want_h && !l.h_direct) {
        s.out = dhidden;
        s.rows = h.tokens;
        s.ldo = lddh;
        s.parts = at<float>(ws, l.dh);
        s.nparts = l.h_slices;
        s.part_stride = l.np * l.dp;
        s.rank = g.rows.rank;
        s.count = g.rows.count;
        s.row_factor = g.by_row ? g.undo_row : nullptr;
        GB_TRY(lib_launch_status(sum_rows_launch(s, sms, stream), "sum_rows"));
    }
    return GEMM_OK;
}

}  // namespace

extern "C" {

gemm_status_t gemm_head_workspace(const gemm_head_t* head, int32_t distill, int32_t backward, int64_t* bytes) {
    if (!bytes || distill < 0 || distill > 1 || backward < 0 || backward > 1) return GEMM_ERR_INVALID_VALUE;
    GB_TRY(check_head(head, distill));
    *bytes = head->tokens == 0 ? 0 : layout_of(with_strides(*head), distill, backward).bytes;
    return GEMM_OK;
}

gemm_status_t gemm_ce_forward(const gemm_head_t* head, float* loss, float* lse, void* workspace,
                              int64_t workspace_bytes, gemm_stream_t stream) {
    return forward(head, 0, loss, lse, workspace, workspace_bytes, stream);
}

gemm_status_t gemm_ce_stall_selftest(const gemm_head_t* head, float* loss, float* lse, void* workspace,
                                     int64_t workspace_bytes, int32_t limit_ms, int32_t stall_cluster,
                                     int32_t stall_fill, gemm_stream_t stream) {
    if (limit_ms < 1 || limit_ms > 2000) return lib_invalid("limit_ms");
    const HeadStall t{static_cast<uint64_t>(limit_ms) * 1000000ull, stall_cluster, stall_fill};
    return forward(head, 0, loss, lse, workspace, workspace_bytes, stream, &t);
}

gemm_status_t gemm_distill_forward(const gemm_head_t* head, float* loss, float* lse, void* workspace,
                                   int64_t workspace_bytes, gemm_stream_t stream) {
    return forward(head, 1, loss, lse, workspace, workspace_bytes, stream);
}

gemm_status_t gemm_ce_backward(const gemm_head_t* head, const float* lse, const float* grad_loss,
                               int64_t grad_stride, void* dhidden, int64_t lddh, void* dweight,
                               int64_t lddw, void* workspace, int64_t workspace_bytes,
                               gemm_stream_t stream) {
    return backward(head, 0, lse, grad_loss, grad_stride, dhidden, lddh, dweight, lddw, workspace,
                    workspace_bytes, stream);
}

gemm_status_t gemm_distill_backward(const gemm_head_t* head, const float* lse, const float* grad_loss,
                                    int64_t grad_stride, void* dhidden, int64_t lddh, void* dweight,
                                    int64_t lddw, void* workspace, int64_t workspace_bytes,
                                    gemm_stream_t stream) {
    return backward(head, 1, lse, grad_loss, grad_stride, dhidden, lddh, dweight, lddw, workspace,
                    workspace_bytes, stream);
}

}  // extern "C"
