// head.h -- the output layer's losses: what head_api.cu (argument checks,
// workspace, order of launches) hands to head.cu (kernels).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace gb300 {

constexpr int kHeadTile = 128;   // words to a softmax statistic

// Where each token's target comes from, and the compact order of the tokens
// that have one: perm[r] is the token at place r, rank[n] the place of token
// n; the first *count places hold the tokens with a target in their own
// order, the rest the others in theirs.  Without an order (perm, count NULL)
// each token is its own place and is asked for its target.
struct HeadRows {
    int64_t tokens, vocab, dim;
    int distill;
    // cross entropy
    const int64_t* target;
    int64_t target_stride, ignore_index;
    // distillation, written by teacher_launch: the entries of each token in
    // the order of their words (kNoWord past the last), log q, and whether
    // there is any
    int top_k;
    int32_t* words;
    float* logq;
    uint8_t* active;
    // the order
    int32_t* count;
    int32_t* perm;
    int32_t* rank;
    int32_t* target_c;   // cross entropy: target by place
};

constexpr int32_t kNoWord = 0x7FFFFFFF;

// Cross entropy: the word that token i is to become, kNoWord if it has none
// (the ignored word, or one outside the vocabulary).
__device__ __forceinline__ int32_t head_target(const int64_t* target, int64_t stride, int64_t ignore_index,
                                               int64_t vocab, int i) {
    const int64_t t = target[static_cast<int64_t>(i) * stride];
    return t != ignore_index && t >= 0 && t < vocab ? static_cast<int32_t>(t) : kNoWord;
}

// Gathers hidden rows into the compact order (row stride ldc, a multiple of
// 8; the columns from dim to ldc are zeros) and fills HeadRows' order.  The
// rows from *count up to the next multiple of pad_rows are zeros.  With lse
// (backward), it also lays out by place what the logits' gradient takes:
// lse2 = lse log2 e, gain = grad_loss / top * unit and boost = 1 + 2 z_loss
// lse, and writes the factor that undoes the gain's scaling, factor = top *
// undo.  top is the largest of size = |grad_loss|
// (1 + |2 z_loss lse|), which bounds a token's gradient of the logits, so that
// none passes unit in size.  It is the largest of the finite ones: an infinite
// or NaN grad_loss stays with its token's row, and with the sums that the row
// goes into.
// by_row (a type with few exponents, and dhidden is wanted): where sizes
// differ by more than kHeadSpread, a row of dhidden would be summed from
// numbers that fall below the type's normal ones.  *spread is then 1, every
// row has a gain of its own, unit / (1 + |2 z_loss lse|), and ratio turns it
// into the gain relative to top, which dweight needs, as its sums run over
// rows.  undo_row undoes a row's gain, whichever it is.
// With zero_rows, the rows there of tokens without a target are zeroed
// (element type zero_ct).
struct GatherArgs {
    HeadRows rows;
    const uint16_t* hidden;
    int64_t ldh;
    uint16_t* out;
    int64_t ldc;
    int pad_rows;
    const float* lse;
    const float* grad_loss;
    int64_t grad_stride;
    float z_loss, unit, undo;
    float *lse2, *gain, *boost, *factor, *undo_row, *ratio;
    int by_row;
    int32_t* spread;
    void* zero_rows;
    int64_t ld_zero;
    int zero_ct;
};
constexpr float kHeadSpread = 16.0f;
cudaError_t gather_launch(const GatherArgs& a, int sms, cudaStream_t stream);

struct TeacherArgs {
    const int64_t* index;
    int64_t ld_index;
    const void* logits;
    int64_t ld_logits;
    int dtype;   // 0 FP32, 1 FP16, 2 BF16
    int64_t tokens, vocab;
    int top_k;
    float temperature;
    int32_t* words;
    float* logq;
    uint8_t* active;
};
cudaError_t teacher_launch(const TeacherArgs& a, cudaStream_t stream);

// Copies rows of 16-bit elements to rows of stride ldc (a multiple of 8),
// zeros from cols to ldc.
cudaError_t pack_rows_launch(const uint16_t* in, int64_t ld, int64_t rows, int64_t cols,
                             uint16_t* out, int64_t ldc, int sms, cudaStream_t stream);

// Joins the statistics of all tiles -- stats[tile * ld_stats + place] is the
// largest z log2 e of a tile's words and the sum of 2^(z log2 e - largest),
// zsum the plain sum of logits, z_at the logits at the target ([place]) or at
// the teacher's words ([token * top_k + entry]) -- and writes loss and lse by
// token.
struct JoinArgs {
    HeadRows rows;
    const float2* stats;
    const float* zsum;
    int64_t ld_stats;
    int tiles;
    const float* z_at;
    float scale, scale2;     // logits to z, and to z log2 e
    float label_smoothing, z_loss, temperature;
    float *loss, *lse;
};
cudaError_t join_launch(const JoinArgs& a, cudaStream_t stream);

// out[i][j] = f * sum_s parts[s][row(i)][j], row(i) = rank[i] if rank (and
// zeros where that is not below *count), else i; f = row_factor[row(i)] if
// row_factor, else *factor.
struct SumRowsArgs {
    void* out;
    int ct;   // 0 FP32, 1 FP16, 2 BF16
    int64_t rows, cols, ldo;
    const float* parts;
    int nparts;
    int64_t part_stride, ld;
    const int32_t* rank;
    const int32_t* count;
    const float* factor;
    const float* row_factor;
};
cudaError_t sum_rows_launch(const SumRowsArgs& a, int sms, cudaStream_t stream);

}  // namespace gb300
