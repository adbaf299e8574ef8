// head_gemm.h -- one launch of the tensor-core kernel behind the output
// layer's losses (head_gemm.cu), as head_api.cu plans it.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "head.h"
#include "internal.h"

namespace gb300 {

constexpr int kHeadTileM = 256, kHeadTileN = 256;   // output tile of a CTA pair
constexpr int kHeadStepK = 128;                     // K of one pipeline stage

// What becomes of a tile of products.
enum HeadMode {
    kHeadStatsCe = 0,    // softmax statistics, and the logits at the targets
    kHeadStatsKd = 1,    // the same, and the logits at the teacher's words
    kHeadGradCe = 2,     // the logits' gradient, 16 bits
    kHeadGradKd = 3,
    kHeadProduct = 4,    // the products themselves
    // the logits' gradient with its copy by rows: forms of their own, since
    // holding a tile for a second store costs 2 us of 170 (4096 x 32001 x 2048)
    kHeadGradCeRows = 5,
    kHeadGradKdRows = 6
};

// A 16-bit matrix as it is stored: `outer` rows of `inner` elements, `ld`
// apart.  kmajor: the rows run along K (else K runs down the rows).
struct HeadOperand {
    const void* base;
    int64_t inner, outer, ld;
    int kmajor;
};

struct HeadGemm {
    HeadMode mode;
    int bf16;
    HeadOperand p, q;        // M x K and N x K
    int64_t m, n, k;
    int count_is;            // 0: sizes as given; 1: m = *rows.count; 2: k = *rows.count
    int splits;              // slices of K (products only): slice s goes to rows s * split_rows of the output
    int chunk;               // stages summed in tensor memory before they are added in registers
    // output (gradient and products)
    void* out;
    int ct;                  // 0 FP32, 1 FP16, 2 BF16
    int64_t out_inner, out_outer, ldo, split_rows;
    int add;                 // add to the output (FP32, tensor stores only)
    const int32_t* out_perm; // products: row r goes to row out_perm[r], or NULL
    const float* factor;     // products: multiply by *factor, or NULL
    const float* row_factor; // products: multiply row r by row_factor[r], or NULL
    // Where *spread is not 0 (NULL: never), the logits' gradient goes to
    // by_row as it is and to out times ratio[r] in row r; a product takes P
    // from by_row, which is laid out as p.
    const int32_t* spread;
    void* by_row;
    const float* ratio;
    // the loss
    HeadRows rows;
    int64_t w0;              // first word
    float scale2;            // logit_scale log2 e (/ temperature)
    float label_smoothing;
    float2* stats;
    float* zsum;
    int64_t ld_stats;
    float* z_at;
    const float *lse2, *gain, *boost;
    // Self-test of the kernel's own bounded waits; 0 and 0 for ordinary calls.
    uint64_t wait_limit_ns;  // 0: two seconds
    int stall_cluster;       // cluster whose copying threads stop
    int stall_fill;          // 1 + number of stages they fill before; 0: they do not stop
};

// True if the output can leave through tensor stores: base and row stride on
// 16-byte boundaries and rows that end on one (a store is clipped there).
bool head_gemm_tensor_store(const void* out, int ct, int64_t inner, int64_t ld);

// Clusters that a launch has, of `clusters` that fit at once.
int64_t head_gemm_clusters(const HeadGemm& g, const HeadGemm* and_then, int clusters);

// Launches one product, or two that do not depend on each other (products
// only; the one with the longer K first) as one kernel.
cudaError_t head_gemm_launch(const HeadGemm& g, const HeadGemm* and_then, int clusters, EncodeTiledFn encode,
                             cudaStream_t stream);

// Device address of this kernel's error word (same bits as tc_error_word's).
cudaError_t head_error_word(uint32_t** ptr);

}  // namespace gb300
