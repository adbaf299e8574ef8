// head.cu -- kernels of the output layer's losses (cross entropy and
// distillation over a large vocabulary without the tokens x vocab logits).
//
// The mathematics, for z = scale * hidden weight^T of one token:
//   lse = log sum_v e^{z_v}, computed tile by tile of 128 words as a largest
//   value m and a sum s of 2^{z log2 e - m}; two tiles join as
//   M = max(m1, m2), S = s1 2^{m1 - M} + s2 2^{m2 - M}.
//   d loss / d z_v = p_v - y_v with p = e^{z - lse} and y the target
//   distribution (one word, a smoothed word, or the teacher's list).
// Tokens without a target are moved behind the others first and cost no
// product.  All statistics are FP32; the one rounding to 16 bits is that of
// the logits' gradient, which the tensor cores then take as an operand.
// The products and what is computed on their tiles are in head_gemm.cu.

#include <algorithm>
#include <cmath>

#include "cstore.cuh"
#include "head.h"
#include "ptx.cuh"
#include "row_blocks.h"

namespace gb300 {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ bool has_target(const HeadRows& r, int i) {
    if (r.distill) return r.active[i] != 0;
    return head_target(r.target, r.target_stride, r.ignore_index, r.vocab, i) != kNoWord;
}

// The first `valid` of the eight 16-bit elements that start `shift` bytes into
// two 16-byte blocks, zeros after them.
__device__ __forceinline__ uint4 cut8(const uint4& x, const uint4& y, uint32_t shift, int64_t valid) {
    uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
    const bool by2 = shift & 8, by1 = shift & 4;
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = by2 ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = by1 ? w[i + 1] : w[i];
    const uint32_t bits = (shift & 2) * 8;
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        o[i] = __funnelshift_r(w[i], w[i + 1], bits);
        if (2 * i + 1 >= valid) o[i] = 2 * i >= valid ? 0u : (o[i] & 0xFFFFu);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// Eight 16-bit elements p[0..7], of which the first `valid` exist; lo and hi
// bound the matrix they are in.  Off a 16-byte boundary they are cut out of
// the two aligned 16-byte blocks they lie in (a row of odd length starts
// anywhere); elements are read one by one only where such a block is partly
// outside the matrix.
__device__ __forceinline__ uint4 load8(const uint16_t* p, int64_t valid, uintptr_t lo, uintptr_t hi) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(p);
    const uint32_t shift = static_cast<uint32_t>(at & 15);
    const uintptr_t block = at - shift;
    if (valid >= 8 && shift == 0) return __ldg(reinterpret_cast<const uint4*>(p));
    if (pair_inside(at, lo, hi))
        return cut8(__ldg(reinterpret_cast<const uint4*>(block)), __ldg(reinterpret_cast<const uint4*>(block + 16)),
                    shift, valid);
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t low = 2 * i < valid ? __ldg(p + 2 * i) : 0u;
        const uint32_t high = 2 * i + 1 < valid ? __ldg(p + 2 * i + 1) : 0u;
        o[i] = low | (high << 16);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// d loss / d z = p (1 + t) - y with t = 2 z_loss lse: p and y are in [0, 1], so
// it is at most 1 + |t| in size.
__device__ __forceinline__ float z_term(const GatherArgs& a, int i) {
    return a.z_loss > 0.0f ? 2.0f * a.z_loss * a.lse[i] : 0.0f;
}

// ---- the compact order --------------------------------------------------------
//
// Every block counts all targets (they sit in L2 after the first block's
// read), so one launch finds each token's place, without a scan across
// blocks, and copies the rows.  Blocks own consecutive tokens.

constexpr int kGatherThreads = 256;

// BY_ROW: with the smallest size and the rows' own scales (a.by_row); a form of
// its own, since it costs 2 us of 15 (4096 tokens, 2048 channels).
template <bool BY_ROW>
__global__ void __launch_bounds__(kGatherThreads) gather_kernel(const GatherArgs a, int rows_per_block) {
    grid_dep_launch_dependents();
    grid_dep_wait();
    __shared__ int s_before[8], s_total[8], s_warp[8];
    __shared__ float s_top[8], s_low[8];
    __shared__ int s_rank[kGatherThreads];
    const HeadRows& r = a.rows;
    const int n = static_cast<int>(r.tokens);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int first = min(n, static_cast<int>(blockIdx.x) * rows_per_block);
    const int last = min(n, first + rows_per_block);

    int before = 0, total = 0;
    float top = 0.0f, low = INFINITY;   // of the sizes that are finite and not 0
    for (int i = tid; i < n; i += kGatherThreads) {
        if (!has_target(r, i)) continue;
        ++total;
        before += i < first;
        if (a.lse) {
            const float size =
                fabsf(a.grad_loss[static_cast<int64_t>(i) * a.grad_stride]) * (1.0f + fabsf(z_term(a, i)));
            if (isfinite(size)) top = fmaxf(top, size);
            if (BY_ROW && size > 0.0f) low = fminf(low, size);
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        before += __shfl_xor_sync(~0u, before, o);
        total += __shfl_xor_sync(~0u, total, o);
        top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
        if (BY_ROW) low = fminf(low, __shfl_xor_sync(~0u, low, o));
    }
    if (lane == 0) {
        if (BY_ROW) s_low[warp] = low;
        s_before[warp] = before;
        s_total[warp] = total;
        s_top[warp] = top;
    }
    __syncthreads();
    before = total = 0;
    top = 0.0f;
    low = INFINITY;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
        if (BY_ROW) low = fminf(low, s_low[w]);
        before += s_before[w];
        total += s_total[w];
        top = fmaxf(top, s_top[w]);
    }
    const bool spread = BY_ROW && low < top / kHeadSpread;
    const float factor = top > 0.0f ? top * a.undo : a.undo;
    if (blockIdx.x == 0 && tid == 0) {
        *r.count = total;
        if (a.lse) {
            *a.factor = factor;
            if (BY_ROW) *a.spread = spread;
        }
    }
    const int zero_end = (total + a.pad_rows - 1) / a.pad_rows * a.pad_rows;
    const uintptr_t lo = reinterpret_cast<uintptr_t>(a.hidden);
    const uintptr_t hi = lo + 2 * static_cast<uintptr_t>((r.tokens - 1) * a.ldh + r.dim);
    const bool zero_vec = (reinterpret_cast<uintptr_t>(a.zero_rows) & 15) == 0 && (a.ld_zero & 3) == 0;
    const int chunks = static_cast<int>(a.ldc >> 3);

    for (int c0 = first; c0 < last; c0 += kGatherThreads) {
        const int i = c0 + tid;
        const bool in = i < last;
        const bool act = in && has_target(r, i);
        const unsigned bal = __ballot_sync(~0u, act);
        if (lane == 0) s_warp[warp] = __popc(bal);
        __syncthreads();
        int ahead = __popc(bal & ((1u << lane) - 1u));
        int whole = 0;
#pragma unroll
        for (int w = 0; w < 8; ++w) {
            if (w < warp) ahead += s_warp[w];
            whole += s_warp[w];
        }
        const int act_before = before + ahead;
        const int place = act ? act_before : total + (i - act_before);
        s_rank[tid] = place;
        if (in) {
            r.rank[i] = place;
            r.perm[place] = i;
            if (act && !r.distill)
                r.target_c[place] = static_cast<int32_t>(r.target[static_cast<int64_t>(i) * r.target_stride]);
            if (act && a.lse) {
                a.lse2[place] = a.lse[i] * kLog2e;
                // divided first: the largest may be close to the smallest
                // numbers there are; infinities and NaN stay, and so do
                // zeros where there is no largest
                const float own = a.grad_loss[static_cast<int64_t>(i) * a.grad_stride];
                const float term = z_term(a, i), most = 1.0f + fabsf(term);
                if (spread) {
                    a.gain[place] = a.unit / most;
                    a.undo_row[place] = own * most * a.undo;
                    a.ratio[place] = own * most / top;
                } else {
                    a.gain[place] = top > 0.0f ? own / top * a.unit : own;
                    if (BY_ROW) a.undo_row[place] = factor;
                }
                a.boost[place] = 1.0f + term;
            }
        }
        __syncthreads();
        // 32 threads to a row, more where the block has fewer than 8 rows
        const int here = min(kGatherThreads, last - c0);
        const int per = here >= 8 ? 32 : here > 3 ? 64 : here > 1 ? 128 : 256;
        for (int j = tid / per; j < here; j += kGatherThreads / per) {
            const int to = s_rank[j];
            if (to >= total && a.zero_rows) {
                for (int ch = tid % per; ch < chunks; ch += per) {
                    const int64_t o = static_cast<int64_t>(c0 + j) * a.ld_zero + ch * 8;
                    if (zero_vec && ch * 8 + 8 <= r.dim) {
                        c_store4(a.zero_rows, o, 0.0f, 0.0f, 0.0f, 0.0f, a.zero_ct);
                        c_store4(a.zero_rows, o + 4, 0.0f, 0.0f, 0.0f, 0.0f, a.zero_ct);
                    } else {
                        for (int k = 0; k < 8 && ch * 8 + k < r.dim; ++k)
                            c_store(a.zero_rows, o + k, 0.0f, a.zero_ct);
                    }
                }
            }
            if (to >= zero_end) continue;
            const uint16_t* from = a.hidden + static_cast<int64_t>(c0 + j) * a.ldh;
            uint4* row = reinterpret_cast<uint4*>(a.out + static_cast<int64_t>(to) * a.ldc);
            for (int ch0 = tid % per; ch0 < chunks; ch0 += 4 * per) {
                uint4 v[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int ch = ch0 + k * per;
                    v[k] = make_uint4(0, 0, 0, 0);
                    if (to < total && ch * 8 < r.dim) v[k] = load8(from + ch * 8, r.dim - ch * 8, lo, hi);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (ch0 + k * per < chunks) row[ch0 + k * per] = v[k];
            }
        }
        before += whole;
        __syncthreads();
    }
}

// One warp to a row at a time.
__global__ void __launch_bounds__(256) pack_rows_kernel(const uint16_t* in, int64_t ld, int64_t rows,
                                                        int64_t cols, uint16_t* out, int64_t ldc) {
    grid_dep_launch_dependents();
    grid_dep_wait();
    const uintptr_t lo = reinterpret_cast<uintptr_t>(in);
    const uintptr_t hi = lo + 2 * static_cast<uintptr_t>((rows - 1) * ld + cols);
    const int lane = threadIdx.x & 31;
    for (int64_t i = blockIdx.x * 8ll + (threadIdx.x >> 5); i < rows; i += gridDim.x * 8ll) {
        const uint16_t* from = in + i * ld;
        uint16_t* to = out + i * ldc;
        if (!row_inside(reinterpret_cast<uintptr_t>(from), cols, lo, hi)) {   // near the matrix's ends
            for (int64_t c = lane * 8; c < ldc; c += 256)
                *reinterpret_cast<uint4*>(to + c) =
                    c < cols ? load8(from + c, cols - c, lo, hi) : make_uint4(0, 0, 0, 0);
            continue;
        }
        // chunks are 16 bytes apart, so one shift serves the row; four reads under way
        const uint32_t shift = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(from) & 15);
        const char* blocks = reinterpret_cast<const char*>(from) - shift;
        for (int64_t c0 = lane * 8; c0 < ldc; c0 += 1024) {
            uint4 x[4], y[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int64_t c = c0 + 256 * k;
                x[k] = y[k] = make_uint4(0, 0, 0, 0);
                if (c < cols) {
                    x[k] = __ldg(reinterpret_cast<const uint4*>(blocks + 2 * c));
                    y[k] = __ldg(reinterpret_cast<const uint4*>(blocks + 2 * c + 16));
                }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int64_t c = c0 + 256 * k;
                if (c < ldc) *reinterpret_cast<uint4*>(to + c) = cut8(x[k], y[k], shift, cols - c);
            }
        }
    }
}

// ---- the teacher's list ---------------------------------------------------------
//
// One warp to a token: softmax over the entries that are there (divided by the
// temperature once the largest has been taken off: a finite logit may pass
// FP32's range when it is divided first, and entries masked by their type's
// lowest number are finite), then the entries in the order of their words
// (bitonic sort in shared memory), so that a tile of the vocabulary finds its
// own entries as one run.

constexpr int kTeacherWarps = 8;
constexpr int kTeacherMost = 256;

__device__ __forceinline__ float teacher_logit(const TeacherArgs& a, int64_t i) {
    if (a.dtype == 0) return static_cast<const float*>(a.logits)[i];
    return c_widen(static_cast<const uint16_t*>(a.logits)[i], a.dtype);
}

__global__ void __launch_bounds__(kTeacherWarps * 32) teacher_kernel(const TeacherArgs a, int size) {
    grid_dep_launch_dependents();
    grid_dep_wait();
    __shared__ uint64_t s_key[kTeacherWarps][kTeacherMost];
    __shared__ float s_val[kTeacherWarps][kTeacherMost];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t n = static_cast<int64_t>(blockIdx.x) * kTeacherWarps + warp;
    if (n >= a.tokens) return;
    uint64_t* key = s_key[warp];
    float* val = s_val[warp];
    float top = -INFINITY;
    for (int j = lane; j < size; j += 32) {
        int32_t word = kNoWord;
        float t = -INFINITY;
        if (j < a.top_k) {
            const int64_t w = a.index[n * a.ld_index + j];
            const float x = teacher_logit(a, n * a.ld_logits + j);
            if (w >= 0 && w < a.vocab && x != -INFINITY) {
                word = static_cast<int32_t>(w);
                t = x;
            }
        }
        key[j] = (static_cast<uint64_t>(static_cast<uint32_t>(word)) << 32) | static_cast<uint32_t>(j);
        val[j] = t;
        top = fmaxf(top, t);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
    float sum = 0.0f;
    int some = 0;
    __syncwarp();
    for (int j = lane; j < size; j += 32) {
        if (static_cast<int32_t>(key[j] >> 32) == kNoWord) continue;
        some = 1;
        sum += expf((val[j] - top) / a.temperature);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
    some = __any_sync(~0u, some);
    const float log_sum = logf(sum);
    for (int k = 2; k <= size; k <<= 1) {
        for (int j = k >> 1; j; j >>= 1) {
            __syncwarp();
            for (int i = lane; i < size; i += 32) {
                const int o = i ^ j;
                if (o > i) {
                    const uint64_t x = key[i], y = key[o];
                    if ((x > y) == ((i & k) == 0)) {
                        key[i] = y;
                        key[o] = x;
                    }
                }
            }
        }
    }
    __syncwarp();
    for (int j = lane; j < a.top_k; j += 32) {
        const uint64_t x = key[j];
        const int32_t word = static_cast<int32_t>(x >> 32);
        a.words[n * a.top_k + j] = word;
        a.logq[n * a.top_k + j] =
            word == kNoWord ? -INFINITY : (val[static_cast<uint32_t>(x)] - top) / a.temperature - log_sum;
    }
    if (lane == 0) a.active[n] = some ? 1 : 0;
}

// ---- joining the tiles ------------------------------------------------------------
//
// A block of 1024 threads takes WIDTH tokens, 1024 / WIDTH threads each: 4,
// so that a single token's tiles (1024 for 131072 words) are four loads deep;
// 8 up to 4096 tokens; 16 above, where whole 128-byte lines of statistics
// count (8192 tokens: 19 us against 24 with 8; 2048 tokens: 12 against 10).
// The sums are taken in a fixed tree.

constexpr int kJoinThreads = 1024;

template <int WIDTH>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const JoinArgs a) {
    constexpr int width = WIDTH, groups = kJoinThreads / WIDTH;
    grid_dep_launch_dependents();
    grid_dep_wait();
    __shared__ float s_m[kJoinThreads], s_s[kJoinThreads], s_z[kJoinThreads];
    const HeadRows& r = a.rows;
    const int me = static_cast<int>(threadIdx.x), row = me & (width - 1), grp = me / width;
    const int place = static_cast<int>(blockIdx.x) * width + row;
    const bool live = r.perm ? place < *r.count : place < r.tokens && has_target(r, place);
    const int token = place >= r.tokens ? 0 : r.perm ? r.perm[place] : place;
    float m = -INFINITY, s = 0.0f, x = 0.0f;
    if (live) {
        for (int t = grp; t < a.tiles; t += groups) {
            const float2 v = a.stats[static_cast<int64_t>(t) * a.ld_stats + place];
            const float top = fmaxf(m, v.x);
            const float base = top == -INFINITY ? 0.0f : top;
            s = s * exp2f(m - base) + v.y * exp2f(v.x - base);
            m = top;
            if (a.zsum) x += a.zsum[static_cast<int64_t>(t) * a.ld_stats + place];
        }
    }
    s_m[me] = m;
    s_s[me] = s;
    s_z[me] = x;
    __syncthreads();
    for (int o = groups / 2; o; o >>= 1) {
        if (grp < o) {
            const float m2 = s_m[me + o * width], top = fmaxf(m, m2);
            const float base = top == -INFINITY ? 0.0f : top;
            s = s * exp2f(m - base) + s_s[me + o * width] * exp2f(m2 - base);
            m = top;
            x += s_z[me + o * width];
            s_m[me] = m;
            s_s[me] = s;
            s_z[me] = x;
        }
        __syncthreads();
    }
    // lse - z is taken as log2 of the sum plus (largest - z log2 e), the
    // difference formed before it is rounded: a likely word's loss is much
    // smaller than either term
    const float top = s_m[row], log_sum = log2f(s_s[row]);
    const float lse = (top + log_sum) * kLn2;
    auto below_lse = [&](float logit) { return (log_sum + fmaf(-logit, a.scale2, top)) * kLn2; };
    float loss = 0.0f;
    if (r.distill) {
        // the divergence's terms, split over the token's threads
        if (live)
            for (int j = grp; j < r.top_k; j += groups) {
                const int64_t at = static_cast<int64_t>(token) * r.top_k + j;
                if (r.words[at] == kNoWord) continue;
                const float lq = r.logq[at];
                const float q = expf(lq);
                if (q != 0.0f) loss += q * (lq + below_lse(a.z_at[at]));
            }
        __syncthreads();
        s_z[me] = loss;
        __syncthreads();
        for (int o = groups / 2; o; o >>= 1) {
            if (grp < o) s_z[me] += s_z[me + o * width];
            __syncthreads();
        }
        loss = s_z[row] * a.temperature * a.temperature;
    } else if (live) {
        const float logit = a.z_at[place];
        loss = below_lse(logit) + a.z_loss * lse * lse;
        if (a.zsum) loss += a.label_smoothing * (a.scale * (logit - s_z[row] / static_cast<float>(r.vocab)));
    }
    if (grp == 0 && place < r.tokens) {
        if (!live) {
            loss = 0.0f;
            if (!r.distill && r.target[static_cast<int64_t>(token) * r.target_stride] != r.ignore_index)
                loss = __int_as_float(0x7FC00000);   // a target outside the vocabulary
        }
        a.loss[token] = loss;
        a.lse[token] = live ? lse : 0.0f;
    }
}

// ---- sums of partial rows -----------------------------------------------------------

__global__ void __launch_bounds__(256) sum_rows_kernel(const SumRowsArgs a, bool vec) {
    grid_dep_launch_dependents();
    grid_dep_wait();
    const int64_t quads = (a.cols + 3) >> 2;
    const int64_t all = a.rows * quads;
    const float all_rows = a.row_factor ? 0.0f : *a.factor;
    const int count = a.rank ? *a.count : 0;
    for (int64_t x = blockIdx.x * 256ll + threadIdx.x; x < all; x += gridDim.x * 256ll) {
        const int64_t i = x / quads, c = (x - i * quads) * 4;
        int64_t from = i;
        bool live = true;
        if (a.rank) {
            from = a.rank[i];
            live = from < count;
        }
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (live) {
            const float factor = a.row_factor ? a.row_factor[from] : all_rows;
            const float* p = a.parts + from * a.ld + c;
            for (int s = 0; s < a.nparts; ++s) {
                const float4 t = *reinterpret_cast<const float4*>(p + s * a.part_stride);
                v.x += t.x;
                v.y += t.y;
                v.z += t.z;
                v.w += t.w;
            }
            v.x *= factor;
            v.y *= factor;
            v.z *= factor;
            v.w *= factor;
        }
        const int64_t o = i * a.ldo + c;
        if (vec && c + 4 <= a.cols) {
            c_store4(a.out, o, v.x, v.y, v.z, v.w, a.ct);
        } else {
            const float e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (c + k < a.cols) c_store(a.out, o + k, e[k], a.ct);
        }
    }
}

// Every kernel of a call is launched with programmatic stream serialization:
// it may be set up while the kernel before it still runs, and waits for that
// one to complete before it touches memory (grid_dep_wait).
template <class... P, class... A>
cudaError_t chain(void (*kernel)(P...), unsigned grid, unsigned block, cudaStream_t stream, A... args) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

unsigned blocks_for(int64_t threads, int sms) {
    return static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>((threads + 255) / 256, 8ll * sms)));
}

}  // namespace

cudaError_t gather_launch(const GatherArgs& a, int sms, cudaStream_t stream) {
    const int64_t n = a.rows.tokens;
    const int64_t rows = std::max<int64_t>(1, (n + 2 * sms - 1) / (2 * sms));
    const unsigned grid = static_cast<unsigned>(std::max<int64_t>(1, (n + rows - 1) / rows));
    return chain(a.by_row ? gather_kernel<true> : gather_kernel<false>, grid, kGatherThreads, stream, a, static_cast<int>(rows));
}

cudaError_t teacher_launch(const TeacherArgs& a, cudaStream_t stream) {
    int size = 32;
    while (size < a.top_k) size <<= 1;
    const unsigned grid = static_cast<unsigned>((a.tokens + kTeacherWarps - 1) / kTeacherWarps);
    return chain(teacher_kernel, grid, kTeacherWarps * 32, stream, a, size);
}

cudaError_t pack_rows_launch(const uint16_t* in, int64_t ld, int64_t rows, int64_t cols,
                             uint16_t* out, int64_t ldc, int sms, cudaStream_t stream) {
    return chain(pack_rows_kernel, blocks_for(rows * 32, sms), 256, stream, in, ld, rows, cols, out, ldc);
}

cudaError_t join_launch(const JoinArgs& a, cudaStream_t stream) {
    const int width = a.rows.tokens <= 4 ? 4 : a.rows.tokens <= 4096 ? 8 : 16;
    const unsigned grid = static_cast<unsigned>((a.rows.tokens + width - 1) / width);
    auto kernel = width == 4 ? join_kernel<4> : width == 8 ? join_kernel<8> : join_kernel<16>;
    return chain(kernel, grid, kJoinThreads, stream, a);
}

cudaError_t sum_rows_launch(const SumRowsArgs& a, int sms, cudaStream_t stream) {
    const uintptr_t align = a.ct == kCF32 ? 15 : 7;
    const bool vec = (reinterpret_cast<uintptr_t>(a.out) & align) == 0 && (a.ldo & 3) == 0;
    return chain(sum_rows_kernel, blocks_for(a.rows * ((a.cols + 3) >> 2), sms), 256, stream, a, vec);
}

}  // namespace gb300
