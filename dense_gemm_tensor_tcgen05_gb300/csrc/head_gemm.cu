// head_gemm.cu -- the tensor-core kernel behind the output layer's losses.
//
// One kernel form computes every product of the losses, P (M x K) times
// Q^T (N x K), in 256 x 256 tiles of a CTA pair:
//
//   logits    P = hidden (tokens x dim), Q = weight (words x dim).  A tile of
//             logits never leaves the SM: its rows' softmax statistics do
//             (largest value and sum of 128 words), or the logits' gradient,
//             rounded to 16 bits.
//   dhidden   P = logits' gradient (tokens x words), Q = weight^T
//   dweight   P = logits' gradient^T (words x tokens), Q = hidden^T
//
// Roles, per CTA of the pair: warps 0 and 2 copy P and Q (TMA, 128-byte
// swizzle, a ring of stages of 128 K); warp 1 of the even CTA issues
// tcgen05.mma for both; warps 4..11 own 32 rows x 128 columns of the CTA's
// 128 x 256 results each (warp 3 only completes the first warpgroup, which
// hands registers to the other two: 56 a thread against 224).
//
// Sums.  The tensor core's FP32 accumulator truncates toward zero as it adds
// (a product of 4096 channels came out 2e-5 too small in its largest logits),
// so K is cut into chunks of `chunk` stages: each chunk is summed in tensor
// memory (two buffers of 256 columns, so the next chunk's products run
// meanwhile) and added, rounded to nearest, to 128 sums a thread holds in
// registers.  The error falls with the chunk's share of K.  The sums are
// handed back by relaxed arrivals: a release at cluster scope waited for the
// warps' stores to global memory and cost a quarter of the time.
//
// What bounds it.  Long products run at the tensor cores' power-limited rate:
// 8192 x 131072 x 4096 takes 4.7 to 5.0 ms with the statistics, by the card
// (1750 to 1870 TFLOP/s; the same product alone, with a 16-bit result written,
// 1700 to 1780 by this library's GEMM where the statistics ran at 1744).  With
// few tokens the weight's read is the bound: 16 x 65536 x 4096 takes 94 us,
// 5.7 TB/s.  Below a thousand channels the forming
// of a tile's results (128 exponentials a thread) takes as long as its
// products.
//
// Why 256 x 256 tiles of a pair for every size: with 256 rows of tokens or
// fewer, rows that are not there cost no traffic, and a tile's 256 words are
// read once either way.
//
// The row of a logits tile is one thread's (128 words of it), so a softmax
// statistic needs no exchange between threads.  Exponentials are ex2.approx
// (relative error 2^-22) of logits scaled by log2 e in the same multiply-add
// that takes off the largest.
//
// The number of tokens that have a target is read on the device: it bounds
// the rows of the logits and of dhidden, and K of dweight.
//
// Every wait gives up after two seconds, sets the device error word and
// makes the pair leave; copies and products in flight are waited for
// (bounded) and tensor memory is freed on every path.  A self-test shortens
// the limit and has one cluster's copies stop.

#include <algorithm>
#include <cmath>
#include <cstring>

#include "cstore.cuh"
#include "head_gemm.h"
#include "ptx.cuh"

namespace gb300 {

namespace {

__device__ uint32_t g_head_error;   // bits as in the GEMM kernels' error word

constexpr uint32_t kErrProducer = 1u, kErrMma = 2u, kErrEpilogue = 4u, kErrDrain = 8u;
constexpr uint64_t kWaitNs = 2000000000ull, kDrainNs = 200000000ull, kPairDrainNs = 3 * kWaitNs;   // kWaitNs: default

constexpr int kThreads = 384;
constexpr int kFirstSumWarp = 4;
// 128 x 56 + 256 x 224 = 384 x 168, the registers the block is launched with.  At
// 8192 x 131072 x 4096 the statistics took 5023 us with 56 and 224, 5072 with 72
// and 216, and 7385 with 88 and 208, where the sums no longer fit.
constexpr int kRegsCopy = 56, kRegsSum = 224;
constexpr int kMaxStages = 5;
constexpr int kRowBytes = 128;                    // 64 16-bit elements of K, one row of an atom
constexpr int kQBytes = 2 * 128 * kRowBytes;      // a stage's 128 rows x 128 K of Q
constexpr int kFullStages = 3;
constexpr int kRingBytes = kFullStages * 2 * kQBytes;   // stages of 128 rows of P and Q each
constexpr int kStoreBytes = 8 * 4096;             // one 4 KiB box for each epilogue warp
constexpr int kBars = 2 * kMaxStages + 5;
constexpr int kSmemBytes = 1024 + kRingBytes + kStoreBytes + kBars * 8 + 16;
constexpr int kCols = 128;                        // columns of a thread
constexpr int kLines = 8;                         // rows that store_lines has under way
static_assert(kSmemBytes <= 227 * 1024 && kSmemBytes > 114 * 1024, "one CTA per SM");
static_assert(kHeadTile == kCols, "a softmax statistic is one thread's columns");

struct Args {
    int32_t m, n, k, count_is, splits, chunk, group;
    int32_t p_kmajor, q_kmajor;
    // FEW: rows of P that the even CTA copies (the odd one none), and stages
    int32_t p_rows, stages;
    uint32_t idesc;
    // how long a wait may take; the stage from which on the copying threads
    // of one cluster withhold their copies (self-test; cluster -1: none)
    uint64_t wait_limit_ns;
    int32_t stall_cluster, stall_fill;
    const int32_t* count;
    // output
    void* out;
    int64_t ldo;
    int32_t ct, tensor_store, add, out_rows, out_cols, split_rows;
    const int32_t* out_perm;   // row r goes to out_perm[r], or NULL
    const float *factor, *row_factor;
    const int32_t* spread;
    const float* ratio;
    // loss
    const int32_t* target_c;
    const int64_t* target;   // read where there is no order (perm NULL)
    int64_t target_stride, ignore_index, vocab;
    const int32_t* perm;
    const int32_t* words;
    const float* logq;
    int32_t top_k, w0;
    float scale2, flat, hit;
    float2* stats;
    float* zsum;
    int64_t ld_stats;
    float* z_at;
    const float *lse2, *gain, *boost;
};

// One product: its operands' and output's tensor maps (by_row: of the copy of
// the logits' gradient that has a scale for each row) and its arguments.
struct Params {
    CUtensorMap p, q, o, by_row;
    Args a;
};

struct Wait {
    volatile uint32_t* abort_flag;   // this CTA's (the peer may raise it)
    uint32_t peer_abort;             // shared::cluster address of the peer's
    volatile uint64_t* limit_ns;     // this CTA's copy of the launch's limit
};

__device__ __forceinline__ void raise_abort(const Wait& w) {
    *w.abort_flag = 1;
    st_shared_cluster_u32(w.peer_abort, 1);
}

template <bool CLUSTER>
__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity, const Wait& w, uint32_t err) {
    auto done = [&]() { return CLUSTER ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity); };
    if (done()) return true;
    const uint64_t last = globaltimer_ns() + *w.limit_ns;
    while (true) {
        if (done()) return true;
        if (*w.abort_flag) return false;
        if (globaltimer_ns() > last) {
            atomicOr(&g_head_error, err);
            raise_abort(w);
            return false;
        }
    }
}

__device__ __forceinline__ void drain(uint32_t bar, uint32_t parity, uint64_t limit) {
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(bar, parity)) {
        if (globaltimer_ns() - t0 > limit) {
            atomicOr(&g_head_error, kErrDrain);
            return;
        }
    }
}

// Adds one box from shared memory to global memory, element by element.
__device__ __forceinline__ void tma_add_2d(const CUtensorMap* map, uint32_t src, int32_t c0, int32_t c1) {
    asm volatile(
        "cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3}], [%1];"
        ::"l"(reinterpret_cast<uint64_t>(map)), "r"(src), "r"(c0), "r"(c1)
        : "memory");
}

// Tells the even CTA's product thread that this warp has read its part of a
// buffer of sums.  Relaxed: the reads have completed (tcgen05.wait::ld) and
// nothing else is handed over; a release at cluster scope would wait for the
// warp's stores to global memory too.
__device__ __forceinline__ void mbar_arrive_relaxed_cluster(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

template <int N>
__device__ __forceinline__ void regs_give() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

template <int N>
__device__ __forceinline__ void regs_take() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A stage of an operand, 128 K of this CTA's rows, in two copies: the issuing
// thread has about 1000 cycles for a stage, and with four copies for an operand
// whose rows run across K the tensor pipe of dweight (two of them) was 80 %
// busy, of the logits (none) 92 %.  Along K: 64 K of all rows each, 128-byte
// rows, atom_bytes apart.  Across K: 64 rows each, 128 lines of K, 16 KiB apart.
__device__ __forceinline__ void load_stage(uint32_t dst, const CUtensorMap* map, uint32_t bar, bool kmajor,
                                           int atom_bytes, int r0, int k0) {
    if (kmajor) {
        tma_load_2d_pair(dst, map, bar, k0, r0);
        tma_load_2d_pair(dst + atom_bytes, map, bar, k0 + 64, r0);
    } else {
        tma_load_2d_pair(dst, map, bar, r0, k0);
        tma_load_2d_pair(dst + kQBytes / 2, map, bar, r0 + 64, k0);
    }
}

// What there is to do, from the number of tokens with a target.
struct Work {
    int tiles_p = 0, tiles_q = 0, units = 0, steps = 0, m = 0;

    __device__ __forceinline__ Work() {}
    __device__ __forceinline__ explicit Work(const Args& a) {
        const int count = a.count_is ? *a.count : 0;
        m = a.count_is == 1 ? count : a.m;
        const int k = a.count_is == 2 ? count : a.k;
        tiles_p = (m + kHeadTileM - 1) / kHeadTileM;
        tiles_q = (a.n + kHeadTileN - 1) / kHeadTileN;
        steps = (k + kHeadStepK - 1) / kHeadStepK;
        units = tiles_p * tiles_q * a.splits;
    }
};

// The units of one cluster, in turn; every role walks the same ones.  Units of
// the first product go round the clusters, then those of the second.  When the
// first's last round is not full, the clusters it leaves out start on the
// second with as many units as take them as long (kTurnSteps: what a unit
// costs beside its K steps, in steps).
constexpr int kTurnSteps = 4;

struct Turns {
    int cid, ncl, n1, n2, left, extra, next1, j;

    __device__ __forceinline__ Turns(const Work& w1, int len1, const Work& w2, int len2)
        : cid(static_cast<int>(cluster_id_x())), ncl(static_cast<int>(cluster_count_x())), n1(w1.units),
          n2(w2.units), next1(cid), j(0) {
        left = n1 % ncl;
        extra = 0;
        if (n2 > 0 && left > 0)
            extra = min((len1 + kTurnSteps) / (len2 + kTurnSteps), n2 / (ncl - left));
    }

    // false: no more
    __device__ __forceinline__ bool next(bool& two, int& u) {
        if (next1 < n1) {
            two = false;
            u = next1;
            next1 += ncl;
            return true;
        }
        if (n2 == 0) return false;
        const bool early = left > 0 && cid >= left;
        two = true;
        if (early && j < extra) u = j * (ncl - left) + cid - left;
        else u = extra * (ncl - left) + (j - (early ? extra : 0)) * ncl + cid;
        ++j;
        return u < n2;
    }
};

struct Unit {
    int pb, qb, seg, k0, k1;
};

// Tiles go in groups of `group` along M, column by column, odd groups
// backwards, so the pairs at work share operand rows in L2.
__device__ __forceinline__ Unit unit_of(const Args& a, const Work& w, int u) {
    Unit r;
    int tile = u;
    r.seg = 0;
    r.k0 = 0;
    r.k1 = w.steps;
    if (a.splits > 1) {
        tile = u / a.splits;
        r.seg = u - tile * a.splits;
        r.k0 = static_cast<int>(static_cast<int64_t>(w.steps) * r.seg / a.splits);
        r.k1 = static_cast<int>(static_cast<int64_t>(w.steps) * (r.seg + 1) / a.splits);
    }
    const int per_group = a.group * w.tiles_q;
    const int g = tile / per_group;
    const int first = g * a.group;
    const int high = min(w.tiles_p - first, a.group);
    const int x = tile - g * per_group;
    r.pb = first + x % high;
    r.qb = x / high;
    if (g & 1) r.qb = w.tiles_q - 1 - r.qb;
    return r;
}

// v[i0 .. i0 + 31] += r, two sums to an instruction.
__device__ __forceinline__ void add32(float (&v)[kCols], int i0, const uint32_t (&r)[32]) {
#pragma unroll
    for (int i = 0; i < 32; i += 2)
        asm volatile(
            "{\n\t.reg .b64 a, b;\n\t"
            "mov.b64 a, {%0, %1};\n\t"
            "mov.b64 b, {%2, %3};\n\t"
            "add.rn.f32x2 a, a, b;\n\t"
            "mov.b64 {%0, %1}, a;\n\t}"
            : "+f"(v[i0 + i]), "+f"(v[i0 + i + 1])
            : "f"(__uint_as_float(r[i])), "f"(__uint_as_float(r[i + 1])));
}

// v *= factor, two to an instruction.
__device__ __forceinline__ void scale_all(float (&v)[kCols], float factor) {
#pragma unroll
    for (int i = 0; i < kCols; i += 2)
        asm volatile(
            "{\n\t.reg .b64 a, b;\n\t"
            "mov.b64 a, {%0, %1};\n\t"
            "mov.b64 b, {%2, %2};\n\t"
            "mul.rn.f32x2 a, a, b;\n\t"
            "mov.b64 {%0, %1}, a;\n\t}"
            : "+f"(v[i]), "+f"(v[i + 1])
            : "f"(factor));
}

// First entry of a token's sorted list whose word is at least w.
__device__ __forceinline__ int first_entry(const int32_t* words, int k, int32_t w) {
    int lo = 0, hi = k;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (words[mid] < w) lo = mid + 1;
        else hi = mid;
    }
    return lo;
}

// The entries of a row that fall in this thread's columns: cross entropy has
// one, the target; a teacher's list is sorted, so they are one run of it.
struct Hits {
    int32_t next = kNoWord;          // word of the next entry (kNoWord: none)
    int32_t ahead = kNoWord;         // and of the one after it, read ahead
    int at = 0, end = 0;
    const int32_t* words = nullptr;
    int64_t row = 0;                 // index of the list's first entry

    template <bool KD>
    __device__ __forceinline__ void start(const Args& a, int place, int32_t word0) {
        if (!KD) {
            const int32_t t = a.perm ? a.target_c[place]
                                     : head_target(a.target, a.target_stride, a.ignore_index, a.vocab, place);
            if (t >= word0) next = t;
            row = place;
        } else {
            row = static_cast<int64_t>(a.perm ? a.perm[place] : place) * a.top_k;
            words = a.words + row;
            end = a.top_k;
            at = first_entry(words, end, word0);
            if (at < end) next = words[at];
            if (at + 1 < end) ahead = words[at + 1];
        }
    }
    template <bool KD>
    __device__ __forceinline__ void advance() {
        next = ahead;
        ahead = kNoWord;
        if (KD && ++at + 1 < end) ahead = words[at + 1];
    }
};

// A thread's 32 columns in its row of the warp's 4 KiB box, where they can be
// indexed: value i sits at i ^ lane, which keeps the warp's accesses to one
// i apart in the banks.
__device__ __forceinline__ uint32_t scratch_at(uint32_t box, int lane, int i) {
    return box + static_cast<uint32_t>(lane * 128 + ((i ^ lane) & 31) * 4);
}

__device__ __forceinline__ float ld_shared(uint32_t addr) {
    float x;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x) : "r"(addr) : "memory");
    return x;
}

__device__ __forceinline__ uint32_t ld_shared_u32(uint32_t addr) {
    uint32_t x;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(x) : "r"(addr));
    return x;
}

// Word `lane` of row r of a box.
__device__ __forceinline__ uint32_t box_word(uint32_t box, int r, int lane) {
    return ld_shared_u32(box + static_cast<uint32_t>(r) * 128u +
                         (static_cast<uint32_t>((lane >> 2) ^ (r & 7)) << 4) + static_cast<uint32_t>(lane & 3) * 4u);
}

__device__ __forceinline__ void st_shared(uint32_t addr, float x) {
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(x) : "memory");
}

// This lane's row of a box: 64 results from v[i0] on, rounded to 16 bits.
template <int CT>
__device__ __forceinline__ void fill_box16(uint32_t line, int lane, const float (&v)[kCols], int i0) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int i = i0 + j * 8;
        st_shared_v4_u32(line + (static_cast<uint32_t>(j ^ (lane & 7)) << 4), c_pack2(v[i], v[i + 1], CT),
                         c_pack2(v[i + 2], v[i + 3], CT), c_pack2(v[i + 4], v[i + 5], CT),
                         c_pack2(v[i + 6], v[i + 7], CT));
    }
}

// Where a tile goes, in registers: Args may lie behind an address (one of two
// products), and each read of it past a memory clobber would be a load.
struct Out {
    void* out;
    int64_t ldo;
    const int32_t* perm;
    int ct, add, rows, cols;

    __device__ __forceinline__ explicit Out(const Args& a)
        : out(a.out), ldo(a.ldo), perm(a.out_perm), ct(a.ct), add(a.add), rows(a.out_rows), cols(a.out_cols) {}
};

// Stores this warp's 32 rows x 128 columns through its 4 KiB box (or two of
// them in turn), 128 bytes of each row at a time; the tensor unit clips at the output's edges.
__device__ __forceinline__ void store_boxes(const Out& a, const CUtensorMap* map, uint32_t box0, uint32_t box1,
                                            const float (&v)[kCols], int lane, int row0, int out_row0, int col0) {
    const bool rows_in = row0 < a.rows;
    if (a.ct == kCF32) {
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const uint32_t box = b & 1 ? box1 : box0, line = box + static_cast<uint32_t>(lane) * 128u;
            if (lane == 0) {   // the last store from this box has read it
                if (box0 != box1) bulk_wait_group_read<1>();
                else bulk_wait_group_read<0>();
            }
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int i = b * 32 + j * 4;
                st_shared_v4(line + (static_cast<uint32_t>(j ^ (lane & 7)) << 4), v[i], v[i + 1], v[i + 2], v[i + 3]);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                if (rows_in && col0 + b * 32 < a.cols) {
                    if (a.add) tma_add_2d(map, box, col0 + b * 32, out_row0);
                    else tma_store_2d(map, box, col0 + b * 32, out_row0);
                }
                bulk_commit_group();   // an empty group too, so that the boxes' groups alternate
            }
        }
    } else {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const uint32_t box = b & 1 ? box1 : box0, line = box + static_cast<uint32_t>(lane) * 128u;
            if (lane == 0) {   // the last store from this box has read it
                if (box0 != box1) bulk_wait_group_read<1>();
                else bulk_wait_group_read<0>();
            }
            __syncwarp();
            if (a.ct == kCF16) fill_box16<kCF16>(line, lane, v, b * 64);
            else fill_box16<kCBF16>(line, lane, v, b * 64);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                if (rows_in && col0 + b * 64 < a.cols) tma_store_2d(map, box, col0 + b * 64, out_row0);
                bulk_commit_group();
            }
        }
    }
}

// The same results to rows whose place or alignment the tensor unit cannot
// take: rows in another order, or a base, row stride or width off 16 bytes.
// The box turns the tile around, so that a warp writes 128 bytes of one row
// at a time; a row of 16-bit numbers that starts between two words is shifted
// by one number to meet them.
__device__ __forceinline__ void store_lines(const Out& a, uint32_t box, const float (&v)[kCols], int lane, int row0,
                                            int rows, int col0) {
    const int row = row0 + lane;
    const int place = a.perm && row < rows ? a.perm[row] : row;
    const int high = min(32, rows - row0);
    const uint32_t line = box + static_cast<uint32_t>(lane) * 128u;
    if (a.ct == kCF32) {
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            if (col0 + b * 32 >= a.cols) break;
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int i = b * 32 + j * 4;
                st_shared_v4(line + (static_cast<uint32_t>(j ^ (lane & 7)) << 4), v[i], v[i + 1], v[i + 2], v[i + 3]);
            }
            __syncwarp();
            const bool in = col0 + b * 32 + lane < a.cols;
#pragma unroll 1
            for (int r0 = 0; r0 < high; r0 += kLines) {
                uint32_t word[kLines];
                int64_t at[kLines];
#pragma unroll
                for (int k = 0; k < kLines; ++k) word[k] = box_word(box, r0 + k, lane);
#pragma unroll
                for (int k = 0; k < kLines; ++k) at[k] = static_cast<int64_t>(__shfl_sync(~0u, place, r0 + k)) * a.ldo;
#pragma unroll
                for (int k = 0; k < kLines; ++k)
                    if (r0 + k < high && in) static_cast<uint32_t*>(a.out)[at[k] + col0 + b * 32 + lane] = word[k];
            }
        }
    } else {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            if (col0 + b * 64 >= a.cols) break;
            __syncwarp();
            if (a.ct == kCF16) fill_box16<kCF16>(line, lane, v, b * 64);
            else fill_box16<kCBF16>(line, lane, v, b * 64);
            __syncwarp();
            const int left = a.cols - (col0 + b * 64);   // columns of this box that exist
#pragma unroll 1
            for (int r0 = 0; r0 < high; r0 += kLines) {
                uint32_t word[kLines];
                uint16_t* to[kLines];
#pragma unroll
                for (int k = 0; k < kLines; ++k) word[k] = box_word(box, r0 + k, lane);
#pragma unroll
                for (int k = 0; k < kLines; ++k)
                    to[k] = static_cast<uint16_t*>(a.out) +
                            (static_cast<int64_t>(__shfl_sync(~0u, place, r0 + k)) * a.ldo + col0 + b * 64);
#pragma unroll
                for (int k = 0; k < kLines; ++k) {
                    // numbers c and c + 1 of the row make this lane's word
                    const uint32_t odd = (reinterpret_cast<uintptr_t>(to[k]) >> 1) & 1;
                    const uint32_t next = __shfl_down_sync(~0u, word[k], 1);
                    const uint32_t pair = __funnelshift_r(word[k], next, odd * 16);
                    const int c = 2 * lane + static_cast<int>(odd);
                    const bool row_in = r0 + k < high;
                    const bool whole = row_in && c + 1 < left && c < 63;
                    if (whole) *reinterpret_cast<uint32_t*>(to[k] + c) = pair;
                    if (row_in && !whole && c < left) to[k][c] = static_cast<uint16_t>(pair & 0xFFFFu);
                    if (row_in && odd && lane == 0) to[k][0] = static_cast<uint16_t>(word[k] & 0xFFFFu);
                }
            }
        }
    }
    __syncwarp();
}

// FEW: the pair copies only p_rows <= 64 rows of P (few tokens), and the ring
// has up to five stages.  The full form keeps the ring's geometry constant:
// computing it as it went cost the issuing thread 9 % at 8192 x 131072 x 4096.
template <int MODE, bool FEW>
__global__ void __launch_bounds__(kThreads, 1)
head_gemm_kernel(const __grid_constant__ Params first, const __grid_constant__ Params second) {
    // The two products of a gradient go in one launch: units of the first,
    // then units of the second.  The other modes have one.
    constexpr bool kTwo = MODE == kHeadProduct && !FEW;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    const uint32_t base = smem_u32(smem);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kRingBytes + kStoreBytes);
    const uint32_t bar0 = smem_u32(bars);
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (kMaxStages + s); };
    auto accf_bar = [&](int b) { return bar0 + 8u * (2 * kMaxStages + b); };
    auto acce_bar = [&](int b) { return bar0 + 8u * (2 * kMaxStages + 2 + b); };
    const uint32_t drain_bar = bar0 + 8u * (2 * kMaxStages + 4);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + kBars);
    volatile uint32_t* abort_flag = tmem_slot + 1;
    volatile uint64_t* limit_ns = reinterpret_cast<volatile uint64_t*>(tmem_slot + 2);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kMaxStages; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(accf_bar(b), 1);
            mbar_init(acce_bar(b), 16);   // eight epilogue warps in each CTA
        }
        mbar_init(drain_bar, 1);
        *abort_flag = 0;
        *limit_ns = first.a.wait_limit_ns;
        fence_barrier_init();
        tma_prefetch_map(&first.p);
        tma_prefetch_map(&first.q);
    }
    if (warp == 1) {
        tmem_alloc_pair(smem_u32(tmem_slot), 512);
        tmem_relinquish_pair();
    }
    tc_fence_before_sync();
    cluster_sync();
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    grid_dep_launch_dependents();
    const Wait wait{abort_flag, mapa_shared(smem_u32(const_cast<uint32_t*>(abort_flag)), rank ^ 1u),
                    limit_ns};
    // every role reads global memory (the number of tokens, at least)
    grid_dep_wait();
    const int p_bytes = FEW ? 2 * first.a.p_rows * kRowBytes : kQBytes, stage_bytes = p_bytes + kQBytes;
    // a product on its own with one or two steps of K leaves the third stage
    // to the results: a second box for each warp
    const int stages = FEW || MODE == kHeadProduct ? first.a.stages : kFullStages;

    if (warp < kFirstSumWarp) {
        regs_give<kRegsCopy>();
        if (warp == 0 || warp == 2) {
            // ---- operand copies (both CTAs): warp 0 P's, warp 2 Q's ----
            const bool p_side = warp == 0;
            if (lane == 0) {
                const Work w1(first.a), w2 = kTwo ? Work(second.a) : Work();
                Turns turns(w1, w1.steps / first.a.splits, w2, kTwo && second.a.splits ? w2.steps / second.a.splits : 0);
                const bool alt1 = MODE == kHeadProduct && first.a.spread && *first.a.spread;
                const bool alt2 = kTwo && second.a.spread && *second.a.spread;
                bool two;
                int u;
                int stage = 0;
                uint32_t phase = 0, armed = 0, armed_parity = 0;
                bool ok = true;
                int items = 0;
                // self-test: the tile in which the pair's four copying threads
                // stop, and after how many of its stages
                int stall_item = -1, stall_step = 0;
                if (static_cast<int>(cluster_id_x()) == first.a.stall_cluster && w1.steps > 0) {
                    stall_item = first.a.stall_fill / w1.steps;
                    stall_step = first.a.stall_fill % w1.steps;
                }
                while (ok && turns.next(two, u)) {
                    const Params& x = kTwo && two ? second : first;
                    const Args& a = x.a;
                    const Unit it = unit_of(a, kTwo && two ? w2 : w1, u);
                    const int r0 = (p_side ? it.pb * kHeadTileM : it.qb * kHeadTileN) + static_cast<int>(rank) * 128;
                    // every other unit walks K backwards: it starts on the operand
                    // slices that the wave before it read last (still in L2)
                    const bool down = (items & 1) != 0;
                    const int k_end = items == stall_item ? it.k0 + stall_step : it.k1;
                    ok = items++ != stall_item;
                    const bool alt = kTwo && two ? alt2 : alt1;
                    const CUtensorMap* map = !p_side ? &x.q : alt ? &x.by_row : &x.p;
                    const bool kmajor = p_side ? a.p_kmajor : a.q_kmajor;
                    for (int s = it.k0; s < k_end; ++s) {
                        const int ks = down ? it.k1 - 1 - (s - it.k0) : s;
                        if (!wait_phase<false>(empty_bar(stage), phase ^ 1u, wait, kErrProducer)) {
                            ok = false;
                            break;
                        }
                        const uint32_t fb = mapa_shared(full_bar(stage), 0);
                        const uint32_t sp = base + stage * stage_bytes;
                        if (p_side) {
                            if (leader) {   // all four threads' bytes complete on the even CTA's barrier
                                mbar_arrive_expect_tx(full_bar(stage), static_cast<uint32_t>(
                                    FEW ? p_bytes + 2 * kQBytes : 2 * stage_bytes));
                                armed |= 1u << stage;
                                armed_parity = (armed_parity & ~(1u << stage)) | (phase << stage);
                            }
                            if (!FEW || leader) load_stage(sp, map, fb, kmajor, p_bytes / 2, r0, ks * kHeadStepK);
                        } else {
                            load_stage(sp + p_bytes, map, fb, kmajor, kQBytes / 2, r0, ks * kHeadStepK);
                        }
                        if (++stage == stages) {
                            stage = 0;
                            phase ^= 1u;
                        }
                    }
                }
                if (leader && p_side)
                    for (int s = 0; s < stages; ++s)
                        if (armed & (1u << s)) drain(full_bar(s), (armed_parity >> s) & 1u, kDrainNs);
            }
            __syncwarp();
        } else if (warp == 1) {
            // ---- products (even CTA, for both) ----
            if (lane == 0 && leader) {
                const Work w1(first.a), w2 = kTwo ? Work(second.a) : Work();
                Turns turns(w1, w1.steps / first.a.splits, w2, kTwo && second.a.splits ? w2.steps / second.a.splits : 0);
                bool two;
                int u;
                int stage = 0, acc = 0;
                uint32_t phase = 0, acc_phase = 0;
                bool ok = true;
                while (ok && turns.next(two, u)) {
                    const Params& x = kTwo && two ? second : first;
                    const Args& a = x.a;
                    const Unit it = unit_of(a, kTwo && two ? w2 : w1, u);
                    // along K: 16 K further is 32 bytes along a row, 64 K further the
                    // next atom; across K: 16 or 64 lines of 128 bytes, and the
                    // next 64 rows 16 KiB on
                    const uint64_t dp = a.p_kmajor ? smem_desc_sw128(base, 16, 1024)
                                                   : smem_desc_sw128(base, kQBytes / 2, 1024);
                    const uint64_t dq = a.q_kmajor ? smem_desc_sw128(base + p_bytes, 16, 1024)
                                                   : smem_desc_sw128(base + p_bytes, kQBytes / 2, 1024);
                    const uint32_t step_p = a.p_kmajor ? 2u : 128u, step_q = a.q_kmajor ? 2u : 128u;
                    const uint32_t atom_p = a.p_kmajor ? static_cast<uint32_t>(p_bytes / 2) >> 4 : 512u;
                    const uint32_t atom_q = a.q_kmajor ? (kQBytes / 2) >> 4 : 512u;
                    const uint32_t idesc = a.idesc;
                    const int chunk = a.chunk;
                    for (int c0 = it.k0; ok && c0 < it.k1; c0 += chunk) {
                        const int c1 = min(it.k1, c0 + chunk);
                        if (!wait_phase<true>(acce_bar(acc), acc_phase ^ 1u, wait, kErrMma)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after_sync();
                        const uint32_t d = tmem + static_cast<uint32_t>(acc * 256);
                        for (int s = c0; s < c1; ++s) {
                            if (!wait_phase<false>(full_bar(stage), phase, wait, kErrMma)) {
                                ok = false;
                                break;
                            }
                            tc_fence_after_sync();
                            const uint64_t so = static_cast<uint64_t>((stage * stage_bytes) >> 4);
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                const uint64_t op = so + j * atom_p, oq = so + j * atom_q;
#pragma unroll
                                for (int kk = 0; kk < 4; ++kk)
                                    tc_mma_pair<0>(d, dp + op + kk * step_p, dq + oq + kk * step_q, idesc,
                                                   (s > c0 || j > 0 || kk > 0) ? 1u : 0u);
                            }
                            tc_commit_pair_multicast(empty_bar(stage), 0x3);
                            if (++stage == stages) {
                                stage = 0;
                                phase ^= 1u;
                            }
                        }
                        if (!ok) break;
                        tc_commit_pair_multicast(accf_bar(acc), 0x3);
                        acc ^= 1;
                        if (acc == 0) acc_phase ^= 1u;
                    }
                }
                tc_commit_pair_multicast(drain_bar, 0x3);
            }
            __syncwarp();
        }
    } else {
        // ---- sums and results (both CTAs) ----
        regs_take<kRegsSum>();
        const Work w1(first.a), w2 = kTwo ? Work(second.a) : Work();
        Turns turns(w1, w1.steps / first.a.splits, w2, kTwo && second.a.splits ? w2.steps / second.a.splits : 0);
        bool two;
        int u;
        constexpr bool kRows = MODE == kHeadGradCeRows || MODE == kHeadGradKdRows;
        constexpr bool kKd = MODE == kHeadStatsKd || MODE == kHeadGradKd || MODE == kHeadGradKdRows;
        constexpr bool kStats = MODE == kHeadStatsCe || MODE == kHeadStatsKd;
        constexpr bool kGrad = MODE == kHeadGradCe || MODE == kHeadGradKd || kRows;
        const int quarter = warp & 3;                   // tensor-memory lanes 32 * quarter ..
        const int half = (warp - kFirstSumWarp) >> 2;   // columns 128 * half ..
        const uint32_t box = base + kRingBytes + static_cast<uint32_t>(warp - kFirstSumWarp) * 4096u;
        const uint32_t box1 = MODE == kHeadProduct && !FEW && stages < kFullStages
                                  ? base + (kFullStages - 1) * stage_bytes + static_cast<uint32_t>(warp - kFirstSumWarp) * 4096u
                                  : box;
        const uint32_t lanes = (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(half * kCols);
        const float factor1 = MODE == kHeadProduct && first.a.factor ? *first.a.factor : 1.0f;
        const float factor2 = kTwo && second.a.factor ? *second.a.factor : 1.0f;
        const bool spread = kRows && *first.a.spread;
        int acc = 0;
        uint32_t acc_phase = 0;
        bool ok = true;
        while (ok && turns.next(two, u)) {
            const Params& x = kTwo && two ? second : first;
            const Args& a = x.a;
            const Work& w = kTwo && two ? w2 : w1;
            const Unit it = unit_of(a, w, u);
            const int row0 = it.pb * kHeadTileM + static_cast<int>(rank) * 128 + quarter * 32;
            const int col0 = it.qb * kHeadTileN + half * kCols;
            const int row = row0 + lane;
            const bool some = row0 < w.m && col0 < a.n;   // of this warp's results are wanted
            const int32_t word0 = a.w0 + col0;
            Hits hits;
            float lse2 = 0.0f, gain = 0.0f, boost = 0.0f, ratio = 0.0f;
            float factor = kTwo && two ? factor2 : factor1;
            if (MODE == kHeadProduct && a.row_factor && row < w.m) factor = a.row_factor[row];
            if (!kKd && (kStats || kGrad) && row < w.m) hits.start<kKd>(a, row, word0);
            if (kGrad && row < w.m) {
                lse2 = a.lse2[row];
                gain = a.gain[row];
                boost = a.boost[row];
                if (kRows && spread) ratio = a.ratio[row];
            }
            float v[kCols];
            if (it.k0 == it.k1) {   // the empty sum
#pragma unroll
                for (int i = 0; i < kCols; ++i) v[i] = 0.0f;
            }
            const int chunk = a.chunk;
            for (int c0 = it.k0; c0 < it.k1; c0 += chunk) {
                ok = wait_phase<false>(accf_bar(acc), acc_phase, wait, kErrEpilogue);
                if (!__all_sync(~0u, ok)) {
                    if (lane == 0) raise_abort(wait);
                    ok = false;
                    break;
                }
                tc_fence_after_sync();
                const uint32_t from = tmem + static_cast<uint32_t>(acc * 256) + lanes;
                const uint32_t freed = mapa_shared(acce_bar(acc), 0);
                auto free_buffer = [&]() {   // all of it has been read
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_relaxed_cluster(freed);
                };
                if (!some) {
                    free_buffer();
                } else if (c0 == it.k0) {   // the first chunk is the sum so far
                    uint32_t r[kCols / 32][32];
#pragma unroll
                    for (int c = 0; c < kCols / 32; ++c) tmem_ld_32x32b_x32(from + c * 32, r[c]);
                    tmem_wait_ld();
                    free_buffer();
#pragma unroll
                    for (int i = 0; i < kCols; ++i) v[i] = __uint_as_float(r[i / 32][i % 32]);
                } else {
                    // 32 columns at a time, the next read under way while the
                    // last one's are added
                    uint32_t r[2][32];
                    tmem_ld_32x32b_x32(from, r[0]);
#pragma unroll
                    for (int c = 0; c < kCols / 32; ++c) {
                        tmem_wait_ld();
                        if (c + 1 < kCols / 32) tmem_ld_32x32b_x32(from + (c + 1) * 32, r[(c + 1) & 1]);
                        else free_buffer();
                        add32(v, c * 32, r[c & 1]);
                    }
                }
                acc ^= 1;
                if (acc == 0) acc_phase ^= 1u;
                // A list is searched (a chain of reads) after the unit's first
                // chunk: before it, the search would add to the time in which
                // the last unit's results are formed and no buffer is freed.
                if (kKd && c0 == it.k0 && row < w.m) hits.start<kKd>(a, row, word0);
            }
            if (!ok) break;
            if (kKd && it.k0 == it.k1 && row < w.m) hits.start<kKd>(a, row, word0);

            const int wide = min(kCols, a.n - col0);   // columns that exist (may be <= 0)
            if constexpr (kStats) {
                if (!some) continue;
                const int32_t hi = word0 + wide;
#pragma unroll
                for (int c = 0; c < kCols / 32; ++c) {
                    const int32_t stop = min(hi, word0 + 32 * (c + 1));
                    if (!__any_sync(~0u, hits.next < stop)) continue;
#pragma unroll
                    for (int i = 0; i < 32; ++i) st_shared(scratch_at(box, lane, i), v[c * 32 + i]);
                    while (hits.next < stop) {
                        a.z_at[kKd ? hits.row + hits.at : hits.row] =
                            ld_shared(scratch_at(box, lane, hits.next - word0 - 32 * c));
                        hits.advance<kKd>();
                    }
                    __syncwarp();
                }
                if (a.zsum) {
                    float x0 = 0.0f, x1 = 0.0f, x2 = 0.0f, x3 = 0.0f;
#pragma unroll
                    for (int i = 0; i < kCols; i += 4) {   // columns past the last are zeros
                        x0 += v[i];
                        x1 += v[i + 1];
                        x2 += v[i + 2];
                        x3 += v[i + 3];
                    }
                    if (row < w.m) a.zsum[static_cast<int64_t>(word0 / kCols) * a.ld_stats + row] = (x0 + x1) + (x2 + x3);
                }
                if (wide < kCols) {
#pragma unroll
                    for (int i = 0; i < kCols; ++i) v[i] = i < wide ? v[i] : -INFINITY;
                }
                float t0 = -INFINITY, t1 = t0, t2 = t0, t3 = t0;
#pragma unroll
                for (int i = 0; i < kCols; i += 4) {
                    t0 = fmaxf(t0, v[i]);
                    t1 = fmaxf(t1, v[i + 1]);
                    t2 = fmaxf(t2, v[i + 2]);
                    t3 = fmaxf(t3, v[i + 3]);
                }
                const float top = fmaxf(fmaxf(t0, t1), fmaxf(t2, t3)) * a.scale2;
                const float off = top == -INFINITY ? 0.0f : -top;
                float s0 = 0.0f, s1 = 0.0f, s2 = 0.0f, s3 = 0.0f;
#pragma unroll
                for (int i = 0; i < kCols; i += 4) {
                    s0 += exp2_fast(fmaf(v[i], a.scale2, off));
                    s1 += exp2_fast(fmaf(v[i + 1], a.scale2, off));
                    s2 += exp2_fast(fmaf(v[i + 2], a.scale2, off));
                    s3 += exp2_fast(fmaf(v[i + 3], a.scale2, off));
                }
                if (row < w.m)
                    a.stats[static_cast<int64_t>(word0 / kCols) * a.ld_stats + row] =
                        make_float2(top, (s0 + s1) + (s2 + s3));
            } else if constexpr (kGrad) {
                const float slope = boost * gain, shift = -a.flat * gain;
#pragma unroll
                for (int i = 0; i < kCols; ++i)
                    v[i] = fmaf(exp2_fast(fmaf(v[i], a.scale2, -lse2)), slope, shift);
                const int32_t hi = word0 + wide;
#pragma unroll
                for (int c = 0; c < kCols / 32; ++c) {
                    const int32_t stop = min(hi, word0 + 32 * (c + 1));
                    if (!__any_sync(~0u, hits.next < stop)) continue;
                    if (lane == 0) bulk_wait_group_read<0>();   // the box's last store has left it
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 32; ++i) st_shared(scratch_at(box, lane, i), v[c * 32 + i]);
                    while (hits.next < stop) {
                        const float y = kKd ? expf(a.logq[hits.row + hits.at]) : a.hit;
                        const uint32_t x = scratch_at(box, lane, hits.next - word0 - 32 * c);
                        st_shared(x, ld_shared(x) - y * gain);
                        hits.advance<kKd>();
                    }
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[c * 32 + i] = ld_shared(scratch_at(box, lane, i));
                }
                // zeros in rows past the last token, which K of dweight may
                // read, and in words past the last, which K of dhidden may
                if (row0 + 32 > w.m) {
#pragma unroll
                    for (int i = 0; i < kCols; ++i) v[i] = row < w.m ? v[i] : 0.0f;
                }
                if (wide < kCols) {
#pragma unroll
                    for (int i = 0; i < kCols; ++i) v[i] = i < wide ? v[i] : 0.0f;
                }
                __syncwarp();
                const Out to(a);
                // where weights differ, the copy with a scale for each row first
#pragma unroll 1
                for (bool by_row = kRows && spread;; by_row = false) {
                    store_boxes(to, by_row ? &x.by_row : &x.o, box, box, v, lane, row0, row0, col0);
                    if (!by_row) break;
                    scale_all(v, ratio);
                }
            } else {
                if (!some) continue;
                const Out to(a);
                const bool tensor_store = a.tensor_store;
                const int split_rows = a.split_rows;
                scale_all(v, factor);
                if (tensor_store) {
                    store_boxes(to, &x.o, box, box1, v, lane, row0, row0 + it.seg * split_rows, col0);
                } else {
                    if (lane == 0) bulk_wait_group_read<0>();   // the other product's last store has left the box
                    store_lines(to, box, v, lane, row0, w.m, col0);
                }
            }
        }
        if (lane == 0) bulk_wait_group<0>();   // every tensor store has completed
        __syncwarp();
    }

    tc_fence_before_sync();
    __syncthreads();
    if (warp == 1 && lane == 0) {
        // every product of the pair has finished (it may read this CTA's
        // shared memory and write its tensor memory)
        drain(drain_bar, 0, kPairDrainNs);
        if (*abort_flag) {   // give copies issued just before an abort time to land
            const uint64_t t1 = globaltimer_ns();
            while (globaltimer_ns() - t1 < 50000ull) {
            }
        }
    }
    __syncwarp();
    tc_fence_before_sync();
    cluster_sync();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc_pair(tmem, 512);
    }
}

bool encode(EncodeTiledFn fn, CUtensorMap* map, CUtensorMapDataType type, int64_t esize, const void* base,
            int64_t inner, int64_t outer, int64_t ld, uint32_t box_inner, uint32_t box_outer,
            CUtensorMapL2promotion promotion) {
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(outer)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld * esize)};
    const cuuint32_t box[2] = {box_inner, box_outer};
    const cuuint32_t ones[2] = {1, 1};
    return fn(map, type, 2, const_cast<void*>(base), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, promotion, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int MODE, bool FEW>
cudaError_t launch_form(int grid, const Params& first, const Params& second, cudaStream_t stream) {
    auto kernel = head_gemm_kernel<MODE, FEW>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemBytes;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, first, second);
}

template <int MODE>
cudaError_t launch(int grid, bool few, const Params& first, const Params& second, cudaStream_t stream) {
    return few ? launch_form<MODE, true>(grid, first, second, stream)
               : launch_form<MODE, false>(grid, first, second, stream);
}

}  // namespace

cudaError_t head_error_word(uint32_t** ptr) {
    return cudaGetSymbolAddress(reinterpret_cast<void**>(ptr), g_head_error);
}

bool head_gemm_tensor_store(const void* out, int ct, int64_t inner, int64_t ld) {
    const int64_t quantum = 16 / c_elem_bytes(ct);
    return (reinterpret_cast<uintptr_t>(out) & 15) == 0 && ld % quantum == 0 && inner % quantum == 0;
}

static int64_t units_of(const HeadGemm& g) {
    return ceil_div(g.m, kHeadTileM) * ceil_div(g.n, kHeadTileN) * g.splits;
}

static bool params_of(const HeadGemm& g, int p_rows, int stages, EncodeTiledFn fn, Params* x) {
    memset(x, 0, sizeof(*x));
    const CUtensorMapDataType t16 = g.bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    // along K: 64 K x rows; across K: 64 rows x 128 K
    const uint32_t box_p = g.p.kmajor ? static_cast<uint32_t>(p_rows) : kHeadStepK, box_q = 128;
    if (!encode(fn, &x->p, t16, 2, g.p.base, g.p.inner, g.p.outer, g.p.ld, 64, box_p, CU_TENSOR_MAP_L2_PROMOTION_L2_256B) ||
        !encode(fn, &x->q, t16, 2, g.q.base, g.q.inner, g.q.outer, g.q.ld, 64, box_q, CU_TENSOR_MAP_L2_PROMOTION_L2_256B))
        return false;
    Args& a = x->a;
    if (g.out && !g.out_perm && head_gemm_tensor_store(g.out, g.ct, g.out_inner, g.ldo)) {
        const int64_t es = c_elem_bytes(g.ct);
        const CUtensorMapDataType t = g.ct == kCF32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                      : g.ct == kCF16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                      : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
        if (!encode(fn, &x->o, t, es, g.out, g.out_inner, g.out_outer, g.ldo, static_cast<uint32_t>(128 / es), 32,
                    CU_TENSOR_MAP_L2_PROMOTION_NONE))
            return false;
        a.tensor_store = 1;
        if (g.by_row && g.mode != kHeadProduct &&
            !encode(fn, &x->by_row, t, es, g.by_row, g.out_inner, g.out_outer, g.ldo, static_cast<uint32_t>(128 / es),
                    32, CU_TENSOR_MAP_L2_PROMOTION_NONE))
            return false;
    }
    if (g.by_row && g.mode == kHeadProduct &&
        !encode(fn, &x->by_row, t16, 2, g.by_row, g.p.inner, g.p.outer, g.p.ld, 64, box_p,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B))
        return false;
    // slices, sums onto the output and the logits' gradient leave through tensor stores only
    if (!a.tensor_store && (g.splits > 1 || g.add || (g.out && g.mode != kHeadProduct))) return false;
    a.m = static_cast<int32_t>(g.m);
    a.n = static_cast<int32_t>(g.n);
    a.k = static_cast<int32_t>(g.k);
    a.count_is = g.count_is;
    a.splits = g.splits;
    a.chunk = g.chunk;
    // Rows of tiles to a raster group.  Logits (8192 x 131072 x 4096, statistics):
    // 4, 8, 16 and 32 took 5336, 5130, 5020 and 5168 us; the products differ by
    // less than 1 % from 4 to 16 and lose 2 % at 32.
    a.group = static_cast<int32_t>(std::min<int64_t>(g.mode == kHeadProduct ? 8 : 16, ceil_div(g.m, kHeadTileM)));
    a.p_kmajor = g.p.kmajor;
    a.q_kmajor = g.q.kmajor;
    a.p_rows = p_rows;
    a.stages = stages;
    a.idesc = idesc_f16_f32(g.bf16 ? 1u : 0u, !g.p.kmajor, !g.q.kmajor, kHeadTileM, kHeadTileN);
    a.wait_limit_ns = g.wait_limit_ns ? g.wait_limit_ns : kWaitNs;
    a.stall_cluster = g.stall_fill > 0 ? g.stall_cluster : -1;
    a.stall_fill = g.stall_fill - 1;
    a.count = g.rows.count;
    a.out = g.out;
    a.ldo = g.ldo;
    a.ct = g.ct;
    a.add = g.add;
    a.out_rows = static_cast<int32_t>(g.splits > 1 ? g.split_rows : g.out_outer);
    a.out_cols = static_cast<int32_t>(g.out_inner);
    a.split_rows = static_cast<int32_t>(g.split_rows);
    a.out_perm = g.out_perm;
    a.factor = g.factor;
    a.row_factor = g.row_factor;
    a.spread = g.by_row ? g.spread : nullptr;
    a.ratio = g.ratio;
    a.target_c = g.rows.target_c;
    a.target = g.rows.target;
    a.target_stride = g.rows.target_stride;
    a.ignore_index = g.rows.ignore_index;
    a.vocab = g.rows.vocab;
    a.perm = g.rows.perm;
    a.words = g.rows.words;
    a.logq = g.rows.logq;
    a.top_k = g.rows.top_k;
    a.w0 = static_cast<int32_t>(g.w0);
    a.scale2 = g.scale2;
    a.flat = g.rows.vocab > 0 ? g.label_smoothing / static_cast<float>(g.rows.vocab) : 0.0f;
    a.hit = 1.0f - g.label_smoothing;
    a.stats = g.stats;
    a.zsum = g.zsum;
    a.ld_stats = g.ld_stats;
    a.z_at = g.z_at;
    a.lse2 = g.lse2;
    a.gain = g.gain;
    a.boost = g.boost;
    return true;
}

int64_t head_gemm_clusters(const HeadGemm& g, const HeadGemm* and_then, int clusters) {
    return std::min<int64_t>(units_of(g) + (and_then ? units_of(*and_then) : 0), clusters);
}

cudaError_t head_gemm_launch(const HeadGemm& g, const HeadGemm* and_then, int clusters, EncodeTiledFn fn,
                             cudaStream_t stream) {
    const int64_t units = units_of(g) + (and_then ? units_of(*and_then) : 0);
    if (clusters < 1 || units < 1 || units > INT32_MAX || g.chunk < 1) return cudaErrorInvalidValue;
    if (and_then && (g.mode != kHeadProduct || and_then->mode != kHeadProduct || and_then->chunk < 1))
        return cudaErrorInvalidValue;
    // Few rows of P (few tokens): copy only as many of the pair's 256, so
    // that the ring has room for more stages of Q.  Q is then all the
    // traffic, and more of it is in flight.
    int p_rows = 128;
    if (!and_then && g.p.kmajor && g.m <= 64) p_rows = g.m <= 16 ? 16 : g.m <= 32 ? 32 : 64;
    int stages = std::min(kMaxStages, kRingBytes / (2 * p_rows * kRowBytes + kQBytes));
    if (g.mode == kHeadProduct && !and_then && p_rows == 128 && g.k <= 2 * kHeadStepK) stages = 2;
    Params first, second;
    if (!params_of(g, p_rows, stages, fn, &first)) return cudaErrorInvalidValue;
    memset(&second, 0, sizeof(second));
    if (and_then && !params_of(*and_then, p_rows, stages, fn, &second)) return cudaErrorInvalidValue;
    const int grid = 2 * static_cast<int>(head_gemm_clusters(g, and_then, clusters));
    const bool few = p_rows < 128;
    switch (g.mode) {
        case kHeadStatsCe: return launch<kHeadStatsCe>(grid, few, first, second, stream);
        case kHeadStatsKd: return launch<kHeadStatsKd>(grid, few, first, second, stream);
        case kHeadGradCe: return launch<kHeadGradCe>(grid, few, first, second, stream);
        case kHeadGradCeRows: return launch<kHeadGradCeRows>(grid, few, first, second, stream);
        case kHeadGradKdRows: return launch<kHeadGradKdRows>(grid, few, first, second, stream);
        case kHeadGradKd: return launch<kHeadGradKd>(grid, few, first, second, stream);
        case kHeadProduct: return launch<kHeadProduct>(grid, few, first, second, stream);
    }
    return cudaErrorInvalidValue;
}

}  // namespace gb300
