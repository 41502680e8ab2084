// Key bounds of cache blocks (pkv_block_bounds) and the choice of blocks by
// them (pkv_select_blocks).
//
// A block's keys lie, dimension by dimension, between lo_d and hi_d, so a
// query's dot product with any of them is at most
//   sum_d max(q_d hi_d, q_d lo_d) = sum_d max(q_d, 0) hi_d + min(q_d, 0) lo_d,
// the block's score: a dot product of length 2 D that reads 2 D bytes where the
// keys themselves are 32 D.  Bounds and query are held as 8-bit codes of a
// power-of-two unit, so a code's product with a code is a whole number, a sum
// of D of them stays below 128 * 127 * 127 < 2^24, and the units only move the
// exponent: every score is exact in single precision.  The choice is thus a
// function of the inputs alone, whatever order the sums are taken in.
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>

#include "launch_cache.h"
#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "sparse_common.cuh"

namespace pkv {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kUnbounded = 127;      // exponent of a block with a key that is not finite

// The least e with amax <= 127 * 2^e, kept within -50 .. 50 (two such exponents
// and a code sum below 2^21 multiply without leaving the normal range).
__device__ __forceinline__ int code_exponent(float amax) {
    const uint32_t b = __float_as_uint(amax);
    // amax = 1.f * 2^(x - 127): 127 = 1.984375 * 2^6
    const int e = int(b >> 23) - 127 - 6 + ((b & 0x7fffffu) > 0x7e0000u ? 1 : 0);
    return min(max(e, -50), 50);
}

__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }

// ---- bounds -------------------------------------------------------------------
struct BoundsParams {
    int8_t* bounds;             // [num_blocks][Hkv][2][D]: hi codes, lo codes
    int8_t* exps;               // [num_blocks][Hkv]
    const void* k_cache;
    const int32_t* block_tables;
    const int32_t* start;       // [n + 1] or null
    const int32_t* ctx;
    int32_t table_stride, n, tokens, num_blocks, num_kv_heads;
    int span;                   // tokens that one CTA looks at
    int* err;
};

constexpr int kBoundsWarps = 8;
constexpr int kMaxSpan = 16;

template <typename T, int V>
__device__ __forceinline__ void load_vec(const T* p, float (&x)[V]);
template <>
__device__ __forceinline__ void load_vec<float, 4>(const float* p, float (&x)[4]) {
    const float4 v = __ldg(reinterpret_cast<const float4*>(p));
    x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
}
template <>
__device__ __forceinline__ void load_vec<__nv_bfloat16, 8>(const __nv_bfloat16* p, float (&x)[8]) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

// A CTA looks at `span` query tokens; a token that is the first of its sequence
// in the step, or the first row of its block, stands for that block.  Each of
// the blocks found, times the KV heads, is one warp's tile: the warp reads the
// rows that hold tokens, keeps the largest and the smallest value of each
// dimension, and writes codes rounded outwards.
template <typename T, int D>
__global__ void __launch_bounds__(kBoundsWarps * 32) block_bounds_kernel(BoundsParams p) {
    constexpr int V = 16 / int(sizeof(T));       // elements of a 16-byte load
    constexpr int LPR = D / V;                   // lanes of a row
    constexpr int RPI = 32 / LPR;                // rows of a load
    __shared__ int32_t blk[kMaxSpan], rows[kMaxSpan];
    __shared__ int count;
    pdl_wait_prerequisites();
    pdl_launch_dependents();
    if (threadIdx.x == 0) count = 0;
    __syncthreads();
    const int t = blockIdx.x * p.span + threadIdx.x;
    if (int(threadIdx.x) < p.span && t < p.tokens) {
        int first, q;
        const int s = token_seq(p.start, p.n, t, first, q, p.err);
        if (s >= 0) {
            const int ctx = p.ctx[s];
            const int pos = ctx - q + (t - first);
            if (ctx < q) {
                if (t == first) flag_error(p.err, PKV_DEV_BAD_CONTEXT_LEN);
            } else if (t == first || pos % kBlockTokens == 0) {
                const int b = pos / kBlockTokens;
                if (b >= p.table_stride) {
                    flag_error(p.err, PKV_DEV_TABLE_TOO_NARROW);
                } else {
                    const int id = p.block_tables[size_t(s) * p.table_stride + b];
                    if (id < 0 || id >= p.num_blocks) {
                        flag_error(p.err, PKV_DEV_BAD_BLOCK_ID);
                    } else {
                        const int at = atomicAdd(&count, 1);
                        blk[at] = id;
                        rows[at] = min(kBlockTokens, ctx - b * kBlockTokens);
                    }
                }
            }
        }
    }
    __syncthreads();
    const int lane = threadIdx.x & 31;
    const int tiles = count * p.num_kv_heads;
    for (int i = threadIdx.x >> 5; i < tiles; i += kBoundsWarps) {
        const int a = i / p.num_kv_heads, h = i % p.num_kv_heads;
        const size_t tile = size_t(blk[a]) * p.num_kv_heads + h;
        const int nrow = rows[a];
        const T* k = static_cast<const T*>(p.k_cache) + tile * (kBlockTokens * D) +
                     (lane / LPR) * D + (lane % LPR) * V;
        float hi[V], lo[V];
        bool odd = false;                        // a value that is not finite
#pragma unroll
        for (int j = 0; j < V; ++j) hi[j] = -INFINITY, lo[j] = INFINITY;
#pragma unroll
        for (int r = 0; r < kBlockTokens; r += RPI) {
            if (r + lane / LPR < nrow) {
                float x[V];
                load_vec<T, V>(k + r * D, x);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    odd |= !(fabsf(x[j]) <= FLT_MAX);
                    hi[j] = fmaxf(hi[j], x[j]);
                    lo[j] = fminf(lo[j], x[j]);
                }
            }
        }
#pragma unroll
        for (int o = LPR; o < 32; o <<= 1)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                hi[j] = fmaxf(hi[j], __shfl_xor_sync(kFull, hi[j], o));
                lo[j] = fminf(lo[j], __shfl_xor_sync(kFull, lo[j], o));
            }
        float amax = 0.f;
#pragma unroll
        for (int j = 0; j < V; ++j) amax = fmaxf(amax, fmaxf(fabsf(hi[j]), fabsf(lo[j])));
#pragma unroll
        for (int o = 1; o < LPR; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, o));
        odd = __any_sync(kFull, odd);
        const int e = code_exponent(amax);
        const float unit = odd ? 0.f : pow2(-e);
        if (lane < LPR) {
            alignas(8) int8_t ch[V], cl[V];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                // (a block with values that are not finite has codes of 0)
                ch[j] = odd ? 0 : int8_t(fminf(fmaxf(ceilf(hi[j] * unit), -127.f), 127.f));
                cl[j] = odd ? 0 : int8_t(fminf(fmaxf(floorf(lo[j] * unit), -127.f), 127.f));
            }
            int8_t* dst = p.bounds + tile * (2 * D) + lane * V;
            if constexpr (V == 8) {
                *reinterpret_cast<uint2*>(dst) = *reinterpret_cast<const uint2*>(ch);
                *reinterpret_cast<uint2*>(dst + D) = *reinterpret_cast<const uint2*>(cl);
            } else {
                *reinterpret_cast<uint32_t*>(dst) = *reinterpret_cast<const uint32_t*>(ch);
                *reinterpret_cast<uint32_t*>(dst + D) = *reinterpret_cast<const uint32_t*>(cl);
            }
        }
        if (lane == 0) p.exps[tile] = int8_t(odd ? kUnbounded : e);
    }
}

// ---- selection ------------------------------------------------------------------
struct SelectParams {
    int32_t* selected;          // [tokens][Hkv][top_k]
    const void* q;
    const int8_t* bounds;
    const int8_t* exps;
    QueryRows rows;
    uint32_t* far_keys;         // [tokens][Hkv][stride] where a row's keys do not fit on chip
    int32_t stride;             // blocks of max_context_len, a multiple of 4
    int32_t num_blocks, num_q_heads, num_kv_heads;
    int32_t top_k, sink, recent;
    int32_t q_f32;              // q is fp32, else bf16
    int* err;
};

constexpr int kSelThreads = 256;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kWarpBlocks = 16;      // blocks that a warp scores at a time
constexpr int kBins = 1024;
constexpr int kMaxCand = kSelThreads;
constexpr int kKeyBytes = 192 << 10; // most shared memory for a CTA's keys

// Floats in an order that unsigned compare keeps (no NaN among the scores).
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t b = __float_as_uint(x);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

struct PickScratch {
    uint32_t hist[kBins];
    uint32_t cand[kMaxCand];
    uint32_t warp_a[kSelWarps], warp_b[kSelWarps];
    uint32_t bin, above, inside, count, cut, take;
};

// Exclusive sums over the CTA of two values per thread.
__device__ __forceinline__ void scan_two(uint32_t& a, uint32_t& b, PickScratch& s) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t a0 = a, b0 = b;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t ua = __shfl_up_sync(kFull, a, o), ub = __shfl_up_sync(kFull, b, o);
        if (lane >= o) a += ua, b += ub;
    }
    if (lane == 31) s.warp_a[warp] = a, s.warp_b[warp] = b;
    __syncthreads();
    for (int w = 0; w < warp; ++w) a += s.warp_a[w], b += s.warp_b[w];
    a -= a0;
    b -= b0;
}

// The list of one row from the keys of its blocks, by the whole CTA.  Wanted
// are the `want` largest keys of blocks sink .. blocks - recent - 1 (the ends are
// always taken).  A histogram over the keys' range finds the bin that holds the
// want-th; its few keys are ranked against one another, or, while they are more
// than a CTA ranks at once, the bin becomes the next range.  Scores of a real
// query spread over the bins, so one histogram and one ranking is the rule.
__device__ __forceinline__ void pick_row(const SelectParams& p, const uint32_t* keys, int blocks,
                                         int32_t* out, PickScratch& s) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int b0 = p.sink, b1 = blocks - p.recent;
    uint32_t want = uint32_t(p.top_k - p.sink - p.recent);
    uint32_t cut = 0xffffffffu, take = 0;        // taken: keys above `cut`, `take` equal to it
    if (want > 0) {
        uint32_t lo = 0xffffffffu, hi = 0;
        for (int b = b0 + tid; b < b1; b += kSelThreads) {
            lo = min(lo, keys[b]);
            hi = max(hi, keys[b]);
        }
        lo = __reduce_min_sync(kFull, lo);
        hi = __reduce_max_sync(kFull, hi);
        if (lane == 0) s.warp_a[warp] = lo, s.warp_b[warp] = hi;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kSelWarps; ++w) {
            lo = min(lo, s.warp_a[w]);
            hi = max(hi, s.warp_b[w]);
        }
        for (;;) {                               // the range lo .. hi holds the want-th
            int shift = 0;
            while ((hi - lo) >> shift >= kBins) ++shift;
            for (int i = tid; i < kBins; i += kSelThreads) s.hist[i] = 0;
            if (tid == 0) s.count = 0;
            __syncthreads();
            for (int b = b0 + tid; b < b1; b += kSelThreads) {
                const uint32_t k = keys[b];
                if (k >= lo && k <= hi) atomicAdd(&s.hist[(k - lo) >> shift], 1u);
            }
            __syncthreads();
            // bins from above, four to a thread
            const uint4 c = *reinterpret_cast<const uint4*>(&s.hist[kBins - 4 - 4 * tid]);
            const uint32_t four[4] = {c.w, c.z, c.y, c.x};
            uint32_t sum = c.x + c.y + c.z + c.w, none = 0;
            scan_two(sum, none, s);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (sum < want && want <= sum + four[i]) {
                    s.bin = uint32_t(kBins - 1 - 4 * tid - i);
                    s.above = sum;
                    s.inside = four[i];
                }
                sum += four[i];
            }
            __syncthreads();
            const uint32_t inside = s.inside;
            want -= s.above;
            const uint32_t first = lo + (s.bin << shift);
            const uint32_t last = min(hi, first + ((1u << shift) - 1u));
            if (want == inside) {                // the whole bin (no key is 0: -inf's is above)
                cut = first - 1;
                break;
            }
            if (first == last) {                 // equal keys: the lower indices
                cut = first;
                take = want;
                break;
            }
            if (inside <= kMaxCand) {
                for (int b = b0 + tid; b < b1; b += kSelThreads) {
                    const uint32_t k = keys[b];
                    if (k >= first && k <= last) s.cand[atomicAdd(&s.count, 1u)] = k;
                }
                __syncthreads();
                if (tid < int(inside)) {
                    const uint32_t k = s.cand[tid];
                    uint32_t gt = 0, ge = 0;
                    for (uint32_t i = 0; i < inside; ++i) {
                        gt += s.cand[i] > k;
                        ge += s.cand[i] >= k;
                    }
                    if (gt < want && want <= ge) {   // the same for all keys equal to the cut
                        s.cut = k;
                        s.take = want - gt;
                    }
                }
                __syncthreads();
                cut = s.cut;
                take = s.take;
                break;
            }
            lo = first;
            hi = last;
            __syncthreads();                     // (the bin was read by all)
        }
    }
    // in ascending order: neighbouring blocks to a thread, so that one scan of
    // the counts places them
    const int per = (blocks + kSelThreads - 1) / kSelThreads;
    const int f = min(blocks, tid * per), e = min(blocks, f + per);
    uint32_t above = 0, equal = 0;
    for (int b = f; b < e; ++b) {
        const bool end = b < b0 || b >= b1;
        above += end || keys[b] > cut;
        equal += !end && keys[b] == cut;
    }
    __syncthreads();
    scan_two(above, equal, s);
    for (int b = f; b < e; ++b) {
        const bool end = b < b0 || b >= b1;
        if (end || keys[b] > cut) {
            out[above + min(equal, take)] = b;
            ++above;
        } else if (keys[b] == cut) {
            if (equal < take) out[above + equal] = b;
            ++equal;
        }
    }
    __syncthreads();
}

// Codes of one query head (one warp): positive parts, then negative parts.
template <int D>
__device__ __forceinline__ void query_codes(const SelectParams& p, size_t head, uint32_t* dst,
                                            float* unit) {
    constexpr int PL = D / 32;                   // dimensions of a lane: consecutive
    const int lane = threadIdx.x & 31;
    float x[PL];
    if (p.q_f32) {
        Elem<float>::load(static_cast<const float*>(p.q) + head * D + lane * PL, x);
    } else {
        Elem<__nv_bfloat16>::load(static_cast<const __nv_bfloat16*>(p.q) + head * D + lane * PL, x);
    }
    float amax = 0.f;
    bool odd = false;
#pragma unroll
    for (int j = 0; j < PL; ++j) {
        odd |= !(fabsf(x[j]) <= FLT_MAX);
        amax = fmaxf(amax, fabsf(x[j]));
    }
    // (the bits of values that are not negative order as the values do)
    amax = __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(amax)));
    odd = __any_sync(kFull, odd);
    const int eq = code_exponent(amax);
    const float u = pow2(-eq);
    int8_t* pos = reinterpret_cast<int8_t*>(dst) + lane * PL;
#pragma unroll
    for (int j = 0; j < PL; ++j) {
        // (a query with values that are not finite has codes of 0)
        const int c = odd ? 0 : int(fminf(fmaxf(rintf(x[j] * u), -127.f), 127.f));
        pos[j] = int8_t(max(c, 0));
        pos[D + j] = int8_t(min(c, 0));
    }
    if (lane == 0) *unit = odd ? 0.f : pow2(eq);
}

// A cluster chooses the blocks of R neighbouring query rows of one sequence for
// one KV head, R * G query heads being its columns.  Its CTAs share the
// sequence's blocks; a quad of lanes takes two blocks at a time, each lane 64 of
// their 2 D bytes straight from the pool, and the sums run on the packed 8-bit
// dot product with the columns' codes from shared memory.  A score's key goes to
// the CTA that picks the row (through distributed shared memory, or to global
// memory where the keys of a very long context do not fit), so the scores never
// pass through HBM and one launch does it all.
template <int D, int G, int R>
__global__ void __launch_bounds__(kSelThreads) select_blocks_kernel(SelectParams p) {
    constexpr int CH = 2 * D / 64;               // 64-byte chunks of a bounds row
    constexpr int COLS = G * R;
    extern __shared__ __align__(16) uint32_t near_keys[];   // [rows picked here][stride]
    __shared__ __align__(16) uint32_t qc[COLS][2 * D / 4];
    __shared__ float unit[COLS];
    __shared__ __align__(16) PickScratch scratch;
    const uint32_t cs = cluster_size(), rank = cluster_rank();
    const int item = int(blockIdx.x / cs);
    const int h = item % p.num_kv_heads, t = item / p.num_kv_heads;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (cs > 1) cluster_arrive();                // the others' shared memory is there to write to
    pdl_wait_prerequisites();
    pdl_launch_dependents();
    int first, q;
    int* tell = tid == 0 && h == 0 && rank == 0 ? p.err : nullptr;
    const int seq = token_seq(p.rows.start, p.rows.n, t, first, q, tell);
    const int rows = seq < 0 || (t - first) % R ? 0 : min(R, first + q - t);
    if (rows == 0) {                             // another cluster's row, or behind the last one
        if (cs > 1) cluster_wait();
        return;
    }
    const int keys0 = sequence_keys(p.rows, seq, q, tell) ? p.rows.ctx[seq] - q + (t - first) + 1 : 0;
    const int blocks_end = keys0 > 0 ? (keys0 + rows - 1 + kBlockTokens - 1) / kBlockTokens : 0;
    const bool scored = blocks_end > p.top_k;    // otherwise every row takes all its blocks
    for (int c = warp; scored && c < rows * G; c += kSelWarps)
        query_codes<D>(p, size_t(t + c / G) * p.num_q_heads + size_t(h) * G + c % G, qc[c], &unit[c]);
    __syncthreads();
    if (cs > 1) cluster_wait();
    const uint32_t near0 = smem_u32(near_keys);
    if (scored) {
        const int32_t* table = p.rows.block_tables + size_t(seq) * p.rows.table_stride;
        const int quad = lane >> 2, tig = lane & 3;
        const int step = int(cs) * kSelWarps * kWarpBlocks;
        // this lane's block of the 16 (the upper half of the warp repeats the lower)
        auto block_id = [&](int b) { return b < blocks_end ? table[b] : 0; };
        int b0 = (int(rank) * kSelWarps + warp) * kWarpBlocks;
        int ahead = block_id(b0 + (lane & 15));
        for (; b0 < blocks_end; b0 += step) {
            const int id = ahead;
            ahead = block_id(b0 + step + (lane & 15));
            const bool good = id >= 0 && id < p.num_blocks;
            if (!good && h == 0 && lane < 16) flag_error(p.err, PKV_DEV_BAD_BLOCK_ID);
            const size_t tile = good ? size_t(id) * p.num_kv_heads + h : 0;
            const int e = p.exps[tile];
            uint4 w[2][CH];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const size_t tk = __shfl_sync(kFull, (unsigned long long)tile, quad * 2 + k);
                const uint4* src = reinterpret_cast<const uint4*>(p.bounds + tk * (2 * D)) + tig;
#pragma unroll
                for (int c = 0; c < CH; ++c) w[k][c] = __ldg(src + 4 * c);
            }
            // after the quad's sums: lane tig holds block 2 quad + (tig >> 1)
            const int mine = quad * 2 + (tig >> 1);
            const float eu = pow2(__shfl_sync(kFull, e == kUnbounded ? 0 : e, mine));
            const int em = __shfl_sync(kFull, e, mine);
            const bool gm = __shfl_sync(kFull, int(good), mine);
            const int bm = b0 + mine;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                if (r >= rows) break;
                float best = -INFINITY;
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    int s0 = 0, s1 = 0;
#pragma unroll
                    for (int c = 0; c < CH; ++c) {
                        const uint4 v = *reinterpret_cast<const uint4*>(&qc[r * G + g][c * 16 + tig * 4]);
                        s0 = __dp4a(int(w[0][c].x), int(v.x), s0);
                        s0 = __dp4a(int(w[0][c].y), int(v.y), s0);
                        s0 = __dp4a(int(w[0][c].z), int(v.z), s0);
                        s0 = __dp4a(int(w[0][c].w), int(v.w), s0);
                        s1 = __dp4a(int(w[1][c].x), int(v.x), s1);
                        s1 = __dp4a(int(w[1][c].y), int(v.y), s1);
                        s1 = __dp4a(int(w[1][c].z), int(v.z), s1);
                        s1 = __dp4a(int(w[1][c].w), int(v.w), s1);
                    }
                    const bool up = tig & 2;
                    int sum = up ? s1 : s0;
                    sum += __shfl_xor_sync(kFull, up ? s0 : s1, 2);
                    sum += __shfl_xor_sync(kFull, sum, 1);
                    best = fmaxf(best, float(sum) * unit[r * G + g]);
                }
                const float score = !gm ? -INFINITY : em == kUnbounded ? INFINITY : best * eu;
                if ((tig & 1) == 0 && bm < blocks_end) {
                    if (p.far_keys)
                        p.far_keys[(size_t(t + r) * p.num_kv_heads + h) * p.stride + bm] = ordered(score);
                    else
                        st_cluster(map_rank(near0 + (uint32_t(r) / cs * p.stride + bm) * 4, r % cs),
                                   ordered(score));
                }
            }
        }
    }
    if (cs > 1) cluster_sync();
    else __syncthreads();
    for (int r = int(rank); r < rows; r += int(cs)) {
        const int blocks = keys0 > 0 ? (keys0 + r + kBlockTokens - 1) / kBlockTokens : 0;
        const size_t row = size_t(t + r) * p.num_kv_heads + h;
        int32_t* out = p.selected + row * p.top_k;
        if (blocks <= p.top_k) {
            for (int i = tid; i < p.top_k; i += kSelThreads) out[i] = i < blocks ? i : -1;
        } else {
            pick_row(p, p.far_keys ? p.far_keys + row * p.stride : near_keys + r / int(cs) * p.stride,
                     blocks, out, scratch);
        }
    }
}

size_t select_stride(int32_t max_ctx) {
    return align_up(size_t(ceil_div(max_ctx, kBlockTokens)), 4);
}

// CTAs that share a row group: enough for two on every SM, but 128 blocks each.
int select_cluster(int64_t items, int max_blocks) {
    int cs = 1;
    while (cs < 8 && items * cs < 2 * int64_t(num_sms()) && max_blocks >= 256 * cs) cs *= 2;
    return cs;
}

// Shared memory for the keys of the rows that one CTA picks, 0 if they do not fit.
size_t near_bytes(int rows, int cs, int32_t stride) {
    const size_t b = size_t(ceil_div(rows, cs)) * stride * 4;
    return b <= size_t(kKeyBytes) ? b : 0;
}

template <int D, int G, int R>
int launch_select_r(const SelectParams& p0, int64_t tokens, uint32_t* far_keys, cudaStream_t stream) {
    SelectParams p = p0;
    const int64_t items = tokens * p.num_kv_heads;
    const int cs = select_cluster(ceil_div(items, R), p.stride);
    const size_t smem = near_bytes(R, cs, p.stride);
    p.far_keys = smem ? nullptr : far_keys;
    constexpr auto kern = select_blocks_kernel<D, G, R>;
    if (kernel_occupancy<kern>(kSelThreads, kKeyBytes) < 1) return PKV_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(items * cs));
    cfg.blockDim = dim3(kSelThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = unsigned(cs);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cuda_status(cudaLaunchKernelEx(&cfg, kern, p));
}

// Rows of a sequence share the reads of its bounds, up to eight columns.
template <int D, int G>
int launch_select_g(const SelectParams& p, int64_t tokens, uint32_t* far_keys, cudaStream_t s) {
    return p.rows.start ? launch_select_r<D, G, 8 / G>(p, tokens, far_keys, s)
                        : launch_select_r<D, G, 1>(p, tokens, far_keys, s);
}

template <int D>
int launch_select(const SelectParams& p, int64_t tokens, uint32_t* far_keys, cudaStream_t s) {
    switch (p.num_q_heads / p.num_kv_heads) {
        case 1: return launch_select_g<D, 1>(p, tokens, far_keys, s);
        case 2: return launch_select_g<D, 2>(p, tokens, far_keys, s);
        case 4: return launch_select_g<D, 4>(p, tokens, far_keys, s);
        default: return launch_select_g<D, 8>(p, tokens, far_keys, s);
    }
}

bool aligned_to(const void* p, uintptr_t a) {
    return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

template <typename T, int D>
int launch_bounds(const BoundsParams& p, unsigned ctas, cudaStream_t s) {
    return cuda_status(launch_pdl(block_bounds_kernel<T, D>, dim3(ctas), dim3(kBoundsWarps * 32), 0, s, p));
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" int pkv_block_bounds(int8_t* bounds, int8_t* exps, const void* k_cache,
                                const pkv_cache_desc* desc, const int32_t* block_tables,
                                int32_t max_blocks_per_seq, const int32_t* query_start_loc,
                                const int32_t* context_lens, int32_t num_seqs,
                                int32_t num_query_tokens, void* stream) {
    int st = check_desc(desc, true);
    if (st != PKV_OK) return st;
    if (max_blocks_per_seq < 1 || num_seqs < 0 || num_query_tokens < 0) return PKV_ERR_INVALID;
    if (!query_start_loc && num_query_tokens != num_seqs) return PKV_ERR_INVALID;
    if (num_seqs == 0 || num_query_tokens == 0) return PKV_OK;
    if (!bounds || !exps || !k_cache || !block_tables || !context_lens ||
        !aligned_to(bounds, 16) || !aligned_to(k_cache, 16) || !aligned_to(block_tables, 4) ||
        !aligned_to(query_start_loc, 4) || !aligned_to(context_lens, 4))
        return PKV_ERR_INVALID;
    BoundsParams p;
    p.err = device_error_ptr(&st);
    if (st != PKV_OK) return st;
    p.bounds = bounds;
    p.exps = exps;
    p.k_cache = k_cache;
    p.block_tables = block_tables;
    p.start = query_start_loc;
    p.ctx = context_lens;
    p.table_stride = max_blocks_per_seq;
    p.n = num_seqs;
    p.tokens = num_query_tokens;
    p.num_blocks = desc->num_blocks;
    p.num_kv_heads = desc->num_kv_heads;
    // few tokens: one to a CTA, so that their tiles spread over the GPU; many:
    // a block's worth, of which one or two stand for a block
    p.span = 1;
    while (p.span < kMaxSpan && num_query_tokens / p.span > 4 * num_sms()) p.span *= 2;
    const unsigned ctas = unsigned(ceil_div(num_query_tokens, p.span));
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    if (desc->dtype == PKV_BF16)
        return desc->head_dim == 128 ? launch_bounds<__nv_bfloat16, 128>(p, ctas, cs)
                                     : launch_bounds<__nv_bfloat16, 64>(p, ctas, cs);
    return desc->head_dim == 128 ? launch_bounds<float, 128>(p, ctas, cs)
                                 : launch_bounds<float, 64>(p, ctas, cs);
}

extern "C" size_t pkv_select_workspace_bytes(const pkv_cache_desc* desc, int32_t num_query_tokens,
                                             int32_t max_context_len) {
    if (check_desc(desc, true) != PKV_OK || num_query_tokens < 0 || max_context_len < 1) return 0;
    // keys that fit on chip whatever the cluster need no workspace
    const size_t stride = select_stride(max_context_len);
    if (near_bytes(8, 1, int32_t(stride))) return 256;
    return align_up(size_t(num_query_tokens) * desc->num_kv_heads * stride * sizeof(uint32_t), 256);
}

extern "C" int pkv_select_blocks(int32_t* selected, const void* q, const int8_t* bounds,
                                 const int8_t* exps, const pkv_cache_desc* desc,
                                 const int32_t* block_tables, int32_t max_blocks_per_seq,
                                 const int32_t* query_start_loc, const int32_t* context_lens,
                                 int32_t num_seqs, int32_t num_query_tokens,
                                 int32_t max_context_len, int32_t top_k, int32_t num_sink,
                                 int32_t num_recent, void* workspace, size_t workspace_bytes,
                                 void* stream) {
    int st = check_desc(desc, true);
    if (st != PKV_OK) return st;
    if (max_blocks_per_seq < 1 || max_context_len < 1 || num_seqs < 0 || num_query_tokens < 0 ||
        num_sink < 0 || num_recent < 1 || int64_t(num_sink) + num_recent > top_k)
        return PKV_ERR_INVALID;
    if (!query_start_loc && num_query_tokens != num_seqs) return PKV_ERR_INVALID;
    if (int64_t(num_query_tokens) * desc->num_kv_heads * 8 > INT32_MAX) return PKV_ERR_UNSUPPORTED;
    if (num_seqs == 0 || num_query_tokens == 0) return PKV_OK;
    if (!selected || !q || !bounds || !exps || !block_tables || !context_lens ||
        !aligned_to(selected, 4) || !aligned_to(q, 16) || !aligned_to(bounds, 16) ||
        !aligned_to(block_tables, 4) || !aligned_to(query_start_loc, 4) ||
        !aligned_to(context_lens, 4))
        return PKV_ERR_INVALID;
    const size_t need = pkv_select_workspace_bytes(desc, num_query_tokens, max_context_len);
    if (!workspace || !aligned_to(workspace, 256) || workspace_bytes < need)
        return PKV_ERR_WORKSPACE;
    SelectParams p;
    p.err = device_error_ptr(&st);
    if (st != PKV_OK) return st;
    p.selected = selected;
    p.q = q;
    p.bounds = bounds;
    p.exps = exps;
    p.rows = QueryRows{block_tables, query_start_loc, context_lens, max_blocks_per_seq, num_seqs,
                       max_context_len};
    p.far_keys = nullptr;
    p.stride = int32_t(select_stride(max_context_len));
    p.num_blocks = desc->num_blocks;
    p.num_q_heads = desc->num_q_heads;
    p.num_kv_heads = desc->num_kv_heads;
    p.top_k = top_k;
    p.sink = num_sink;
    p.recent = num_recent;
    p.q_f32 = desc->dtype == PKV_F32;
    uint32_t* far_keys = static_cast<uint32_t*>(workspace);
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    return desc->head_dim == 128 ? launch_select<128>(p, num_query_tokens, far_keys, cs)
                                 : launch_select<64>(p, num_query_tokens, far_keys, cs);
}
