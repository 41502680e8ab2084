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
    float* scores;              // [tokens][Hkv][stride]
    int32_t stride;             // blocks of max_context_len, a multiple of 4
    int32_t num_blocks, num_q_heads, num_kv_heads;
    int32_t top_k, sink, recent;
    int* err;
};

constexpr int kScoreWarps = 8;
constexpr int kWarpBlocks = 32;      // blocks that a warp scores at a time

// Scores of kScoreWarps * 32 blocks for one query row and KV head.  The G query
// heads' codes, positive and negative parts, lie in shared memory; a quad of
// lanes takes four blocks at a time, each lane 64 bytes of their 2 D, and the
// sums run on the packed 8-bit dot product.
template <typename T, int D, int G>
__global__ void __launch_bounds__(kScoreWarps * 32) block_scores_kernel(SelectParams p) {
    constexpr int CH = 2 * D / 64;               // 64-byte chunks of a bounds row
    __shared__ uint32_t qc[G][2 * D / 4];        // codes: positive parts, negative parts
    __shared__ float unit[G];
    const int t = blockIdx.z, h = blockIdx.y;
    pdl_wait_prerequisites();
    pdl_launch_dependents();
    int seq;
    const int keys = row_keys(p.rows, t, seq, nullptr);
    const int blocks = (keys + kBlockTokens - 1) / kBlockTokens;
    // a row whose blocks are all taken needs no scores
    if (keys <= 0 || blocks <= p.top_k || int(blockIdx.x) * kScoreWarps * kWarpBlocks >= blocks)
        return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int b0 = (blockIdx.x * kScoreWarps + warp) * kWarpBlocks;
    int id = -1;
    if (b0 + lane < blocks) id = p.rows.block_tables[size_t(seq) * p.rows.table_stride + b0 + lane];
    const bool good = id >= 0 && id < p.num_blocks;
    const size_t tile = good ? size_t(id) * p.num_kv_heads + h : 0;
    const int e = good ? p.exps[tile] : 0;
    const int quad = lane >> 2, tig = lane & 3;
    uint4 w[4][CH];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int from = quad * 4 + k;
        const size_t tk = __shfl_sync(kFull, (unsigned long long)tile, from);
        const bool ok = __shfl_sync(kFull, int(good), from);
        const uint4* src = reinterpret_cast<const uint4*>(p.bounds + tk * (2 * D)) + tig;
#pragma unroll
        for (int c = 0; c < CH; ++c)
            w[k][c] = ok ? __ldg(src + 4 * c) : make_uint4(0u, 0u, 0u, 0u);
    }
    // codes of the query heads: one warp a head
    for (int g = warp; g < G; g += kScoreWarps) {
        constexpr int PL = D / 32;               // dimensions of a lane: consecutive
        const T* q = static_cast<const T*>(p.q) +
                     (size_t(t) * p.num_q_heads + size_t(h) * G + g) * D + lane * PL;
        float x[PL], amax = 0.f;
        bool odd = false;
#pragma unroll
        for (int j = 0; j < PL; ++j) {
            x[j] = float(q[j]);
            odd |= !(fabsf(x[j]) <= FLT_MAX);
            amax = fmaxf(amax, fabsf(x[j]));
        }
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, o));
        odd = __any_sync(kFull, odd);
        const int eq = code_exponent(amax);
        const float u = pow2(-eq);
        int8_t* pos = reinterpret_cast<int8_t*>(qc[g]) + lane * PL;
#pragma unroll
        for (int j = 0; j < PL; ++j) {
            // (a query with values that are not finite has codes of 0)
            const int c = odd ? 0 : int(fminf(fmaxf(rintf(x[j] * u), -127.f), 127.f));
            pos[j] = int8_t(max(c, 0));
            pos[D + j] = int8_t(min(c, 0));
        }
        if (lane == 0) unit[g] = pow2(eq);
    }
    __syncthreads();
    if (b0 >= blocks) return;
    float best = -INFINITY;
#pragma unroll
    for (int g = 0; g < G; ++g) {
        int s[4] = {0, 0, 0, 0};
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const uint4 qv = *reinterpret_cast<const uint4*>(&qc[g][c * 16 + tig * 4]);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                s[k] = __dp4a(int(w[k][c].x), int(qv.x), s[k]);
                s[k] = __dp4a(int(w[k][c].y), int(qv.y), s[k]);
                s[k] = __dp4a(int(w[k][c].z), int(qv.z), s[k]);
                s[k] = __dp4a(int(w[k][c].w), int(qv.w), s[k]);
            }
        }
        // the quad's four sums of four blocks: lane tig ends with block tig's
        const bool up = tig & 2;
        int a0 = up ? s[2] : s[0], a1 = up ? s[3] : s[1];
        a0 += __shfl_xor_sync(kFull, up ? s[0] : s[2], 2);
        a1 += __shfl_xor_sync(kFull, up ? s[1] : s[3], 2);
        const bool odd = tig & 1;
        int sum = odd ? a1 : a0;
        sum += __shfl_xor_sync(kFull, odd ? a0 : a1, 1);
        best = fmaxf(best, float(sum) * unit[g]);
    }
    const int b = b0 + lane;
    if (b < blocks) {
        const float score = !good ? -INFINITY : e == kUnbounded ? INFINITY : best * pow2(e);
        p.scores[(size_t(t) * p.num_kv_heads + h) * p.stride + b] = score;
    }
}

constexpr int kPickThreads = 256;

// Floats in an order that unsigned compare keeps (no NaN among the scores).
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t b = __float_as_uint(x);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// One CTA for a query row and KV head: the top_k-th largest key by four passes
// over 8-bit digits, then the blocks above it and the first ones equal to it,
// in ascending order.  Blocks that are always taken have a key above all scores.
__global__ void __launch_bounds__(kPickThreads) pick_blocks_kernel(SelectParams p) {
    __shared__ uint32_t hist[256];
    __shared__ uint32_t warp_sum[2][kPickThreads / 32];
    __shared__ uint32_t digit_s, above_s;
    pdl_wait_prerequisites();
    pdl_launch_dependents();
    const int h = blockIdx.x % p.num_kv_heads, t = blockIdx.x / p.num_kv_heads;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int seq;
    const int keys = row_keys(p.rows, t, seq, tid == 0 && h == 0 ? p.err : nullptr);
    if (keys < 0) return;                        // behind the last sequence: left as it is
    const int blocks = (keys + kBlockTokens - 1) / kBlockTokens;
    int32_t* out = p.selected + size_t(blockIdx.x) * p.top_k;
    if (blocks <= p.top_k) {
        for (int i = tid; i < p.top_k; i += kPickThreads) out[i] = i < blocks ? i : -1;
        return;
    }
    if (h == 0) {                                // ids outside the pool score below all others
        for (int b = tid; b < blocks; b += kPickThreads) {
            const int id = p.rows.block_tables[size_t(seq) * p.rows.table_stride + b];
            if (id < 0 || id >= p.num_blocks) flag_error(p.err, PKV_DEV_BAD_BLOCK_ID);
        }
    }
    const float* sc = p.scores + size_t(blockIdx.x) * p.stride;
    auto key_of = [&](int b) {
        return b < p.sink || b >= blocks - p.recent ? 0xffffffffu : ordered(sc[b]);
    };
    uint32_t prefix = 0, want = uint32_t(p.top_k);   // the want-th largest key under the prefix
    for (int shift = 24; shift >= 0; shift -= 8) {
        hist[tid] = 0;
        __syncthreads();
        for (int b = tid; b < blocks; b += kPickThreads) {
            const uint32_t k = key_of(b);
            if (shift == 24 || (k ^ prefix) >> (shift + 8) == 0)
                atomicAdd(&hist[k >> shift & 255u], 1u);
        }
        __syncthreads();
        // keys with a larger digit than tid's: a suffix sum over the 256 bins
        const uint32_t mine = hist[255 - tid];
        uint32_t v = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t u = __shfl_up_sync(kFull, v, o);
            if (lane >= o) v += u;
        }
        if (lane == 31) warp_sum[0][warp] = v;
        __syncthreads();
        for (int w = 0; w < warp; ++w) v += warp_sum[0][w];
        if (v >= want && v - mine < want) {      // exactly one bin
            digit_s = uint32_t(255 - tid);
            above_s = v - mine;
        }
        __syncthreads();
        prefix |= digit_s << shift;
        want -= above_s;
        __syncthreads();
    }
    // keys above `prefix` are all taken, and the first `want` equal to it
    uint32_t n_gt = 0, n_eq = 0;
    for (int base = 0; base < blocks; base += kPickThreads) {
        const int b = base + tid;
        const uint32_t k = b < blocks ? key_of(b) : 0u;
        const bool gt = b < blocks && k > prefix, eq = b < blocks && k == prefix;
        const uint32_t mg = __ballot_sync(kFull, gt), me = __ballot_sync(kFull, eq);
        if (lane == 0) {
            warp_sum[0][warp] = __popc(mg);
            warp_sum[1][warp] = __popc(me);
        }
        __syncthreads();
        uint32_t g0 = n_gt, e0 = n_eq;
        for (int w = 0; w < kPickThreads / 32; ++w) {
            if (w < warp) g0 += warp_sum[0][w], e0 += warp_sum[1][w];
            n_gt += warp_sum[0][w];
            n_eq += warp_sum[1][w];
        }
        const uint32_t below = (1u << lane) - 1u;
        g0 += __popc(mg & below);
        e0 += __popc(me & below);
        // place = taken blocks in front of b
        if (gt || (eq && e0 < want)) out[g0 + min(e0, want)] = b;
        __syncthreads();
    }
}

size_t select_stride(int32_t max_ctx) {
    return align_up(size_t(ceil_div(max_ctx, kBlockTokens)), 4);
}

template <typename T, int D, int G>
int launch_scores(const SelectParams& p, dim3 grid, cudaStream_t s) {
    return cuda_status(launch_pdl(block_scores_kernel<T, D, G>, grid, dim3(kScoreWarps * 32), 0, s, p));
}

template <typename T, int D>
int launch_scores_g(const SelectParams& p, dim3 grid, cudaStream_t s) {
    switch (p.num_q_heads / p.num_kv_heads) {
        case 1: return launch_scores<T, D, 1>(p, grid, s);
        case 2: return launch_scores<T, D, 2>(p, grid, s);
        case 4: return launch_scores<T, D, 4>(p, grid, s);
        default: return launch_scores<T, D, 8>(p, grid, s);
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
    return align_up(size_t(num_query_tokens) * desc->num_kv_heads * select_stride(max_context_len) *
                        sizeof(float),
                    256);
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
    if (num_query_tokens > 65535 || desc->num_kv_heads > 65535) return PKV_ERR_UNSUPPORTED;
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
    p.scores = static_cast<float*>(workspace);
    p.stride = int32_t(select_stride(max_context_len));
    p.num_blocks = desc->num_blocks;
    p.num_q_heads = desc->num_q_heads;
    p.num_kv_heads = desc->num_kv_heads;
    p.top_k = top_k;
    p.sink = num_sink;
    p.recent = num_recent;
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    const int max_blocks = ceil_div(max_context_len, kBlockTokens);
    if (max_blocks > top_k) {
        const dim3 grid(unsigned(ceil_div(max_blocks, kScoreWarps * kWarpBlocks)),
                        unsigned(desc->num_kv_heads), unsigned(num_query_tokens));
        if (desc->dtype == PKV_BF16)
            st = desc->head_dim == 128 ? launch_scores_g<__nv_bfloat16, 128>(p, grid, cs)
                                       : launch_scores_g<__nv_bfloat16, 64>(p, grid, cs);
        else
            st = desc->head_dim == 128 ? launch_scores_g<float, 128>(p, grid, cs)
                                       : launch_scores_g<float, 64>(p, grid, cs);
        if (st != PKV_OK) return st;
    }
    return cuda_status(launch_pdl(pick_blocks_kernel,
                                  dim3(unsigned(num_query_tokens) * unsigned(desc->num_kv_heads)),
                                  dim3(kPickThreads), 0, cs, p));
}
