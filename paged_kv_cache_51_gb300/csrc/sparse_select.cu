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
#include <cuda_fp16.h>
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
    int span;                   // tokens that one warp looks at
    int work_ctas;              // the CTAs behind these look over the offsets
    int* err;
};

constexpr int kBoundsWarps = 4;

// Largest and smallest of 16 bytes of values each, element by element; NaN if
// either is.
template <typename T>
struct Extent;
template <>
struct Extent<float> {
    static constexpr int V = 4;
    float hi[4], lo[4];
    __device__ __forceinline__ static float max_nan(float a, float b) {
        float r;
        asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
        return r;
    }
    __device__ __forceinline__ void start(uint4 v) {
        hi[0] = lo[0] = __uint_as_float(v.x);
        hi[1] = lo[1] = __uint_as_float(v.y);
        hi[2] = lo[2] = __uint_as_float(v.z);
        hi[3] = lo[3] = __uint_as_float(v.w);
    }
    __device__ __forceinline__ void add(const float (&h)[4], const float (&l)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            hi[i] = max_nan(hi[i], h[i]);
            lo[i] = -max_nan(-lo[i], -l[i]);
        }
    }
    __device__ __forceinline__ void add(uint4 v) {
        const float x[4] = {__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z),
                            __uint_as_float(v.w)};
        add(x, x);
    }
    __device__ __forceinline__ void fold(int lanes) {
        float h[4], l[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            h[i] = __shfl_xor_sync(kFull, hi[i], lanes);
            l[i] = __shfl_xor_sync(kFull, lo[i], lanes);
        }
        add(h, l);
    }
    __device__ __forceinline__ float top(int i) const { return hi[i]; }
    __device__ __forceinline__ float low(int i) const { return lo[i]; }
};
template <>
struct Extent<__nv_bfloat16> {
    static constexpr int V = 8;
    __nv_bfloat162 hi[4], lo[4];                 // two values at a time
    __device__ __forceinline__ static __nv_bfloat162 two(uint32_t w) {
        return *reinterpret_cast<const __nv_bfloat162*>(&w);
    }
    __device__ __forceinline__ void start(uint4 v) {
        hi[0] = lo[0] = two(v.x);
        hi[1] = lo[1] = two(v.y);
        hi[2] = lo[2] = two(v.z);
        hi[3] = lo[3] = two(v.w);
    }
    __device__ __forceinline__ void add(uint4 v) {
        const __nv_bfloat162 x[4] = {two(v.x), two(v.y), two(v.z), two(v.w)};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            hi[i] = __hmax2_nan(hi[i], x[i]);
            lo[i] = __hmin2_nan(lo[i], x[i]);
        }
    }
    __device__ __forceinline__ void fold(int lanes) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            hi[i] = __hmax2_nan(hi[i], __shfl_xor_sync(kFull, hi[i], lanes));
            lo[i] = __hmin2_nan(lo[i], __shfl_xor_sync(kFull, lo[i], lanes));
        }
    }
    __device__ __forceinline__ static float part(__nv_bfloat162 v, int i) {
        return i & 1 ? __high2float(v) : __low2float(v);
    }
    __device__ __forceinline__ float top(int i) const { return part(hi[i / 2], i); }
    __device__ __forceinline__ float low(int i) const { return part(lo[i / 2], i); }
};

// A warp looks at `span` query tokens for one KV head; a token that is the first
// of its sequence in the step, or the first row of its block, stands for that
// block.  For each block found the warp reads the rows that hold tokens, all of
// them asked for at once, keeps the largest and the smallest value of each
// dimension, and writes codes rounded outwards, half the warp the upper ends and
// half the lower.  One pass over the keys: bound by the chain of lookups in front of
// the tile, which prompts pay in one wave of warps.  Device time of a call: one token
// each of 64 sequences, 32 heads (5 MB, 9 MB in fp32) 3.2 us, 3.5 in fp32; 15000
// prompt tokens, 8 heads (33 MB, 64 MB) 8.2 us, 4.0 TB/s, and 16.2 us, 3.9 TB/s.
template <typename T, int D>
__global__ void __launch_bounds__(kBoundsWarps * 32) block_bounds_kernel(BoundsParams p) {
    constexpr int V = Extent<T>::V;              // elements of a 16-byte load
    constexpr int LPR = D / V;                   // lanes of a row
    constexpr int RPI = 32 / LPR;                // rows of a load
    const int lane = threadIdx.x & 31;
    pdl_wait_prerequisites();
    pdl_launch_dependents();
    const uint32_t unit = blockIdx.x * kBoundsWarps + (threadIdx.x >> 5);
    const int h = int(unit % uint32_t(p.num_kv_heads));
    const int64_t t0 = int64_t(unit / uint32_t(p.num_kv_heads)) * p.span;
    if (int(blockIdx.x) >= p.work_ctas) {        // (beside the work these would delay its lookups)
        const int64_t width = kBoundsWarps * 32;
        check_offsets(p.start, p.n, (blockIdx.x - p.work_ctas) * width + threadIdx.x,
                      (gridDim.x - p.work_ctas) * width, p.err);
        return;
    }
    if (t0 >= p.tokens) return;
    int* const tell = h == 0 ? p.err : nullptr;
    int first, q, id = -1, nrow = 0;
    int s = token_seq(p.start, p.n, p.tokens, int(t0), first, q, lane == 0 ? tell : nullptr);
    const int64_t t = t0 + lane;
    if (lane < p.span && t < p.tokens && s >= 0) {
        // the lane's own token: a later sequence than the first token's, perhaps
        while (t >= int64_t(first) + q && s + 1 < p.n) {
            ++s;
            first = p.start[s];
            q = p.start[s + 1] - first;
        }
        if (t >= first && t < int64_t(first) + q) {
            const int ctx = p.ctx[s];
            const int pos = ctx - q + int(t - first);
            if (ctx < q) {
                if (t == first) flag_error(tell, PKV_DEV_BAD_CONTEXT_LEN);
            } else if (t == first || pos % kBlockTokens == 0) {
                const int b = pos / kBlockTokens;
                if (b >= p.table_stride) {
                    flag_error(tell, PKV_DEV_TABLE_TOO_NARROW);
                } else {
                    id = p.block_tables[size_t(s) * p.table_stride + b];
                    nrow = min(kBlockTokens, ctx - b * kBlockTokens);
                    if (id < 0 || id >= p.num_blocks) {
                        flag_error(tell, PKV_DEV_BAD_BLOCK_ID);
                        nrow = 0;
                    }
                }
            }
        }
    }
    for (uint32_t found = __ballot_sync(kFull, nrow > 0); found; found &= found - 1) {
        const int from = __ffs(found) - 1;
        const int rows = __shfl_sync(kFull, nrow, from);
        const size_t tile = size_t(__shfl_sync(kFull, id, from)) * p.num_kv_heads + h;
        const uint4* k = reinterpret_cast<const uint4*>(static_cast<const T*>(p.k_cache) +
                                                        tile * (kBlockTokens * D)) + lane;
        uint4 x[kBlockTokens / RPI];
#pragma unroll
        for (int i = 0; i < kBlockTokens / RPI; ++i) {
            // (a lane whose row holds no token repeats row 0)
            const bool in = i * RPI + lane / LPR < rows;
            x[i] = __ldg(k + (in ? i * 32 : -(lane / LPR) * LPR));
        }
        Extent<T> ex;
        ex.start(x[0]);
#pragma unroll
        for (int i = 1; i < kBlockTokens / RPI; ++i) ex.add(x[i]);
#pragma unroll
        for (int o = LPR; o < 32; o <<= 1) ex.fold(o);
        float amax = 0.f;
        bool odd = false;                        // a value that is not finite
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float a = fmaxf(fabsf(ex.top(j)), fabsf(ex.low(j)));
            odd |= !(fabsf(ex.top(j)) <= FLT_MAX) || !(fabsf(ex.low(j)) <= FLT_MAX);
            amax = fmaxf(amax, a);
        }
        // (the bits of values that are not negative order as the values do)
        amax = __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(amax)));
        odd = __any_sync(kFull, odd);
        const int e = code_exponent(amax);
        const float unit_inv = pow2(-e);
        int8_t* dst = p.bounds + tile * (2 * D) + (lane % LPR) * V;
        auto write = [&](bool lower) {           // floor(x) = -ceil(-x)
            uint32_t w[V / 4];
#pragma unroll
            for (int j = 0; j < V; j += 4) {
                w[j / 4] = 0u;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float y = lower ? -ex.low(j + i) : ex.top(j + i);
                    // (a product too small for its type is rounded up too: to 1, if positive)
                    const float x = ceilf(__fmul_ru(y, unit_inv));
                    const int c = int(fminf(fmaxf(x, -127.f), 127.f));
                    w[j / 4] |= uint32_t((lower ? -c : c) & 0xff) << (8 * i);
                }
                if (odd) w[j / 4] = 0u;          // (such a block has codes of 0)
            }
            if constexpr (V == 8) *reinterpret_cast<uint2*>(dst + lower * D) = make_uint2(w[0], w[1]);
            else *reinterpret_cast<uint32_t*>(dst + lower * D) = w[0];
        };
        if (RPI > 1) {
            if (lane < 2 * LPR) write(lane >= LPR);
        } else {
            write(false);
            write(true);
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
    uint32_t* keys;             // [tokens][Hkv][stride]: scores in an order unsigned compare keeps
    int32_t stride;             // blocks of max_context_len, a multiple of 4
    int32_t tokens, num_blocks, num_q_heads, num_kv_heads;
    int32_t top_k, sink, recent;
    int32_t q_f32;              // q is fp32, else bf16
    // tiles that one warp scores, and CTAs of a query row: of the first rows, and of
    // the others, which begin at `fine_row` and at CTA `fine_cta`
    int32_t chunk_tiles, row_ctas, fine_tiles, fine_ctas, fine_row, fine_cta;
    int* err;
};

constexpr int kScoreWarps = 4;
constexpr int kTileBlocks = 16;      // blocks of a product tile
constexpr int kScoreStages = 2;      // tiles in flight per warp

// Floats in an order that unsigned compare keeps (no NaN among the scores), and the
// ends of that order, -inf and inf.
constexpr uint32_t kLeastKey = 0x007fffffu, kMostKey = 0xff800000u;
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t b = __float_as_uint(x);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// Four 8-bit codes as two pairs of halves, bytes 0 and 2 and bytes 1 and 3, each
// raised by kBias: a code with its sign bit flipped, below the byte 0x64, is the
// half 1024 + 128 + code.
constexpr float kBias = 1152.f;
__device__ __forceinline__ void raise_codes(uint32_t w, uint32_t& even, uint32_t& odd) {
    even = (w & 0x00ff00ffu) ^ 0x64806480u;
    odd = (w >> 8 & 0x00ff00ffu) ^ 0x64806480u;
}

__device__ __forceinline__ uint32_t bits(__half2 v) { return *reinterpret_cast<const uint32_t*>(&v); }

// d = c + a . b, the sums of two columns starting from c0 and c1
__device__ __forceinline__ void mma16816_f16(float (&d)[4], float c0, float c1, float c2, float c3,
                                             const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2),
          "f"(c3));
}

// Sixteen consecutive values of a query head.
__device__ __forceinline__ void load16(const SelectParams& p, size_t at, float (&x)[16]) {
    if (p.q_f32) {
        const float4* s = reinterpret_cast<const float4*>(static_cast<const float*>(p.q) + at);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 v = __ldg(s + i);
            x[4 * i] = v.x; x[4 * i + 1] = v.y; x[4 * i + 2] = v.z; x[4 * i + 3] = v.w;
        }
    } else {
        const uint4* s = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) + at);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint4 v = __ldg(s + i);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                x[8 * i + 2 * k] = __uint_as_float(w[k] << 16);
                x[8 * i + 2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
            }
        }
    }
}

// Keys of the blocks of up to R neighbouring query rows of one sequence for one
// KV head.  The rows' R * G <= 8 query heads are the columns of a product whose
// rows are blocks: scores = bounds (16 blocks x 2 D) . codes (2 D x 8), on
// m16n8k16 half-precision products with single-precision sums, in which whole
// numbers below 2^24 stay exact.  (The packed 8-bit dot product and the 8-bit
// tensor products run at a quarter of that rate on this GPU: 491 against 1915
// multiply-adds per ns and SM.)  The bounds enter raised by 1152, which three
// instructions on four packed codes do, and each 64-byte chunk's sum starts from
// -1152 times the chunk's codes: all sums of a chunk stay below
// 64 * 127 * 1279 < 2^24.
//
// Every warp works alone on a chunk of a row's tiles: it makes the codes in the
// registers that the product takes them from, and every lane copies the bounds
// that it will use itself (two rows' 16 bytes of each 64) into places of its own
// in shared memory, a tile ahead.  Nothing waits for another lane or warp,
// and the SM's other warps hide the start of each (context, ids, bounds: three
// dependent loads).  256 rows of 64 to 512 blocks, 8 heads (152 MB of bounds): 29 us
// of the call's 35, where a copy of the same rows alone takes 26; bound by HBM's rate
// for gathered 256-byte rows and by the start and the end of the launch.
template <int D, int G, int R>
__global__ void __launch_bounds__(kScoreWarps * 32, 4) block_scores_kernel(SelectParams p) {
    __shared__ __align__(128) uint4 ring_all[kScoreWarps][kScoreStages][2 * D / 32][32];
    constexpr int CH = 2 * D / 64;               // 64-byte chunks: four product steps each
    constexpr int NP = D / 64;                   // ... of which the first half meet positive parts
    constexpr int LR = G > 2 ? G / 2 : 1;        // lanes of a quad that hold a row's columns
    constexpr int NR = G == 1 ? 2 : 1;           // rows of a lane's two columns
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int gid = lane >> 2, tig = lane & 3;
    pdl_wait_prerequisites();
    pdl_launch_dependents();
    // neighbouring warps take neighbouring heads: their bounds lie side by side
    const bool fine = int(blockIdx.x) >= p.fine_cta;
    const int chunk_tiles = fine ? p.fine_tiles : p.chunk_tiles;
    const uint32_t cta = blockIdx.x - (fine ? p.fine_cta : 0);
    const uint32_t ctas = fine ? p.fine_ctas : p.row_ctas;
    const int t = int(cta / ctas) + (fine ? p.fine_row : 0);
    const uint32_t unit = cta % ctas * kScoreWarps + warp;
    const int chunk = int(unit / uint32_t(p.num_kv_heads));
    const int h = int(unit % uint32_t(p.num_kv_heads));
    int first, q;
    const int seq = token_seq(p.rows.start, p.rows.n, p.tokens, t, first, q, nullptr);
    // (the sequence's rows are rows of the call, so the group's are)
    const int rows = seq < 0 || (t - first) % R ? 0 : min(R, first + q - t);
    if (rows == 0) return;                       // another warp's row, or behind the last one
    // asked for at once, before the context is known: the first tile's ids and
    // the values of this lane's query head (column gid)
    const int32_t* table = p.rows.block_tables + size_t(seq) * p.rows.table_stride;
    const int base = chunk * chunk_tiles * kTileBlocks;
    const int last = p.rows.table_stride - 1;
    int id0 = table[min(base + gid, last)], id1 = table[min(base + gid + 8, last)];
    float x[NP][16];
    const bool column = gid < rows * G;
    if (column) {
        const size_t head = size_t(t + gid / G) * p.num_q_heads + size_t(h) * G + gid % G;
#pragma unroll
        for (int c = 0; c < NP; ++c) load16(p, head * D + c * 64 + tig * 16, x[c]);
    }
    if (!sequence_keys(p.rows, seq, q, nullptr)) return;
    const int keys_end = p.rows.ctx[seq] - q + (t - first) + rows;
    const int blocks = (keys_end + kBlockTokens - 1) / kBlockTokens;
    // (a row whose blocks are all taken needs no scores)
    if (blocks <= p.top_k || base >= blocks) return;
    const int end = min(blocks, base + chunk_tiles * kTileBlocks);

    // this lane's two rows of a tile are blocks gid and gid + 8
    constexpr int kBadId = 1000;                 // exponent of an id outside the pool
    uint4* ring = &ring_all[warp][0][0][lane];
    const uint32_t ring_u = smem_u32(ring);
    int e0[kScoreStages], e1[kScoreStages];
    const int8_t* bounds_h = p.bounds + h * (2 * D) + tig * 16;
    const int8_t* exps_h = p.exps + h;
    const int bounds_step = p.num_kv_heads * (2 * D);
    auto request = [&](int b, int js) {          // the tile at block b, into stage js
        if (b < end) {
            const bool good0 = uint32_t(id0) < uint32_t(p.num_blocks);
            const bool good1 = uint32_t(id1) < uint32_t(p.num_blocks);
            const int at0 = good0 ? id0 : 0, at1 = good1 ? id1 : 0;
            const int8_t* src0 = bounds_h + int64_t(at0) * bounds_step;
            const int8_t* src1 = bounds_h + int64_t(at1) * bounds_step;
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                cp_async16(ring_u + (js * 2 * CH + 2 * c) * 512, src0 + 64 * c, true);
                cp_async16(ring_u + (js * 2 * CH + 2 * c + 1) * 512, src1 + 64 * c, true);
            }
            e0[js] = exps_h[int64_t(at0) * p.num_kv_heads];
            e1[js] = exps_h[int64_t(at1) * p.num_kv_heads];
            if (!good0 || !good1) {
                if ((!good0 && b + gid < end) || (!good1 && b + gid + 8 < end))
                    if (h == 0) flag_error(p.err, PKV_DEV_BAD_BLOCK_ID);
                if (!good0) e0[js] = kBadId;
                if (!good1) e1[js] = kBadId;
            }
            // (entries behind the row's blocks may hold anything: clamped, then not used)
            id0 = table[min(b + kTileBlocks + gid, end - 1)];
            id1 = table[min(b + kTileBlocks + gid + 8, end - 1)];
        }
        cp_commit();
    };
    if (base + gid >= end) id0 = 0;
    if (base + gid + 8 >= end) id1 = 0;
#pragma unroll
    for (int js = 0; js < kScoreStages - 1; ++js) request(base + js * kTileBlocks, js);

    // codes of column gid as the product's second operand, in the order in which
    // the bounds are read: of each 64-byte chunk this lane's 16 dimensions
    uint32_t bq[CH][4][2];
    float unit_q, start[CH][2];
    {
        float amax = 0.f;
        bool odd = false;
#pragma unroll
        for (int c = 0; c < NP; ++c)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                if (!column) x[c][i] = 0.f;
                odd |= !(fabsf(x[c][i]) <= FLT_MAX);
                amax = fmaxf(amax, fabsf(x[c][i]));
            }
        odd = __ballot_sync(kFull, odd) >> (lane & 28) & 15u;
        amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 2));
        const int eq = code_exponent(amax);
        const float u = pow2(-eq);
        unit_q = odd ? 0.f : pow2(eq);
        if (odd || eq == 50) {                   // (rare, and the only values past 127 units)
#pragma unroll
            for (int c = 0; c < NP; ++c)
#pragma unroll
                for (int i = 0; i < 16; ++i)     // a query that is not finite has codes of 0
                    x[c][i] = odd ? 0.f : fminf(fmaxf(x[c][i], -127.f * pow2(50)), 127.f * pow2(50));
        }
#pragma unroll
        for (int c = 0; c < NP; ++c) {
            // x / 2^eq to the nearest whole number, ties to even: added to 1.5 * 2^23
            // it is rounded there
            constexpr float kRound = 12582912.f;
            float sum = 0.f, size = 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                x[c][i] = __fsub_rn(__fmaf_rn(x[c][i], u, kRound), kRound);
                sum += x[c][i];
                size += fabsf(x[c][i]);
            }
            const __half2 zero = __float2half2_rn(0.f);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int k = 0; k < 2; ++k) {    // bytes 0 and 2, then 1 and 3
                    const __half2 v = __floats2half2_rn(x[c][4 * i + k], x[c][4 * i + k + 2]);
                    bq[c][i][k] = bits(__hmax2(v, zero));
                    bq[NP + c][i][k] = bits(__hmin2(v, zero));
                }
            float up = 0.5f * (size + sum), down = 0.5f * (sum - size);   // whole numbers: exact
            up += __shfl_xor_sync(kFull, up, 1);
            up += __shfl_xor_sync(kFull, up, 2);
            down += __shfl_xor_sync(kFull, down, 1);
            down += __shfl_xor_sync(kFull, down, 2);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                start[c][k] = -kBias * __shfl_sync(kFull, up, 8 * tig + 4 * k);
                start[NP + c][k] = -kBias * __shfl_sync(kFull, down, 8 * tig + 4 * k);
            }
        }
    }
    const float u0 = __shfl_sync(kFull, unit_q, 8 * tig), u1 = __shfl_sync(kFull, unit_q, 8 * tig + 4);
    uint32_t* out[NR];
    bool mine[NR];
#pragma unroll
    for (int n = 0; n < NR; ++n) {
        const int r = (2 * tig + n) / G;
        mine[n] = r < rows;
        out[n] = p.keys + (size_t(t + (mine[n] ? r : 0)) * p.num_kv_heads + h) * p.stride;
    }
    for (int tile = base; tile < end; tile += kScoreStages * kTileBlocks) {
#pragma unroll
        for (int js = 0; js < kScoreStages; ++js) {
            const int b0 = tile + js * kTileBlocks;
            if (b0 >= end) break;
            request(b0 + (kScoreStages - 1) * kTileBlocks, (js + kScoreStages - 1) % kScoreStages);
            cp_wait<kScoreStages - 1>();
            float d[CH][4];
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const uint4 v = ring[(js * 2 * CH + 2 * c) * 32];
                const uint4 w = ring[(js * 2 * CH + 2 * c + 1) * 32];
                const uint32_t vw[4] = {v.x, v.y, v.z, v.w}, ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    uint32_t a[4];
                    raise_codes(vw[k], a[0], a[2]);
                    raise_codes(ww[k], a[1], a[3]);
                    if (k == 0)
                        mma16816_f16(d[c], start[c][0], start[c][1], start[c][0], start[c][1], a,
                                     bq[c][k][0], bq[c][k][1]);
                    else
                        mma16816_f16(d[c], d[c][0], d[c][1], d[c][2], d[c][3], a, bq[c][k][0],
                                     bq[c][k][1]);
                }
            }
            // this lane: blocks gid and gid + 8, columns 2 tig and 2 tig + 1
            float s[2][NR];
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                float x0 = d[0][2 * half], x1 = d[0][2 * half + 1];
#pragma unroll
                for (int c = 1; c < CH; ++c) x0 += d[c][2 * half], x1 += d[c][2 * half + 1];
                s[half][0] = x0 * u0;
                if (NR == 2) s[half][NR - 1] = x1 * u1;
                else s[half][0] = fmaxf(s[half][0], x1 * u1);
                if (G > 4) s[half][0] = fmaxf(s[half][0], __shfl_xor_sync(kFull, s[half][0], 2));
            }
            int e = e0[js], f = e1[js], b = b0 + gid;
            bool writes0 = true, writes1 = LR == 1;
            if (LR > 1) {                        // a block each for lanes that share a row's columns
                const bool up = tig & 1;
                const float mine_s = up ? s[1][0] : s[0][0], other = up ? s[0][0] : s[1][0];
                s[0][0] = fmaxf(mine_s, __shfl_xor_sync(kFull, other, 1));
                if (up) e = f, b += 8;
                writes0 = tig % LR < 2;
            }
            auto put = [&](int at, int ex, const float (&sc)[NR]) {
                float x[NR];
#pragma unroll
                for (int n = 0; n < NR; ++n) x[n] = sc[n] * pow2(ex);
                if (ex > 50 || ex < -126) {      // (an exponent that no bounds call writes: any value)
#pragma unroll
                    for (int n = 0; n < NR; ++n)
                        x[n] = ex == kBadId ? -INFINITY : ex == kUnbounded ? INFINITY : 0.f;
                }
#pragma unroll
                for (int n = 0; n < NR; ++n)
                    if (mine[n]) out[n][at] = ordered(x[n] + 0.f);   // (one zero, not two)
            };
            if (writes0 && b < end) put(b, e, s[0]);
            if (writes1 && b + 8 < end) put(b + 8, f, s[1]);
        }
    }
    cp_wait<0>();
}

// ---- the lists ------------------------------------------------------------------

template <int NT>
struct PickScratch {
    static constexpr int kWarps = NT / 32;
    static constexpr int kBins = 4 * NT;
    uint32_t hist[kBins];
    uint4 cand[16];                              // two (key, block) of the last bin in each
    uint32_t warp_a[kWarps], warp_b[kWarps];
    uint32_t bin, above, inside, count;
};

// Sums of a value over the warps in front of this one (the same for a warp's
// lanes, and written to `of_warps` by all of them before a barrier).
__device__ __forceinline__ uint32_t warps_before(const uint32_t* of_warps) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    return __reduce_add_sync(kFull, lane < warp ? of_warps[lane] : 0u);
}

// One CTA of NT threads for the list of a (query row, KV head).  Wanted are the
// `want` largest keys of blocks sink .. blocks - recent - 1 (the ends are always
// taken).  A histogram over the keys' range finds the bin that holds the want-th.
// Its few keys are ranked by every warp for itself, with the lower index first
// among equals, and where each warp's part of the list begins follows from the
// same ranks: one barrier between the histogram and the list.  While the bin holds
// more keys than a warp ranks at once it becomes the next range.  Scores of a real
// query spread over the bins, so one histogram and one ranking is the rule.  A
// row's keys stay in registers, kHeld to a thread, asked for before the row's
// context is known; with kHeld 0 (rows longer than that) every pass reads them
// again.  Keys of real blocks lie between those of the two infinities; the ends
// carry a key above all and places behind the row one below all, so that no pass
// has to look at indices.  (They are held to that: where the offsets of the batch are
// out of order a row may find keys that no warp wrote, and the counts below are
// those of the list only while every block's key is between the ends.)  2048 rows of
// up to 512 blocks: 5.5 us behind the scores, of which 2.4 start the CTAs and 2.0 rank
// and write; 32 rows of 2048: 2.9 us, a chain of barriers.
template <int NT, int kHeld>
__global__ void __launch_bounds__(NT) pick_blocks_kernel(SelectParams p) {
    using S = PickScratch<NT>;
    constexpr bool Held = kHeld > 0;
    constexpr uint32_t kEnd = 0xffffffffu, kNone = 0u;
    __shared__ __align__(16) S s;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
#pragma unroll
    for (int i = 0; i < 4; ++i) s.hist[i * NT + tid] = 0;
    if (tid < 16) s.cand[tid] = make_uint4(0u, 0u, 0u, 0u);
    if (tid == 0) s.count = 0;
    const int h = int(blockIdx.x % uint32_t(p.num_kv_heads));
    const int t = int(blockIdx.x / uint32_t(p.num_kv_heads));
    const uint32_t* far = p.keys + size_t(blockIdx.x) * p.stride;
    pdl_wait_prerequisites();
    pdl_launch_dependents();
    const int mine = warp * 32 * kHeld + lane;
    uint32_t held[Held ? kHeld : 1];
    if (Held) {
#pragma unroll
        for (int i = 0; i < kHeld; ++i)
            held[i] = mine + 32 * i < p.stride ? far[mine + 32 * i] : kNone;
    }
    const OffsetStep step(p.rows.start, p.rows.n);
    int seq;
    const int row_sees = row_keys(p.rows, t, seq, tid == 0 && h == 0 ? p.err : nullptr);
    step.check(p.err);
    if (row_sees < 0) return;                    // behind the last sequence: left as it is
    const int blocks = (row_sees + kBlockTokens - 1) / kBlockTokens;
    int32_t* out = p.selected + size_t(blockIdx.x) * p.top_k;
    if (blocks <= p.top_k) {
        for (int i = tid; i < p.top_k; i += NT) out[i] = i < blocks ? i : -1;
        return;
    }
    const int b0 = p.sink, b1 = blocks - p.recent;
    auto between = [](uint32_t k) { return min(max(k, kLeastKey), kMostKey); };
    auto marked = [&](int b, uint32_t k) {
        return b >= blocks ? kNone : b < b0 || b >= b1 ? kEnd : k;
    };
    if (Held) {
        if (p.rows.start) {
#pragma unroll
            for (int i = 0; i < kHeld; ++i) held[i] = between(held[i]);
        }
#pragma unroll
        for (int i = 0; i < kHeld; ++i) held[i] = marked(mine + 32 * i, held[i]);
    }
    auto each = [&](auto f) {                    // f(key) for each of this thread's keys
        if (Held) {
#pragma unroll
            for (int i = 0; i < kHeld; ++i) f(held[i]);
        } else {
            for (int b = b0 + tid; b < b1; b += NT) f(between(far[b]));
        }
    };
    // this warp's stretch of the row (ascending with the warps), 32 blocks at a time
    const int stretch = Held ? 32 * kHeld : ((blocks + S::kWarps - 1) / S::kWarps + 31) & ~31;
    auto in_order = [&](auto f) {                // f(block, key)
        if (Held) {
#pragma unroll
            for (int i = 0; i < kHeld; ++i) f(mine + 32 * i, held[i]);
        } else {
            const int end = min(blocks, (warp + 1) * stretch);
            for (int b = warp * stretch + lane; b - lane < end; b += 32)
                f(b, b < end ? marked(b, between(far[b])) : kNone);
        }
    };
    const uint32_t below = (1u << lane) - 1u;
    uint32_t want = uint32_t(p.top_k - p.sink - p.recent);
    uint32_t cut = kEnd - 1, take = 0;           // taken: keys above `cut`, `take` equal to it
    if (want > 0) {
        uint32_t lo = 0xffffffffu, hi = 0;
        each([&](uint32_t k) {
            lo = min(lo, k - 1);                 // (kNone wraps to the top)
            hi = max(hi, k + 1);                 // (kEnd wraps to 0)
        });
        lo = __reduce_min_sync(kFull, lo);
        hi = __reduce_max_sync(kFull, hi);
        if (lane == 0) s.warp_a[warp] = lo, s.warp_b[warp] = hi;
        __syncthreads();
        lo = __reduce_min_sync(kFull, s.warp_a[lane % S::kWarps]) + 1;
        hi = __reduce_max_sync(kFull, s.warp_b[lane % S::kWarps]) - 1;
        for (;;) {                               // the range lo .. hi holds the want-th
            if (lo == hi) {                      // equal keys (a query of zeros): the lower indices
                cut = lo;
                take = want;
                break;
            }
            const int shift = max(0, 32 - __clz(hi - lo) - (31 - __clz(S::kBins)));
            each([&](uint32_t k) {
                if (k - lo <= hi - lo) atomicAdd(&s.hist[(k - lo) >> shift], 1u);
            });
            __syncthreads();
            // bins from above, four to a thread
            const uint4 c = *reinterpret_cast<const uint4*>(&s.hist[S::kBins - 4 - 4 * tid]);
            const uint32_t four[4] = {c.w, c.z, c.y, c.x};
            const uint32_t own = c.x + c.y + c.z + c.w;
            uint32_t sum = own;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t u = __shfl_up_sync(kFull, sum, o);
                if (lane >= o) sum += u;
            }
            if (lane == 31) s.warp_a[warp] = sum;
            __syncthreads();
            sum += warps_before(s.warp_a) - own;
            if (sum < want && want <= sum + own) {   // exactly one thread
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (sum < want && want <= sum + four[i]) {
                        s.bin = uint32_t(S::kBins - 1 - 4 * tid - i);
                        s.above = sum;
                        s.inside = four[i];
                    }
                    sum += four[i];
                }
            }
            __syncthreads();
            const uint32_t inside = s.inside;
            want -= s.above;
            const uint32_t first = lo + (s.bin << shift);
            const uint32_t last = min(hi, first + ((1u << shift) - 1u));
            if (inside <= 32) {
                uint32_t n = 0;
                in_order([&](int b, uint32_t k) {
                    n += __popc(__ballot_sync(kFull, k > last));
                    if (k - first <= last - first)
                        reinterpret_cast<uint2*>(s.cand)[atomicAdd(&s.count, 1u)] =
                            make_uint2(k, uint32_t(b));
                });
                if (lane == 0) s.warp_a[warp] = n;
                __syncthreads();
                const uint2 c = reinterpret_cast<const uint2*>(s.cand)[lane];
                uint32_t rank = lane < int(inside) ? 0u : want;
                for (uint32_t j = 0; j < inside; j += 4) {   // (places behind the last hold 0)
                    const uint4 o = s.cand[j / 2], u = s.cand[j / 2 + 1];
                    rank += o.x > c.x || (o.x == c.x && o.y < c.y);
                    rank += o.z > c.x || (o.z == c.x && o.w < c.y);
                    rank += u.x > c.x || (u.x == c.x && u.y < c.y);
                    rank += u.z > c.x || (u.z == c.x && u.w < c.y);
                }
                // the last one taken
                const int at = __ffs(__ballot_sync(kFull, rank == want - 1)) - 1;
                const uint32_t ck = __shfl_sync(kFull, c.x, at);
                const int cb = int(__shfl_sync(kFull, c.y, at));
                n = warps_before(s.warp_a) +
                    __popc(__ballot_sync(kFull, rank < want && int(c.y) < warp * stretch));
                in_order([&](int b, uint32_t k) {
                    const bool in = k > ck || (k == ck && b <= cb);
                    const uint32_t m = __ballot_sync(kFull, in);
                    if (in) out[n + __popc(m & below)] = b;
                    n += __popc(m);
                });
                return;
            }
            if (want == inside) {                // the whole bin (no key is 0: -inf's is above)
                cut = first - 1;
                break;
            }
            lo = first;
            hi = last;
            __syncthreads();                     // (the bin was read by all)
#pragma unroll
            for (int i = 0; i < 4; ++i) s.hist[i * NT + tid] = 0;
            __syncthreads();
        }
    }
    // in ascending order: each warp's counts are summed first
    uint32_t n_above = 0, n_equal = 0;
    in_order([&](int, uint32_t k) {
        n_above += __popc(__ballot_sync(kFull, k > cut));
        n_equal += __popc(__ballot_sync(kFull, k == cut));
    });
    __syncthreads();                             // (what the warps left there was read by all)
    if (lane == 0) s.warp_a[warp] = n_above, s.warp_b[warp] = n_equal;
    __syncthreads();
    n_above = warps_before(s.warp_a);
    n_equal = warps_before(s.warp_b);
    in_order([&](int b, uint32_t k) {
        const uint32_t ma = __ballot_sync(kFull, k > cut), me = __ballot_sync(kFull, k == cut);
        const uint32_t at = n_above + __popc(ma & below), nth = n_equal + __popc(me & below);
        if (k > cut || (k == cut && nth < take)) out[at + min(nth, take)] = b;
        n_above += __popc(ma);
        n_equal += __popc(me);
    });
}

size_t select_stride(int32_t max_ctx) {
    return align_up(size_t(ceil_div(max_ctx, kBlockTokens)), 4);
}

template <int D, int G, int R>
int launch_scores_r(SelectParams p, cudaStream_t stream) {
    // (Device times, calls back to back, each rule beside its alternatives at its step.)
    // Chunks of 4 to 16 tiles that give every SM some warps, of 2 for a few rows (8
    // items of 2048 blocks: 6.1 us, 7.1 with chunks of 4; 32 items: 9.0 and 8.7).
    // Where they are longer than 4, the last fifth of the rows goes in chunks of 4,
    // so that the SMs run dry at about the same time.  The whole call, 256 rows of 64
    // to 512 blocks / 48 x 2 of 2048: 34.7 / 35.2 us; with no fine rows 37.2 / 36.8,
    // with half of them fine 35.8 / 37.5, with chunks of 8 throughout 36.8 / 37.5.
    const int64_t items = ceil_div(int64_t(p.tokens), R) * int64_t(p.num_kv_heads);
    const int tiles = ceil_div(p.stride, kTileBlocks);
    auto ctas = [&](int chunk_tiles) {           // of a row
        return ceil_div(ceil_div(tiles, chunk_tiles) * int64_t(p.num_kv_heads), kScoreWarps);
    };
    p.chunk_tiles = 16;
    while (p.chunk_tiles > 2 && items * ceil_div(tiles, p.chunk_tiles) <
                                    (p.chunk_tiles > 4 ? 8 : 2) * int64_t(num_sms()))
        p.chunk_tiles /= 2;
    p.fine_tiles = std::min(p.chunk_tiles, 4);
    p.fine_row = p.fine_tiles < p.chunk_tiles ? p.tokens - p.tokens / 5 : p.tokens;
    p.row_ctas = ctas(p.chunk_tiles);
    p.fine_ctas = ctas(p.fine_tiles);
    const int64_t coarse = int64_t(p.fine_row) * p.row_ctas;
    const int64_t all = coarse + int64_t(p.tokens - p.fine_row) * p.fine_ctas;
    if (all > INT32_MAX) return PKV_ERR_UNSUPPORTED;
    p.fine_cta = int32_t(coarse);
    return cuda_status(launch_pdl(block_scores_kernel<D, G, R>, dim3(unsigned(all)),
                                  dim3(kScoreWarps * 32), 0, stream, p));
}

// Rows of a sequence share the reads of its bounds, up to eight columns.
template <int D, int G>
int launch_scores_g(const SelectParams& p, cudaStream_t s) {
    return p.rows.start ? launch_scores_r<D, G, 8 / G>(p, s) : launch_scores_r<D, G, 1>(p, s);
}

template <int D>
int launch_scores(const SelectParams& p, cudaStream_t s) {
    switch (p.num_q_heads / p.num_kv_heads) {
        case 1: return launch_scores_g<D, 1>(p, s);
        case 2: return launch_scores_g<D, 2>(p, s);
        case 4: return launch_scores_g<D, 4>(p, s);
        default: return launch_scores_g<D, 8>(p, s);
    }
}

template <int NT, int kHeld>
int launch_pick_t(const SelectParams& p, cudaStream_t s) {
    return cuda_status(launch_pdl(pick_blocks_kernel<NT, kHeld>,
                                  dim3(unsigned(p.tokens) * unsigned(p.num_kv_heads)), dim3(NT), 0,
                                  s, p));
}

// Threads that hold a row's keys, four to sixteen each.  Device time of the whole call
// with one or the other, at the step that chose (32 rows now 8.3 us): 32 rows of
// 2048 blocks 8.5 us with 256 threads, 8.9 with 512, 9.6 with 128; 768 such rows 38,
// 39 and 39.5; 8 rows of 8192 blocks 10.7 us with 512 threads, 12.9 with 256, 14.1
// by passes over memory.  Longer rows take as many threads as there are: 8 rows of
// 16384 blocks 18 to 21 us, 28 with 512 (34 MB, 5 us at HBM's rate: eight CTAs read
// their rows' keys in four passes, one after the other).
int launch_pick(const SelectParams& p, cudaStream_t s) {
    if (p.stride <= 128 * 4) return launch_pick_t<128, 4>(p, s);
    if (p.stride <= 256 * 8) return launch_pick_t<256, 8>(p, s);
    if (p.stride <= 512 * 16) return launch_pick_t<512, 16>(p, s);
    return launch_pick_t<1024, 0>(p, s);
}

bool aligned_to(const void* p, uintptr_t a) {
    return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

template <typename T, int D>
int launch_bounds(BoundsParams p, cudaStream_t s) {
    const int64_t units = ceil_div(p.tokens, p.span) * int64_t(p.num_kv_heads);
    p.work_ctas = int((units + kBoundsWarps - 1) / kBoundsWarps);
    // (two offsets a thread)
    const int checks = p.start ? std::min(ceil_div(p.n, 2 * kBoundsWarps * 32), num_sms()) : 0;
    return cuda_status(launch_pdl(block_bounds_kernel<T, D>, dim3(unsigned(p.work_ctas + checks)),
                                  dim3(kBoundsWarps * 32), 0, s, p));
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
    if (int64_t(num_query_tokens) * desc->num_kv_heads > INT32_MAX) return PKV_ERR_UNSUPPORTED;
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
    // few tokens: one to a warp; many: a block's worth, of which one or two stand
    // for a block
    p.span = 1;
    while (p.span < kBlockTokens &&
           int64_t(num_query_tokens) * desc->num_kv_heads / p.span > 64 * int64_t(num_sms()))
        p.span *= 2;
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    if (desc->dtype == PKV_BF16)
        return desc->head_dim == 128 ? launch_bounds<__nv_bfloat16, 128>(p, cs)
                                     : launch_bounds<__nv_bfloat16, 64>(p, cs);
    return desc->head_dim == 128 ? launch_bounds<float, 128>(p, cs) : launch_bounds<float, 64>(p, cs);
}

extern "C" size_t pkv_select_workspace_bytes(const pkv_cache_desc* desc, int32_t num_query_tokens,
                                             int32_t max_context_len) {
    if (check_desc(desc, true) != PKV_OK || num_query_tokens < 0 || max_context_len < 1) return 0;
    return align_up(size_t(num_query_tokens) * desc->num_kv_heads * select_stride(max_context_len) *
                        sizeof(uint32_t),
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
    // (launch sizes and indices within 32 bits)
    if (int64_t(num_query_tokens) * desc->num_kv_heads > INT32_MAX || top_k > PKV_SPARSE_MAX_TOP_K ||
        ceil_div(max_context_len, kBlockTokens) * int64_t(desc->num_kv_heads) > INT32_MAX)
        return PKV_ERR_UNSUPPORTED;
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
                       max_context_len, num_query_tokens};
    p.keys = static_cast<uint32_t*>(workspace);
    p.stride = int32_t(select_stride(max_context_len));
    p.tokens = num_query_tokens;
    p.num_blocks = desc->num_blocks;
    p.num_q_heads = desc->num_q_heads;
    p.num_kv_heads = desc->num_kv_heads;
    p.top_k = top_k;
    p.sink = num_sink;
    p.recent = num_recent;
    p.q_f32 = desc->dtype == PKV_F32;
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    // (a batch whose lists hold every block needs no scores)
    if (ceil_div(max_context_len, kBlockTokens) > top_k) {
        st = desc->head_dim == 128 ? launch_scores<128>(p, cs) : launch_scores<64>(p, cs);
        if (st != PKV_OK) return st;
    }
    return launch_pick(p, cs);
}
