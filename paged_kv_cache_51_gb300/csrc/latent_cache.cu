// The latent cache's entry points: append with normalisation and rotation, the gather, and
// the attention's argument checks and workspace.
//
// Both kernels (append, gather) move bytes and are bound by HBM (by launch latency for one
// decode step): 16-byte vectors, every load of a warp's share issued before its first store.
// Whole blocks are copied by append.cu's kernel.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "latent_common.cuh"
#include "launch_cache.h"

namespace pkv {

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// ---- append ---------------------------------------------------------------------
struct AppendParams {
    const void* latent;
    const void* k_rope;
    const void* weight;
    const int64_t* slots;
    const int32_t* positions;
    const float* cos_sin;
    void* cache;
    const void* q;
    void* q_out;
    int64_t latent_stride, k_stride, q_token, q_head, o_token, o_head;
    int64_t num_slots;
    int64_t warps;            // tokens x tasks
    int32_t tasks;            // of a token: its cache row, then its query heads in groups
    int32_t heads;
    int32_t latent_dim;
    int32_t max_position;
    float eps;
    int* err;
};

// Values of one lane's part of a row: 8 pairs, bf16 (2 vectors) or fp32 (4).
template <typename T>
struct Values {
    uint4 w[sizeof(T)];
    __device__ void load(const T* a, const T* b) {
        constexpr int n = sizeof(T) / 2;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            w[i] = __ldg(reinterpret_cast<const uint4*>(a) + i);
            w[n + i] = __ldg(reinterpret_cast<const uint4*>(b) + i);
        }
    }
    __device__ void store(T* a, T* b) const {
        constexpr int n = sizeof(T) / 2;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            reinterpret_cast<uint4*>(a)[i] = w[i];
            reinterpret_cast<uint4*>(b)[i] = w[n + i];
        }
    }
    __device__ void wide(float (&x)[16]) const {
        if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[8 * i + 2 * e] = __uint_as_float(u[e] << 16);
                    x[8 * i + 2 * e + 1] = __uint_as_float(u[e] & 0xffff0000u);
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[4 * i] = __uint_as_float(w[i].x);
                x[4 * i + 1] = __uint_as_float(w[i].y);
                x[4 * i + 2] = __uint_as_float(w[i].z);
                x[4 * i + 3] = __uint_as_float(w[i].w);
            }
        }
    }
    __device__ void narrow(const float (&x)[16]) {
        if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                w[i] = make_uint4(pack_bf16x2(x[8 * i], x[8 * i + 1]), pack_bf16x2(x[8 * i + 2], x[8 * i + 3]),
                                  pack_bf16x2(x[8 * i + 4], x[8 * i + 5]), pack_bf16x2(x[8 * i + 6], x[8 * i + 7]));
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = make_uint4(__float_as_uint(x[4 * i]), __float_as_uint(x[4 * i + 1]),
                                  __float_as_uint(x[4 * i + 2]), __float_as_uint(x[4 * i + 3]));
        }
    }
};

// Pairs 8c .. 8c + 7 of a row of 64 values: where a lane's two runs of 8 values begin.
template <bool kInter>
__device__ __forceinline__ int run_a(int c) { return kInter ? 16 * c : 8 * c; }
template <bool kInter>
__device__ __forceinline__ int run_b(int c) { return kInter ? 16 * c + 8 : 32 + 8 * c; }

// Each product and sum rounded on its own, as the rotary append of the other caches.
template <typename T, bool kInter>
__device__ __forceinline__ void rotate(Values<T>& v, const float (&co)[8], const float (&si)[8]) {
    float x[16];
    v.wide(x);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int ia = kInter ? 2 * i : i, ib = kInter ? 2 * i + 1 : 8 + i;
        const float a = x[ia], b = x[ib];
        x[ia] = __fsub_rn(__fmul_rn(a, co[i]), __fmul_rn(b, si[i]));
        x[ib] = __fadd_rn(__fmul_rn(a, si[i]), __fmul_rn(b, co[i]));
    }
    v.narrow(x);
}

__device__ __forceinline__ void load_angles(const float* table, int64_t pos, int c, float (&co)[8],
                                            float (&si)[8]) {
    const float4* t = reinterpret_cast<const float4*>(table + pos * kLatentRope + 8 * c);
    const float4 a = __ldg(t), b = __ldg(t + 1), d = __ldg(t + 8), e = __ldg(t + 9);
    co[0] = a.x; co[1] = a.y; co[2] = a.z; co[3] = a.w;
    co[4] = b.x; co[5] = b.y; co[6] = b.z; co[7] = b.w;
    si[0] = d.x; si[1] = d.y; si[2] = d.z; si[3] = d.w;
    si[4] = e.x; si[5] = e.y; si[6] = e.z; si[7] = e.w;
}

constexpr int kHeadsPerWarp = 16;          // 4 lanes a row, two rows a lane

// One warp a task.  Task 0 of a token is its cache row: the lanes hold the latent
// vector, sum its squares by shuffles and write it, and lanes 0-3 rotate the key.
// The other tasks rotate 16 query heads each, 4 lanes a head.  Bound by how many loads are on
// their way: 40 warps an SM at 48 registers (12 bytes of which spill) and CTAs of four of them
// take 31.5 us for 16384 tokens of 32 heads, 32 warps at 64 in CTAs of eight 33.9, 32 heads a
// warp 33.3, 8 heads 42.  fp32: 80 registers, 24 warps, 8192 such tokens 30.0 us.
template <typename T, bool kInter>
__global__ void __launch_bounds__(128, sizeof(T) == 2 ? 10 : 6) latent_append_kernel(AppendParams p) {
    pdl_wait_prerequisites();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t id = int64_t(blockIdx.x) * (blockDim.x / 32) + (threadIdx.x >> 5);
    if (id >= p.warps) return;
    const int64_t t = id / p.tasks;
    const int task = int(id - t * p.tasks);
    const int64_t pos = __ldg(p.positions + t);
    const bool pos_ok = pos >= 0 && pos < p.max_position;
    const int c = lane & 3;
    float co[8], si[8];
    if (task > 0) {
        // the values are asked for next to the position, before it is looked at
        Values<T> v[2];
        int h[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            h[u] = (task - 1) * kHeadsPerWarp + u * 8 + (lane >> 2);
            const T* src = static_cast<const T*>(p.q) + t * p.q_token + h[u] * p.q_head;
            if (h[u] < p.heads) v[u].load(src + run_a<kInter>(c), src + run_b<kInter>(c));
        }
        if (!pos_ok) {
            if (task == 1 && lane == 0) flag_error(p.err, PKV_DEV_BAD_POSITION);
            return;
        }
        load_angles(p.cos_sin, pos, c, co, si);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            if (h[u] >= p.heads) continue;
            rotate<T, kInter>(v[u], co, si);
            T* dst = static_cast<T*>(p.q_out) + t * p.o_token + h[u] * p.o_head;
            v[u].store(dst + run_a<kInter>(c), dst + run_b<kInter>(c));
        }
        return;
    }
    const int64_t slot = __ldg(p.slots + t);
    const T* src = static_cast<const T*>(p.latent) + t * p.latent_stride;
    // the vector and the key are asked for before slot and position are looked at
    Values<T> key;
    if (lane < 4) {
        const T* k = static_cast<const T*>(p.k_rope) + t * p.k_stride;
        key.load(k + run_a<kInter>(c), k + run_b<kInter>(c));
    }
    constexpr int kPer = 16 / sizeof(T);                   // values of a vector
    constexpr int kMost = 512 / kPer / 32;                 // vectors of a lane at most
    const int vecs = p.latent_dim / kPer;
    uint4 x[kMost], w[kMost];
#pragma unroll
    for (int i = 0; i < kMost; ++i) {
        const int at = lane + 32 * i;
        if (at < vecs) {
            x[i] = __ldg(reinterpret_cast<const uint4*>(src) + at);
            if (p.weight) w[i] = __ldg(static_cast<const uint4*>(p.weight) + at);
        }
    }
    if (slot < 0 || slot >= p.num_slots) {
        if (slot >= 0 && lane == 0) flag_error(p.err, PKV_DEV_BAD_SLOT);
        return;
    }
    if (!pos_ok) {
        if (lane == 0) flag_error(p.err, PKV_DEV_BAD_POSITION);
        return;
    }
    T* row = static_cast<T*>(p.cache) + slot * (p.latent_dim + kLatentRope);
    if (lane < 4) load_angles(p.cos_sin, pos, c, co, si);
    if (p.weight) {
        auto get = [](const uint4& v, int e) {
            const uint32_t u[4] = {v.x, v.y, v.z, v.w};
            if constexpr (sizeof(T) == 2)
                return __uint_as_float(e & 1 ? u[e / 2] & 0xffff0000u : u[e / 2] << 16);
            else
                return __uint_as_float(u[e]);
        };
        float sq = 0.f;
#pragma unroll
        for (int i = 0; i < kMost; ++i)
            if (lane + 32 * i < vecs)
#pragma unroll
                for (int e = 0; e < kPer; ++e) sq = fmaf(get(x[i], e), get(x[i], e), sq);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, d);
        const float inv = 1.f / sqrtf(sq / float(p.latent_dim) + p.eps);
#pragma unroll
        for (int i = 0; i < kMost; ++i) {
            float y[kPer];
#pragma unroll
            for (int e = 0; e < kPer; ++e) y[e] = get(x[i], e) * inv * get(w[i], e);
            if constexpr (sizeof(T) == 2)
                x[i] = make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]),
                                  pack_bf16x2(y[6], y[7]));
            else
                x[i] = make_uint4(__float_as_uint(y[0]), __float_as_uint(y[1]), __float_as_uint(y[2]),
                                  __float_as_uint(y[3]));
        }
    }
#pragma unroll
    for (int i = 0; i < kMost; ++i)
        if (lane + 32 * i < vecs) reinterpret_cast<uint4*>(row)[lane + 32 * i] = x[i];
    if (lane < 4) {
        rotate<T, kInter>(key, co, si);
        T* dst = row + p.latent_dim;
        key.store(dst + run_a<kInter>(c), dst + run_b<kInter>(c));
    }
}

// ---- gather ---------------------------------------------------------------------
struct GatherParams {
    uint4* latent;
    uint4* rope;
    const uint4* cache;
    const int32_t* tables;
    const int32_t* starts;
    int64_t stride;           // of a table row
    int32_t num_seqs;
    int32_t num_keys;
    int32_t num_blocks;
    int* err;
};

constexpr int kGatherRows = 8;             // rows a warp

// A warp moves 8 rows in a row: lanes 0-7 look their rows up (a search over the offsets,
// then the table), and all lanes copy the rows' vectors one after the other.  VECS: 16-byte
// vectors of a cached row, RVECS of its rotary part (with sizes known at run time only, two
// divisions a vector made the kernel instruction-bound: 65 us for 129536 rows of 1152 bytes;
// now 46.6, 0.94 of what a copy of them takes).
template <int VECS, int RVECS>
__global__ void __launch_bounds__(256) latent_gather_kernel(GatherParams p) {
    pdl_wait_prerequisites();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t t0 = (int64_t(blockIdx.x) * (blockDim.x / 32) + (threadIdx.x >> 5)) * kGatherRows;
    const int end = __ldg(p.starts + p.num_seqs);
    if (end > p.num_keys) {
        if (t0 == 0 && lane == 0) flag_error(p.err, PKV_DEV_BAD_QUERY_LAYOUT);
        return;
    }
    if (t0 >= end) return;
    int64_t row = -1;
    if (lane < kGatherRows && t0 + lane < end) {
        const int t = int(t0) + lane;
        int lo = 0, hi = p.num_seqs;       // the last sequence that begins at or before t
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (__ldg(p.starts + mid) <= t) lo = mid;
            else hi = mid;
        }
        const int first = __ldg(p.starts + lo), next = __ldg(p.starts + lo + 1);
        if (first > t || first < 0 || next <= t || next > end) {
            flag_error(p.err, PKV_DEV_BAD_QUERY_LAYOUT);
        } else {
            const int pos = t - first, blk_at = pos / kBlockTokens;
            if (blk_at >= p.stride) {
                flag_error(p.err, PKV_DEV_TABLE_TOO_NARROW);
            } else {
                const int blk = __ldg(p.tables + lo * p.stride + blk_at);
                if (blk < 0 || blk >= p.num_blocks) flag_error(p.err, PKV_DEV_BAD_BLOCK_ID);
                else row = int64_t(blk) * kBlockTokens + pos % kBlockTokens;
            }
        }
    }
    __syncwarp();
    constexpr int kLatent = VECS - RVECS, kTotal = VECS * kGatherRows;
    constexpr int kUnroll = kTotal / 32 % 9 == 0 ? 9 : kTotal / 32 % 6 == 0 ? 6 : kTotal / 32 % 7 == 0 ? 7 : 5;
    static_assert(kTotal % (32 * kUnroll) == 0, "whole passes");
    uint4* latent = p.latent + t0 * kLatent;
    uint4* rope = p.rope + t0 * RVECS;
#pragma unroll
    for (int pass = 0; pass < kTotal / 32 / kUnroll; ++pass) {
        uint4 x[kUnroll];
        bool there[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const uint32_t v = lane + 32 * (pass * kUnroll + u), r = v / VECS;
            const int64_t src = __shfl_sync(0xffffffffu, row, int(r));
            there[u] = src >= 0;
            if (there[u]) x[u] = __ldg(p.cache + src * VECS + (v - r * VECS));
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const uint32_t v = lane + 32 * (pass * kUnroll + u), r = v / VECS, c = v - r * VECS;
            if (!there[u]) continue;
            if (c < kLatent) latent[r * kLatent + c] = x[u];
            else rope[r * RVECS + c - kLatent] = x[u];
        }
    }
}

}  // namespace

int check_latent_desc(const pkv_latent_desc* d) {
    if (!d) return PKV_ERR_INVALID;
    if (d->dtype != PKV_F32 && d->dtype != PKV_BF16) return PKV_ERR_UNSUPPORTED;
    if (d->num_blocks < 1 || d->block_size < 1 || d->latent_dim < 1 || d->rope_dim < 1 ||
        d->num_q_heads < 1)
        return PKV_ERR_INVALID;
    if (d->block_size != kBlockTokens || d->rope_dim != kLatentRope || d->latent_dim % 128 ||
        d->latent_dim > 512 || d->num_q_heads > 65536)
        return PKV_ERR_UNSUPPORTED;
    // row indices of the cache are 32-bit
    if (int64_t(d->num_blocks) * kBlockTokens >= (int64_t(1) << 31)) return PKV_ERR_UNSUPPORTED;
    return PKV_OK;
}

size_t latent_workspace_layout(const pkv_latent_desc* d, void* base, LatentWorkspace* ws) {
    const size_t ctas = size_t(std::max(num_sms(), 1));
    const size_t o_ml = align_up(ctas * sizeof(LatentMerge), 256);
    const size_t o_o = align_up(o_ml + 2 * ctas * kLatentRowTile * sizeof(float2), 256);
    if (ws) {
        char* b = static_cast<char*>(base);
        ws->merge = reinterpret_cast<LatentMerge*>(b);
        ws->ml = reinterpret_cast<float2*>(b + o_ml);
        ws->o = reinterpret_cast<float*>(b + o_o);
    }
    return o_o + 2 * ctas * kLatentRowTile * size_t(d->latent_dim) * sizeof(float);
}

}  // namespace pkv

using namespace pkv;

extern "C" int paged_latent_append(const void* latent, int64_t latent_stride, const void* k_rope,
                                   int64_t k_rope_stride, const void* norm_weight, float eps,
                                   const int64_t* slot_mapping, const int32_t* positions,
                                   const float* cos_sin, int32_t max_position, int32_t rope_layout,
                                   int32_t num_tokens, void* latent_cache, const void* q,
                                   int64_t q_token_stride, int64_t q_head_stride, void* q_out,
                                   int64_t q_out_token_stride, int64_t q_out_head_stride,
                                   const pkv_latent_desc* desc, void* stream) {
    int st = check_latent_desc(desc);
    if (st != PKV_OK) return st;
    if (num_tokens < 0 || max_position < 1) return PKV_ERR_INVALID;
    if (rope_layout != PKV_ROPE_HALF && rope_layout != PKV_ROPE_INTERLEAVED) return PKV_ERR_UNSUPPORTED;
    if (norm_weight && !(eps >= 0.f && std::isfinite(eps))) return PKV_ERR_INVALID;
    if (num_tokens == 0) return PKV_OK;
    if (!latent || !k_rope || !slot_mapping || !positions || !cos_sin || !latent_cache ||
        (q == nullptr) != (q_out == nullptr))
        return PKV_ERR_INVALID;
    const int64_t per = desc->dtype == PKV_BF16 ? 8 : 4;       // values of 16 bytes
    if (!aligned(latent, 16) || !aligned(k_rope, 16) || !aligned(norm_weight, 16) ||
        !aligned(cos_sin, 16) || !aligned(latent_cache, 16) || !aligned(q, 16) || !aligned(q_out, 16) ||
        !aligned(slot_mapping, 8) || !aligned(positions, 4) || latent_stride % per || k_rope_stride % per)
        return PKV_ERR_INVALID;
    if (q && (q_token_stride % per || q_head_stride % per || q_out_token_stride % per ||
              q_out_head_stride % per))
        return PKV_ERR_INVALID;
    AppendParams p;
    p.err = device_error_ptr(&st);
    if (st != PKV_OK) return st;
    p.latent = latent;
    p.k_rope = k_rope;
    p.weight = norm_weight;
    p.slots = slot_mapping;
    p.positions = positions;
    p.cos_sin = cos_sin;
    p.cache = latent_cache;
    p.q = q;
    p.q_out = q_out;
    p.latent_stride = latent_stride;
    p.k_stride = k_rope_stride;
    p.q_token = q_token_stride;
    p.q_head = q_head_stride;
    p.o_token = q_out_token_stride;
    p.o_head = q_out_head_stride;
    p.num_slots = int64_t(desc->num_blocks) * desc->block_size;
    p.tasks = 1 + (q ? ceil_div(desc->num_q_heads, kHeadsPerWarp) : 0);
    p.warps = int64_t(num_tokens) * p.tasks;
    p.heads = desc->num_q_heads;
    p.latent_dim = desc->latent_dim;
    p.max_position = max_position;
    p.eps = eps;
    // one warp a CTA while that leaves SMs free: a decode step's chain is short
    const int warps = p.warps <= 2 * int64_t(std::max(num_sms(), 1)) ? 1 : 4;
    const int64_t blocks = (p.warps + warps - 1) / warps;
    if (blocks > INT32_MAX) return PKV_ERR_UNSUPPORTED;
    const bool inter = rope_layout == PKV_ROPE_INTERLEAVED;
    auto kern = desc->dtype == PKV_BF16
                    ? (inter ? latent_append_kernel<__nv_bfloat16, true> : latent_append_kernel<__nv_bfloat16, false>)
                    : (inter ? latent_append_kernel<float, true> : latent_append_kernel<float, false>);
    return cuda_status(launch_pdl(kern, dim3(unsigned(blocks)), dim3(32 * warps), 0,
                                  static_cast<cudaStream_t>(stream), p));
}

extern "C" int paged_latent_gather(void* latent_out, void* rope_out, const void* latent_cache,
                                   const pkv_latent_desc* desc, const int32_t* block_tables,
                                   int32_t max_blocks_per_seq, const int32_t* key_start_loc,
                                   int32_t num_seqs, int32_t num_keys, void* stream) {
    int st = check_latent_desc(desc);
    if (st != PKV_OK) return st;
    if (num_seqs < 0 || num_keys < 0 || max_blocks_per_seq < 1) return PKV_ERR_INVALID;
    if (num_seqs == 0 || num_keys == 0) return PKV_OK;
    if (!latent_out || !rope_out || !latent_cache || !block_tables || !key_start_loc ||
        !aligned(latent_out, 16) || !aligned(rope_out, 16) || !aligned(latent_cache, 16) ||
        !aligned(block_tables, 4) || !aligned(key_start_loc, 4))
        return PKV_ERR_INVALID;
    GatherParams p;
    p.err = device_error_ptr(&st);
    if (st != PKV_OK) return st;
    const int per = desc->dtype == PKV_BF16 ? 8 : 4;
    p.latent = static_cast<uint4*>(latent_out);
    p.rope = static_cast<uint4*>(rope_out);
    p.cache = static_cast<const uint4*>(latent_cache);
    p.tables = block_tables;
    p.starts = key_start_loc;
    p.stride = max_blocks_per_seq;
    p.num_seqs = num_seqs;
    p.num_keys = num_keys;
    p.num_blocks = desc->num_blocks;
    const auto kern = [&]() -> void (*)(GatherParams) {
        switch ((desc->latent_dim + desc->rope_dim) / per) {
            case 24: return latent_gather_kernel<24, 8>;
            case 40: return latent_gather_kernel<40, 8>;
            case 56: return latent_gather_kernel<56, 8>;
            case 72: return latent_gather_kernel<72, 8>;
            case 48: return latent_gather_kernel<48, 16>;
            case 80: return latent_gather_kernel<80, 16>;
            case 112: return latent_gather_kernel<112, 16>;
            default: return latent_gather_kernel<144, 16>;
        }
    }();
    const int rows = kGatherRows * 8;
    return cuda_status(launch_pdl(kern, dim3(unsigned((int64_t(num_keys) + rows - 1) / rows)), dim3(256), 0,
                                  static_cast<cudaStream_t>(stream), p));
}

extern "C" size_t pkv_latent_workspace_bytes(const pkv_latent_desc* desc, int32_t num_seqs,
                                             int32_t num_query_tokens, int32_t max_context_len) {
    if (check_latent_desc(desc) != PKV_OK || num_seqs < 0 || num_query_tokens < 0 || max_context_len < 1)
        return 0;
    return latent_workspace_layout(desc, nullptr, nullptr);
}

extern "C" int paged_attention_latent(void* out, const void* q, const void* latent_cache,
                                      const pkv_latent_desc* desc, const int32_t* block_tables,
                                      int32_t max_blocks_per_seq, const int32_t* query_start_loc,
                                      const int32_t* context_lens, int32_t num_seqs,
                                      int32_t num_query_tokens, int32_t max_context_len, float scale,
                                      void* workspace, size_t workspace_bytes, void* stream) {
    int st = check_latent_desc(desc);
    if (st != PKV_OK) return st;
    if (num_seqs < 0 || num_query_tokens < 0 || max_blocks_per_seq < 1 || max_context_len < 1 ||
        !(scale > 0.f && std::isfinite(scale)) || (!query_start_loc && num_query_tokens != num_seqs))
        return PKV_ERR_INVALID;
    if (num_seqs == 0 || num_query_tokens == 0) return PKV_OK;
    // rows of q are counted in 32 bits, with up to 8 tiles of 128 behind the last
    if (int64_t(num_query_tokens) * desc->num_q_heads >= (int64_t(1) << 31) - 2048) return PKV_ERR_UNSUPPORTED;
    if (!out || !q || !latent_cache || !block_tables || !context_lens || !aligned(out, 16) ||
        !aligned(q, 16) || !aligned(latent_cache, 16) || !aligned(block_tables, 4) ||
        !aligned(context_lens, 4) || !aligned(query_start_loc, 4))
        return PKV_ERR_INVALID;
    LatentArgs a;
    const size_t need = latent_workspace_layout(desc, workspace, &a.ws);
    if (!workspace || !aligned(workspace, 256) || workspace_bytes < need) return PKV_ERR_WORKSPACE;
    a.batch.err = device_error_ptr(&st);
    if (st != PKV_OK) return st;
    a.out = out;
    a.q = q;
    a.cache = latent_cache;
    a.desc = desc;
    a.batch.block_tables = block_tables;
    a.batch.context_lens = context_lens;
    a.batch.query_start_loc = query_start_loc;
    a.batch.table_stride = max_blocks_per_seq;
    a.batch.num_blocks = desc->num_blocks;
    a.batch.num_seqs = num_seqs;
    a.batch.num_query_tokens = num_query_tokens;
    a.batch.max_context_len = max_context_len;
    a.batch.heads = desc->num_q_heads;
    a.batch.latent = desc->latent_dim;
    a.batch.scale_log2 = float(double(scale) * 1.4426950408889634);
    a.stream = static_cast<cudaStream_t>(stream);
    return desc->dtype == PKV_BF16 ? launch_latent_bf16(a) : launch_latent_f32(a);
}
