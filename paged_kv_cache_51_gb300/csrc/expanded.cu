// Attention over expanded keys: argument checks, the plan, and the single-precision
// kernel.  (expanded_tc.cu holds the bf16 kernel.)
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "expanded_common.h"
#include "launch_cache.h"
#include "pkv_device.cuh"

namespace pkv {
namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// ---- plan -----------------------------------------------------------------------
struct PlanParams {
    const int32_t* q_start;
    const int32_t* k_start;
    int32_t num_seqs, num_query_tokens, num_keys, max_query_len;
    int32_t rows, group;
    ExpandedWorkspace ws;
    int* err;
};

constexpr int kBins = 1024;

// One CTA counts the units by their keys (in tiles of 128, the last bin takes all longer
// ones) and writes them longest first, so that the CTAs that take them one by one end
// together.  Within a bin the order is that of the threads' arrival, which no result
// depends on.
__global__ void __launch_bounds__(1024) expanded_plan_kernel(PlanParams p) {
    __shared__ int32_t bin[kBins];
    __shared__ int32_t sums[32];
    const int tid = threadIdx.x;
    bin[tid] = 0;
    pdl_wait_prerequisites();
    pdl_launch_dependents();
    __syncthreads();
    auto each = [&](bool flag, auto&& take) {
        for (int s = tid; s < p.num_seqs; s += 1024) {
            const int q0 = __ldg(p.q_start + s), q1 = __ldg(p.q_start + s + 1);
            const int k0 = __ldg(p.k_start + s), k1 = __ldg(p.k_start + s + 1);
            if (q0 < 0 || q1 < q0 || q1 > p.num_query_tokens || q1 - q0 > p.max_query_len || k0 < 0 ||
                k1 < k0 || k1 > p.num_keys || (s == 0 && (q0 != 0 || k0 != 0))) {
                if (flag) flag_error(p.err, PKV_DEV_BAD_QUERY_LAYOUT);
                continue;
            }
            // groups from the sequence's last unit on, each in the bin of its longest
            for (int left = (q1 - q0 + p.rows - 1) / p.rows; left > 0; left -= p.group) {
                const int n = min(p.group, left), r = (left - 1) * p.rows;
                ExpandedItem x;
                x.q0 = q0 + r;
                x.rows = min(p.rows, q1 - q0 - r);
                x.k0 = k0;
                x.keys = (k1 - k0) - (q1 - q0) + r + x.rows;
                x.members = n;
                take(x, kBins - 1 - min(kBins - 1, (max(x.keys, 0) + 127) / 128));
            }
        }
    };
    each(true, [&](const ExpandedItem& x, int b) { atomicAdd(&bin[b], x.members); });
    __syncthreads();
    // where each bin begins
    const int mine = bin[tid];
    int upto = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, upto, d);
        if ((tid & 31) >= d) upto += v;
    }
    if ((tid & 31) == 31) sums[tid >> 5] = upto;
    __syncthreads();
    for (int w = 0; w < (tid >> 5); ++w) upto += sums[w];
    bin[tid] = upto - mine;
    if (tid == 1023) {
        p.ws.counters[0] = min(upto, p.ws.max_items);
        p.ws.counters[1] = 0;
    }
    __syncthreads();
    each(false, [&](ExpandedItem x, int b) {
        x.group = atomicAdd(&bin[b], x.members);
        // (rows that offsets out of order name twice may leave no room)
        x.members = min(x.members, p.ws.max_items - x.group);
        for (int i = 0; i < x.members; ++i) {
            p.ws.items[x.group + i] = x;
            x.keys -= x.rows;              // the unit in front of it
            x.q0 -= p.rows;
            x.rows = p.rows;
        }
    });
}

// ---- single precision -------------------------------------------------------------
// A CTA takes 64 or 128 query rows of one head and tiles of 64 keys; a thread keeps RI x 4
// scores and RI rows x D / 16 values of the output in registers.  Bound by what shared memory
// returns: a read of 16 bytes a lane costs a warp four cycles, the time of 16 FMAs, and there
// are RI + 4 of them for 16 RI.  Eight rows a thread (two prompts of 1000 to 1500 tokens, 16
// heads of 64: 294 us, 311 with four) leave a CTA of 64 rows four warps, too few where it is
// alone on its SM (D = 128).  Where units of 64 rows would not give every SM two, they have 32
// and a cluster of four CTAs takes turns at the tiles of the keys and meets at the end: the
// tiles of a unit follow one another, and six prompts of up to 300 tokens with 4 heads took 52
// us with one CTA a unit and take 25 with four.  P lies over the keys that it was made of, so
// that three such CTAs (heads of 128: two) fit on an SM.
struct F32Params {
    ExpandedWorkspace ws;
    const float *q, *k, *v, *k_rope;
    float* out;
    int64_t k_token, k_head, v_token, v_head;
    int32_t heads;
    float scale_log2;
};

constexpr int kT = 64;                     // keys of a tile
constexpr int kPPitch = kT + 4;

template <int D, int ROWS>
constexpr int f32_smem_floats() {
    return (ROWS + kT) * (D + kExpandedRope + 4) + kT * (D + 4);
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(there ? 16 : 0)
                 : "memory");
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// the value at this address of the cluster's CTA `rank`
__device__ __forceinline__ float load_cluster(const float* at, int rank) {
    uint32_t a;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(at)), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}

// RI: rows of a thread; a unit has THREADS / 16 as many.  CTAS of a cluster share a unit.
template <int D, int THREADS, int RI, int CTAS>
__global__ void __cluster_dims__(CTAS, 1, 1) __launch_bounds__(THREADS) expanded_f32_kernel(F32Params p) {
    constexpr int kTy = THREADS / 16, kRows = kTy * RI;
    constexpr int kDim = D + kExpandedRope, kPitch = kDim + 4, kVPitch = D + 4;
    constexpr int kCols = D / 16;          // output values of a thread in a row
    static_assert(kRows * kPPitch <= kT * kPitch, "P lies over the keys");
    extern __shared__ float4 smem4[];
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    float* qs = reinterpret_cast<float*>(smem4);
    float* ks = qs + kRows * kPitch;
    float* vs = ks + kT * kPitch;
    float* ps = ks;
    pdl_wait_prerequisites();
    pdl_launch_dependents();
    const int unit = blockIdx.x / CTAS, rank = blockIdx.x % CTAS;
    if (unit / p.heads >= p.ws.counters[0]) return;
    int h;
    const ExpandedItem x = expanded_unit(p.ws, unit, p.heads, h);
    const int keys = max(x.keys, 0);

    for (int i = threadIdx.x; i < kRows * (kDim / 4); i += THREADS) {
        const int r = i / (kDim / 4), c = i - r * (kDim / 4);
        cp_async16(smem_u32(qs + r * kPitch + 4 * c),
                   p.q + ((int64_t(x.q0) + min(r, x.rows - 1)) * p.heads + h) * kDim + 4 * c, r < x.rows);
    }
    // rows ty + kTy i, keys and values tx + 16 j (in fours)
    float m[RI], l[RI], o[RI][kCols];
    int limit[RI];
#pragma unroll
    for (int i = 0; i < RI; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
        const int r = ty + kTy * i;
        limit[i] = r < x.rows ? x.keys - x.rows + r : -1;
#pragma unroll
        for (int c = 0; c < kCols; ++c) o[i][c] = 0.f;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    for (int k0 = rank * kT; k0 < keys; k0 += CTAS * kT) {
        __syncthreads();                   // the last tile's readers are done
        for (int i = tid; i < kT * (kDim / 4); i += THREADS) {
            const int r = i / (kDim / 4), c = i - r * (kDim / 4);
            const bool there = k0 + r < keys;
            const int64_t row = int64_t(x.k0) + (there ? k0 + r : 0);
            const float* src = c < D / 4 ? p.k + row * p.k_token + h * p.k_head + 4 * c
                                         : p.k_rope + row * kExpandedRope + 4 * (c - D / 4);
            cp_async16(smem_u32(ks + r * kPitch + 4 * c), src, there);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        for (int i = tid; i < kT * (D / 4); i += THREADS) {
            const int r = i / (D / 4), c = i - r * (D / 4);
            const bool there = k0 + r < keys;
            const int64_t row = int64_t(x.k0) + (there ? k0 + r : 0);
            cp_async16(smem_u32(vs + r * kVPitch + 4 * c), p.v + row * p.v_token + h * p.v_head + 4 * c, there);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        __syncthreads();
        float s[RI][4] = {};
#pragma unroll 4
        for (int c = 0; c < kDim / 4; ++c) {
            float4 a[RI], b[4];
#pragma unroll
            for (int i = 0; i < RI; ++i)
                a[i] = *reinterpret_cast<const float4*>(qs + (ty + kTy * i) * kPitch + 4 * c);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                b[i] = *reinterpret_cast<const float4*>(ks + (tx + 16 * i) * kPitch + 4 * c);
#pragma unroll
            for (int i = 0; i < RI; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    s[i][j] = fmaf(a[i].x, b[j].x, fmaf(a[i].y, b[j].y, fmaf(a[i].z, b[j].z, fmaf(a[i].w, b[j].w, s[i][j]))));
        }
        __syncthreads();                   // the keys have been read
#pragma unroll
        for (int i = 0; i < RI; ++i) {
            float mx = -INFINITY;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[i][j] = k0 + tx + 16 * j <= limit[i] ? s[i][j] * p.scale_log2 : -INFINITY;
                mx = fmaxf(mx, s[i][j]);
            }
#pragma unroll
            for (int d = 8; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
            const float m_new = fmaxf(m[i], mx);
            const float a = m_new == -INFINITY ? 1.f : exp2f(m[i] - m_new);
            const float ref = m_new == -INFINITY ? 0.f : m_new;
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float e = exp2f(s[i][j] - ref);
                ps[(ty + kTy * i) * kPPitch + tx + 16 * j] = e;
                sum += e;
            }
#pragma unroll
            for (int d = 8; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
            m[i] = m_new;
            l[i] = l[i] * a + sum;
#pragma unroll
            for (int c = 0; c < kCols; ++c) o[i][c] *= a;
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();
#pragma unroll 4
        for (int k = 0; k < kT; k += 4) {
            float4 e[RI];
#pragma unroll
            for (int i = 0; i < RI; ++i)
                e[i] = *reinterpret_cast<const float4*>(ps + (ty + kTy * i) * kPPitch + k);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
#pragma unroll
                for (int c = 0; c < kCols; c += 4) {
                    const float4 v = *reinterpret_cast<const float4*>(vs + (k + kk) * kVPitch + 16 * c + 4 * tx);
#pragma unroll
                    for (int i = 0; i < RI; ++i) {
                        const float w = kk == 0 ? e[i].x : kk == 1 ? e[i].y : kk == 2 ? e[i].z : e[i].w;
                        o[i][c] = fmaf(w, v.x, o[i][c]);
                        o[i][c + 1] = fmaf(w, v.y, o[i][c + 1]);
                        o[i][c + 2] = fmaf(w, v.z, o[i][c + 2]);
                        o[i][c + 3] = fmaf(w, v.w, o[i][c + 3]);
                    }
                }
            }
        }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");   // (the queries, where there was no tile)
    if constexpr (CTAS > 1) {
        // the CTAs' states: a thread's rows and columns are the same in all of them.  CTA r of
        // the cluster joins the rows i = r
        constexpr int kState = kCols + 2;
        static_assert(RI == CTAS && RI * kState * THREADS <= kT * kPitch, "states");
        __syncthreads();                   // the last tile's readers are done
#pragma unroll
        for (int i = 0; i < RI; ++i) {
            float* mine = ks + i * kState * THREADS + tid;
            mine[0] = m[i];
            mine[THREADS] = l[i];
#pragma unroll
            for (int c = 0; c < kCols; ++c) mine[(2 + c) * THREADS] = o[i][c];
        }
        cluster_sync();
#pragma unroll
        for (int i = 0; i < RI; ++i) {
            if (i != rank) continue;
            float part[CTAS][kState];
#pragma unroll
            for (int q = 0; q < CTAS; ++q)
#pragma unroll
                for (int c = 0; c < kState; ++c) part[q][c] = load_cluster(ks + (i * kState + c) * THREADS + tid, q);
            const float top = fmaxf(fmaxf(part[0][0], part[1][0]), fmaxf(part[2][0], part[3][0]));
            const float ref = top == -INFINITY ? 0.f : top;
            l[i] = 0.f;
#pragma unroll
            for (int c = 0; c < kCols; ++c) o[i][c] = 0.f;
#pragma unroll
            for (int q = 0; q < CTAS; ++q) {
                const float f = exp2f(part[q][0] - ref);
                l[i] += f * part[q][1];
#pragma unroll
                for (int c = 0; c < kCols; ++c) o[i][c] += f * part[q][2 + c];
            }
        }
        cluster_sync();                    // nobody leaves while its states are being read
    }
#pragma unroll
    for (int i = 0; i < RI; ++i) {
        const int r = ty + kTy * i;
        if (r >= x.rows || (CTAS > 1 && i != rank)) continue;
        const float inv = limit[i] >= 0 ? 1.f / l[i] : 0.f;      // a query without keys: zeros
        float* dst = p.out + ((int64_t(x.q0) + r) * p.heads + h) * D + 4 * tx;
#pragma unroll
        for (int c = 0; c < kCols; c += 4)
            *reinterpret_cast<float4*>(dst + 16 * c) =
                make_float4(o[i][c] * inv, o[i][c + 1] * inv, o[i][c + 2] * inv, o[i][c + 3] * inv);
    }
}

template <int D, int THREADS, int RI, int CTAS>
int launch_f32(const ExpandedArgs& a, const F32Params& p) {
    constexpr int rows = THREADS / 16 * RI, smem = f32_smem_floats<D, rows>() * int(sizeof(float));
    static_assert(smem <= 232448, "shared memory");
    const int st = launch_expanded_plan(a, rows);
    if (st != PKV_OK) return st;
    if (kernel_occupancy<expanded_f32_kernel<D, THREADS, RI, CTAS>>(THREADS, smem) < 1) return PKV_ERR_CUDA;
    const int64_t items = std::min<int64_t>(a.ws.max_items, ceil_div(a.num_query_tokens, rows) + int64_t(a.num_seqs));
    const int64_t grid = items * a.desc->num_heads * CTAS;
    if (grid > INT32_MAX) return PKV_ERR_UNSUPPORTED;
    return cuda_status(launch_pdl(expanded_f32_kernel<D, THREADS, RI, CTAS>, dim3(unsigned(grid)), dim3(THREADS),
                                  size_t(smem), a.stream, p));
}

int check_expanded_desc(const pkv_expanded_desc* d) {
    if (!d) return PKV_ERR_INVALID;
    if (d->dtype != PKV_F32 && d->dtype != PKV_BF16) return PKV_ERR_UNSUPPORTED;
    if (d->num_heads < 1 || d->head_dim < 1 || d->rope_dim < 1) return PKV_ERR_INVALID;
    if ((d->head_dim != 64 && d->head_dim != 128) || d->rope_dim != kExpandedRope || d->num_heads > 65536)
        return PKV_ERR_UNSUPPORTED;
    return PKV_OK;
}

// rows of the smallest unit (sizes the workspace)
int row_tile(const pkv_expanded_desc* d) {
    return d->dtype == PKV_BF16 ? kExpandedRowsBf16 : kExpandedRowsF32;
}

size_t layout(const pkv_expanded_desc* d, int32_t num_seqs, int32_t num_query_tokens, void* base,
              ExpandedWorkspace* ws) {
    const int64_t items = ceil_div(num_query_tokens, row_tile(d)) + int64_t(num_seqs);
    if (ws) {
        ws->counters = static_cast<int32_t*>(base);
        ws->items = reinterpret_cast<ExpandedItem*>(static_cast<char*>(base) + 256);
        ws->max_items = int32_t(items);
    }
    return align_up(256 + size_t(items) * sizeof(ExpandedItem), 256);
}

}  // namespace

int launch_expanded_plan(const ExpandedArgs& a, int rows) {
    const int64_t units = int64_t(ceil_div(a.num_query_tokens, rows)) * a.desc->num_heads;
    PlanParams p{a.query_start_loc, a.key_start_loc, a.num_seqs, a.num_query_tokens, a.num_keys,
                 a.max_query_len, rows, units >= 8 * int64_t(num_sms()) ? 4 : 1, a.ws, a.err};
    return cuda_status(launch_pdl(expanded_plan_kernel, dim3(1), dim3(1024), 0, a.stream, p));
}

int launch_expanded_f32(const ExpandedArgs& a) {
    F32Params p{a.ws,
                static_cast<const float*>(a.q),
                static_cast<const float*>(a.k),
                static_cast<const float*>(a.v),
                static_cast<const float*>(a.k_rope),
                static_cast<float*>(a.out),
                a.desc->k_token_stride,
                a.desc->k_head_stride,
                a.desc->v_token_stride,
                a.desc->v_head_stride,
                a.desc->num_heads,
                float(double(a.scale) * 1.4426950408889634)};
    const bool wide = a.desc->head_dim == 128;
    const int64_t units = int64_t(a.num_query_tokens) * a.desc->num_heads / 64;
    if (units < 2 * std::max(num_sms(), 1))
        return wide ? launch_f32<128, 128, 4, 4>(a, p) : launch_f32<64, 128, 4, 4>(a, p);
    if (!wide) return launch_f32<64, 128, 8, 1>(a, p);
    // (two prompts of 1000 to 1500 tokens, 16 heads: 554 us with 64 rows, 484 with 128; six of up
    // to 300, 32 heads: 172 and 199)
    return ceil_div(a.num_query_tokens, a.num_seqs) >= 512 ? launch_f32<128, 256, 8, 1>(a, p)
                                                           : launch_f32<128, 256, 4, 1>(a, p);
}

}  // namespace pkv

using namespace pkv;

extern "C" size_t pkv_expanded_workspace_bytes(const pkv_expanded_desc* desc, int32_t num_seqs,
                                               int32_t num_query_tokens) {
    if (check_expanded_desc(desc) != PKV_OK || num_seqs < 0 || num_query_tokens < 0) return 0;
    return layout(desc, num_seqs, num_query_tokens, nullptr, nullptr);
}

extern "C" int pkv_attention_expanded(void* out, const void* q, const void* k, const void* v,
                                      const void* k_rope, const pkv_expanded_desc* desc,
                                      const int32_t* query_start_loc, const int32_t* key_start_loc,
                                      int32_t num_seqs, int32_t num_query_tokens, int32_t num_keys,
                                      int32_t max_query_len, float scale, void* workspace,
                                      size_t workspace_bytes, void* stream) {
    int st = check_expanded_desc(desc);
    if (st != PKV_OK) return st;
    if (num_seqs < 0 || num_query_tokens < 0 || num_keys < 0 || max_query_len < 0 ||
        !(scale > 0.f && std::isfinite(scale)))
        return PKV_ERR_INVALID;
    if (num_seqs == 0 || num_query_tokens == 0) return PKV_OK;
    const int64_t per = desc->dtype == PKV_BF16 ? 8 : 4;
    if (!out || !q || !query_start_loc || !key_start_loc || (num_keys > 0 && (!k || !v || !k_rope)) ||
        !aligned(out, 16) || !aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(k_rope, 16) ||
        !aligned(query_start_loc, 4) || !aligned(key_start_loc, 4))
        return PKV_ERR_INVALID;
    // (the stride of a dimension of one is not used)
    const bool heads = desc->num_heads > 1, tokens = num_keys > 1;
    if ((tokens && (desc->k_token_stride < 1 || desc->k_token_stride % per || desc->v_token_stride < 1 ||
                    desc->v_token_stride % per)) ||
        (heads && num_keys > 0 && (desc->k_head_stride < 1 || desc->k_head_stride % per ||
                                   desc->v_head_stride < 1 || desc->v_head_stride % per)))
        return PKV_ERR_INVALID;
    ExpandedArgs a{out, q, k, v, k_rope, desc, query_start_loc, key_start_loc, num_seqs, num_query_tokens,
                   num_keys, max_query_len, scale, {}, nullptr, static_cast<cudaStream_t>(stream)};
    const size_t need = layout(desc, num_seqs, num_query_tokens, workspace, &a.ws);
    if (!workspace || !aligned(workspace, 256) || workspace_bytes < need) return PKV_ERR_WORKSPACE;
    a.err = device_error_ptr(&st);
    if (st != PKV_OK) return st;
    return desc->dtype == PKV_BF16 ? launch_expanded_bf16(a) : launch_expanded_f32(a);
}
