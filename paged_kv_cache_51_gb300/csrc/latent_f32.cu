// Attention over a paged latent cache in single precision, on the CUDA cores.
//
// A CTA of eight warps takes ROWS (token, head) rows of one sequence and tiles of 32 keys,
// two of them in flight (cp.async).  Products in fp32 have no tensor-core form that keeps
// their bits, so what bounds it beyond a few heads is the FMA rate, and shared memory in
// front of it: a thread therefore keeps a key's part (S) or a value's part (O) in
// registers against all rows.
//   S: warp w holds an eighth of the dimensions, lane = key, one sum per row: per 4
//      dimensions one read of its own and ROWS reads that all lanes share.
//      The eighths meet in shared memory.
//   O: a thread owns two dimensions and ROWS (or, for short vectors, a share of the) rows.
// Rows of keys lie four floats further apart than they are long, so that 32 lanes reading
// 16 bytes of 32 rows meet no bank twice.
// 8 rows where that covers a sequence's rows, else 16: with 16, half of the products of an
// 8-head decode step would be for nothing.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "latent_common.cuh"
#include "latent_merge.cuh"
#include "launch_cache.h"

namespace pkv {
namespace {

constexpr int kKeys = 32;
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kLeastSteps = 2;

struct Params {
    LatentBatch b;
    LatentWorkspace ws;
    float* out;
    const float* q;
    const float* cache;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(there ? 16 : 0)
                 : "memory");
}

// floats of shared memory: two key tiles, queries, eighths of S, P, alpha
__host__ __device__ constexpr int smem_floats(int latent, int rows) {
    return (2 * kKeys + rows) * (latent + kLatentRope + 4) + kWarps * rows * kKeys + kKeys * rows + 3 * rows;
}

// RPT: rows of a thread in the second product.
template <int ROWS, int RPT>
__global__ void __launch_bounds__(kThreads) latent_f32_kernel(Params p) {
    extern __shared__ float4 smem4[];
    float* smem = reinterpret_cast<float*>(smem4);
    const int R = p.b.latent, D = R + kLatentRope, pitch = D + 4;
    float* kt = smem;                                      // [2][kKeys][pitch]
    float* qs = kt + 2 * kKeys * pitch;                    // [ROWS][pitch]
    float* part = qs + ROWS * pitch;                       // [kWarps][ROWS][kKeys]
    float* pt = part + kWarps * ROWS * kKeys;              // [kKeys][ROWS]
    float* alpha = pt + kKeys * ROWS;                      // [ROWS]
    float* row_m = alpha + ROWS;                           // [ROWS], at the end of a fragment
    float* row_l = row_m + ROWS;
    __shared__ int64_t sums[kWarps + 2];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int vecs = D / 4;

    pdl_wait_prerequisites();
    pdl_launch_dependents();
    LatentWalk<ROWS, kKeys> w = latent_plan<ROWS, kKeys, kThreads>(p.b, sums, kLeastSteps, blockIdx.x, gridDim.x);
    if (tid == 0) p.ws.merge[blockIdx.x].nrows = 0;
    // sequences with lengths that the call does not allow: zeros
    for (int s = blockIdx.x; s < p.b.num_seqs; s += gridDim.x) {
        const LatentSeq x = latent_seq<false>(p.b, s);
        if (!x.zero) continue;
        const int64_t n = int64_t(p.b.heads) * R;
        for (int64_t i = tid; i < n * x.qlen; i += kThreads) p.out[x.q0 * n + i] = 0.f;
    }

    LatentFrag f;
    while (w.next(p.b, f)) {
        // a warp loads four of a tile's 32 rows; their block's id is asked for a tile ahead
        const int32_t* table = p.b.block_tables + int64_t(f.seq) * p.b.table_stride;
        auto block_of = [&](int j) {
            const int key = (f.kt0 + j) * kKeys + warp * 4;   // (four rows are of one block)
            return j < f.n && key < f.ctx ? __ldg(table + key / kBlockTokens) : 0;
        };
        auto load = [&](int j, int blk) {
            float* dst = kt + (j & 1) * kKeys * pitch + warp * 4 * pitch;
            const int key0 = (f.kt0 + j) * kKeys + warp * 4;
            const bool good = blk >= 0 && blk < p.b.num_blocks;
            if (!good && lane == 0 && key0 < f.ctx) flag_error(p.b.err, PKV_DEV_BAD_BLOCK_ID);
            const float* src = p.cache + (int64_t(good ? blk : 0) * kBlockTokens + key0 % kBlockTokens) * D;
#pragma unroll
            for (int r = 0; r < 4; ++r)
                for (int c = lane; c < vecs; c += 32)
                    cp_async16(smem_u32(dst + r * pitch + 4 * c), src + r * D + 4 * c, good && key0 + r < f.ctx);
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        int blk = block_of(0);
        __syncthreads();                                   // the last fragment's readers are done
        for (int i = tid; i < ROWS * vecs && f.n > 0; i += kThreads) {
            const int r = i / vecs, c = i - r * vecs;
            const bool there = r < f.nrows;
            cp_async16(smem_u32(qs + r * pitch + 4 * c),
                       p.q + (there ? (int64_t(f.row0) + r) * D + 4 * c : 0), there);
        }
        if (f.n > 0) load(0, blk);
        blk = block_of(1);

        float acc[RPT][2];
#pragma unroll
        for (int i = 0; i < RPT; ++i) acc[i][0] = acc[i][1] = 0.f;
        const int pairs = R / 2;
        const int d2 = tid % pairs, rg = tid / pairs;      // a thread's dimensions and rows
        const bool owner = rg * RPT < ROWS;
        constexpr int kMine = ROWS / kWarps;               // softmax rows of a warp
        float m[kMine], l[kMine];
        int limit[kMine];
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            m[i] = -INFINITY;
            l[i] = 0.f;
            const int r = warp * kMine + i;
            limit[i] = r < f.nrows ? f.first_pos + f.t0 + (f.rest + r) / p.b.heads : -1;
        }

        for (int j = 0; j < f.n; ++j) {
            if (j + 1 < f.n) load(j + 1, blk);
            blk = block_of(j + 2);
            if (j + 1 < f.n) asm volatile("cp.async.wait_group 1;" ::: "memory");
            else asm volatile("cp.async.wait_group 0;" ::: "memory");
            __syncthreads();
            const float* kb = kt + (j & 1) * kKeys * pitch;
            {
                float s[ROWS];
#pragma unroll
                for (int i = 0; i < ROWS; ++i) s[i] = 0.f;
                const int c1 = vecs / kWarps;              // (D is a multiple of 32)
                const float4* krow = reinterpret_cast<const float4*>(kb + lane * pitch) + warp * c1;
                const float4* qrow = reinterpret_cast<const float4*>(qs) + warp * c1;
                for (int c = 0; c < c1; ++c) {
                    const float4 k = krow[c];
#pragma unroll
                    for (int i = 0; i < ROWS; ++i) {
                        const float4 q = qrow[i * (pitch / 4) + c];
                        s[i] = fmaf(q.x, k.x, fmaf(q.y, k.y, fmaf(q.z, k.z, fmaf(q.w, k.w, s[i]))));
                    }
                }
#pragma unroll
                for (int i = 0; i < ROWS; ++i) part[(warp * ROWS + i) * kKeys + lane] = s[i];
            }
            __syncthreads();
            const int key = (f.kt0 + j) * kKeys + lane;
#pragma unroll
            for (int i = 0; i < kMine; ++i) {
                const int r = warp * kMine + i;
                float s = 0.f;
#pragma unroll
                for (int e = 0; e < kWarps; ++e) s += part[(e * ROWS + r) * kKeys + lane];
                s = key <= limit[i] ? s * p.b.scale_log2 : -INFINITY;
                float mx = s;
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
                const float m_new = fmaxf(m[i], mx);
                const float a = m_new == -INFINITY ? 1.f : exp2f(m[i] - m_new);
                const float e = exp2f(s - (m_new == -INFINITY ? 0.f : m_new));
                float sum = e;
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
                m[i] = m_new;
                l[i] = l[i] * a + sum;
                pt[lane * ROWS + r] = e;
                if (lane == 0) alpha[r] = a;
            }
            __syncthreads();
            if (owner) {
#pragma unroll
                for (int i = 0; i < RPT; ++i) {
                    const float a = alpha[rg * RPT + i];
                    acc[i][0] *= a;
                    acc[i][1] *= a;
                }
#pragma unroll 4
                for (int k = 0; k < kKeys; ++k) {
                    const float2 v = *reinterpret_cast<const float2*>(kb + k * pitch + 2 * d2);
                    const float* pk = pt + k * ROWS + rg * RPT;
#pragma unroll
                    for (int i = 0; i < RPT; ++i) {
                        acc[i][0] = fmaf(pk[i], v.x, acc[i][0]);
                        acc[i][1] = fmaf(pk[i], v.y, acc[i][1]);
                    }
                }
            }
            __syncthreads();                               // the buffer may be filled again
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        if (lane == 0) {
#pragma unroll
            for (int i = 0; i < kMine; ++i) {
                const int r = warp * kMine + i;
                row_l[r] = l[i];
                if (!f.whole) p.ws.ml[f.slot * kLatentRowTile + r] = make_float2(m[i], l[i]);
            }
        }
        if (f.starts && tid == 0)
            p.ws.merge[blockIdx.x] = LatentMerge{f.row0, f.nrows, int(blockIdx.x), f.last_cta, f.slot};
        __syncthreads();
        if (owner && f.n > 0) {
            float* part_o = p.ws.o + int64_t(f.slot) * kLatentRowTile * R;
#pragma unroll
            for (int i = 0; i < RPT; ++i) {
                const int r = rg * RPT + i;
                if (r >= f.nrows) continue;
                if (f.whole) {
                    const float inv = 1.f / row_l[r];
                    *reinterpret_cast<float2*>(p.out + (int64_t(f.row0) + r) * R + 2 * d2) =
                        make_float2(acc[i][0] * inv, acc[i][1] * inv);
                } else {
                    *reinterpret_cast<float2*>(part_o + r * R + 2 * d2) = make_float2(acc[i][0], acc[i][1]);
                }
            }
        }
    }
}

template <int ROWS, int RPT>
int launch(const LatentArgs& a, const Params& p) {
    const int smem = smem_floats(a.desc->latent_dim, ROWS) * int(sizeof(float));
    if (kernel_occupancy<latent_f32_kernel<ROWS, RPT>>(kThreads, smem_floats(512, ROWS) * int(sizeof(float))) < 1)
        return PKV_ERR_CUDA;
    cudaError_t e = launch_pdl(latent_f32_kernel<ROWS, RPT>, dim3(num_sms()), dim3(kThreads), size_t(smem),
                               a.stream, p);
    if (e != cudaSuccess) return cuda_status(e);
    return launch_latent_merge<float>(a.stream, p.b, p.ws, p.out, num_sms(), 0);
}

}  // namespace

int launch_latent_f32(const LatentArgs& a) {
    Params p;
    p.b = a.batch;
    p.ws = a.ws;
    p.out = static_cast<float*>(a.out);
    p.q = static_cast<const float*>(a.q);
    p.cache = static_cast<const float*>(a.cache);
    static_assert(smem_floats(512, 16) * 4 <= 232448, "shared memory");
    // rows of a sequence, on average
    const int64_t rows = int64_t(ceil_div(p.b.num_query_tokens, p.b.num_seqs)) * p.b.heads;
    p.b.team = latent_team(p.b, rows <= 8 ? 8 : 16);
    const int groups = std::max(1, kThreads / (p.b.latent / 2));   // threads of one pair of dimensions
    if (rows <= 8)
        return groups == 1 ? launch<8, 8>(a, p) : groups == 2 ? launch<8, 4>(a, p) : launch<8, 2>(a, p);
    return groups == 1 ? launch<16, 16>(a, p) : groups == 2 ? launch<16, 8>(a, p) : launch<16, 4>(a, p);
}

}  // namespace pkv
