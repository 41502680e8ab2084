// Attention over a paged latent cache in single precision, on the CUDA cores.
//
// A CTA of eight warps takes ROWS (token, head) rows of one sequence and tiles of KEYS keys,
// two of them in flight (cp.async).  Tensor cores take no fp32 operands; an fp32 value is the
// sum of three bf16 values, and six to nine such products in place of one would keep its bits,
// which is not built.  So what bounds it beyond a few heads is the FMA rate, and in front of
// it what shared memory returns: 128 bytes a cycle, so that a read of 16 bytes a lane costs a warp
// four cycles even where all lanes read the same, the time of 16 FMAs of a warp.
//   S: warp w holds an eighth of the dimensions of all ROWS x KEYS scores, a lane a part of
//      RT x KT: RT + KT reads for 4 RT KT FMAs (rows against one key of a lane, 17 reads for
//      64 FMAs, ran at 13 TFLOP/s).  The eighths meet in shared memory.
//   O: a thread owns four dimensions of a share of the rows.
// Rows of keys lie four floats further apart than they are long, so that 8 lanes reading 16
// bytes of 8 rows meet no bank twice.
// 8, 16 or 32 rows, the least that covers a sequence's rows: with more, products would be
// for nothing.  32 rows of 512 + 64 dimensions leave room for tiles of 16 keys only.
// Measured: 9 requests of two tokens over up to 3985, 91 heads, latent 384: 180 us (31 TFLOP/s);
// 8 of up to 2048, 8 heads, latent 256: 17.5 us, of which the merge takes 4.5.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "latent_common.cuh"
#include "latent_merge.cuh"
#include "launch_cache.h"

namespace pkv {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kLeastSteps = 1;             // of a CTA (one request of 8000 keys, 8 heads: 18.4 us, with two 21.4)
constexpr int kStart = 1;                  // steps that a unit costs beside its tiles

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

// floats of a row of the eighths: the rows that a warp writes at once begin on different banks
template <int KEYS>
constexpr int kPartPitch = KEYS == 32 ? 40 : 20;

// floats of shared memory: two key tiles, queries, eighths of S, P, alpha
template <int ROWS, int KEYS>
constexpr int smem_floats(int latent) {
    return (2 * KEYS + ROWS) * (latent + kLatentRope + 4) + kWarps * ROWS * kPartPitch<KEYS> +
           KEYS * (ROWS + 4) + 3 * ROWS;
}

// RG: shares of the rows in the second product.
template <int ROWS, int KEYS, int RG>
__global__ void __launch_bounds__(kThreads) latent_f32_kernel(Params p) {
    static_assert(ROWS <= kLatentRowTile, "states");
    constexpr int RPT = ROWS / RG, kPtPitch = ROWS + 4, kPitch = kPartPitch<KEYS>;
    extern __shared__ float4 smem4[];
    float* smem = reinterpret_cast<float*>(smem4);
    const int R = p.b.latent, D = R + kLatentRope, pitch = D + 4;
    float* kt = smem;                                      // [2][KEYS][pitch]
    float* qs = kt + 2 * KEYS * pitch;                     // [ROWS][pitch]
    float* part = qs + ROWS * pitch;                       // [kWarps][ROWS][kPitch]
    float* pt = part + kWarps * ROWS * kPitch;             // [KEYS][kPtPitch]
    float* alpha = pt + KEYS * kPtPitch;                   // [ROWS]
    float* row_m = alpha + ROWS;                           // [ROWS], at the end of a fragment
    float* row_l = row_m + ROWS;
    __shared__ int64_t sums[kWarps + 2];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int vecs = D / 4;

    pdl_wait_prerequisites();
    pdl_launch_dependents();
    LatentWalk<ROWS, KEYS, kStart> w = latent_plan<ROWS, KEYS, kStart, kThreads>(p.b, sums, kLeastSteps, blockIdx.x, gridDim.x);
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
        // a warp loads an eighth of a tile's rows; their block's id is asked for a tile ahead
        constexpr int kLoad = KEYS / kWarps;               // (of one block)
        const int32_t* table = p.b.block_tables + int64_t(f.seq) * p.b.table_stride;
        auto block_of = [&](int j) {
            const int key = (f.kt0 + j) * KEYS + warp * kLoad;
            return j < f.n && key < f.ctx ? __ldg(table + key / kBlockTokens) : 0;
        };
        auto load = [&](int j, int blk) {
            float* dst = kt + ((j & 1) * KEYS + warp * kLoad) * pitch;
            const int key0 = (f.kt0 + j) * KEYS + warp * kLoad;
            const bool good = blk >= 0 && blk < p.b.num_blocks;
            if (!good && lane == 0 && key0 < f.ctx) flag_error(p.b.err, PKV_DEV_BAD_BLOCK_ID);
            const float* src = p.cache + (int64_t(good ? blk : 0) * kBlockTokens + key0 % kBlockTokens) * D;
#pragma unroll
            for (int r = 0; r < kLoad; ++r)
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

        float acc[RPT][4];
#pragma unroll
        for (int i = 0; i < RPT; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
        const int fours = R / 4;
        const int d4 = tid % fours, rg = tid / fours;      // a thread's dimensions and rows
        const bool owner = rg < RG;
        // softmax: KEYS lanes a row, kOnce rows of a warp at once
        constexpr int kOnce = 32 / KEYS, kMine = ROWS / kWarps, kTurns = kMine / kOnce;
        static_assert(kTurns * kOnce == kMine, "rows of a warp");
        const int key_lane = lane % KEYS;
        float m[kTurns], l[kTurns];
        int limit[kTurns];
        auto row_of = [&](int i) { return warp * kMine + i * kOnce + lane / KEYS; };
#pragma unroll
        for (int i = 0; i < kTurns; ++i) {
            m[i] = -INFINITY;
            l[i] = 0.f;
            const int r = row_of(i);
            limit[i] = r < f.nrows ? f.first_pos + f.t0 + (f.rest + r) / p.b.heads : -1;
        }

        for (int j = 0; j < f.n; ++j) {
            if (j + 1 < f.n) load(j + 1, blk);
            blk = block_of(j + 2);
            if (j + 1 < f.n) asm volatile("cp.async.wait_group 1;" ::: "memory");
            else asm volatile("cp.async.wait_group 0;" ::: "memory");
            __syncthreads();
            const float* kb = kt + (j & 1) * KEYS * pitch;
            {
                // lanes: kLr by kLk; a lane's rows kLr apart, its keys kLk apart
                constexpr int kLr = KEYS == 32 ? 4 : 8, kLk = 32 / kLr, RT = ROWS / kLr, KT = KEYS / kLk;
                const int lr = lane / kLk, lk = lane % kLk;
                float s[RT][KT] = {};
                const int c1 = vecs / kWarps;              // (D is a multiple of 32)
                const float* krow = kb + lk * pitch + 4 * warp * c1;
                const float* qrow = qs + lr * pitch + 4 * warp * c1;
#pragma unroll 2
                for (int c = 0; c < c1; ++c) {
                    float4 q[RT], k[KT];
#pragma unroll
                    for (int i = 0; i < RT; ++i) q[i] = *reinterpret_cast<const float4*>(qrow + i * kLr * pitch + 4 * c);
#pragma unroll
                    for (int e = 0; e < KT; ++e) k[e] = *reinterpret_cast<const float4*>(krow + e * kLk * pitch + 4 * c);
#pragma unroll
                    for (int i = 0; i < RT; ++i)
#pragma unroll
                        for (int e = 0; e < KT; ++e)
                            s[i][e] = fmaf(q[i].x, k[e].x, fmaf(q[i].y, k[e].y,
                                          fmaf(q[i].z, k[e].z, fmaf(q[i].w, k[e].w, s[i][e]))));
                }
#pragma unroll
                for (int i = 0; i < RT; ++i)
#pragma unroll
                    for (int e = 0; e < KT; ++e)
                        part[(warp * ROWS + lr + i * kLr) * kPitch + lk + e * kLk] = s[i][e];
            }
            __syncthreads();
            const int key = (f.kt0 + j) * KEYS + key_lane;
#pragma unroll
            for (int i = 0; i < kTurns; ++i) {
                const int r = row_of(i);
                float s = 0.f;
#pragma unroll
                for (int e = 0; e < kWarps; ++e) s += part[(e * ROWS + r) * kPitch + key_lane];
                s = key <= limit[i] ? s * p.b.scale_log2 : -INFINITY;
                float mx = s;
#pragma unroll
                for (int d = KEYS / 2; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
                const float m_new = fmaxf(m[i], mx);
                const float a = m_new == -INFINITY ? 1.f : exp2f(m[i] - m_new);
                const float e = exp2f(s - (m_new == -INFINITY ? 0.f : m_new));
                float sum = e;
#pragma unroll
                for (int d = KEYS / 2; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
                m[i] = m_new;
                l[i] = l[i] * a + sum;
                pt[key_lane * kPtPitch + r] = e;
                if (key_lane == 0) alpha[r] = a;
            }
            __syncthreads();
            if (owner) {
#pragma unroll
                for (int i = 0; i < RPT; ++i) {
                    const float a = alpha[rg * RPT + i];
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[i][e] *= a;
                }
#pragma unroll 8
                for (int k = 0; k < KEYS; ++k) {
                    const float4 v = *reinterpret_cast<const float4*>(kb + k * pitch + 4 * d4);
                    float w[RPT];
                    const float* pk = pt + k * kPtPitch + rg * RPT;
                    if constexpr (RPT % 4 == 0) {
#pragma unroll
                        for (int i = 0; i < RPT; i += 4) {
                            const float4 x = *reinterpret_cast<const float4*>(pk + i);
                            w[i] = x.x; w[i + 1] = x.y; w[i + 2] = x.z; w[i + 3] = x.w;
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < RPT; ++i) w[i] = pk[i];
                    }
#pragma unroll
                    for (int i = 0; i < RPT; ++i) {
                        acc[i][0] = fmaf(w[i], v.x, acc[i][0]);
                        acc[i][1] = fmaf(w[i], v.y, acc[i][1]);
                        acc[i][2] = fmaf(w[i], v.z, acc[i][2]);
                        acc[i][3] = fmaf(w[i], v.w, acc[i][3]);
                    }
                }
            }
            __syncthreads();                               // the buffer may be filled again
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        if (key_lane == 0) {
#pragma unroll
            for (int i = 0; i < kTurns; ++i) {
                const int r = row_of(i);
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
                    *reinterpret_cast<float4*>(p.out + (int64_t(f.row0) + r) * R + 4 * d4) =
                        make_float4(acc[i][0] * inv, acc[i][1] * inv, acc[i][2] * inv, acc[i][3] * inv);
                } else {
                    *reinterpret_cast<float4*>(part_o + r * R + 4 * d4) =
                        make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
                }
            }
        }
    }
}

template <int ROWS, int KEYS, int RG>
int launch(const LatentArgs& a, Params& p) {
    p.b.team = latent_team(p.b, ROWS);
    const int smem = smem_floats<ROWS, KEYS>(a.desc->latent_dim) * int(sizeof(float));
    constexpr int most = RG == 8 ? 128 : RG == 4 ? 256 : ROWS == 32 && KEYS == 32 ? 384 : 512;
    constexpr int limit = smem_floats<ROWS, KEYS>(most) * int(sizeof(float));
    static_assert(limit + (kWarps + 2) * 8 <= 232448, "shared memory");
    if (kernel_occupancy<latent_f32_kernel<ROWS, KEYS, RG>>(kThreads, limit) < 1) return PKV_ERR_CUDA;
    cudaError_t e = launch_pdl(latent_f32_kernel<ROWS, KEYS, RG>, dim3(num_sms()), dim3(kThreads), size_t(smem),
                               a.stream, p);
    if (e != cudaSuccess) return cuda_status(e);
    return launch_latent_merge<float>(a.stream, p.b, p.ws, p.out, num_sms(), 0);
}

// threads of four dimensions: 256 of 32, 64, 96 or 128
template <int ROWS>
int launch_rows(const LatentArgs& a, Params& p) {
    switch (a.desc->latent_dim) {
        case 128: return launch<ROWS, 32, 8>(a, p);
        case 256: return launch<ROWS, 32, 4>(a, p);
        case 384: return launch<ROWS, 32, 2>(a, p);
        default: return launch<ROWS, ROWS == 32 ? 16 : 32, 2>(a, p);
    }
}

}  // namespace

int launch_latent_f32(const LatentArgs& a) {
    Params p;
    p.b = a.batch;
    p.ws = a.ws;
    p.out = static_cast<float*>(a.out);
    p.q = static_cast<const float*>(a.q);
    p.cache = static_cast<const float*>(a.cache);
    const int64_t rows = latent_rows(p.b);
    return rows <= 8 ? launch_rows<8>(a, p) : rows <= 16 ? launch_rows<16>(a, p) : launch_rows<32>(a, p);
}

}  // namespace pkv
