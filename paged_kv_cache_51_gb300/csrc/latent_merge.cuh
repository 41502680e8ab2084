// States of the cut units of a latent attention, joined in the order of their keys:
//   M = max m_i,  out = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i.
//
// One wave of CTAs, launched while the attention still runs.  (Its CTAs want 15 KB each: next to
// an attention CTA there is room for none of them at latent 512 and for one at 256, so that most
// start as the attention's leave; what the early launch hides is the launch.)
// Every CTA lists the cut units for itself; a warp takes 256 values of a unit at a time and asks for the states of several
// CTAs at once, so that what it waits for is one trip to L2 (reading state by state took
// 13 us for 64 requests of 512 to 4096 tokens).  Where there are fewer such items than
// warps, 2, 4 or 8 warps of a CTA share one, each with a share of the states, and meet in
// shared memory.
//
// An item's values lie as the attention left them.  bf16: [4 columns][128 lanes][4], lane
// h * 64 + r being row r and half h of each product's columns (half0 of the first, the
// others of the second); an item is 32 lanes and 8 columns.  fp32: [row][latent]; an item is
// (up to) 256 values of a row.
#pragma once

#include "latent_common.cuh"
#include "launch_cache.h"

namespace pkv {
namespace {

constexpr int kMergeThreads = 256, kMergeWarps = kMergeThreads / 32;
// states in flight a warp and CTAs of an SM: many warps of few states where there are many
// short lists (bf16, 96 requests with 128 heads, the whole call: 125.1 us with 2 and 4, 126.2
// with 4 and 3, 130.5 with 2 and 6), few of many in single precision's small calls (17.5 and 18)
template <typename T>
constexpr int kMergeBatch = sizeof(T) == 4 ? 4 : 2;
template <typename T>
constexpr int kMergeCtas = sizeof(T) == 4 ? 3 : 4;

template <typename T>
__global__ void __launch_bounds__(kMergeThreads, kMergeCtas<T>)
    latent_merge_kernel(LatentBatch b, LatentWorkspace ws, T* out, int ctas, int half0) {
    constexpr bool kWide = sizeof(T) == 4;
    constexpr int kBatch = kMergeBatch<T>;
    __shared__ LatentMerge list[kMergeThreads];
    __shared__ int counts[kMergeWarps], tallest;
    __shared__ float shared[kMergeWarps][10][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int latent = b.latent, team = b.team;
    const int64_t stride = int64_t(kLatentRowTile) * latent;
    const int n0 = 2 * half0, half1 = (latent - n0) / 2;
    pdl_wait_prerequisites();
    pdl_launch_dependents();
    for (int base = 0; base < ctas; base += kMergeThreads) {
        LatentMerge e{};
        if (base + int(threadIdx.x) < ctas) e = ws.merge[base + threadIdx.x];
        const unsigned mask = __ballot_sync(0xffffffffu, e.nrows > 0);
        if (lane == 0) counts[warp] = __popc(mask);
        if (threadIdx.x == 0) tallest = 0;
        __syncthreads();
        int at = __popc(mask & ((1u << lane) - 1)), units = 0;
#pragma unroll
        for (int w = 0; w < kMergeWarps; ++w) {
            if (w < warp) at += counts[w];
            units += counts[w];
        }
        if (e.nrows > 0) {
            list[at] = e;
            atomicMax(&tallest, e.nrows);
        }
        __syncthreads();
        // items of a unit: bf16 quarters of the lanes (rows 0-31 first) by 8 columns, fp32
        // rows by 256 columns
        const int inner = kWide ? (latent + 255) / 256 : tallest > 32 ? 4 : 2;
        const int each = kWide ? tallest * inner : latent / 16 * inner;
        const int items = units * each, all = int(gridDim.x) * kMergeWarps;
        const int share = items * 8 <= all ? 8 : items * 4 <= all ? 4 : items * 2 <= all ? 2 : 1;
        const int per_cta = kMergeWarps / share, mine = warp % share;
        for (int i0 = blockIdx.x * per_cta; i0 < items; i0 += gridDim.x * per_cta) {
            const int item = i0 + warp / share;
            bool live = item < items;
            const int u = live ? item / each : 0, rest = live ? item - u * each : 0;
            const int x = rest / inner, y = rest - x * inner;
            const LatentMerge m = list[u];
            int r, d, from;                // row, first of 8 values in it, and where they lie
            bool second = true;            // the upper four of them
            if (kWide) {
                r = x;
                d = y * 256 + lane * 4;
                from = r * latent + d;
                second = d + 128 < latent;
            } else {
                const int h = y & 1, c = x * 8;
                r = (y >> 1) * 32 + lane;
                d = c < half0 ? h * half0 + c : n0 + h * half1 + c - half0;
                from = (x * 256 + h * 64 + r) * 4;
            }
            live = live && r < m.nrows;
            const float* o0 = ws.o + from;
            constexpr int kSecond = kWide ? 128 : 512;
            float acc[8] = {}, sum = 0.f, big = -INFINITY;
            const int n = (m.last - m.first) / team + 1;
            for (int c0 = mine; live && c0 < n; c0 += kBatch * share) {
                float2 ml[kBatch];
                float4 o[kBatch][2];
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    const int c = c0 + i * share, slot = c == 0 ? m.first_slot : 2 * (m.first + c * team);
                    ml[i] = make_float2(-INFINITY, 0.f);
                    o[i][1] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (c < n) {
                        ml[i] = ws.ml[slot * kLatentRowTile + r];
                        o[i][0] = __ldcg(reinterpret_cast<const float4*>(o0 + slot * stride));
                        if (second) o[i][1] = __ldcg(reinterpret_cast<const float4*>(o0 + slot * stride + kSecond));
                    }
                }
                float top = big;
#pragma unroll
                for (int i = 0; i < kBatch; ++i) top = fmaxf(top, ml[i].x);
                const float a = top == -INFINITY ? 1.f : exp2f(big - top);
                big = top;
                sum *= a;
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[i] *= a;
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    if (!(ml[i].y != 0.f)) continue;      // no visible keys: nothing was written
                    const float w = exp2f(ml[i].x - big);
                    sum += w * ml[i].y;
                    acc[0] += w * o[i][0].x; acc[1] += w * o[i][0].y;
                    acc[2] += w * o[i][0].z; acc[3] += w * o[i][0].w;
                    acc[4] += w * o[i][1].x; acc[5] += w * o[i][1].y;
                    acc[6] += w * o[i][1].z; acc[7] += w * o[i][1].w;
                }
            }
            if (share > 1) {
                float (*mem)[32] = shared[warp];
                mem[8][lane] = sum;
                mem[9][lane] = big;
#pragma unroll
                for (int i = 0; i < 8; ++i) mem[i][lane] = acc[i];
                __syncthreads();
                if (mine == 0) {
                    float top = big;
                    for (int w = 1; w < share; ++w) top = fmaxf(top, shared[warp + w][9][lane]);
                    const float a = top == -INFINITY ? 1.f : exp2f(big - top);
                    sum *= a;
#pragma unroll
                    for (int i = 0; i < 8; ++i) acc[i] *= a;
                    for (int w = 1; w < share; ++w) {
                        const float top_w = shared[warp + w][9][lane], l = shared[warp + w][8][lane];
                        if (!(l != 0.f)) continue;
                        const float f = exp2f(top_w - top);
                        sum += f * l;
#pragma unroll
                        for (int i = 0; i < 8; ++i) acc[i] += f * shared[warp + w][i][lane];
                    }
                }
                __syncthreads();
            }
            if (mine != 0 || !live) continue;
            const float inv = 1.f / sum;
            T* dst = out + (int64_t(m.row0) + r) * latent + d;
            if constexpr (kWide) {
                *reinterpret_cast<float4*>(dst) = make_float4(acc[0] * inv, acc[1] * inv, acc[2] * inv, acc[3] * inv);
                if (second)
                    *reinterpret_cast<float4*>(dst + 128) =
                        make_float4(acc[4] * inv, acc[5] * inv, acc[6] * inv, acc[7] * inv);
            } else {
                *reinterpret_cast<uint4*>(dst) =
                    make_uint4(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv),
                               pack_bf16x2(acc[4] * inv, acc[5] * inv), pack_bf16x2(acc[6] * inv, acc[7] * inv));
            }
        }
        __syncthreads();
    }
}

template <typename T>
int launch_latent_merge(cudaStream_t stream, const LatentBatch& b, const LatentWorkspace& ws, T* out, int ctas,
                        int half0) {
    return cuda_status(launch_pdl(latent_merge_kernel<T>, dim3(kMergeCtas<T> * num_sms()), dim3(kMergeThreads), 0,
                                  stream, b, ws, out, ctas, half0));
}

}  // namespace
}  // namespace pkv
