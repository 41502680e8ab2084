// Attention over a paged latent cache (absorbed form) on the tcgen05 tensor cores.
//
//   S = Q K^T      rows x keys, over the latent_dim + 64 values of a cached row
//   O += P C       rows x latent_dim, C being the first latent_dim values of the same rows
//
// with the online softmax between them (base 2, one pass).  A tile of cached rows is
// staged once in shared memory and is both operands: K-major for the first product,
// and, through another descriptor over the same bytes, MN-major for the second.
//
// Shapes.  A CTA takes 64 (token, head) rows of one sequence and tiles of 64 keys.  A
// product of 64 rows in its plain form runs at half the rate of 128 (measured: 128
// cycles for 64 x 256 x 16, the same as 128 x 256 x 16); the .ws form spreads the
// columns' halves over all 128 TMEM lanes and takes 80, bound by the 10 KB of shared
// memory it reads at 128 bytes a cycle.  O of 512 values then needs 256 TMEM columns
// (in the plain form with 128 rows it would take all 512 and leave none for S).
// A thread of the softmax holds one row's 32 keys (lanes 0-63: the tile's first 32,
// lanes 64-127 the others) and, when O is read, half of the row's values.
//
// Shared memory: 64 query rows (latent 512: 72 KB), two key tiles (144 KB), P (8 KB).
// Rows lie as [8-row group][64-value column][8 rows][128 bytes, swizzled], which one
// TMA box a group fills (9 KB) and whose groups and columns are both evenly spaced,
// as the two descriptors need.
//
// Warps: 0 loads (queries, tiles), 1 issues the products, 2 and 3 zero the rows of
// sequences that the call does not allow, 4-7 are the softmax.  S of the next tile goes
// out while the softmax works on this one; the issuer takes whichever of the two
// products is ready, so a tile that has not landed does not hold back the P C that
// frees the other.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "latent_common.cuh"
#include "launch_cache.h"

namespace pkv {
namespace {

constexpr int kRows = 64;
constexpr int kKeys = 64;
constexpr int kThreads = 256;
constexpr int kSoftWarp0 = 4;
constexpr int kSoftWarps = 4;
constexpr int kLoadWarp = 0;
constexpr int kMmaWarp = 1;
constexpr int kGroups = kKeys / 8;         // 8-row groups of a tile
constexpr int kPBytes = kRows * kKeys * 2;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kSCol = 256;            // S buffers: 32 columns each behind O
constexpr float kRescale = 8.f;            // log2 units: O is rescaled when a row's max grows by more
constexpr int kLeastSteps = 2;             // a CTA takes at least 128 keys

enum {
    B_K_FULL = 0,                          // [tile buffer]
    B_S_FULL = B_K_FULL + 2,               // [S buffer]
    B_S_EMPTY = B_S_FULL + 2,              // [S buffer]: the softmax has loaded it
    B_O_DONE = B_S_EMPTY + 2,              // [tile buffer]: its P C is complete, the buffer is free
    B_P_FULL = B_O_DONE + 2,
    B_Q_FULL,
    B_Q_EMPTY,                             // the fragment's last S is complete
    B_O_EMPTY,                             // the softmax has read the fragment's O
    B_XM,                                  // [row half]: both key halves' maxima are there
    B_SUM = B_XM + 2,                      // [row half]: both key halves' sums are there
    B_DRAIN = B_SUM + 2,
    B_COUNT
};

struct Smem {                              // behind the operands
    uint64_t bars[B_COUNT];
    int64_t sums[kThreads / 32 + 2];
    float xm[2][128];
    float sum[128];
    uint32_t tmem;
    int abort;
};

__device__ __forceinline__ void mma_ws(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t acc) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.ws.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}

struct Params {
    LatentBatch b;
    LatentWorkspace ws;
    __nv_bfloat16* out;
};

using Walk = LatentWalk<kRows, kKeys>;

// The fragments' tiles one after the other, skipping fragments without any.
struct Tiles {
    Walk w;
    LatentFrag f;
    int j;                                 // tile of the fragment
    uint32_t g, k;                         // tiles and fragments (of any tiles) so far
    bool live;
    __device__ void start(const LatentBatch& b, const Walk& from) {
        w = from;
        g = k = 0;
        live = false;
        frag(b);
    }
    __device__ void frag(const LatentBatch& b) {
        j = 0;
        do {
            live = w.next(b, f);
        } while (live && f.n == 0);
    }
    __device__ void next(const LatentBatch& b) {
        ++g;
        if (++j == f.n) {
            ++k;
            frag(b);
        }
    }
};

__global__ void __launch_bounds__(kThreads, 1)
    latent_kernel(const __grid_constant__ CUtensorMap map_kv, const __grid_constant__ CUtensorMap map_q,
                  Params p) {
    extern __shared__ unsigned char smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    unsigned char* smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
    const uint32_t base = smem_u32(smem);
    const int cols = p.b.latent / 64 + 1;                 // 64-value columns of a row
    const uint32_t group = uint32_t(cols) * 1024;         // bytes of an 8-row group
    const uint32_t tile = group * kGroups;
    const uint32_t k_at = base + tile, p_at = base + 3 * tile;
    unsigned char* k_ptr = smem + tile;
    unsigned char* p_ptr = smem + 3 * tile;
    Smem& sh = *reinterpret_cast<Smem*>(smem + 3 * tile + kPBytes);
    uint64_t* bars = sh.bars;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile int* abort_flag = &sh.abort;
    int* err = p.b.err;

    if (threadIdx.x == 0) {
        for (int i = 0; i < B_COUNT; ++i) {
            int n = 1;
            if (i == B_S_EMPTY || i == B_S_EMPTY + 1 || i == B_P_FULL || i == B_O_EMPTY) n = kSoftWarps;
            if (i >= B_XM && i < B_DRAIN) n = 2;
            mbar_init(&bars[i], n);
        }
        sh.abort = 0;
        fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(&sh.tmem)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    pdl_wait_prerequisites();
    pdl_launch_dependents();
    tc_fence_before();
    const Walk plan = latent_plan<kRows, kKeys, kThreads>(p.b, sh.sums, kLeastSteps);
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&sh.tmem);

    if (warp == kLoadWarp) {
        // ---- queries and key tiles: lane i < 8 loads the 8 rows of group i ----
        Tiles t;
        bool ok = true;
        uint32_t q_loads = 0, k_loads = 0;
        for (t.start(p.b, plan); t.live; t.next(p.b)) {
            const int32_t* table = p.b.block_tables + int64_t(t.f.seq) * p.b.table_stride;
            if (t.j == 0) {
                ok = __all_sync(0xffffffffu, t.k == 0 || mbar_wait(&bars[B_Q_EMPTY], (t.k - 1) & 1, err));
                if (!ok || *abort_flag) break;
                const int groups = (t.f.nrows + 7) / 8;
                if (lane == 0) mbar_arrive_expect_tx(&bars[B_Q_FULL], uint32_t(groups) * group);
                ++q_loads;
                __syncwarp();
                if (lane < groups)
                    tc_load_3d(base + uint32_t(lane) * group, &map_q, 0, t.f.row0 + lane * 8, 0,
                               &bars[B_Q_FULL]);
            }
            const int key0 = (t.f.kt0 + t.j) * kKeys;
            const int keys = min(kKeys, t.f.ctx - key0);
            const int groups = (keys + 7) / 8;
            int blk = lane < groups ? __ldg(table + key0 / kBlockTokens + (lane >> 1)) : 0;
            const uint32_t st = t.g & 1;
            ok = __all_sync(0xffffffffu,
                            t.g < 2 || mbar_wait(&bars[B_O_DONE + st], ((t.g - 2) >> 1) & 1, err));
            if (!ok || *abort_flag) break;
            const bool good = lane < groups && blk >= 0 && blk < p.b.num_blocks;
            if (lane < groups && !good) flag_error(err, PKV_DEV_BAD_BLOCK_ID);
            const unsigned mask = __ballot_sync(0xffffffffu, good);
            if (lane == 0) mbar_arrive_expect_tx(&bars[B_K_FULL + st], uint32_t(__popc(mask)) * group);
            ++k_loads;
            __syncwarp();
            if (good)
                tc_load_3d(k_at + st * tile + uint32_t(lane) * group, &map_kv, 0,
                           blk * kBlockTokens + (lane & 1) * 8, 0, &bars[B_K_FULL + st]);
            __syncwarp();
        }
        if (t.live) *abort_flag = 1;
        // never leave with copies in flight
        if (lane == 0) {
            if (q_loads > 0) mbar_wait(&bars[B_Q_FULL], (q_loads - 1) & 1, err);
            for (uint32_t i = 0; i < 2 && i < k_loads; ++i) {
                const uint32_t last = k_loads - 1 - i;
                mbar_wait(&bars[B_K_FULL + (last & 1)], (last >> 1) & 1, err);
            }
        }
        __syncwarp();
    } else if (warp == kMmaWarp) {
        if (lane == 0) {
            // S of tile g goes to S buffer g & 1 and P C of tile g follows it; whichever is
            // ready first goes out, S in front where both are
            const uint32_t idesc_s = tc_idesc(kRows, kKeys, false);
            const int n0 = min(256, p.b.latent), n1 = p.b.latent - n0;
            const uint32_t idesc_o0 = tc_idesc(kRows, n0, true), idesc_o1 = tc_idesc(kRows, n1, true);
            const uint64_t qd = tc_smem_desc(base, 16, group);
            const uint64_t kd = tc_smem_desc(k_at, 16, group);
            const uint64_t vd = tc_smem_desc(k_at, 1024, group);
            const uint64_t pd = tc_smem_desc(p_at, 16, 1024);
            Tiles s, o;
            s.start(p.b, plan);
            o.start(p.b, plan);
            bool ok = true;
            uint64_t t0 = 0;
            uint32_t spins = 0;
            while (o.live && ok) {
                bool moved = false;
                if (s.live && s.g <= o.g + 1 && (s.g < 2 || mbar_test(&bars[B_S_EMPTY + (s.g & 1)], ((s.g - 2) >> 1) & 1)) &&
                    mbar_test(&bars[B_K_FULL + (s.g & 1)], (s.g >> 1) & 1) &&
                    (s.j != 0 || mbar_test(&bars[B_Q_FULL], s.k & 1))) {
                    tc_fence_after();
                    const uint32_t d = tmem + kSCol + (s.g & 1) * 32;
                    const uint64_t k0 = kd + uint64_t((s.g & 1) * (tile >> 4));
                    for (int c = 0; c < cols; ++c) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            mma_ws(d, qd + uint64_t(c * 64 + i * 2), k0 + uint64_t(c * 64 + i * 2),
                                   idesc_s, (c | i) != 0);
                    }
                    tc_commit(&bars[B_S_FULL + (s.g & 1)]);
                    if (s.j == s.f.n - 1) tc_commit(&bars[B_Q_EMPTY]);
                    s.next(p.b);
                    moved = true;
                }
                if (o.g < s.g && mbar_test(&bars[B_P_FULL], o.g & 1) &&
                    (o.j != 0 || o.k == 0 || mbar_test(&bars[B_O_EMPTY], (o.k - 1) & 1))) {
                    tc_fence_after();
                    const uint64_t v0 = vd + uint64_t((o.g & 1) * (tile >> 4));
#pragma unroll
                    for (int i = 0; i < kKeys / 16; ++i) {
                        const uint32_t acc = (o.j | i) != 0;
                        const uint64_t v = v0 + uint64_t(i * 2 * (group >> 4));
                        mma_ws(tmem, pd + uint64_t(i * 2), v, idesc_o0, acc);
                        if (n1 > 0) mma_ws(tmem + 128, pd + uint64_t(i * 2), v + 4 * 64, idesc_o1, acc);
                    }
                    tc_commit(&bars[B_O_DONE + (o.g & 1)]);
                    o.next(p.b);
                    moved = true;
                }
                if (moved) {
                    spins = 0;
                } else if (++spins == 64) {
                    t0 = global_ns();
                } else if (spins > 64 && (spins & 63) == 0 &&
                           (*abort_flag || global_ns() - t0 > kWaitLimitNs)) {
                    if (!*abort_flag) flag_error(err, PKV_DEV_WAIT_TIMEOUT);
                    ok = false;
                }
            }
            if (!ok) *abort_flag = 1;
            tc_commit(&bars[B_DRAIN]);
            mbar_wait(&bars[B_DRAIN], 0, err);
        }
        __syncwarp();
    } else if (warp < kSoftWarp0) {
        // ---- sequences with lengths that the call does not allow: zeros ----
        for (int s = blockIdx.x; s < p.b.num_seqs; s += gridDim.x) {
            const LatentSeq x = latent_seq<false>(p.b, s);
            if (!x.zero) continue;
            const int64_t row_vecs = int64_t(p.b.heads) * p.b.latent / 8;
            uint4* dst = reinterpret_cast<uint4*>(p.out) + int64_t(x.q0) * row_vecs;
            for (int64_t i = (warp - 2) * 32 + lane; i < row_vecs * x.qlen; i += 64)
                dst[i] = make_uint4(0, 0, 0, 0);
        }
    } else {
        // ---- softmax: thread = (row r, key half h) ----
        const int w4 = warp - kSoftWarp0;
        const int r = (w4 & 1) * 32 + lane, h = w4 >> 1;
        const uint32_t lanes = uint32_t(w4 * 32) << 16;
        const int n0 = min(256, p.b.latent);
        const int half0 = n0 / 2, half1 = (p.b.latent - n0) / 2;
        const int ocols = half0 + half1;                  // TMEM columns of O
        Walk w = plan;
        LatentFrag f;
        uint32_t g = 0, k = 0;
        bool ok = true;
        if (int(threadIdx.x) == kSoftWarp0 * 32) p.ws.merge[blockIdx.x].nrows = 0;
        while (w.next(p.b, f)) {
            const int tok = f.t0 + (f.rest + r) / p.b.heads;
            const int limit = r < f.nrows ? f.first_pos + tok : -1;   // last key that the row sees
            float m = -INFINITY, l = 0.f;
            for (int j = 0; j < f.n; ++j, ++g) {
                ok = __all_sync(0xffffffffu, mbar_wait(&bars[B_S_FULL + (g & 1)], (g >> 1) & 1, err));
                if (!ok) break;
                tc_fence_after();
                float s[32];
                {
                    uint32_t v[32];
                    tc_ld32(tmem + lanes + kSCol + (g & 1) * 32, v);
                    tc_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i) s[i] = __uint_as_float(v[i]) * p.b.scale_log2;
                }
                const int key0 = (f.kt0 + j) * kKeys;
                const int khalf = key0 + h * 32;
                if (khalf + 31 > limit) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) s[i] = khalf + i <= limit ? s[i] : -INFINITY;
                }
                float mx4[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) mx4[i] = fmaxf(s[i], s[i + 4]);
#pragma unroll
                for (int i = 8; i < 32; ++i) mx4[i & 3] = fmaxf(mx4[i & 3], s[i]);
                const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
                // the row's other key half is the same lane of the warp two on
                sh.xm[g & 1][h * 64 + r] = mx;
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&bars[B_XM + (w4 & 1)]);
                    mbar_arrive(&bars[B_S_EMPTY + (g & 1)]);
                }
                ok = __all_sync(0xffffffffu, mbar_wait(&bars[B_XM + (w4 & 1)], g & 1, err));
                if (!ok) break;
                const float m_new = fmaxf(m, fmaxf(mx, sh.xm[g & 1][(h ^ 1) * 64 + r]));
                const bool need = m_new > m + kRescale;   // first visible keys included
                float alpha = 1.f;
                if (need) {
                    alpha = exp2_fast(m - m_new);
                    m = m_new;
                    l *= alpha;
                }
                // P in bf16: 2^-8 of a weight at most; the sum is taken of the same rounded
                // weights, so that what is lost does not shift the weighted mean
                const float neg_m = m == -INFINITY ? 0.f : -m;
                uint32_t pk[16];
                float sum[2] = {0.f, 0.f};
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    pk[i] = pack_bf16x2(exp2_fast(s[2 * i] + neg_m), exp2_fast(s[2 * i + 1] + neg_m));
                    sum[0] += __uint_as_float(pk[i] << 16);
                    sum[1] += __uint_as_float(pk[i] & 0xffff0000u);
                }
                l += sum[0] + sum[1];
                // the previous tile's P C reads P and O
                if (g > 0) {
                    ok = __all_sync(0xffffffffu, mbar_wait(&bars[B_O_DONE + ((g - 1) & 1)],
                                                           ((g - 1) >> 1) & 1, err));
                    if (!ok) break;
                }
                tc_fence_after();
                if (j > 0 && __any_sync(0xffffffffu, need)) {
                    for (int c = 0; c < ocols; c += 32) {
                        uint32_t v[32];
                        const uint32_t at = tmem + lanes + (c < half0 ? c : 128 + c - half0);
                        tc_ld32(at, v);
                        tc_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * alpha);
                        tc_st32(at, v);
                    }
                    tc_wait_st();
                }
                unsigned char* row = p_ptr + r * 128;
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    *reinterpret_cast<uint4*>(row + (((h * 4 + c) ^ (r & 7)) * 16)) =
                        make_uint4(pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]);
                // rows behind the context hold another tile's or nothing: their values are
                // zeroed, since 0 times anything must stay 0
                const int keys = f.ctx - key0;
                if (keys < kKeys) {
                    unsigned char* ks = k_ptr + (g & 1) * tile;
                    const int vecs = cols * 8;             // 16-byte vectors of a row
                    for (int i = w4 * 32 + lane; i < (kKeys - keys) * vecs; i += 128) {
                        const int row_i = keys + i / vecs, c = i % vecs;
                        *reinterpret_cast<uint4*>(ks + uint32_t(row_i >> 3) * group + (c >> 3) * 1024 +
                                                  (row_i & 7) * 128 + (c & 7) * 16) =
                            make_uint4(0, 0, 0, 0);
                    }
                }
                fence_proxy_async_shared();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[B_P_FULL]);
            }
            if (!ok) break;
            // ---- the fragment's output or state ----
            if (f.n > 0) {
                ok = __all_sync(0xffffffffu, mbar_wait(&bars[B_O_DONE + ((g - 1) & 1)],
                                                       ((g - 1) >> 1) & 1, err));
                if (!ok) break;
                tc_fence_after();
                sh.sum[h * 64 + r] = l;
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[B_SUM + (w4 & 1)]);
                ok = __all_sync(0xffffffffu, mbar_wait(&bars[B_SUM + (w4 & 1)], k & 1, err));
                if (!ok) break;
                l += sh.sum[(h ^ 1) * 64 + r];
            }
            if (!f.whole && h == 0) p.ws.ml[f.slot * kLatentRowTile + r] = make_float2(m, l);
            if (f.starts && int(threadIdx.x) == kSoftWarp0 * 32)
                p.ws.merge[blockIdx.x] = LatentMerge{f.row0, f.nrows, int(blockIdx.x), f.last_cta, f.slot};
            if (f.n > 0) {
                const float inv = 1.f / l;
                __nv_bfloat16* dst = p.out + int64_t(f.row0 + r) * p.b.latent;
                float* part = p.ws.o + int64_t(f.slot) * kLatentRowTile * p.b.latent;
                for (int c = 0; c < ocols; c += 32) {
                    uint32_t v[32];
                    tc_ld32(tmem + lanes + (c < half0 ? c : 128 + c - half0), v);
                    tc_wait_ld();
                    if (f.whole) {
                        if (r < f.nrows) {
                            const int d = c < half0 ? h * half0 + c : n0 + h * half1 + c - half0;
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                uint32_t o[4];
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    o[e] = pack_bf16x2(__uint_as_float(v[8 * i + 2 * e]) * inv,
                                                       __uint_as_float(v[8 * i + 2 * e + 1]) * inv);
                                *reinterpret_cast<uint4*>(dst + d + 8 * i) = make_uint4(o[0], o[1], o[2], o[3]);
                            }
                        }
                    } else {
                        // [4 columns][lane]: a warp writes 512 bytes in a row
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            *reinterpret_cast<uint4*>(part + ((c / 4 + i) * 128 + h * 64 + r) * 4) =
                                make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[B_O_EMPTY]);
                ++k;
            }
        }
        if (!ok) *abort_flag = 1;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols)
                     : "memory");
}

// States of a cut unit, joined in the order of its keys:
//   M = max m_i,  out = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i.
// CTA (i, y): merge i, 8 values of each lane y holds.  A thread reads its values of every
// state (16 bytes, neighbours side by side) and writes 16 bytes of a row.
__global__ void __launch_bounds__(128) latent_merge_kernel(Params p) {
    pdl_wait_prerequisites();
    const LatentMerge e = p.ws.merge[blockIdx.x];
    const int r = threadIdx.x & 63, h = threadIdx.x >> 6;
    if (r >= e.nrows) return;
    float big = -INFINITY;
    for (int c = e.first; c <= e.last; ++c)
        big = fmaxf(big, p.ws.ml[(c == e.first ? e.first_slot : 2 * c) * kLatentRowTile + r].x);
    float acc[8] = {}, sum = 0.f;
    const int64_t stride = int64_t(kLatentRowTile) * p.b.latent;
    const int at = (blockIdx.y * 2 * 128 + threadIdx.x) * 4;
    for (int c = e.first; c <= e.last; ++c) {
        const int slot = c == e.first ? e.first_slot : 2 * c;
        const float2 ml = p.ws.ml[slot * kLatentRowTile + r];
        if (!(ml.y != 0.f)) continue;                     // no visible keys: nothing was written
        const float w = exp2f(ml.x - big);
        sum += w * ml.y;
        const float* o = p.ws.o + slot * stride + at;
        const float4 a = *reinterpret_cast<const float4*>(o), b = *reinterpret_cast<const float4*>(o + 512);
        acc[0] += w * a.x; acc[1] += w * a.y; acc[2] += w * a.z; acc[3] += w * a.w;
        acc[4] += w * b.x; acc[5] += w * b.y; acc[6] += w * b.z; acc[7] += w * b.w;
    }
    const float inv = 1.f / sum;
    const int n0 = min(256, p.b.latent), half0 = n0 / 2, half1 = (p.b.latent - n0) / 2;
    const int c = blockIdx.y * 8;
    const int d = c < half0 ? h * half0 + c : n0 + h * half1 + c - half0;
    uint4 v;
    v.x = pack_bf16x2(acc[0] * inv, acc[1] * inv);
    v.y = pack_bf16x2(acc[2] * inv, acc[3] * inv);
    v.z = pack_bf16x2(acc[4] * inv, acc[5] * inv);
    v.w = pack_bf16x2(acc[6] * inv, acc[7] * inv);
    *reinterpret_cast<uint4*>(p.out + int64_t(e.row0 + r) * p.b.latent + d) = v;
}

}  // namespace

int launch_latent_bf16(const LatentArgs& a) {
    const pkv_latent_desc* d = a.desc;
    const int cols = d->latent_dim / 64 + 1;
    CUtensorMap kv, q;
    if (!make_latent_tensor_map(&kv, a.cache, int64_t(d->num_blocks) * kBlockTokens, cols, 8) ||
        !make_latent_tensor_map(&q, a.q, int64_t(a.batch.num_query_tokens) * d->num_q_heads, cols, 8))
        return PKV_ERR_CUDA;
    Params p;
    p.b = a.batch;
    p.ws = a.ws;
    p.out = static_cast<__nv_bfloat16*>(a.out);
    const int smem = 3 * kGroups * cols * 1024 + kPBytes + int(sizeof(Smem)) + 1024;
    static_assert(3 * kGroups * 9 * 1024 + kPBytes + sizeof(Smem) + 1024 <= 232448, "shared memory");
    // one limit for all latent_dims
    if (kernel_occupancy<latent_kernel>(kThreads, 232448) < 1) return PKV_ERR_CUDA;
    cudaError_t e = launch_pdl(latent_kernel, dim3(num_sms()), dim3(kThreads), size_t(smem), a.stream, kv,
                               q, p);
    if (e != cudaSuccess) return cuda_status(e);
    return cuda_status(launch_pdl(latent_merge_kernel, dim3(num_sms(), d->latent_dim / 16), dim3(128), 0,
                                  a.stream, p));
}

}  // namespace pkv
