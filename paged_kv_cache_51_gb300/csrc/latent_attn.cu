// Attention over a paged latent cache (absorbed form) on the tcgen05 tensor cores.
//
//   S = Q K^T      rows x keys, over the latent_dim + 64 values of a cached row
//   O += P C       rows x latent_dim, C being the first latent_dim values of the same rows
//
// with the online softmax between them (base 2, one pass).  A tile of cached rows is
// staged once in shared memory and is both operands: K-major for the first product,
// and, through another descriptor over the same bytes, MN-major for the second.
//
// Shapes.  A CTA takes 64 (token, head) rows of one sequence and tiles of 32 keys (batches of
// more rows a sequence on average go to pairs of CTAs, latent_pair.cu; a sequence of more rows
// in a batch of few is several units here).
// Products of this size are bound by the shared memory they read (128 bytes a cycle;
// measured, in cycles: 64 x 32 x 16 takes 24, 64 x 64 x 16 32, 64 x 256 x 16 80 in the .ws
// form, which spreads the halves of the columns over all 128 TMEM lanes, and 128 in the
// plain form): a tile's S takes 864 and its P C 320, of the 1575 that an SM's share of HBM
// needs for its 36 KB.  64-key tiles take 896 in all, but only two of them fit beside the
// queries (72 KB of 227): with two buffers that are empty at about the same time the SM
// computes on both while nothing is being loaded, and 4 x 32k keys took 40 us instead of 31.
//
// S (plain form: row 16 w + i in lane 32 w + i) is read with the 16x256b shape, so a
// thread holds 8 keys of two rows and four threads share a row.  O (.ws form: row r in
// lanes r and 64 + r, a half of the columns each) is read a lane a thread.  The two meet
// only where O has to be rescaled, which the warps tell one another through shared memory.
//
// Shared memory: the query rows (latent 512: 72 KB for 64 rows, less for fewer), as many
// tile buffers as fit (4 to 8), two P buffers (4 KB each).  Rows lie as [8-row group]
// [64-value column][8 rows][128 bytes, swizzled], which one TMA box a group fills (9 KB)
// and whose groups and columns are both evenly spaced, as the two descriptors need.
//
// Warps: 0 loads (queries, tiles), 1 issues S, 2 P C, 3 zeroes the rows of sequences that
// the call does not allow, 4-7 are the softmax.  (One thread that issued both took 1727
// cycles a tile, 450 of them its own waits and bookkeeping between the two.)
//
// Measured, with the merge: 4 requests of 32k tokens, 64 heads, 42 us; 64 of 512 to 4096, 32
// heads, 45 us.  The tiles run at HBM's rate, 1650 cycles each; a start of 5 us, outputs of
// 2.5 and the merge of 6 are the rest.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "latent_common.cuh"
#include "latent_merge.cuh"
#include "launch_cache.h"

namespace pkv {
namespace {

constexpr int kRows = 64;
static_assert(kRows == kLatentRowTile, "states");
constexpr int kKeys = 32;
constexpr int kThreads = 256;
constexpr int kSoftWarp0 = 4;
constexpr int kSoftWarps = 4;
constexpr int kLoadWarp = 0;
constexpr int kMmaWarp = 1;                // S; owns TMEM
constexpr int kPcWarp = 2;                 // P C
constexpr int kGroups = kKeys / 8;         // 8-row groups of a tile
constexpr int kPBytes = 2 * kRows * kKeys * 2;
constexpr int kSBufs = 4;
constexpr int kMostSlots = 8;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kSCol = 256;            // S buffers: 32 columns each behind O
constexpr float kRescale = 8.f;            // log2 units: O is rescaled when a row's max grows by more
constexpr int kLeastSteps = 4;             // of a CTA
constexpr int kStart = 4;                  // steps that a unit costs beside its tiles

enum {
    B_K_FULL = 0,                          // [tile buffer]
    B_O_DONE = B_K_FULL + kMostSlots,      // [tile buffer]: its P C is complete, the buffer is free
    B_S_FULL = B_O_DONE + kMostSlots,      // [S buffer]
    B_S_EMPTY = B_S_FULL + kSBufs,         // [S buffer]: the softmax has loaded it
    B_P_FULL = B_S_EMPTY + kSBufs,         // [P buffer]
    B_Q_FULL = B_P_FULL + 2,
    B_Q_EMPTY,                             // the fragment's last S is complete
    B_O_EMPTY,                             // the softmax has read the fragment's O
    B_NEED,                                // every warp has said whether its rows' O is rescaled
    B_SUM,                                 // the rows' sums are there
    B_DRAIN,                               // [issuer]
    B_COUNT = B_DRAIN + 2
};

struct Smem {                              // behind the operands
    uint64_t bars[B_COUNT];
    int64_t sums[kThreads / 32 + 2];
    float alpha[2][kRows];                 // [tile parity]
    uint8_t need[2][kSoftWarps];
    float m[kRows], l[kRows];              // at the end of a fragment
    uint32_t tmem;
    int abort;
};

// A place in the ring of tile buffers: tile g is in buffer g % slots.
struct Ring {
    uint32_t slot = 0, phase = 0;
    __device__ void next(uint32_t slots) {
        if (++slot == slots) {
            slot = 0;
            phase ^= 1;
        }
    }
};

__device__ __forceinline__ void mma_ws(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t acc) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.ws.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}

__device__ __forceinline__ void mma_plain(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                          uint32_t acc) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
// 16 lanes x 32 columns: register 4 i + e of lane t is row t / 4 + 8 (e / 2), column
// 8 i + 2 (t % 4) + e % 2
__device__ __forceinline__ void tc_ld_16x32(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15},"
        " [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
          "=r"(r[15])
        : "r"(taddr));
}

struct Params {
    LatentBatch b;
    LatentWorkspace ws;
    __nv_bfloat16* out;
    int32_t q_groups;                      // 8-row groups of the query buffer
    int32_t slots;
    bool whole_sectors;                    // out begins on 32 bytes
};

using Walk = LatentWalk<kRows, kKeys, kStart>;

using Tiles = LatentTiles<kRows, kKeys, kStart>;

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
    const uint32_t slots = uint32_t(p.slots);
    // P first: the products read 64 query rows whatever the buffer holds, and then what
    // lies behind it, which is still shared memory (the tile buffers)
    const uint32_t p_at = base, q_at = base + kPBytes;
    const uint32_t k_off = kPBytes + uint32_t(p.q_groups) * group, k_at = base + k_off;
    unsigned char* p_ptr = smem;
    unsigned char* k_ptr = smem + k_off;
    Smem& sh = *reinterpret_cast<Smem*>(k_ptr + slots * tile);
    uint64_t* bars = sh.bars;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile int* abort_flag = &sh.abort;
    int* err = p.b.err;

    if (threadIdx.x == 0) {
        for (int i = 0; i < B_COUNT; ++i) {
            int n = 1;
            if (i >= B_S_EMPTY && i < B_Q_FULL) n = kSoftWarps;
            if (i == B_O_EMPTY || i == B_NEED || i == B_SUM) n = kSoftWarps;
            mbar_init(&bars[i], n);
        }
        sh.abort = 0;
        fence_mbar_init();
    }
    // Tensor memory is taken behind the wait, and the next kernel let in behind the plan's
    // barriers: a kernel that held it while it waited for one that has yet to take its own
    // would wait for ever where their CTAs share an SM.
    pdl_wait_prerequisites();
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(&sh.tmem)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    const Walk plan = latent_plan<kRows, kKeys, kStart, kThreads>(p.b, sh.sums, kLeastSteps, blockIdx.x, gridDim.x);
    pdl_launch_dependents();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&sh.tmem);

    if (warp == kLoadWarp) {
        // ---- queries and key tiles: lane i < 4 loads the 8 rows of group i ----
        Tiles t;
        Ring at;
        bool ok = true;
        uint32_t q_loads = 0, k_loads = 0;
        for (t.start(p.b, plan); t.live; t.next(p.b)) {
            const int32_t* table = p.b.block_tables + int64_t(t.f.seq) * p.b.table_stride;
            const int key0 = (t.f.kt0 + t.j) * kKeys;
            const int groups = (min(kKeys, t.f.ctx - key0) + 7) / 8;
            const int blk = lane < groups ? __ldg(table + key0 / kBlockTokens + (lane >> 1)) : 0;
            if (t.j == 0) {
                const bool stop = *abort_flag;             // (lanes may read it before and after it is set)
                ok = __all_sync(0xffffffffu, !stop && (t.k == 0 || mbar_wait_asleep(&bars[B_Q_EMPTY],
                                                                                 (t.k - 1) & 1, err)));
                if (!ok) break;
                const int rows = (t.f.nrows + 7) / 8;
                if (lane == 0) mbar_arrive_expect_tx(&bars[B_Q_FULL], uint32_t(rows) * group);
                ++q_loads;
                __syncwarp();
                if (lane < rows)
                    tc_load_3d(q_at + uint32_t(lane) * group, &map_q, 0, t.f.row0 + lane * 8, 0,
                               &bars[B_Q_FULL]);
            }
            const bool good = lane < groups && blk >= 0 && blk < p.b.num_blocks;
            if (lane < groups && !good) flag_error(err, PKV_DEV_BAD_BLOCK_ID);
            const unsigned mask = __ballot_sync(0xffffffffu, good);
            uint64_t* full = &bars[B_K_FULL + at.slot];
            const bool stop = *abort_flag;
            ok = __all_sync(0xffffffffu, !stop && (t.g < slots || mbar_wait_asleep(&bars[B_O_DONE + at.slot],
                                                                             at.phase ^ 1, err)));
            if (!ok) break;
            ++k_loads;
#ifdef PKV_TEST_SKIP_TILE
            // wait-timeout test build only: neither copied nor expected, so that the waits for
            // this tile run out (no copy is in flight for it at any time).  Its place in the ring
            // has been waited for like any other's: a loader a lap ahead would arrive on a
            // barrier whose phase is not over
            if (t.g == uint32_t(PKV_TEST_SKIP_TILE)) {
                at.next(slots);
                continue;
            }
#endif
            if (lane == 0) mbar_arrive_expect_tx(full, uint32_t(__popc(mask)) * group);
            __syncwarp();
            if (good)
                tc_load_3d(k_at + at.slot * tile + uint32_t(lane) * group, &map_kv, 0,
                           blk * kBlockTokens + (lane & 1) * 8, 0, full);
            __syncwarp();
            at.next(slots);
        }
        if (t.live) *abort_flag = 1;
        // never leave with copies in flight
        if (lane == 0) {
            if (q_loads > 0) mbar_wait_asleep(&bars[B_Q_FULL], (q_loads - 1) & 1, err);
            for (uint32_t i = 0; i < slots && i < k_loads; ++i) {
                const uint32_t last = k_loads - 1 - i;
                mbar_wait_asleep(&bars[B_K_FULL + last % slots], (last / slots) & 1, err);
            }
        }
        __syncwarp();
    } else if (warp == kMmaWarp) {
        if (elect_one()) {
            constexpr uint32_t idesc = tc_idesc(kRows, kKeys, false);
            const uint64_t qd = tc_smem_desc(q_at, 16, group);
            const uint64_t kd = tc_smem_desc(k_at, 16, group);
            // The pipe idles for whatever this thread does between two tiles beyond the other
            // issuer's products, so the next tile's barriers are tested before this one's
            // last products go out and the answer is looked at behind them.
            Tiles t;
            Ring at;
            bool ok = true, ready = false;
            for (t.start(p.b, plan); t.live; t.next(p.b)) {
                const uint32_t sb = t.g & (kSBufs - 1);
                const uint32_t d = tmem + kSCol + sb * 32;
                const uint64_t k0 = kd + uint64_t(at.slot * (tile >> 4));
                if (t.j == 0) ok = !*abort_flag && mbar_wait_asleep(&bars[B_Q_FULL], t.k & 1, err);
                if (!ready)
                    ok = ok &&
                         (t.g < kSBufs || mbar_wait_asleep(&bars[B_S_EMPTY + sb], ((t.g / kSBufs) & 1) ^ 1, err)) &&
                         mbar_wait_asleep(&bars[B_K_FULL + at.slot], at.phase, err);
                if (!ok) break;
                tc_fence_after();
                uint64_t qa = qd, ka = k0;
                for (int c = 0; c < cols - 1; ++c, qa += 64, ka += 64) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) mma_plain(d, qa + uint64_t(i * 2), ka + uint64_t(i * 2), idesc,
                                                          (c | i) != 0);
                }
                at.next(slots);
                const uint32_t nb = (t.g + 1) & (kSBufs - 1);
                ready = mbar_test2(&bars[B_K_FULL + at.slot], at.phase, &bars[B_S_EMPTY + nb],
                                   (((t.g + 1) / kSBufs) & 1) ^ 1) && t.g + 1 >= kSBufs;
#pragma unroll
                for (int i = 0; i < 4; ++i) mma_plain(d, qa + uint64_t(i * 2), ka + uint64_t(i * 2), idesc, 1);
                tc_commit(&bars[B_S_FULL + sb]);
                if (t.j == t.f.n - 1) tc_commit(&bars[B_Q_EMPTY]);
            }
            if (t.live) *abort_flag = 1;
            tc_commit(&bars[B_DRAIN]);
            mbar_wait_asleep(&bars[B_DRAIN], 0, err);
        }
        __syncwarp();
    } else if (warp == kPcWarp) {
        if (elect_one()) {
            const int n0 = min(256, p.b.latent), n1 = p.b.latent - n0;
            const uint32_t idesc0 = tc_idesc(kRows, n0, true), idesc1 = tc_idesc(kRows, n1, true);
            const uint64_t vd = tc_smem_desc(k_at, 1024, group);
            const uint64_t pd = tc_smem_desc(p_at, 16, 1024);
            Tiles t;
            Ring at;
            bool ok = true;
            for (t.start(p.b, plan); t.live; t.next(p.b)) {
                const uint64_t v0 = vd + uint64_t(at.slot * (tile >> 4));
                const uint64_t p0 = pd + uint64_t((t.g & 1) * 4);
                if (t.j == 0)
                    ok = !*abort_flag && (t.k == 0 || mbar_wait_asleep(&bars[B_O_EMPTY], (t.k - 1) & 1, err));
                ok = ok && mbar_wait_asleep(&bars[B_P_FULL + (t.g & 1)], (t.g >> 1) & 1, err);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int i = 0; i < kKeys / 16; ++i) {
                    const uint32_t acc = (t.j | i) != 0;
                    const uint64_t v = v0 + uint64_t(i * 2 * (group >> 4));
                    mma_ws(tmem, p0 + uint64_t(i * 2), v, idesc0, acc);
                    if (n1 > 0) mma_ws(tmem + 128, p0 + uint64_t(i * 2), v + 4 * 64, idesc1, acc);
                }
                tc_commit(&bars[B_O_DONE + at.slot]);
                at.next(slots);
            }
            if (t.live) *abort_flag = 1;
            tc_commit(&bars[B_DRAIN + 1]);
            mbar_wait_asleep(&bars[B_DRAIN + 1], 0, err);
        }
        __syncwarp();
    } else if (warp < kSoftWarp0) {
        // ---- sequences with lengths that the call does not allow: zeros ----
        for (int s = blockIdx.x; s < p.b.num_seqs; s += gridDim.x) {
            const LatentSeq x = latent_seq<false>(p.b, s);
            if (!x.zero) continue;
            const int64_t row_vecs = int64_t(p.b.heads) * p.b.latent / 8;
            uint4* dst = reinterpret_cast<uint4*>(p.out) + int64_t(x.q0) * row_vecs;
            for (int64_t i = lane; i < row_vecs * x.qlen; i += 32)
                dst[i] = make_uint4(0, 0, 0, 0);
        }
    } else {
        // ---- softmax: thread = 8 keys of rows ra and ra + 8 ----
        const int w4 = warp - kSoftWarp0;
        const int ra = w4 * 16 + (lane >> 2), quad = lane & 3;
        const uint32_t lanes = uint32_t(w4 * 32) << 16;
        // O: row r, half h of the columns of each product
        const int r = (w4 & 1) * 32 + lane, h = w4 >> 1;
        const int n0 = min(256, p.b.latent);
        const int half0 = n0 / 2, half1 = (p.b.latent - n0) / 2;
        const int ocols = half0 + half1;                  // TMEM columns of O
        Walk w = plan;
        LatentFrag f;
        uint32_t g = 0, k = 0;
        Ring at, prev, prev2;                             // tiles g, g - 1 and g - 2
        bool ok = true;
        if (int(threadIdx.x) == kSoftWarp0 * 32) p.ws.merge[blockIdx.x].nrows = 0;
        while (w.next(p.b, f)) {
            int limit[2];                                 // last key that the row sees
            float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int row = ra + 8 * e;
                limit[e] = f.first_pos + f.t0 + (f.rest + min(row, f.nrows - 1)) / p.b.heads;
            }
            for (int j = 0; j < f.n; ++j, ++g) {
                const uint32_t sb = g & (kSBufs - 1);
                // (that the P buffer is free, the tile before the last, is nearly always so)
                const bool free = g < 2 || mbar_test(&bars[B_O_DONE + prev2.slot], prev2.phase);
                ok = mbar_wait_asleep(&bars[B_S_FULL + sb], (g / kSBufs) & 1, err);
                __syncwarp();
                tc_fence_after();
                float s[16];
                {
                    uint32_t v[16];
                    tc_ld_16x32(tmem + lanes + kSCol + sb * 32, v);
                    tc_wait_ld();
#pragma unroll
                    for (int i = 0; i < 16; ++i) s[i] = __uint_as_float(v[i]);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[B_S_EMPTY + sb]);
                const int key0 = (f.kt0 + j) * kKeys;
                if (key0 + kKeys - 1 > min(limit[0], limit[1])) {
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        s[i] = key0 + 8 * (i >> 2) + 2 * quad + (i & 1) <= limit[(i >> 1) & 1] ? s[i] : -INFINITY;
                }
                float alpha[2], neg_m[2];
                bool need = false;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float mx = fmaxf(s[2 * e], s[2 * e + 1]);
#pragma unroll
                    for (int i = 1; i < 4; ++i) mx = fmaxf(mx, fmaxf(s[4 * i + 2 * e], s[4 * i + 2 * e + 1]));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                    const float m_new = fmaxf(m[e], mx * p.b.scale_log2);
                    alpha[e] = 1.f;
                    if (m_new > m[e] + kRescale) {         // first visible keys included
                        alpha[e] = exp2_fast(m[e] - m_new);
                        m[e] = m_new;
                        l[e] *= alpha[e];
                        need = true;
                    }
                    neg_m[e] = m[e] == -INFINITY ? 0.f : -m[e];
                }
                // O has nothing to rescale in a fragment's first tile
                const bool tell = j > 0 && __any_sync(0xffffffffu, need);
                if (tell && quad == 0) {
                    sh.alpha[g & 1][ra] = alpha[0];
                    sh.alpha[g & 1][ra + 8] = alpha[1];
                }
                if (lane == 0) sh.need[g & 1][w4] = tell;
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[B_NEED]);
                // P in bf16: 2^-8 of a weight at most; the sum is taken of the same rounded
                // weights, so that what is lost does not shift the weighted mean
                uint32_t pk[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int e = i & 1;
                    pk[i] = pack_bf16x2(exp2_fast(fmaf(s[2 * i], p.b.scale_log2, neg_m[e])),
                                        exp2_fast(fmaf(s[2 * i + 1], p.b.scale_log2, neg_m[e])));
                    l[e] += __uint_as_float(pk[i] << 16) + __uint_as_float(pk[i] & 0xffff0000u);
                }
                if (!free) ok = mbar_wait_asleep(&bars[B_O_DONE + prev2.slot], prev2.phase, err) && ok;
                // (row & 7) is lane / 4 for both rows
                unsigned char* row = p_ptr + ra * 128 + quad * 4;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int c = ((((g & 1) * 4 + i) ^ (lane >> 2)) * 16);
                    *reinterpret_cast<uint32_t*>(row + c) = pk[2 * i];
                    *reinterpret_cast<uint32_t*>(row + 8 * 128 + c) = pk[2 * i + 1];
                }
                // rows behind the context hold another tile's or nothing: their values are
                // zeroed, since 0 times anything must stay 0
                const int keys = f.ctx - key0;
                if (keys < kKeys) {
                    unsigned char* ks = k_ptr + at.slot * tile;
                    const int vecs = cols * 8;             // 16-byte vectors of a row
                    for (int i = w4 * 32 + lane; i < (kKeys - keys) * vecs; i += 128) {
                        const int row_i = keys + i / vecs, c = i % vecs;
                        *reinterpret_cast<uint4*>(ks + uint32_t(row_i >> 3) * group + (c >> 3) * 1024 +
                                                  (row_i & 7) * 128 + (c & 7) * 16) =
                            make_uint4(0, 0, 0, 0);
                    }
                }
                fence_proxy_async_shared();
                ok = __all_sync(0xffffffffu, mbar_wait_asleep(&bars[B_NEED], g & 1, err) && ok);
                if (!ok) break;
                const uint32_t any = *reinterpret_cast<const volatile uint32_t*>(sh.need[g & 1]);
                if (any) {
                    // the previous tile's P C adds to O
                    ok = __all_sync(0xffffffffu, mbar_wait_asleep(&bars[B_O_DONE + prev.slot], prev.phase, err));
                    if (!ok) break;
                    tc_fence_after();
                    const float a = (any >> (8 * (r >> 4))) & 0xff ? sh.alpha[g & 1][r] : 1.f;
                    for (int c = 0; c < ocols; c += 32) {
                        uint32_t v[32];
                        const uint32_t to = tmem + lanes + (c < half0 ? c : 128 + c - half0);
                        tc_ld32(to, v);
                        tc_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * a);
                        tc_st32(to, v);
                    }
                    tc_wait_st();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[B_P_FULL + (g & 1)]);
                prev2 = prev;
                prev = at;
                at.next(slots);
            }
            if (!ok) break;
            // ---- the fragment's output or state ----
            float mr = -INFINITY, lr = 0.f;                // of row r
            if (f.n > 0) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
                    l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
                    if (quad == 0) {
                        sh.m[ra + 8 * e] = m[e];
                        sh.l[ra + 8 * e] = l[e];
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[B_SUM]);
                ok = __all_sync(0xffffffffu, mbar_wait_asleep(&bars[B_O_DONE + prev.slot], prev.phase, err) &&
                                                 mbar_wait_asleep(&bars[B_SUM], k & 1, err));
                if (!ok) break;
                tc_fence_after();
                mr = sh.m[r];
                lr = sh.l[r];
            }
            if (!f.whole && h == 0) p.ws.ml[f.slot * kLatentRowTile + r] = make_float2(mr, lr);
            if (f.starts && int(threadIdx.x) == kSoftWarp0 * 32)
                p.ws.merge[blockIdx.x] = LatentMerge{f.row0, f.nrows, int(blockIdx.x), f.last_cta, f.slot};
            __syncwarp();                                  // the TMEM reads want all lanes at once
            if (f.n > 0) {
                const float inv = 1.f / lr;
                __nv_bfloat16* dst = p.out + int64_t(f.row0 + r) * p.b.latent;
                float* part = p.ws.o + int64_t(f.slot) * kLatentRowTile * p.b.latent;
                for (int c = 0; c < ocols; c += 32) {
                    uint32_t v[32];
                    tc_ld32(tmem + lanes + (c < half0 ? c : 128 + c - half0), v);
                    tc_wait_ld();
                    if (r >= f.nrows) {
                    } else if (f.whole) {
                        const int d = c < half0 ? h * half0 + c : n0 + h * half1 + c - half0;
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            uint32_t o[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                o[e] = pack_bf16x2(__uint_as_float(v[16 * i + 2 * e]) * inv,
                                                   __uint_as_float(v[16 * i + 2 * e + 1]) * inv);
                            store_sector(dst + d + 16 * i, o, p.whole_sectors);
                        }
                    } else {
                        // [4 columns][lane]: a warp writes 512 bytes in a row
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            *reinterpret_cast<uint4*>(part + ((c / 4 + i) * 128 + h * 64 + r) * 4) =
                                make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                    }
                    __syncwarp();
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

}  // namespace

int launch_latent_bf16(const LatentArgs& a) {
    const pkv_latent_desc* d = a.desc;
    // more rows than a unit's go to pairs of CTAs (latent 512, us here and there: 96 requests of
    // 1k to 8k keys with 128 rows 161 and 127, 32 with 72 rows 65 and 58)
    if (latent_rows(a.batch) > kRows) return launch_latent_pair(a);
    const int cols = d->latent_dim / 64 + 1;
    CUtensorMap kv, q;
    if (!make_latent_tensor_map(&kv, a.cache, int64_t(d->num_blocks) * kBlockTokens, cols, 8, cols) ||
        !make_latent_tensor_map(&q, a.q, int64_t(a.batch.num_query_tokens) * d->num_q_heads, cols, 8, cols))
        return PKV_ERR_CUDA;
    Params p;
    p.b = a.batch;
    p.ws = a.ws;
    p.out = static_cast<__nv_bfloat16*>(a.out);
    p.b.team = 1;                          // (a sequence has one tile of rows on average, or less)
    p.whole_sectors = (reinterpret_cast<uintptr_t>(a.out) & 31) == 0;
    // query rows of a unit: all 64, or those of the longest sequence if it has fewer (a
    // call of one token a sequence; with offsets the rows of a sequence are not known here)
    const int64_t rows = a.batch.query_start_loc ? kRows : std::min<int64_t>(kRows, a.batch.heads);
    p.q_groups = int(rows + 7) / 8;
    const int group = cols * 1024, rest = int(sizeof(Smem)) + 1024 + kPBytes + p.q_groups * group;
    static_assert(kPBytes + (8 + 4 * kGroups) * 9 * 1024 + sizeof(Smem) + 1024 <= 232448, "shared memory");
    p.slots = std::min(kMostSlots, (232448 - rest) / (kGroups * group));
    const int smem = rest + p.slots * kGroups * group;
    // one limit for all latent_dims
    if (kernel_occupancy<latent_kernel>(kThreads, 232448) < 1) return PKV_ERR_CUDA;
    cudaError_t e = launch_pdl(latent_kernel, dim3(num_sms()), dim3(kThreads), size_t(smem), a.stream, kv,
                               q, p);
    if (e != cudaSuccess) return cuda_status(e);
    return launch_latent_merge<__nv_bfloat16>(a.stream, p.b, p.ws, p.out, num_sms(),
                                              std::min(256, d->latent_dim) / 2);
}

}  // namespace pkv
