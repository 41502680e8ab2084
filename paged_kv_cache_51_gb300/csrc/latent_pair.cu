// Attention over a paged latent cache for more than 64 (token, head) rows of a sequence: a
// pair of CTAs on one tile of 128 rows and 128 keys (tcgen05, cta_group::2).
//
//   S = Q K^T      128 rows x 128 keys: each CTA holds 64 of the rows and 64 of the keys
//   O += P C       128 rows x latent_dim: each CTA holds P of its rows and, of all 128 keys,
//                  one half of the latent values
//
// Measured, a pair's product of 128 x 128 x 16 takes 32 cycles and one of 128 x 256 x 16 64:
// a step of 128 keys costs each SM 2176 cycles of products for 128 rows, where two CTAs of
// 64 rows (latent_attn.cu) cost 4736 each; HBM needs 3300 for a step's rows.  What a CTA
// keeps in shared memory grows in turn: its rows' queries (latent 512: 72 KB), its 64 keys in
// full (72 KB), half of the values of all 128 keys (64 KB) and P (16 KB) fill it.  So keys
// come in chunks of three 64-value columns and values in chunks of 32 keys, each loaded again
// as soon as its own products are complete: loads never pause for a whole step.
//
// The accumulators of such products lie like this in each CTA's TMEM: row r of its 64 in
// lanes r and 64 + r, the first half of the columns in the former.  So a thread of the
// softmax holds 64 keys of one row, and O's halves of the values of the same row.
//
// Warps of each CTA: 0 loads queries and keys, 2 values, 4-7 are the softmax; 1 and 3 of the
// first CTA issue S and P C for both.  Loads count on the first CTA's barriers, which expect
// both CTAs' bytes (always whole chunks of keys: rows behind the context are read from some
// block and masked in S); a product's completion arrives in both CTAs.
//
// Measured: 96 requests of 1k to 8k tokens, latent 512, 128 heads: 126 us with the merge (4.3
// TB/s, 980 TFLOP/s); a step takes 4150 cycles, what L2 delivers to an SM 2570 of them and
// chunks that are 3000 on their way the rest.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "latent_common.cuh"
#include "latent_merge.cuh"
#include "launch_cache.h"

namespace pkv {
namespace {

constexpr int kRows = 128;                 // of the pair
constexpr int kKeys = 128;
constexpr int kMine = 64;                  // rows and keys of a CTA
constexpr int kThreads = 256;
constexpr int kSoftWarp0 = 4;
constexpr int kSoftWarps = 4;
constexpr int kPBytes = kMine * kKeys * 2;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kSCol = 256;            // S buffers: 64 columns each behind O
constexpr float kRescale = 8.f;            // log2 units
constexpr int kLeastSteps = 2;             // of a pair (one request of 8000 keys: 18.1 us, with one 20.1)
constexpr int kStart = 2;                  // steps that a unit costs beside its tiles
constexpr int kSmemMost = 232448;

constexpr int kKCols = 3;                  // 64-value columns of a chunk of keys
constexpr int kVKeys = 32;                 // keys of a chunk of values
constexpr int kMostK = 4, kMostV = 8;      // chunks

enum {
    B_K_FULL = 0,                          // [key chunk]       (first CTA)
    B_V_FULL = B_K_FULL + kMostK,          // [value chunk]     (first CTA)
    B_Q_FULL = B_V_FULL + kMostV,          //                   (first CTA)
    B_S_EMPTY,                             // [S buffer]: both CTAs' softmax have loaded it (first)
    B_P_FULL = B_S_EMPTY + 2,              // both CTAs' P are there (first)
    B_K_EMPTY,                             // [key chunk]: its products are complete
    B_V_EMPTY = B_K_EMPTY + kMostK,        // [value chunk]: its products are complete
    B_S_FULL = B_V_EMPTY + kMostV,         // [S buffer]
    B_O_DONE = B_S_FULL + 2,               // the tile's P C is complete
    B_Q_EMPTY,                             // the fragment's last S is complete
    B_V_TAIL,                              // [value chunk]: a chunk that the context ends in has landed
    B_XM = B_V_TAIL + kMostV,              // [row half]: both key halves' maxima are there
    B_SUM = B_XM + 2,                      // [row half]: both key halves' sums are there
    B_DRAIN = B_SUM + 2,                   // [issuer]          (first CTA)
    B_COUNT = B_DRAIN + 2
};

struct Smem {                              // behind the operands
    uint64_t bars[B_COUNT];
    int64_t sums[kThreads / 32 + 2];
    float xm[2][128];
    float sum[128];
    uint32_t tmem;
    int abort;
};
static_assert(sizeof(Smem) <= 2048, "shared memory");
static_assert(kMine == kLatentRowTile, "a CTA of a pair writes the states of its own rows");

// Chunks and shared memory for a latent_dim: two tiles of keys where they fit, at the longest
// latent vectors one; then as many chunks of values as fit.
struct Slots {
    int k, v, smem;
};
constexpr Slots slots_of(int latent) {
    const int cols = latent / 64 + 1, vcols = latent / 128, chunks = (cols + kKCols - 1) / kKCols;
    const int kchunk = kKCols * 1024 * (kMine / 8), vchunk = vcols * 1024 * (kVKeys / 8);
    const int fixed = 1024 + int(sizeof(Smem)) + kPBytes + cols * 1024 * (kMine / 8);
    const int k = fixed + 2 * chunks * kchunk + 4 * vchunk <= kSmemMost ? 2 * chunks : chunks;
    const int room = (kSmemMost - fixed - k * kchunk) / vchunk, v = room < kMostV ? room : kMostV;
    return {k, v, fixed + k * kchunk + v * vchunk};
}
// The value ring holds a tile at least: the softmax waits for the chunk that the context ends
// in before its P lets the chunks in front of it go, and finds a chunk's slot by one subtraction.
constexpr bool slots_fit(int latent) {
    const Slots s = slots_of(latent);
    return s.k >= 1 && s.k <= kMostK && s.v >= kKeys / kVKeys && s.v <= kMostV && s.smem <= kSmemMost;
}
static_assert(slots_fit(128) && slots_fit(256) && slots_fit(384) && slots_fit(512), "shared memory");

struct Params {
    LatentBatch b;
    LatentWorkspace ws;
    __nv_bfloat16* out;
    int32_t k_slots, v_slots;
    bool whole_sectors;
};

using Walk = LatentWalk<kRows, kKeys, kStart>;
using Tiles = LatentTiles<kRows, kKeys, kStart>;

// ---- the pair ------------------------------------------------------------------
__device__ __forceinline__ uint32_t cta_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void pair_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// the first CTA's copy of a shared-memory address
__device__ __forceinline__ uint32_t in_first(const void* p) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(smem_u32(p)));
    return a;
}
// Tells the first CTA that this warp's P or its reads of S are there.  What it orders is what
// this CTA's own tensor core reads next, behind each writer's fence for that proxy (a release
// at the scope of the cluster, which no thread of the other CTA needs, took 1000 to 3500
// cycles; one thread that passed the warps' arrivals on with such a release: 96 requests with
// 128 heads 163 us instead of 127).
__device__ __forceinline__ void arrive_first(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(in_first(bar)) : "memory");
}
// a box to this CTA's shared memory, counted on a barrier of the first CTA
__device__ __forceinline__ void load_pair(uint32_t dst, const CUtensorMap* map, int x, int y, int z,
                                          uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void commit_pair(uint64_t* bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"(uint16_t(3))
        : "memory");
}
__device__ __forceinline__ void commit_first(uint64_t* bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}

// A place in a ring of chunks.
struct Ring {
    uint32_t slot = 0, phase = 0;
    __device__ void next(uint32_t slots) {
        if (++slot == slots) {
            slot = 0;
            phase ^= 1;
        }
    }
};

// After a wait ran out: time for this CTA's copies to land before it leaves (what they count
// on may be the other CTA's barrier).
__device__ __forceinline__ void let_copies_land() {
    const uint64_t t0 = global_ns();
    while (global_ns() - t0 < 1000000) {
    }
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    latent_pair_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                       const __grid_constant__ CUtensorMap map_q, Params p) {
    extern __shared__ unsigned char smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    // (the same offset in both CTAs, whose dynamic shared memory begins at the same address)
    unsigned char* smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
    const uint32_t base = smem_u32(smem);
    const int cols = p.b.latent / 64 + 1, vcols = p.b.latent / 128;   // 64-value columns of a row, and of half a value
    const int chunks = (cols + kKCols - 1) / kKCols;
    const uint32_t group = uint32_t(cols) * 1024;         // 8 rows: queries,
    constexpr uint32_t kgroup = kKCols * 1024;            // a chunk of keys,
    const uint32_t vgroup = uint32_t(vcols) * 1024;       // values
    constexpr uint32_t kchunk = kgroup * (kMine / 8);
    const uint32_t qbytes = group * (kMine / 8), vchunk = vgroup * (kVKeys / 8);
    const uint32_t k_slots = uint32_t(p.k_slots), v_slots = uint32_t(p.v_slots);
    const uint32_t p_off = 0, q_off = kPBytes, k_off = q_off + qbytes, v_off = k_off + k_slots * kchunk;
    Smem& sh = *reinterpret_cast<Smem*>(smem + v_off + v_slots * vchunk);
    uint64_t* bars = sh.bars;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = int(cta_rank()), pair = int(blockIdx.x) >> 1;
    volatile int* abort_flag = &sh.abort;
    int* err = p.b.err;

    if (threadIdx.x == 0) {
        for (int i = 0; i < B_COUNT; ++i) {
            int n = 1;
            if (i >= B_S_EMPTY && i < B_K_EMPTY) n = 2 * kSoftWarps;
            if (i >= B_XM && i < B_DRAIN) n = 2;
            mbar_init(&bars[i], n);
        }
        sh.abort = 0;
        fence_mbar_init();
    }
    // (as in latent_attn.cu, tensor memory is taken behind the wait)
    pdl_wait_prerequisites();
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(&sh.tmem)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    const Walk plan = latent_plan<kRows, kKeys, kStart, kThreads>(p.b, sh.sums, kLeastSteps, pair, int(gridDim.x) / 2);
    pdl_launch_dependents();
    pair_sync();                                          // the other CTA's barriers are initialised
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&sh.tmem);

    if (warp == 0) {
        // ---- queries and keys (one thread, as elect_one's comment says: eight lanes of a warp
        // took 800 cycles for a chunk's eight copies) ----
        if (elect_one()) {
            const uint32_t full0 = in_first(&bars[B_K_FULL]), q_full = in_first(&bars[B_Q_FULL]);
            Tiles t;
            Ring at;
            bool ok = true;
            uint32_t n = 0;                               // chunks so far
            for (t.start(p.b, plan); t.live; t.next(p.b)) {
                const int32_t* table = p.b.block_tables + int64_t(t.f.seq) * p.b.table_stride;
                const int key0 = (t.f.kt0 + t.j) * kKeys + rank * kMine;
                int row[kMine / kBlockTokens];
#pragma unroll
                for (int i = 0; i < kMine / kBlockTokens; ++i) {
                    const int key = key0 + i * kBlockTokens;
                    row[i] = key < t.f.ctx ? __ldg(table + key / kBlockTokens) : 0;
                }
                if (t.j == 0) {                            // (while the ids are on their way)
                    ok = !*abort_flag && (t.k == 0 || mbar_wait_asleep(&bars[B_Q_EMPTY], (t.k - 1) & 1, err));
                    if (!ok) break;
                    if (rank == 0) mbar_arrive_expect_tx(&bars[B_Q_FULL], 2 * qbytes);
                    const int row0 = t.f.row0 + rank * (t.f.nrows > kMine ? kMine : kMine / 2);
#pragma unroll
                    for (int i = 0; i < kMine / 8; ++i)
                        load_pair(base + q_off + uint32_t(i) * group, &map_q, 0, row0 + i * 8, 0, q_full);
                }
#pragma unroll
                for (int i = 0; i < kMine / kBlockTokens; ++i) {
                    if (row[i] < 0 || row[i] >= p.b.num_blocks) {
                        flag_error(err, PKV_DEV_BAD_BLOCK_ID);
                        row[i] = 0;
                    }
                    row[i] *= kBlockTokens;
                }
                for (int c = 0; c < chunks; ++c, ++n) {
                    ok = !*abort_flag && (n < k_slots || mbar_wait_asleep(&bars[B_K_EMPTY + at.slot], at.phase ^ 1, err));
                    if (!ok) break;
#ifdef PKV_TEST_SKIP_TILE
                    // wait-timeout test build only, as in latent_attn.cu
                    if (t.g == uint32_t(PKV_TEST_SKIP_TILE)) {
                        at.next(k_slots);
                        continue;
                    }
#endif
                    if (rank == 0) mbar_arrive_expect_tx(&bars[B_K_FULL + at.slot], 2 * kchunk);
                    const uint32_t dst = base + k_off + at.slot * kchunk, full = full0 + at.slot * 8;
#pragma unroll
                    for (int i = 0; i < kMine / 8; ++i)
                        load_pair(dst + uint32_t(i) * kgroup, &map_k, 0, row[i / 2] + (i & 1) * 8, c * kKCols, full);
                    at.next(k_slots);
                }
                if (!ok) break;
            }
            // (nothing arrives here once this CTA has left)
            if (ok && t.k > 0) ok = mbar_wait_asleep(&bars[B_Q_EMPTY], (t.k - 1) & 1, err);
            for (uint32_t i = 0; ok && i < k_slots && i < n; ++i) {
                const uint32_t last = n - 1 - i;
                ok = mbar_wait_asleep(&bars[B_K_EMPTY + last % k_slots], (last / k_slots) & 1, err);
            }
            if (!ok) {
                *abort_flag = 1;
                let_copies_land();
            }
        }
        __syncwarp();
    } else if (warp == 2) {
        // ---- values ----
        if (elect_one()) {
            const uint32_t full0 = in_first(&bars[B_V_FULL]);
            Tiles t;
            Ring at;
            bool ok = true;
            uint32_t n = 0;
            for (t.start(p.b, plan); t.live; t.next(p.b)) {
                const int32_t* table = p.b.block_tables + int64_t(t.f.seq) * p.b.table_stride;
                const int key0 = (t.f.kt0 + t.j) * kKeys, keys = min(kKeys, t.f.ctx - key0);
                int row[kKeys / kBlockTokens];
#pragma unroll
                for (int i = 0; i < kKeys / kBlockTokens; ++i)
                    row[i] = i * kBlockTokens < keys ? __ldg(table + key0 / kBlockTokens + i) : 0;
#pragma unroll
                for (int i = 0; i < kKeys / kBlockTokens; ++i)    // (bad ids: flagged by warp 0)
                    row[i] = row[i] < 0 || row[i] >= p.b.num_blocks ? 0 : row[i] * kBlockTokens;
#pragma unroll
                for (int c = 0; c < kKeys / kVKeys; ++c) {
                    if (c * kVKeys >= keys) break;
                    ok = !*abort_flag && (n < v_slots || mbar_wait_asleep(&bars[B_V_EMPTY + at.slot], at.phase ^ 1, err));
                    if (!ok) break;
                    const int groups = (min(kVKeys, keys - c * kVKeys) + 7) / 8;
                    const uint32_t dst = base + v_off + at.slot * vchunk;
                    // a chunk whose last 16 keys are not all of the context's is seen by the softmax
                    // of its CTA, whose P says that it is there; any other one by the issuer
                    if (keys - c * kVKeys < kVKeys && (keys & 15) != 0) {
                        mbar_arrive_expect_tx(&bars[B_V_TAIL + at.slot], uint32_t(groups) * vgroup);
                        if (rank == 0) mbar_arrive(&bars[B_V_FULL + at.slot]);
#pragma unroll
                        for (int i = 0; i < kVKeys / 8; ++i)
                            if (i < groups)
                                tc_load_3d(dst + uint32_t(i) * vgroup, &map_v, 0, row[2 * c + i / 2] + (i & 1) * 8,
                                           rank * vcols, &bars[B_V_TAIL + at.slot]);
                    } else {
                        if (rank == 0)
                            mbar_arrive_expect_tx(&bars[B_V_FULL + at.slot], 2 * uint32_t(groups) * vgroup);
#pragma unroll
                        for (int i = 0; i < kVKeys / 8; ++i)
                            if (i < groups)
                                load_pair(dst + uint32_t(i) * vgroup, &map_v, 0, row[2 * c + i / 2] + (i & 1) * 8,
                                          rank * vcols, full0 + at.slot * 8);
                    }
                    at.next(v_slots);
                    ++n;
                }
                if (!ok) break;
            }
            for (uint32_t i = 0; ok && i < v_slots && i < n; ++i) {
                const uint32_t last = n - 1 - i;
                ok = mbar_wait_asleep(&bars[B_V_EMPTY + last % v_slots], (last / v_slots) & 1, err);
            }
            if (!ok) {
                *abort_flag = 1;
                let_copies_land();
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        if (rank == 0 && elect_one()) {
            constexpr uint32_t idesc = tc_idesc(kRows, kKeys, false);
            const uint64_t qd = tc_smem_desc(base + q_off, 16, group);
            const uint64_t kd = tc_smem_desc(base + k_off, 16, kgroup);
            Tiles t;
            Ring at;
            bool ok = true;
            for (t.start(p.b, plan); t.live; t.next(p.b)) {
                const uint32_t sb = t.g & 1;
                const uint32_t d = tmem + kSCol + sb * 64;
                uint64_t qa = qd;
                if (t.j == 0) ok = !*abort_flag && mbar_wait_asleep(&bars[B_Q_FULL], t.k & 1, err);
                ok = ok && (t.g < 2 || mbar_wait_asleep(&bars[B_S_EMPTY + sb], ((t.g - 2) >> 1) & 1, err));
                for (int c0 = 0; ok && c0 < cols; c0 += kKCols) {
                    ok = mbar_wait_asleep(&bars[B_K_FULL + at.slot], at.phase, err);
                    if (!ok) break;
                    tc_fence_after();
                    uint64_t ka = kd + uint64_t(at.slot * (kchunk >> 4));
                    for (int c = c0; c < min(cols, c0 + kKCols); ++c, qa += 64, ka += 64) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            mma_pair(d, qa + uint64_t(i * 2), ka + uint64_t(i * 2), idesc, (c | i) != 0);
                    }
                    commit_pair(&bars[B_K_EMPTY + at.slot]);
                    at.next(k_slots);
                }
                if (!ok) break;
                commit_pair(&bars[B_S_FULL + sb]);
                if (t.j == t.f.n - 1) commit_pair(&bars[B_Q_EMPTY]);
            }
            if (t.live) *abort_flag = 1;
            commit_first(&bars[B_DRAIN]);
            mbar_wait_asleep(&bars[B_DRAIN], 0, err);
        }
        __syncwarp();
    } else if (warp == 3) {
        if (rank == 0 && elect_one()) {
            const int half = p.b.latent / 2, n0 = min(128, half), n1 = half - n0;   // columns of a CTA
            const uint32_t idesc0 = tc_idesc(kRows, 2 * n0, true), idesc1 = tc_idesc(kRows, 2 * n1, true);
            const uint64_t vd = tc_smem_desc(base + v_off, 1024, vgroup);
            const uint64_t pd = tc_smem_desc(base + p_off, 16, 1024);
            Tiles t;
            Ring at;
            bool ok = true;
            for (t.start(p.b, plan); t.live; t.next(p.b)) {
                const int keys = min(kKeys, t.f.ctx - (t.f.kt0 + t.j) * kKeys);
                ok = !*abort_flag && mbar_wait_asleep(&bars[B_P_FULL], t.g & 1, err);
                for (int i0 = 0; ok && i0 < keys; i0 += kVKeys) {
                    ok = mbar_wait_asleep(&bars[B_V_FULL + at.slot], at.phase, err);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t v0 = vd + uint64_t(at.slot * (vchunk >> 4));
#pragma unroll
                    for (int i = 0; i < kVKeys / 16; ++i) {
                        const int k0 = i0 + 16 * i;
                        if (k0 >= keys) break;
                        const uint32_t acc = (t.j | k0) != 0;
                        const uint64_t a = pd + uint64_t((k0 >> 6) * (kMine * 128 >> 4) + ((k0 >> 4) & 3) * 2);
                        const uint64_t v = v0 + uint64_t(i * 2 * (vgroup >> 4));
                        mma_pair(tmem, a, v, idesc0, acc);
                        if (n1 > 0) mma_pair(tmem + 128, a, v + 2 * 64, idesc1, acc);
                    }
                    commit_pair(&bars[B_V_EMPTY + at.slot]);
                    at.next(v_slots);
                }
                if (!ok) break;
                commit_pair(&bars[B_O_DONE]);
            }
            if (t.live) *abort_flag = 1;
            commit_first(&bars[B_DRAIN + 1]);
            mbar_wait_asleep(&bars[B_DRAIN + 1], 0, err);
        }
        __syncwarp();
        // sequences with lengths that the call does not allow: zeros
        for (int s = blockIdx.x; s < p.b.num_seqs; s += gridDim.x) {
            const LatentSeq x = latent_seq<false>(p.b, s);
            if (!x.zero) continue;
            const int64_t row_vecs = int64_t(p.b.heads) * p.b.latent / 8;
            uint4* dst = reinterpret_cast<uint4*>(p.out) + int64_t(x.q0) * row_vecs;
            for (int64_t i = lane; i < row_vecs * x.qlen; i += 32) dst[i] = make_uint4(0, 0, 0, 0);
        }
        __syncwarp();
    } else {
        // ---- softmax: thread = (row r, key half h); O: the same row, half h of the values ----
        const int w4 = warp - kSoftWarp0;
        const int r = (w4 & 1) * 32 + lane, h = w4 >> 1;
        const uint32_t lanes = uint32_t(w4 * 32) << 16;
        const int half = p.b.latent / 2;                  // TMEM columns of O
        Walk w = plan;
        LatentFrag f;
        uint32_t g = 0, k = 0;
        uint32_t at = 0;                                  // the tile's first value chunk
        uint32_t tails = 0;                               // phases of B_V_TAIL
        bool ok = true;
        if (int(threadIdx.x) == kSoftWarp0 * 32) p.ws.merge[blockIdx.x].nrows = 0;
        __syncwarp();
        while (w.next(p.b, f)) {
            // this CTA's rows of the pair's: 64 and the rest, or two halves of up to 32
            const int split = f.nrows > kMine ? kMine : kMine / 2;
            const int first = rank * split, nrows = max(0, min(split, f.nrows - first));
            const int row = min(first + r, max(0, f.nrows - 1));
            const int limit = f.first_pos + f.t0 + (f.rest + row) / p.b.heads;   // last key that the row sees
            float m = -INFINITY, l = 0.f;
            for (int j = 0; j < f.n; ++j, ++g) {
                ok = mbar_wait_asleep(&bars[B_S_FULL + (g & 1)], (g >> 1) & 1, err);
                __syncwarp();
                tc_fence_after();
                float s[64];
                {
                    uint32_t v0[32], v1[32];
                    tc_ld32(tmem + lanes + kSCol + (g & 1) * 64, v0);
                    tc_ld32(tmem + lanes + kSCol + (g & 1) * 64 + 32, v1);
                    tc_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        s[i] = __uint_as_float(v0[i]);
                        s[32 + i] = __uint_as_float(v1[i]);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive_first(&bars[B_S_EMPTY + (g & 1)]);
                const int key0 = (f.kt0 + j) * kKeys, lim = limit - key0 - h * kMine;
                if (lim < kMine - 1) {
#pragma unroll
                    for (int i = 0; i < 64; ++i) s[i] = i <= lim ? s[i] : -INFINITY;
                }
                float mx4[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) mx4[i] = fmaxf(s[i], s[i + 4]);
#pragma unroll
                for (int i = 8; i < 64; ++i) mx4[i & 3] = fmaxf(mx4[i & 3], s[i]);
                const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * p.b.scale_log2;
                // the row's other key half is the same lane of the warp two on
                sh.xm[g & 1][h * 64 + r] = mx;
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[B_XM + (w4 & 1)]);
                ok = mbar_wait_asleep(&bars[B_XM + (w4 & 1)], g & 1, err) && ok;
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
                uint32_t pk[32];
                float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    pk[i] = pack_bf16x2(exp2_fast(fmaf(s[2 * i], p.b.scale_log2, neg_m)),
                                        exp2_fast(fmaf(s[2 * i + 1], p.b.scale_log2, neg_m)));
                    sum[i & 1] += __uint_as_float(pk[i] << 16);
                    sum[2 + (i & 1)] += __uint_as_float(pk[i] & 0xffff0000u);
                }
                l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                // the previous tile's P C reads P and adds to O
                if (g > 0) ok = mbar_wait_asleep(&bars[B_O_DONE], (g - 1) & 1, err) && ok;
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                if (j > 0 && __any_sync(0xffffffffu, need)) {
                    for (int c = 0; c < half; c += 32) {
                        uint32_t v[32];
                        tc_ld32(tmem + lanes + c, v);
                        tc_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * alpha);
                        tc_st32(tmem + lanes + c, v);
                    }
                    tc_wait_st();
                }
                unsigned char* dst = smem + p_off + h * (kMine * 128) + r * 128;
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    *reinterpret_cast<uint4*>(dst + ((c ^ (r & 7)) * 16)) =
                        make_uint4(pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]);
                // the 16 keys that the context ends in: the values behind it are another tile's or
                // nothing's and are zeroed, since 0 times anything must stay 0
                const int keys = min(kKeys, f.ctx - key0);
                if (keys & 15) {
                    const int chunk = keys / kVKeys, from = keys - chunk * kVKeys;
                    uint32_t slot = at + uint32_t(chunk);
                    if (slot >= v_slots) slot -= v_slots;
                    ok = __all_sync(0xffffffffu,
                                    mbar_wait_asleep(&bars[B_V_TAIL + slot], (tails >> slot) & 1, err));
                    if (!ok) break;
                    tails ^= 1u << slot;
                    unsigned char* vs = smem + v_off + slot * vchunk;
                    const int vecs = vcols * 8;            // 16-byte vectors of a row
                    for (int i = w4 * 32 + lane; i < (16 - (keys & 15)) * vecs; i += 128) {
                        const int row_i = from + i / vecs, c = i % vecs;
                        *reinterpret_cast<uint4*>(vs + uint32_t(row_i >> 3) * vgroup + (c >> 3) * 1024 +
                                                  (row_i & 7) * 128 + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
                    }
                }
                at += uint32_t(keys + kVKeys - 1) / kVKeys;
                if (at >= v_slots) at -= v_slots;
                fence_proxy_async_shared();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive_first(&bars[B_P_FULL]);
            }
            if (!ok) break;
            // ---- the fragment's output or state ----
            if (f.n > 0) {
                ok = mbar_wait_asleep(&bars[B_O_DONE], (g - 1) & 1, err);
                sh.sum[h * 64 + r] = l;
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[B_SUM + (w4 & 1)]);
                ok = mbar_wait_asleep(&bars[B_SUM + (w4 & 1)], k & 1, err) && ok;
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                l += sh.sum[(h ^ 1) * 64 + r];
            }
            const int slot = 2 * int(blockIdx.x) + (f.slot & 1);
            if (!f.whole && h == 0) p.ws.ml[slot * kLatentRowTile + r] = make_float2(m, l);
            if (f.starts && nrows > 0 && int(threadIdx.x) == kSoftWarp0 * 32)
                p.ws.merge[blockIdx.x] =
                    LatentMerge{f.row0 + first, nrows, int(blockIdx.x), 2 * f.last_cta + rank, slot};
            __syncwarp();                                  // the TMEM reads want all lanes at once
            if (f.n > 0) {
                const float inv = 1.f / l;
                __nv_bfloat16* dst = p.out + (int64_t(f.row0) + first + r) * p.b.latent + h * half;
                float* part = p.ws.o + int64_t(slot) * kLatentRowTile * p.b.latent;
                for (int c = 0; c < half; c += 32) {
                    uint32_t v[32];
                    tc_ld32(tmem + lanes + c, v);
                    tc_wait_ld();
                    if (r >= nrows) {
                    } else if (f.whole) {
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            uint32_t o[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                o[e] = pack_bf16x2(__uint_as_float(v[16 * i + 2 * e]) * inv,
                                                   __uint_as_float(v[16 * i + 2 * e + 1]) * inv);
                            store_sector(dst + c + 16 * i, o, p.whole_sectors);
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
                // (that O has been read, the next fragment's first P tells)
                ++k;
            }
        }
        if (!ok) *abort_flag = 1;
        __syncwarp();
    }
    // neither CTA leaves, or frees TMEM, while copies, products or arrivals of the other are
    // on their way
    tc_fence_before();
    __syncthreads();
    pair_sync();
    tc_fence_after();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols)
                     : "memory");
}

}  // namespace

int launch_latent_pair(const LatentArgs& a) {
    const pkv_latent_desc* d = a.desc;
    const int cols = d->latent_dim / 64 + 1, vcols = d->latent_dim / 128;
    const int64_t rows = int64_t(d->num_blocks) * kBlockTokens;
    CUtensorMap k, v, q;
    if (!make_latent_tensor_map(&k, a.cache, rows, cols, 8, kKCols) ||
        !make_latent_tensor_map(&v, a.cache, rows, cols, 8, vcols) ||
        !make_latent_tensor_map(&q, a.q, int64_t(a.batch.num_query_tokens) * d->num_q_heads, cols, 8, cols))
        return PKV_ERR_CUDA;
    Params p;
    p.b = a.batch;
    p.ws = a.ws;
    p.out = static_cast<__nv_bfloat16*>(a.out);
    p.b.team = latent_team(p.b, kRows);
    p.whole_sectors = (reinterpret_cast<uintptr_t>(a.out) & 31) == 0;
    const Slots slots = slots_of(d->latent_dim);
    p.k_slots = slots.k;
    p.v_slots = slots.v;
    if (kernel_occupancy<latent_pair_kernel>(kThreads, kSmemMost) < 1) return PKV_ERR_CUDA;
    const int ctas = num_sms() & ~1;                      // whole pairs
    cudaError_t e = launch_pdl(latent_pair_kernel, dim3(unsigned(ctas)), dim3(kThreads), size_t(slots.smem), a.stream, k,
                               v, q, p);
    if (e != cudaSuccess) return cuda_status(e);
    LatentBatch b = p.b;
    b.team *= 2;                                          // CTAs from one state of a unit to the next
    return launch_latent_merge<__nv_bfloat16>(a.stream, b, p.ws, p.out, ctas, d->latent_dim / 2);
}

}  // namespace pkv
