// Attention over expanded keys in bf16 on the tcgen05 tensor cores.
//
//   S = Q K^T   128 query rows x 128 keys over D + 64 dimensions
//   O += P V    128 query rows x D values over 128 keys
//
// with fp32 accumulators in TMEM, the online softmax in base 2 between them and P in
// TMEM in front of the second product.  A key's last 64 dimensions come from the rotary
// part that all heads share, so the keys are never laid out in full anywhere.
//
// Two query tiles a CTA.  One tile alone leaves the tensor cores idle while its softmax
// runs (S 768 cycles, P V 512, and in between the chain of load, maximum, exponentials
// and store); so a unit is 256 query rows of one head, two streams of 128 rows that read
// the same keys and values, and the products of one run under the softmax of the other.
// TMEM is then full: two S (128 columns each, P overwrites its own S) and two O.
//
// Warps: 0-3 and 4-7 are the streams' softmax (a thread a row, so a row's maximum and sum
// need no exchange), 8 loads, 9 issues all products.  Shared memory: the two query tiles
// (D = 128: 96 KB) and a ring of 16 KB slots that takes keys and values in the order of
// their use: 3 slots of a key tile (64 dimensions each), 2 of a value tile (64 keys each);
// 8 slots are 1.6 tiles, where a ring each for keys and values would have held 1.3 and 2.
// A slot is given back on its own, the first half of the values before the second (chunks:
// 91.5 us where all of a tile's values came back together, 87.5).  Landing is told by the
// tile: a wait for each slot costs the issuer more than it gains where units are short (50
// prompts of up to 976 tokens, 26 heads: 223 us against 182).
//
// Units come longest first from a ticket.  Where there are so few that four or two CTAs for
// each find SMs, a cluster shares one: every CTA takes its part of the key tiles, and they
// meet through one another's shared memory at the end (one head of 16 queries over 16k keys
// took 180 us with one CTA and takes 52 with four, 8 heads over 4k 51 and 19; two sequences
// of 256 queries over 3256 keys, 16 heads, 55 and 37 with two).
//
// Measured, D = 128, 32 heads: 8 prompts of 1700 to 4096 tokens 561 to 569 us (1290 TFLOP/s, at
// the power limit), 4 chunks of about 450 over 512 to 3584 cached 90 us; D = 64: 406 us (1080
// TFLOP/s) and 73.  A tile of both
// streams takes 3350 to 3600 cycles, of which products 2560: a stream's softmax (1500 to 1600)
// and its products (1280) cannot overlap, since S and P share their columns.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "expanded_common.h"
#include "latent_common.cuh"
#include "launch_cache.h"

namespace pkv {
namespace {

constexpr int kT = 128;                    // query rows of a stream, keys of a tile
constexpr int kBox = kT * 128;             // bytes of 128 rows x 64 values
constexpr int kThreads = 384;
constexpr int kLoadWarp = 8;
constexpr int kMmaWarp = 9;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kOCol = 256;            // S of stream x at 128 x, O at 256 + 128 x
constexpr float kRescale = 8.f;            // log2 units: O is rescaled when a row's max grows by more
// registers: 384 threads start with 168 each; the softmax warps hold a row's 128 scores
constexpr int kSoftRegs = 208, kOtherRegs = 88;
static_assert(256 * kSoftRegs + 128 * kOtherRegs <= 384 * 168, "register split");

constexpr int kMostSlots = 8;

enum {
    B_K_FULL = 0,                          // [tile parity]
    B_V_FULL = B_K_FULL + 2,
    B_EMPTY = B_V_FULL + 2,                // [slot]: its products are complete
    B_Q_FULL = B_EMPTY + kMostSlots,                // [stream]
    B_Q_EMPTY = B_Q_FULL + 2,              // the unit's last S of the stream is complete
    B_S_FULL = B_Q_EMPTY + 2,
    B_P_FULL = B_S_FULL + 2,               // [stream][half of the keys]
    B_O_FULL = B_P_FULL + 4,               // the unit's last P V of the stream is complete
    B_O_EMPTY = B_O_FULL + 2,
    B_U_FULL = B_O_EMPTY + 2,              // [unit parity]
    B_U_EMPTY = B_U_FULL + 2,
    B_DRAIN = B_U_EMPTY + 2,
    B_COUNT
};
constexpr int kUnitReaders = 1 + 8;        // issuer, softmax warps

struct Unit {
    int32_t live;                          // 0: no more work
    int32_t head, q0, rows, k0, keys;
    int32_t most;                          // key tiles at most (a cluster's CTA: its share)
};

struct Smem {                              // behind the operands
    uint64_t bars[B_COUNT];
    Unit unit[2];
    uint32_t tmem;
    int abort;
};

template <int D>
struct Shape {
    static constexpr int kKBoxes = D / 64 + 1;             // slots of a key tile
    static constexpr int kVBoxes = D / 64;                 // and of a value tile
    static constexpr int kBoxes = kKBoxes + kVBoxes;
    // a slot's earlier use must be at most two tiles back (the tiles' barriers come in twos)
    static constexpr int kSlots = D == 128 ? 8 : 6;
    static constexpr int kQBytes = kKBoxes * kBox;
    static constexpr int kRing = 2 * kQBytes;
    static constexpr int kSmem = kRing + kSlots * kBox + int(sizeof(Smem)) + 1024;
    static_assert(kSmem <= 232448, "shared memory");
};

struct Params {
    ExpandedWorkspace ws;
    __nv_bfloat16* out;
    int32_t heads;
    bool whole_sectors;                    // out begins on 32 bytes
    float scale_log2;
    int* err;
};

// Tiles of each stream: rows 128 x .. of the unit see keys up to their last row's.
__device__ __forceinline__ int tiles_of(const Unit& u, int x) {
    const int rows = min(kT, u.rows - x * kT);
    if (rows <= 0) return 0;
    const int keys = u.keys - u.rows + x * kT + rows;
    return keys <= 0 ? 0 : min(u.most, (keys + kT - 1) / kT);
}

// four K = 16 steps over one 64-value column of both operands
__device__ __forceinline__ void mma_ss4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n .reg .pred pf, pa;\n .reg .b64 a1, a2, a3, b1, b2, b3;\n"
        " setp.ne.b32 pf, %4, 0;\n setp.eq.b32 pa, %4, %4;\n"
        " add.u64 a1, %1, 2;\n add.u64 a2, %1, 4;\n add.u64 a3, %1, 6;\n"
        " add.u64 b1, %2, 2;\n add.u64 b2, %2, 4;\n add.u64 b3, %2, 6;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, pf;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, pa;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, pa;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, pa;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
// four K = 16 steps over 64 keys: A (P, pairs of bf16) from TMEM, B 2048 bytes a step
__device__ __forceinline__ void mma_ts4(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n .reg .pred pf, pa;\n .reg .b32 a1, a2, a3;\n .reg .b64 b1, b2, b3;\n"
        " setp.ne.b32 pf, %4, 0;\n setp.eq.b32 pa, %4, %4;\n"
        " add.u32 a1, %1, 8;\n add.u32 a2, %1, 16;\n add.u32 a3, %1, 24;\n"
        " add.u64 b1, %2, 128;\n add.u64 b2, %2, 256;\n add.u64 b3, %2, 384;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, pf;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, pa;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], b2, %3, pa;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], b3, %3, pa;\n}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}

// s += (low, high) half of a pair of bf16, in one instruction each
__device__ __forceinline__ void add_pair(float2& s, uint32_t w) {
    asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n add.f32.bf16 %0, a, %0;\n add.f32.bf16 %1, b, %1;\n}\n"
        : "+f"(s.x), "+f"(s.y)
        : "r"(w));
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

__device__ __forceinline__ bool read_unit(Smem& sh, uint32_t n, int* err, Unit& u) {
    if (!mbar_wait(&sh.bars[B_U_FULL + (n & 1)], (n >> 1) & 1, err)) return false;
    u = sh.unit[n & 1];
    return true;
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t in_cta(const void* p, int rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    return a;
}
__device__ __forceinline__ float load_cluster(uint32_t at) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ float4 load_cluster4(uint32_t at) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(at)
                 : "memory");
    return v;
}

// The parts of a cluster's unit, in shared memory where queries and ring were: O of 256 rows,
// then their maxima and sums.
template <int D>
struct Parts {
    float o[2 * kT][D + 4];
    float m[2 * kT], l[2 * kT];
};

template <int D, int CTAS>
__global__ void __cluster_dims__(CTAS, 1, 1) __launch_bounds__(kThreads, 1)
    expanded_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                    const __grid_constant__ CUtensorMap map_r, const __grid_constant__ CUtensorMap map_v,
                    Params p) {
    using S = Shape<D>;
    extern __shared__ unsigned char smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    unsigned char* smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
    const uint32_t base = smem_u32(smem);
    Smem& sh = *reinterpret_cast<Smem*>(smem + S::kRing + S::kSlots * kBox);
    uint64_t* bars = sh.bars;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile int* abort_flag = &sh.abort;
    int* err = p.err;

    if (threadIdx.x == 0) {
        for (int i = 0; i < B_COUNT; ++i) {
            int n = 1;
            if (i >= B_P_FULL && i < B_O_FULL) n = 4;
            if (i >= B_O_EMPTY && i < B_U_FULL) n = 4;
            if (i >= B_U_EMPTY && i < B_DRAIN) n = kUnitReaders;
            mbar_init(&bars[i], n);
        }
        sh.abort = 0;
        fence_mbar_init();
    }
    // (as in latent_attn.cu, tensor memory is taken behind the wait)
    pdl_wait_prerequisites();
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(&sh.tmem)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    pdl_launch_dependents();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&sh.tmem);

    if (warp >= kLoadWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (warp == kLoadWarp && lane == 0) {
            const int units = p.ws.counters[0] * p.heads;
            int next = blockIdx.x / CTAS;
            uint32_t tile = 0, box = 0;                    // tiles and boxes so far
            uint32_t used[2] = {0, 0};                     // units with tiles of each stream
            bool ok = true;
            // the slot of the next box, once the box that it held is done with
            auto slot = [&](uint32_t& dst) {
                if (box >= uint32_t(S::kSlots)) {
                    ok = ok && mbar_wait(&bars[B_EMPTY + box % S::kSlots], (box / S::kSlots - 1) & 1, err);
                }
                dst = base + S::kRing + (box % S::kSlots) * kBox;
                ++box;
                return ok;
            };
            uint32_t n = 0;
            for (; ok; ++n) {
                ok = n < 2 || mbar_wait(&bars[B_U_EMPTY + (n & 1)], ((n - 2) >> 1) & 1, err);
                if (!ok || *abort_flag) break;
                Unit u = {};
                if (next < units) {
                    const ExpandedItem x = expanded_unit(p.ws, next, p.heads, u.head);
                    u = Unit{1, u.head, x.q0, x.rows, x.k0, x.keys, INT32_MAX};
                    if (CTAS > 1) {
                        u.most = ((max(x.keys, 0) + kT - 1) / kT + CTAS - 1) / CTAS;
                        const int skip = int(blockIdx.x % CTAS) * u.most * kT;
                        u.k0 += skip;
                        u.keys -= skip;
                    }
                }
                sh.unit[n & 1] = u;
                mbar_arrive(&bars[B_U_FULL + (n & 1)]);
                if (!u.live) break;
                next = CTAS > 1 ? units : int(gridDim.x) + atomicAdd(p.ws.counters + 1, 1);
                const int tiles[2] = {tiles_of(u, 0), tiles_of(u, 1)};
                const int most = max(tiles[0], tiles[1]);
                auto load_q = [&](int x) {
                    if (tiles[x] == 0) return;
                    ok = ok && (used[x] == 0 || mbar_wait(&bars[B_Q_EMPTY + x], (used[x] - 1) & 1, err));
                    if (!ok) return;
                    mbar_arrive_expect_tx(&bars[B_Q_FULL + x], S::kQBytes);
                    for (int c = 0; c < S::kKBoxes; ++c)
                        tc_load_3d(base + x * S::kQBytes + c * kBox, &map_q, c * 64, u.head, u.q0 + x * kT,
                                   &bars[B_Q_FULL + x]);
                    ++used[x];
                };
                load_q(0);
                for (int j = 0; j < most && ok; ++j, ++tile) {
                    const int row = u.k0 + j * kT;
                    uint32_t dst;
#ifdef PKV_TEST_SKIP_TILE
                    // wait-timeout test build only, as in latent_attn.cu
                    const bool skip = tile == uint32_t(PKV_TEST_SKIP_TILE);
#else
                    constexpr bool skip = false;
#endif
                    for (int c = 0; c < S::kKBoxes; ++c) {
                        if (!slot(dst)) break;
                        if (skip) continue;
                        if (c == 0) mbar_arrive_expect_tx(&bars[B_K_FULL + (tile & 1)], S::kKBoxes * kBox);
                        if (c < D / 64) tc_load_3d(dst, &map_k, c * 64, u.head, row, &bars[B_K_FULL + (tile & 1)]);
                        else tc_load_3d(dst, &map_r, 0, 0, row, &bars[B_K_FULL + (tile & 1)]);
                    }
                    if (j == 0) load_q(1);
                    for (int c = 0; c < S::kVBoxes && ok; ++c) {
                        if (!slot(dst)) break;
                        if (skip) continue;
                        if (c == 0) mbar_arrive_expect_tx(&bars[B_V_FULL + (tile & 1)], S::kVBoxes * kBox);
                        // D = 128: 64 keys of both halves of the values; D = 64: 128 keys
                        for (int e = 0; e < 2; ++e)
                            tc_load_3d(dst + e * (kBox / 2), &map_v, D == 128 ? e * 64 : 0, u.head,
                                       row + (D == 128 ? c : e) * 64, &bars[B_V_FULL + (tile & 1)]);
                    }
                }
                if (!ok) break;
            }
            if (!ok) *abort_flag = 1;
            // never leave with copies in flight: a group whose boxes were all issued completes
            for (int x = 0; x < 2; ++x)
                if (used[x] > 0) mbar_wait(&bars[B_Q_FULL + x], (used[x] - 1) & 1, err);
            for (uint32_t i = 0; i < 2 && i < tile; ++i) {
                const uint32_t t = tile - 1 - i;
                mbar_wait(&bars[B_K_FULL + (t & 1)], (t >> 1) & 1, err);
                mbar_wait(&bars[B_V_FULL + (t & 1)], (t >> 1) & 1, err);
            }
            if (!ok) {
                // a tile that was cut short by a failed wait: its copies land within the limit
                const uint64_t t0 = global_ns();
                while (global_ns() - t0 < 1000000ull) {
                }
            }
        } else if (warp == kMmaWarp && elect_one()) {
            constexpr uint32_t idesc_s = tc_idesc(kT, kT, false), idesc_o = tc_idesc(kT, D, true);
            const uint64_t qd = tc_smem_desc(base, 16, 1024);
            const uint64_t kd = tc_smem_desc(base + S::kRing, 16, 1024);
            const uint64_t vd = tc_smem_desc(base + S::kRing, kBox / 2, 1024);
            uint32_t tile = 0;                             // the unit's first tile
            uint32_t slot0 = 0;                            // its first slot
            uint32_t used[2] = {0, 0}, steps[2] = {0, 0};
            bool ok = true;
            auto wrap = [](uint32_t s) { return s >= uint32_t(S::kSlots) ? s - S::kSlots : s; };
            for (uint32_t n = 0; ok; ++n) {
                Unit u;
                ok = read_unit(sh, n, err, u);
                mbar_arrive(&bars[B_U_EMPTY + (n & 1)]);
                if (!ok || !u.live || *abort_flag) break;
                const int tiles[2] = {tiles_of(u, 0), tiles_of(u, 1)};
                const int most = max(tiles[0], tiles[1]);
                // S of tile j (slots from `at`) for stream x
                auto issue_s = [&](int x, int j, uint32_t at) {
                    tc_fence_after();
#pragma unroll
                    for (int c = 0; c < S::kKBoxes; ++c)
                        mma_ss4(tmem + x * kT, qd + uint64_t((x * S::kQBytes + c * kBox) >> 4),
                                kd + uint64_t(wrap(at + c) * (kBox >> 4)), idesc_s, c != 0);
                    tc_commit(&bars[B_S_FULL + x]);
                    if (j == tiles[x] - 1) tc_commit(&bars[B_Q_EMPTY + x]);
                    // the last stream that takes the tile gives it back
                    if (x == 1 || j >= tiles[1]) {
#pragma unroll
                        for (int c = 0; c < S::kKBoxes; ++c) tc_commit(&bars[B_EMPTY + wrap(at + c)]);
                    }
                };
                if (most > 0) {
                    ok = mbar_wait(&bars[B_K_FULL + (tile & 1)], (tile >> 1) & 1, err);
                    for (int x = 0; x < 2 && ok; ++x) {
                        if (tiles[x] == 0) continue;
                        ok = mbar_wait(&bars[B_Q_FULL + x], used[x] & 1, err);
                        if (ok) issue_s(x, 0, slot0);
                    }
                }
                for (int j = 0; j < most && ok; ++j) {
                    const uint32_t t = tile + j;
                    const uint32_t v_at = wrap(slot0 + S::kKBoxes);
                    const uint32_t k_next = wrap(slot0 + S::kBoxes);
                    ok = mbar_wait(&bars[B_V_FULL + (t & 1)], (t >> 1) & 1, err);
                    for (int x = 0; x < 2 && ok; ++x) {
                        if (j >= tiles[x]) continue;
                        ok = mbar_wait(&bars[B_P_FULL + 2 * x], steps[x] & 1, err) &&
                             (j != 0 || used[x] == 0 || mbar_wait(&bars[B_O_EMPTY + x], (used[x] - 1) & 1, err));
                        if (!ok) break;
                        tc_fence_after();
                        mma_ts4(tmem + kOCol + x * kT, tmem + x * kT, vd + uint64_t(v_at * (kBox >> 4)), idesc_o,
                                j != 0);
                        const bool last = x == 1 || j >= tiles[1];
                        if (last && D == 128) tc_commit(&bars[B_EMPTY + v_at]);
                        ok = mbar_wait(&bars[B_P_FULL + 2 * x + 1], steps[x] & 1, err);
                        if (!ok) break;
                        tc_fence_after();
                        mma_ts4(tmem + kOCol + x * kT, tmem + x * kT + 32,
                                vd + (D == 128 ? uint64_t(wrap(v_at + 1) * (kBox >> 4))
                                               : uint64_t(v_at * (kBox >> 4) + (kBox >> 5))),
                                idesc_o, 1);
                        ++steps[x];
                        if (j == tiles[x] - 1) tc_commit(&bars[B_O_FULL + x]);
                        if (last) tc_commit(&bars[B_EMPTY + (D == 128 ? wrap(v_at + 1) : v_at)]);
                        if (j + 1 < tiles[x]) {
                            ok = mbar_wait(&bars[B_K_FULL + ((t + 1) & 1)], ((t + 1) >> 1) & 1, err);
                            if (ok) issue_s(x, j + 1, k_next);
                        }
                    }
                    slot0 = k_next;
                }
                tile += most;
                for (int x = 0; x < 2; ++x) used[x] += tiles[x] > 0;
            }
            if (!ok) *abort_flag = 1;
            tc_commit(&bars[B_DRAIN]);
            mbar_wait(&bars[B_DRAIN], 0, err);
        }
        __syncwarp();
        if (CTAS > 1) {
            cluster_sync();
            cluster_sync();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
        const int x = warp >> 2;                           // stream
        const int r = (warp & 3) * 32 + lane;              // its row
        const uint32_t lanes = uint32_t((warp & 3) * 32) << 16;
        const uint32_t s_at = tmem + lanes + x * kT, o_at = tmem + lanes + kOCol + x * kT;
        uint32_t tile = 0, slot0 = 0, steps = 0, used = 0;
        bool ok = true;
        Parts<D>& parts = *reinterpret_cast<Parts<D>*>(smem);
        static_assert(sizeof(Parts<D>) <= S::kRing + S::kSlots * kBox, "shared memory");
        Unit whole = {};                                   // (a cluster's)
        float last_m = -INFINITY, last_l = 0.f;
        for (uint32_t n = 0;; ++n) {
            Unit u;
            ok = __all_sync(0xffffffffu, read_unit(sh, n, err, u));
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[B_U_EMPTY + (n & 1)]);
            if (!ok || !u.live) break;
            const int mine = tiles_of(u, x), most = max(mine, tiles_of(u, x ^ 1));
            const int row = x * kT + r;                    // of the unit
            const int limit = min(row, u.rows - 1) + u.keys - u.rows;   // last key that it sees
            float m = -INFINITY, l = 0.f;
            for (int j = 0; j < mine; ++j, ++steps) {
                ok = __all_sync(0xffffffffu, mbar_wait(&bars[B_S_FULL + x], steps & 1, err));
                if (!ok) break;
                tc_fence_after();
                float s[128];
                {
                    uint32_t v[4][32];
#pragma unroll
                    for (int i = 0; i < 4; ++i) tc_ld32(s_at + 32 * i, v[i]);
                    tc_wait_ld();
#pragma unroll
                    for (int i = 0; i < 128; ++i) s[i] = __uint_as_float(v[i >> 5][i & 31]);
                }
                const int key0 = j * kT;
                if (key0 + kT - 1 > limit) {
#pragma unroll
                    for (int i = 0; i < 128; ++i) s[i] = key0 + i <= limit ? s[i] : -INFINITY;
                }
                float mx[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) mx[i] = max3(s[i], s[i + 4], s[i + 8]);
#pragma unroll
                for (int i = 12; i < 124; i += 8)
#pragma unroll
                    for (int e = 0; e < 4; ++e) mx[e] = max3(mx[e], s[i + e], s[i + 4 + e]);
#pragma unroll
                for (int i = 0; i < 4; ++i) mx[i] = fmaxf(mx[i], s[124 + i]);
                const float top = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]) * p.scale_log2;
                const float m_new = fmaxf(m, top);
                const bool need = m_new > m + kRescale;    // first visible keys included
                float alpha = 1.f;
                if (need) {
                    alpha = exp2_fast(m - m_new);
                    m = m_new;
                    l *= alpha;
                }
                const float ref = m == -INFINITY ? 0.f : -m;
                // S of this tile was issued behind the P V of the one before: O is complete
                if (j > 0 && __any_sync(0xffffffffu, need)) {
#pragma unroll 1
                    for (int c = 0; c < D; c += 32) {
                        uint32_t v[32];
                        tc_ld32(o_at + c, v);
                        tc_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * alpha);
                        tc_st32(o_at + c, v);
                    }
                }
                // values behind the unit's keys are another sequence's or nothing's: zeroed,
                // since 0 times anything must stay 0 (by both streams, each before its P V)
                const int keys = u.keys - key0;
                if (keys < kT) {
                    const uint32_t t = tile + j;
                    ok = __all_sync(0xffffffffu, mbar_wait(&bars[B_V_FULL + (t & 1)], (t >> 1) & 1, err));
                    if (!ok) break;
                    uint32_t first = slot0 + uint32_t(j) * S::kBoxes + S::kKBoxes;
                    constexpr int kVecs = D / 8;           // 16-byte vectors of a row
                    for (int i = r; i < (kT - keys) * kVecs; i += kT) {
                        const int key = keys + i / kVecs, c = i % kVecs;
                        const uint32_t sl = D == 128 ? (first + (key >> 6)) % S::kSlots : first % S::kSlots;
                        const uint32_t at = D == 128 ? (c >> 3) * (kBox / 2) + (key & 63) * 128 + (c & 7) * 16
                                                     : key * 128 + c * 16;
                        *reinterpret_cast<uint4*>(smem + S::kRing + sl * kBox + at) = make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_shared();
                    __syncwarp();                          // the TMEM stores want all lanes at once
                }
                // P = 2^(s scale - m) in bf16 (2^-8 of a weight at most), over S's own columns; the
                // sum is taken of the same rounded weights, so that what is lost does not shift the
                // weighted mean (of equal values too)
                const float2 sc2 = make_float2(p.scale_log2, p.scale_log2);
                // (keeps the arithmetic of the second half behind the store of the first)
                float refc = ref;
                uint32_t w[2][32];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    asm volatile("" : "+f"(refc));
                    const float2 ref2 = make_float2(refc, refc);
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const int at = 64 * c + 2 * i;
                        const float2 e = __ffma2_rn(make_float2(s[at], s[at + 1]), sc2, ref2);
                        w[c][i] = pack_bf16x2(exp2_fast(e.x), exp2_fast(e.y));
                    }
                    tc_st32(s_at + 32 * c, w[c]);
                    tc_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars[B_P_FULL + 2 * x + c]);
                }
                // Beside the product that P has just been stored for (the empty statement keeps the
                // additions here).  Summed in front of the store, with the halves taken apart by
                // shifts, prompts of 64-value heads took 418 us, and take 401; 394 with the
                // weights summed before their rounding
                float2 sum[4] = {};
#pragma unroll
                for (int i = 0; i < 64; ++i) {
                    uint32_t v = w[i >> 5][i & 31];
                    asm volatile("" : "+r"(v));
                    add_pair(sum[i & 3], v);
                }
                l += ((sum[0].x + sum[0].y) + (sum[1].x + sum[1].y)) +
                     ((sum[2].x + sum[2].y) + (sum[3].x + sum[3].y));
            }
            if (!ok) break;
            if (CTAS > 1) {                                // the only one
                whole = u;
                last_m = m;
                last_l = l;
                used = mine;
                continue;
            }
            __nv_bfloat16* dst = p.out + ((int64_t(u.q0) + row) * p.heads + u.head) * D;
            if (mine > 0) {
                ok = __all_sync(0xffffffffu, mbar_wait(&bars[B_O_FULL + x], used & 1, err));
                if (!ok) break;
                tc_fence_after();
                const float inv = limit >= 0 ? 1.f / l : 0.f;
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    uint32_t v[32];
                    tc_ld32(o_at + c, v);
                    tc_wait_ld();
                    if (row < u.rows) {
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            uint32_t o[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                o[e] = limit < 0 ? 0u
                                                 : pack_bf16x2(__uint_as_float(v[16 * i + 2 * e]) * inv,
                                                               __uint_as_float(v[16 * i + 2 * e + 1]) * inv);
                            store_sector(dst + c + 16 * i, o, p.whole_sectors);
                        }
                    }
                    __syncwarp();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[B_O_EMPTY + x]);
                ++used;
            } else if (row < u.rows) {                     // no query of the stream sees a key
                for (int c = 0; c < D; c += 8) *reinterpret_cast<uint4*>(dst + c) = make_uint4(0, 0, 0, 0);
            }
            tile += most;
            slot0 = (slot0 + uint32_t(most) * S::kBoxes) % S::kSlots;
        }
        if (!ok) *abort_flag = 1;
        if (CTAS > 1) {
            // once all products are complete, queries and ring are free
            const int row = x * kT + r;
            ok = __all_sync(0xffffffffu, mbar_wait(&bars[B_DRAIN], 0, err)) && ok;
            tc_fence_after();
            if (used > 0) {
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    uint32_t v[32];
                    tc_ld32(o_at + c, v);
                    tc_wait_ld();
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        *reinterpret_cast<uint4*>(&parts.o[row][c + 4 * i]) =
                            make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                }
            }
            parts.m[row] = last_m;
            parts.l[row] = last_l;
            cluster_sync();
            // a warp a row, every CTAS-th row each
            const int rank = blockIdx.x % CTAS;
            const int keys = whole.keys + rank * whole.most * kT;   // of the unit, not of this CTA's part
            for (int y = rank + CTAS * warp; y < whole.rows && ok; y += CTAS * 8) {
                float pm[CTAS], pl[CTAS], top = -INFINITY, sum = 0.f;
#pragma unroll
                for (int q = 0; q < CTAS; ++q) {
                    pm[q] = load_cluster(in_cta(&parts.m[y], q));
                    pl[q] = load_cluster(in_cta(&parts.l[y], q));
                }
#pragma unroll
                for (int q = 0; q < CTAS; ++q) top = fmaxf(top, pm[q]);
                float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int q = 0; q < CTAS; ++q) {
                    if (!(pl[q] != 0.f)) continue;         // saw no key: nothing was written
                    const float4 v = lane < D / 4 ? load_cluster4(in_cta(&parts.o[y][lane * 4], q)) : acc;
                    const float w = exp2f(pm[q] - top);
                    sum += w * pl[q];
                    acc.x += w * v.x;
                    acc.y += w * v.y;
                    acc.z += w * v.z;
                    acc.w += w * v.w;
                }
                // a query without keys: zeros (one whose scores are all -inf: 0 / 0, as in a CTA alone)
                const float inv = y + keys >= whole.rows ? 1.f / sum : 0.f;
                if (lane < D / 4)
                    *reinterpret_cast<uint2*>(p.out + ((int64_t(whole.q0) + y) * p.heads + whole.head) * D + lane * 4) =
                        make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
            }
            __syncwarp();
            cluster_sync();                                // nobody leaves while its parts are being read
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols)
                     : "memory");
}

// units of a batch whose rows belong to one sequence each: ceil(q / 256) <= 1 + (q - 1) / 256
int64_t fewest_units(const ExpandedArgs& a) {
    const int64_t items = a.num_seqs + int64_t(std::max(0, a.num_query_tokens - a.num_seqs)) / kExpandedRowsBf16;
    return std::min<int64_t>(items, a.ws.max_items) * a.desc->num_heads;
}

template <int D, int CTAS>
int launch(const ExpandedArgs& a) {
    const pkv_expanded_desc* d = a.desc;
    const int H = d->num_heads, dim = D + kExpandedRope;
    // without keys no tile is loaded; the maps then stand on the queries
    const bool none = a.num_keys == 0;
    const int keys = none ? 1 : a.num_keys;
    const int64_t kh = H == 1 || none ? D : d->k_head_stride, vh = H == 1 || none ? D : d->v_head_stride;
    const int64_t kt = keys == 1 ? int64_t(H) * dim : d->k_token_stride;
    const int64_t vt = keys == 1 ? int64_t(H) * dim : d->v_token_stride;
    CUtensorMap mq, mk, mr, mv;
    if (!make_strided_tensor_map(&mq, a.q, dim, H, a.num_query_tokens, dim, int64_t(H) * dim, kT) ||
        !make_strided_tensor_map(&mk, none ? a.q : a.k, D, H, keys, kh, kt, kT) ||
        !make_strided_tensor_map(&mr, none ? a.q : a.k_rope, kExpandedRope, 1, keys, kExpandedRope, kExpandedRope, kT) ||
        !make_strided_tensor_map(&mv, none ? a.q : a.v, D, H, keys, vh, vt, kT / 2))
        return PKV_ERR_CUDA;
    const int st = launch_expanded_plan(a, kExpandedRowsBf16);
    if (st != PKV_OK) return st;
    Params p{a.ws, static_cast<__nv_bfloat16*>(a.out), H, (reinterpret_cast<uintptr_t>(a.out) & 31) == 0,
             float(double(a.scale) * 1.4426950408889634), a.err};
    if (kernel_occupancy<expanded_kernel<D, CTAS>>(kThreads, Shape<D>::kSmem) < 1) return PKV_ERR_CUDA;
    const int64_t units = CTAS > 1 ? fewest_units(a) : int64_t(a.ws.max_items) * H;
    if (units > INT32_MAX - 1024) return PKV_ERR_UNSUPPORTED;
    const int64_t grid = CTAS > 1 ? CTAS * units : std::min<int64_t>(num_sms(), units);
    return cuda_status(launch_pdl(expanded_kernel<D, CTAS>, dim3(unsigned(grid)), dim3(kThreads),
                                  size_t(Shape<D>::kSmem), a.stream, mq, mk, mr, mv, p));
}

}  // namespace

int launch_expanded_bf16(const ExpandedArgs& a) {
    // a cluster for a unit where all find SMs and the keys are tiles enough to share (one head
    // set of 30 units over 556 keys: 18 us by two CTAs, 15 by one)
    const bool wide = a.desc->head_dim == 128;
    if (a.num_keys >= 1024 * int64_t(a.num_seqs)) {
        if (4 * fewest_units(a) <= num_sms()) return wide ? launch<128, 4>(a) : launch<64, 4>(a);
        if (2 * fewest_units(a) <= num_sms()) return wide ? launch<128, 2>(a) : launch<64, 2>(a);
    }
    return wide ? launch<128, 1>(a) : launch<64, 1>(a);
}

}  // namespace pkv
