// What the kernels over a latent cache share: the batch, how its work is split over
// the CTAs, and the tcgen05 / TMA instructions.
//
// Latent attention keeps one vector per token for all heads: latent_dim values c and
// 64 rotated key values k.  A head's absorbed query (a, b) scores a token with
// a . c + b . k and sums the c themselves:  out = sum_j p_j c_j.  All heads read the
// same keys, so a row of the products is a (token, head) pair of one sequence.
//
// Split.  CTAs work in teams: the members of a team take neighbouring tiles of ROWS rows
// of the same sequence over the same keys at the same time, so that what one of them
// brings into L2 the others find there (one after the other, 128 heads over more keys than
// L2 holds read HBM twice).  A unit is (sequence, row tiles of a team); it costs one step
// for each tile of KEYS keys of its context.  The steps of all units, one after the other,
// are cut into as many equal stretches as there are teams, so every SM reads the same
// number of keys whatever the lengths.  A unit also costs START steps in front of its tiles,
// in which nothing is done: they stand for the time of its queries, its output and the gap
// between two units, so that the stretches with several short units do not end last (64
// requests of 512 to 4096 tokens, 32 heads: 46.9 us without, 45.1 with four; 99 of 43 to 398
// tokens, 48 heads: 22.3 and 18.5).  A stretch is a run of fragments; one that holds
// all keys of its unit writes the output, another one its partial state (max, sum, output)
// to a slot of its CTA: only a CTA's first and last fragment can be partial, so there are
// two slots a CTA and the workspace does not grow with the batch.  A merge kernel joins
// the states of each cut unit in the order of its keys.
#pragma once

#include <cuda.h>

#include <algorithm>

#include "latent_split.h"
#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {

constexpr int kLatentRope = 64;            // rotated key values of a token
constexpr int kLatentRowTile = 64;         // most rows whose state one CTA writes (sizes the workspace)

struct LatentBatch {
    const int32_t* block_tables;
    const int32_t* context_lens;
    const int32_t* query_start_loc;        // null: one query token a sequence
    int32_t table_stride;
    int32_t num_blocks;
    int32_t num_seqs;
    int32_t num_query_tokens;
    int32_t max_context_len;
    int32_t heads;
    int32_t latent;                        // latent_dim
    int32_t team;                          // CTAs of a team
    float scale_log2;
    int* err;
};

// One merge: the rows of a cut unit and the CTAs whose slots hold its fragments.
struct LatentMerge {
    int32_t row0, nrows;                   // rows of q and out ([token][head] order)
    int32_t first, last;                   // CTAs, a team's size apart; nrows 0: nothing to merge
    int32_t first_slot;                    // the first fragment's slot (the others': 2 c)
};

struct LatentWorkspace {
    LatentMerge* merge;                    // [CTAs]
    float2* ml;                            // [2 CTAs][kLatentRowTile] (max in log2 units, sum)
    float* o;                              // [2 CTAs][kLatentRowTile * latent]
};

// A sequence's share of the batch.  Lengths that the call does not allow are flagged
// by `flag` and leave no rows; `zero` says that its output rows are to be zeroed.
struct LatentSeq {
    int q0, qlen, ctx;
    bool zero;
};
template <bool kFlag>
__device__ __forceinline__ LatentSeq latent_seq(const LatentBatch& b, int s) {
    LatentSeq x;
    x.q0 = s;
    x.qlen = 1;
    x.zero = false;
    x.ctx = __ldg(b.context_lens + s);
    if (b.query_start_loc) {
        x.q0 = __ldg(b.query_start_loc + s);
        const int q1 = __ldg(b.query_start_loc + s + 1);
        if (x.q0 < 0 || q1 < x.q0 || q1 > b.num_query_tokens || (s == 0 && x.q0 != 0)) {
            if (kFlag) flag_error(b.err, PKV_DEV_BAD_QUERY_LAYOUT);
            x.qlen = 0;
            return x;
        }
        x.qlen = q1 - x.q0;
    }
    if (x.qlen > 0) {
        if (x.ctx < x.qlen || x.ctx > b.max_context_len) {
            if (kFlag) flag_error(b.err, PKV_DEV_BAD_CONTEXT_LEN);
            x.zero = true;
        } else if ((x.ctx - 1) / kBlockTokens >= b.table_stride) {
            if (kFlag) flag_error(b.err, PKV_DEV_TABLE_TOO_NARROW);
            x.zero = true;
        }
    }
    return x;
}

// A stretch's part of one unit: key tiles kt0 .. kt0 + n - 1 (n may be 0 where the
// rows' causal limit lies in front of them).
struct LatentFrag {
    int seq, ctx;
    int row0, nrows;                       // rows of q and out
    int t0;                                // (row in sequence of row0) / heads is row r's token
    int rest;                              // row in sequence of row0, modulo heads
    int first_pos;                         // position of the sequence's first query token
    int kt0, n;
    bool whole;                            // holds all keys of its unit
    bool starts;                           // begins with the unit's first key, but is cut
    int slot;
    int last_cta;                          // the CTA of the rows' last key (starts)
};

template <int ROWS, int KEYS, int START>
struct LatentWalk {
    int s;
    int64_t off;                           // step within sequence s
    int64_t left;                          // steps left of this team's stretch
    int64_t pos, total;                    // position among all steps
    int teams;
    int cta;                               // (of the kernel's work; a pair counts as one)
    bool begun;

    __device__ static int groups(const LatentBatch& b, int rows) {
        return ((rows + ROWS - 1) / ROWS + b.team - 1) / b.team;
    }
    __device__ static int64_t steps(const LatentBatch& b, const LatentSeq& x) {
        if (x.qlen == 0 || x.zero) return 0;
        return int64_t(groups(b, x.qlen * b.heads)) * ((x.ctx + KEYS - 1) / KEYS + START);
    }
    __device__ bool next(const LatentBatch& b, LatentFrag& f) {
        for (;;) {
            if (left <= 0) return false;
            if (step(b, f)) return true;
        }
    }
    // one unit's part of the stretch; false if that lies in front of the unit's tiles
    __device__ bool step(const LatentBatch& b, LatentFrag& f) {
        LatentSeq x = latent_seq<false>(b, s);
        while (steps(b, x) == 0) x = latent_seq<false>(b, ++s);
        const int seq = s;
        const int rows = x.qlen * b.heads;
        const int kt = (x.ctx + KEYS - 1) / KEYS, len = kt + START;
        const int group = int((off >> 32) == 0 ? uint32_t(off) / uint32_t(len) : off / len);
        const int at = int(off - int64_t(group) * len);    // step of the unit
        int n = len - at;
        if (n > left) n = int(left);
        const int64_t last = pos + len - at - 1;           // the unit's last step
        left -= n;
        pos += n;
        off += n;
        if (off == int64_t(groups(b, rows)) * len) {
            off = 0;
            ++s;
        }
        const int end = at + n - START;
        if (end <= 0) return false;
        f.kt0 = max(0, at - START);
        const int r0 = (group * b.team + cta % b.team) * ROWS;
        f.seq = seq;
        f.ctx = x.ctx;
        f.nrows = max(0, min(ROWS, rows - r0));
        f.row0 = x.q0 * b.heads + r0;
        f.t0 = r0 / b.heads;
        f.rest = r0 - f.t0 * b.heads;
        f.first_pos = x.ctx - x.qlen;
        f.whole = f.kt0 == 0 && end == kt;
        f.starts = f.kt0 == 0 && end < kt;
        f.slot = 2 * cta + (begun ? 1 : 0);
        f.last_cta = 0;
        f.n = 0;
        if (f.nrows == 0) {                // this member has no rows of the unit
            f.whole = true;
            f.starts = false;
        } else {
            const int last_tok = (r0 + f.nrows - 1) / b.heads;
            const int want = (f.first_pos + last_tok) / KEYS + 1;   // tiles that any row sees
            f.n = max(0, min(end, want) - f.kt0);
            if (f.starts)
                f.last_cta = stretch_of(last, total, teams) * b.team + cta % b.team;
        }
        begun = true;
        return true;
    }
};

// Every CTA sums the steps of all sequences for itself and finds the sequence that
// its stretch begins in: threads 0 .. T-1 take runs of sequences, `sums` is shared
// memory for T / 32 + 2 values.  Steps fewer than `least` a team go to fewer teams.
// (All T threads call it; CTA 0 flags bad lengths.)
template <int ROWS, int KEYS, int START, int T>
__device__ __forceinline__ LatentWalk<ROWS, KEYS, START> latent_plan(const LatentBatch& b, int64_t* sums,
                                                             int least, int cta, int ctas) {
    using Walk = LatentWalk<ROWS, KEYS, START>;
    constexpr int kWarps = T / 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (b.num_seqs + T - 1) / T;
    const int s0 = min(b.num_seqs, tid * per), s1 = min(b.num_seqs, s0 + per);
    int64_t mine = 0;
    for (int s = s0; s < s1; ++s)
        mine += Walk::steps(b, blockIdx.x == 0 ? latent_seq<true>(b, s) : latent_seq<false>(b, s));
    int64_t upto = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d) upto += v;
    }
    if (lane == 31) sums[warp] = upto;
    __syncthreads();
    int64_t total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) upto += sums[w];
        total += sums[w];
    }
    Walk x;
    x.total = total;
    x.cta = cta;
    const int team = cta / b.team;
    x.teams = int(max(int64_t(1), min(int64_t(ctas) / b.team, total / least)));
    x.begun = false;
    const int64_t from = stretch_begin(team, total, x.teams);
    x.left = team < x.teams ? stretch_begin(team + 1, total, x.teams) - from : 0;
    x.pos = from;
    if (x.left > 0 && from < upto && from >= upto - mine) {
        int64_t at = upto - mine;
        int s = s0;
        if (per > 1) {                     // (a run of one is the sequence itself)
            for (;; ++s) {
                const int64_t n = Walk::steps(b, latent_seq<false>(b, s));
                if (from < at + n) break;
                at += n;
            }
        }
        sums[kWarps] = s;
        sums[kWarps + 1] = from - at;
    }
    __syncthreads();
    x.s = int(sums[kWarps]);
    x.off = sums[kWarps + 1];
    return x;
}

// Rows of a sequence, on average: what the host knows of a batch whose offsets lie on the device.
// It chooses the kernel and the size of its units, and neither changes what is computed: a
// sequence of more rows than a unit's is several units.  Rows behind the last sequence (a
// captured call's padding) count, so a call padded far beyond its tokens takes larger units
// than its sequences fill.
inline int64_t latent_rows(const LatentBatch& b) {
    return int64_t(ceil_div(b.num_query_tokens, b.num_seqs)) * b.heads;
}
// CTAs (or pairs) of a team: all row tiles of a sequence, on average, up to 8 of them; of more
// tiles two, since a team's last tiles then seldom have members without rows (41 requests of 28
// tiles: 185 us with two, 196 with eight; keys read by one CTA after the other, without teams:
// 64 requests of two tiles over 2k to 8k tokens 173 us against 160)
inline int latent_team(const LatentBatch& b, int rows) {
    const int64_t tiles = std::max<int64_t>(1, (latent_rows(b) + rows - 1) / rows);
    return tiles <= 8 ? int(tiles) : 2;
}

// The fragments' tiles one after the other, skipping fragments without any.
template <int ROWS, int KEYS, int START>
struct LatentTiles {
    LatentWalk<ROWS, KEYS, START> w;
    LatentFrag f;
    int j;                                 // tile of the fragment
    uint32_t g, k;                         // tiles and fragments (of any tiles) so far
    bool live;
    __device__ void start(const LatentBatch& b, const LatentWalk<ROWS, KEYS, START>& from) {
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

// ---- tcgen05 and TMA ---------------------------------------------------------
__device__ __forceinline__ uint64_t tc_smem_desc(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
    return uint64_t((saddr >> 4) & 0x3FFFu) | uint64_t((lbo >> 4) & 0x3FFFu) << 16 |
           uint64_t((sbo >> 4) & 0x3FFFu) << 32 | uint64_t(1) << 46 /* version */ |
           uint64_t(2) << 61 /* 128-byte swizzle */;
}
// kind::f16, bf16 x bf16 -> fp32, A K-major
__host__ __device__ constexpr uint32_t tc_idesc(int m, int n, bool b_mn_major) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((b_mn_major ? 1u : 0u) << 16) |
           (uint32_t(n >> 3) << 17) | (uint32_t(m >> 4) << 24);
}
// One lane of a converged warp.  Products are issued inside a branch on this and not on a
// lane's number: only then does the compiler know that one thread is active, and takes
// their operands to uniform registers once instead of looping over the lanes (measured: a
// product costs 45 cycles to issue in a branch on the lane's number, whatever its size;
// 24 and less in this one).
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(one));
    return one != 0;
}
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
    asm volatile(
        "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
            smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void tc_fence_before() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_wait_ld() {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tc_wait_st() {
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
#define PKV_TC_R32(r)                                                                           \
    "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),         \
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), \
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),           \
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),           \
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
#define PKV_TC_W32(r)                                                                       \
    "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), \
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),   \
        "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), \
        "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), \
        "r"(r[29]), "r"(r[30]), "r"(r[31])
// 32 consecutive fp32 columns of this thread's TMEM lane
__device__ __forceinline__ void tc_ld32(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
        "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : PKV_TC_R32(r)
        : "r"(taddr));
}
__device__ __forceinline__ void tc_st32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
        "%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(
            taddr),
        PKV_TC_W32(r)
        : "memory");
}
__device__ __forceinline__ void tc_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y,
                                           int z, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
        " selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}
// As mbar_wait, but asleep while it waits: the attempt is given a time that the hardware may
// suspend the thread for.  Without it an attempt comes back soon, and the warps that wait
// take issue slots and shared-memory cycles from the ones that work.
__device__ __forceinline__ bool mbar_wait_asleep(uint64_t* bar, uint32_t parity, int* err) {
    uint64_t t0 = 0;
    for (;;) {
        uint32_t ok;
        asm volatile(
            "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n"
            " selp.u32 %0, 1, 0, p;\n}\n"
            : "=r"(ok)
            : "r"(smem_u32(bar)), "r"(parity), "r"(1000000u)
            : "memory");
        if (ok) return true;
        const uint64_t now = global_ns();
        if (t0 == 0) t0 = now;
        if (now - t0 > kWaitLimitNs) {
            flag_error(err, PKV_DEV_WAIT_TIMEOUT);
            return false;
        }
    }
}

// Tests of two barriers' phases side by side (a round trip of one costs about 90 cycles).
__device__ __forceinline__ bool mbar_test2(uint64_t* a, uint32_t pa, uint64_t* b, uint32_t pb) {
    uint32_t x, y;
    asm volatile(
        "{\n .reg .pred p, q;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%2], %3;\n"
        " mbarrier.test_wait.parity.shared::cta.b64 q, [%4], %5;\n"
        " selp.u32 %0, 1, 0, p;\n selp.u32 %1, 1, 0, q;\n}\n"
        : "=r"(x), "=r"(y)
        : "r"(smem_u32(a)), "r"(pa), "r"(smem_u32(b)), "r"(pb)
        : "memory");
    return x != 0 && y != 0;
}
// a -> low half, b -> high half
__device__ __forceinline__ uint32_t pack_bf16x2(float a, float b) {
    __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&v);
}
// 32 bytes of a row by one thread; a row a thread, so that the halves of a sector written
// one after the other would be two transactions
__device__ __forceinline__ void store_sector(void* dst, const uint32_t (&v)[8], bool whole) {
    if (whole) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(v[0]),
                     "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                     : "memory");
    } else {
        reinterpret_cast<uint4*>(dst)[0] = make_uint4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<uint4*>(dst)[1] = make_uint4(v[4], v[5], v[6], v[7]);
    }
}
// 2^x in one instruction (a few ulps, subnormal results flushed to zero): softmax
// weights and rescale factors only
__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// ---- host ---------------------------------------------------------------------
size_t latent_workspace_layout(const pkv_latent_desc* d, void* base, LatentWorkspace* ws);

struct LatentArgs {
    void* out;
    const void* q;
    const void* cache;
    const pkv_latent_desc* desc;
    LatentBatch batch;
    LatentWorkspace ws;
    cudaStream_t stream;
};
int launch_latent_bf16(const LatentArgs& a);
int launch_latent_pair(const LatentArgs& a);
int launch_latent_f32(const LatentArgs& a);

// tmap.cu: rows of (latent / 64 + 1) x 64 bf16 values, row_bytes apart, as a 3-D tensor
// (64 values, rows, 64-value columns); a box is `box_rows` rows of `box_columns` columns and
// lands column by column, each row's 128 bytes swizzled
bool make_latent_tensor_map(struct CUtensorMap_st* map, const void* base, int64_t rows,
                            int32_t columns, int32_t box_rows, int32_t box_columns);
// tmap.cu: bf16 [tokens][heads][dim] with strides in elements, as (dims, heads, tokens); a
// box is 64 dims of one head, `box_tokens` tokens
bool make_strided_tensor_map(struct CUtensorMap_st* map, const void* base, int32_t dim,
                             int32_t heads, int32_t tokens, int64_t head_stride,
                             int64_t token_stride, int32_t box_tokens);

}  // namespace pkv
