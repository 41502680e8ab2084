// Attention over a list of blocks for each query row and KV head
// (paged_attention_sparse): exact softmax(q K^T * scale) V over the keys of the
// listed blocks that the row sees.
//
// Each (query row, KV head) reads top_k tiles of K and of V, scattered over the
// pool, and nothing is read twice, so the work is bound by HBM for a batch and
// by latency for a few rows.  A cluster of CTAs shares one (row, head): the
// listed blocks go round the cluster's warps, every warp keeps a running
// (max, sum, output) and tiles of its own that it fills with asynchronous copies
// itself, so that no warp waits for another before the end; the states are then
// merged inside the CTA and, through distributed shared memory, across the
// cluster, in a fixed order and without a workspace.
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>

#include "launch_cache.h"
#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "sparse_common.cuh"

namespace pkv {
namespace {

constexpr unsigned kFull = 0xffffffffu;

struct SparseParams {
    void* out;
    const void* q;
    const void* k_cache;
    const void* v_cache;
    const int32_t* selected;       // [tokens][Hkv][top_k]
    QueryRows rows;
    int32_t num_blocks, num_q_heads, num_kv_heads, top_k;
    float scale_log2;
    int* err;
};

// Floats of a head's outputs in a warp's record: eight more than D, so that the lanes
// that write two dimensions each of eight heads meet different banks (4 rows of 128
// blocks: 9.4 us, 9.5 without).
constexpr int head_floats(int d) { return d + 8; }

// Floats of a warp's record: outputs [G][head_floats], max [G], sum [G], keys seen.
constexpr int record_floats(int g, int d) { return (g * (head_floats(d) + 2) + 1 + 3) & ~3; }

// Floats behind the warps' records: their factors [warp][G], and a CTA's sums [G].
constexpr int factor_floats(int g, int warps) { return ((warps + 1) * g + 3) & ~3; }

// Where a CTA of a cluster finds what the others send it: from each its part of
// the outputs (G * D / cluster floats) and its (max, sum) per head.
template <int D, int kMaxG>
struct Inbox {
    static constexpr int kMaxCluster = 8;
    static constexpr int kFloats = kMaxG * D + kMaxCluster * 2 * kMaxG;
};

// The sum of a CTA that saw no key.
constexpr uint32_t kNoKeys = 0x80000000u;

template <int D, int G>
struct SparseF32Cfg {
    static constexpr int kWarps = 4;
    static constexpr int kThreads = kWarps * 32;
    static constexpr int kTileBytes = kBlockTokens * D * 4;
    static constexpr int kStageBytes = 2 * kTileBytes;
    static constexpr int kQOff = kWarps * kStageBytes;                // q as fp32 [G][D]
    static constexpr int kPOff = kQOff + G * D * 4;                   // weights [warp][G][16]
    static constexpr int kRec = record_floats(G, D);
    static constexpr int kCombOff = kPOff + kWarps * G * kBlockTokens * 4;
    static constexpr int kInboxOff = kCombOff + (kWarps * kRec + factor_floats(G, kWarps)) * 4;
    static constexpr int kSmem = kInboxOff + Inbox<D, G>::kFloats * 4;
};

// 16-byte chunk c of tile row r, so that the reads of eight lanes (four rows,
// two neighbouring chunks) fall into eight different bank groups
__device__ __forceinline__ int chunk_at(int r, int c) { return c ^ ((r & 3) << 1); }

// What this CTA will get from the cluster's CTAs, itself among them, announced
// before any of them can send it.
__device__ __forceinline__ void expect_parts(uint64_t* arrived, int G, int D, uint32_t cs) {
    if (threadIdx.x == 0) {
        mbar_init(arrived, 1);
        fence_mbar_init();
        mbar_arrive_expect_tx(arrived, uint32_t(G * D + int(cs) * 2 * G) * 4);
    }
    __syncwarp();
    cluster_arrive();                                // (waited for before the others are written to)
}

// Merge the CTA's warp states (records in shared memory), then the cluster's,
// and write the outputs of the (row, head): shared by every variant.  Each CTA
// owns a part of the outputs; the others send it theirs by stores that count on
// the owner's mbarrier, so that between the merges a CTA waits for nothing but
// what it needs (with a cluster barrier there the call of 4 rows of 128 blocks and
// that of 8 rows of fp32 took 0.4 us more).  The factors of a head are made once, not
// by every output.
template <typename T, int D, int kMaxG, int kWarps>
__device__ __forceinline__ void merge_and_write(const SparseParams& p, float* comb, float* inbox,
                                                uint64_t* arrived, int t, int h, int G) {
    constexpr int kThreads = kWarps * 32;
    constexpr int kRec = record_floats(kMaxG, D), kHead = head_floats(D);
    const uint32_t cs = cluster_size(), rank = cluster_rank();
    const int part_log2 = 31 - __clz(G * D) - (31 - __clz(int(cs)));   // all powers of two
    const int part = 1 << part_log2;
    const uint32_t in_u = smem_u32(inbox), stats_u = in_u + kMaxG * D * 4;
    const uint32_t bar_u = smem_u32(arrived);
    float* fac = comb + kWarps * kRec;
    T* out = static_cast<T*>(p.out) + (size_t(t) * p.num_q_heads + size_t(h) * G) * D;
    __syncthreads();
    if (cs > 1) cluster_wait();                      // the others have started
    // one head each, and one receiver: the warps' factors over the maxima, and the
    // CTA's statistics
    static_assert(kMaxG * Inbox<D, kMaxG>::kMaxCluster <= kThreads, "a thread for each");
    if (threadIdx.x < uint32_t(G) * cs) {
        const int g = threadIdx.x & (G - 1);
        const uint32_t c = threadIdx.x / uint32_t(G);
        float M = -INFINITY, L = 0.f, seen = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, comb[w * kRec + G * kHead + g]);
        const float Mx = M == -INFINITY ? 0.f : M;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float s = exp2f(comb[w * kRec + G * kHead + g] - Mx);
            L = fmaf(comb[w * kRec + G * kHead + G + g], s, L);
            seen += comb[w * kRec + G * kHead + 2 * G];
            if (c == 0) fac[w * G + g] = s;
        }
        if (cs == 1) {
            // (a row whose list names no key it sees is 0)
            fac[kWarps * G + g] = seen > 0.f ? L : INFINITY;
        } else {
            if (!(seen > 0.f)) L = __uint_as_float(kNoKeys);
            st_async(map_rank(stats_u + (rank * G + g) * 8, c), map_rank(bar_u, c),
                     make_float2(M, L));
        }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < (kMaxG * D / 4 + kThreads - 1) / kThreads; ++k) {
        const int i = (k * kThreads + threadIdx.x) * 4;
        if (i >= G * D) break;
        const int g = i / D;
        float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float4 o = *reinterpret_cast<const float4*>(comb + w * kRec + g * kHead + i % D);
            const float s = fac[w * G + g];
            O.x = fmaf(o.x, s, O.x);
            O.y = fmaf(o.y, s, O.y);
            O.z = fmaf(o.z, s, O.z);
            O.w = fmaf(o.w, s, O.w);
        }
        if (cs == 1) {
            const float L = fac[kWarps * G + g];
            const float v[4] = {O.x / L, O.y / L, O.z / L, O.w / L};
#pragma unroll
            for (int e = 0; e < 4; ++e) out[i + e] = Elem<T>::store_val(v[e]);
        } else {
            const uint32_t owner = uint32_t(i >> part_log2);
            st_async(map_rank(in_u + (rank * part + (i & (part - 1))) * 4, owner),
                     map_rank(bar_u, owner), O);
        }
    }
    if (cs == 1) return;
    if (!mbar_wait(arrived, 0, p.err)) return;
    const float2* stats = reinterpret_cast<const float2*>(inbox + kMaxG * D);
    for (int i = threadIdx.x; i < part; i += kThreads) {
        const int at = int(rank) * part + i, g = at / D;
        float M = -INFINITY, L = 0.f, O = 0.f;
        bool seen = false;
        for (uint32_t c = 0; c < cs; ++c) M = fmaxf(M, stats[c * G + g].x);
        const float Mx = M == -INFINITY ? 0.f : M;
        for (uint32_t c = 0; c < cs; ++c) {
            const float2 ml = stats[c * G + g];
            const float s = exp2f(ml.x - Mx);
            L = fmaf(ml.y, s, L);
            O = fmaf(inbox[c * part + i], s, O);
            seen |= __float_as_uint(ml.y) != kNoKeys;
        }
        out[at] = Elem<T>::store_val(seen ? O / L : 0.f);
    }
}

// A warp's own list entries: tile j of the warp is entry first + j * stride.
// Entry `e`, block b -> physical block, 32 tiles at a time.
struct ListCursor {
    int phys, logical;                   // this lane's tile of the current 32
};
__device__ __forceinline__ ListCursor fetch_tiles(const SparseParams& p, int b, int seq,
                                                  int blocks, int e) {
    ListCursor c{-1, 0};
    if (e < p.top_k && blocks > 0) {             // (a context out of range is flagged as such)
        if (b >= blocks) {
            flag_error(p.err, PKV_DEV_BAD_BLOCK_ID);
        } else if (b >= 0) {
            const int id = p.rows.block_tables[size_t(seq) * p.rows.table_stride + b];
            if (id < 0 || id >= p.num_blocks) flag_error(p.err, PKV_DEV_BAD_BLOCK_ID);
            else c = ListCursor{id, b};
        }
    }
    return c;
}

// On CUDA cores (fp32 caches).  A warp holds one tile at a time: the products are
// long next to its copy, and three or more CTAs on an SM hide one warp's copy
// behind the others' products better than a ring of tiles in one CTA does (at the
// step that chose, groups of 4, 64 dimensions, four tiles a warp took 1.8 times as
// long).  64 rows x 8 heads x 64 blocks, groups of 1 / 4 / 8: 64 dimensions (269 MB,
// 40 us at HBM's rate) 50 / 46 / 75 us, 128 dimensions (538 MB, 80 us) 83 / 89 / 112
// us; in groups of 8 bound by the products.
template <int D, int G>
__global__ void __launch_bounds__(SparseF32Cfg<D, G>::kThreads) sparse_attn_f32_kernel(SparseParams p) {
    using C = SparseF32Cfg<D, G>;
    constexpr int RC = D / 4;                    // 16-byte chunks of a row
    constexpr int DL = D / 32;                   // output dimensions of a lane
    constexpr int kHead = head_floats(D);
    extern __shared__ __align__(128) unsigned char smem[];
    float* qs = reinterpret_cast<float*>(smem + C::kQOff);
    float* comb = reinterpret_cast<float*>(smem + C::kCombOff);
    float* inbox = reinterpret_cast<float*>(smem + C::kInboxOff);
    __shared__ uint64_t arrived;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t cs = cluster_size(), rank = cluster_rank();
    const int item = int(blockIdx.x / cs);
    const int t = item / p.num_kv_heads, h = item % p.num_kv_heads;
    if (cs > 1) expect_parts(&arrived, G, D, cs);
    pdl_wait_prerequisites();
    pdl_launch_dependents();
    const int32_t* list = p.selected + size_t(item) * p.top_k;
    const int first = int(rank) * C::kWarps + warp, stride = int(cs) * C::kWarps;
    // the first entries, asked for before the row's context is known
    const int entry0 = first + lane * stride < p.top_k ? list[first + lane * stride] : -1;
    const OffsetStep step(p.rows.start, p.rows.n);
    int seq;
    const int keys = row_keys(p.rows, t, seq,
                              threadIdx.x == 0 && h == 0 && rank == 0 ? p.err : nullptr);
    step.check(p.err);
    if (keys < 0) {                              // the whole cluster: left as it is
        if (cs > 1) cluster_wait();
        return;
    }
    const int blocks = (keys + kBlockTokens - 1) / kBlockTokens;
    for (int i = threadIdx.x; i < G * D; i += C::kThreads)
        qs[i] = static_cast<const float*>(p.q)[(size_t(t) * p.num_q_heads + size_t(h) * G) * D + i];
    __syncthreads();

    const int tiles = p.top_k > first ? (p.top_k - first + stride - 1) / stride : 0;
    unsigned char* kt = smem + warp * C::kStageBytes;
    unsigned char* vt = kt + C::kTileBytes;
    float* ps = reinterpret_cast<float*>(smem + C::kPOff) + warp * (G * kBlockTokens);
    ListCursor now{-1, 0};

    float o[G][DL], m[G], l[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
        m[g] = -INFINITY;
        l[g] = 0.f;
#pragma unroll
        for (int d = 0; d < DL; ++d) o[g][d] = 0.f;
    }
    int seen = 0;
    const int key = lane >> 1, half = lane & 1;
    for (int j = 0; j < tiles; ++j) {
        if (j % 32 == 0) {
            const int e = first + (j + lane) * stride;
            now = fetch_tiles(p, j ? (e < p.top_k ? list[e] : -1) : entry0, seq, blocks, e);
        }
        const int id = __shfl_sync(kFull, now.phys, j % 32);
        const int b = __shfl_sync(kFull, now.logical, j % 32);
        if (id < 0) continue;
        const size_t off = (size_t(id) * p.num_kv_heads + h) * (kBlockTokens * D);
        const float* ks = static_cast<const float*>(p.k_cache) + off;
        const float* vs = static_cast<const float*>(p.v_cache) + off;
        // rows past the row's keys are zero (they may hold anything; 0 x NaN is NaN)
        const int live = keys - b * kBlockTokens;
        const uint32_t dst = smem_u32(kt);
#pragma unroll
        for (int i = 0; i < kBlockTokens * RC / 32; ++i) {
            const int idx = i * 32 + lane, r = idx / RC, c = idx % RC;
            const uint32_t at = dst + (r * RC + chunk_at(r, c)) * 16;
            cp_async16(at, ks + idx * 4, r < live);
            cp_async16(at + C::kTileBytes, vs + idx * 4, r < live);
        }
        cp_commit();
        cp_wait<0>();
        __syncwarp();
        const int nvalid = min(kBlockTokens, keys - b * kBlockTokens);
        seen += nvalid;
        // scores: two lanes a key, chunks taken in turn
        float s[G];
#pragma unroll
        for (int g = 0; g < G; ++g) s[g] = 0.f;
#pragma unroll
        for (int i = 0; i < RC / 2; ++i) {
            const int c = 2 * i + half;
            const float4 x = *reinterpret_cast<const float4*>(kt + (key * RC + chunk_at(key, c)) * 16);
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const float4 qv = *reinterpret_cast<const float4*>(qs + g * D + c * 4);
                s[g] = fmaf(x.x, qv.x, s[g]);
                s[g] = fmaf(x.y, qv.y, s[g]);
                s[g] = fmaf(x.z, qv.z, s[g]);
                s[g] = fmaf(x.w, qv.w, s[g]);
            }
        }
#pragma unroll
        for (int g = 0; g < G; ++g) {
            s[g] += __shfl_xor_sync(kFull, s[g], 1);
            s[g] = key < nvalid ? s[g] * p.scale_log2 : -INFINITY;
            float mx = s[g];
#pragma unroll
            for (int of = 2; of < 32; of <<= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, of));
            const float mn = fmaxf(m[g], mx);
            const float mz = mn == -INFINITY ? 0.f : mn;    // nothing above -inf so far
            const float alpha = exp2f(m[g] - mz), w = exp2f(s[g] - mz);
            m[g] = mn;
            l[g] = l[g] * alpha + (half ? 0.f : w);
#pragma unroll
            for (int d = 0; d < DL; ++d) o[g][d] *= alpha;
            if (!half) ps[g * kBlockTokens + key] = w;
        }
        __syncwarp();
        // four keys at a time, their weights in one load a head
#pragma unroll
        for (int k = 0; k < kBlockTokens; k += 4) {
            float v[4][DL];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int byte = lane * DL * 4;
                const int chunk = (k + e) * RC + chunk_at(k + e, byte / 16);
                const unsigned char* src = vt + chunk * 16 + byte % 16;
                Elem<float>::load(reinterpret_cast<const float*>(src), v[e]);
            }
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const float4 w = *reinterpret_cast<const float4*>(ps + g * kBlockTokens + k);
#pragma unroll
                for (int d = 0; d < DL; ++d) {
                    o[g][d] = fmaf(w.x, v[0][d], o[g][d]);
                    o[g][d] = fmaf(w.y, v[1][d], o[g][d]);
                    o[g][d] = fmaf(w.z, v[2][d], o[g][d]);
                    o[g][d] = fmaf(w.w, v[3][d], o[g][d]);
                }
            }
        }
        __syncwarp();
    }
    float* rec = comb + warp * C::kRec;
#pragma unroll
    for (int g = 0; g < G; ++g) {
#pragma unroll
        for (int of = 1; of < 32; of <<= 1) l[g] += __shfl_xor_sync(kFull, l[g], of);
#pragma unroll
        for (int d = 0; d < DL; ++d) rec[g * kHead + lane * DL + d] = o[g][d];
        if (lane == 0) {
            rec[G * kHead + g] = m[g];
            rec[G * kHead + G + g] = l[g];
        }
    }
    if (lane == 0) rec[G * (kHead + 2)] = float(seen);
    merge_and_write<float, D, G, C::kWarps>(p, comb, inbox, &arrived, t, h, G);
}

// ---- bf16 on tensor cores -------------------------------------------------------
__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
// d += a (16 x 16) . b (16 x 8): this lane's a0, a2 of row lane / 4, a1, a3 of row lane / 4 + 8
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same for rows lane / 4 + 8 alone: d2, d3 += a . b, rows of zeros above them.  (Those
// rows' sums go nowhere: zeros times an infinite b are not zero.)
__device__ __forceinline__ void mma16816_lower(float (&d)[4], uint32_t a1, uint32_t a3, uint32_t b0,
                                               uint32_t b1) {
    float above[2];
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%4,%6}, "
        "{%7,%8}, {%9,%9,%2,%3};"
        : "=f"(above[0]), "=f"(above[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(0u), "r"(a1), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// The upper halves of two words: bf16 values that are the words' leading bits.
__device__ __forceinline__ uint32_t upper2(uint32_t lo, uint32_t hi) {
    return __byte_perm(lo, hi, 0x7632);
}

template <int D>
struct SparseBf16Cfg {
    static constexpr int kWarps = 4;
    static constexpr int kThreads = kWarps * 32;
    static constexpr int kMaxG = 8;
    static constexpr int kTileBytes = kBlockTokens * D * 2;
    static constexpr int kStageBytes = 2 * kTileBytes;
    static constexpr int kStages = D == 128 ? 3 : 6;
    static constexpr int kRingBytes = kWarps * kStages * kStageBytes;
    static constexpr int kRec = record_floats(kMaxG, D);
    // (the warps' records go over the ring)
    static constexpr int kSmem = kRingBytes + Inbox<D, kMaxG>::kFloats * 4;
    static_assert((kWarps * kRec + factor_floats(kMaxG, kWarps)) * 4 <= kRingBytes,
                  "records fit into the ring");
};

// The same work on warp-level tensor-core products (m16n8k16): S = q K^T with
// the group's query heads as rows 0 .. G-1, then O += P V.  A weight of P enters the
// product whole, as three bf16 values of eight of its 24 bits each: rows 0-7 carry
// the leading bits and rows 8-15, which the heads leave free, the next ones; the last
// ones go through a second product into rows 8-15.  (Without the second product, P to
// 2^-17, 0.23 % of the outputs were a bf16 step away from the nearest value; 0.02 %
// are, 0.04 % of those of a sum in single precision.  It costs 0.4 us of 9.4 for 4
// rows of 128 blocks and 1 % of a batch.  As O^T = V^T P^T, the heads as columns, the
// three parts take three products of 16 dimensions in place of four, but the call
// 10.3 us.)  A ring of three tiles a warp and two CTAs an SM keep 192 KB in flight:
// 256 rows x 8 heads x 64 blocks (1.07 GB) 161 us, 6.7 TB/s (two tiles and three CTAs
// 4 % more); 4 rows x 8 heads x 128 blocks (34 MB), in clusters of 8, 9.8 us.
template <int D>
__global__ void __launch_bounds__(SparseBf16Cfg<D>::kThreads) sparse_attn_bf16_kernel(SparseParams p) {
    using C = SparseBf16Cfg<D>;
    constexpr int RC = D / 8;                    // 16-byte chunks of a row
    constexpr int kHead = head_floats(D);
    extern __shared__ __align__(128) unsigned char smem[];
    float* comb = reinterpret_cast<float*>(smem);
    float* inbox = reinterpret_cast<float*>(smem + C::kRingBytes);
    __shared__ uint64_t arrived;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int gid = lane >> 2, tig = lane & 3, mi = lane >> 3;
    const int G = p.num_q_heads / p.num_kv_heads;
    const uint32_t cs = cluster_size(), rank = cluster_rank();
    const int item = int(blockIdx.x / cs);
    const int t = item / p.num_kv_heads, h = item % p.num_kv_heads;
    if (cs > 1) expect_parts(&arrived, G, D, cs);
    pdl_wait_prerequisites();
    pdl_launch_dependents();
    const int32_t* list = p.selected + size_t(item) * p.top_k;
    const int first = int(rank) * C::kWarps + warp, stride = int(cs) * C::kWarps;
    // the first entries, asked for before the row's context is known
    const int entry0 = first + lane * stride < p.top_k ? list[first + lane * stride] : -1;
    const OffsetStep step(p.rows.start, p.rows.n);
    int seq;
    const int keys = row_keys(p.rows, t, seq,
                              threadIdx.x == 0 && h == 0 && rank == 0 ? p.err : nullptr);
    step.check(p.err);
    if (keys < 0) {                              // the whole cluster: left as it is
        if (cs > 1) cluster_wait();
        return;
    }
    const int blocks = (keys + kBlockTokens - 1) / kBlockTokens;
    const int tiles = p.top_k > first ? (p.top_k - first + stride - 1) / stride : 0;
    const uint32_t ring = smem_u32(smem) + warp * (C::kStages * C::kStageBytes);

    auto fetch = [&](int j) {
        const int e = first + (j + lane) * stride;
        return fetch_tiles(p, j ? (e < p.top_k ? list[e] : -1) : entry0, seq, blocks, e);
    };
    ListCursor next{-1, 0}, now{-1, 0};
    auto request = [&](int j) {
        if (j < tiles) {
            if (j % 32 == 0) next = fetch(j);
            const int id = __shfl_sync(kFull, next.phys, j % 32);
            if (id >= 0) {
                const size_t off = (size_t(id) * p.num_kv_heads + h) * (kBlockTokens * D);
                const __nv_bfloat16* ks = static_cast<const __nv_bfloat16*>(p.k_cache) + off;
                const __nv_bfloat16* vs = static_cast<const __nv_bfloat16*>(p.v_cache) + off;
                const uint32_t dst = ring + (j % C::kStages) * C::kStageBytes;
                // rows past the row's keys are zero (they may hold anything; 0 x NaN is NaN)
                const int live = keys - __shfl_sync(kFull, next.logical, j % 32) * kBlockTokens;
#pragma unroll
                for (int i = 0; i < kBlockTokens * RC / 32; ++i) {
                    const int idx = i * 32 + lane, r = idx / RC, c = idx % RC;
                    // chunk c of row r lies at c ^ (r % 8): ldmatrix reads without conflicts
                    const uint32_t at = dst + (r * RC + (c ^ (r & 7))) * 16;
                    cp_async16(at, ks + idx * 8, r < live);
                    cp_async16(at + C::kTileBytes, vs + idx * 8, r < live);
                }
            }
        }
        cp_commit();
    };
    for (int j = 0; j < C::kStages - 1; ++j) request(j);

    // q as the A operand: row gid is query head gid of the group
    uint32_t q0[D / 16], q2[D / 16];
    {
        const uint32_t* q = reinterpret_cast<const uint32_t*>(p.q) +
                            (size_t(t) * p.num_q_heads + size_t(h) * G + (gid < G ? gid : 0)) * (D / 2);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
            q0[ks] = gid < G ? q[ks * 8 + tig] : 0u;
            q2[ks] = gid < G ? q[ks * 8 + 4 + tig] : 0u;
        }
    }
    float o[D / 8][4];
#pragma unroll
    for (int n = 0; n < D / 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
    float m = -INFINITY, l = 0.f;
    int seen = 0;
    for (int j = 0; j < tiles; ++j) {
        request(j + C::kStages - 1);
        if (j % 32 == 0) now = j ? fetch(j) : next;
        const int id = __shfl_sync(kFull, now.phys, j % 32);
        const int b = __shfl_sync(kFull, now.logical, j % 32);
        cp_wait<C::kStages - 1>();
        __syncwarp();
        if (id < 0) continue;
        const uint32_t kt = ring + (j % C::kStages) * C::kStageBytes, vt = kt + C::kTileBytes;
        const int nvalid = min(kBlockTokens, keys - b * kBlockTokens);
        seen += nvalid;
        // S: keys 0-7 and 8-15
        float s0[4] = {0.f, 0.f, 0.f, 0.f}, s1[4] = {0.f, 0.f, 0.f, 0.f};
        {
            const int r = ((mi >> 1) << 3) + (lane & 7);
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                uint32_t f[4];
                ldsm_x4(kt + (r * RC + ((ks * 2 + (mi & 1)) ^ (r & 7))) * 16, f);
                mma16816(s0, q0[ks], 0u, q2[ks], 0u, f[0], f[1]);
                mma16816(s1, q0[ks], 0u, q2[ks], 0u, f[2], f[3]);
            }
        }
        // this lane's keys of row gid: 2 tig, 2 tig + 1, 8 + 2 tig, 9 + 2 tig
        float v[4] = {s0[0], s0[1], s1[0], s1[1]};
        float mx = -INFINITY;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int key = (i >> 1) * 8 + 2 * tig + (i & 1);
            v[i] = key < nvalid ? v[i] * p.scale_log2 : -INFINITY;
            mx = fmaxf(mx, v[i]);
        }
        mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 2));
        const float mn = fmaxf(m, mx);
        const float mz = mn == -INFINITY ? 0.f : mn;     // nothing above -inf so far
        const float alpha = exp2f(m - mz);
        uint32_t part[3][4];                     // eight leading bits, the next eight, the last
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float w = exp2f(v[i] - mz);
            sum += w;
            part[0][i] = __float_as_uint(w) & 0xffff0000u;
            const float behind = w - __uint_as_float(part[0][i]);
            part[1][i] = __float_as_uint(behind) & 0xffff0000u;
            part[2][i] = __float_as_uint(behind - __uint_as_float(part[1][i]));
        }
        l = l * alpha + sum;
        m = mn;
        if (__any_sync(kFull, alpha != 1.f)) {
#pragma unroll
            for (int n = 0; n < D / 8; ++n) {
                o[n][0] *= alpha;
                o[n][1] *= alpha;
                o[n][2] *= alpha;
                o[n][3] *= alpha;
            }
        }
        const uint32_t a0 = upper2(part[0][0], part[0][1]), a2 = upper2(part[0][2], part[0][3]);
        const uint32_t a1 = upper2(part[1][0], part[1][1]), a3 = upper2(part[1][2], part[1][3]);
        const uint32_t b1 = upper2(part[2][0], part[2][1]), b3 = upper2(part[2][2], part[2][3]);
        {
            const int r = ((mi & 1) << 3) + (lane & 7);
            uint32_t f[D / 16][4];
#pragma unroll
            for (int n = 0; n < D / 16; ++n) {
                ldsm_x4_t(vt + (r * RC + ((n * 2 + (mi >> 1)) ^ (r & 7))) * 16, f[n]);
                mma16816(o[2 * n], a0, a1, a2, a3, f[n][0], f[n][1]);
                mma16816(o[2 * n + 1], a0, a1, a2, a3, f[n][2], f[n][3]);
            }
#pragma unroll
            for (int n = 0; n < D / 16; ++n) {
                mma16816_lower(o[2 * n], b1, b3, f[n][0], f[n][1]);
                mma16816_lower(o[2 * n + 1], b1, b3, f[n][2], f[n][3]);
            }
        }
        __syncwarp();
    }
    cp_wait<0>();
    __syncthreads();                             // every warp is done with the ring
    l += __shfl_xor_sync(kFull, l, 1);
    l += __shfl_xor_sync(kFull, l, 2);
    float* rec = comb + warp * C::kRec;
    if (gid < G) {
#pragma unroll
        for (int n = 0; n < D / 8; ++n) {
            // (where an infinite value of V makes the sum infinite, P's remainders,
            // of either sign or 0, would turn it into NaN)
            const bool f0 = fabsf(o[n][0]) <= FLT_MAX, f1 = fabsf(o[n][1]) <= FLT_MAX;
            rec[gid * kHead + n * 8 + 2 * tig] = o[n][0] + (f0 ? o[n][2] : 0.f);
            rec[gid * kHead + n * 8 + 2 * tig + 1] = o[n][1] + (f1 ? o[n][3] : 0.f);
        }
        if (tig == 0) {
            rec[G * kHead + gid] = m;
            rec[G * kHead + G + gid] = l;
        }
    }
    if (lane == 0) rec[G * (kHead + 2)] = float(seen);
    merge_and_write<__nv_bfloat16, D, C::kMaxG, C::kWarps>(p, comb, inbox, &arrived, t, h, G);
}

// CTAs that share one (row, head): those that take the fewest steps, when `slots`
// CTAs run at a time.  A step is a tile of every warp; the start of a CTA (three
// dependent loads) and its merge cost about four, the exchange in a cluster one
// more.  (56 items x 169 blocks: 21 us with 8 CTAs each, which is a second wave,
// 16 us with 4.)
int cluster_for(int64_t items, int top_k, int warps, int64_t slots) {
    int best = 1;
    int64_t least = INT64_MAX;
    for (int cs = 1; cs <= 8; cs *= 2) {
        const int64_t waves = (items * cs + slots - 1) / slots;
        const int64_t steps = waves * (ceil_div(top_k, cs * warps) + (cs > 1 ? 5 : 4));
        if (steps < least) least = steps, best = cs;
    }
    return best;
}

template <typename C, auto Kern>
int launch_sparse(const SparseParams& p, int64_t items, cudaStream_t stream) {
    const int per_sm = kernel_occupancy<Kern>(C::kThreads, C::kSmem);
    if (per_sm < 1) return PKV_ERR_CUDA;
    const int cs = cluster_for(items, p.top_k, C::kWarps, int64_t(per_sm) * num_sms());
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(items * cs));
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = unsigned(cs);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cuda_status(cudaLaunchKernelEx(&cfg, Kern, p));
}

template <int D>
int launch_sparse_f32(const SparseParams& p, int64_t items, cudaStream_t s) {
    switch (p.num_q_heads / p.num_kv_heads) {
        case 1: return launch_sparse<SparseF32Cfg<D, 1>, sparse_attn_f32_kernel<D, 1>>(p, items, s);
        case 2: return launch_sparse<SparseF32Cfg<D, 2>, sparse_attn_f32_kernel<D, 2>>(p, items, s);
        case 4: return launch_sparse<SparseF32Cfg<D, 4>, sparse_attn_f32_kernel<D, 4>>(p, items, s);
        default: return launch_sparse<SparseF32Cfg<D, 8>, sparse_attn_f32_kernel<D, 8>>(p, items, s);
    }
}

bool aligned_to(const void* p, uintptr_t a) {
    return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" int paged_attention_sparse(void* out, const void* q, const void* k_cache,
                                      const void* v_cache, const pkv_cache_desc* desc,
                                      const int32_t* block_tables, int32_t max_blocks_per_seq,
                                      const int32_t* query_start_loc, const int32_t* context_lens,
                                      const int32_t* selected, int32_t top_k, int32_t num_seqs,
                                      int32_t num_query_tokens, float scale, void* stream) {
    int st = check_desc(desc, true);
    if (st != PKV_OK) return st;
    if (max_blocks_per_seq < 1 || num_seqs < 0 || num_query_tokens < 0 || top_k < 1 ||
        !(scale - scale == 0.f))
        return PKV_ERR_INVALID;
    if (!query_start_loc && num_query_tokens != num_seqs) return PKV_ERR_INVALID;
    const int64_t items = int64_t(num_query_tokens) * desc->num_kv_heads;
    if (items * 8 > INT32_MAX || top_k > PKV_SPARSE_MAX_TOP_K) return PKV_ERR_UNSUPPORTED;
    if (num_seqs == 0 || num_query_tokens == 0) return PKV_OK;
    if (!out || !q || !k_cache || !v_cache || !block_tables || !context_lens || !selected ||
        !aligned_to(out, 16) || !aligned_to(q, 16) || !aligned_to(k_cache, 16) ||
        !aligned_to(v_cache, 16) || !aligned_to(block_tables, 4) ||
        !aligned_to(query_start_loc, 4) || !aligned_to(context_lens, 4) ||
        !aligned_to(selected, 4))
        return PKV_ERR_INVALID;
    SparseParams p;
    p.err = device_error_ptr(&st);
    if (st != PKV_OK) return st;
    p.out = out;
    p.q = q;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.selected = selected;
    p.rows = QueryRows{block_tables, query_start_loc, context_lens, max_blocks_per_seq, num_seqs,
                       INT32_MAX, num_query_tokens};
    p.num_blocks = desc->num_blocks;
    p.num_q_heads = desc->num_q_heads;
    p.num_kv_heads = desc->num_kv_heads;
    p.top_k = top_k;
    p.scale_log2 = scale * 1.4426950408889634f;
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    if (desc->dtype == PKV_BF16)
        return desc->head_dim == 128
                   ? launch_sparse<SparseBf16Cfg<128>, sparse_attn_bf16_kernel<128>>(p, items, cs)
                   : launch_sparse<SparseBf16Cfg<64>, sparse_attn_bf16_kernel<64>>(p, items, cs);
    return desc->head_dim == 128 ? launch_sparse_f32<128>(p, items, cs)
                                 : launch_sparse_f32<64>(p, items, cs);
}
