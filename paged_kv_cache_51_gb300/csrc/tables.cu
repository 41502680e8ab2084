// Block tables and slots built on the device from the requests' lengths
// (pkv_tables_step), and their release (pkv_tables_release).
//
// A step is a prefix sum.  Request i holds cached_i tokens and adds new_i, so it
// needs ceil((cached_i + new_i) / bs) - ceil(cached_i / bs) new blocks; with
// N_i the sum of the needs before it, its k-th new block is entry
// count - 1 - (N_i + k) of the free stack, exactly the block that a host pool
// serving the requests one after the other would pop.  Token j of request i
// goes to row j of the batch's tokens behind the T_i tokens of the requests
// before it, at position cached_i + j, slot table[position / bs] * bs +
// position % bs.
//
// The step moves a few hundred KB to a few MB, so it is bound by latency.  Where
// the outputs are not the inputs it is one launch (tables_step_kernel): every CTA
// makes the prefix sums for itself, so that nothing has to be waited for, and
// fills its share of the outputs from them.  A step in place, or of very many
// requests, takes two: tables_plan_kernel (one CTA) does what is sequential by
// nature, the checks, both sums and the few new table entries; tables_fill_kernel
// spreads the copies over the GPU.
#include <cuda_runtime.h>

#include <algorithm>

#include "launch_cache.h"
#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int kPlanThreads = 1024;
constexpr uint32_t kFull = 0xffffffffu;
// Sums saturate here: needs and tokens of a batch may pass 32 bits, the
// capacities they are compared with may not.
constexpr uint32_t kSat = 1u << 30;

struct TablesParams {
    int32_t* table;            // [max_seqs][max_blocks]
    const int32_t* free_list;  // [num_blocks]
    const int32_t* free_count;
    int32_t* free_count_out;
    const int32_t* seq_rows;   // [n] or null (row i)
    const int32_t* cached;     // [n]
    const int32_t* fresh;      // [n] or null (one token each)
    int32_t* out_tables;       // [n][width] or null
    int32_t* ctx;              // [n]
    int32_t* start;            // [n + 1]
    int64_t* slots;            // [max_tokens]
    int32_t* positions;        // [max_tokens] or null
    int32_t n, max_seqs, max_blocks, num_blocks, block_size, width, max_tokens;
    int* err;
};

__device__ __forceinline__ uint32_t sat_add(uint32_t a, uint32_t b) { return min(a + b, kSat); }

// Inclusive saturating scans of two values per thread over a CTA of NT threads;
// `total_*` are the CTA's sums.  (min(a + b, cap) is associative on 0 .. cap.)
template <int NT>
struct ScanScratch {
    uint32_t a[NT / 32], b[NT / 32];
};
template <int NT>
__device__ __forceinline__ void scan_inclusive(uint32_t& a, uint32_t& b, ScanScratch<NT>& s,
                                               uint32_t& total_a, uint32_t& total_b) {
    constexpr int kWarps = NT / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t u = __shfl_up_sync(kFull, a, o), v = __shfl_up_sync(kFull, b, o);
        if (lane >= o) a = sat_add(a, u), b = sat_add(b, v);
    }
    if (lane == 31) s.a[warp] = a, s.b[warp] = b;
    __syncthreads();
    // every warp sums the warps for itself
    uint32_t wa = lane < kWarps ? s.a[lane] : 0u, wb = lane < kWarps ? s.b[lane] : 0u;
#pragma unroll
    for (int o = 1; o < kWarps; o <<= 1) {
        const uint32_t u = __shfl_up_sync(kFull, wa, o), v = __shfl_up_sync(kFull, wb, o);
        if (lane >= o) wa = sat_add(wa, u), wb = sat_add(wb, v);
    }
    total_a = __shfl_sync(kFull, wa, kWarps - 1);
    total_b = __shfl_sync(kFull, wb, kWarps - 1);
    const uint32_t pa = __shfl_sync(kFull, wa, max(warp - 1, 0));
    const uint32_t pb = __shfl_sync(kFull, wb, max(warp - 1, 0));
    if (warp > 0) a = sat_add(a, pa), b = sat_add(b, pb);
    __syncthreads();                              // (the scratch may be written again)
}

// Marks the rows that the batch names more than once: two bit planes over
// max_seqs rows in shared memory, `seen` and `twice`.  `mine` is this thread's
// first row, which it has loaded already.
template <int NT>
__device__ __forceinline__ void mark_rows(const int32_t* rows, int mine, int n, int max_seqs,
                                          uint32_t* seen, uint32_t* twice) {
    const int words = (max_seqs + 31) / 32;
    for (int i = threadIdx.x; i < words; i += NT) seen[i] = twice[i] = 0u;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += NT) {
        const int r = i < NT ? mine : rows[i];
        if (r < 0 || r >= max_seqs) continue;
        const uint32_t bit = 1u << (r & 31);
        if (atomicOr(seen + (r >> 5), bit) & bit) atomicOr(twice + (r >> 5), bit);
    }
    __syncthreads();
}

// The row that request i names, if it is one and named once; else -1.
__device__ __forceinline__ int checked_row(int r, bool listed, int max_seqs, const uint32_t* twice) {
    if (r < 0 || r >= max_seqs) return -1;
    return listed && (twice[r >> 5] >> (r & 31) & 1u) ? -1 : r;
}

__device__ __forceinline__ int64_t blocks_of(int64_t tokens, int bs) {
    return (tokens + bs - 1) / bs;
}

// What a step hands out: running sums over the passes of kPlanThreads requests.
struct StepSums {
    uint32_t need_base = 0, tok_base = 0;         // of the requests before this pass
    uint32_t used = 0, placed = 0;                // of the served ones
};
// Request i as the caller gave it.
struct Given {
    int row, cached, fresh;
};
__device__ __forceinline__ Given load_request(const TablesParams& p, int i) {
    Given g{-1, 0, 0};
    if (i < p.n) {
        g.row = p.seq_rows ? p.seq_rows[i] : i;
        g.cached = p.cached[i];
        g.fresh = p.fresh ? p.fresh[i] : 1;
    }
    return g;
}
struct Request {
    int row, cached, fresh;
    uint32_t need_in, tok_in;                     // sums that include it
    uint32_t need_sum, tok_sum;                   // of the whole pass
    bool ok, served;
};

// One pass: request `i` of this thread, checked and summed.  Served in order up
// to the first request that does not fit: both sums only grow, so no later
// request fits either.
template <int NT>
__device__ __forceinline__ Request plan_pass(const TablesParams& p, int i, Given g,
                                             const uint32_t* twice,
                                             uint32_t have, int64_t limit, ScanScratch<NT>& scratch,
                                             StepSums& s, int* tell) {
    Request r{-1, 0, 0, 0, 0, 0, 0, false, false};
    uint32_t need = 0, tok = 0;
    if (i < p.n) {
        r.row = checked_row(g.row, p.seq_rows != nullptr, p.max_seqs, twice);
        r.cached = g.cached;
        r.fresh = g.fresh;
        if (r.row < 0) {
            flag_error(tell, PKV_DEV_BAD_SEQ_ROW);
        } else if (r.cached < 0 || r.fresh < 0) {
            flag_error(tell, PKV_DEV_BAD_CONTEXT_LEN);
        } else if (int64_t(r.cached) + r.fresh > limit) {
            flag_error(tell, PKV_DEV_TABLE_TOO_NARROW);
        } else {
            r.ok = true;
            need = uint32_t(blocks_of(int64_t(r.cached) + r.fresh, p.block_size) -
                            blocks_of(r.cached, p.block_size));
            tok = min(uint32_t(r.fresh), kSat);
        }
    }
    scan_inclusive<NT>(need, tok, scratch, r.need_sum, r.tok_sum);
    r.need_in = sat_add(s.need_base, need);
    r.tok_in = sat_add(s.tok_base, tok);
    const bool fits = r.need_in <= have && r.tok_in <= uint32_t(p.max_tokens);
    r.served = r.ok && fits;
    if (r.ok && !fits)
        flag_error(tell, r.need_in > have ? PKV_DEV_NO_FREE_BLOCKS : PKV_DEV_BAD_QUERY_LAYOUT);
    // the sums of served requests: the largest, over the CTA
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t u = __reduce_max_sync(kFull, r.served ? r.need_in : 0u);
    const uint32_t q = __reduce_max_sync(kFull, r.served ? r.tok_in : 0u);
    if (lane == 0) scratch.a[warp] = u, scratch.b[warp] = q;
    __syncthreads();
    s.used = max(s.used, __reduce_max_sync(kFull, scratch.a[lane % (NT / 32)]));
    s.placed = max(s.placed, __reduce_max_sync(kFull, scratch.b[lane % (NT / 32)]));
    __syncthreads();
    return r;
}

// The free blocks that a step may take; a count out of range gives none.
__device__ __forceinline__ uint32_t free_blocks(const TablesParams& p, int count, bool& ok) {
    ok = count >= 0 && count <= p.num_blocks;
    return ok ? uint32_t(count) : 0u;
}

// Entry `k` from the top of the free stack: the id, or -1 if it is none.
__device__ __forceinline__ int take_block(const TablesParams& p, uint32_t have, uint32_t k,
                                          int* tell) {
    const int blk = p.free_list[have - 1 - k];
    if (blk >= 0 && blk < p.num_blocks) return blk;
    flag_error(tell, PKV_DEV_BAD_BLOCK_ID);
    return -1;
}

__device__ __forceinline__ int64_t token_limit(const TablesParams& p) {
    return int64_t(min(p.max_blocks, p.out_tables ? p.width : p.max_blocks)) * p.block_size;
}

__global__ void __launch_bounds__(kPlanThreads) tables_plan_kernel(TablesParams p) {
    extern __shared__ uint32_t bits[];            // two planes of max_seqs bits
    __shared__ ScanScratch<kPlanThreads> scratch;
    __shared__ uint32_t need_end[kPlanThreads];   // inclusive needs of the pass's served requests
    __shared__ int32_t dest[kPlanThreads];        // first new table entry of a request ...
    __shared__ int32_t dest_row[kPlanThreads];    // ... in this row
    const uint32_t* twice = bits + (p.max_seqs + 31) / 32;
    pdl_wait_prerequisites();
    pdl_launch_dependents();
    const int free0 = *p.free_count;
    const Given given = load_request(p, threadIdx.x);
    if (p.seq_rows)
        mark_rows<kPlanThreads>(p.seq_rows, given.row, p.n, p.max_seqs, bits,
                                bits + (p.max_seqs + 31) / 32);
    bool free_ok;
    const uint32_t have = free_blocks(p, free0, free_ok);
    if (!free_ok && threadIdx.x == 0) flag_error(p.err, PKV_DEV_BAD_BLOCK_ID);
    __syncthreads();                              // everyone read the count before it is written
    const int64_t limit = token_limit(p);
    StepSums s;
    for (int base = 0; base < p.n; base += kPlanThreads) {
        const int i = base + threadIdx.x;
        const Request r = plan_pass<kPlanThreads>(p, i, base ? load_request(p, i) : given, twice,
                                                  have, limit, scratch, s, p.err);
        if (i < p.n) {
            p.ctx[i] = r.ok ? r.cached + (r.served ? r.fresh : 0) : 0;
            p.start[i + 1] = int32_t(min(r.tok_in, s.placed));
        }
        need_end[threadIdx.x] = min(r.need_in, s.used);
        dest[threadIdx.x] = r.ok ? int32_t(blocks_of(r.cached, p.block_size)) : 0;
        dest_row[threadIdx.x] = r.row;
        __syncthreads();
        // new entries of the pass, one thread each: the request by bisection
        const uint32_t first = min(s.need_base, s.used);
        for (uint32_t b = first + threadIdx.x; b < s.used; b += kPlanThreads) {
            int lo = 0, hi = kPlanThreads - 1;
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (need_end[mid] > b) hi = mid;
                else lo = mid + 1;
            }
            const uint32_t before = lo ? need_end[lo - 1] : first;
            p.table[size_t(dest_row[lo]) * p.max_blocks + dest[lo] + (b - before)] =
                take_block(p, have, b, p.err);
        }
        __syncthreads();
        s.need_base = sat_add(s.need_base, r.need_sum);
        s.tok_base = sat_add(s.tok_base, r.tok_sum);
    }
    if (threadIdx.x == 0) {
        p.start[0] = 0;
        *p.free_count_out = free_ok ? int32_t(have - s.used) : free0;
    }
}

constexpr int kFillThreads = 256;
constexpr int kSegment = 256;     // table entries copied by a warp: eight loads in flight a lane

__global__ void __launch_bounds__(kFillThreads) tables_fill_kernel(TablesParams p, int segments,
                                                                   int copy_warps) {
    pdl_wait_prerequisites();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t warp = (int64_t(blockIdx.x) * kFillThreads + threadIdx.x) >> 5;
    if (warp < copy_warps) {
        const int i = int(warp / segments), j0 = int(warp % segments) * kSegment;
        int row = p.seq_rows ? p.seq_rows[i] : i;
        const int blocks = int(blocks_of(p.ctx[i], p.block_size));   // 0 for a refused request
        if (row < 0 || row >= p.max_seqs) row = 0;
        const int32_t* src = p.table + size_t(row) * p.max_blocks + j0;
        int32_t* dst = p.out_tables + size_t(i) * p.width + j0;
        int32_t v[kSegment / 32];
#pragma unroll
        for (int k = 0; k < kSegment / 32; ++k) {
            const int j = lane + 32 * k;
            v[k] = j0 + j < blocks ? src[j] : -1;
        }
#pragma unroll
        for (int k = 0; k < kSegment / 32; ++k) {
            const int j = lane + 32 * k;
            if (j0 + j < p.width) dst[j] = v[k];
        }
        return;
    }
    const int64_t t64 = (warp - copy_warps) * 32 + lane;
    if (t64 >= p.max_tokens) return;
    const int t = int(t64);
    if (t >= p.start[p.n]) {
        p.slots[t] = -1;
        if (p.positions) p.positions[t] = 0;
        return;
    }
    // the request of token t: itself in a decode batch, else by bisection
    int i = t;
    if (!(t < p.n && p.start[t] <= t && t < p.start[t + 1])) {
        int lo = 0, hi = p.n - 1;
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (p.start[mid + 1] > t) hi = mid;
            else lo = mid + 1;
        }
        i = lo;
    }
    const int pos = p.ctx[i] - (p.start[i + 1] - t);
    const int row = p.seq_rows ? p.seq_rows[i] : i;
    const int blk = p.table[size_t(row) * p.max_blocks + pos / p.block_size];
    if (blk < 0 || blk >= p.num_blocks) flag_error(p.err, PKV_DEV_BAD_BLOCK_ID);
    p.slots[t] = blk < 0 || blk >= p.num_blocks
                     ? -1
                     : int64_t(blk) * p.block_size + pos % p.block_size;
    if (p.positions) p.positions[t] = pos;
}

constexpr int kStepSeqs = 2048;   // most requests of a step in one launch

// A step in one launch, for outputs that are not inputs.  Every CTA checks and
// sums all requests and keeps what the outputs are made of in shared memory; then
// the CTAs fill the outputs side by side.  What another CTA writes is never read:
// a new entry is taken from the free list wherever it is needed.  Device time of a
// call: 64 requests 3.7 us, 515 requests with 2048 tokens 5.2 us, 1024 requests x
// 2049 entries (12.8 MB) 6.8 us; the two launches take 6.0, 7.2 and 7.9 us.
template <int NT>
__global__ void __launch_bounds__(NT) tables_step_kernel(TablesParams p, int segments,
                                                         int copy_warps) {
    extern __shared__ uint32_t dyn[];             // 6 n + 1 words, then two planes of max_seqs bits
    __shared__ ScanScratch<NT> scratch;
    int32_t* row = reinterpret_cast<int32_t*>(dyn);    // -1: refused
    int32_t* old_blocks = row + p.n;              // blocks held, and with the new ones
    int32_t* now_blocks = old_blocks + p.n;
    uint32_t* before = reinterpret_cast<uint32_t*>(now_blocks + p.n);   // new blocks in front
    int32_t* ctx = reinterpret_cast<int32_t*>(before + p.n);
    int32_t* start = ctx + p.n;
    uint32_t* bits = dyn + 6 * p.n + 1;
    const uint32_t* twice = bits + (p.max_seqs + 31) / 32;
    int* const tell = blockIdx.x == 0 ? p.err : nullptr;
    const int lane = threadIdx.x & 31;
    pdl_wait_prerequisites();
    pdl_launch_dependents();
    const int free0 = *p.free_count;
    const Given given = load_request(p, threadIdx.x);
    if (p.seq_rows)
        mark_rows<NT>(p.seq_rows, given.row, p.n, p.max_seqs, bits,
                      bits + (p.max_seqs + 31) / 32);
    bool free_ok;
    const uint32_t have = free_blocks(p, free0, free_ok);
    if (!free_ok && threadIdx.x == 0) flag_error(tell, PKV_DEV_BAD_BLOCK_ID);
    const int64_t limit = token_limit(p);
    StepSums s;
    if (threadIdx.x == 0) start[0] = 0;
    for (int base = 0; base < p.n; base += NT) {
        const int i = base + threadIdx.x;
        const Request r = plan_pass<NT>(p, i, base ? load_request(p, i) : given, twice, have,
                                        limit, scratch, s, tell);
        if (i < p.n) {
            const int held = r.ok ? int(blocks_of(r.cached, p.block_size)) : 0;
            ctx[i] = r.ok ? r.cached + (r.served ? r.fresh : 0) : 0;
            row[i] = r.ok ? r.row : -1;
            old_blocks[i] = held;
            now_blocks[i] = r.ok ? int(blocks_of(ctx[i], p.block_size)) : 0;
            before[i] = r.need_in - (now_blocks[i] - held);
            start[i + 1] = int32_t(min(r.tok_in, s.placed));
        }
        s.need_base = sat_add(s.need_base, r.need_sum);
        s.tok_base = sat_add(s.tok_base, r.tok_sum);
    }
    __syncthreads();
    // block j of request i, as the step leaves it
    auto block = [&](int i, int j, int* flag) {
        if (j >= old_blocks[i]) return take_block(p, have, before[i] + (j - old_blocks[i]), flag);
        return p.table[size_t(row[i]) * p.max_blocks + j];
    };
    const int threads = int(gridDim.x) * NT, me = int(blockIdx.x) * NT + threadIdx.x;
    for (int i = me; i <= p.n; i += threads) {
        if (i < p.n) p.ctx[i] = ctx[i];
        p.start[i] = start[i];
    }
    if (me == 0) *p.free_count_out = free_ok ? int32_t(have - s.used) : free0;
    // a warp copies a segment of a row, or makes 32 tokens and as many of the new
    // entries (each of which holds a new token: there are no more of them)
    const int total = start[p.n], units = copy_warps + (p.max_tokens + 31) / 32;
    for (int w = me >> 5; w < units; w += threads >> 5) {
        if (w < copy_warps) {
            const int i = w / segments, j0 = (w % segments) * kSegment;
            int32_t* dst = p.out_tables + size_t(i) * p.width + j0;
            int32_t v[kSegment / 32];
#pragma unroll
            for (int k = 0; k < kSegment / 32; ++k) {
                const int j = j0 + lane + 32 * k;
                v[k] = j < now_blocks[i] ? block(i, j, nullptr) : -1;
            }
#pragma unroll
            for (int k = 0; k < kSegment / 32; ++k) {
                const int j = lane + 32 * k;
                if (j0 + j < p.width) dst[j] = v[k];
            }
            continue;
        }
        const int t = (w - copy_warps) * 32 + lane;
        if (uint32_t(t) < s.used) {              // the request by bisection
            int lo = 0, hi = p.n - 1;
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (before[mid] + (now_blocks[mid] - old_blocks[mid]) > uint32_t(t)) hi = mid;
                else lo = mid + 1;
            }
            p.table[size_t(row[lo]) * p.max_blocks + old_blocks[lo] + (t - before[lo])] =
                take_block(p, have, t, p.err);
        }
        if (t >= p.max_tokens) continue;
        int64_t slot = -1;
        int pos = 0;
        if (t < total) {
            int lo = 0, hi = p.n - 1;
            if (t < p.n && start[t] <= t && t < start[t + 1]) lo = hi = t;   // a decode batch
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (start[mid + 1] > t) hi = mid;
                else lo = mid + 1;
            }
            pos = ctx[lo] - (start[lo + 1] - t);
            const int blk = block(lo, pos / p.block_size, nullptr);
            if (blk < 0 || blk >= p.num_blocks) flag_error(p.err, PKV_DEV_BAD_BLOCK_ID);
            else slot = int64_t(blk) * p.block_size + pos % p.block_size;
        }
        p.slots[t] = slot;
        if (p.positions) p.positions[t] = pos;
    }
}

struct ReleaseParams {
    int32_t* table;
    int32_t* free_list;
    int32_t* free_count;
    const int32_t* seq_rows;
    const int32_t* lens;
    int32_t n, max_seqs, max_blocks, num_blocks, block_size;
    int* err;
};

// One CTA: blocks of the released rows go back on the stack, request by
// request in table order, and their table entries are set to -1.  1024 rows of 2048
// blocks 1.6 ms, the moves of two million entries through one SM, the row of each
// found by bisection.
__global__ void __launch_bounds__(kPlanThreads) tables_release_kernel(ReleaseParams p) {
    extern __shared__ uint32_t bits[];
    __shared__ ScanScratch<kPlanThreads> scratch;
    __shared__ uint32_t end[kPlanThreads];
    __shared__ int32_t rows[kPlanThreads];
    const uint32_t* twice = bits + (p.max_seqs + 31) / 32;
    pdl_wait_prerequisites();
    pdl_launch_dependents();
    if (p.seq_rows)
        mark_rows<kPlanThreads>(p.seq_rows, int(threadIdx.x) < p.n ? p.seq_rows[threadIdx.x] : -1,
                                p.n, p.max_seqs, bits, bits + (p.max_seqs + 31) / 32);
    const int free0 = *p.free_count;
    const bool free_ok = free0 >= 0 && free0 <= p.num_blocks;
    const uint32_t room = free_ok ? uint32_t(p.num_blocks - free0) : 0u;
    if (!free_ok && threadIdx.x == 0) flag_error(p.err, PKV_DEV_BAD_BLOCK_ID);
    __syncthreads();
    uint32_t base_sum = 0, top = 0;
    for (int base = 0; base < p.n; base += kPlanThreads) {
        const int i = base + threadIdx.x;
        uint32_t blocks = 0;
        int row = -1;
        if (i < p.n) {
            row = checked_row(p.seq_rows ? p.seq_rows[i] : i, p.seq_rows != nullptr, p.max_seqs,
                              twice);
            const int len = p.lens[i];
            if (row < 0) {
                flag_error(p.err, PKV_DEV_BAD_SEQ_ROW);
            } else if (len < 0) {
                flag_error(p.err, PKV_DEV_BAD_CONTEXT_LEN);
            } else if (len > int64_t(p.max_blocks) * p.block_size) {
                flag_error(p.err, PKV_DEV_TABLE_TOO_NARROW);
            } else if (len > 0) {
                // a row that was released already, or holds fewer blocks, has -1 there:
                // nothing is given back (entries between them are looked at below)
                const int32_t* e = p.table + size_t(row) * p.max_blocks;
                const int64_t held = blocks_of(len, p.block_size);
                if (e[0] < 0 || e[held - 1] < 0) flag_error(p.err, PKV_DEV_BAD_SEQ_ROW);
                else blocks = uint32_t(held);
            }
        }
        uint32_t sum, incl, first;
        const uint32_t top_before = top;
        for (bool again = false;; again = true) {
            uint32_t in_pass = blocks, none = 0, none_sum;
            scan_inclusive<kPlanThreads>(in_pass, none, scratch, sum, none_sum);
            incl = sat_add(base_sum, in_pass);
            // more blocks than the pool has: the stack takes no request past its end
            const uint32_t got = blocks && incl <= room ? incl : 0u;
            top = max(top_before, __reduce_max_sync(kFull, got));
            if ((threadIdx.x & 31) == 0) end[threadIdx.x >> 5] = top;
            __syncthreads();
            for (int w = 0; w < kPlanThreads / 32; ++w) top = max(top, end[w]);
            __syncthreads();
            end[threadIdx.x] = min(incl, top);
            rows[threadIdx.x] = row;
            __syncthreads();
            first = min(base_sum, top);
            auto entry = [&](uint32_t b) {           // of the b-th block given back
                int lo = 0, hi = kPlanThreads - 1;
                while (lo < hi) {
                    const int mid = (lo + hi) >> 1;
                    if (end[mid] > b) hi = mid;
                    else lo = mid + 1;
                }
                return p.table + size_t(rows[lo]) * p.max_blocks +
                       (b - (lo ? end[lo - 1] : first));
            };
            bool odd = false;
            for (uint32_t b = first + threadIdx.x; b < top; b += kPlanThreads) {
                int32_t* e = entry(b);
                const int blk = *e;
                odd |= blk < 0 || blk >= p.num_blocks;
                p.free_list[uint32_t(free0) + b] = blk;
                *e = -1;
            }
            if (!__syncthreads_or(odd) || again) break;
            // A row has an entry that is no block: the pass's rows get their entries back
            // (what lies above the stack's count counts for nothing), and are given back
            // without the rows that have one.
            for (uint32_t b = first + threadIdx.x; b < top; b += kPlanThreads)
                *entry(b) = p.free_list[uint32_t(free0) + b];
            __syncthreads();
            const int32_t* e = p.table + size_t(max(row, 0)) * p.max_blocks;
            for (uint32_t j = 0; j < blocks; ++j) {
                if (e[j] < 0 || e[j] >= p.num_blocks) {
                    flag_error(p.err, PKV_DEV_BAD_BLOCK_ID);
                    blocks = 0;
                }
            }
        }
        if (blocks && incl > room) flag_error(p.err, PKV_DEV_BAD_BLOCK_ID);
        base_sum = sat_add(base_sum, sum);
    }
    if (threadIdx.x == 0 && free_ok) *p.free_count = int32_t(free0 + top);
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

int check_tables(const pkv_device_tables* t) {
    if (!t) return PKV_ERR_INVALID;
    if (t->max_seqs < 1 || t->max_blocks < 1 || t->num_blocks < 1 || t->block_size < 1)
        return PKV_ERR_INVALID;
    if (t->max_seqs > PKV_TABLES_MAX_SEQS || t->num_blocks >= int32_t(kSat) ||
        int64_t(t->max_blocks) * t->block_size > INT32_MAX)
        return PKV_ERR_UNSUPPORTED;
    return PKV_OK;
}

int check_tables_pointers(const pkv_device_tables* t) {
    if (!t->block_table || !t->free_list || !t->free_count || !aligned4(t->block_table) ||
        !aligned4(t->free_list) || !aligned4(t->free_count))
        return PKV_ERR_INVALID;
    return PKV_OK;
}

int plane_bytes(int max_seqs) { return 2 * ((max_seqs + 31) / 32) * 4; }

template <int NT>
int launch_step(const TablesParams& p, int segments, int64_t copy_warps, int planes,
                cudaStream_t s) {
    const int fixed = (6 * kStepSeqs + 1) * 4;
    if (kernel_occupancy<tables_step_kernel<NT>>(NT, fixed + plane_bytes(PKV_TABLES_MAX_SEQS)) < 1)
        return PKV_ERR_CUDA;
    const int64_t warps = copy_warps + ceil_div(p.max_tokens, 32);
    const int64_t ctas = std::max<int64_t>(
        1, std::min<int64_t>((warps + NT / 32 - 1) / (NT / 32), 1024 / NT * int64_t(num_sms())));
    return cuda_status(launch_pdl(tables_step_kernel<NT>, dim3(unsigned(ctas)), dim3(NT),
                                  size_t((6 * p.n + 1) * 4 + planes), s, p, segments,
                                  int(copy_warps)));
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" int pkv_tables_step(const pkv_device_tables* tables, const int32_t* seq_rows,
                               const int32_t* cached_lens, const int32_t* new_lens,
                               int32_t num_seqs, int32_t max_tokens, int32_t* free_count_out,
                               int32_t* block_tables, int32_t max_blocks_per_seq,
                               int32_t* context_lens, int32_t* query_start_loc,
                               int64_t* slot_mapping, int32_t* positions, void* stream) {
    int st = check_tables(tables);
    if (st != PKV_OK) return st;
    if (num_seqs < 0 || max_tokens < 0) return PKV_ERR_INVALID;
    if (max_tokens >= int32_t(kSat) || max_blocks_per_seq >= int32_t(kSat))
        return PKV_ERR_UNSUPPORTED;
    if (block_tables && max_blocks_per_seq < 1) return PKV_ERR_INVALID;
    st = check_tables_pointers(tables);
    if (st != PKV_OK) return st;
    if (block_tables == tables->block_table ||   // the state itself is not an output
        !query_start_loc || (num_seqs > 0 && (!cached_lens || !context_lens)) ||
        (max_tokens > 0 && !slot_mapping) ||
        !aligned4(seq_rows) || !aligned4(cached_lens) || !aligned4(new_lens) ||
        !aligned4(free_count_out) || !aligned4(block_tables) || !aligned4(context_lens) ||
        !aligned4(query_start_loc) || !aligned4(positions) ||
        (reinterpret_cast<uintptr_t>(slot_mapping) & 7u))
        return PKV_ERR_INVALID;
    const int segments = block_tables ? ceil_div(max_blocks_per_seq, kSegment) : 0;
    const int64_t copy_warps = int64_t(num_seqs) * segments;
    const int64_t warps = copy_warps + ceil_div(max_tokens, 32);
    if (warps > INT32_MAX / 2) return PKV_ERR_UNSUPPORTED;
    TablesParams p;
    p.err = device_error_ptr(&st);
    if (st != PKV_OK) return st;
    p.table = tables->block_table;
    p.free_list = tables->free_list;
    p.free_count = tables->free_count;
    p.free_count_out = free_count_out ? free_count_out : tables->free_count;
    p.seq_rows = seq_rows;
    p.cached = cached_lens;
    p.fresh = new_lens;
    p.out_tables = block_tables;
    p.ctx = context_lens;
    p.start = query_start_loc;
    p.slots = slot_mapping;
    p.positions = positions;
    p.n = num_seqs;
    p.max_seqs = tables->max_seqs;
    p.max_blocks = tables->max_blocks;
    p.num_blocks = tables->num_blocks;
    p.block_size = tables->block_size;
    p.width = max_blocks_per_seq;
    p.max_tokens = max_tokens;
    const int smem = seq_rows ? plane_bytes(p.max_seqs) : 0;
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    // one launch where nothing is written that the other CTAs still read
    if (num_seqs <= kStepSeqs && context_lens != cached_lens &&
        p.free_count_out != tables->free_count) {
        return num_seqs <= 256 ? launch_step<256>(p, segments, copy_warps, smem, cs)
                               : launch_step<1024>(p, segments, copy_warps, smem, cs);
    }
    if (kernel_occupancy<tables_plan_kernel>(kPlanThreads, plane_bytes(PKV_TABLES_MAX_SEQS)) < 1)
        return PKV_ERR_CUDA;
    st = cuda_status(launch_pdl(tables_plan_kernel, dim3(1), dim3(kPlanThreads), size_t(smem), cs, p));
    if (st != PKV_OK || warps == 0) return st;
    const int64_t ctas = (warps + kFillThreads / 32 - 1) / (kFillThreads / 32);
    return cuda_status(launch_pdl(tables_fill_kernel, dim3(unsigned(ctas)), dim3(kFillThreads), 0,
                                  cs, p, segments, int(copy_warps)));
}

extern "C" int pkv_tables_release(const pkv_device_tables* tables, const int32_t* seq_rows,
                                  const int32_t* lens, int32_t num_seqs, void* stream) {
    int st = check_tables(tables);
    if (st != PKV_OK) return st;
    if (num_seqs < 0) return PKV_ERR_INVALID;
    if (num_seqs == 0) return PKV_OK;
    st = check_tables_pointers(tables);
    if (st != PKV_OK) return st;
    if (!lens || !aligned4(lens) || !aligned4(seq_rows)) return PKV_ERR_INVALID;
    ReleaseParams p;
    p.err = device_error_ptr(&st);
    if (st != PKV_OK) return st;
    p.table = tables->block_table;
    p.free_list = tables->free_list;
    p.free_count = tables->free_count;
    p.seq_rows = seq_rows;
    p.lens = lens;
    p.n = num_seqs;
    p.max_seqs = tables->max_seqs;
    p.max_blocks = tables->max_blocks;
    p.num_blocks = tables->num_blocks;
    p.block_size = tables->block_size;
    const int smem = seq_rows ? plane_bytes(p.max_seqs) : 0;
    if (kernel_occupancy<tables_release_kernel>(kPlanThreads, plane_bytes(PKV_TABLES_MAX_SEQS)) < 1)
        return PKV_ERR_CUDA;
    return cuda_status(launch_pdl(tables_release_kernel, dim3(1), dim3(kPlanThreads), size_t(smem),
                                  static_cast<cudaStream_t>(stream), p));
}
