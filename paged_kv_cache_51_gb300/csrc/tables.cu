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
// Two launches.  tables_plan_kernel (one CTA) does what is sequential by
// nature: the checks, both prefix sums and the few new table entries.
// tables_fill_kernel spreads the rest over the GPU: rows of tables copied out
// and padded, slots and positions of the tokens.  The step moves a few hundred
// KB to a few MB, so it is bound by the latency of the two launches.
#include <cuda_runtime.h>

#include <algorithm>

#include "launch_cache.h"
#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;
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

// Inclusive saturating scan of one value per thread; `total` is the CTA's sum.
// (min(a + b, cap) is associative on values of 0 .. cap.)
__device__ __forceinline__ uint32_t scan_inclusive(uint32_t v, uint32_t* warp_sums,
                                                   uint32_t& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t u = __shfl_up_sync(kFull, v, o);
        if (lane >= o) v = sat_add(v, u);
    }
    if (lane == 31) warp_sums[warp] = v;
    __syncthreads();
    if (warp == 0) {
        uint32_t w = lane < kPlanWarps ? warp_sums[lane] : 0u;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t u = __shfl_up_sync(kFull, w, o);
            if (lane >= o) w = sat_add(w, u);
        }
        if (lane < kPlanWarps) warp_sums[lane] = w;
    }
    __syncthreads();
    if (warp > 0) v = sat_add(v, warp_sums[warp - 1]);
    total = warp_sums[kPlanWarps - 1];
    __syncthreads();
    return v;
}

// Marks the rows that the batch names more than once: two bit planes over
// max_seqs rows in shared memory, `seen` and `twice`.
__device__ __forceinline__ void mark_rows(const int32_t* rows, int n, int max_seqs,
                                          uint32_t* seen, uint32_t* twice) {
    const int words = (max_seqs + 31) / 32;
    for (int i = threadIdx.x; i < words; i += kPlanThreads) seen[i] = twice[i] = 0u;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kPlanThreads) {
        const int r = rows[i];
        if (r < 0 || r >= max_seqs) continue;
        const uint32_t bit = 1u << (r & 31);
        if (atomicOr(seen + (r >> 5), bit) & bit) atomicOr(twice + (r >> 5), bit);
    }
    __syncthreads();
}

__device__ __forceinline__ int row_of(const int32_t* rows, int i, int max_seqs,
                                      const uint32_t* twice) {
    if (!rows) return i < max_seqs ? i : -1;
    const int r = rows[i];
    if (r < 0 || r >= max_seqs) return -1;
    return twice[r >> 5] >> (r & 31) & 1u ? -1 : r;
}

__device__ __forceinline__ int64_t blocks_of(int64_t tokens, int bs) {
    return (tokens + bs - 1) / bs;
}

__global__ void __launch_bounds__(kPlanThreads) tables_plan_kernel(TablesParams p) {
    extern __shared__ uint32_t bits[];            // two planes of max_seqs bits
    __shared__ uint32_t warp_sums[kPlanWarps];
    __shared__ uint32_t need_end[kPlanThreads];   // inclusive needs of the pass's served requests
    __shared__ int32_t dest[kPlanThreads];        // first new table entry of a request ...
    __shared__ int32_t dest_row[kPlanThreads];    // ... in this row
    const uint32_t* twice = bits + (p.max_seqs + 31) / 32;
    pdl_wait_prerequisites();
    pdl_launch_dependents();
    if (p.seq_rows)
        mark_rows(p.seq_rows, p.n, p.max_seqs, bits, bits + (p.max_seqs + 31) / 32);
    const int free0 = *p.free_count;
    const bool free_ok = free0 >= 0 && free0 <= p.num_blocks;
    const uint32_t have = free_ok ? uint32_t(free0) : 0u;
    if (!free_ok && threadIdx.x == 0) flag_error(p.err, PKV_DEV_BAD_BLOCK_ID);
    __syncthreads();                              // everyone read the count before it is written
    const int64_t limit = int64_t(min(p.max_blocks, p.out_tables ? p.width : p.max_blocks)) *
                          p.block_size;
    uint32_t need_base = 0, tok_base = 0;         // of the requests before this pass
    uint32_t used = 0, placed = 0;                // of the served ones
    for (int base = 0; base < p.n; base += kPlanThreads) {
        const int i = base + threadIdx.x;
        int row = -1, cached = 0, fresh = 0;
        uint32_t need = 0;
        bool ok = false;
        if (i < p.n) {
            row = row_of(p.seq_rows, i, p.max_seqs, twice);
            cached = p.cached[i];
            fresh = p.fresh ? p.fresh[i] : 1;
            if (row < 0) {
                flag_error(p.err, PKV_DEV_BAD_SEQ_ROW);
            } else if (cached < 0 || fresh < 0) {
                flag_error(p.err, PKV_DEV_BAD_CONTEXT_LEN);
            } else if (int64_t(cached) + fresh > limit) {
                flag_error(p.err, PKV_DEV_TABLE_TOO_NARROW);
            } else {
                ok = true;
                need = uint32_t(blocks_of(int64_t(cached) + fresh, p.block_size) -
                                blocks_of(cached, p.block_size));
            }
        }
        const uint32_t tok = ok ? min(uint32_t(fresh), kSat) : 0u;
        uint32_t need_sum, tok_sum;
        const uint32_t need_in = sat_add(need_base, scan_inclusive(need, warp_sums, need_sum));
        const uint32_t tok_in = sat_add(tok_base, scan_inclusive(tok, warp_sums, tok_sum));
        // served in order up to the first request that does not fit: both sums
        // only grow, so no later request fits either
        const bool fits = need_in <= have && tok_in <= uint32_t(p.max_tokens);
        const bool served = ok && fits;
        if (ok && !fits)
            flag_error(p.err, need_in > have ? PKV_DEV_NO_FREE_BLOCKS : PKV_DEV_BAD_QUERY_LAYOUT);
        // the sums of served requests: those in front of the first that does not fit
        const uint32_t need_got = served ? need_in : 0u, tok_got = served ? tok_in : 0u;
        used = max(used, __reduce_max_sync(kFull, need_got));
        placed = max(placed, __reduce_max_sync(kFull, tok_got));
        if ((threadIdx.x & 31) == 0) need_end[threadIdx.x >> 5] = used;
        if ((threadIdx.x & 31) == 0) dest[threadIdx.x >> 5] = int32_t(placed);
        __syncthreads();
        used = need_end[0];
        placed = uint32_t(dest[0]);
        for (int w = 1; w < kPlanWarps; ++w) {
            used = max(used, need_end[w]);
            placed = max(placed, uint32_t(dest[w]));
        }
        __syncthreads();
        if (i < p.n) {
            p.ctx[i] = ok ? cached + (served ? fresh : 0) : 0;
            p.start[i + 1] = int32_t(min(tok_in, placed));
        }
        need_end[threadIdx.x] = min(need_in, used);
        dest[threadIdx.x] = ok ? int32_t(blocks_of(cached, p.block_size)) : 0;
        dest_row[threadIdx.x] = row;
        __syncthreads();
        // new entries of the pass, one thread each: the request by bisection
        const uint32_t first = min(need_base, used);
        for (uint32_t b = first + threadIdx.x; b < used; b += kPlanThreads) {
            int lo = 0, hi = kPlanThreads - 1;
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (need_end[mid] > b) hi = mid;
                else lo = mid + 1;
            }
            const uint32_t before = lo ? need_end[lo - 1] : first;
            int blk = p.free_list[have - 1 - b];
            if (blk < 0 || blk >= p.num_blocks) {
                flag_error(p.err, PKV_DEV_BAD_BLOCK_ID);
                blk = -1;
            }
            p.table[size_t(dest_row[lo]) * p.max_blocks + dest[lo] + (b - before)] = blk;
        }
        __syncthreads();
        need_base = sat_add(need_base, need_sum);
        tok_base = sat_add(tok_base, tok_sum);
    }
    if (threadIdx.x == 0) {
        p.start[0] = 0;
        *p.free_count_out = free_ok ? int32_t(have - used) : free0;
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
// request in table order, and their table entries are set to -1.
__global__ void __launch_bounds__(kPlanThreads) tables_release_kernel(ReleaseParams p) {
    extern __shared__ uint32_t bits[];
    __shared__ uint32_t warp_sums[kPlanWarps];
    __shared__ uint32_t end[kPlanThreads];
    __shared__ int32_t rows[kPlanThreads];
    const uint32_t* twice = bits + (p.max_seqs + 31) / 32;
    pdl_wait_prerequisites();
    pdl_launch_dependents();
    if (p.seq_rows)
        mark_rows(p.seq_rows, p.n, p.max_seqs, bits, bits + (p.max_seqs + 31) / 32);
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
            row = row_of(p.seq_rows, i, p.max_seqs, twice);
            const int len = p.lens[i];
            if (row < 0) {
                flag_error(p.err, PKV_DEV_BAD_SEQ_ROW);
            } else if (len < 0) {
                flag_error(p.err, PKV_DEV_BAD_CONTEXT_LEN);
            } else if (len > int64_t(p.max_blocks) * p.block_size) {
                flag_error(p.err, PKV_DEV_TABLE_TOO_NARROW);
            } else if (len > 0) {
                // a row that was released already holds -1: nothing to give back
                if (p.table[size_t(row) * p.max_blocks] < 0) flag_error(p.err, PKV_DEV_BAD_SEQ_ROW);
                else blocks = uint32_t(blocks_of(len, p.block_size));
            }
        }
        uint32_t sum;
        const uint32_t incl = sat_add(base_sum, scan_inclusive(blocks, warp_sums, sum));
        if (blocks && incl > room) flag_error(p.err, PKV_DEV_BAD_BLOCK_ID);
        // more blocks than the pool has: the stack takes no request past its end
        const uint32_t got = blocks && incl <= room ? incl : 0u;
        top = max(top, __reduce_max_sync(kFull, got));
        if ((threadIdx.x & 31) == 0) end[threadIdx.x >> 5] = top;
        __syncthreads();
        for (int w = 0; w < kPlanWarps; ++w) top = max(top, end[w]);
        __syncthreads();
        end[threadIdx.x] = min(incl, top);
        rows[threadIdx.x] = row;
        __syncthreads();
        const uint32_t first = min(base_sum, top);
        for (uint32_t b = first + threadIdx.x; b < top; b += kPlanThreads) {
            int lo = 0, hi = kPlanThreads - 1;
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (end[mid] > b) hi = mid;
                else lo = mid + 1;
            }
            int32_t* e = p.table + size_t(rows[lo]) * p.max_blocks + (b - (lo ? end[lo - 1] : first));
            const int blk = *e;
            if (blk < 0 || blk >= p.num_blocks) flag_error(p.err, PKV_DEV_BAD_BLOCK_ID);
            p.free_list[uint32_t(free0) + b] = blk;
            *e = -1;
        }
        __syncthreads();
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
    if (max_tokens >= int32_t(kSat)) return PKV_ERR_UNSUPPORTED;
    if (block_tables && max_blocks_per_seq < 1) return PKV_ERR_INVALID;
    st = check_tables_pointers(tables);
    if (st != PKV_OK) return st;
    if (!query_start_loc || (num_seqs > 0 && (!cached_lens || !context_lens)) ||
        (max_tokens > 0 && !slot_mapping) ||
        !aligned4(seq_rows) || !aligned4(cached_lens) || !aligned4(new_lens) ||
        !aligned4(free_count_out) || !aligned4(block_tables) || !aligned4(context_lens) ||
        !aligned4(query_start_loc) || !aligned4(positions) ||
        (reinterpret_cast<uintptr_t>(slot_mapping) & 7u))
        return PKV_ERR_INVALID;
    const int segments = block_tables ? ceil_div(max_blocks_per_seq, kSegment) : 0;
    const int64_t copy_warps = int64_t(num_seqs) * segments;
    const int64_t warps = copy_warps + ceil_div(max_tokens, 32);
    if (copy_warps > INT32_MAX) return PKV_ERR_UNSUPPORTED;
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
    if (kernel_occupancy<tables_plan_kernel>(kPlanThreads, plane_bytes(PKV_TABLES_MAX_SEQS)) < 1)
        return PKV_ERR_CUDA;
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
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
