// Query rows of the sparse entry points (the sequence of a row and the keys it
// sees), and thread-block clusters.
#pragma once

#include "pkv_device.cuh"

namespace pkv {

struct QueryRows {
    const int32_t* block_tables;   // [n][table_stride]
    const int32_t* start;          // query_start_loc [n + 1], or null: one row per sequence
    const int32_t* ctx;            // context_lens [n]
    int32_t table_stride, n, max_ctx;
    int32_t tokens;                // query rows that the call was given
};

// Sequence of query token t, found by a whole warp: t itself without
// query_start_loc, else the last one that starts at or before t; -1 for a token
// behind the last sequence.  `first` is the sequence's first token, `count` its
// number of tokens, all of them among the `tokens` rows of the call: where the
// offsets end above that, or a sequence above their end, the answer is -1 too.
// A batch of single tokens or of up to 32 sequences is answered by one round of
// loads, others by one more for every factor of 32 in their number.
__device__ __forceinline__ int token_seq(const int32_t* start, int n, int tokens, int t, int& first,
                                         int& count, int* err) {
    if (!start) {
        first = t;
        count = 1;
        return t < n ? t : -1;
    }
    const int lane = threadIdx.x & 31;
    int step = (n + 31) / 32;
    const int coarse = lane * step < n ? start[lane * step] : INT32_MAX;
    const int total = start[n];
    int lo = min(t, n - 1);
    first = start[lo];
    int next = start[lo + 1];
    if (total > tokens) {
        flag_error(err, PKV_DEV_BAD_QUERY_LAYOUT);
        return -1;
    }
    if (t >= total) return -1;
    if (t < first || t >= next) {
        // (of several sequences that start there, those before the last are empty)
        lo = 31 - __clz(__ballot_sync(0xffffffffu, lane == 0 || coarse <= t));
        first = __shfl_sync(0xffffffffu, coarse, lo);
        next = __shfl_sync(0xffffffffu, coarse, min(lo + 1, 31));
        if (lo + 1 >= min(n, 32)) next = total;
        if (step > 1) {
            int width = min(step, n - lo * step);
            lo *= step;
            while (width > 1) {                  // the sequence is one of lo .. lo + width - 1
                step = (width + 31) / 32;
                const bool before = lane == 0 || (lane * step < width && start[lo + lane * step] <= t);
                const int k = 31 - __clz(__ballot_sync(0xffffffffu, before));
                lo += k * step;
                width = min(step, width - k * step);
            }
            first = start[lo];
            next = start[lo + 1];
        }
        if (t < first || t >= next) {            // offsets that are not in order
            flag_error(err, PKV_DEV_BAD_QUERY_LAYOUT);
            return -1;
        }
    }
    if (first < 0 || next > total) {
        flag_error(err, PKV_DEV_BAD_QUERY_LAYOUT);
        return -1;
    }
    count = next - first;
    return lo;
}

// Flags offsets that do not rise from 0 (one out of order between two others shows in
// no row of theirs): the steps i, i + threads, ... of one of `threads` threads.
__device__ __forceinline__ void check_offsets(const int32_t* start, int n, int64_t i,
                                              int64_t threads, int* err) {
    for (; i < n; i += threads)
        if (start[i + 1] < start[i] || (i == 0 && start[0] != 0))
            flag_error(err, PKV_DEV_BAD_QUERY_LAYOUT);
}

// The same by all threads of a grid beside their own work: each one's first step is
// asked for when this is made and looked at by `check`, behind the lookup of the
// thread's own row.
struct OffsetStep {
    const int32_t* start;
    int32_t n, from, to;
    __device__ __forceinline__ OffsetStep(const int32_t* start_, int32_t n_)
        : start(start_), n(n_), from(0), to(0) {
        const int64_t i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
        if (start && i < n) from = start[i], to = start[i + 1];
    }
    __device__ __forceinline__ void check(int* err) const {
        if (!start) return;
        if (to < from || ((blockIdx.x | threadIdx.x) == 0 && from != 0))
            flag_error(err, PKV_DEV_BAD_QUERY_LAYOUT);
        const int64_t threads = int64_t(gridDim.x) * blockDim.x;
        if (threads < n)
            check_offsets(start, n, threads + int64_t(blockIdx.x) * blockDim.x + threadIdx.x,
                          threads, err);
    }
};

// Whether a sequence of q query rows has a context that can be read (flagged
// where `err` is given).
__device__ __forceinline__ bool sequence_keys(const QueryRows& r, int seq, int q, int* err) {
    const int ctx = r.ctx[seq];
    if (ctx < q || ctx > r.max_ctx) {
        flag_error(err, PKV_DEV_BAD_CONTEXT_LEN);
        return false;
    }
    if (ctx > int64_t(r.table_stride) * kBlockTokens) {
        flag_error(err, PKV_DEV_TABLE_TOO_NARROW);
        return false;
    }
    return true;
}

// Keys that query row `t` of sequence `seq` sees: its context up to the row's
// own position.  0 for a sequence whose length is out of range, -1 for a row
// behind the last sequence.
__device__ __forceinline__ int row_keys(const QueryRows& r, int t, int& seq, int* err) {
    int first, q;
    seq = token_seq(r.start, r.n, r.tokens, t, first, q, err);
    if (seq < 0) return -1;
    return sequence_keys(r, seq, q, err) ? r.ctx[seq] - q + (t - first) + 1 : 0;
}

// ---- asynchronous copies -----------------------------------------------------------
// 16 bytes to shared memory, or 16 bytes of zeros without reading (`live` false)
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool live) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(live ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// ---- thread-block clusters --------------------------------------------------------
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// shared::cluster address of `addr` (this CTA's shared memory) in CTA `rank`
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
// Stores into the shared memory of a CTA of the cluster that count their bytes on
// an mbarrier there (both addresses from map_rank): the receiver waits for what it
// gets, the sender for nothing.
__device__ __forceinline__ void st_async(uint32_t addr, uint32_t bar, float4 v) {
    asm volatile(
        "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::
            "r"(addr), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void st_async(uint32_t addr, uint32_t bar, float2 v) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::
                     "r"(addr), "f"(v.x), "f"(v.y), "r"(bar)
                 : "memory");
}

}  // namespace pkv
