// Query rows of the sparse entry points: the sequence of a row and the keys it sees.
#pragma once

#include "pkv_device.cuh"

namespace pkv {

struct QueryRows {
    const int32_t* block_tables;   // [n][table_stride]
    const int32_t* start;          // query_start_loc [n + 1], or null: one row per sequence
    const int32_t* ctx;            // context_lens [n]
    int32_t table_stride, n, max_ctx;
};

// Sequence of query token t: t itself without query_start_loc, else by
// bisection; -1 for a token behind the last sequence.  `first` is the
// sequence's first token, `count` its number of tokens.
__device__ __forceinline__ int token_seq(const int32_t* start, int n, int t, int& first,
                                         int& count, int* err) {
    if (!start) {
        first = t;
        count = 1;
        return t < n ? t : -1;
    }
    if (t >= start[n]) return -1;
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (start[mid + 1] > t) hi = mid;
        else lo = mid + 1;
    }
    first = start[lo];
    count = start[lo + 1] - first;
    if (first < 0 || t < first || t >= first + count) {   // offsets that are not in order
        flag_error(err, PKV_DEV_BAD_QUERY_LAYOUT);
        return -1;
    }
    return lo;
}

// Keys that query row `t` of sequence `seq` sees: its context up to the row's
// own position.  0 for a sequence whose length is out of range (flagged where
// `err` is given), -1 for a row behind the last sequence.
__device__ __forceinline__ int row_keys(const QueryRows& r, int t, int& seq, int* err) {
    int first, q;
    seq = token_seq(r.start, r.n, t, first, q, err);
    if (seq < 0) return -1;
    const int ctx = r.ctx[seq];
    if (ctx < q || ctx > r.max_ctx) {
        flag_error(err, PKV_DEV_BAD_CONTEXT_LEN);
        return 0;
    }
    if (ctx > int64_t(r.table_stride) * kBlockTokens) {
        flag_error(err, PKV_DEV_TABLE_TOO_NARROW);
        return 0;
    }
    return ctx - q + (t - first) + 1;
}

}  // namespace pkv
