// What the kernels over expanded keys share: the batch, its plan and the launchers.
#pragma once

#include "pkv_internal.h"

namespace pkv {

// A planned unit: query rows of one sequence (of one head; heads are the units' inner
// index), cheapest last.
struct ExpandedItem {
    int32_t q0, rows;        // first query row of the call, rows of the unit
    int32_t k0, keys;        // first key row of the sequence, keys that the last row sees (may be <= 0)
};

struct ExpandedWorkspace {
    int32_t* counters;       // [0] items, [1] ticket
    ExpandedItem* items;
    int32_t max_items;
};

struct ExpandedArgs {
    void* out;
    const void* q;
    const void* k;
    const void* v;
    const void* k_rope;
    const pkv_expanded_desc* desc;
    const int32_t* query_start_loc;
    const int32_t* key_start_loc;
    int32_t num_seqs, num_query_tokens, num_keys, max_query_len;
    float scale;
    ExpandedWorkspace ws;
    int* err;
    cudaStream_t stream;
};

constexpr int kExpandedRope = 64;
constexpr int kExpandedRowsF32 = 32;       // query rows of a unit (fp32: 32 or 64)
constexpr int kExpandedRowsBf16 = 256;

int launch_expanded_plan(const ExpandedArgs& a, int rows);
int launch_expanded_bf16(const ExpandedArgs& a);
int launch_expanded_f32(const ExpandedArgs& a);

}  // namespace pkv
