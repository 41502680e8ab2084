// What the kernels over expanded keys share: the batch, its plan and the launchers.
#pragma once

#include "pkv_internal.h"

namespace pkv {

// A planned unit: query rows of one sequence (of one head), cheapest last.  Up to four
// neighbouring units of a sequence form a group, and the units of all heads of a group are
// taken head by head: those that run at the same time then read the same keys.  (Unit by unit
// over all heads, eight prompts of up to 4096 tokens with 32 heads read 2.6 GB from HBM, three
// times their keys and values, and took 590 us instead of 546; now they read 1.1 GB, 0.67 GB
// being their keys, values and queries.)  With fewer than eight units an SM they mostly run at the same time anyway, and groups of one end more evenly (4 prompts
// of 2048 tokens, 19 heads: 83 us against 91).
struct ExpandedItem {
    int32_t q0, rows;        // first query row of the call, rows of the unit
    int32_t k0, keys;        // first key row of the sequence, keys that the last row sees (may be <= 0)
    int32_t group, members;  // first item of the group, and how many
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
constexpr int kExpandedRowsF32 = 32;       // query rows of a unit (fp32: 32, 64 or 128)
constexpr int kExpandedRowsBf16 = 256;

#ifdef __CUDACC__
// unit `ticket` of all, in the order of their groups
__device__ __forceinline__ ExpandedItem expanded_unit(const ExpandedWorkspace& ws, int ticket, int heads, int& head) {
    const ExpandedItem x = ws.items[ticket / heads];
    const int local = ticket - x.group * heads;
    head = local / x.members;
    return ws.items[x.group + local - head * x.members];
}
#endif

int launch_expanded_plan(const ExpandedArgs& a, int rows);
int launch_expanded_bf16(const ExpandedArgs& a);
int launch_expanded_f32(const ExpandedArgs& a);

}  // namespace pkv
