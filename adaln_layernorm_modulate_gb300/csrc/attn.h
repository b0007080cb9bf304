// Host-side entry points of the attention kernels (csrc/attn.cu, internal to libadaln).
#pragma once

#include <cuda_runtime.h>

#include "common.cuh"

namespace adaln {

constexpr int kAttnTile = 128;       // rows of an operand tile, keys of a step
constexpr int kAttnMaxD = 128;       // elements of a head
constexpr int kAttnMaxRows = 1 << 30;  // of either side: row and key numbers and their sums are 32 bits

// One tile of rows of a segment (of queries; of keys for dk and dv) and what it meets.
struct AttnItem {
    int32_t row0;    // its first row
    int32_t rows;    // its rows
    int32_t other0;  // first row of the segment's other side
    int32_t others;  // the other side's rows
    // Queries: row r of the tile sees the keys j < min(others, shift + r + 1) of its segment. Keys: key c
    // of the tile is seen by the queries i >= max(0, shift + c) of its segment.
    int32_t shift;
    int32_t end;     // the segment's last row is the tensor's last: nothing follows (bit 0: of the other side)
    int32_t pad[2];
};

constexpr int kAttnClasses = 128;    // work items in descending order of cost, a quarter octave each

struct AttnTables {
    const int32_t* cu_q;  // [nseg + 1], or null: nseg segments of Rq / nseg rows
    const int32_t* cu_k;
    int64_t nseg, Rq, Rk;
    int causal;
};

struct AttnPlanArgs {
    AttnTables t;
    AttnItem* items[2];   // list 0 over queries, list 1 over keys (or null)
    int32_t* count;       // [2]
    int64_t most[2];      // entries of the lists
    int tile[2];          // rows a tile
    uint32_t* status;     // [2]
    WsHeader* header;
};

struct AttnFwdArgs {
    const AttnItem* items;
    const int32_t* count;
    void* o;
    float* lse;            // [Hq, Rq]
    float* part;           // splits > 1: [splits][Hq][Rq][d] sums of p v
    float2* ml;            // and [splits][Hq][Rq] (maximum, sum of p)
    uint32_t* status;
    int64_t Rq, o_ld, most;
    int Hq, group, d, splits;
    float scale;
};

struct AttnJoinArgs {
    const float* part;
    const float2* ml;
    void* o;
    float* lse;
    int64_t Rq, o_ld;
    int Hq, d, splits;
    float scale;
    const uint32_t* bad;   // the plan's status: nothing was computed
};

struct AttnDeltaArgs {
    const void* dout;
    const void* o;
    const float* lse;
    float* delta;          // [Hq, Rq] sum of dout * o
    float* lse2;           // [Hq, Rq] lse in units of log 2
    int64_t Rq, do_ld, o_ld;
    int Hq, d;
};

struct AttnBwdArgs {
    const AttnItem* items;
    const int32_t* count;
    const float* delta;
    const float* lse2;
    void* dx;              // dq; dk
    void* dv;
    uint32_t* status;
    int64_t Rq, dx_ld, dv_ld, most;
    int Hq, group, d;
    float scale;
};

// A side's rows as the kernels' TMA maps take them.
struct AttnRows {
    const void* p;
    int64_t R, ld;
    int H;
};

cudaError_t launch_attn_plan(const AttnPlanArgs& args, cudaStream_t stream);
cudaError_t launch_attn_fwd(const AttnFwdArgs& args, const AttnRows& q, const AttnRows& k, const AttnRows& v, int sms,
                            cudaStream_t stream);
cudaError_t launch_attn_join(const AttnJoinArgs& args, int sms, cudaStream_t stream);
cudaError_t launch_attn_delta(const AttnDeltaArgs& args, int sms, cudaStream_t stream);
cudaError_t launch_attn_dq(const AttnBwdArgs& args, const AttnRows& dout, const AttnRows& q, const AttnRows& k,
                           const AttnRows& v, int sms, cudaStream_t stream);
cudaError_t launch_attn_dkv(const AttnBwdArgs& args, const AttnRows& dout, const AttnRows& q, const AttnRows& k,
                            const AttnRows& v, int sms, cudaStream_t stream);
cudaError_t debug_word_attn(uint32_t* out, bool reset);

}  // namespace adaln
