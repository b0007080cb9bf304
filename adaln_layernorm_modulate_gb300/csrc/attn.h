// Host-side entry points of the attention kernels (csrc/attn.cu, internal to libadaln).
#pragma once

#include <cuda_runtime.h>

#include "common.cuh"

namespace adaln {

constexpr uint32_t kDbgAttn = 2048u;  // debug builds: rows, heads, work items, statistics, pieces
constexpr int kAttnTile = 128;       // rows of an operand tile, keys of a step
constexpr int kAttnMaxD = 128;       // elements of a head
constexpr int kAttnMaxCtas = 256;    // of one launch
constexpr int kAttnFewKeys = 32;     // rows of queries that see no more take delta from the scores
constexpr int kAttnFewBlocks = kAttnFewKeys / 16;  // of 16 such rows, a causal segment
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
    int32_t end;     // the segment's last row of the other side is the tensor's last: nothing follows
    int32_t unseen;  // keys: the segment's first queries that see no key at all
    int32_t pad;
};

// A unit of work is an item and a head: unit u is head u / items, item u % items. Its cost is its
// steps (tiles of the other side) and what its beginning and end take, in steps. Units are laid end to end and
// shared out evenly, so that a CTA may begin or end inside one; what it computes of such a unit is a
// piece, left in fp32 and joined with the others in their order by another kernel. With whole units a CTA,
// 64 x 12 units on 152 SMs would take six rounds for 5.05.
// A piece has at least this many steps: writing and joining one costs about as much as two.
constexpr int kAttnMinPiece = 4;
struct AttnCursor {
    int32_t unit, tile;
};

struct AttnTables {
    const int32_t* cu_q;  // [nseg + 1], or null: nseg segments of Rq / nseg rows
    const int32_t* cu_k;
    int64_t nseg, Rq, Rk;
    int causal;
};

// A work list.
struct AttnList {
    AttnItem* items;
    int32_t* count;       // its entries
    longlong2* segs;      // [nseg]: entries and cost of the segments before each
    AttnCursor* cursors;  // [ctas + 1]: where each CTA begins
    int64_t most;         // entries it has room for
    int tile;             // rows an entry
    int heads;            // units an entry
    int group;            // keys: heads of queries that a step is repeated for
    int unit_cost;        // what a unit takes beside its steps, in steps
    int ctas;
};

struct AttnPlanArgs {
    AttnTables t;
    AttnList list[2];     // over queries; over keys (items null: not wanted)
    uint32_t* status;     // [2]
    WsHeader* header;
};

struct AttnFwdArgs {
    AttnList list;
    void* o;
    float* lse;            // [Hq, Rq]
    float* part;           // pieces: [2 * ctas][d / 4][slot_rows][4] sums of p v
    float2* ml;            // and [2 * ctas][slot_rows] (maximum, sum of p)
    uint32_t* status;
    int64_t Rq, o_ld;
    int Hq, group, d, slot_rows;
    float scale;
};

struct AttnBwdArgs {
    AttnList list;
    const float* delta;
    const float* lse2;
    void* dx;              // dq; dk
    void* dv;
    float* part;           // pieces: [2 * ctas][d / 4][slot_rows][4] of dq; [2 * ctas][2].. of dv, dk
    uint32_t* status;
    int64_t Rq, dx_ld, dv_ld;
    int Hq, group, d, slot_rows;
    float scale;
};

// Pieces of up to two lists joined: the forward's, or dq's and dk's and dv's.
struct AttnJoinArgs {
    AttnList list[2];
    const float* part[2];
    const float2* ml;      // forward
    void* out[2];          // o, or dq; dk
    void* dv;
    float* lse;
    int64_t Rq, ld[2], dv_ld;
    int d, slot_rows[2];
    float scale;
};

struct AttnDeltaArgs {
    const void* dout;
    const void* o;
    const float* lse;
    float* delta;          // [Hq, Rq] sum of dout * o
    float* lse2;           // [Hq, Rq] lse in units of log 2
    int64_t Rq, do_ld, o_ld;
    int Hq, d;
    const void *q, *k, *v;  // rows of few keys
    int64_t Rk, q_ld, k_ld, v_ld;
    int group, few;         // CTAs for them (of the launch; 0: there are none)
    float scale;
};

// A side's rows as the kernels' TMA maps take them.
struct AttnRows {
    const void* p;
    int64_t R, ld;
    int H;
};

// The forward's work list; the backward's lists and delta.
cudaError_t launch_attn_plan(const AttnPlanArgs& plan, cudaStream_t stream);
cudaError_t launch_attn_prepare(const AttnPlanArgs& plan, const AttnDeltaArgs& delta, int sms, cudaStream_t stream);
cudaError_t launch_attn_fwd(const AttnFwdArgs& args, const AttnRows& q, const AttnRows& k, const AttnRows& v,
                            cudaStream_t stream);
cudaError_t launch_attn_join(const AttnJoinArgs& args, bool bwd, cudaStream_t stream);
// dk and dv, dq; either's list may have no CTAs.
cudaError_t launch_attn_bwd(const AttnBwdArgs& dkv, const AttnBwdArgs& dq, const AttnRows& dout, const AttnRows& q,
                            const AttnRows& k, const AttnRows& v, cudaStream_t stream);
cudaError_t debug_word_attn(uint32_t* out, bool reset);

}  // namespace adaln
