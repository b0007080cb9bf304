// Host-side entry points of the vocabulary loss's kernels (csrc/xent.cu, internal to libadaln).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "common.cuh"

namespace adaln {

// Output tile of a CTA pair's matrix product (at most kTileN columns, see tile_cols) and its K
// step; a CTA's share of the rows.
constexpr int kTileM = 256, kTileN = 256, kTileK = 64;
constexpr int kCtaM = kTileM / 2;
constexpr int kPairs = 76;  // CTA pairs the tiles are shared out to
// Columns a tile: 256, or 128 where that leaves pairs without one: a pair's product takes the same
// time a column whatever its rows hold, so a few rows are through sooner in narrower tiles (96 x
// 8192 x 1024, forward: 12.8 us against 14.8; backward 31.0 against 33.6).
inline int tile_cols(int64_t row_tiles, int64_t cols) {
    return row_tiles * ((cols + kTileN - 1) / kTileN) < kPairs ? kTileN / 2 : kTileN;
}
// dweight takes what rounding dz of the target left off in fp32: from a list of the word's rows in the
// epilogue of its products if they are at most kHits, else in finish_kernel.
constexpr int kHits = 8;
// Rows whose targets one look at them covers. Up to these a word's rows are looked for among all
// targets; with more rows (and more such words) that would grow with their product, so that every word's
// rows are listed first. Words of more than kSortRows are few and are looked for all the same.
// Backward at 262144 x 20000 x 512: 20.0 ms, without lists 30.4 (and 19.9 without remainders).
constexpr int kListRows = 8192, kSortRows = 512;
constexpr int kPackThreads = 256;
constexpr int kPackCtas = 608;  // four per SM: every CTA also counts the rows before its own

// Words that are the target of more than kHits rows: at most slots, a place each, in the order in
// which they were found (nothing that is computed depends on it).
struct ManyRows {
    int32_t* count;   // places taken
    int32_t* word;    // [slots]
    int32_t* slot;    // [V]: the place of a word that has one
    float* sums;      // [slots][D]: dweight without the remainders
    int64_t slots;
    // More than kListRows rows: the words' packed rows in any order, each word's from first on.
    int32_t* listed;  // entries of rows taken; null: no lists
    int32_t* first;   // [slots]
    int32_t* next;    // [slots]
    int32_t* rows;    // [Np]
};

struct PackArgs {
    const void* x;          // [N, D]
    const int64_t* target;  // [N]
    const float* lse;       // backward: [N], or null
    const float* dloss;
    const float* dlse;      // or null
    void* xp;               // packed rows [Np, D]
    int32_t* row;           // [Np]: the packed row's row
    int32_t* tgt;           // [Np]
    float* row_lse;         // backward: lse, dloss + dlse, dloss of the packed row
    float* row_gs;
    float* row_gt;
    int32_t* nact;          // packed rows
    int32_t* word_hits;     // backward: zeros [V], or null
    ManyRows many;          // backward with word_hits: its count, zero
    float* loss_out;        // forward: zeros for rows without a loss, or null
    float* lse_out;
    void* dx;               // backward: zeros for rows without a loss, or null
    uint32_t* status;
    WsHeader* header;
    int64_t N, Np, D, V, ignore;
};

struct LogitsArgs {
    const int32_t* nact;
    const int32_t* tgt;
    float2* parts;          // statistics: [2 * tiles][Np] (max, sum exp)
    float* zt;              // statistics: [Np], the target's logit
    const float* row_lse;   // dz
    const float* row_gs;
    const float* row_gt;
    float* row_lo;          // dz: [Np], what rounding dz of the target left off
    int32_t* word_hits;     // dz: rows whose target each word is [V], and the first kHits of them
    int32_t* word_rows;     // in the order they came [V, kHits]; or null
    ManyRows many;          // dz, with word_hits: count, word and slot
    __nv_bfloat16* probs;   // dz [Np, ldp]
    int64_t ldp;
    uint32_t* status;
    int64_t Np, D, V, v0, v1;  // columns [v0, v1) of the vocabulary
    int tn;                 // columns a tile
};

struct GradArgs {
    const int32_t* nact;
    float* dxacc;           // [splits][Np][D] fp32, or null
    __nv_bfloat16* dweight; // [V, D], or null
    const void* xp;
    const int32_t* word_hits;
    const int32_t* word_rows;
    ManyRows many;          // writes sums
    const float* row_lo;
    uint32_t* status;
    int64_t Np, D, V, v0, v1;
    int splits;             // parts of dx's K range
    int tn;                 // columns a tile
};

struct LseArgs {
    const int32_t* nact;
    const int32_t* row;
    const float2* parts;
    const float* zt;
    float* loss;
    float* lse;
    int64_t N, Np;
    int nparts;
};

struct FinishArgs {
    const int32_t* nact;
    const int32_t* row;
    const float* dxacc;
    const void* weight;
    const void* xp;
    const int32_t* tgt;
    const float* row_lo;
    const int32_t* word_hits;
    ManyRows many;
    void* dx;               // or null
    __nv_bfloat16* dweight; // or null
    int64_t N, Np, D, V;
    int splits;
    int many_ctas;          // set by launch_finish
};

cudaError_t launch_pack(const PackArgs& args, int ctas, cudaStream_t stream);
cudaError_t launch_logits(const LogitsArgs& args, bool probs, const void* xp, const void* weight, int sms,
                          cudaStream_t stream);
cudaError_t launch_grad(const GradArgs& args, const void* probs, int64_t ldp, const void* xp, const void* weight,
                        int sms, cudaStream_t stream);
cudaError_t launch_lse(const LseArgs& args, int sms, cudaStream_t stream);
cudaError_t launch_lists(const FinishArgs& args, int sms, cudaStream_t stream);
cudaError_t launch_finish(const FinishArgs& args, int sms, cudaStream_t stream);
cudaError_t debug_word_xent(uint32_t* out, bool reset);

}  // namespace adaln
