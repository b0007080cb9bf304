// Host-side entry points of the head norm and rotation kernels (csrc/rope.cu, internal to libadaln).
#pragma once

#include <cuda_runtime.h>

#include "common.cuh"

namespace adaln {

constexpr uint32_t kDbgHeads = 1024u;  // debug builds: rows, heads, positions
constexpr int kRopeThreads = 256;
constexpr int kRopeMaxD = 256;      // elements of a head
constexpr int kRopeMaxAxes = 8;

// One side (queries or keys): H heads of d elements a token, rows ld elements apart.
struct RopeSide {
    const void* x;        // the projection; backward without a norm: null
    const void* dy;       // backward: the rotated output's gradient
    const void* weight;   // [d], or null (ones)
    void* out;            // forward: the result; backward: dx
    int64_t x_ld, dy_ld, out_ld;
    int heads;
};

struct RopeArgs {
    RopeSide side[2];     // queries, keys
    const int32_t* pos;   // [R, naxes], or null (no rotation)
    float* partials;      // backward: [CTAs][2][d] sums of dy * xhat, or null (not wanted)
    uint32_t* status;     // backward, or null
    WsHeader* header;
    int64_t R;
    int d, naxes, chunk, chunks;  // heads a work item (of the queries' and keys' together), items a token
    int norm;
    float eps;
    // Turns a position step of each pair as a binary fraction (2^-64 of a turn), and its axis.
    unsigned long long freq[kRopeMaxD / 2];
    unsigned char axis[kRopeMaxD / 2];
};

struct RopeReduceArgs {
    const float* partials;
    float* dw[2];         // either may be null
    int64_t G;
    int d;
};

// Resident CTAs an SM.
cudaError_t rope_blocks_per_sm(int dtype, int d, bool bwd, int* out);
cudaError_t launch_rope(const RopeArgs& args, int dtype, bool bwd, int64_t G, cudaStream_t stream);
cudaError_t launch_rope_reduce(const RopeReduceArgs& args, cudaStream_t stream);
// Lanes that share a head: d elements, eight a lane, rounded up to a power of two.
inline int rope_lanes(int64_t d) {
    int l = 1;
    while (8 * l < d) l *= 2;
    return l;
}
cudaError_t debug_word_rope(uint32_t* out, bool reset);

}  // namespace adaln
