// Norms of queries and keys for each head, with their rotation by positions, in one pass:
//
//     xhat = x / sqrt(mean(x^2) + eps),  y = xhat * w,
//     (out[2i], out[2i+1]) = (y[2i] cos t - y[2i+1] sin t,  y[2i] sin t + y[2i+1] cos t)
//
// t = position * theta^(-2i / w) on the pair's axis (of w elements). Backward, with dy the outputs'
// gradient turned back by t:
//
//     dw = sum dy * xhat,  g = dy * w,  dx = rstd * (g - xhat * mean(g * xhat))
//
// Bound by HBM. A power of two of lanes shares a head, eight elements a lane, so that a head's sums
// are a few shuffles and a pair never leaves its lane. A group of lanes takes a token and goes through
// its heads, several on their way at once: the token's angles are computed once for all of them. Short
// batches go in items of fewer heads (rope_items). 32760 x 12 x 128 (queries and keys each), bf16: 75 us
// forward (5.4 TB/s), 118 us backward (5.1 TB/s); 40 heads 225 us (6.0 TB/s); fp32 128 and 195 us
// (6.3 and 6.2 TB/s). Heads whose eighths are no power of two leave lanes idle (15000 x 12 x 72: 3.3 TB/s).
//
// Angles: a position times a frequency is far more than fp32 holds (position 500,000 at frequency 1 is
// off by 0.03 rad). Frequencies are turns as binary fractions of 64 bits; the product with the integer
// position wraps at whole turns by itself. What is left, the fraction of a turn, has the frequency's own
// rounding (a double's, five times 2^-53 of the angle at most), its cut after 64 bits (2^-33 of a turn at any
// position), the product's after 32, and the rounding to the fp32 argument of sine and cosine: 2^-26 of a
// turn, the largest.
#include <atomic>

#include "rope.h"

namespace adaln {

#define ADALN_IN_HEADS(cond) ADALN_IN(::adaln::kDbgHeads, cond)

template <typename T>
struct Lane {
    static constexpr int VE = Io<T>::VE;   // elements of a 16-byte vector
    static constexpr int NV = 8 / VE;      // vectors a lane: v = lane + j * GL of the head's
    static constexpr int NP = VE / 2;      // pairs of a vector
};

template <int GL>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int o = GL / 2; o >= 1; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// Heads on their way at once, and CTAs an SM that the registers are to hold. Forward, bf16, 32760 x 40 x
// 128: four heads and three CTAs 225 us; two and four 256, six and three 231, eight and two 218 (but 81
// instead of 75 us for 12 heads). Backward, bf16, 32760 x 12 x 128: four and two 118 us; two and two 141,
// two and three 140, six and two 114 (but slower with few rows). fp32 backward, 32760 x 12 x 128: two and
// two 195 us, four and one 229.
template <typename T, bool BWD>
__host__ __device__ constexpr int rope_heads() { return sizeof(T) == 4 && BWD ? 2 : 4; }
template <typename T, bool BWD>
__host__ __device__ constexpr int rope_ctas() { return sizeof(T) == 2 && !BWD ? 3 : 2; }

template <typename T>
__device__ __forceinline__ float inv_sqrt(float v) {
    return sizeof(T) == 2 ? rsqrtf(v) : __frsqrt_rn(v);  // (2 steps of fp32 are nothing to bf16)
}

// What a token's heads share is in registers: the angles' cosines and sines, forward times the weights.
template <typename T, int GL, bool BWD>
__global__ void __launch_bounds__(kRopeThreads, rope_ctas<T, BWD>()) rope_kernel(const __grid_constant__ RopeArgs a) {
    using L = Lane<T>;
    constexpr int U = rope_heads<T, BWD>();
    constexpr int GROUPS = kRopeThreads / GL;
    const int lane = threadIdx.x % GL, group = threadIdx.x / GL;
    const int vecs = a.d / L::VE;
    const float inv_d = 1.0f / (float)a.d;
    pdl_begin();
    [[maybe_unused]] f2r dw[2][L::NV][L::NP];
    if constexpr (BWD) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
#pragma unroll
            for (int j = 0; j < L::NV; ++j) {
#pragma unroll
                for (int p = 0; p < L::NP; ++p) dw[s][j][p] = kPairZero;
            }
        }
    }

    const int64_t items = a.R * a.chunks, step = (int64_t)gridDim.x * GROUPS;
    // The lanes of a warp stay together: its groups run as many rounds as its first one.
    const int64_t first = (int64_t)blockIdx.x * GROUPS + group;
    const int64_t warp_first = (int64_t)blockIdx.x * GROUPS + (threadIdx.x & ~31) / GL;
    for (int64_t off = 0; warp_first + off < items; off += step) {
        const int64_t item = first + off;
        const bool live = item < items;
        const int64_t r = !live ? 0 : a.chunks == 1 ? item : item / a.chunks;
        const int h0 = !live || a.chunks == 1 ? 0 : (int)(item % a.chunks) * a.chunk;
        float c[L::NV][L::NP], sn[L::NV][L::NP];
#pragma unroll
        for (int j = 0; j < L::NV; ++j) {
            const int v = lane + j * GL;
#pragma unroll
            for (int p = 0; p < L::NP; ++p) {
                c[j][p] = 1.0f;
                sn[j][p] = 0.0f;
                if (a.pos && v < vecs && ADALN_IN_HEADS(r < a.R)) {
                    const long long at = __ldg(a.pos + r * a.naxes + a.axis[v * L::NP + p]);
                    const int turn32 = (int)(((unsigned long long)at * a.freq[v * L::NP + p]) >> 32);
                    sincospif((float)turn32 * 0x1p-31f, &sn[j][p], &c[j][p]);  // half turns
                }
            }
        }
        // One side's heads [b, e).
        auto heads = [&](int s, int b, int e) {
            const RopeSide& sd = a.side[s];
            const int most = __reduce_max_sync(0xFFFFFFFFu, live ? e - b : 0);
            if (most <= 0) return;
            f2r w[L::NV][L::NP];
#pragma unroll
            for (int j = 0; j < L::NV; ++j) {
#pragma unroll
                for (int p = 0; p < L::NP; ++p) w[j][p] = p_splat(1.0f);
                if (sd.weight && lane + j * GL < vecs)
                    Io<T>::unpackp(ld_keep(reinterpret_cast<const uint4*>(sd.weight) + lane + j * GL), w[j]);
            }
            // Forward: out = x0 * ac + x1 * bd, what the pair's elements have of both results.
            [[maybe_unused]] float2 ac[L::NV][L::NP], bd[L::NV][L::NP];
            if constexpr (!BWD) {
#pragma unroll
                for (int j = 0; j < L::NV; ++j) {
#pragma unroll
                    for (int p = 0; p < L::NP; ++p) {
                        const float2 f = p_get(w[j][p]);
                        ac[j][p] = make_float2(f.x * c[j][p], f.x * sn[j][p]);
                        bd[j][p] = make_float2(-f.y * sn[j][p], f.y * c[j][p]);
                    }
                }
            }
            const T* x0 = reinterpret_cast<const T*>(sd.x) + r * sd.x_ld + lane * L::VE;
            [[maybe_unused]] const T* y0 = reinterpret_cast<const T*>(sd.dy) + r * sd.dy_ld + lane * L::VE;
            T* o0 = reinterpret_cast<T*>(sd.out) + r * sd.out_ld + lane * L::VE;
            for (int i = 0; i < most; i += U) {
                uint4 x[U][L::NV];
                [[maybe_unused]] uint4 y[U][L::NV];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int h = b + i + u, at = h * a.d;
#pragma unroll
                    for (int j = 0; j < L::NV; ++j) {
                        x[u][j] = make_uint4(0, 0, 0, 0);
                        if (BWD) y[u][j] = x[u][j];
                        if (live && h < e && lane + j * GL < vecs && ADALN_IN_HEADS(r < a.R && h >= 0 && h < sd.heads)) {
                            if (!BWD || a.norm) x[u][j] = ld_stream(x0 + at + j * GL * L::VE);
                            if (BWD) y[u][j] = ld_stream(y0 + at + j * GL * L::VE);
                        }
                    }
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int h = b + i + u, at = h * a.d;
                    f2r f[L::NV][L::NP];
                    [[maybe_unused]] f2r g[L::NV][L::NP], dy[L::NV][L::NP];
                    f2r ss = kPairZero, gs = kPairZero;
#pragma unroll
                    for (int j = 0; j < L::NV; ++j) {
                        Io<T>::unpackp(x[u][j], f[j]);
                        if (BWD) Io<T>::unpackp(y[u][j], dy[j]);
#pragma unroll
                        for (int p = 0; p < L::NP; ++p) {
                            ss = p_fma(f[j][p], f[j][p], ss);
                            if constexpr (BWD) {
                                const float2 d = p_get(dy[j][p]);
                                dy[j][p] = p_make(fmaf(d.y, sn[j][p], d.x * c[j][p]), fmaf(d.y, c[j][p], -d.x * sn[j][p]));
                                g[j][p] = p_mul(w[j][p], dy[j][p]);
                                gs = p_fma(g[j][p], f[j][p], gs);
                            }
                        }
                    }
                    float rstd = 1.0f, m = 0.0f;
                    if (a.norm) {
                        rstd = inv_sqrt<T>(fmaf(group_sum<GL>(p_hsum(ss)), inv_d, a.eps));
                        if (BWD) m = group_sum<GL>(p_hsum(gs)) * rstd * inv_d;
                    }
                    const f2r rs = p_splat(rstd);
                    [[maybe_unused]] const f2r nm = p_splat(-m);
#pragma unroll
                    for (int j = 0; j < L::NV; ++j) {
                        f2r o[L::NP];
#pragma unroll
                        for (int p = 0; p < L::NP; ++p) {
                            if constexpr (!BWD) {
                                const float2 e2 = p_get(f[j][p]);
                                o[p] = p_mul(p_make(fmaf(e2.y, bd[j][p].x, e2.x * ac[j][p].x),
                                                    fmaf(e2.y, bd[j][p].y, e2.x * ac[j][p].y)),
                                             rs);
                            } else {
                                o[p] = g[j][p];
                                if (a.norm) {
                                    const f2r xhat = p_mul(f[j][p], rs);
                                    dw[s][j][p] = p_fma(dy[j][p], xhat, dw[s][j][p]);
                                    o[p] = p_mul(rs, p_fma(xhat, nm, g[j][p]));
                                }
                            }
                        }
                        if (live && h < e && lane + j * GL < vecs && ADALN_IN_HEADS(r < a.R && h < sd.heads))
                            st_vec(o0 + at + j * GL * L::VE, Io<T>::packp(o));
                    }
                }
            }
        };
        const int Hq = a.side[0].heads, h1 = min(h0 + a.chunk, Hq + a.side[1].heads);
        heads(0, h0, min(h1, Hq));
        heads(1, max(h0, Hq) - Hq, h1 - Hq);
    }

    if constexpr (BWD) {
        if (a.partials) {
            // The groups' sums, added in the groups' order.
            __shared__ float red[2 * 8 * kRopeThreads];
            const int n = 8 * GL;
#pragma unroll
            for (int s = 0; s < 2; ++s) {
#pragma unroll
                for (int j = 0; j < L::NV; ++j) {
#pragma unroll
                    for (int p = 0; p < L::NP; ++p)
                        *reinterpret_cast<float2*>(red + (s * GROUPS + group) * n + (lane + j * GL) * L::VE + 2 * p) =
                            p_get(dw[s][j][p]);
                }
            }
            __syncthreads();
            for (int i = threadIdx.x; i < 2 * a.d; i += kRopeThreads) {
                const int s = i >= a.d, col = i - s * a.d;
                float sum = 0.0f;
                for (int q = 0; q < GROUPS; ++q) sum += red[(s * GROUPS + q) * n + col];
                a.partials[(int64_t)blockIdx.x * 2 * a.d + i] = sum;
            }
        }
        publish_status(0, a.status, a.header);
    }
}

// Columns of the partials, 32 a CTA: 32 threads a column take every 32nd row each, then add up in a
// fixed order.
__global__ void __launch_bounds__(1024) rope_reduce_kernel(const RopeReduceArgs a) {
    pdl_begin();
    __shared__ float red[32][33];
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + x;
    float sum = 0.0f;
    if (col < 2 * a.d) {
#pragma unroll 4
        for (int64_t g = y; g < a.G; g += 32) sum += a.partials[g * 2 * a.d + col];
    }
    red[y][x] = sum;
    __syncthreads();
    float v[1] = {red[x][y]};
    warp_sum(v);
    const int out = blockIdx.x * 32 + y;
    if (x == 0 && out < 2 * a.d) {
        const int s = out >= a.d;
        if (a.dw[s]) a.dw[s][out - s * a.d] = v[0];
    }
}

namespace {

template <typename T, bool BWD>
const void* rope_fn(int lanes) {
    switch (lanes) {
        case 1: return reinterpret_cast<const void*>(&rope_kernel<T, 1, BWD>);
        case 2: return reinterpret_cast<const void*>(&rope_kernel<T, 2, BWD>);
        case 4: return reinterpret_cast<const void*>(&rope_kernel<T, 4, BWD>);
        case 8: return reinterpret_cast<const void*>(&rope_kernel<T, 8, BWD>);
        case 16: return reinterpret_cast<const void*>(&rope_kernel<T, 16, BWD>);
        default: return reinterpret_cast<const void*>(&rope_kernel<T, 32, BWD>);
    }
}

const void* rope_fn(int dtype, int d, bool bwd) {
    const int lanes = rope_lanes(d);
    if (dtype == 0) return bwd ? rope_fn<float, true>(lanes) : rope_fn<float, false>(lanes);
    return bwd ? rope_fn<__nv_bfloat16, true>(lanes) : rope_fn<__nv_bfloat16, false>(lanes);
}

}  // namespace

cudaError_t rope_blocks_per_sm(int dtype, int d, bool bwd, int* out) {
    return cudaOccupancyMaxActiveBlocksPerMultiprocessor(out, rope_fn(dtype, d, bwd), kRopeThreads, 0);
}

cudaError_t launch_rope(const RopeArgs& args, int dtype, bool bwd, int64_t G, cudaStream_t stream) {
    RopeArgs a = args;
    void* params[] = {&a};
    return launch_dependent(rope_fn(dtype, a.d, bwd), dim3((unsigned)G), dim3(kRopeThreads), params, 0, stream);
}

cudaError_t launch_rope_reduce(const RopeReduceArgs& args, cudaStream_t stream) {
    RopeReduceArgs a = args;
    void* params[] = {&a};
    return launch_dependent(reinterpret_cast<const void*>(&rope_reduce_kernel), dim3((unsigned)((2 * a.d + 31) / 32)),
                            dim3(1024), params, 0, stream);
}

cudaError_t debug_word_rope(uint32_t* out, bool reset) { return debug_word(out, reset); }

}  // namespace adaln
