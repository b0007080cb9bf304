// Softmax cross entropy over a vocabulary, from hidden rows and the head's weight, with its
// gradient; the logits are never kept.
//
//     z = x W^T,  lse = log sum_v exp(z_v),  loss = lse - z_target
//     dz = softmax(z) * (dloss + dlse) - onehot(target) * dloss,  dx = dz W,  dW = dz^T x
//
// Rows whose target is ignore_index carry no loss. Masked-token training has many of them, so
// the first kernel packs the other rows densely (and their count stays on the device: the
// kernels after it read it). Then
//   forward:  logits_kernel<false>: tiles of z in tensor memory, reduced to (max, sum exp) a
//             row and half tile; lse_kernel joins them in a fixed order;
//   backward, a piece of the vocabulary at a time: logits_kernel<true> computes the piece's
//             tiles again and writes dz in bf16; grad_kernel forms dW of the piece (whole) and
//             adds the piece's part of dx to an fp32 buffer; finish_kernel rounds dx once.
// The products run on the tensor cores with fp32 accumulators; exp, sums and lse are fp32. dz is
// rounded to bf16 as an operand of the next two products (up to half a step, 2^-8, of each value).
// The target's dz is often most of its row's and its word's gradient, and much the same in all rows
// of a word (a mean's, of small probabilities), so that its roundings need not average out: what
// they leave off is kept and added in fp32, to dx, and to dW in the order of the word's rows.
//
// Bound by the tensor cores from a few hundred rows on: 8192 rows, 50,257 words, D = 2048 take
// 0.81 ms forward (2.1 PFLOP/s, the tensor pipe 96% active) and 2.8 ms backward; with a few rows by
// the chain of launches (1 row, 1000 words, D = 512: 9.6 us forward, 17.2 us backward on the device).
#include <algorithm>
#include <atomic>

#include "tensor.cuh"
#include "xent.h"

namespace adaln {

constexpr int kAccs = 2;              // accumulator tiles in tensor memory
constexpr int kEpiWarp = 4;           // first epilogue warp
constexpr int kEpiWarps = 8;          // two per 32 lanes of tensor memory, every other 64 columns each
constexpr int kGemmThreads = (kEpiWarp + kEpiWarps) * 32;
constexpr uint32_t kABytes = kCtaM * kTileK * 2, kBBytes = kTileN / 2 * kTileK * 2;
constexpr uint32_t kStageBytes = kABytes + kBBytes;
// Six stages measured the same or slower (96 x 8192 x 1024 backward: 32.9 us against 31.4).
constexpr int kGemmStages = 5;
constexpr uint32_t kOutBytes = 32 * 128;  // an epilogue warp's rows on their way out
constexpr size_t kGemmSmem = 1024 + (size_t)kGemmStages * kStageBytes + (size_t)kEpiWarps * kOutBytes;
constexpr uint32_t kMnBlock = 64 * kTileK * 2;  // 64 m of all the tile's k (MN-major operands)
constexpr float kLog2e = 1.4426950408889634f;

#define ADALN_IN_LOSS(cond) ADALN_IN(::adaln::kDbgLoss, cond)

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }
// 2^x, results below 2^-126 as 0.
__device__ __forceinline__ float exp2_ftz(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// The epilogue warps' own barrier; true if `ok` is, in all of them.
__device__ __forceinline__ bool epilogue_all(bool ok) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.and.pred q, 1, %2, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)ok), "n"(kEpiWarps * 32)
        : "memory");
    return r != 0;
}

// ---------------------------------------------------------------------------------------
// Packing: CTA b counts the rows that carry a loss before its range, then places its own
// behind them, so the packed order is the row order, whatever the CTAs' timing, and one launch
// does it. Reads x and writes the packed copy once: 13 us for 8192 rows of 2048 (5.1 TB/s), its
// loads eight at a time.
// ---------------------------------------------------------------------------------------
__global__ void __launch_bounds__(kPackThreads) pack_kernel(const PackArgs a) {
    pdl_begin();
    __shared__ int warp_tot[kPackThreads / 32];
    __shared__ int list[kPackThreads];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int NW = kPackThreads / 32;
    const int64_t G = gridDim.x, b = blockIdx.x;
    const int64_t r0 = tile_begin(b, a.N, G), r1 = tile_begin(b + 1, a.N, G);
    bool bad = false;
    auto counts = [&](int64_t r, int64_t* t) {
        if (!ADALN_IN_LOSS(r >= 0 && r < a.N)) return false;
        *t = a.target[r];
        return *t != a.ignore && *t >= 0 && *t < a.V;
    };
    // Rows that count before r0.
    int n = 0;
    int64_t first = tid;
    for (; first + 7 * kPackThreads < r0; first += 8 * kPackThreads) {  // eight loads on their way
        int64_t t[8];
        bool on[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) on[i] = counts(first + i * kPackThreads, t + i);
#pragma unroll
        for (int i = 0; i < 8; ++i) n += on[i] ? 1 : 0;
    }
    for (; first < r0; first += kPackThreads) {
        int64_t t;
        n += counts(first, &t) ? 1 : 0;
    }
    for (int o = 16; o >= 1; o >>= 1) n += __shfl_xor_sync(0xFFFFFFFFu, n, o);
    if (lane == 0) warp_tot[warp] = n;
    __syncthreads();
    int base = 0;
    for (int w = 0; w < NW; ++w) base += warp_tot[w];
    const int64_t vecs = a.D / 8;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    for (int64_t c0 = r0; c0 < r1; c0 += kPackThreads) {
        const int64_t r = c0 + tid;
        int64_t t = 0;
        const bool in = r < r1;
        const bool on = in && counts(r, &t);
        if (in && !on && t != a.ignore) bad = true;
        const uint32_t ballot = __ballot_sync(0xFFFFFFFFu, on);
        __syncthreads();  // the last chunk's list and totals have been read
        if (lane == 0) warp_tot[warp] = __popc(ballot);
        __syncthreads();
        int at = base, all = 0;
        for (int w = 0; w < NW; ++w) {
            if (w < warp) at += warp_tot[w];
            all += warp_tot[w];
        }
        at += __popc(ballot & ((1u << lane) - 1u));
        list[tid] = on ? at : -1;
        if (on && ADALN_IN_LOSS(at < a.Np)) {
            a.row[at] = (int32_t)r;
            a.tgt[at] = (int32_t)t;
            if (a.lse) {
                a.row_lse[at] = a.lse[r];
                const float up = a.dloss[r];
                a.row_gt[at] = up;
                a.row_gs[at] = a.dlse ? up + a.dlse[r] : up;
            }
        } else if (in && !on && a.loss_out) {
            a.loss_out[r] = 0.0f;
            a.lse_out[r] = 0.0f;
        }
        __syncthreads();
        // One warp a row: pack the rows that count, zero the gradient rows of the others.
        for (int i = warp; i < kPackThreads && c0 + i < r1; i += NW) {
            const int to = list[i];
            if (to >= 0) {
                const uint4* src = reinterpret_cast<const uint4*>(a.x) + (c0 + i) * vecs;
                uint4* dst = reinterpret_cast<uint4*>(a.xp) + (int64_t)to * vecs;
                if (!ADALN_IN_LOSS(c0 + i < a.N && to < a.Np)) continue;
                int64_t v = lane;
                for (; v + 7 * 32 < vecs; v += 8 * 32) {  // eight loads on their way
                    uint4 q[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) q[j] = ld_stream(src + v + 32 * j);
#pragma unroll
                    for (int j = 0; j < 8; ++j) dst[v + 32 * j] = q[j];
                }
                for (; v < vecs; v += 32) dst[v] = ld_stream(src + v);
            } else if (a.dx) {
                uint4* dst = reinterpret_cast<uint4*>(a.dx) + (c0 + i) * vecs;
                for (int64_t v = lane; v < vecs; v += 32)
                    if (ADALN_IN_LOSS(c0 + i < a.N)) dst[v] = zero;
            }
        }
        base += all;
    }
    if (a.word_hits) {
        for (int64_t v = b * kPackThreads + tid; v < a.V; v += G * kPackThreads) a.word_hits[v] = 0;
    }
    // The rows between the packed ones and the next K step of dweight are operands of it: zeros.
    // Those from N on are shared out, the others (rows without a loss made room) the last CTA's.
    // The rest of the last row tile only makes rows of products that nothing reads.
    uint4* xp = reinterpret_cast<uint4*>(a.xp);
    auto clear = [&](int64_t r0, int64_t r1, int64_t first, int64_t step) {
        for (int64_t v = r0 * vecs + first; v < r1 * vecs; v += step)
            if (ADALN_IN_LOSS(v < a.Np * vecs)) xp[v] = zero;
    };
    const int64_t kpad = ((int64_t)a.N + kTileK - 1) / kTileK * kTileK;
    if (a.lse) clear(a.N, kpad, b * kPackThreads + tid, G * kPackThreads);
    if (b == G - 1) {
        if (a.lse) clear(base, min(((int64_t)base + kTileK - 1) / kTileK * kTileK, a.N), tid, kPackThreads);
        const int64_t end = ((int64_t)base + kTileM - 1) / kTileM * kTileM;
        for (int64_t r = base + tid; r < end; r += kPackThreads) {
            if (!ADALN_IN_LOSS(r < a.Np)) continue;
            a.tgt[r] = -1;
            if (a.lse) a.row_lse[r] = a.row_gt[r] = a.row_gs[r] = 0.0f;
        }
        if (tid == 0) {
            *a.nact = base;
            if (a.many.count) *a.many.count = 0;
            if (a.many.listed) *a.many.listed = 0;
        }
    }
    const bool any_bad = __syncthreads_or(bad);
    if (tid == 0) {
        a.status[b] = any_bad ? kErrTarget : 0u;
        if (b == 0) {
            a.status[G] = 0u;  // the tensor-core kernels' word
            a.header->magic = kStatusMagic;
            a.header->nwords = (uint32_t)G + 1u;
        }
    }
}

// ---------------------------------------------------------------------------------------
// Matrix products. A persistent CTA pair on every two SMs walks its units (output tiles): warps 0 and 3
// of each CTA fill its half of a ring of shared-memory stages by TMA (all of a stage completes on
// CTA 0's barrier), warp 1 of CTA 0 issues the pair's products into one of two accumulators,
// warps 4.. of each CTA read its rows of the other one back and run the epilogue.
// ---------------------------------------------------------------------------------------
struct Unit {
    const CUtensorMap* ma;
    const CUtensorMap* mb;
    int64_t m0, n0;     // output tile: rows of A, rows of B
    int64_t k0;         // first k of A
    int64_t kb0;        // first k of B
    int iters;          // K steps of kTileK
    bool a_mn, b_mn;    // operand layouts
    int kind;           // 0: logits; 1: dx; 2: dweight
    int64_t slot;       // dx: which part of the K range
};

// decode(u): unit u. prologue(unit): run by the epilogue threads while the unit's products are
// still under way. epilogue(unit, accumulator, row of the tile, half (which 64 columns), out, release):
// calls release() when it has read the accumulator; `out` is the warp's buffer for results, read
// by stores that lane 0 issues. units() is called, and global memory first
// read, after the kernel ahead has finished; barriers and tensor memory are set up before.
// TN: columns a tile; a template argument because a loading thread that computes with it is late
// (8192 x 50257 x 2048 backward: 8% slower).
// HALVES: the second half of the K steps is accumulated TN columns further on, for the epilogue to add.
// The tensor cores cut sums towards zero at every K step, so that errors of long sums do not average
// out; narrow tiles leave the columns free (300 rows, 16 words, D = 2048: losses off by 5.7e-7 of
// themselves, 1.2e-6 in one sum; 0.1 us a kernel). Wide tiles use all of tensor memory.
template <int TN, bool HALVES, class Units, class Decode, class Prologue, class Epilogue>
__device__ __forceinline__ void gemm_loop(Units count, uint32_t* status, Decode decode, Prologue prologue,
                                          Epilogue epilogue) {
    extern __shared__ uint4 dyn[];
    __shared__ __align__(8) uint64_t bars[2 * kGemmStages + 2 * kAccs + 1];
    __shared__ uint32_t tmem_base;
    __shared__ uint32_t fills[4];  // CTA 0: stages filled by each loading warp of the pair
    __shared__ int abort_flag;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = cluster_ctarank();
    const uint32_t first = blockIdx.x >> 1, step = gridDim.x >> 1;  // units of this pair
    const uint32_t data = (smem_addr(dyn) + 1023u) & ~1023u;
    const uint32_t full = smem_addr(bars), empty = full + 8u * kGemmStages;
    const uint32_t afull = empty + 8u * kGemmStages, aempty = afull + 8u * kAccs, drain = aempty + 8u * kAccs;
    if (tid == 0) {
        for (int i = 0; i < kGemmStages; ++i) {
            mbar_init(full + 8u * i, 1);
            mbar_init(empty + 8u * i, 1);
        }
        for (int i = 0; i < kAccs; ++i) {
            mbar_init(afull + 8u * i, 1);
            mbar_init(aempty + 8u * i, 2 * kEpiWarps);  // CTA 0's: both CTAs' epilogues
        }
        mbar_init(drain, 1);
        abort_flag = 0;
        mbar_fence_init();
    }
    if (warp == 2) tmem_alloc(smem_addr(&tmem_base), kAccs * kTileN);
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // the other CTA's barriers are ready too
    tc_fence_after();
    const uint32_t tmem = tmem_base;
    pdl_wait();
    const uint32_t units = count();
    bool issued = false;  // products, by warp 1 of CTA 0

    const int role = __shfl_sync(0xFFFFFFFFu, warp, 0);  // the warp's number, known to be uniform
    if (role == 0 || role == 3) {
        // Warp 0 loads this CTA's half of A, warp 3 its half of B, both into the same stages: one
        // thread issuing both is late (the loads of an MN-major operand are one a 64 columns).
        fence_async_proxy();
        const bool is_b = role == 3;
        const uint32_t base = data + (is_b ? kABytes : 0u), bars0 = cluster_map(full, 0);
        int s = 0;
        uint32_t lap = 0;
        bool live = true;
        for (uint32_t u = first; live && u < units; u += step) {
            const Unit t = decode(u);
            const CUtensorMap* map = is_b ? t.mb : t.ma;
            const int x0 = is_b ? (int)t.n0 + (int)rank * (TN / 2) : (int)t.m0 + (int)rank * kCtaM;
            const int blocks = !(is_b ? t.b_mn : t.a_mn) ? 0 : is_b ? TN / 128 : kCtaM / 64;
            int k = (int)(is_b ? t.kb0 : t.k0);
            for (int i = 0; i < t.iters; ++i, k += kTileK) {
                // The lanes go on together or stop together.
                live = __all_sync(0xFFFFFFFFu, lap == 0 || mbar_wait_bounded(empty + 8u * s, (lap - 1) & 1u, &abort_flag));
                if (!live) break;
                if (elect_lane()) {
                    const uint32_t bar = bars0 + 8u * s, dst = base + s * kStageBytes;
                    if (rank == 0 && !is_b)
                        mbar_arrive_expect_tx(full + 8u * s, 2 * kABytes + (uint32_t)TN * kTileK * 2);
                    if (blocks == 0) {
                        tma_load(dst, map, k, x0, bar);
                    } else {
                        tma_load(dst, map, x0, k, bar);
                        if (blocks == 2) tma_load(dst + kMnBlock, map, x0 + 64, k, bar);
                    }
                }
                if (++s == kGemmStages) {
                    s = 0;
                    ++lap;
                }
            }
        }
        if (lane == 0)
            st_cluster_u32(cluster_map(smem_addr(fills) + 4u * (2 * rank + (is_b ? 1 : 0)), 0), lap * kGemmStages + s);
    } else if (role == 1) {
        if (rank == 0) {
            // Descriptors of stage 0; a stage and a K step move the address field (the low bits).
            const uint64_t da0 = smem_desc(data, kMnBlock), db0 = smem_desc(data + kABytes, kMnBlock);
            int s = 0, acc = 0;
            uint32_t lap = 0, alap = 0;
            bool live = true;
            for (uint32_t u = first; live && u < units; u += step) {
                const Unit t = decode(u);
                const uint32_t idesc = mma_desc(kTileM, TN, t.a_mn, t.b_mn);
                // 16 k: 32 bytes of a K-major row, 16 rows of an MN-major tile.
                const uint32_t ak = (t.a_mn ? 2048u : 32u) >> 4, bk = (t.b_mn ? 2048u : 32u) >> 4;
                live = __all_sync(0xFFFFFFFFu, alap == 0 || mbar_wait_cluster_bounded(aempty + 8u * acc,
                                                                                      (alap - 1) & 1u, &abort_flag));
                if (!live) break;
                tc_fence_after();
                const uint32_t d0 = tmem + (uint32_t)acc * kTileN;
                const int second = HALVES ? (t.iters + 1) / 2 : t.iters;
                for (int i = 0; i < t.iters; ++i) {
                    live = __all_sync(0xFFFFFFFFu, mbar_wait_cluster_bounded(full + 8u * s, lap & 1u, &abort_flag));
                    if (!live) break;
                    tc_fence_after();
                    if (elect_lane()) {
                        const uint64_t off = (uint64_t)(uint32_t)(s * (int)(kStageBytes >> 4));
                        const uint64_t da = da0 + off, db = db0 + off;
                        const uint32_t d = HALVES && i >= second ? d0 + TN : d0;
                        const bool fresh = i == 0 || (HALVES && i == second);
#pragma unroll
                        for (int k = 0; k < kTileK / 16; ++k)
                            mma_bf16(d, da + (uint64_t)(k * ak), db + (uint64_t)(k * bk), idesc, !fresh || k > 0);
                        mma_commit(empty + 8u * s);
                    }
                    issued = true;
                    if (++s == kGemmStages) {
                        s = 0;
                        ++lap;
                    }
                }
                if (!live) break;
                if (elect_lane()) mma_commit(afull + 8u * acc);
                if (++acc == kAccs) {
                    acc = 0;
                    ++alap;
                }
            }
        }
    } else if (role >= kEpiWarp) {
        const int q = warp & 3, half = (warp - kEpiWarp) >> 2;
        const uint32_t out = data + kGemmStages * kStageBytes + (uint32_t)(warp - kEpiWarp) * kOutBytes;
        int acc = 0;
        uint32_t alap = 0;
        for (uint32_t u = first; u < units; u += step) {
            const Unit t = decode(u);
            prologue(t);
            // All epilogue warps go on or none: they meet at barriers of their own.
            if (!epilogue_all(mbar_wait_bounded(afull + 8u * acc, alap & 1u, &abort_flag))) break;
            tc_fence_after();
            const uint32_t src = tmem + (uint32_t)acc * kTileN + ((uint32_t)q << 21);
            epilogue(t, src, (int)rank * kCtaM + q * 32 + lane, half, out, [&]() {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_relaxed(cluster_map(aempty + 8u * acc, 0));
            });
            if (++acc == kAccs) {
                acc = 0;
                ++alap;
            }
        }
        if (lane == 0) tma_store_wait();
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (tid == 0 && *(volatile int*)&abort_flag) st_cluster_u32(cluster_map(smem_addr(&abort_flag), rank ^ 1u), 1);
    cluster_sync();  // every wait of the pair is over, nothing more is issued, and both flags agree
    // Without a timeout no product, copy or arrival is left. After one, whichever warp's it was,
    // copies and products may still be on their way: CTA 0 gives each stage's last copies and the
    // products a further bounded wait before memory is given back.
    if (__builtin_expect(*(volatile int*)&abort_flag, 0)) {
        volatile int never = 0;
        if (rank == 0 && tid == 0) {
            const uint32_t most = max(max(fills[0], fills[1]), max(fills[2], fills[3]));
            for (uint32_t q = 0; q < min(most, (uint32_t)kGemmStages); ++q)
                mbar_wait_bounded(full + 8u * q, ((most - 1 - q) / kGemmStages) & 1u, &never);
        }
        if (rank == 0 && warp == 1 && issued && elect_lane()) {
            mma_commit(drain);
            mbar_wait_bounded(drain, 0, &never);
        }
        __syncwarp();
        cluster_sync();
    }
    tc_fence_after();
    if (warp == 2) tmem_free(tmem, kAccs * kTileN);
    __syncwarp();
    cluster_sync();
    if (tid == 0 && abort_flag) atomicOr(status, kErrTimeout);
}

// The tile's logits, as row statistics (PROBS false) or as dz (PROBS true). Tiles of all rows first:
// x stays in L2 and the weight is read once. 8192 x 50257 x 2048: 782 us for the statistics (2.16
// PFLOP/s); dz, whose epilogue also writes 0.8 GB through shared memory, 929 us (1.82 PFLOP/s).
template <bool PROBS, int TN>
__global__ void __launch_bounds__(kGemmThreads, 1) logits_kernel(const __grid_constant__ CUtensorMap mx,
                                                              const __grid_constant__ CUtensorMap mw,
                                                              const __grid_constant__ CUtensorMap mp,
                                                              const LogitsArgs a) {
    pdl_trigger();
    if (threadIdx.x == 0) {
        tma_prefetch_map(&mx);
        tma_prefetch_map(&mw);
        if (PROBS) tma_prefetch_map(&mp);
    }
    int64_t nact = 0;
    uint32_t mt = 0;  // tile counts are 32 bits (checked on the host): their quotients are cheap
    const uint32_t nt = (uint32_t)((a.v1 - a.v0 + TN - 1) / TN);
    auto count = [&]() {
        nact = *a.nact;
        mt = (uint32_t)((nact + kTileM - 1) / kTileM);
        return mt * nt;
    };
    auto decode = [&](uint32_t u) {
        Unit t{};
        t.ma = &mx;
        t.mb = &mw;
        t.m0 = (int64_t)(u % mt) * kTileM;
        t.n0 = a.v0 + (int64_t)(u / mt) * TN;
        t.iters = (int)((a.D + kTileK - 1) / kTileK);
        return t;
    };
    // This thread's row, read while the tile's products are under way.
    const int lane = threadIdx.x & 31;
    const int64_t rank0 = (int64_t)cluster_ctarank() * kCtaM;
    int tgt = -1;
    int64_t mine = -1;
    [[maybe_unused]] float lse = 0.0f, gs = 0.0f, gt = 0.0f;
    auto prologue = [&](const Unit& t) {
        const int64_t row = t.m0 + rank0 + (threadIdx.x & 127);
        if (row == mine || !ADALN_IN_LOSS(row < a.Np)) return;
        mine = row;
        tgt = a.tgt[row];
        if constexpr (PROBS) {
            lse = a.row_lse[row];
            gs = a.row_gs[row];
            gt = a.row_gt[row];
        }
    };
    constexpr bool HALVES = TN < kTileN;
    gemm_loop<TN, HALVES>(count, a.status, decode, prologue, [&](const Unit& t, uint32_t src, int r, int half,
                                                             [[maybe_unused]] uint32_t out, auto release) {
        const int64_t row = t.m0 + r;
        const bool in = ADALN_IN_LOSS(row < a.Np);
        [[maybe_unused]] const int64_t krows = (nact + kTileK - 1) / kTileK * kTileK;
        const int64_t c0 = t.n0;
        const f2r l2e = p_splat(kLog2e);
        [[maybe_unused]] float top = neg_inf(), sum = 0.0f;
#pragma unroll 1
        for (int c = 64 * half; c < TN; c += 128) {
            float v[64];
            __syncwarp();
            tmem_ld64(src + c, v);
            if (HALVES && t.iters > 1) {
#pragma unroll
                for (int h = 0; h < 64; h += 32) {
                    float w[32];
                    tmem_ld32(src + TN + c + h, w);
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[h + j] += w[j];
                }
            }
            const int64_t col = c0 + c;
            const int hit = (int64_t)tgt >= col && (int64_t)tgt < col + 64 ? (int)(tgt - col) : -1;
            float zt = 0.0f;
            if (hit >= 0) {
#pragma unroll
                for (int j = 0; j < 64; ++j) zt = j == hit ? v[j] : zt;
            }
            if constexpr (!PROBS) {
                if (col + 64 > a.V) {
#pragma unroll
                    for (int j = 0; j < 64; ++j)
                        if (col + j >= a.V) v[j] = neg_inf();
                }
                if (hit >= 0 && in) a.zt[row] = zt;
                float m4[4] = {top, neg_inf(), neg_inf(), neg_inf()};
#pragma unroll
                for (int j = 0; j < 64; ++j) m4[j & 3] = fmaxf(m4[j & 3], v[j]);
                const float m = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
                // A chunk with no finite value at all adds nothing (and NaN is kept below).
                const float mm = m == neg_inf() ? 0.0f : m;
                const f2r m2 = p_splat(-mm);
                f2r s[2] = {kPairZero, kPairZero};
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    // The difference first: the maximum's exponential is exactly 1.
                    const float2 e = p_get(p_mul(p_add(p_make(v[2 * j], v[2 * j + 1]), m2), l2e));
                    s[j & 1] = p_add(s[j & 1], p_make(exp2_ftz(e.x), exp2_ftz(e.y)));
                }
                sum = sum * exp2_ftz((top - mm) * kLog2e) + p_hsum(p_add(s[0], s[1]));
                top = m;
            } else {
                const f2r nl = p_splat(-lse), g2 = p_splat(gs);
                uint32_t w[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    const float2 e = p_get(p_mul(p_add(p_make(v[2 * j], v[2 * j + 1]), nl), l2e));
                    const float2 p = p_get(p_mul(p_make(exp2_ftz(e.x), exp2_ftz(e.y)), g2));
                    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[j]) : "f"(p.y), "f"(p.x));
                }
                if (hit >= 0) {
                    // The target's dz: what its rounding leaves off is kept.
                    const float d = exp2_ftz((zt - lse) * kLog2e) * gs - gt;
                    const uint32_t bits = __bfloat16_as_ushort(__float2bfloat16_rn(d));
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (j == hit >> 1) w[j] = hit & 1 ? (w[j] & 0xFFFFu) | bits << 16 : (w[j] & 0xFFFF0000u) | bits;
                    if (in) a.row_lo[row] = d - __uint_as_float(bits << 16);
                    if (in && a.word_hits && ADALN_IN_LOSS(tgt < a.V)) {
                        const int k = atomicAdd(a.word_hits + tgt, 1);
                        if (k < kHits) a.word_rows[(int64_t)tgt * kHits + k] = (int32_t)row;
                        if (k == kHits) {  // more than the epilogue of dweight takes
                            const int slot = atomicAdd(a.many.count, 1);
                            if (ADALN_IN_LOSS(slot < a.many.slots)) {
                                a.many.word[slot] = tgt;
                                a.many.slot[tgt] = slot;
                            }
                        }
                    }
                }
                // Columns past the vocabulary and rows past the packed ones, up to a whole K step of
                // dweight, are operands too: zeros.
                if (col + 64 > a.V || row >= nact) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        if (col + 2 * j >= a.V || row >= nact) w[j] = 0u;
                        else if (col + 2 * j + 1 >= a.V) w[j] &= 0xFFFFu;
                    }
                }
                if (lane == 0) tma_store_read();
                __syncwarp();
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    st_swizzled(out + (uint32_t)lane * 128u, lane, j, w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
                fence_shared_async();
                __syncwarp();
                // Rows 32 at a time: krows is a multiple of 32.
                if (lane == 0 && row < krows && ADALN_IN_LOSS(row + 32 <= a.Np && col - a.v0 + 64 <= a.ldp))
                    tma_store(&mp, (int)(col - a.v0), (int)row, out, false);
            }
        }
        release();
        if constexpr (!PROBS) {
            const int64_t part = (int64_t)((uint32_t)(t.n0 - a.v0) / TN) * 2 + half;
            if (in && row < nact) a.parts[part * a.Np + row] = make_float2(top, sum);
        }
    });
}

// dx += dz W and dweight = dz^T x of one piece of the vocabulary, as one list of units: dx
// tiles, each in `splits` parts of the piece's columns, then dweight tiles (one list, so that only
// one wave is partly filled). 8192 x 50257 x 2048: 1.8 ms in four pieces (1.88 PFLOP/s).
template <int TN>
__global__ void __launch_bounds__(kGemmThreads, 1) grad_kernel(const __grid_constant__ CUtensorMap mp,
                                                            const __grid_constant__ CUtensorMap mw,
                                                            const __grid_constant__ CUtensorMap mx,
                                                            const __grid_constant__ CUtensorMap mpt,
                                                            const __grid_constant__ CUtensorMap mdx,
                                                            const __grid_constant__ CUtensorMap mdw,
                                                            const GradArgs a) {
    pdl_trigger();
    if (threadIdx.x == 0) {
        for (const CUtensorMap* m : {&mp, &mw, &mx, &mpt}) tma_prefetch_map(m);
        if (a.dxacc) tma_prefetch_map(&mdx);
        if (a.dweight) tma_prefetch_map(&mdw);
    }
    int64_t nact = 0;
    uint32_t per = 0, ndx = 0;  // units of one part of dx, and of all
    const uint32_t dt = (uint32_t)((a.D + TN - 1) / TN);
    const uint32_t kv = (uint32_t)((a.v1 - a.v0 + kTileK - 1) / kTileK);  // K steps of dx
    const uint32_t vt = (uint32_t)((a.v1 - a.v0 + kTileM - 1) / kTileM);
    auto count = [&]() {
        nact = *a.nact;
        per = (uint32_t)((nact + kTileM - 1) / kTileM) * dt;
        ndx = a.dxacc ? per * (uint32_t)a.splits : 0;
        return ndx + (a.dweight ? vt * dt : 0);
    };
    auto decode = [&](uint32_t u) {
        Unit t{};
        t.b_mn = true;
        if (u < ndx) {
            t.kind = 1;
            const uint32_t slot = u / per, w = u - slot * per;
            const uint32_t k0 = slot * kv / (uint32_t)a.splits, k1 = (slot + 1) * kv / (uint32_t)a.splits;
            t.slot = slot;
            t.ma = &mp;
            t.mb = &mw;
            // dz is read once, by the units of all columns of dx side by side.
            t.m0 = (int64_t)(w / dt) * kTileM;
            t.n0 = (int64_t)(w % dt) * TN;
            t.k0 = (int64_t)k0 * kTileK;
            t.kb0 = a.v0 + t.k0;
            t.iters = (int)(k1 - k0);
        } else {
            t.kind = 2;
            const uint32_t w = u - ndx;
            t.ma = &mpt;
            t.mb = &mx;
            t.a_mn = true;
            t.m0 = (int64_t)(w / dt) * kTileM;
            t.n0 = (int64_t)(w % dt) * TN;
            t.iters = (int)((nact + kTileK - 1) / kTileK);
        }
        return t;
    };
    // dweight: the rows whose target is this thread's word, if they are at most kHits; else its place
    // among the words of more.
    const int64_t rank0 = (int64_t)cluster_ctarank() * kCtaM;
    int hits = 0, slot = -1;
    int32_t hit_row[kHits];
    auto prologue = [&](const Unit& t) {
        hits = 0;
        slot = -1;
        if (t.kind != 2) return;
        const int64_t word = a.v0 + t.m0 + rank0 + (threadIdx.x & 127);
        if (word >= a.v1 || !ADALN_IN_LOSS(word < a.V)) return;
        hits = a.word_hits[word];
        if (hits > kHits) {
            slot = a.many.slot[word];
            hits = 0;
        }
        if (hits == 0) return;
        const int4* list = reinterpret_cast<const int4*>(a.word_rows + word * kHits);
        const int4 lo = list[0], hi = list[1];
        const int32_t r[kHits] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
        for (int i = 0; i < kHits; ++i) hit_row[i] = i < hits ? r[i] : INT32_MAX;
    };
    gemm_loop<TN, false>(count, a.status, decode, prologue, [&](const Unit& t, uint32_t src, int r, int half,
                                                            uint32_t out, auto release) {
        const int lane = threadIdx.x & 31;
        const int64_t row = t.m0 + r;
        const int64_t c0 = t.n0;
        const uint32_t mine = out + (uint32_t)lane * 128u;
#pragma unroll 1
        for (int c = 64 * half; c < TN; c += 128) {
            float v[64];
            __syncwarp();
            tmem_ld64(src + c, v);
            if (t.iters == 0) {  // nothing was accumulated
#pragma unroll
                for (int j = 0; j < 64; ++j) v[j] = 0.0f;
            }
            const int64_t col = c0 + c;
            if (t.kind == 1) {
                // A later piece adds in place (one addition a launch to each element, so the order
                // is the pieces').
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    if (lane == 0) tma_store_read();
                    __syncwarp();
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float* f = v + 32 * b + 4 * j;
                        st_swizzled(mine, lane, j, __float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                                    __float_as_uint(f[3]));
                    }
                    fence_shared_async();
                    __syncwarp();
                    if (lane == 0 && row < nact && col + 32 * b < a.D &&
                        ADALN_IN_LOSS(row + 32 <= a.Np && t.slot < a.splits))
                        tma_store(&mdx, (int)col + 32 * b, (int)(t.slot * a.Np + row), out, a.v0 > 0);
                }
            } else {
                const int64_t word = a.v0 + row;
                int32_t last = -1;
                for (int h = 0; h < hits; ++h) {
                    // In row order: the order of the list is that in which the rows came.
                    int32_t i = INT32_MAX;
#pragma unroll
                    for (int k = 0; k < kHits; ++k)
                        if (hit_row[k] > last && hit_row[k] < i) i = hit_row[k];
                    last = i;
                    if (!ADALN_IN_LOSS(i >= 0 && i < nact)) continue;
                    const f2r lo = p_splat(a.row_lo[i]);
                    const uint4* xr = reinterpret_cast<const uint4*>(a.xp) + ((int64_t)i * a.D + col) / 8;
#pragma unroll
                    for (int j = 0; j < 64; j += 8) {
                        if (col + j >= a.D) continue;
                        f2r x[4];
                        Io<__nv_bfloat16>::unpackp(xr[j / 8], x);
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float2 s = p_get(p_fma(lo, x[k], p_make(v[j + 2 * k], v[j + 2 * k + 1])));
                            v[j + 2 * k] = s.x;
                            v[j + 2 * k + 1] = s.y;
                        }
                    }
                }
                // A word of more rows is left to finish_kernel, unrounded.
                if (slot >= 0 && ADALN_IN_LOSS(slot < a.many.slots)) {
                    float4* sum = reinterpret_cast<float4*>(a.many.sums + (int64_t)slot * a.D + col);
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        if (col + 4 * j < a.D) sum[j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
                }
                uint32_t w[32];
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[j]) : "f"(v[2 * j + 1]), "f"(v[2 * j]));
                if (lane == 0) tma_store_read();
                __syncwarp();
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    st_swizzled(mine, lane, j, w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
                fence_shared_async();
                __syncwarp();
                if (lane == 0 && word < a.v1 && col < a.D) tma_store(&mdw, (int)col, (int)word, out, false);
            }
        }
        release();
    });
}

// Joins a row's partial (max, sum exp) in a fixed order: 32 threads a row, each a run of parts
// (its maximum first, then the sums taken to it, so that neither waits for the other's chain),
// then the 32 in a tree. 32 rows a CTA, so that a warp reads 32 rows' parts side by side. 14 us for
// 8192 rows of 394 parts; 11 us for 1023 rows of 1024 (63 us with 8 threads a row).
__global__ void __launch_bounds__(1024) lse_kernel(const LseArgs a) {
    pdl_begin();
    __shared__ float2 red[32][33];
    const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
    const int64_t nact = *a.nact;
    for (int64_t t = blockIdx.x; t * 32 < nact; t += gridDim.x) {
        const int64_t row = t * 32 + lane;
        const int64_t p0 = (int64_t)g * a.nparts / 32, p1 = (int64_t)(g + 1) * a.nparts / 32;
        const int64_t mine = t * 32 + g;  // the row this warp joins below
        const bool own = mine < nact && ADALN_IN_LOSS(mine < a.Np);
        const int64_t r = own ? a.row[mine] : 0;
        const float zt = own ? a.zt[mine] : 0.0f;
        float m = neg_inf(), s = 0.0f;
        if (row < nact && ADALN_IN_LOSS(row < a.Np)) {
            const float2* part = a.parts + row;
#pragma unroll 4
            for (int64_t p = p0; p < p1; ++p) m = fmaxf(m, part[p * a.Np].x);
            const float mm = m == neg_inf() ? 0.0f : m;
#pragma unroll 4
            for (int64_t p = p0; p < p1; ++p) {
                const float2 q = part[p * a.Np];
                s += q.y * exp2_ftz((q.x - mm) * kLog2e);
            }
        }
        red[g][lane] = make_float2(m, s);
        __syncthreads();
        // Warp g joins row g of the 32: every lane a part, the same maximum, sums in a fixed tree.
        const float2 q = red[lane][g];
        m = q.x;
        for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        const float mm = m == neg_inf() ? 0.0f : m;
        s = q.y * exp2_ftz((q.x - mm) * kLog2e);
        for (int o = 16; o >= 1; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
        if (lane == 0 && own && ADALN_IN_LOSS(r >= 0 && r < a.N)) {
            // The loss not as lse - zt: where the target's logit is the maximum (or near it), lse has
            // rounded away what is left of it. As it is here it is never negative.
            const float l = logf(s);
            a.lse[r] = m + l;
            a.loss[r] = (m - zt) + l;
        }
        __syncthreads();
    }
}

// Lists the rows of the words of more than kHits: room for each word's, then the rows.
__global__ void __launch_bounds__(256) list_words_kernel(const FinishArgs a) {
    pdl_begin();
    const int n = *a.many.count, lane = threadIdx.x & 31;
    for (int s0 = blockIdx.x * 256; s0 < n; s0 += gridDim.x * 256) {
        const int s = s0 + threadIdx.x;
        const bool in = s < n && ADALN_IN_LOSS(s < a.many.slots);
        const int hits = in ? a.word_hits[a.many.word[s]] : 0;
        int upto = hits;
        for (int o = 1; o < 32; o *= 2) {
            const int v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
            if (lane >= o) upto += v;
        }
        int at = 0;
        if (lane == 31) at = atomicAdd(a.many.listed, upto);
        at = __shfl_sync(0xFFFFFFFFu, at, 31) + upto - hits;
        if (in) a.many.first[s] = a.many.next[s] = at;
    }
}
__global__ void __launch_bounds__(256) list_rows_kernel(const FinishArgs a) {
    pdl_begin();
    const int64_t nact = *a.nact;
    for (int64_t r = (int64_t)blockIdx.x * 256 + threadIdx.x; r < nact; r += (int64_t)gridDim.x * 256) {
        if (!ADALN_IN_LOSS(r < a.Np)) continue;
        const int32_t word = a.tgt[r];
        if (!ADALN_IN_LOSS(word >= 0 && word < a.V) || a.word_hits[word] <= kHits) continue;
        const int32_t slot = a.many.slot[word];
        if (!ADALN_IN_LOSS(slot >= 0 && slot < a.many.slots)) continue;
        const int at = atomicAdd(a.many.next + slot, 1);
        if (ADALN_IN_LOSS(at >= 0 && at < a.Np)) a.many.rows[at] = (int32_t)r;
    }
}

// dweight of the words of more than kHits rows: what the products left, and the remainders of all their
// rows' targets. A CTA takes a word and some columns at a time: it puts the word's rows in order, from
// the targets of kListRows rows at a time or from the word's list, and adds them up in groups of threads, every group a fixed
// share of the list; then the groups' sums in their order. The more such words, the more columns at a
// time (64 columns are 32 groups of 8 threads): as few as leave no CTA a second word, so that a few words
// of many rows are shared out and many words are listed once or twice. What it adds to a backward, without
// such words and with them: nothing at 96 x 8192 x 1024 (30.2 us), 29.7 -> 33.4 us at 4096 x 24 x 256,
// 96 -> 108 us at 8192 x 1000 x 1024, 48 -> 64 us at 8192 x 2 x 512.
__device__ __forceinline__ void add_remainders(const FinishArgs& a, int64_t nact) {
    __shared__ __align__(16) uint16_t list[kListRows];
    __shared__ int totals[8][8];
    __shared__ __align__(16) float red[2048];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // Thread tid looks at rows r0 + 1024 j + 4 tid ..; without lists before anything else is known.
    int4 t[8];
    auto targets = [&](int64_t r0) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int64_t row = r0 + 1024 * j + 4 * tid;
            t[j] = make_int4(-1, -1, -1, -1);
            if (row < nact && ADALN_IN_LOSS(row + 4 <= a.Np)) t[j] = *reinterpret_cast<const int4*>(a.tgt + row);
        }
    };
    if (!a.many.listed) targets(0);
    const int64_t n = *a.many.count;
    int lanes = 8;  // threads a group
    while (lanes < 256 && 8 * lanes < a.D && n * ((a.D + 8 * lanes - 1) / (8 * lanes)) > a.many_ctas) lanes *= 2;
    const int groups = 256 / lanes, group = tid / lanes, cols = 8 * lanes;
    const int64_t chunks = (a.D + cols - 1) / cols;
    for (int64_t u = blockIdx.x; u < n * chunks; u += a.many_ctas) {
        const int64_t slot = u / chunks, col = u % chunks * cols + tid % lanes * 8;
        if (!ADALN_IN_LOSS(slot < a.many.slots)) break;
        const int32_t word = a.many.word[slot];
        const char* x = reinterpret_cast<const char*>(a.xp) + col * 2;
        f2r s[4] = {kPairZero, kPairZero, kPairZero, kPairZero};
        auto add = [&](int count, auto row_of) {
            for (int k = group; k < count; k += 8 * groups) {  // eight loads on their way
                uint4 q[8];
                float lo[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    q[j] = make_uint4(0, 0, 0, 0);
                    lo[j] = 0.0f;
                    if (k + j * groups < count) {
                        const int64_t row = row_of(k + j * groups);
                        if (!ADALN_IN_LOSS(row >= 0 && row < nact)) continue;
                        lo[j] = a.row_lo[row];
                        if (col < a.D) q[j] = ld_keep(x + row * a.D * 2);
                    }
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    f2r v[4];
                    Io<__nv_bfloat16>::unpackp(q[j], v);
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[e] = p_fma(p_splat(lo[j]), v[e], s[e]);
                }
            }
            __syncthreads();  // the list has been read
        };
        const int hits = a.many.listed && ADALN_IN_LOSS(word >= 0 && word < a.V) ? a.word_hits[word] : INT32_MAX;
        if (hits <= kSortRows) {
            // In order: a row's place is the number of rows before it.
            int* unsorted = reinterpret_cast<int*>(list);
            int* sorted = unsorted + kSortRows;
            const int64_t first = a.many.first[slot];
            for (int k = tid; k < hits; k += 256)
                unsorted[k] = ADALN_IN_LOSS(first + k < a.Np) ? a.many.rows[first + k] : 0;
            __syncthreads();
            for (int k = tid; k < hits; k += 256) {
                const int row = unsorted[k];
                int place = 0;
                for (int i = 0; i < hits; ++i) place += unsorted[i] < row;
                sorted[place] = row;
            }
            __syncthreads();
            add(hits, [&](int k) { return (int64_t)sorted[k]; });
        }
        for (int64_t r0 = 0; hits > kSortRows && r0 < nact; r0 += kListRows) {
            if (a.many.listed) targets(r0);  // else all of them are in one look
            uint32_t on[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int64_t row = r0 + 1024 * j + 4 * tid;
                on[j] = (t[j].x == word) | (t[j].y == word && row + 1 < nact) << 1 |
                        (t[j].z == word && row + 2 < nact) << 2 | (t[j].w == word && row + 3 < nact) << 3;
            }
            int before[8];  // of the warp's rows of this j
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                int all = 0;
                before[j] = 0;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const uint32_t b = __ballot_sync(0xFFFFFFFFu, on[j] >> c & 1u);
                    before[j] += __popc(b & ((1u << lane) - 1u));
                    all += __popc(b);
                }
                if (lane == 0) totals[j][warp] = all;
            }
            __syncthreads();
            int count = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
#pragma unroll
                for (int w = 0; w < 8; ++w) {
                    before[j] += w < warp ? totals[j][w] : 0;
                }
                before[j] += count;
#pragma unroll
                for (int w = 0; w < 8; ++w) count += totals[j][w];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    if (on[j] >> c & 1u) list[before[j]++] = (uint16_t)(1024 * j + 4 * tid + c);
                }
            }
            __syncthreads();
            add(count, [&](int k) { return r0 + list[k]; });
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) *reinterpret_cast<float2*>(red + 8 * tid + 2 * e) = p_get(s[e]);
        __syncthreads();
        for (int c = tid; c < cols; c += 256) {
            const int64_t out = u % chunks * cols + c;
            if (out >= a.D || !ADALN_IN_LOSS(word >= 0 && word < a.V)) break;
            float sum = a.many.sums[slot * a.D + out];
            for (int g = 0; g < groups; ++g) sum += red[g * cols + c];
            a.dweight[word * a.D + out] = __float2bfloat16_rn(sum);
        }
        __syncthreads();
    }
}

// dx of the packed rows: the parts added in order, then what rounding dz of the target left off,
// rounded once, back to the rows' places. 32 us for 8192 rows of 2048 (4.2 TB/s). MANY: the first
// a.many_ctas CTAs have dweight of the words of more than kHits rows instead.
template <bool MANY>
__global__ void __launch_bounds__(256, MANY ? 2 : 3) finish_kernel(const FinishArgs a) {
    pdl_begin();
    const int64_t nact = *a.nact, vecs = a.D / 8;
    if constexpr (MANY) {
        if ((int)blockIdx.x < a.many_ctas) {
            add_remainders(a, nact);
            return;
        }
    }
    const int many = MANY ? a.many_ctas : 0;
    const int64_t block = (int64_t)blockIdx.x - many, step = (int64_t)(gridDim.x - many) * 256;
    for (int64_t i = block * 256 + threadIdx.x; i < nact * vecs; i += step) {
        const int64_t p = i / vecs, v = i % vecs;
        if (!ADALN_IN_LOSS(p < a.Np)) continue;
        const int64_t r = a.row[p];
        const float rest = a.row_lo[p];
        const uint4 word = ld_keep(reinterpret_cast<const uint4*>(a.weight) + a.tgt[p] * vecs + v);
        float s[8] = {};
        for (int k = 0; k < a.splits; ++k) {
            const float4* src = reinterpret_cast<const float4*>(a.dxacc + ((int64_t)k * a.Np + p) * a.D + v * 8);
            const float4 lo = src[0], hi = src[1];
            s[0] += lo.x; s[1] += lo.y; s[2] += lo.z; s[3] += lo.w;
            s[4] += hi.x; s[5] += hi.y; s[6] += hi.z; s[7] += hi.w;
        }
        f2r t[4];
        Io<__nv_bfloat16>::unpackp(word, t);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 f = p_get(t[j]);
            s[2 * j] = fmaf(rest, f.x, s[2 * j]);
            s[2 * j + 1] = fmaf(rest, f.y, s[2 * j + 1]);
        }
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[j]) : "f"(s[2 * j + 1]), "f"(s[2 * j]));
        if (ADALN_IN_LOSS(r >= 0 && r < a.N))
            reinterpret_cast<uint4*>(a.dx)[r * vecs + v] = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// ---- launches ------------------------------------------------------------------------------
namespace {

unsigned cap(int64_t want, int64_t most) { return (unsigned)(want < 1 ? 1 : want < most ? want : most); }

// Lets kernel variant `which` use its shared memory, once a device.
cudaError_t allow_gemm_smem(const void* fn, int which) {
    constexpr int kDevices = 64;
    static std::atomic<bool> done[kDevices][6];
    int dev = 0;
    if (cudaError_t e = cudaGetDevice(&dev)) return e;
    if (dev >= 0 && dev < kDevices && done[dev][which].load(std::memory_order_acquire)) return cudaSuccess;
    cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kGemmSmem);
    if (e == cudaSuccess && dev >= 0 && dev < kDevices) done[dev][which].store(true, std::memory_order_release);
    return e;
}

// Tiled tensor map of a row-major bf16 (or fp32) [rows, cols] matrix (row stride ld elements),
// boxes of 128 bytes of a row by `box_rows` rows, 128-byte swizzle.
bool tile_map(CUtensorMap* m, const void* base, int64_t rows, int64_t cols, int64_t ld, int box_rows,
              bool f32 = false) {
    using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static const Encode encode = [] {
        void* fn = nullptr;
        cudaDriverEntryPointQueryResult res;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &res) !=
                cudaSuccess ||
            res != cudaDriverEntryPointSuccess)
            fn = nullptr;
        return reinterpret_cast<Encode>(fn);
    }();
    if (!encode) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)ld * (f32 ? 4 : 2)};
    const cuuint32_t box[2] = {f32 ? 32u : 64u, (cuuint32_t)box_rows}, one[2] = {1, 1};
    return encode(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, one,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

cudaError_t launch_pack(const PackArgs& args, int ctas, cudaStream_t stream) {
    PackArgs a = args;
    void* params[] = {&a};
    return launch_dependent(reinterpret_cast<const void*>(&pack_kernel), dim3((unsigned)ctas), dim3(kPackThreads),
                            params, 0, stream);
}

cudaError_t launch_logits(const LogitsArgs& args, bool probs, const void* xp, const void* weight, int sms,
                          cudaStream_t stream) {
    LogitsArgs a = args;
    CUtensorMap mx, mw, mp{};
    if (!tile_map(&mx, xp, a.Np, a.D, a.D, kCtaM) || !tile_map(&mw, weight, a.V, a.D, a.D, a.tn / 2) ||
        (probs && !tile_map(&mp, a.probs, a.Np, a.ldp, a.ldp, 32)))
        return cudaErrorInvalidValue;
    const void* fn = a.tn == kTileN ? (probs ? reinterpret_cast<const void*>(&logits_kernel<true, kTileN>)
                                             : reinterpret_cast<const void*>(&logits_kernel<false, kTileN>))
                                    : (probs ? reinterpret_cast<const void*>(&logits_kernel<true, kTileN / 2>)
                                             : reinterpret_cast<const void*>(&logits_kernel<false, kTileN / 2>));
    if (cudaError_t e = allow_gemm_smem(fn, (a.tn == kTileN ? 0 : 1) + (probs ? 2 : 0))) return e;
    const int64_t units = (a.Np / kTileM) * ((a.v1 - a.v0 + a.tn - 1) / a.tn);
    void* params[] = {&mx, &mw, &mp, &a};
    return launch_dependent(fn, dim3(2 * cap(units, sms / 2)), dim3(kGemmThreads), params, kGemmSmem, stream, 2);
}

cudaError_t launch_grad(const GradArgs& args, const void* probs, int64_t ldp, const void* xp, const void* weight,
                        int sms, cudaStream_t stream) {
    GradArgs a = args;
    CUtensorMap mp, mw, mx, mpt, mdx{}, mdw{};
    if (!tile_map(&mp, probs, a.Np, ldp, ldp, kCtaM) || !tile_map(&mw, weight, a.V, a.D, a.D, kTileK) ||
        !tile_map(&mx, xp, a.Np, a.D, a.D, kTileK) || !tile_map(&mpt, probs, a.Np, ldp, ldp, kTileK) ||
        (a.dxacc && !tile_map(&mdx, a.dxacc, a.splits * a.Np, a.D, a.D, 32, true)) ||
        (a.dweight && !tile_map(&mdw, a.dweight, a.V, a.D, a.D, 32)))
        return cudaErrorInvalidValue;
    const void* fn = a.tn == kTileN ? reinterpret_cast<const void*>(&grad_kernel<kTileN>)
                                    : reinterpret_cast<const void*>(&grad_kernel<kTileN / 2>);
    if (cudaError_t e = allow_gemm_smem(fn, a.tn == kTileN ? 4 : 5)) return e;
    const int64_t dt = (a.D + a.tn - 1) / a.tn;
    const int64_t units = (a.dxacc ? a.Np / kTileM * dt * a.splits : 0) +
                          (a.dweight ? (a.v1 - a.v0 + kTileM - 1) / kTileM * dt : 0);
    void* params[] = {&mp, &mw, &mx, &mpt, &mdx, &mdw, &a};
    return launch_dependent(fn, dim3(2 * cap(units, sms / 2)), dim3(kGemmThreads), params, kGemmSmem, stream, 2);
}

cudaError_t launch_lse(const LseArgs& args, int sms, cudaStream_t stream) {
    LseArgs a = args;
    void* params[] = {&a};
    return launch_dependent(reinterpret_cast<const void*>(&lse_kernel), dim3(cap(a.Np / 32, 2 * (int64_t)sms)),
                            dim3(1024), params, 0, stream);
}

cudaError_t launch_lists(const FinishArgs& args, int sms, cudaStream_t stream) {
    FinishArgs a = args;
    void* params[] = {&a};
    const unsigned words = cap((a.many.slots + 255) / 256, 4 * (int64_t)sms), rows = cap(a.Np / 256, 8 * (int64_t)sms);
    if (cudaError_t e = launch_dependent(reinterpret_cast<const void*>(&list_words_kernel), dim3(words), dim3(256), params,
                                         0, stream))
        return e;
    return launch_dependent(reinterpret_cast<const void*>(&list_rows_kernel), dim3(rows), dim3(256), params, 0, stream);
}

cudaError_t launch_finish(const FinishArgs& args, int sms, cudaStream_t stream) {
    FinishArgs a = args;
    void* params[] = {&a};
    const bool many = a.dweight != nullptr;
    // One of the two CTAs that an SM holds; the other is left to dx (both: the same time; the last CTAs
    // instead of the first: 119 us against 108 at 8192 x 1000 x 1024).
    a.many_ctas = many ? (int)cap(a.many.slots * ((a.D + 63) / 64), (int64_t)sms) : 0;
    const unsigned dx_ctas = a.dx ? cap((a.Np * (a.D / 8) + 255) / 256, 8 * (int64_t)sms) : 0;
    const void* fn = many ? reinterpret_cast<const void*>(&finish_kernel<true>)
                          : reinterpret_cast<const void*>(&finish_kernel<false>);
    return launch_dependent(fn, dim3(a.many_ctas + dx_ctas), dim3(256), params, 0, stream);
}

cudaError_t debug_word_xent(uint32_t* out, bool reset) { return debug_word(out, reset); }

}  // namespace adaln
