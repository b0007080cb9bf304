// Softmax attention over packed sequences, with its gradient; the scores are never kept.
//
//     z = scale q k^T (masked),  lse = log sum_j exp(z_j),  p = exp(z - lse),  o = p v
//     dv = p^T dout,  dp = dout v^T,  dz = p (dp - delta),  delta = dout . o
//     dq = scale dz k,  dk = scale dz^T q
//
// attn_plan lists the tiles of rows of all segments and cuts them, with the heads, into equal shares;
// persistent CTAs, one an SM, walk theirs. Every product is a tcgen05.mma of 128 rows with its accumulator in
// tensor memory, its operands brought by TMA; p and dz (bf16, the products' types) are written back to
// tensor memory over the scores that they come from and are operands from there, so that they never pass
// through shared memory.
//
//   attn_fwd_kernel: two tiles of 128 queries share the keys and values in shared memory; a
//       warpgroup each has a thread a row, so that the softmax needs no exchange between threads. The
//       two alternate: while one computes exponentials, the tensor cores run the other's products.
//   attn_dq: a tile of 128 queries over its keys: z, dp, dq += dz k.
//   attn_dkv: a tile of 128 keys over its queries, transposed: z^T, dp^T, dv += p^T dout,
//       dk += dz^T q, over all heads that share the keys.
//
// dq and dk, dv are CTAs of their own that both compute z and dp (7 products where one would need 5): each
// sum then stays in tensor memory in a fixed order, without atomics and without an fp32 dq in memory.
//
// Sums, maxima, exponentials and lse are fp32. Rounded to bf16 as operands: p (half a step, 2^-8 of
// each value) and dz. delta is taken from the caller's bf16 o, of rows of few keys from the scores.
//
// Bound by the tensor cores from some thousand rows on: 32760 rows, 12 heads of 128, 4.2 ms forward (1.55
// PFLOP/s, the tensor pipe 72% active; a step of 128 keys and 256 queries takes 2,800 cycles, its products 2,048).
// 16384 rows 1.0 ms forward (1.6 PFLOP/s) and 3.4-3.6 ms backward (1.13-1.2 PFLOP/s, 1.6-1.7 with the second z
// and dp; 75% active: operands and incoming tiles take all that shared memory gives), causal 0.54 and 1.8 ms. Short
// segments by the units' beginnings and ends, the smallest calls by the chain of launches (153 rows: 11 + 20 us).
// Times of one direction are of replayed graphs of 20 equal calls; a pass with changing inputs takes 2-5% more
// than their sum (16384: 4.6-4.7 ms).
#include <algorithm>
#include <atomic>

#include "attn.h"
#include "tensor.cuh"

namespace adaln {

#define ADALN_IN_ATTN(cond) ADALN_IN(::adaln::kDbgAttn, cond)

constexpr int kAttnThreads = 384;  // two warpgroups of rows, one warp of products, one of loads
constexpr int kMmaWarp = 8, kLoadWarp = 9, kAllocWarp = 10;
constexpr uint32_t kPanel = kAttnTile * 128;  // 128 rows of 64 elements, 128-byte swizzle

// Shared memory: two resident tiles, a ring of tiles, and in the forward 4 KB a warp for its results on
// their way out.
enum AttnKernel : int { kAttnFwd = 0, kAttnDq = 1, kAttnDkv = 2 };
constexpr uint32_t kAttnOut = 32 * 128;  // 32 rows of 64 elements
template <int DP, int KIND>
struct AttnShape {
    static constexpr uint32_t kTile = DP / 64 * kPanel;
    static constexpr int kStages = DP == 128 ? (KIND == kAttnFwd ? 4 : 5) : 8;
    static constexpr uint32_t kTiles = (2 + kStages) * kTile;
    // The gradients keep nothing in static shared memory: the dynamic memory then begins on a 1024-byte
    // boundary, without which the fifth stage would not fit. Behind the tiles: results on their way out (of
    // wide heads they fit the second resident tile), barriers and two words, for dk and dv the row statistics.
    static constexpr uint32_t kOut = DP == 64 ? 8 * kAttnOut : 0, kBars = kTiles + kOut;
    static constexpr size_t kSmem = KIND == kAttnFwd ? 1024 + kTiles + 8 * kAttnOut : kBars + 320 + 2048;
};

// ---- work list -----------------------------------------------------------------------------
__device__ __forceinline__ int64_t attn_start(const int32_t* cu, int64_t s, int64_t nseg, int64_t R) {
    if (!ADALN_IN_ATTN(s >= 0 && s <= nseg)) return 0;
    return cu ? (int64_t)__ldg(cu + s) : s * (R / nseg);
}

// A segment's rows on both sides.
struct AttnSegment {
    int q0, nq, k0, nk;
};
__device__ __forceinline__ int floor_div(int a, int b) { return a >= 0 ? a / b : -((b - 1 - a) / b); }

// Entry `at / tile` of a list's segment.
__device__ __forceinline__ AttnItem attn_entry(const AttnTables& t, const AttnList& l, int list, const AttnSegment& g,
                                               int at) {
    AttnItem it{};
    const int len = list ? g.nk : g.nq;
    it.rows = min(l.tile, len - at);
    it.row0 = (list ? g.k0 : g.q0) + at;
    it.other0 = list ? g.q0 : g.k0;
    it.others = list ? g.nq : g.nk;
    it.end = it.other0 + it.others == (int)(list ? t.Rq : t.Rk);
    if (list == 0)
        it.shift = t.causal ? at + g.nk - g.nq : g.nk;
    else
        it.shift = t.causal ? at - g.nk + g.nq : -kAttnTile;
    it.unseen = list && t.causal ? max(0, g.nq - g.nk) : 0;
    return it;
}

// Cost of a segment's first `tiles` entries: their steps (as the kernels count them from the entry) and
// l.unit_cost each, summed in closed form.
__device__ __forceinline__ int64_t attn_cost(const AttnTables& t, const AttnList& l, int list, const AttnSegment& g,
                                             int tiles) {
    const int len = list ? g.nk : g.nq, other = list ? g.nq : g.nk;
    const int64_t steps = (other + kAttnTile - 1) / kAttnTile;
    int64_t sum = 0;
    if (!t.causal) {
        sum = steps * tiles;
    } else if (list == 0) {
        // A full entry's last query, (i + 1) k tiles of 128 on, sees a + (i + 1) k tiles of keys; the last
        // entry, full or not, sees all keys.
        const int k = l.tile / kAttnTile /* 1 or 2 */, a = -floor_div(g.nq - g.nk, kAttnTile);
        const int64_t full = min(tiles, len / l.tile), none = a + k > 0 ? 0 : min((int64_t)(-a >> (k - 1)), full);
        sum = (full - none) * a + k * (full * (full + 1) - none * (none + 1)) / 2;
        if (tiles > full) sum += steps;
    } else {
        // Entry i is seen by the tiles of queries from max(0, b + i) on.
        const int64_t b = floor_div(g.nq - g.nk, kAttnTile), n = tiles;
        const int64_t whole = min(max(1 - b, (int64_t)0), n), end = min(n, max(whole, steps - b));
        sum = whole * steps + (end - whole) * (steps - b) - (end * (end - 1) - whole * (whole - 1)) / 2;
    }
    return sum * l.group + (int64_t)l.unit_cost * tiles;
}

__device__ __forceinline__ int64_t warp_before(int64_t v, int lane, int64_t* total) {
    int64_t s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xFFFFFFFFu, s, o);
        if (lane >= o) s += x;
    }
    *total = __shfl_sync(0xFFFFFFFFu, s, 31);
    return s - v;
}

constexpr int kPlanThreads = 512;
constexpr int kAttnFewSegs = 1024;  // kept in shared memory while they are planned

// One CTA a list. The entries are in the order of the rows: entries and cost of every segment, sums over
// those before it, then the entries and where each CTA begins. Everything follows
// from the tables alone, so that pieces, and with them the order of sums, are the same every time.
__device__ __forceinline__ void attn_plan(const AttnPlanArgs& a, int list) {
    constexpr int NW = kPlanThreads / 32;
    __shared__ int64_t sums[2][NW];
    __shared__ longlong2 few[kAttnFewSegs];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const AttnTables& t = a.t;
    const AttnList& l = a.list[list];
    longlong2* segs = t.nseg <= kAttnFewSegs ? few : l.segs;
    auto segment = [&](int64_t s, bool* bad) {
        const int64_t q0 = attn_start(t.cu_q, s, t.nseg, t.Rq), q1 = attn_start(t.cu_q, s + 1, t.nseg, t.Rq);
        const int64_t k0 = attn_start(t.cu_k, s, t.nseg, t.Rk), k1 = attn_start(t.cu_k, s + 1, t.nseg, t.Rk);
        *bad |= q0 < 0 || q1 < q0 || q1 > t.Rq || k0 < 0 || k1 < k0 || k1 > t.Rk;
        *bad |= (s == 0 && (q0 != 0 || k0 != 0)) || (s == t.nseg - 1 && (q1 != t.Rq || k1 != t.Rk));
        return AttnSegment{(int)q0, (int)(q1 - q0), (int)k0, (int)(k1 - k0)};
    };
    auto tiles_of = [&](const AttnSegment& g) { return ((list ? g.nk : g.nq) + l.tile - 1) / l.tile; };
    bool any_bad = t.nseg == 0 && (t.Rq != 0 || t.Rk != 0);
    int64_t run[2] = {0, 0};  // entries and cost so far
    for (int64_t base = 0; base < t.nseg && !any_bad; base += kPlanThreads) {
        const int64_t s = base + tid;
        bool bad = false;
        int64_t v[2] = {0, 0}, all[2];
        if (s < t.nseg) {
            const AttnSegment g = segment(s, &bad);
            if (!bad) {
                v[0] = tiles_of(g);
                v[1] = attn_cost(t, l, list, g, (int)v[0]);
            }
        }
        int64_t before[2] = {warp_before(v[0], lane, &all[0]), warp_before(v[1], lane, &all[1])};
        if (lane == 0) {
            sums[0][warp] = all[0];
            sums[1][warp] = all[1];
        }
        any_bad = __syncthreads_or(bad);
        const int warps = (int)min((int64_t)NW, (t.nseg - base + 31) / 32);  // that have segments
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            before[x] += run[x];
            for (int w = 0; w < warps; ++w) {
                const int64_t n = sums[x][w];
                before[x] += w < warp ? n : 0;
                run[x] += n;
            }
        }
        if (s < t.nseg) segs[s] = make_longlong2(before[0], before[1]);
        __syncthreads();
    }
    if (tid == 0 && list == 0) {
        a.status[0] = any_bad ? kErrSeqlens : 0u;
        a.status[1] = 0u;  // the kernels' word
        a.header->magic = kStatusMagic;
        a.header->nwords = 2;
    }
    if (l.items == nullptr) return;
    const int64_t count = any_bad ? 0 : min(run[0], l.most), total = any_bad ? 0 : run[1];
    if (tid == 0) *l.count = (int32_t)count;
    // CTA c begins at cost c / ctas of all heads' together.
    const int64_t every = total * l.heads;
    for (int c = tid; c <= l.ctas; c += kPlanThreads) {
        AttnCursor cur{(int32_t)(count * l.heads), 0};
        if (c < l.ctas && total > 0) {
            const int64_t x = every / l.ctas * c + every % l.ctas * c / l.ctas;
            const int64_t head = x / total, in = x - head * total;
            int64_t lo = 0, hi = t.nseg - 1;  // the last segment that begins at or before `in`
            while (lo < hi) {
                const int64_t mid = (lo + hi + 1) >> 1;
                if (segs[mid].y <= in) lo = mid;
                else hi = mid - 1;
            }
            bool bad = false;
            const AttnSegment g = segment(lo, &bad);
            const int64_t rest = in - segs[lo].y;
            int first = 0, last = tiles_of(g) - 1;  // and its last entry that does
            while (first < last) {
                const int mid = (first + last + 1) >> 1;
                if (attn_cost(t, l, list, g, mid) <= rest) first = mid;
                else last = mid - 1;
            }
            const int64_t begin = attn_cost(t, l, list, g, first);
            const int n = (int)(attn_cost(t, l, list, g, first + 1) - begin) - l.unit_cost;
            int tile = (int)(rest - begin) - l.unit_cost / 2;
            cur.unit = (int32_t)(head * count + segs[lo].x + first);
            if (tile < kAttnMinPiece) tile = 0;
            if (tile > 0 && n - tile < kAttnMinPiece) {
                tile = 0;
                ++cur.unit;
            }
            cur.tile = tile;
        }
        l.cursors[c] = cur;
    }
    // A thread an entry, the last ones first: the first threads have the cursors.
    for (int64_t i = kPlanThreads - 1 - tid; i < count; i += kPlanThreads) {
        int64_t lo = 0, hi = t.nseg - 1;  // the last segment that begins at or before the entry
        while (lo < hi) {
            const int64_t mid = (lo + hi + 1) >> 1;
            if (segs[mid].x <= i) lo = mid;
            else hi = mid - 1;
        }
        bool bad = false;
        const AttnSegment g = segment(lo, &bad);
        if (ADALN_IN_ATTN(i < l.most)) l.items[i] = attn_entry(t, l, list, g, (int)(i - segs[lo].x) * l.tile);
    }
}

// What row r of the queries sees: `seen` keys from k0 on, of segment s; -1 where the tables say nothing usable (they
// are reported, and nothing is computed).
struct AttnSeen {
    int s, k0, seen;
    __device__ __forceinline__ bool few() const { return seen > 0 && seen <= kAttnFewKeys; }
};
__device__ __forceinline__ AttnSeen attn_seen(const AttnTables& t, int64_t s, int64_t r) {
    const int64_t q0 = attn_start(t.cu_q, s, t.nseg, t.Rq), q1 = attn_start(t.cu_q, s + 1, t.nseg, t.Rq);
    const int64_t k0 = attn_start(t.cu_k, s, t.nseg, t.Rk), k1 = attn_start(t.cu_k, s + 1, t.nseg, t.Rk);
    if (r < q0 || r >= q1 || k0 < 0 || k1 < k0 || k1 > t.Rk) return AttnSeen{(int)s, 0, -1};
    const int64_t seen = t.causal ? min(k1 - k0, r + 1 - q1 + k1 - k0) : k1 - k0;
    return AttnSeen{(int)s, (int)k0, (int)max(seen, (int64_t)0)};
}
__device__ __forceinline__ AttnSeen attn_seen(const AttnTables& t, int64_t r) {
    int64_t lo = 0, hi = t.nseg - 1;  // the last segment that begins at or before r
    while (lo < hi) {
        const int64_t mid = (lo + hi + 1) >> 1;
        if (attn_start(t.cu_q, mid, t.nseg, t.Rq) <= r) lo = mid;
        else hi = mid - 1;
    }
    return attn_seen(t, lo, r);
}

// delta = dout . o of every row and head, and lse in units of log 2: 16 lanes a head, a warp two heads of a row,
// four such pairs on their way. FEW: there may be rows of few keys, whose delta is attn_delta_few's.
template <bool FEW>
__device__ __forceinline__ void attn_delta(const AttnTables& t, const AttnDeltaArgs& a, int64_t block, int64_t blocks) {
    constexpr int U = 4, NW = kPlanThreads / 32;
    const int lane = threadIdx.x & 15, group = threadIdx.x >> 4 & 1, vecs = a.d / 8, pairs = (a.Hq + 1) / 2;
    const int64_t first = block * NW + (threadIdx.x >> 5), step = blocks * NW;
    // The warp's next pair, and what a step adds to it.
    int64_t r = first / pairs;
    int at = (int)(first % pairs);
    const int64_t dr = step / pairs;
    const int da = (int)(step % pairs);
    uint32_t few = 0;  // of the warp's next 32 pairs, those whose row is attn_delta_few's
    for (int n = 0; r < a.Rq; n += U) {
        uint4 x[U], y[U];
        float lse[U], v[U];
        int64_t rows[U];
        int heads[U];
        const int64_t pair = r * pairs + at;
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const int h = heads[j] = 2 * at + group;
            rows[j] = r;
            x[j] = y[j] = make_uint4(0, 0, 0, 0);
            lse[j] = 0.0f;
            if (r < a.Rq && h < a.Hq && lane < vecs && ADALN_IN_ATTN(r >= 0)) {
                const int64_t off = (int64_t)h * a.d + 8 * lane;
                x[j] = ld_stream(reinterpret_cast<const __nv_bfloat16*>(a.dout) + r * a.do_ld + off);
                // (o and lse are of a kernel that may be close ahead: from L2.)
                y[j] = __ldcg(reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(a.o) + r * a.o_ld + off));
                if (lane == 0) lse[j] = __ldcg(a.lse + (int64_t)h * a.Rq + r);
            }
            r += dr;
            at += da;
            if (at >= pairs) {
                at -= pairs;
                ++r;
            }
        }
#pragma unroll
        for (int j = 0; j < U; ++j) {
            f2r p[4], q[4], sum = kPairZero;
            Io<__nv_bfloat16>::unpackp(x[j], p);
            Io<__nv_bfloat16>::unpackp(y[j], q);
#pragma unroll
            for (int e = 0; e < 4; ++e) sum = p_fma(p[e], q[e], sum);
            v[j] = p_hsum(sum);
#pragma unroll
            for (int o = 8; o >= 1; o >>= 1) v[j] += __shfl_xor_sync(0xFFFFFFFFu, v[j], o);
        }
        if (FEW) few >>= U;
        if (FEW && n % 32 == 0) {  // a lane a pair, behind the loads
            const int64_t row = (pair + (threadIdx.x & 31) * step) / pairs;
            few = __ballot_sync(0xFFFFFFFFu, row < a.Rq && attn_seen(t, row).few());
        }
#pragma unroll
        for (int j = 0; j < U; ++j) {
            if (lane == 0 && rows[j] < a.Rq && heads[j] < a.Hq && ADALN_IN_ATTN(rows[j] >= 0)) {
                if (!FEW || !(few >> j & 1)) a.delta[(int64_t)heads[j] * a.Rq + rows[j]] = v[j];
                a.lse2[(int64_t)heads[j] * a.Rq + rows[j]] = lse[j] * kLog2e;
            }
        }
    }
}

__device__ __forceinline__ void mma_m16n8k16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                             uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// delta of rows that see at most kAttnFewKeys keys, from its definition: sum p dp. delta = dout . o has the rounding of
// the caller's bf16 o, and of p in it: little beside what a row of many keys sums, but with few keys dp - delta is
// a difference of near values. In the 2-norm, where one rounding is 0.0017, dq of rows over 2, 3, 8, 17, 33 keys was
// off by 0.0048, 0.0040, 0.0032, 0.0029, 0.0028 (three rows of three: 0.0060) and now 0.0024 up to 32, 0.0030 at
// worst. Backward of 153 causal rows 17.2 -> 19.9 us, causal 15927 x 16 x 64 679 -> 684, 200 causal segments of 200
// 364 -> 392, 1000 of 30 688 -> 762, 32760 rows over 16 keys 179 -> 276 (12 heads of 128); rows of 64 keys too:
// 23 us for the 153 rows and 440 for the 200 segments. Calls without such rows as before.
//
// A warp takes 16 rows and a head (tcgen05's tiles of 128 rows would be mostly empty), the keys of one segment after
// another's, 16 at a time. The sum over a head's elements may go in any order: lane t of four holds elements
// 8 t .. 8 t + 7 of every 32, one 16-byte load, as two steps of the product.
__device__ __forceinline__ void attn_delta_few(const AttnTables& t, const AttnDeltaArgs& a, int64_t block, int64_t blocks) {
    constexpr int NW = kPlanThreads / 32, NT = 2;  // tiles of 8 keys at once
    using T = __nv_bfloat16;
    const int lane = threadIdx.x & 31, g = lane >> 2, q4 = lane & 3;
    // Causal: the first rows of every segment that see a key. Else all groups of 16 rows are looked at.
    const int64_t units = (t.causal ? t.nseg * kAttnFewBlocks : (a.Rq + 15) / 16) * a.Hq;
    const float sl2 = a.scale * kLog2e;
    auto load = [&](const void* p, int64_t ld, int64_t row, bool in, int head, int e) {
        return in && e < a.d ? *reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(p) + row * ld + (int64_t)head * a.d + e)
                             : make_uint4(0, 0, 0, 0);
    };
    for (int64_t u = block * NW + (threadIdx.x >> 5); u < units; u += blocks * NW) {
        const int h = (int)(u % a.Hq), kv = h / a.group;
        int64_t r0 = u / a.Hq * 16;
        AttnSeen own{-1, 0, -1};  // lanes 0 .. 15: a row each
        if (t.causal) {
            const int64_t s = u / a.Hq / kAttnFewBlocks;
            const int64_t q0 = attn_start(t.cu_q, s, t.nseg, t.Rq), q1 = attn_start(t.cu_q, s + 1, t.nseg, t.Rq);
            const int64_t nk = attn_start(t.cu_k, s + 1, t.nseg, t.Rk) - attn_start(t.cu_k, s, t.nseg, t.Rk);
            if (q0 < 0 || q1 > a.Rq) continue;
            r0 = max(q0, q1 - nk) + 16 * (u / a.Hq % kAttnFewBlocks);
            if (lane < 16) own = attn_seen(t, s, r0 + lane);
        } else if (lane < 16 && r0 + lane < a.Rq) {
            own = attn_seen(t, r0 + lane);
        }
        uint32_t left = __ballot_sync(0xFFFFFFFFu, own.few());
        if (left == 0) continue;
        // This lane's two rows: as the products have them.
        const int64_t ra = r0 + g, rb = ra + 8;
        const bool ina = ra < a.Rq && ADALN_IN_ATTN(ra >= 0 && h < a.Hq), inb = rb < a.Rq && ADALN_IN_ATTN(rb >= 0);
        const float la = ina ? __ldcg(a.lse + (int64_t)h * a.Rq + ra) * kLog2e : 0.0f;
        const float lb = inb ? __ldcg(a.lse + (int64_t)h * a.Rq + rb) * kLog2e : 0.0f;
        const int sa = __shfl_sync(0xFFFFFFFFu, own.seen, g), sb = __shfl_sync(0xFFFFFFFFu, own.seen, g + 8);
        while (left) {
            const int lead = 31 - __clz(left);  // a segment's last row here sees most
            const int s = __shfl_sync(0xFFFFFFFFu, own.s, lead), k0 = __shfl_sync(0xFFFFFFFFu, own.k0, lead);
            const int keys = __shfl_sync(0xFFFFFFFFu, own.seen, lead);
            const uint32_t mine = left & __ballot_sync(0xFFFFFFFFu, own.s == s);
            left &= ~mine;
            float va = 0.0f, vb = 0.0f;
            for (int j0 = 0; j0 < keys; j0 += 8 * NT) {
                float z[NT][4] = {}, dp[NT][4] = {};
#pragma unroll 1
                for (int e = 8 * q4; e - 8 * q4 < a.d; e += 32) {
                    const uint4 xa = load(a.q, a.q_ld, ra, ina, h, e), xb = load(a.q, a.q_ld, rb, inb, h, e);
                    const uint4 ya = load(a.dout, a.do_ld, ra, ina, h, e), yb = load(a.dout, a.do_ld, rb, inb, h, e);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const int j = j0 + 8 * n + g;
                        const bool in = j < keys && ADALN_IN_ATTN(k0 >= 0 && (int64_t)k0 + j < a.Rk);
                        const uint4 k = load(a.k, a.k_ld, (int64_t)k0 + j, in, kv, e), v = load(a.v, a.v_ld, (int64_t)k0 + j, in, kv, e);
                        mma_m16n8k16(z[n], xa.x, xb.x, xa.y, xb.y, k.x, k.y);
                        mma_m16n8k16(z[n], xa.z, xb.z, xa.w, xb.w, k.z, k.w);
                        mma_m16n8k16(dp[n], ya.x, yb.x, ya.y, yb.y, v.x, v.y);
                        mma_m16n8k16(dp[n], ya.z, yb.z, ya.w, yb.w, v.z, v.w);
                    }
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const int j = j0 + 8 * n + 2 * q4 + c;
                        if (j < sa) va = fmaf(exp2_ftz(fmaf(z[n][c], sl2, -la)), dp[n][c], va);
                        if (j < sb) vb = fmaf(exp2_ftz(fmaf(z[n][2 + c], sl2, -lb)), dp[n][2 + c], vb);
                    }
                }
            }
#pragma unroll
            for (int o = 2; o >= 1; o >>= 1) {
                va += __shfl_xor_sync(0xFFFFFFFFu, va, o);
                vb += __shfl_xor_sync(0xFFFFFFFFu, vb, o);
            }
            if (q4 == 0 && (mine >> g & 1) && ina) a.delta[(int64_t)h * a.Rq + ra] = va;
            if (q4 == 0 && (mine >> (g + 8) & 1) && inb) a.delta[(int64_t)h * a.Rq + rb] = vb;
        }
    }
}

// Whether any row sees 1 .. kAttnFewKeys keys: the whole CTA looks through the tables. (Causal: the first rows of
// every segment do.)
__device__ __forceinline__ bool attn_any_few(const AttnTables& t) {
    bool any = t.causal != 0;
    for (int64_t s = threadIdx.x; s < t.nseg && !any; s += kPlanThreads) {
        const int64_t nk = attn_start(t.cu_k, s + 1, t.nseg, t.Rk) - attn_start(t.cu_k, s, t.nseg, t.Rk);
        any = nk > 0 && nk <= kAttnFewKeys;
    }
    return __syncthreads_or(any);
}

// The forward's work list. (A kernel of its own: as a part of the backward's, with its spills, 1 over 32760 took 52.4 us
// instead of 50.2.)
__global__ void __launch_bounds__(kPlanThreads) attn_plan_kernel(const __grid_constant__ AttnPlanArgs p) {
    pdl_begin();
    attn_plan(p, 0);
}

// The backward's work lists, a CTA each, and beside them delta: CTAs for rows of few keys, which wait for copies most of
// the time, and the others in turn. Two CTAs an SM: delta needs their loads (32760 over 512: 344 us with one).
__global__ void __launch_bounds__(kPlanThreads, 2) attn_prepare_kernel(const __grid_constant__ AttnPlanArgs p,
                                                               const __grid_constant__ AttnDeltaArgs d, int lists) {
    pdl_begin();
    const int at = (int)blockIdx.x - lists, all = (int)gridDim.x - lists - d.few, both = 2 * min(d.few, all);
    if (at < 0) {
        attn_plan(p, blockIdx.x);
        return;
    }
    const bool any_few = d.few > 0 && attn_any_few(p.t);
    if (at < both ? at % 2 != 0 : d.few <= all)
        any_few ? attn_delta<true>(p.t, d, at < both ? at / 2 : at - d.few, all)
                : attn_delta<false>(p.t, d, at < both ? at / 2 : at - d.few, all);
    else if (any_few)
        attn_delta_few(p.t, d, at < both ? at / 2 : at - all, d.few);
}

// The work list is written by the kernel ahead, which this kernel may have been scheduled before: read
// from L2.
__device__ __forceinline__ AttnItem attn_item(const AttnList& l, int64_t i) {
    AttnItem it{};
    if (!ADALN_IN_ATTN(i >= 0 && i < l.most)) return it;
    const int4 a = __ldcg(reinterpret_cast<const int4*>(l.items + i));
    const int4 b = __ldcg(reinterpret_cast<const int4*>(l.items + i) + 1);
    it.row0 = a.x;
    it.rows = a.y;
    it.other0 = a.z;
    it.others = a.w;
    it.shift = b.x;
    it.end = b.y;
    it.unseen = b.z;
    return it;
}
__device__ __forceinline__ AttnCursor attn_cursor(const AttnList& l, int c) {
    if (!ADALN_IN_ATTN(c >= 0 && c <= l.ctas)) return AttnCursor{0, 0};
    const int2 v = __ldcg(reinterpret_cast<const int2*>(l.cursors + c));
    return AttnCursor{v.x, v.y};
}

// The units of this CTA, one after another: entry and head, and the steps [t0, t1) of the unit's n that are
// its own.
struct AttnWalk {
    const AttnList& l;
    int cta;
    AttnCursor from, to;
    int count, unit, entry;
    AttnItem it, ahead;
    int head, t0, t1, all, shift;
    uint32_t elapsed = 0;  // steps so far
    __device__ __forceinline__ AttnWalk(const AttnList& list, int at) : l(list), cta(at) {
        from = attn_cursor(l, cta);
        to = attn_cursor(l, cta + 1);
        count = __ldcg(l.count);
        unit = from.unit - 1;
        head = count > 0 ? from.unit / count : 0;
        entry = count > 0 ? from.unit % count - 1 : 0;
        fetch();
    }
    // Loads the next unit's entry, once before every next(): early, since it takes as long as a step.
    __device__ __forceinline__ void fetch() {
        const int u = unit + 1;
        if (u < to.unit || (u == to.unit && to.tile > 0)) ahead = attn_item(l, entry + 1 < count ? entry + 1 : 0);
    }
    __device__ __forceinline__ bool next() {
        ++unit;
        if (unit > to.unit || (unit == to.unit && to.tile == 0)) return false;
        if (++entry == count) {
            entry = 0;
            ++head;
        }
        it = ahead;
        return true;
    }
    // With the unit's steps known. `turn`: its steps may go in any order; a whole unit then begins with the step
    // that the CTA would be at had it begun with step 0 of its first unit, and goes round. CTAs that work on
    // one head so read the same tiles at about the same time, wherever they began (32760 x 12 x 128: the keys
    // and values of all heads are more than L2 holds; 5065 us without, 4315 with).
    __device__ __forceinline__ void steps(int n, bool turn) {
        t0 = unit == from.unit ? from.tile : 0;
        t1 = unit == to.unit ? to.tile : n;
        all = n;
        shift = turn && n > 0 && whole(n) ? (int)(elapsed % (uint32_t)n) : 0;
        elapsed += (uint32_t)(t1 - t0);
    }
    // The tile of step t of the unit.
    __device__ __forceinline__ int tile(int t) const { return t + shift < all ? t + shift : t + shift - all; }
    __device__ __forceinline__ bool whole(int n) const { return t0 == 0 && t1 == n; }
    // Where a piece goes: a CTA has at most one that does not begin its unit and one that does.
    __device__ __forceinline__ int slot() const { return 2 * cta + (t0 == 0 ? 1 : 0); }
};

// ---- operands --------------------------------------------------------------------------------
template <int DP>
__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap* map, int head, int row, uint32_t bar) {
    tma_load3(dst, map, 0, head, row, bar);
    if (DP == 128) tma_load3(dst + kPanel, map, 64, head, row, bar);
}
// Rows [from, to) of a tile become zeros: what follows a segment may hold anything, and 0 * NaN is NaN.
template <int DP>
__device__ __forceinline__ void zero_rows(uint32_t tile, int from, int to, int lane) {
#pragma unroll
    for (int p = 0; p < DP / 64; ++p) {
        for (uint32_t at = (uint32_t)from * 128 + 16 * lane; at < (uint32_t)to * 128; at += 512)
            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(tile + p * kPanel + at), "r"(0u) : "memory");
    }
}
// D = A B^T over d: both tiles with d contiguous.
template <int DP>
__device__ __forceinline__ void mma_rows(uint32_t d_tmem, uint32_t a, uint32_t b, int d) {
    const uint64_t da = smem_desc(a, 0), db = smem_desc(b, 0);
    constexpr uint32_t idesc = mma_desc(128, kAttnTile, false, false);
#pragma unroll
    for (int k = 0; k < DP / 16; ++k) {
        const uint64_t off = (uint64_t)((k & 3) * 2 + (k >> 2) * (kPanel >> 4));
        if (16 * k < d) mma_bf16_ss(d_tmem, da + off, db + off, idesc, k > 0);
    }
}
// D (+)= A B with A [128, 128] bf16 in tensor memory, its columns 0..63 from `a`, the others from
// `a2`; B a tile whose 128 rows are the sum's, d columns.
__device__ __forceinline__ void mma_cols(uint32_t d_tmem, uint32_t a, uint32_t a2, uint32_t b, int d, bool accumulate) {
    const uint64_t db = smem_desc(b, kPanel);
    const uint32_t idesc = mma_desc(128, (d + 15) / 16 * 16, false, true);
#pragma unroll
    for (int k = 0; k < kAttnTile / 16; ++k)
        mma_bf16_ts(d_tmem, k < 4 ? a + 8 * k : a2 + 8 * (k - 4), db + (uint64_t)(k * (2048 >> 4)), idesc,
                    accumulate || k > 0);
}

// The same over 64 of the sum's rows.
__device__ __forceinline__ void mma_cols64(uint32_t d_tmem, uint32_t a, uint32_t b, int d, bool accumulate) {
    const uint64_t db = smem_desc(b, kPanel);
    const uint32_t idesc = mma_desc(128, (d + 15) / 16 * 16, false, true);
#pragma unroll
    for (int k = 0; k < kAttnTile / 32; ++k)
        mma_bf16_ts(d_tmem, a + 8 * k, db + (uint64_t)(k * (2048 >> 4)), idesc, accumulate || k > 0);
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t w;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
    return w;
}

// A warp's 32 rows, 64 columns from `col` on, through its 4 KB of shared memory and out by one TMA store
// (every lane's own 16-byte stores took 10,000 cycles for two tiles of 128 x 128); rows that another
// segment follows within the warp's 32 go directly. The buffer's last store has been read.
__device__ __forceinline__ void out64(const CUtensorMap* map, uint32_t buf, const uint32_t (&w)[32], int col, int head,
                                      int64_t row0, int rows, void* row, int d, int lane) {
    if (rows >= 32) {
        const uint32_t to = buf + 128 * lane;
#pragma unroll
        for (int c = 0; c < 8; ++c) st_swizzled(to, lane, c, w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
        fence_shared_async();
        __syncwarp();
        if (elect_lane()) tma_store3(map, col, head, (int)row0, buf);
    } else if (lane < rows) {
#pragma unroll
        for (int c = 0; c < 8; ++c)
            if (col + 8 * c < d)
                st_vec(reinterpret_cast<__nv_bfloat16*>(row) + col + 8 * c,
                       make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]));
    }
}
// 64 accumulator columns times f, rounded.
__device__ __forceinline__ void read64(uint32_t from, float f, uint32_t (&w)[32]) {
    float v[64];
    tmem_ld64(from, v);
#pragma unroll
    for (int j = 0; j < 32; ++j) w[j] = pack2(v[2 * j] * f, v[2 * j + 1] * f);
}
__device__ __forceinline__ void store_zeros(void* row, int c0, int c1, int d) {
    for (int c = c0; c < min(c1, d); c += 8)
        st_vec(reinterpret_cast<__nv_bfloat16*>(row) + c, make_uint4(0, 0, 0, 0));
}

// 32 columns of a row to a piece, which holds [d / 4][rows] vectors of four columns: the lanes of a warp, a row
// each, write side by side.
__device__ __forceinline__ void store_piece32(float* piece, int row, int rows, int col, int d, const float (&v)[32]) {
#pragma unroll
    for (int j = 0; j < 32; j += 4)
        if (col + j < d)
            reinterpret_cast<float4*>(piece)[(int64_t)((col + j) / 4) * rows + row] = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
}

// What a CTA has issued, for the drain after a timeout: copies and products must not land in memory
// that has been given back.
struct AttnIssued {
    uint32_t ring = 0, pair = 0, pair2 = 0, tail = 0;  // fills of the ring, of the resident tiles (of the second), of tails
    bool mma = false;
};

// Registers a thread of the forward: at launch, then of the rows' warps and of the others. (The compiler keeps
// to the launch's and spills: -Xptxas -v, 232 bytes of loads at 128 elements, 220 at 64.)
constexpr int kFwdRegs = 168, kRowRegs = 208, kOtherRegs = 88;
static_assert(256 * kRowRegs + 128 * kOtherRegs <= kAttnThreads * kFwdRegs, "no more than the launch brought");

// ---- forward ---------------------------------------------------------------------------------
template <int DP>
__global__ void __launch_bounds__(kAttnThreads, 1) attn_fwd_kernel(const __grid_constant__ CUtensorMap mq,
                                                                const __grid_constant__ CUtensorMap mk,
                                                                const __grid_constant__ CUtensorMap mv,
                                                                const __grid_constant__ CUtensorMap mo,
                                                                const AttnFwdArgs a) {
    using S = AttnShape<DP, kAttnFwd>;
    constexpr int ST = S::kStages;
    extern __shared__ uint4 dyn[];
    __shared__ __align__(8) uint64_t bars[2 * ST + 14];
    __shared__ uint32_t tmem_base;
    __shared__ int abort_flag;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t qt = (smem_addr(dyn) + 1023u) & ~1023u, ring = qt + 2 * S::kTile;
    const uint32_t full = smem_addr(bars), empty = full + 8 * ST, qfull = empty + 8 * ST, qempty = qfull + 8;
    const uint32_t sfull = qempty + 8, pfull = sfull + 16, pfull2 = pfull + 16, odone = pfull2 + 16, ofree = odone + 16;
    const uint32_t tail = ofree + 16, drain = tail + 8;
    if (tid == 0) {
        for (int i = 0; i < ST; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(empty + 8 * i, 1);
        }
        mbar_init(qfull, 1);
        mbar_init(qempty, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(sfull + 8 * i, 1);
            mbar_init(pfull + 8 * i, 4);
            mbar_init(pfull2 + 8 * i, 4);
            mbar_init(odone + 8 * i, 1);
            mbar_init(ofree + 8 * i, 4);
        }
        mbar_init(tail, 1);
        mbar_init(drain, 1);
        abort_flag = 0;
        mbar_fence_init();
        tma_prefetch_map(&mq);
        tma_prefetch_map(&mk);
        tma_prefetch_map(&mv);
        tma_prefetch_map(&mo);
    }
    if (warp == kAllocWarp) tmem_alloc1(smem_addr(&tmem_base), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_trigger();  // behind the allocation: a dependent CTA on this SM must not get the columns first
    const uint32_t tmem = tmem_base;
    pdl_wait();
    AttnIssued issued;
    const int role = __shfl_sync(0xFFFFFFFFu, warp, 0);
    // Steps [t0, t1[i]) of a unit for its two tiles of queries; n of the unit in all.
    AttnWalk walk(a.list, blockIdx.x);
    const AttnItem& it = walk.it;
    const int& head = walk.head;
    int t0 = 0, t1[2], n = 0;
    auto next = [&]() {
        if (!walk.next()) return false;
        int of[2];
        n = 0;
        for (int i = 0; i < 2; ++i) {
            const int rows = min(max(walk.it.rows - i * kAttnTile, 0), kAttnTile);
            const int seen = rows > 0 ? max(0, min(walk.it.others, walk.it.shift + i * kAttnTile + rows)) : 0;
            of[i] = (seen + kAttnTile - 1) / kAttnTile;
            n = max(n, of[i]);
        }
        walk.steps(n, of[0] == n && (of[1] == n || it.rows <= kAttnTile));
        t0 = walk.t0;
        for (int i = 0; i < 2; ++i) t1[i] = max(t0, min(of[i], walk.t1));
        return true;
    };

    // Registers: the launch's 384 x 168 go as 256 x 208 to the rows' warps, which hold 128 scores each, and
    // 128 x 88 to the others.
    if (role >= kMmaWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (role == kLoadWarp) {
            bool live = true;
            fence_async_proxy();
            while (live && next()) {
                walk.fetch();
                const int end = max(t1[0], t1[1]);
                if (end == t0) continue;
                live = __all_sync(0xFFFFFFFFu, issued.pair == 0 || mbar_wait_bounded(qempty, (issued.pair - 1) & 1u, &abort_flag));
                if (!live) break;
                const int tiles = it.rows > kAttnTile ? 2 : 1;
                if (elect_lane()) {
                    mbar_arrive_expect_tx(qfull, tiles * S::kTile);
                    for (int i = 0; i < tiles; ++i)
                        load_tile<DP>(qt + i * S::kTile, &mq, head, it.row0 + i * kAttnTile, qfull);
                }
                ++issued.pair;
                const int kv = head / a.group;
                for (int t = t0; t < end && live; ++t) {
                    const int at = walk.tile(t) * kAttnTile, row = it.other0 + at, left = it.others - at;
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const uint32_t s = issued.ring % ST, lap_ = issued.ring / ST;
                        live = __all_sync(0xFFFFFFFFu, lap_ == 0 || mbar_wait_bounded(empty + 8 * s, (lap_ - 1) & 1u, &abort_flag));
                        if (!live) break;
                        const uint32_t dst = ring + s * S::kTile;
                        // The values' last tile of a segment that something follows goes through this warp.
                        const bool cut = x == 1 && left < kAttnTile && !it.end;
                        if (elect_lane()) {
                            const uint32_t bar = cut ? tail : full + 8 * s;
                            mbar_arrive_expect_tx(bar, S::kTile);
                            load_tile<DP>(dst, x ? &mv : &mk, kv, row, bar);
                        }
                        if (cut) {
                            live = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(tail, issued.tail & 1u, &abort_flag));
                            ++issued.tail;
                            if (live) {
                                zero_rows<DP>(dst, left, kAttnTile, lane);
                                fence_shared_async();
                            }
                            __syncwarp();
                            if (elect_lane()) mbar_arrive(full + 8 * s);
                        }
                        ++issued.ring;
                        if (!live) break;
                    }
                }
            }
        } else if (role == kMmaWarp) {
            bool live = true;
            uint32_t used = 0, pairs = 0, np[2] = {0, 0}, nu[2] = {0, 0};  // ring tiles, units, tiles and units a warpgroup
            auto wait = [&](uint32_t bar, uint32_t parity) {
                live = live && __all_sync(0xFFFFFFFFu, mbar_wait_bounded(bar, parity & 1u, &abort_flag));
                return live;
            };
            auto stage = [&](uint32_t n) { return n % ST; };
            auto scores = [&](int i, uint32_t n) {
                if (elect_lane()) {
                    mma_rows<DP>(tmem + 128 * i, qt + i * S::kTile, ring + stage(n) * S::kTile, a.d);
                    mma_commit1(sfull + 8 * i);
                }
            };
            while (live && next()) {
                walk.fetch();
                const int end = max(t1[0], t1[1]);
                if (end == t0) continue;
                if (!wait(qfull, pairs) || !wait(full + 8 * stage(used), used / ST)) break;
                tc_fence_after();
                issued.mma = true;
                for (int i = 0; i < 2; ++i)
                    if (t1[i] > t0) scores(i, used);
                if (elect_lane()) {
                    mma_commit1(empty + 8 * stage(used));
                    if (end == t0 + 1) mma_commit1(qempty);
                }
                for (int t = t0; t < end; ++t, used += 2) {
                    const bool more = t + 1 < end;
                    if (more && !wait(full + 8 * stage(used + 2), (used + 2) / ST)) break;
                    if (!wait(full + 8 * stage(used + 1), (used + 1) / ST)) break;
                    for (int i = 0; i < 2; ++i) {
                        if (t >= t1[i]) continue;
                        if (t == t0 && nu[i] > 0 && !wait(ofree + 8 * i, nu[i] - 1)) break;
                        // Each half of the keys as soon as its p is there.
                        const uint32_t acc = tmem + 256 + 128 * i, v = ring + stage(used + 1) * S::kTile;
                        if (!wait(pfull + 8 * i, np[i])) break;
                        tc_fence_after();
                        if (elect_lane()) mma_cols64(acc, tmem + 128 * i, v, a.d, t > t0);
                        if (!wait(pfull2 + 8 * i, np[i])) break;
                        tc_fence_after();
                        if (elect_lane()) {
                            mma_cols64(acc, tmem + 128 * i + 32, v + kPanel / 2, a.d, true);
                            mma_commit1(odone + 8 * i);
                        }
                        ++np[i];
                        if (t + 1 < t1[i]) scores(i, used + 2);
                    }
                    if (!live) break;
                    if (t + 2 == end && elect_lane()) mma_commit1(qempty);  // behind the unit's last scores
                    if (elect_lane()) {
                        mma_commit1(empty + 8 * stage(used + 1));
                        if (more) mma_commit1(empty + 8 * stage(used + 2));
                    }
                }
                if (!live) break;
                ++pairs;
                for (int i = 0; i < 2; ++i)
                    if (t1[i] > t0) ++nu[i];
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRowRegs));
        const int i = warp >> 2;  // this warpgroup's tile of queries
        const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21), st = lanes + 128 * i, ot = lanes + 256 + 128 * i;
        const int r = (warp & 3) * 32 + lane;
        const float sl2 = a.scale * kLog2e;
        const uint32_t out_buf = ring + ST * S::kTile + warp * kAttnOut;
        uint32_t tiles = 0;
        bool live = true;
        while (live && next()) {
            const int row = i * kAttnTile + r, end = i ? t1[1] : t1[0];
            // Keys that this row sees.
            const int seen = max(0, min(it.others, it.shift + row + 1));
            float m = neg_inf(), l = 0.0f;  // the exponentials' reference, their sum
            for (int t = t0; t < end; ++t, ++tiles) {
                live = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(sfull + 8 * i, tiles & 1u, &abort_flag));
                if (!live) break;
                tc_fence_after();
                float v[64], w[64];
                const int lim = seen - walk.tile(t) * kAttnTile;
                const bool cut = __any_sync(0xFFFFFFFFu, lim < kAttnTile);
                tmem_ld128(st, v, w);
                if (cut) {
#pragma unroll
                    for (int j = 0; j < 64; ++j) {
                        v[j] = j < lim ? v[j] : neg_inf();
                        w[j] = 64 + j < lim ? w[j] : neg_inf();
                    }
                }
                float m4[4] = {v[0], v[1], w[0], w[1]};
#pragma unroll
                for (int j = 2; j < 64; j += 2) {
                    m4[0] = fmaxf(m4[0], v[j]);
                    m4[1] = fmaxf(m4[1], v[j + 1]);
                    m4[2] = fmaxf(m4[2], w[j]);
                    m4[3] = fmaxf(m4[3], w[j + 1]);
                }
                const float mt = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
                const f2r s2 = p_splat(sl2);
                f2r c2, sum[2];
                uint32_t b[32];
                // Exponentials of 64 scores against the reference, their sum; a row that has seen nothing yet
                // has none but 0 (and NaN stays).
                auto half = [&](const float (&x)[64]) {
                    c2 = p_splat(m == neg_inf() ? 0.0f : -m * sl2);
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        const float2 e = p_get(p_fma(p_make(x[2 * j], x[2 * j + 1]), s2, c2));
                        const float e0 = exp2_ftz(e.x), e1 = exp2_ftz(e.y);
                        sum[j & 1] = p_add(sum[j & 1], p_make(e0, e1));
                        b[j] = pack2(e0, e1);
                    }
                };
                // The first half's against the reference of the step before, while the maximum is still being
                // found; it seldom has to be done again.
                sum[0] = sum[1] = kPairZero;
                half(v);
                // The reference may lag behind the maximum by 2^8, which fp32 sums and bf16 p take as well as 1;
                // beyond it, what has been summed is brought to the new one. Each row goes by its own scores: the
                // others' decide only whether the warp comes here, where a row whose reference stays is
                // multiplied by 1. Rows behind the segment's last, which meet its keys too, do not ask for it.
                const bool jump = (mt - m) * sl2 > 8.0f;
                if (__any_sync(0xFFFFFFFFu, t == t0 || (jump && row < it.rows))) {
                    const float to = t == t0 || jump ? mt : m;
                    if (t > t0) {
                        const float f = to == m ? 1.0f : exp2_ftz((m - to) * sl2);
                        live = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(odone + 8 * i, (tiles - 1) & 1u, &abort_flag));
                        if (!live) break;
                        tc_fence_after();
                        l *= f;
#pragma unroll 1
                        for (int c = 0; c < a.d; c += 32) {
                            float o[32];
                            tmem_ld32(ot + c, o);
#pragma unroll
                            for (int j = 0; j < 32; ++j) b[j] = __float_as_uint(o[j] * f);
                            tmem_st32(ot + c, b);
                        }
                    }
                    m = to;
                    tmem_ld64(st, v);
                    if (cut) {
#pragma unroll
                        for (int j = 0; j < 64; ++j) v[j] = j < lim ? v[j] : neg_inf();
                    }
                    sum[0] = sum[1] = kPairZero;
                    half(v);
                }
                tmem_st32(st, b);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(pfull + 8 * i);
                half(w);
                tmem_st32(st + 32, b);
                l += p_hsum(p_add(sum[0], sum[1]));
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(pfull2 + 8 * i);
            }
            if (!live) break;
            walk.fetch();
            const bool mine = row < it.rows;
            const int64_t at = (int64_t)it.row0 + row;
            const bool in = mine && ADALN_IN_ATTN(at >= 0 && at < a.Rq && head < a.Hq);
            const bool none = l == 0.0f;  // no key seen: zeros
            if (end > t0) {
                live = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(odone + 8 * i, (tiles - 1) & 1u, &abort_flag));
                if (!live) break;
                tc_fence_after();
            }
            if (walk.whole(n)) {
                if (in) a.lse[(int64_t)head * a.Rq + at] = none ? neg_inf() : fmaf(m, a.scale, logf(l));
                const float f = 1.0f / l;
                const int first = i * kAttnTile + (warp & 3) * 32, rows = min(32, it.rows - first);
#pragma unroll 1
                for (int c = 0; c < a.d && rows > 0; c += 64) {
                    uint32_t b[32];
                    if (end > t0) read64(ot + c, f, b);
#pragma unroll
                    for (int j = 0; j < 32; ++j) b[j] = none ? 0u : b[j];
                    tma_store_read();  // the lane that issued the buffer's last store has it read
                    __syncwarp();
                    out64(&mo, out_buf, b, c, head, it.row0 + first, in || !mine ? rows : 0,
                          reinterpret_cast<__nv_bfloat16*>(a.o) + at * a.o_ld + (int64_t)head * a.d, a.d, lane);
                }
            } else {
                const int64_t place = (int64_t)walk.slot() * a.slot_rows + row;
                if (end > t0) {
#pragma unroll 1
                    for (int c = 0; c < a.d; c += 32) {
                        float o[32];
                        tmem_ld32(ot + c, o);
                        if (in && ADALN_IN_ATTN(row < a.slot_rows))
                            store_piece32(a.part + (int64_t)walk.slot() * a.slot_rows * a.d, row, a.slot_rows, c, a.d, o);
                    }
                }
                if (in && ADALN_IN_ATTN(row < a.slot_rows)) a.ml[place] = make_float2(m, l);
            }
            if (end > t0) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(ofree + 8 * i);
            }
        }
        tma_store_wait();
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (__builtin_expect(*(volatile int*)&abort_flag, 0)) {
        volatile int never = 0;
        if (warp == kLoadWarp && lane == 0) {
            if (issued.pair) mbar_wait_bounded(qfull, (issued.pair - 1) & 1u, &never);
            if (issued.tail) mbar_wait_bounded(tail, (issued.tail - 1) & 1u, &never);
            for (uint32_t s = 0; s < min(issued.ring, (uint32_t)ST); ++s)
                mbar_wait_bounded(full + 8 * s, ((issued.ring - 1 - s) / ST) & 1u, &never);
        }
        if (warp == kMmaWarp && issued.mma && elect_lane()) {
            mma_commit1(drain);
            mbar_wait_bounded(drain, 0, &never);
        }
        __syncwarp();
        __syncthreads();
    }
    tc_fence_after();
    if (warp == kAllocWarp) tmem_free1(tmem, 512);
    if (tid == 0 && abort_flag) atomicOr(a.status, kErrTimeout);
}

// Pieces joined, in the order of the CTAs that left them. CTA (c, y, list): if CTA c of the list is the first
// that began inside its unit, the y-th eighth of that unit's rows. Forward: o = sum_s w_s o_s / sum_s w_s l_s
// with w_s = 2^(m_s - max m); backward: plain sums.
template <bool BWD>
__global__ void __launch_bounds__(256) attn_join_kernel(const __grid_constant__ AttnJoinArgs a) {
    pdl_begin();
    const int list = blockIdx.z, c = blockIdx.x;
    const AttnList& l = a.list[list];
    if (l.items == nullptr || c == 0 || c >= l.ctas) return;
    const AttnCursor cur = attn_cursor(l, c), prev = attn_cursor(l, c - 1);
    if (cur.tile == 0 || (prev.unit == cur.unit && prev.tile > 0)) return;
    // The pieces: CTA c - 1's, which begins the unit, then of every CTA that begins inside it (one of two that
    // begin at one place has none).
    __shared__ int16_t slots[kAttnMaxCtas + 1];
    __shared__ float weight[BWD ? 1 : 32][kAttnMaxCtas + 1];  // forward: of a row's pieces, 0 for none
    int begun = 0;
    for (int x0 = c + 1; x0 < l.ctas; x0 += 256) {
        const int x = x0 + threadIdx.x;
        begun += __syncthreads_count(x < l.ctas && attn_cursor(l, x).unit == cur.unit);
    }
    const int pieces = 2 + begun;
    for (int x = threadIdx.x; x < pieces; x += 256) {
        const int at = c - 1 + x;
        const bool none = x > 0 && x < pieces - 1 && attn_cursor(l, at).tile == attn_cursor(l, at + 1).tile;
        slots[x] = none ? -1 : (int16_t)(x == 0 ? 2 * at + 1 : 2 * at);
    }
    __syncthreads();
    const int count = __ldcg(l.count), head = cur.unit / count;
    const AttnItem it = attn_item(l, cur.unit % count);
    const int vecs = a.d / 8, rows = a.slot_rows[list], parts = BWD && list == 1 ? 2 : 1;
    const int64_t plane = (int64_t)rows * a.d;
    const float sl2 = a.scale * kLog2e;
    const int per = (rows + 7) / 8, items = per * vecs * parts;
    if (!BWD) {
        // A warp a row, a lane a piece: the maximum, the weights, the sum.
        const int lane = threadIdx.x & 31;
        for (int k = threadIdx.x >> 5; k < per; k += 8) {
            const int row = (int)blockIdx.y * per + k;
            const int64_t at = (int64_t)it.row0 + row;
            if (row >= it.rows || !ADALN_IN_ATTN(row < rows && k < 32)) continue;
            float top = neg_inf(), sum = 0.0f;
            auto load = [&](int x) {
                const int s = x < pieces ? slots[x] : -1;
                return s < 0 ? make_float2(0.0f, 0.0f) : __ldcg(a.ml + (int64_t)s * rows + row);
            };
            float2 first = load(lane);  // (sum 0: the row sees nothing of the piece)
            for (int x = lane; x < pieces; x += 32) {
                const float2 ml = x == lane ? first : load(x);
                if (ml.y != 0.0f) top = fmaxf(top, ml.x);
            }
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
            for (int x = lane; x < pieces; x += 32) {
                const float2 ml = x == lane ? first : load(x);
                const float w = ml.y == 0.0f ? 0.0f : top == neg_inf() ? 1.0f : exp2_ftz((ml.x - top) * sl2);
                weight[k][x] = ml.y == 0.0f ? 0.0f : w;
                sum = fmaf(w, ml.y, sum);
            }
            float v[1] = {sum};
            warp_sum(v);
            sum = v[0];
            for (int x = lane; x < pieces; x += 32) weight[k][x] *= sum == 0.0f ? 0.0f : 1.0f / sum;
            if (lane == 0) a.lse[(int64_t)head * a.Rq + at] = sum == 0.0f ? neg_inf() : fmaf(top, a.scale, logf(sum));
        }
        __syncthreads();
    }
    for (int i = threadIdx.x; i < items; i += 256) {
        // Rows side by side, as the pieces have them.
        const int k = i % per, row = (int)blockIdx.y * per + k, v = i / per % vecs, part = i / per / vecs;
        const int64_t at = (int64_t)it.row0 + row;
        if (row >= it.rows || !ADALN_IN_ATTN(row < rows)) continue;
        float o[8] = {};
        for (int x0 = 0; x0 < pieces; x0 += 4) {  // four pieces on their way
            float4 f[4], g[4];
            float w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int x = x0 + j, s = x < pieces ? slots[x] : -1;
                w[j] = s < 0 ? 0.0f : BWD ? 1.0f : weight[BWD ? 0 : k][x];
                f[j] = g[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (w[j] == 0.0f) continue;
                const float4* p = reinterpret_cast<const float4*>(a.part[list] + ((int64_t)s * parts + part) * plane) +
                                  (int64_t)2 * v * rows + row;
                f[j] = __ldcg(p);
                g[j] = __ldcg(p + rows);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                o[0] = fmaf(w[j], f[j].x, o[0]);
                o[1] = fmaf(w[j], f[j].y, o[1]);
                o[2] = fmaf(w[j], f[j].z, o[2]);
                o[3] = fmaf(w[j], f[j].w, o[3]);
                o[4] = fmaf(w[j], g[j].x, o[4]);
                o[5] = fmaf(w[j], g[j].y, o[5]);
                o[6] = fmaf(w[j], g[j].z, o[6]);
                o[7] = fmaf(w[j], g[j].w, o[7]);
            }
        }
        const bool dv = BWD && list == 1 && part == 0;
        const float f = !BWD || dv ? 1.0f : a.scale;
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = pack2(o[2 * j] * f, o[2 * j + 1] * f);
        __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(dv ? a.dv : a.out[list]) + at * (dv ? a.dv_ld : a.ld[list]);
        st_vec(out + (int64_t)head * a.d + 8 * v, make_uint4(w[0], w[1], w[2], w[3]));
    }
}

// ---- backward --------------------------------------------------------------------------------
// 64 values of a row, those outside [from, to) 0.
__device__ __forceinline__ void mask64(float (&p)[64], int from, int to) {
#pragma unroll
    for (int j = 0; j < 64; ++j) p[j] = j >= from && j < to ? p[j] : 0.0f;
}

// dq of a tile of 128 queries. Its scores have two places in tensor memory: dz goes over the scores that
// it came from, and the next scores and dp are formed while the warps are at it. The two warpgroups
// take 64 keys of a step each, a thread a row. The queries' shared memory is free behind the unit's last
// scores, so that the next unit's scores are there when dq has gone out, through dout's.
template <int DP>
__device__ __forceinline__ void attn_dq(const CUtensorMap& mdo, const CUtensorMap& mq, const CUtensorMap& mk,
                                        const CUtensorMap& mv, const CUtensorMap& mdq, const AttnBwdArgs& a, int cta) {
    using S = AttnShape<DP, kAttnDq>;
    // Keys are held from their scores to dq, two steps on; values from dp of their step alone. With a ring
    // for both, a values' tile would wait for the keys three tiles before it.
    constexpr int KS = DP == 128 ? 3 : 4, VS = DP == 128 ? 2 : 4, ST = KS + VS;
    static_assert(ST == S::kStages, "the rings fill the shared memory");
    extern __shared__ __align__(1024) unsigned char bwd_shared[];
    uint64_t* bars = reinterpret_cast<uint64_t*>(bwd_shared + S::kBars);
    static_assert((2 * ST + 14) * 8 <= 312, "barriers and two words in 320 bytes");
    uint32_t* tmem_word = reinterpret_cast<uint32_t*>(bwd_shared + S::kBars + 312);
    volatile int& abort_flag = *reinterpret_cast<volatile int*>(bwd_shared + S::kBars + 316);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t qt = smem_addr(bwd_shared), ring = qt + 2 * S::kTile;
    const uint32_t full = smem_addr(bars), empty = full + 8 * ST, qfull = empty + 8 * ST, dofull = qfull + 8, doempty = dofull + 8, qempty = doempty + 8;
    const uint32_t sfull = qempty + 8, pfull = sfull + 16, pfree = pfull + 8, dsfull = pfree + 8;
    const uint32_t done = dsfull + 16, freed = done + 8, tail = freed + 8, drain = tail + 8;
    if (tid == 0) {
        for (int i = 0; i < ST; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(empty + 8 * i, 1);
        }
        mbar_init(qfull, 1);
        mbar_init(qempty, 1);
        mbar_init(dofull, 1);
        mbar_init(doempty, 9);  // the products that read it, and the warps that sent dq out through it
        mbar_init(sfull, 1);
        mbar_init(sfull + 8, 1);
        mbar_init(pfull, 1);
        mbar_init(pfree, 8);
        // Two: a warp may be through a step before another one has written its dz of the step before (dp
        // of a step needs only that the last dp has been read), but not two.
        mbar_init(dsfull, 8);
        mbar_init(dsfull + 8, 8);
        mbar_init(done, 1);
        mbar_init(freed, 8);
        mbar_init(tail, 1);
        mbar_init(drain, 1);
        abort_flag = 0;
        mbar_fence_init();
        tma_prefetch_map(&mdo);
        tma_prefetch_map(&mq);
        tma_prefetch_map(&mk);
        tma_prefetch_map(&mv);
        tma_prefetch_map(&mdq);
    }
    if (warp == kAllocWarp) tmem_alloc1(smem_addr(tmem_word), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_trigger();
    const uint32_t tmem = *tmem_word, dp_tmem = tmem + 256, acc = tmem + 384;
    pdl_wait();
    AttnIssued issued;
    const int role = __shfl_sync(0xFFFFFFFFu, warp, 0);
    // n steps of a unit, from step t0 of it on; `all` is the unit's.
    AttnWalk walk(a.list, cta);
    int t0 = 0, n = 0, all = 0;
    auto next = [&]() {
        if (!walk.next()) return false;
        all = (max(0, min(walk.it.others, walk.it.shift + walk.it.rows)) + kAttnTile - 1) / kAttnTile;
        walk.steps(all, true);
        t0 = walk.t0;
        n = walk.t1 - t0;
        return true;
    };
    const AttnItem& it = walk.it;
    const int& head = walk.head;

    if (role == kLoadWarp) {
        bool live = true;
        uint32_t steps = 0;
        fence_async_proxy();
        while (live && next()) {
            walk.fetch();
            if (n == 0) continue;
            live = __all_sync(0xFFFFFFFFu, issued.pair == 0 || mbar_wait_bounded(qempty, (issued.pair - 1) & 1u, &abort_flag));
            if (!live) break;
            if (elect_lane()) {
                mbar_arrive_expect_tx(qfull, S::kTile);
                load_tile<DP>(qt, &mq, head, it.row0, qfull);
            }
            ++issued.pair;
            const int kv = head / a.group;
            for (int t = t0; t < t0 + n && live; ++t, ++steps) {
                const int at = walk.tile(t) * kAttnTile, row = it.other0 + at, left = it.others - at;
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const uint32_t s = x ? KS + steps % VS : steps % KS, l = x ? steps / VS : steps / KS;
                    live = __all_sync(0xFFFFFFFFu, l == 0 || mbar_wait_bounded(empty + 8 * s, (l - 1) & 1u, &abort_flag));
                    if (!live) break;
                    const uint32_t dst = ring + s * S::kTile;
                    const bool cut = x == 0 && left < kAttnTile && !it.end;  // dz k: keys past the segment's end
                    if (elect_lane()) {
                        const uint32_t bar = cut ? tail : full + 8 * s;
                        mbar_arrive_expect_tx(bar, S::kTile);
                        load_tile<DP>(dst, x ? &mv : &mk, kv, row, bar);
                    }
                    if (cut) {
                        live = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(tail, issued.tail & 1u, &abort_flag));
                        ++issued.tail;
                        if (live) {
                            zero_rows<DP>(dst, left, kAttnTile, lane);
                            fence_shared_async();
                        }
                        __syncwarp();
                        if (elect_lane()) mbar_arrive(full + 8 * s);
                    }
                    ++issued.ring;
                    if (!live) break;
                    if (n > 1 ? x == 0 && t == t0 + 1 : x == 1) {  // dout behind what goes before it
                        live = __all_sync(0xFFFFFFFFu,
                                          issued.pair2 == 0 || mbar_wait_bounded(doempty, (issued.pair2 - 1) & 1u, &abort_flag));
                        if (!live) break;
                        if (elect_lane()) {
                            mbar_arrive_expect_tx(dofull, S::kTile);
                            load_tile<DP>(qt + S::kTile, &mdo, head, it.row0, dofull);
                        }
                        ++issued.pair2;
                    }
                }
            }
        }
    } else if (role == kMmaWarp) {
        bool live = true;
        uint32_t laps = 0, steps = 0;  // units, steps
        auto wait = [&](uint32_t bar, uint32_t parity) {
            live = live && __all_sync(0xFFFFFFFFu, mbar_wait_bounded(bar, parity & 1u, &abort_flag));
            return live;
        };
        // Places of the keys and the values of step j of this unit, and waits for them.
        auto kslot = [&](int j) { return (steps + j) % KS; };
        auto vslot = [&](int j) { return KS + (steps + j) % VS; };
        auto keys = [&](int j) { return wait(full + 8 * kslot(j), (steps + j) / KS); };
        auto values = [&](int j) { return wait(full + 8 * vslot(j), (steps + j) / VS); };
        // z of step j (of this unit), dp of step j.
        auto scores = [&](int j) {
            const uint32_t b = (steps + j) & 1u;
            if (elect_lane()) {
                mma_rows<DP>(tmem + 128 * b, qt, ring + kslot(j) * S::kTile, a.d);
                mma_commit1(sfull + 8 * b);
            }
        };
        auto dprobs = [&](int j) {
            if (elect_lane()) {
                mma_rows<DP>(dp_tmem, qt + S::kTile, ring + vslot(j) * S::kTile, a.d);
                mma_commit1(pfull);
                mma_commit1(empty + 8 * vslot(j));
            }
        };
        while (live && next()) {
            walk.fetch();
            if (n == 0) continue;
            if (!wait(qfull, laps) || !keys(0)) break;
            tc_fence_after();
            issued.mma = true;
            scores(0);
            if (n > 1) {
                if (!keys(1)) break;
                tc_fence_after();
                scores(1);
            }
            if (n <= 2 && elect_lane()) mma_commit1(qempty);
            if (!wait(dofull, laps) || !values(0)) break;
            tc_fence_after();
            dprobs(0);
            for (int j = 0; j < n; ++j) {
                if (j + 1 < n) {
                    if (!values(j + 1) || !wait(pfree, steps + j)) break;
                    tc_fence_after();
                    dprobs(j + 1);
                }
                if (j == 0 && laps > 0 && !wait(freed, laps - 1)) break;
                if (!wait(dsfull + 8 * ((steps + j) & 1u), (steps + j) >> 1)) break;
                tc_fence_after();
                if (elect_lane()) {
                    const uint32_t z = tmem + 128 * ((steps + j) & 1u);
                    mma_cols(acc, z, z + 64, ring + kslot(j) * S::kTile, a.d, j > 0);
                    mma_commit1(empty + 8 * kslot(j));
                }
                if (j + 2 < n) {
                    if (!keys(j + 2)) break;
                    tc_fence_after();
                    scores(j + 2);
                    if (j + 3 == n && elect_lane()) mma_commit1(qempty);  // behind the unit's last scores
                }
            }
            if (!live) break;
            if (elect_lane()) {
                mma_commit1(done);
                mma_commit1(doempty);
            }
            steps += n;
            ++laps;
        }
    } else if (role < kMmaWarp) {
        const int wg = warp >> 2, r = (warp & 3) * 32 + lane;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;
        const float sl2 = a.scale * kLog2e;
        const f2r s2 = p_splat(sl2);
        uint32_t steps = 0, laps = 0;
        bool live = true;
        while (live && next()) {
            const int64_t at = (int64_t)it.row0 + r;
            const bool in = r < it.rows && ADALN_IN_ATTN(at >= 0 && at < a.Rq && head < a.Hq);
            const float lse2 = in ? __ldcg(a.lse2 + (int64_t)head * a.Rq + at) : 0.0f;
            const float delta = in ? __ldcg(a.delta + (int64_t)head * a.Rq + at) : 0.0f;
            const int seen = max(0, min(it.others, it.shift + r + 1));
            const f2r nl = p_splat(-lse2), nd = p_splat(-delta);
            for (int t = t0; t < t0 + n; ++t, ++steps) {
                const uint32_t b = steps & 1u, z = tmem + lanes + 128 * b + 64 * wg;
                live = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(sfull + 8 * b, (steps >> 1) & 1u, &abort_flag));
                if (!live) break;
                tc_fence_after();
                float p[64];
                tmem_ld64(z, p);
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    const float2 e = p_get(p_fma(p_make(p[2 * j], p[2 * j + 1]), s2, nl));
                    p[2 * j] = exp2_ftz(e.x);
                    p[2 * j + 1] = exp2_ftz(e.y);
                }
                const int lim = seen - walk.tile(t) * kAttnTile - 64 * wg;
                const bool cut = __any_sync(0xFFFFFFFFu, lim < 64);
                live = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(pfull, steps & 1u, &abort_flag));
                if (!live) break;
                tc_fence_after();
                float dp[64];
                tmem_ld64(dp_tmem + lanes + 64 * wg, dp);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(pfree);
                uint32_t w[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    const float2 x = p_get(p_mul(p_add(p_make(dp[2 * j], dp[2 * j + 1]), nd), p_make(p[2 * j], p[2 * j + 1])));
                    dp[2 * j] = x.x;
                    dp[2 * j + 1] = x.y;
                }
                if (cut) mask64(dp, 0, lim);  // dz itself: p, dp and delta of what is masked may be infinite or NaN
#pragma unroll
                for (int j = 0; j < 32; ++j) w[j] = pack2(dp[2 * j], dp[2 * j + 1]);
                tmem_st32(z, w);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(dsfull + 8 * b);
            }
            if (!live) break;
            walk.fetch();
            __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(a.dx) + at * a.dx_ld + (int64_t)head * a.d;
            if (n == 0) {  // nothing of the unit, or nothing in it
                if (in && all == 0) store_zeros(out, wg * (DP / 2), (wg + 1) * (DP / 2), a.d);
                continue;
            }
            live = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(done, laps & 1u, &abort_flag));
            if (!live) break;
            tc_fence_after();
            // 64 columns a warpgroup, out through dout's shared memory.
            if (walk.whole(all)) {
                const int rows = min(32, it.rows - (warp & 3) * 32);
                if (64 * wg < a.d && rows > 0) {
                    uint32_t w[32];
                    read64(acc + lanes + 64 * wg, a.scale, w);
                    out64(&mdq, (DP == 64 ? qt + S::kTiles : qt + S::kTile) + warp * kAttnOut, w, 64 * wg, head, it.row0 + (warp & 3) * 32, rows, out, a.d, lane);
                    tma_store_read();
                }
            } else {
                float* piece = a.part + (int64_t)walk.slot() * a.slot_rows * a.d;
#pragma unroll 1
                for (int c = 64 * wg; c < min(64 * (wg + 1), a.d); c += 32) {
                    float o[32];
                    tmem_ld32(acc + lanes + c, o);
                    if (in && ADALN_IN_ATTN(r < a.slot_rows)) store_piece32(piece, r, a.slot_rows, c, a.d, o);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(freed);
                mbar_arrive(doempty);
            }
            ++laps;
        }
        tma_store_wait();
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (__builtin_expect(abort_flag, 0)) {
        volatile int never = 0;
        if (warp == kLoadWarp && lane == 0) {
            if (issued.pair) mbar_wait_bounded(qfull, (issued.pair - 1) & 1u, &never);
            if (issued.pair2) mbar_wait_bounded(dofull, (issued.pair2 - 1) & 1u, &never);
            if (issued.tail) mbar_wait_bounded(tail, (issued.tail - 1) & 1u, &never);
            // ring counts tiles of both rings, the keys' first.
            const uint32_t ks = (issued.ring + 1) / 2, vs = issued.ring / 2;
            for (uint32_t s = 0; s < min(ks, (uint32_t)KS); ++s)
                mbar_wait_bounded(full + 8 * s, ((ks - 1 - s) / KS) & 1u, &never);
            for (uint32_t s = 0; s < min(vs, (uint32_t)VS); ++s)
                mbar_wait_bounded(full + 8 * (KS + s), ((vs - 1 - s) / VS) & 1u, &never);
        }
        if (warp == kMmaWarp && issued.mma && elect_lane()) {
            mma_commit1(drain);
            mbar_wait_bounded(drain, 0, &never);
        }
        __syncwarp();
        __syncthreads();
    }
    tc_fence_after();
    if (warp == kAllocWarp) tmem_free1(tmem, 512);
    if (tid == 0 && abort_flag) atomicOr(a.status, kErrTimeout);
}

// dk and dv of a tile of 128 keys, over the queries of all heads that share them; everything transposed,
// a thread a key. The two warpgroups take 64 queries of a step each. p goes over the scores and dz
// over dp; the tensor cores form dv and the next scores while the warps are at dz, dk and the next dp while
// they are at the next p. The keys' shared memory is free behind the unit's last scores; dk and dv go out
// through the values'.
template <int DP>
__device__ __forceinline__ void attn_dkv(const CUtensorMap& mdo, const CUtensorMap& mq, const CUtensorMap& mk,
                                         const CUtensorMap& mv, const CUtensorMap& mdk, const CUtensorMap& mdv,
                                         const AttnBwdArgs& a, int cta) {
    using S = AttnShape<DP, kAttnDkv>;
    constexpr int ST = S::kStages, SS = 2;  // slots of row statistics
    extern __shared__ __align__(1024) unsigned char bwd_shared[];
    uint64_t* bars = reinterpret_cast<uint64_t*>(bwd_shared + S::kBars);  // 2 * ST + 2 * SS + 13 of them, in 312 bytes
    static_assert((2 * ST + 2 * SS + 13) * 8 <= 312, "barriers and two words in 320 bytes");
    uint32_t* tmem_word = reinterpret_cast<uint32_t*>(bwd_shared + S::kBars + 312);
    volatile int& abort_flag = *reinterpret_cast<volatile int*>(bwd_shared + S::kBars + 316);
    // lse (units of log 2) and delta of a step's queries: [SS][2][kAttnTile]
    float* stats = reinterpret_cast<float*>(bwd_shared + S::kBars + 320);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t kt = smem_addr(bwd_shared), ring = kt + 2 * S::kTile;
    const uint32_t full = smem_addr(bars), empty = full + 8 * ST, sready = empty + 8 * ST, sfree = sready + 8 * SS, kfull = sfree + 8 * SS, vfull = kfull + 8;
    const uint32_t kempty = vfull + 8, vempty = kempty + 8, sfull = vempty + 8, pready = sfull + 8, pfull = pready + 8, dsready = pfull + 8;
    const uint32_t done = dsready + 8, freed = done + 8, tail = freed + 8, drain = tail + 8;
    if (tid == 0) {
        for (int i = 0; i < ST; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(empty + 8 * i, 1);
        }
        for (int i = 0; i < SS; ++i) {
            mbar_init(sready + 8 * i, 32);
            mbar_init(sfree + 8 * i, 8);
        }
        mbar_init(kfull, 1);
        mbar_init(kempty, 1);
        mbar_init(vfull, 1);
        mbar_init(vempty, 9);  // the products that read them, and the warps that sent dk and dv out through them
        mbar_init(sfull, 1);
        mbar_init(pready, 8);
        mbar_init(pfull, 1);
        mbar_init(dsready, 8);
        mbar_init(done, 1);
        mbar_init(freed, 8);
        mbar_init(tail, 1);
        mbar_init(drain, 1);
        abort_flag = 0;
        mbar_fence_init();
        tma_prefetch_map(&mdo);
        tma_prefetch_map(&mq);
        tma_prefetch_map(&mk);
        tma_prefetch_map(&mv);
        tma_prefetch_map(&mdk);
        tma_prefetch_map(&mdv);
    }
    if (warp == kAllocWarp) tmem_alloc1(smem_addr(tmem_word), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_trigger();
    const uint32_t tmem = *tmem_word, dp_tmem = tmem + 128, dv_tmem = tmem + 256, dk_tmem = tmem + 384;
    pdl_wait();
    AttnIssued issued;
    const int role = __shfl_sync(0xFFFFFFFFu, warp, 0);
    // n steps of a unit, from step t0 of it on; `all` is the unit's: `tiles` of queries, from the first
    // that sees one of the keys, for every head of the group.
    AttnWalk walk(a.list, cta);
    int first = 0, tiles = 0, t0 = 0, n = 0, all = 0;
    auto next = [&]() {
        if (!walk.next()) return false;
        first = max(0, walk.it.shift) / kAttnTile;
        tiles = max(0, (walk.it.others + kAttnTile - 1) / kAttnTile - first);
        all = tiles * a.group;
        walk.steps(all, true);
        t0 = walk.t0;
        n = walk.t1 - t0;
        return true;
    };
    const AttnItem& it = walk.it;
    const int& head = walk.head;

    if (role == kLoadWarp) {
        bool live = true;
        uint32_t slots = 0;
        fence_async_proxy();
        while (live && next()) {
            walk.fetch();
            if (n == 0) continue;
            live = __all_sync(0xFFFFFFFFu, issued.pair == 0 || mbar_wait_bounded(kempty, (issued.pair - 1) & 1u, &abort_flag));
            if (!live) break;
            if (elect_lane()) {
                mbar_arrive_expect_tx(kfull, S::kTile);
                load_tile<DP>(kt, &mk, head, it.row0, kfull);
            }
            ++issued.pair;
            for (int j = 0; j < n && live; ++j, ++slots) {
                const int step = walk.tile(t0 + j), h = head * a.group + step / tiles, t = first + step % tiles;
                const int row = it.other0 + t * kAttnTile, left = it.others - t * kAttnTile;
                // Both are operands of sums over the queries: what follows the segment, and queries that see no
                // key (a gradient of theirs may be infinite or NaN, where a loss divides by what they saw).
                const int unseen = it.unseen - t * kAttnTile;
                const bool cut = (left < kAttnTile && !it.end) || unseen > 0;
                float stat[8];  // four rows' lse, then their delta
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int q = (lane + 32 * i) & (kAttnTile - 1);
                    const bool in = q < left && ADALN_IN_ATTN(row >= 0 && (int64_t)row + q < a.Rq && h < a.Hq);
                    stat[i] = in ? __ldcg((i < 4 ? a.lse2 : a.delta) + (int64_t)h * a.Rq + row + q) : 0.0f;
                }
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const uint32_t s = issued.ring % ST, l = issued.ring / ST;
                    live = __all_sync(0xFFFFFFFFu, l == 0 || mbar_wait_bounded(empty + 8 * s, (l - 1) & 1u, &abort_flag));
                    if (!live) break;
                    const uint32_t dst = ring + s * S::kTile;
                    if (elect_lane()) {
                        const uint32_t bar = cut ? tail : full + 8 * s;
                        mbar_arrive_expect_tx(bar, S::kTile);
                        load_tile<DP>(dst, x ? &mdo : &mq, h, row, bar);
                    }
                    if (x == 1) {
                        if (slots >= SS)
                            live = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(sfree + 8 * (slots % SS), (slots / SS - 1) & 1u, &abort_flag));
                        float* dst2 = stats + slots % SS * 2 * kAttnTile;
#pragma unroll
                        for (int i = 0; i < 8; ++i) dst2[lane + 32 * i] = stat[i];
                        mbar_arrive(sready + 8 * (slots % SS));
                    }
                    if (cut) {
                        live = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(tail, issued.tail & 1u, &abort_flag));
                        ++issued.tail;
                        if (live) {
                            if (unseen > 0) zero_rows<DP>(dst, 0, min(unseen, kAttnTile), lane);
                            if (left < kAttnTile) zero_rows<DP>(dst, left, kAttnTile, lane);
                            fence_shared_async();
                        }
                        __syncwarp();
                        if (elect_lane()) mbar_arrive(full + 8 * s);
                    }
                    ++issued.ring;
                    if (!live) break;
                    if (n > 1 ? x == 0 && j == 1 : x == 1) {  // the values behind what goes before them
                        live = __all_sync(0xFFFFFFFFu,
                                          issued.pair2 == 0 || mbar_wait_bounded(vempty, (issued.pair2 - 1) & 1u, &abort_flag));
                        if (!live) break;
                        if (elect_lane()) {
                            mbar_arrive_expect_tx(vfull, S::kTile);
                            load_tile<DP>(kt + S::kTile, &mv, head, it.row0, vfull);
                        }
                        ++issued.pair2;
                    }
                }
            }
        }
    } else if (role == kMmaWarp) {
        bool live = true;
        uint32_t used = 0, laps = 0, steps = 0;
        auto wait = [&](uint32_t bar, uint32_t parity) {
            live = live && __all_sync(0xFFFFFFFFu, mbar_wait_bounded(bar, parity & 1u, &abort_flag));
            return live;
        };
        auto tile = [&](uint32_t x) { return ring + x % ST * S::kTile; };
        auto loaded = [&](uint32_t x) { return wait(full + 8 * (x % ST), x / ST); };
        auto scores = [&](int j) {
            if (elect_lane()) {
                mma_rows<DP>(tmem, kt, tile(used + 2 * j), a.d);
                mma_commit1(sfull);
            }
        };
        auto dprobs = [&](int j) {
            if (elect_lane()) {
                mma_rows<DP>(dp_tmem, kt + S::kTile, tile(used + 2 * j + 1), a.d);
                mma_commit1(pfull);
            }
        };
        while (live && next()) {
            walk.fetch();
            if (n == 0) continue;
            if (!wait(kfull, laps) || !loaded(used)) break;
            tc_fence_after();
            issued.mma = true;
            scores(0);
            if (n == 1 && elect_lane()) mma_commit1(kempty);
            if (!wait(vfull, laps) || !loaded(used + 1)) break;
            tc_fence_after();
            dprobs(0);
            if (laps > 0 && !wait(freed, laps - 1)) break;
            for (int j = 0; j < n; ++j) {
                if (!wait(pready, steps + j)) break;
                tc_fence_after();
                if (elect_lane()) {
                    mma_cols(dv_tmem, tmem, tmem + 64, tile(used + 2 * j + 1), a.d, j > 0);
                    mma_commit1(empty + 8 * ((used + 2 * j + 1) % ST));
                }
                if (j + 1 < n) {
                    if (!loaded(used + 2 * j + 2)) break;
                    tc_fence_after();
                    scores(j + 1);
                    if (j + 2 == n && elect_lane()) mma_commit1(kempty);  // behind the unit's last scores
                }
                if (!wait(dsready, steps + j)) break;
                tc_fence_after();
                if (elect_lane()) {
                    mma_cols(dk_tmem, dp_tmem, dp_tmem + 64, tile(used + 2 * j), a.d, j > 0);
                    mma_commit1(empty + 8 * ((used + 2 * j) % ST));
                }
                if (j + 1 < n) {
                    if (!loaded(used + 2 * j + 3)) break;
                    tc_fence_after();
                    dprobs(j + 1);
                }
            }
            if (!live) break;
            if (elect_lane()) {
                mma_commit1(done);
                mma_commit1(vempty);
            }
            used += 2 * n;
            steps += n;
            ++laps;
        }
    } else if (role < kMmaWarp) {
        const int wg = warp >> 2, c = (warp & 3) * 32 + lane;  // this thread's key of the tile
        const uint32_t lanes = ((uint32_t)(warp & 3) << 21) + 64 * wg;
        const f2r s2 = p_splat(a.scale * kLog2e);
        const uint32_t out_buf = (DP == 64 ? kt + S::kTiles : kt + S::kTile) + warp * kAttnOut;
        uint32_t steps = 0, laps = 0;
        bool live = true;
        while (live && next()) {
            const int from = max(0, it.shift + c);  // the first query that sees this key
            for (int j = 0; j < n; ++j, ++steps) {
                const int q0 = (first + walk.tile(t0 + j) % tiles) * kAttnTile + 64 * wg;
                const bool cut = __any_sync(0xFFFFFFFFu, from > q0 || it.others < q0 + 64);
                const uint32_t slot = smem_addr(stats) + steps % SS * 1024 + 256 * wg;
                live = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(sready + 8 * (steps % SS), (steps / SS) & 1u, &abort_flag) &&
                                                   mbar_wait_bounded(sfull, steps & 1u, &abort_flag));
                if (!live) break;
                tc_fence_after();
                float p[64];
                tmem_ld64(tmem + lanes, p);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const uint4 l = lds128(slot + 16 * i);
                    const f2r x = p_fma(p_make(p[4 * i], p[4 * i + 1]), s2, p_make(-__uint_as_float(l.x), -__uint_as_float(l.y)));
                    const f2r y = p_fma(p_make(p[4 * i + 2], p[4 * i + 3]), s2, p_make(-__uint_as_float(l.z), -__uint_as_float(l.w)));
                    p[4 * i] = exp2_ftz(p_get(x).x);
                    p[4 * i + 1] = exp2_ftz(p_get(x).y);
                    p[4 * i + 2] = exp2_ftz(p_get(y).x);
                    p[4 * i + 3] = exp2_ftz(p_get(y).y);
                }
                if (cut) mask64(p, from - q0, it.others - q0);
                uint32_t w[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) w[i] = pack2(p[2 * i], p[2 * i + 1]);
                tmem_st32(tmem + lanes, w);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(pready);
                live = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(pfull, steps & 1u, &abort_flag));
                if (!live) break;
                tc_fence_after();
                float dp[64];
                tmem_ld64(dp_tmem + lanes, dp);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const uint4 l = lds128(slot + 512 + 16 * i);
                    const f2r x = p_mul(p_sub(p_make(dp[4 * i], dp[4 * i + 1]), p_make(__uint_as_float(l.x), __uint_as_float(l.y))),
                                        p_make(p[4 * i], p[4 * i + 1]));
                    const f2r y = p_mul(p_sub(p_make(dp[4 * i + 2], dp[4 * i + 3]), p_make(__uint_as_float(l.z), __uint_as_float(l.w))),
                                        p_make(p[4 * i + 2], p[4 * i + 3]));
                    dp[4 * i] = p_get(x).x;
                    dp[4 * i + 1] = p_get(x).y;
                    dp[4 * i + 2] = p_get(y).x;
                    dp[4 * i + 3] = p_get(y).y;
                }
                if (cut) mask64(dp, from - q0, it.others - q0);  // dz itself: dp and delta may be infinite or NaN
#pragma unroll
                for (int i = 0; i < 32; ++i) w[i] = pack2(dp[2 * i], dp[2 * i + 1]);
                tmem_st32(dp_tmem + lanes, w);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(dsready);
                    mbar_arrive(sfree + 8 * (steps % SS));
                }
            }
            if (!live) break;
            walk.fetch();
            // One warpgroup writes dv, the other dk.
            const int64_t at = (int64_t)it.row0 + c;
            const bool in = c < it.rows && ADALN_IN_ATTN(at >= 0 && head < a.Hq / a.group);
            __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(wg ? a.dx : a.dv) + at * (wg ? a.dx_ld : a.dv_ld) +
                                 (int64_t)head * a.d;
            if (n == 0) {
                if (in && all == 0) store_zeros(out, 0, a.d, a.d);
                continue;
            }
            live = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(done, laps & 1u, &abort_flag));
            if (!live) break;
            tc_fence_after();
            const uint32_t src = (wg ? dk_tmem : dv_tmem) + ((uint32_t)(warp & 3) << 21);
            const float f = wg ? a.scale : 1.0f;
            if (walk.whole(all)) {
                const int rows = min(32, it.rows - (warp & 3) * 32);
#pragma unroll 1
                for (int x = 0; x < a.d && rows > 0; x += 64) {
                    uint32_t w[32];
                    read64(src + x, f, w);
                    tma_store_read();  // the first half, out of the buffer
                    __syncwarp();
                    out64(wg ? &mdk : &mdv, out_buf, w, x, head, it.row0 + (warp & 3) * 32, rows, out, a.d, lane);
                }
                tma_store_read();
            } else {
                float* piece = a.part + ((int64_t)walk.slot() * 2 + wg) * a.slot_rows * a.d;
#pragma unroll 1
                for (int x = 0; x < a.d; x += 32) {
                    float o[32];
                    tmem_ld32(src + x, o);
                    if (in && ADALN_IN_ATTN(c < a.slot_rows)) store_piece32(piece, c, a.slot_rows, x, a.d, o);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(freed);
                mbar_arrive(vempty);
            }
            ++laps;
        }
        tma_store_wait();
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (__builtin_expect(abort_flag, 0)) {
        volatile int never = 0;
        if (warp == kLoadWarp && lane == 0) {
            if (issued.pair) mbar_wait_bounded(kfull, (issued.pair - 1) & 1u, &never);
            if (issued.pair2) mbar_wait_bounded(vfull, (issued.pair2 - 1) & 1u, &never);
            if (issued.tail) mbar_wait_bounded(tail, (issued.tail - 1) & 1u, &never);
            for (uint32_t s = 0; s < min(issued.ring, (uint32_t)ST); ++s)
                mbar_wait_bounded(full + 8 * s, ((issued.ring - 1 - s) / ST) & 1u, &never);
        }
        if (warp == kMmaWarp && issued.mma && elect_lane()) {
            mma_commit1(drain);
            mbar_wait_bounded(drain, 0, &never);
        }
        __syncwarp();
        __syncthreads();
    }
    tc_fence_after();
    if (warp == kAllocWarp) tmem_free1(tmem, 512);
    if (tid == 0 && abort_flag) atomicOr(a.status, kErrTimeout);
}

// Both gradients in one launch: with few units the two run side by side (17 + 130 + 5 + 1 rows, 4 heads:
// 23.1 us one after the other, 16.7 together), with many one begins on the SMs that the other leaves.
template <int DP>
__global__ void __launch_bounds__(kAttnThreads, 1) attn_bwd_kernel(const __grid_constant__ CUtensorMap mdo,
                                                                const __grid_constant__ CUtensorMap mq,
                                                                const __grid_constant__ CUtensorMap mk,
                                                                const __grid_constant__ CUtensorMap mv,
                                                                const __grid_constant__ CUtensorMap mdq,
                                                                const __grid_constant__ CUtensorMap mdk,
                                                                const __grid_constant__ CUtensorMap mdv,
                                                                const __grid_constant__ AttnBwdArgs dkv,
                                                                const __grid_constant__ AttnBwdArgs dq) {
    if ((int)blockIdx.x < dkv.list.ctas)
        attn_dkv<DP>(mdo, mq, mk, mv, mdk, mdv, dkv, blockIdx.x);
    else
        attn_dq<DP>(mdo, mq, mk, mv, mdq, dq, (int)blockIdx.x - dkv.list.ctas);
}

// ---- launches ------------------------------------------------------------------------------
namespace {

unsigned cap(int64_t want, int64_t most) { return (unsigned)(want < 1 ? 1 : want < most ? want : most); }

// Lets kernel variant `which` use its shared memory, once a device. `regs`: what its threads must have been
// given at launch (setmaxnreg would wait forever for more).
cudaError_t allow_attn_smem(const void* fn, int which, size_t bytes, int regs = 0) {
    constexpr int kDevices = 64;
    static std::atomic<bool> done[kDevices][4];
    int dev = 0;
    if (cudaError_t e = cudaGetDevice(&dev)) return e;
    if (dev >= 0 && dev < kDevices && done[dev][which].load(std::memory_order_acquire)) return cudaSuccess;
    cudaFuncAttributes attr{};
    cudaError_t e = cudaFuncGetAttributes(&attr, fn);
    if (e == cudaSuccess && attr.numRegs < regs) e = cudaErrorInvalidKernelImage;
    if (e == cudaSuccess) e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess && dev >= 0 && dev < kDevices) done[dev][which].store(true, std::memory_order_release);
    return e;
}

// Tensor map of rows of H heads of d elements: boxes of 64 elements of one head by 128 rows, 128-byte
// swizzle; what is past d, or past the last row, arrives as zeros.
bool rows_map(CUtensorMap* m, const AttnRows& x, int d, int box_rows = kAttnTile) {
    const TensorMapEncode encode = tensor_map_encode();
    if (!encode) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)x.H, (cuuint64_t)x.R};
    const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)x.ld * 2};
    const cuuint32_t box[3] = {64u, 1u, (cuuint32_t)box_rows}, one[3] = {1, 1, 1};
    return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(x.p), dims, strides, box, one,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

cudaError_t launch_attn_plan(const AttnPlanArgs& plan, cudaStream_t stream) {
    AttnPlanArgs p = plan;
    void* params[] = {&p};
    return launch_dependent(reinterpret_cast<const void*>(&attn_plan_kernel), dim3(1), dim3(kPlanThreads), params, 0, stream);
}

cudaError_t launch_attn_prepare(const AttnPlanArgs& plan, const AttnDeltaArgs& delta, int sms, cudaStream_t stream) {
    AttnPlanArgs p = plan;
    AttnDeltaArgs d = delta;
    int lists = p.list[1].items ? 2 : 1;
    unsigned ctas = d.Rq > 0 ? cap((d.Rq * ((d.Hq + 1) / 2) + 63) / 64, 4 * (int64_t)sms) : 0;
    // Segments of equal lengths tell whether any row sees few keys; tables are on the device.
    const bool few = ctas && (p.t.causal || p.t.Rk <= kAttnFewKeys * p.t.nseg || (p.t.nseg > 1 && p.t.cu_k));
    d.few = few ? (int)cap((p.t.causal ? p.t.nseg * kAttnFewBlocks : (d.Rq + 15) / 16) * d.Hq / 16 + 1, 4 * (int64_t)sms) : 0;
    ctas += d.few;
    void* params[] = {&p, &d, &lists};
    return launch_dependent(reinterpret_cast<const void*>(&attn_prepare_kernel), dim3(lists + ctas), dim3(kPlanThreads), params,
                            0, stream);
}

cudaError_t launch_attn_fwd(const AttnFwdArgs& args, const AttnRows& q, const AttnRows& k, const AttnRows& v,
                            cudaStream_t stream) {
    AttnFwdArgs a = args;
    CUtensorMap mq, mk, mv, mo;
    // Without keys nothing is loaded; the maps still have to be maps.
    if (!rows_map(&mq, q, a.d) || !rows_map(&mk, k.R ? k : q, a.d) || !rows_map(&mv, k.R ? v : q, a.d) ||
        !rows_map(&mo, {a.o, q.R, a.o_ld, q.H}, a.d, 32))
        return cudaErrorInvalidValue;
    const bool wide = a.d > 64;
    const void* fn = wide ? reinterpret_cast<const void*>(&attn_fwd_kernel<128>)
                          : reinterpret_cast<const void*>(&attn_fwd_kernel<64>);
    const size_t smem = wide ? AttnShape<128, kAttnFwd>::kSmem : AttnShape<64, kAttnFwd>::kSmem;
    if (cudaError_t e = allow_attn_smem(fn, wide ? 1 : 0, smem, kFwdRegs)) return e;
    void* params[] = {&mq, &mk, &mv, &mo, &a};
    return launch_dependent(fn, dim3((unsigned)a.list.ctas), dim3(kAttnThreads), params, smem, stream);
}

cudaError_t launch_attn_join(const AttnJoinArgs& args, bool bwd, cudaStream_t stream) {
    AttnJoinArgs a = args;
    void* params[] = {&a};
    const void* fn = bwd ? reinterpret_cast<const void*>(&attn_join_kernel<true>)
                         : reinterpret_cast<const void*>(&attn_join_kernel<false>);
    const int ctas = std::max(a.list[0].ctas, bwd ? a.list[1].ctas : 0);
    return launch_dependent(fn, dim3((unsigned)ctas, 8, bwd ? 2 : 1), dim3(256), params, 0, stream);
}

cudaError_t launch_attn_bwd(const AttnBwdArgs& dkv_args, const AttnBwdArgs& dq_args, const AttnRows& dout,
                            const AttnRows& q, const AttnRows& k, const AttnRows& v, cudaStream_t stream) {
    AttnBwdArgs dkv = dkv_args, dq = dq_args;
    const int d = dkv.list.ctas ? dkv.d : dq.d;
    CUtensorMap mdo, mq, mk, mv, mdq{}, mdk{}, mdv{};
    // A side without rows is not loaded; the maps still have to be maps.
    const AttnRows some = q.R ? q : k;
    if (!rows_map(&mdo, q.R ? dout : some, d) || !rows_map(&mq, some, d) || !rows_map(&mk, k.R ? k : some, d) ||
        !rows_map(&mv, k.R ? v : some, d) || !rows_map(&mdq, dq.list.ctas ? AttnRows{dq.dx, q.R, dq.dx_ld, q.H} : some, d, 32) ||
        !rows_map(&mdk, dkv.list.ctas ? AttnRows{dkv.dx, k.R, dkv.dx_ld, k.H} : some, d, 32) ||
        !rows_map(&mdv, dkv.list.ctas ? AttnRows{dkv.dv, k.R, dkv.dv_ld, k.H} : some, d, 32))
        return cudaErrorInvalidValue;
    const bool wide = d > 64;
    const void* fn = wide ? reinterpret_cast<const void*>(&attn_bwd_kernel<128>)
                          : reinterpret_cast<const void*>(&attn_bwd_kernel<64>);
    const size_t smem = wide ? AttnShape<128, kAttnDkv>::kSmem : AttnShape<64, kAttnDkv>::kSmem;
    static_assert(AttnShape<128, kAttnDkv>::kSmem == AttnShape<128, kAttnDq>::kSmem &&
                      AttnShape<64, kAttnDkv>::kSmem == AttnShape<64, kAttnDq>::kSmem, "one launch holds both");
    if (cudaError_t e = allow_attn_smem(fn, wide ? 3 : 2, smem)) return e;
    void* params[] = {&mdo, &mq, &mk, &mv, &mdq, &mdk, &mdv, &dkv, &dq};
    return launch_dependent(fn, dim3((unsigned)(dkv.list.ctas + dq.list.ctas)), dim3(kAttnThreads), params, smem, stream);
}

cudaError_t debug_word_attn(uint32_t* out, bool reset) { return debug_word(out, reset); }

}  // namespace adaln
