// Key blocks and pages: block means, block selection, page copies.
//
// Means.  A block's mean is f32(sum / n) with the sum in f64.  A bf16 value
// has 8 significant bits, so the sum of up to 256 of them is exact in f64
// while their exponents span at most 37 binades: the order of the additions
// does not show, and a mean has the same bits wherever it is computed.
//
// Selection.  score = sum_d qmean[d] * kmean[d] in f64; the `keep` largest
// blocks of each (head, query group), ties to the lowest index.  Scores in
// f64 leave two blocks at the border in the wrong order only when their
// scores agree to about 1e-15.
#include <cooperative_groups.h>

#include "pv_internal.h"

namespace cg = cooperative_groups;

namespace pv {
namespace {

constexpr int kPoolThreads = 256;
constexpr int kPoolWarps = kPoolThreads / 32;

// Adds a row (eight bf16 columns) to f64 sums.
__device__ __forceinline__ void add_row(double* a, const uint4& v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        a[2 * i] += (double)__uint_as_float(w[i] << 16);
        a[2 * i + 1] += (double)__uint_as_float(w[i] & 0xFFFF0000u);
    }
}

// Sums of rows [r0, r1), at most kRows of them, over a strip of 64 columns by
// one warp: `strip` points at the strip's first column of row 0, rows are D
// apart.  Lanes 0..7 end with columns 8 lane .. 8 lane + 7.
template <int D, int kRows>
__device__ __forceinline__ void pool_strip(const bf16* strip, int r0, int r1, double* a) {
    constexpr int kLoads = kRows >= 32 ? 8 : (kRows + 3) / 4;   // in flight, four rows each
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int c = 0; c < 8; ++c) a[c] = 0.0;
#pragma unroll 1
    for (int r = r0 + lane / 8; r < r0 + kRows; r += 4 * kLoads) {
        uint4 v[kLoads];
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            v[i] = r + 4 * i < r1
                       ? __ldg(reinterpret_cast<const uint4*>(strip + (size_t)(r + 4 * i) * D) + (lane & 7))
                       : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < kLoads; ++i) add_row(a, v[i]);
    }
#pragma unroll
    for (int m = 8; m < 32; m *= 2)
#pragma unroll
        for (int c = 0; c < 8; ++c) a[c] += __shfl_xor_sync(0xffffffffu, a[c], m);
}

// kParts warps share the rows of each (block, strip).  Four: the fewest steps
// one after the other, for few blocks.  One: long streams of loads without a
// synchronisation, for many.  Bound by reading the keys.
template <int D, int kParts>
__global__ void __launch_bounds__(kPoolThreads, 3)
    summary_kernel(const __grid_constant__ SummaryParams p) {
    constexpr int kStrips = D / 64;
    constexpr int kPer = kPoolWarps / (kStrips * kParts);    // blocks of a CTA
    __shared__ double part[kParts > 1 ? kPoolWarps * 64 : 1];
    wait_for_stream();
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const int strip = warp / kParts % kStrips, share = warp % kParts;
    const long long idx = (long long)blockIdx.x * kPer + warp / (kStrips * kParts);
    const bool live = idx < (long long)p.n_items * p.heads;
    float* dst = nullptr;
    int rows = 0;
    double a[8];
    if (live) {
        const int head = (int)(idx / p.n_items), item = (int)(idx - (long long)head * p.n_items);
        int i = 0;
        while (i + 1 < p.n_runs && p.item0[i + 1] <= item) ++i;
        const int li = item - p.item0[i];
        const int seg = li / p.bps, blk = li - seg * p.bps;
        const long long ps =
            (long long)blockIdx.y * p.plane_segs + p.seg0[i] + (long long)head * p.head_segs + seg;
        rows = min(p.seg_len - blk * kKeyTile, kKeyTile);
        dst = p.means + (ps * p.bps + blk) * D + strip * 64;
        const bf16* src = p.k + (ps * p.seg_len + blk * kKeyTile) * D + strip * 64;
        pool_strip<D, kKeyTile / kParts>(src, share * (kKeyTile / kParts),
                                         min(rows, (share + 1) * (kKeyTile / kParts)), a);
    }
    if constexpr (kParts == 1) {
        if (live && lane < 8) {
            float m[8];
#pragma unroll
            for (int c = 0; c < 8; ++c) m[c] = (float)(a[c] / (double)rows);
            float4* d4 = reinterpret_cast<float4*>(dst) + lane * 2;
            d4[0] = make_float4(m[0], m[1], m[2], m[3]);
            d4[1] = make_float4(m[4], m[5], m[6], m[7]);
        }
    } else {
        if (live && lane < 8) {
#pragma unroll
            for (int c = 0; c < 8; ++c) part[warp * 64 + lane * 8 + c] = a[c];
        }
        __syncthreads();
        // the first warps of each (block, strip) add up its shares
        if (live && share < 2) {
            const int c = share * 32 + lane;
            double s = 0;
#pragma unroll
            for (int w = 0; w < kParts; ++w) s += part[(warp - share + w) * 64 + c];
            dst[c] = (float)(s / (double)rows);
        }
    }
}

// ------------------------------------------------------------------ select
constexpr int kSelThreads = kPoolThreads;
constexpr int kSelWarps = kPoolWarps;
constexpr int kCountBlocks = 256;   // one block per thread: order by counting
constexpr int kMaxClose = 512;      // blocks at the border that are scored again
constexpr uint32_t kForced = 0xFFFFC000u;   // keys of forced blocks, above +inf's

// Floating-point values as unsigned integers of the same order (-0 and +0
// equal, NaN lowest).
__device__ __forceinline__ unsigned long long order_key(double s) {
    if (!(s == s)) return 0;
    const long long b = __double_as_longlong(s + 0.0);
    return b < 0 ? ~(unsigned long long)b : (unsigned long long)b | 0x8000000000000000ull;
}
__device__ __forceinline__ uint32_t order_key(float s) {
    if (!(s == s)) return 0;
    const uint32_t b = __float_as_uint(s + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}

struct SelShared {
    int warp_a[kSelWarps], warp_b[kSelWarps];
    int hist[256];
    int bin, need, all;
    uint32_t edge;
    uint32_t norm2;                     // largest |kmean|^2 (its bits)
    int close[kMaxClose];               // blocks at the border
    unsigned long long key[kMaxClose];  // and their f64 scores
};

// Threshold of the `need` largest of n keys (radix select, eight bits at a
// time from the top): the keys whose upper bits exceed `prefix` are taken,
// and of those that equal it all (sh->all) or the first sh->need.
template <typename K>
__device__ void radix_threshold(const K* keys, int n, int need, SelShared* sh, int* shift_out,
                                K* prefix_out) {
    constexpr int kBits = sizeof(K) * 8;
    K prefix = 0;
    int shift = kBits;
    const int t = threadIdx.x;
    if (t == 0) {
        sh->need = need;
        sh->all = 0;
    }
    while (shift > 0) {
        shift -= 8;
        sh->hist[t] = 0;
        __syncthreads();
        for (int i = t; i < n; i += kSelThreads) {
            const K k = keys[i] >> shift;
            if (shift == kBits - 8 || (k >> 8) == prefix) atomicAdd(&sh->hist[(int)(k & 255)], 1);
        }
        __syncthreads();
        if (t < 32) {
            // lane l holds bins 255 - 8l down to 248 - 8l
            int c[8], sum = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) sum += c[i] = sh->hist[255 - 8 * t - i];
            int before = sum;
#pragma unroll
            for (int o = 1; o < 32; o *= 2) {
                const int v = __shfl_up_sync(0xffffffffu, before, o);
                if (t >= o) before += v;
            }
            before -= sum;
            const int want = sh->need;
            __syncwarp();
            if (before < want && before + sum >= want) {
                int left = want - before, i = 0;
                while (c[i] < left) left -= c[i++];
                sh->bin = 255 - 8 * t - i;
                sh->need = left;
                sh->all = c[i] == left;
            }
        }
        __syncthreads();
        prefix = (prefix << 8) | (K)sh->bin;
        if (sh->all) break;
    }
    *shift_out = shift;
    *prefix_out = prefix;
    __syncthreads();
}

// Position of this thread among the block's threads whose flag is set, and
// their number.  Ends with every thread past its reads of w.
__device__ __forceinline__ int block_rank(bool f, int* w, int* total) {
    const unsigned b = __ballot_sync(0xffffffffu, f);
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    if (lane == 0) w[warp] = __popc(b);
    __syncthreads();
    int before = 0, sum = 0;
#pragma unroll
    for (int i = 0; i < kSelWarps; ++i) {
        const int c = w[i];
        before += i < warp ? c : 0;
        sum += c;
    }
    *total = sum;
    __syncthreads();
    return before + __popc(b & ((1u << lane) - 1));
}

// The need-th largest of n keys.
__device__ uint32_t nth_key(const uint32_t* keys, int n, int need, SelShared* sh) {
    const int t = threadIdx.x;
    if (n <= kCountBlocks) {
        // the smallest key that fewer than `need` others exceed
        uint32_t mine = 0xFFFFFFFFu;
        if (t < n) {
            const uint32_t k = keys[t];
            const uint4* four = reinterpret_cast<const uint4*>(keys);   // zeros behind n
            int above = 0;
#pragma unroll 4
            for (int i = 0; i < (n + 3) / 4; ++i) {
                const uint4 o = four[i];
                above += (o.x > k) + (o.y > k) + (o.z > k) + (o.w > k);
            }
            if (above < need) mine = k;
        }
        mine = __reduce_min_sync(0xffffffffu, mine);
        if ((t & 31) == 0) atomicMin(&sh->edge, mine);
        __syncthreads();
        return sh->edge;
    }
    int shift;
    uint32_t prefix;
    radix_threshold(keys, n, need, sh, &shift, &prefix);
    if (shift == 0) return prefix;
    // every key of the last bin is among the `need`: the smallest of them
    uint32_t mine = 0xFFFFFFFFu;
    for (int i = t; i < n; i += kSelThreads)
        if (keys[i] >> shift == prefix) mine = min(mine, keys[i]);
    mine = __reduce_min_sync(0xffffffffu, mine);
    if ((t & 31) == 0) atomicMin(&sh->edge, mine);
    __syncthreads();
    return sh->edge;
}

// Ascending indices of the n_sel largest of n f64 keys, ties to the lowest.
__device__ void write_top(const unsigned long long* keys, int n, int n_sel, SelShared* sh, int* out) {
    int shift;
    unsigned long long prefix;
    radix_threshold(keys, n, n_sel, sh, &shift, &prefix);
    const bool all = sh->all != 0;
    const int need = sh->need;
    int base = 0, eq_base = 0;
    for (int i0 = 0; i0 < n; i0 += kSelThreads) {
        const int i = i0 + threadIdx.x;
        const unsigned long long k = i < n ? keys[i] >> shift : 0;
        const bool gt = i < n && k > prefix;
        const bool eq = i < n && k == prefix;
        int eqs, cnt;
        const int er = eq_base + block_rank(eq, sh->warp_a, &eqs);
        const bool f = gt || (eq && (all || er < need));
        const int pos = base + block_rank(f, sh->warp_b, &cnt);
        if (f) out[pos] = i;
        base += cnt;
        eq_base += eqs;
    }
}

// The n_sel best of n blocks, as ascending indices; -1 up to keep.  keys
// holds f32 scores, each finite and off by at most `err` unless that is
// infinite, on entry, f64 scores if they are needed.  Blocks whose f32 score is more than 2 err above the n_sel-th
// largest one are among the best whatever the errors, those more than 2 err
// below are not, and the few between (seldom more than one) are scored in
// f64 by score(b), eight lanes of a warp to a block.
template <typename Score>
__device__ void choose(unsigned long long* keys64, int n, int n_sel, int keep, float err,
                       SelShared* sh, int* out, const Score& score) {
    uint32_t* keys = reinterpret_cast<uint32_t*>(keys64);
    const int t = threadIdx.x, sub = t / 8;   // 32 groups of eight lanes
    const uint32_t edge = nth_key(keys, n, n_sel, sh);
    // taken: keys from `above` on; close: keys from `from` up to it
    uint32_t above, from;
    if (edge >= kForced) {                    // forced blocks alone
        above = from = edge;
    } else if (!(err < INFINITY)) {           // f32 tells nothing: every unforced block in f64
        above = kForced;
        from = 0;
    } else {
        const float at = key_value(edge);
        above = min(order_key(__fadd_ru(at, 2.f * err)), kForced - 1) + 1;
        from = order_key(__fadd_rd(at, -2.f * err));
    }
    int taken = 0, close = 0;
    for (int i0 = 0; i0 < n; i0 += kSelThreads) {
        const int i = i0 + t;
        const uint32_t k = i < n ? keys[i] : 0;
        const bool c = i < n && k >= from && k < above;
        taken += __syncthreads_count(i < n && k >= above);
        int cnt;
        const int pos = close + block_rank(c, sh->warp_a, &cnt);
        if (c && pos < kMaxClose) sh->close[pos] = i;
        close += cnt;
    }
    __syncthreads();
    if (taken + close > n_sel) {
        if (close > kMaxClose) {
            // too close to call (equal blocks, sums beyond f32): all in f64;
            // forced blocks keep their rank
            // (32 blocks at a time from the last one down: a block's f64 key
            // covers f32 keys behind its own, which have been read)
            for (int b0 = (n - 1) / 32 * 32; b0 >= 0; b0 -= 32) {
                const int b = b0 + sub;
                const uint32_t was = b < n ? keys[b] : 0;
                const double s = score(min(b, n - 1));
                __syncthreads();
                if (b < n && (t & 7) == 0)
                    keys64[b] = was >= kForced ? ~0ull : order_key(s);
                __syncthreads();
            }
            write_top(keys64, n, n_sel, sh, out);
            for (int i = n_sel + t; i < keep; i += kSelThreads) out[i] = -1;
            return;
        }
        for (int j0 = 0; j0 < close; j0 += 32) {
            const int j = j0 + sub;
            const double s = score(sh->close[min(j, close - 1)]);
            if (j < close && (t & 7) == 0) sh->key[j] = order_key(s);
        }
        __syncthreads();
        for (int j = t; j < close; j += kSelThreads) {
            const unsigned long long k = sh->key[j];
            int ahead = 0;
            for (int i = 0; i < close; ++i) {
                const unsigned long long o = sh->key[i];
                ahead += o > k || (o == k && i < j);
            }
            keys[sh->close[j]] = ahead < n_sel - taken ? 0xFFFFFFFFu : 0u;
        }
        __syncthreads();
        from = above;     // now marked
    }
    int base = 0;
    for (int i0 = 0; i0 < n; i0 += kSelThreads) {
        const int i = i0 + t;
        const bool f = i < n && keys[i] >= from;
        int cnt;
        const int pos = base + block_rank(f, sh->warp_b, &cnt);
        if (f) out[pos] = i;
        base += cnt;
    }
    for (int i = n_sel + t; i < keep; i += kSelThreads) out[i] = -1;
}

// A cluster of kCluster CTAs per (stream, head, query group).  Its CTAs share
// the group's rows (sums exchanged through distributed shared memory) and the
// blocks to score; the first one picks the top.
template <int D, int kCluster, typename Pages>
__global__ void __launch_bounds__(kSelThreads, 4)
    select_kernel(const __grid_constant__ SelectParams p, const __grid_constant__ Pages pages) {
    cg::cluster_group cl = cg::this_cluster();
    const int rank = kCluster > 1 ? (int)cl.block_rank() : 0;
    extern __shared__ __align__(16) unsigned long long keys64[];   // max_blocks
    constexpr int kStrips = D / 64;
    constexpr int kParts = kSelWarps / kStrips;       // warps that share a strip's rows
    constexpr int kShare = kQBlock / kCluster;        // rows of a CTA
    __shared__ double part[kParts * D];
    __shared__ double mine[D];                        // this CTA's sums
    __shared__ __align__(16) float qm[D];
    __shared__ SelShared sh;
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    const int item = blockIdx.x / kCluster;
    wait_for_stream();
    if (threadIdx.x == 0) {
        sh.norm2 = 0;
        sh.edge = 0xFFFFFFFFu;
    }
    int i = 0;
    while (i + 1 < p.n_streams && p.item0[i + 1] <= item) ++i;
    const int li = item - p.item0[i];
    const int n_q = p.n_q[i];
    const int groups = (n_q + kQBlock - 1) / kQBlock;
    const int head = li / groups, g = li - head * groups;

    // the group's mean query
    const int q0 = g * kQBlock, q1 = min(n_q, q0 + kQBlock);
    {
        const int strip = warp / kParts, share = warp % kParts;
        const bf16* q = p.q + (p.q_row0[i] + (long long)head * n_q) * D + strip * 64;
        const int r0 = q0 + rank * kShare + share * (kShare / kParts);
        double a[8];
        pool_strip<D, kShare / kParts>(q, r0, min(q1, r0 + kShare / kParts), a);
        if (lane < 8) {
#pragma unroll
            for (int c = 0; c < 8; ++c) part[share * D + strip * 64 + lane * 8 + c] = a[c];
        }
    }
    __syncthreads();
    double sum = 0;
    if (threadIdx.x < D) {
#pragma unroll
        for (int w = 0; w < kParts; ++w) sum += part[w * D + threadIdx.x];
    }
    if (kCluster > 1) {
        if (threadIdx.x < D) mine[threadIdx.x] = sum;
        cl.sync();
        if (threadIdx.x < D) {
            sum = 0;
#pragma unroll
            for (int r = 0; r < kCluster; ++r) sum += cl.map_shared_rank(mine, r)[threadIdx.x];
        }
    }
    if (threadIdx.x < D) qm[threadIdx.x] = (float)(sum / (double)(q1 - q0));
    __syncthreads();

    // f32 scores of this CTA's blocks, to the first CTA: eight lanes to a
    // block, each with every eighth run of four columns
    constexpr int kRuns = D / 32;
    const int l8 = lane & 7;
    float4 ql[kRuns];
#pragma unroll
    for (int c = 0; c < kRuns; ++c) ql[c] = reinterpret_cast<const float4*>(qm)[c * 8 + l8];
    uint32_t* keys = reinterpret_cast<uint32_t*>(keys64);
    uint32_t* dst = kCluster > 1 ? cl.map_shared_rank(keys, 0) : keys;
    const int n = p.kb.n_blocks[i];
    const long long hs = p.kb.seg0[i] + (long long)head * p.kb.head_segs;
    auto mean_of = [&](int b) {
        const int seg = segment_of(p.kb, b);
        const long long row = (hs + pages.page(p.kb, i, seg)) * p.kb.bps + (b - seg * p.kb.bps);
        return reinterpret_cast<const float4*>(p.means + row * D) + l8;
    };
    float norm2 = 0.f;
    for (int b0 = (rank * kSelWarps + warp) * 4; b0 < n; b0 += kCluster * kSelWarps * 4) {
        const int b = b0 + lane / 8;
        const float4* src = mean_of(min(b, n - 1));
        float4 m[kRuns];
#pragma unroll
        for (int c = 0; c < kRuns; ++c) m[c] = __ldg(src + c * 8);
        float2 s = make_float2(0.f, 0.f), k2 = make_float2(0.f, 0.f);
#pragma unroll
        for (int c = 0; c < kRuns; ++c) {
            const float2 lo = make_float2(m[c].x, m[c].y), hi = make_float2(m[c].z, m[c].w);
            s = __ffma2_rn(make_float2(ql[c].x, ql[c].y), lo, s);
            s = __ffma2_rn(make_float2(ql[c].z, ql[c].w), hi, s);
            k2 = __ffma2_rn(lo, lo, k2);
            k2 = __ffma2_rn(hi, hi, k2);
        }
        float score = s.x + s.y, len = k2.x + k2.y;
#pragma unroll
        for (int o = 4; o > 0; o /= 2) {
            score += __shfl_xor_sync(0xffffffffu, score, o);
            len += __shfl_xor_sync(0xffffffffu, len, o);
        }
        // NaN lengths count as infinite: the f64 scores decide
        norm2 = fmaxf(norm2, len == len ? len : INFINITY);
        if (l8 == 0 && b < n) {
            const bool forced = (b >= p.force0[i][0] && b < p.force1[i][0]) ||
                                (b >= p.force0[i][1] && b < p.force1[i][1]);
            dst[b] = forced ? kForced | (kMaxSelectBlocks - 1 - b) : order_key(score);
        }
    }
    const uint32_t most = __reduce_max_sync(0xffffffffu, __float_as_uint(norm2));
    if (lane == 0) atomicMax(kCluster > 1 ? cl.map_shared_rank(&sh.norm2, 0) : &sh.norm2, most);
    if (rank == 0 && threadIdx.x < 3) keys[n + threadIdx.x] = 0;   // read in fours
    if (kCluster > 1)
        cl.sync();
    else
        __syncthreads();
    if (rank != 0) return;

    // A score is rounded at most 2 * kRuns times along a lane's columns and
    // four times after, each time by 2^-24 of partial sums that |qmean| |kmean|
    // bounds; 2 * kRuns + 8 leaves room for the roundings of the lengths, the
    // small constants for squares and products that underflow.
    float q2 = 0.f;
#pragma unroll
    for (int c = 0; c < kRuns; ++c)
        q2 += ql[c].x * ql[c].x + ql[c].y * ql[c].y + ql[c].z * ql[c].z + ql[c].w * ql[c].w;
#pragma unroll
    for (int o = 4; o > 0; o /= 2) q2 += __shfl_xor_sync(0xffffffffu, q2, o);
    float err = (2 * kRuns + 8) * 0x1p-24f * (sqrtf(q2) + 1e-18f) *
                    (sqrtf(__uint_as_float(sh.norm2)) + 1e-18f) + 1e-36f;
    // From 2^100 on, and where a length is infinite or NaN, products or partial
    // sums may have overflowed and no f32 score is worth anything; below it
    // |qmean| |kmean| is under 2^121 and every f32 score is finite.
    if (!(err < 0x1p100f)) err = INFINITY;
    choose(keys64, n, min(p.keep, n), p.keep, err, &sh, p.blocks + (long long)item * p.keep,
           [&](int b) {
               const float4* src = mean_of(b);
               double s = 0;
#pragma unroll
               for (int c = 0; c < kRuns; ++c) {
                   const float4 m = __ldg(src + c * 8);
                   s = fma((double)ql[c].x, (double)m.x, s);
                   s = fma((double)ql[c].y, (double)m.y, s);
                   s = fma((double)ql[c].z, (double)m.z, s);
                   s = fma((double)ql[c].w, (double)m.w, s);
               }
#pragma unroll
               for (int o = 4; o > 0; o /= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
               return s;
           });
}

// ------------------------------------------------------------------ copies
constexpr int kCopyThreads = 256;
constexpr int kCopyVecs = 4;   // 16-byte vectors of a thread

// A CTA owns kCopyThreads * kCopyVecs vectors at one place of a segment (run)
// in one (region, plane, head) and makes every move there.  The moves of a
// compaction go down in ascending order, so that a move may write a segment
// that an earlier one has read.  A vector's place inside a segment is the
// same for all moves: one thread's program order is all the ordering they
// need.  Bound by HBM.
__global__ void __launch_bounds__(kCopyThreads)
    copy_kernel(const __grid_constant__ CopyParams p, const __grid_constant__ long long cta0_1,
                const __grid_constant__ long long cta0_2, int parts0, int parts2) {
    wait_for_stream();
    long long c = blockIdx.x;
    const int r = c >= cta0_2 ? 2 : c >= cta0_1 ? 1 : 0;
    c -= r == 2 ? cta0_2 : r == 1 ? cta0_1 : 0;
    const int parts = r == 2 ? parts2 : parts0;
    const long long ph = c / parts;                 // plane, head
    const int part = (int)(c - ph * parts);
    const long long plane = ph / p.heads;
    const int head = (int)(ph - plane * p.heads);
    const long long sb = p.seg_bytes[r];
    char* base = p.base[r] + (plane * p.plane_segs + (long long)head * p.head_segs) * sb;
    const long long len = sb * p.len;
    long long off[kCopyVecs];
    bool in[kCopyVecs];
#pragma unroll
    for (int u = 0; u < kCopyVecs; ++u) {
        off[u] = ((long long)part * kCopyThreads * kCopyVecs + u * kCopyThreads + threadIdx.x) * 16;
        in[u] = off[u] < len;
    }
    uint4 v[kCopyVecs];
    for (int i = 0; i < p.n; ++i) {
        if (i == 0 || !p.fan) {
            const char* s = base + p.src[i] * sb;
#pragma unroll
            for (int u = 0; u < kCopyVecs; ++u)
                if (in[u]) v[u] = *reinterpret_cast<const uint4*>(s + off[u]);
        }
        char* d = base + p.dst[i] * sb;
#pragma unroll
        for (int u = 0; u < kCopyVecs; ++u)
            if (in[u]) *reinterpret_cast<uint4*>(d + off[u]) = v[u];
    }
}

template <int D, int kCluster, typename Pages>
cudaError_t launch_select_c(const SelectParams& p, const Pages& pages, cudaStream_t s) {
    static std::atomic<unsigned long long> configured{0};
    cudaError_t e =
        smem_limit_once(select_kernel<D, kCluster, Pages>, kMaxSelectBlocks * 8, configured);
    if (e != cudaSuccess) return e;
    // (the list of a short sequence still has room for reads in fours)
    const size_t smem = std::max<size_t>(32, (size_t)p.max_blocks * 8);
    return launch_early(select_kernel<D, kCluster, Pages>, (unsigned)p.n_items * kCluster,
                        kSelThreads, smem, kCluster, s, p, pages);
}

template <int D, typename Pages>
cudaError_t launch_select_d(const SelectParams& p, const Pages& pages, cudaStream_t s) {
    // few items: as many CTAs to each as still get an SM of their own, for
    // latency (24 items of 313 blocks: 8.0 us with four, 11.1 with one); many
    // items keep the GPU busy by themselves (1,752 items of 145 blocks: 38.7 us
    // with one CTA each, 56 with two)
    if (p.n_items * 8 <= 148) return launch_select_c<D, 8>(p, pages, s);
    if (p.n_items * 4 <= 148) return launch_select_c<D, 4>(p, pages, s);
    if (p.n_items * 2 <= 148) return launch_select_c<D, 2>(p, pages, s);
    return launch_select_c<D, 1>(p, pages, s);
}

template <int D, int kParts>
cudaError_t launch_summary_p(const SummaryParams& p, cudaStream_t s) {
    constexpr int kPer = kPoolWarps / (D / 64 * kParts);
    const long long ctas = ((long long)p.n_items * p.heads + kPer - 1) / kPer;
    if (ctas >= (1LL << 31)) return cudaErrorInvalidConfiguration;
    return launch_early(summary_kernel<D, kParts>, dim3((unsigned)ctas, p.planes), kPoolThreads, 0,
                        1, s, p);
}
template <int D>
cudaError_t launch_summary_d(const SummaryParams& p, cudaStream_t s) {
    // 168 blocks of 128 x 128: 3.1 us with four warps to a strip, 5.1 with one;
    // 3,480 blocks: 24.6 and 22.5 us
    const bool few = (long long)p.n_items * p.heads * p.planes <= 4 * 148;
    return few ? launch_summary_p<D, 4>(p, s) : launch_summary_p<D, 1>(p, s);
}

}  // namespace

cudaError_t launch_summary(const SummaryParams& p, cudaStream_t s) {
    return p.head_dim == 128 ? launch_summary_d<128>(p, s) : launch_summary_d<64>(p, s);
}

cudaError_t launch_select(const SelectParams& p, const PageTable* pages, cudaStream_t s) {
    if (pages)
        return p.head_dim == 128 ? launch_select_d<128>(p, *pages, s)
                                 : launch_select_d<64>(p, *pages, s);
    return p.head_dim == 128 ? launch_select_d<128>(p, FixedRows{}, s)
                             : launch_select_d<64>(p, FixedRows{}, s);
}

cudaError_t launch_copy(const CopyParams& p, cudaStream_t s) {
    constexpr long long per = (long long)kCopyThreads * kCopyVecs * 16;
    long long parts[3] = {0, 0, 0}, cta0[4] = {0, 0, 0, 0};
    for (int r = 0; r < 3; ++r) {
        if (r < p.n_regions) parts[r] = (p.seg_bytes[r] * p.len + per - 1) / per;
        cta0[r + 1] = cta0[r] + parts[r] * p.planes * p.heads;
    }
    if (cta0[3] >= (1LL << 31) || cta0[3] <= 0) return cudaErrorInvalidConfiguration;
    return launch_early(copy_kernel, (unsigned)cta0[3], kCopyThreads, 0, 1, s, p, cta0[1], cta0[2],
                        (int)parts[0], (int)std::max(1LL, parts[2]));
}

}  // namespace pv
