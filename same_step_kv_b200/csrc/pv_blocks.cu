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
#ifndef PV_LB
#define PV_LB 3
#endif
#ifndef PV_SLB
#define PV_SLB 3
#endif
#ifndef PV_QS
#define PV_QS 0
#endif

namespace cg = cooperative_groups;

namespace pv {
namespace {

constexpr int kPoolThreads = 256;
constexpr int kPoolWarps = kPoolThreads / 32;

__device__ __forceinline__ float2 bf16_pair(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

// Adds rows x and y (eight bf16 columns each) to f64 sums.  The conversions
// to f64 share a slow pipe, so two values are added in f32 first and converted
// once, wherever that addition is exact: s = x + y is, when both s - x == y
// and s - y == x (of the two, the difference with the larger operand is
// exact in f32, and equal to the other operand only if nothing was lost).
// For values within about 16 binades of one another it always is.
__device__ __forceinline__ void add_rows(double* a, const uint4& x4, const uint4& y4) {
    const uint32_t xs[4] = {x4.x, x4.y, x4.z, x4.w}, ys[4] = {y4.x, y4.y, y4.z, y4.w};
    const float2 neg = make_float2(-1.f, -1.f);
    float2 s[4];
    uint32_t lost = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 x = bf16_pair(xs[i]), y = bf16_pair(ys[i]);
        s[i] = __fadd2_rn(x, y);
        const float2 d = __ffma2_rn(y, neg, __ffma2_rn(x, neg, s[i]));
        const float2 e = __ffma2_rn(x, neg, __ffma2_rn(y, neg, s[i]));
        lost |= __float_as_uint(d.x) | __float_as_uint(e.x);
        lost |= __float_as_uint(d.y) | __float_as_uint(e.y);
    }
    if (lost == 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            a[2 * i] += (double)s[i].x;
            a[2 * i + 1] += (double)s[i].y;
        }
    } else {  // also sums beyond f32, infinities and NaN
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 x = bf16_pair(xs[i]), y = bf16_pair(ys[i]);
            a[2 * i] = a[2 * i] + (double)x.x + (double)y.x;
            a[2 * i + 1] = a[2 * i + 1] + (double)x.y + (double)y.y;
        }
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
        uint4 v[kLoads + kLoads % 2];
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            v[i] = r + 4 * i < r1
                       ? __ldg(reinterpret_cast<const uint4*>(strip + (size_t)(r + 4 * i) * D) + (lane & 7))
                       : make_uint4(0, 0, 0, 0);
        if (kLoads % 2) v[kLoads] = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < kLoads; i += 2) add_rows(a, v[i], v[i + 1]);
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
__global__ void __launch_bounds__(kPoolThreads, PV_SLB)
    summary_kernel(const __grid_constant__ SummaryParams p) {
    constexpr int kStrips = D / 64;
    constexpr int kPer = kPoolWarps / (kStrips * kParts);    // blocks of a CTA
    __shared__ double part[kParts > 1 ? kPoolWarps * 64 : 1];
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
constexpr int kRankBlocks = 256;   // one block per thread: order by counting

// f64 -> unsigned integer of the same order (-0 and +0 equal, NaN lowest).
__device__ __forceinline__ unsigned long long order_key(double s) {
    if (!(s == s)) return 0;
    const long long b = __double_as_longlong(s + 0.0);
    return b < 0 ? ~(unsigned long long)b : (unsigned long long)b | 0x8000000000000000ull;
}

struct SelShared {
    int warp_a[kSelWarps], warp_b[kSelWarps];
    int hist[256];
    int bin, need, all;
};

// Threshold of the `need` largest of n keys (radix select, eight bits at a
// time from the top): the keys whose upper bits exceed `prefix` are taken,
// and of those that equal it all (*all) or the first *need.
__device__ void radix_threshold(const unsigned long long* keys, int n, int need, SelShared* sh,
                                int* shift_out, unsigned long long* prefix_out) {
    unsigned long long prefix = 0;
    int shift = 64;
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
            const unsigned long long k = keys[i] >> shift;
            if (shift == 56 || (k >> 8) == prefix) atomicAdd(&sh->hist[(int)(k & 255)], 1);
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
        prefix = (prefix << 8) | (unsigned long long)sh->bin;
        if (sh->all) break;
    }
    *shift_out = shift;
    *prefix_out = prefix;
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

// The n_sel largest of n keys, ties to the lowest index, as ascending
// indices; -1 up to keep.
__device__ void write_top(const unsigned long long* keys, int n, int n_sel, int keep, SelShared* sh,
                          int* out) {
    const int t = threadIdx.x;
    if (n <= kRankBlocks) {
        // every thread counts the keys ahead of its own: equal ones before it,
        // larger ones anywhere (keys holds a 0 behind an odd n)
        bool f = false;
        if (t < n) {
            const unsigned long long k = keys[t];
            const int w0 = t & ~31, w1 = min(n, w0 + 32);
            const ulonglong2* two = reinterpret_cast<const ulonglong2*>(keys);
            int ahead = 0;
#pragma unroll 4
            for (int i = 0; i < w0 / 2; ++i) {
                const ulonglong2 o = two[i];
                ahead += (o.x >= k) + (o.y >= k);
            }
            for (int i = w0; i < w1; ++i) {
                const unsigned long long o = keys[i];
                ahead += o > k || (o == k && i < t);
            }
#pragma unroll 4
            for (int i = (w1 + 1) / 2; i < (n + 1) / 2; ++i) {
                const ulonglong2 o = two[i];
                ahead += (o.x > k) + (o.y > k);
            }
            f = ahead < n_sel;
        }
        int total;
        const int pos = block_rank(f, sh->warp_a, &total);
        if (f) out[pos] = t;
    } else {
        int shift;
        unsigned long long prefix;
        radix_threshold(keys, n, n_sel, sh, &shift, &prefix);
        const bool all = sh->all != 0;
        const int need = sh->need;
        int base = 0, eq_base = 0;
        for (int i0 = 0; i0 < n; i0 += kSelThreads) {
            const int i = i0 + t;
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
    for (int i = n_sel + t; i < keep; i += kSelThreads) out[i] = -1;
}

// A cluster of kCluster CTAs per (stream, head, query group).  Its CTAs share
// the group's rows (sums exchanged through distributed shared memory) and the
// blocks to score; the first one picks the top.
template <int D, int kCluster, typename Pages>
__global__ void __launch_bounds__(kSelThreads, PV_LB)
    select_kernel(const __grid_constant__ SelectParams p, const __grid_constant__ Pages pages) {
    cg::cluster_group cl = cg::this_cluster();
    const int rank = kCluster > 1 ? (int)cl.block_rank() : 0;
    extern __shared__ __align__(16) unsigned long long keys[];   // max_blocks, rounded up to even
    constexpr int kStrips = D / 64;
    constexpr int kParts = kSelWarps / kStrips;       // warps that share a strip's rows
    constexpr int kShare = kQBlock / kCluster;        // rows of a CTA
    __shared__ double part[kParts * D];
    __shared__ double mine[D];                        // this CTA's sums
    __shared__ double qm[D];
    __shared__ SelShared sh;
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    const int item = blockIdx.x / kCluster;
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
    if (threadIdx.x < D) qm[threadIdx.x] = (double)(float)(sum / (double)(q1 - q0));
    __syncthreads();

    // scores of this CTA's blocks, to the first CTA: eight lanes to a block,
    // each with every eighth run of four columns
    constexpr int kRuns = D / 32;
    const int l8 = lane & 7;
    double ql[kRuns][4];
#pragma unroll
    for (int c = 0; c < kRuns; ++c)
#pragma unroll
        for (int k = 0; k < 4; ++k) ql[c][k] = qm[(c * 8 + l8) * 4 + k];
    unsigned long long* dst = kCluster > 1 ? cl.map_shared_rank(keys, 0) : keys;
    const int n = p.kb.n_blocks[i];
    const long long hs = p.kb.seg0[i] + (long long)head * p.kb.head_segs;
    for (int b0 = (rank * kSelWarps + warp) * 4; b0 < n; b0 += kCluster * kSelWarps * 4) {
        const int b = b0 + lane / 8;
        double s = 0, s2 = 0;
        if (b < n) {
            const int seg = b / p.kb.bps;
            const long long row = (hs + pages.page(p.kb, i, seg)) * p.kb.bps + (b - seg * p.kb.bps);
            const float4* src = reinterpret_cast<const float4*>(p.means + row * D) + l8;
            float4 m[kRuns];
#pragma unroll
            for (int c = 0; c < kRuns; ++c) m[c] = __ldg(src + c * 8);
#pragma unroll
            for (int c = 0; c < kRuns; ++c) {
                double2 qa = make_double2(ql[c][0], ql[c][1]), qb = make_double2(ql[c][2], ql[c][3]);
                if (PV_QS) {
                    const volatile double2* q2 = reinterpret_cast<const volatile double2*>(qm + (c * 8 + l8) * 4);
                    qa.x = q2[0].x; qa.y = q2[0].y; qb.x = q2[1].x; qb.y = q2[1].y;
                }
                s = fma(qa.x, (double)m[c].x, s);
                s2 = fma(qa.y, (double)m[c].y, s2);
                s = fma(qb.x, (double)m[c].z, s);
                s2 = fma(qb.y, (double)m[c].w, s2);
            }
            s += s2;
        }
#pragma unroll
        for (int o = 4; o > 0; o /= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (l8 == 0 && b < n) {
            const bool forced = (b >= p.force0[i][0] && b < p.force1[i][0]) ||
                                (b >= p.force0[i][1] && b < p.force1[i][1]);
            dst[b] = forced ? ~0ull : order_key(s);
        }
    }
    if (rank == 0 && threadIdx.x == 0 && (n & 1)) keys[n] = 0;
    if (kCluster > 1)
        cl.sync();
    else
        __syncthreads();
    if (rank == 0)
        write_top(keys, n, min(p.keep, n), p.keep, &sh, p.blocks + (long long)item * p.keep);
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
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)p.n_items * kCluster);
    cfg.blockDim = dim3(kSelThreads);
    cfg.dynamicSmemBytes = (size_t)(p.max_blocks + 1) / 2 * 16;
    cfg.stream = s;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = kCluster;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, select_kernel<D, kCluster, Pages>, p, pages);
}

#ifndef PV_CS
#define PV_CS 0
#endif
template <int D, typename Pages>
cudaError_t launch_select_d(const SelectParams& p, const Pages& pages, cudaStream_t s) {
    int cs = p.n_items <= 148 ? 8 : p.n_items <= 2 * 148 ? 4 : 1;
    if (PV_CS) cs = PV_CS;
    if (cs == 8) return launch_select_c<D, 8>(p, pages, s);
    if (cs == 4) return launch_select_c<D, 4>(p, pages, s);
    if (cs == 2) return launch_select_c<D, 2>(p, pages, s);
    return launch_select_c<D, 1>(p, pages, s);
}

#ifndef PV_SUM
#define PV_SUM 0
#endif
template <int D, int kParts>
cudaError_t launch_summary_p(const SummaryParams& p, cudaStream_t s) {
    constexpr int kPer = kPoolWarps / (D / 64 * kParts);
    const long long ctas = ((long long)p.n_items * p.heads + kPer - 1) / kPer;
    if (ctas >= (1LL << 31)) return cudaErrorInvalidConfiguration;
    summary_kernel<D, kParts><<<dim3((unsigned)ctas, p.planes), kPoolThreads, 0, s>>>(p);
    return cudaGetLastError();
}
template <int D>
cudaError_t launch_summary_d(const SummaryParams& p, cudaStream_t s) {
    bool few = (long long)p.n_items * p.heads * p.planes <= 4 * 148;
    if (PV_SUM) few = PV_SUM == 4;
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
    copy_kernel<<<(unsigned)cta0[3], kCopyThreads, 0, s>>>(p, cta0[1], cta0[2], (int)parts[0],
                                                           (int)std::max(1LL, parts[2]));
    return cudaGetLastError();
}

}  // namespace pv
