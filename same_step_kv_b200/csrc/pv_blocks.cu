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

// Adds eight bf16 values (one 16-byte load) to f64 sums.
__device__ __forceinline__ void add8(double* a, const uint4& v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        a[2 * i] += (double)__uint_as_float(w[i] << 16);
        a[2 * i + 1] += (double)__uint_as_float(w[i] & 0xFFFF0000u);
    }
}

// Sums of the rows [r0, r1) of `rows` (bf16 [.][D]), D columns, by the whole
// block, at most kRows of them: partial sums of the warps in part [kPoolWarps][D];
// the caller synchronises.
template <int D, int kRows>
__device__ __forceinline__ void pool_rows(const bf16* rows, int r0, int r1, double* part) {
    constexpr int kLanes = D / 8;                    // threads across one row
    constexpr int kStep = kPoolThreads / kLanes;     // rows per pass
    constexpr int kPasses = (kRows + kStep - 1) / kStep;
    const int col = threadIdx.x % kLanes, row = threadIdx.x / kLanes;
    uint4 v[kPasses];
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        const int r = r0 + row + i * kStep;
        v[i] = r < r1 ? __ldg(reinterpret_cast<const uint4*>(rows + (size_t)r * D) + col)
                      : make_uint4(0, 0, 0, 0);
    }
    double a[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < kPasses; ++i) add8(a, v[i]);
#pragma unroll
    for (int m = kLanes; m < 32; m *= 2)
#pragma unroll
        for (int i = 0; i < 8; ++i) a[i] += __shfl_xor_sync(0xffffffffu, a[i], m);
    if ((threadIdx.x & 31) < kLanes) {
        double* p = part + (threadIdx.x / 32) * D + col * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = a[i];
    }
}

// One CTA per (block of a run, head, plane).  Bound by reading the keys.
template <int D>
__global__ void __launch_bounds__(kPoolThreads)
    summary_kernel(const __grid_constant__ SummaryParams p) {
    __shared__ double part[kPoolWarps * D];
    const int head = blockIdx.y;
    const int item = blockIdx.x;
    int i = 0;
    while (i + 1 < p.n_runs && p.item0[i + 1] <= item) ++i;
    const int li = item - p.item0[i];
    const int seg = li / p.bps, blk = li - seg * p.bps;
    const long long ps =
        (long long)blockIdx.z * p.plane_segs + p.seg0[i] + (long long)head * p.head_segs + seg;
    const int r0 = blk * kKeyTile;
    const int r1 = min(p.seg_len, r0 + kKeyTile);
    pool_rows<D, kKeyTile>(p.k + ps * p.seg_len * D, r0, r1, part);
    __syncthreads();
    if (threadIdx.x < D) {
        double s = 0;
#pragma unroll
        for (int w = 0; w < kPoolWarps; ++w) s += part[w * D + threadIdx.x];
        p.means[(ps * p.bps + blk) * D + threadIdx.x] = (float)(s / (double)(r1 - r0));
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
        // every thread counts the keys ahead of its own
        bool f = false;
        if (t < n) {
            const unsigned long long k = keys[t];
            int ahead = 0;
            for (int i = 0; i < n; ++i) {
                const unsigned long long o = keys[i];
                ahead += o > k || (o == k && i < t);
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

// One cluster of CTAs per (stream, head, query group): its CTAs share the
// group's rows (sums exchanged through distributed shared memory) and the
// blocks to score; the first one picks the top.
template <int D, typename Pages>
__global__ void __launch_bounds__(kSelThreads)
    select_kernel(const __grid_constant__ SelectParams p, const __grid_constant__ Pages pages) {
    cg::cluster_group cl = cg::this_cluster();
    const int cs = (int)cl.num_blocks(), rank = (int)cl.block_rank();
    extern __shared__ unsigned long long keys[];      // max_blocks
    __shared__ double part[kPoolWarps * D];
    __shared__ double mine[D];                        // this CTA's sums
    __shared__ double qm[D];
    __shared__ SelShared sh;
    const int item = blockIdx.x / cs;
    int i = 0;
    while (i + 1 < p.n_streams && p.item0[i + 1] <= item) ++i;
    const int li = item - p.item0[i];
    const int n_q = p.n_q[i];
    const int groups = (n_q + kQBlock - 1) / kQBlock;
    const int head = li / groups, g = li - head * groups;

    // the group's mean query
    const int q0 = g * kQBlock, q1 = min(n_q, q0 + kQBlock);
    const int share = kQBlock / cs;
    const bf16* q = p.q + (p.q_row0[i] + (long long)head * n_q) * D;
    {
        const int r0 = q0 + rank * share, r1 = min(q1, r0 + share);
        if (cs >= 8)
            pool_rows<D, kQBlock / 8>(q, r0, r1, part);
        else
            for (int r = r0; r < r0 + share; r += kQBlock / 4) {
                // rows in runs of 64, the warps' sums added up
                if (r > r0) __syncthreads();
                pool_rows<D, kQBlock / 4>(q, r, min(r1, r + kQBlock / 4), part);
                __syncthreads();
                if (threadIdx.x < D) {
                    double s = r > r0 ? mine[threadIdx.x] : 0.0;
#pragma unroll
                    for (int w = 0; w < kPoolWarps; ++w) s += part[w * D + threadIdx.x];
                    mine[threadIdx.x] = s;
                }
            }
        if (cs >= 8) {
            __syncthreads();
            if (threadIdx.x < D) {
                double s = 0;
#pragma unroll
                for (int w = 0; w < kPoolWarps; ++w) s += part[w * D + threadIdx.x];
                mine[threadIdx.x] = s;
            }
        }
    }
    cl.sync();
    if (threadIdx.x < D) {
        double s = 0;
        for (int r = 0; r < cs; ++r) s += cl.map_shared_rank(mine, r)[threadIdx.x];
        qm[threadIdx.x] = (double)(float)(s / (double)(q1 - q0));
    }
    __syncthreads();

    // scores of this CTA's blocks, to the first CTA
    constexpr int kPer = D / 32;   // columns of a lane
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    double ql[kPer];
#pragma unroll
    for (int c = 0; c < kPer; ++c) ql[c] = qm[lane * kPer + c];
    unsigned long long* dst = cl.map_shared_rank(keys, 0);
    const int n = p.kb.n_blocks[i];
    const long long hs = p.kb.seg0[i] + (long long)head * p.kb.head_segs;
    const int step = cs * kSelWarps;
    for (int b0 = rank * kSelWarps + warp; b0 < n; b0 += 4 * step) {
        float m[4][kPer];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int b = b0 + u * step;
            if (b < n) {
                const int seg = b / p.kb.bps;
                const long long row =
                    (hs + pages.page(p.kb, i, seg)) * p.kb.bps + (b - seg * p.kb.bps);
                const float* src = p.means + row * D + lane * kPer;
                if constexpr (kPer == 4) {
                    const float4 v = __ldg(reinterpret_cast<const float4*>(src));
                    m[u][0] = v.x, m[u][1] = v.y, m[u][2] = v.z, m[u][3] = v.w;
                } else {
                    const float2 v = __ldg(reinterpret_cast<const float2*>(src));
                    m[u][0] = v.x, m[u][1] = v.y;
                }
            }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int b = b0 + u * step;
            if (b < n) {   // the same for the whole warp
                double s = 0;
#pragma unroll
                for (int c = 0; c < kPer; ++c) s = fma(ql[c], (double)m[u][c], s);
#pragma unroll
                for (int o = 16; o > 0; o /= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
                const bool forced = (b >= p.force0[i][0] && b < p.force1[i][0]) ||
                                    (b >= p.force0[i][1] && b < p.force1[i][1]);
                if (lane == 0) dst[b] = forced ? ~0ull : order_key(s);
            }
        }
    }
    cl.sync();
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

template <int D, typename Pages>
cudaError_t launch_select_d(const SelectParams& p, const Pages& pages, cudaStream_t s) {
    static std::atomic<unsigned long long> configured{0};
    cudaError_t e = smem_limit_once(select_kernel<D, Pages>, kMaxSelectBlocks * 8, configured);
    if (e != cudaSuccess) return e;
    // few items: several CTAs to each, for latency; many: one each
    const int cs = p.n_items <= 148 ? 8 : p.n_items <= 2 * 148 ? 4 : 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)p.n_items * cs);
    cfg.blockDim = dim3(kSelThreads);
    cfg.dynamicSmemBytes = (size_t)p.max_blocks * 8;
    cfg.stream = s;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = cs;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, select_kernel<D, Pages>, p, pages);
}

}  // namespace

cudaError_t launch_summary(const SummaryParams& p, cudaStream_t s) {
    const dim3 grid(p.n_items, p.heads, p.planes);
    if (p.head_dim == 128)
        summary_kernel<128><<<grid, kPoolThreads, 0, s>>>(p);
    else
        summary_kernel<64><<<grid, kPoolThreads, 0, s>>>(p);
    return cudaGetLastError();
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
