// Attention of few queries over listed key blocks: single tokens and other
// short query sets, where the 128-row tiles of the tcgen05 kernel would be
// almost empty and reading K and V is all the time there is.
//
// An item is (stream, head, 16 queries), or 8 when no stream has more.  Its
// keys, in units of 64, are cut into even parts, one CTA of four warps to a
// part, so that few items fill the GPU; a warp takes 16 keys of each unit.
// Keys and values go from global memory straight into the operand registers
// of mma.sync.m16n8k16: nothing is staged, so nothing waits at a barrier
// inside the key loop, and a warp has its next keys in flight while it works.
// Running maximum and sum per warp as in the other kernels; the four warps
// join through shared memory, the parts of an item through global memory by
// the last CTA to arrive, in part order.
//
// Operand registers.  With g = lane / 4 and c = lane % 4, mma wants from a
// lane A rows g, g + 8 and B column g, each at k = 2c, 2c + 1, 2c + 8, 2c + 9.
//  16 queries: S = Q K^T and O = P V, queries along M.
//  8 queries: S^T = K Q^T and O^T = V^T P^T, keys and columns along M: half
//   the products and accumulators; P^T turns into an operand by a transpose
//   of its 8 x 8 tiles.
//  The order of the k positions of S is free as long as Q and K agree, so
//   lane c takes the 16-byte pieces c, c + 4, c + 8, ... of a row, eight
//   dimensions that serve two k steps.
//  The order of the columns of O is free, so column g of tile t stands for
//   column 8 g + t of a 64-column half, and a lane's tiles come from one
//   16-byte piece of each of its four key rows.
//
// Measured, 24 heads of 128, one query over 32 of 313 blocks (50.3 MB): 14 us;
// the tcgen05 kernel 20 us.  The call's fixed chain (launch, list, first keys,
// joins) is about 6 us of it.  Drawing later strips into L2 ahead
// of time (cp.async.bulk.prefetch) made it slower, 18 against 16.6 us.
#include "pv_internal.h"

namespace pv {
namespace {

constexpr int kFewThreads = 128;
constexpr int kFewWarps = kFewThreads / 32;
constexpr float kFewEmpty = -3.0e38f;   // running maximum of a row without keys

__device__ __forceinline__ float few_ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void mma16816(float* d, uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t few_pack(float lo, float hi) {
    __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&b);
}
__device__ __forceinline__ uint4 few_load(const bf16* p, bool in) {
    return in ? __ldg(reinterpret_cast<const uint4*>(p)) : make_uint4(0, 0, 0, 0);
}

// Transposed 8 x 8 tile of 16-bit values, a row's pair to a lane.
__device__ __forceinline__ uint32_t few_transpose(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

template <int D, int kRows>
struct FewShared {
    float o[kFewWarps][kRows][D];
    float m[kFewWarps][kRows], l[kFewWarps][kRows];
    int last;
};

// CTAs of an SM, by registers.
constexpr int few_resident(int D, int rows) {
    return D == 128 ? (rows == 8 ? 3 : 2) : (rows == 8 ? 4 : 3);
}

template <int D, int kRows, typename Pages>
__global__ void __launch_bounds__(kFewThreads, few_resident(D, kRows))
    few_kernel(const __grid_constant__ FewArgs<Pages> p) {
    __shared__ FewShared<D, kRows> sh;
    wait_for_stream();
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    const int g = lane / 4, c = lane % 4;
    constexpr int kPieces = D / 32;   // 16-byte pieces of a row per lane
    constexpr int kHalves = D / 64;
    constexpr bool kSmall = kRows == 8;

    int si = 0;
    while (si + 1 < p.n_streams && p.st[si + 1].cta0 <= (int)blockIdx.x) ++si;
    const FewStream& st = p.st[si];
    const int li = blockIdx.x - st.cta0;
    const int item = li / st.splits, split = li - item * st.splits;
    const int tiles = (st.n_q + kRows - 1) / kRows;
    const int head = item / tiles, rt = item - head * tiles;
    const int row0 = rt * kRows, rows = min(kRows, st.n_q - row0);
    const int groups = (st.n_q + kQBlock - 1) / kQBlock;
    const int* list = p.list ? p.list + (p.list_row0[si] + (long long)head * groups +
                                         row0 / kQBlock) * p.keep
                             : nullptr;

    // Q: rows g and (of 16) g + 8
    uint4 qa[kPieces], qb[kSmall ? 1 : kPieces];
    {
        const bf16* q = p.q + ((long long)st.q_row0 + (long long)head * st.n_q + row0) * D + c * 8;
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            qa[i] = few_load(q + g * D + i * 32, g < rows);
            if (!kSmall) qb[i] = few_load(q + (g + 8) * D + i * 32, g + 8 < rows);
        }
    }

    // unit u: keys [64 (u % 2), + 64) of listed block u / 2; this warp's 16
    // keys from row 16 warp on.  Rows of the block's first key, valid keys.
    const long long base = (long long)p.kb.seg0[si] + (long long)head * p.kb.head_segs;
    const int units = 2 * st.n_sel;
    const int u_end = (int)((split + 1LL) * units / st.splits);
    // list entries: 32 blocks from block0 on and the 32 behind them, one to a lane
    int u = (int)((long long)split * units / st.splits);
    int block0 = u / 2;
    auto fetch = [&](int b) {
        b += lane;
        return b >= st.n_sel ? -1 : list ? __ldg(list + b) : b;
    };
    int near = fetch(block0), far = fetch(block0 + 32);
    auto entry = [&](int u) {
        const int i = u / 2 - block0;
        return __shfl_sync(0xffffffffu, i < 32 ? near : far, i & 31);
    };
    auto locate = [&](int u, int b, long long* row, int* valid) {
        const int k0 = (u % 2) * kFewUnit + warp * 16;
        *row = 0;
        *valid = 0;
        if ((unsigned)b >= (unsigned)p.kb.n_blocks[si]) return;  // an empty block
        const int seg = segment_of(p.kb, b), blk = b - seg * p.kb.bps;
        *valid = (blk == p.kb.bps - 1 ? p.kb.tail : kKeyTile) - k0;
        *row = (base + p.pages.page(p.kb, si, seg)) * p.kb.seg_len + blk * kKeyTile + k0;
    };
    uint4 kk[2][kPieces];       // keys g and g + 8 of the strip
    // values of keys 2c, 2c + 1, 2c + 8, 2c + 9, of this strip and the next
    uint4 vv[4][kHalves], vn[4][kHalves];
    constexpr int kTiles = kHalves * (kSmall ? 4 : 8);   // accumulator tiles
    auto load_k = [&](long long row, int valid) {
        const bf16* k = p.k + row * D + c * 8;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < kPieces; ++i)
                kk[t][i] = few_load(k + (g + 8 * t) * D + i * 32, g + 8 * t < valid);
    };
    auto load_v = [&](uint4 (&dst)[4][kHalves], long long row, int valid) {
        const bf16* v = p.v + row * D + g * 8;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int key = 2 * c + (j & 1) + (j >> 1) * 8;
#pragma unroll
            for (int h = 0; h < kHalves; ++h)
                dst[j][h] = few_load(v + key * D + h * 64, key < valid);
        }
    };

    float o[kTiles][4];
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[t][i] = 0.f;
    // of rows g, g + 8; of eight rows: 2c, 2c + 1
    float m0 = kFewEmpty, m1 = kFewEmpty, l0 = 0.f, l1 = 0.f;

    long long row = 0;
    int valid = 0;
    if (u < u_end) {
        locate(u, entry(u), &row, &valid);
        load_k(row, valid);
        load_v(vv, row, valid);
    }
    while (u < u_end) {
        const int now = valid;
        // scores: s[t] holds rows g, g + 8 at keys 8t + 2c, 8t + 2c + 1; of eight
        // rows, s[0] holds keys g, g + 8 at rows 2c, 2c + 1
        constexpr int kS = kSmall ? 1 : 2;
        float s[kS][4];
#pragma unroll
        for (int t = 0; t < kS; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[t][i] = 0.f;
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            if constexpr (kSmall) {
                mma16816(s[0], kk[0][i].x, kk[1][i].x, kk[0][i].y, kk[1][i].y, qa[i].x, qa[i].y);
                mma16816(s[0], kk[0][i].z, kk[1][i].z, kk[0][i].w, kk[1][i].w, qa[i].z, qa[i].w);
            } else {
#pragma unroll
                for (int t = 0; t < kS; ++t) {
                    mma16816(s[t], qa[i].x, qb[i].x, qa[i].y, qb[i].y, kk[t][i].x, kk[t][i].y);
                    mma16816(s[t], qa[i].z, qb[i].z, qa[i].w, qb[i].w, kk[t][i].z, kk[t][i].w);
                }
            }
        }
        if (++u < u_end) {      // the next strip, while this one is worked on
            if (u / 2 - block0 == 32) {
                block0 += 32;
                near = far;
                far = fetch(block0 + 32);
            }
            locate(u, entry(u), &row, &valid);
            load_k(row, valid);
            load_v(vn, row, valid);
        }
        float x0, x1;   // largest scores of the lane's rows
        if constexpr (kSmall) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                s[0][i] = g + (i >> 1) * 8 < now ? s[0][i] * p.scale_log2 : -INFINITY;
            x0 = fmaxf(s[0][0], s[0][2]);
            x1 = fmaxf(s[0][1], s[0][3]);
        } else {
#pragma unroll
            for (int t = 0; t < kS; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    s[t][i] = 8 * t + 2 * c + (i & 1) < now ? s[t][i] * p.scale_log2 : -INFINITY;
            x0 = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[kS - 1][0], s[kS - 1][1]));
            x1 = fmaxf(fmaxf(s[0][2], s[0][3]), fmaxf(s[kS - 1][2], s[kS - 1][3]));
        }
#pragma unroll
        for (int d = kSmall ? 4 : 1; d < (kSmall ? 32 : 4); d *= 2) {
            x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, d));
            x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, d));
        }
        // the maximum moves only when it grows by more than 8 (log2 units):
        // P stays below 2^8 and O is seldom rescaled
        if (__any_sync(0xffffffffu, x0 > m0 + 8.f || x1 > m1 + 8.f)) {
            const float n0 = fmaxf(m0, x0), n1 = fmaxf(m1, x1);
            const float a0 = few_ex2(m0 - n0), a1 = few_ex2(m1 - n1);
            m0 = n0, m1 = n1;
            l0 *= a0, l1 *= a1;
#pragma unroll
            for (int t = 0; t < kTiles; ++t) {
                o[t][0] *= a0, o[t][1] *= kSmall ? a1 : a0;
                o[t][2] *= kSmall ? a0 : a1, o[t][3] *= a1;
            }
        }
        // P rounded to nearest bf16, its sum over the unrounded values
        uint32_t pa[4];
        if constexpr (kSmall) {
            const float e0 = few_ex2(s[0][0] - m0), e1 = few_ex2(s[0][1] - m1);
            const float e2 = few_ex2(s[0][2] - m0), e3 = few_ex2(s[0][3] - m1);
            l0 += e0 + e2;
            l1 += e1 + e3;
            pa[0] = few_transpose(few_pack(e0, e1));
            pa[1] = few_transpose(few_pack(e2, e3));
        } else {
#pragma unroll
            for (int t = 0; t < kS; ++t) {
                const float e0 = few_ex2(s[t][0] - m0), e1 = few_ex2(s[t][1] - m0);
                const float e2 = few_ex2(s[t][2] - m1), e3 = few_ex2(s[t][3] - m1);
                l0 += e0 + e1;
                l1 += e2 + e3;
                pa[2 * t] = few_pack(e0, e1);
                pa[2 * t + 1] = few_pack(e2, e3);
            }
        }
#pragma unroll
        for (int h = 0; h < kHalves; ++h) {
            const uint32_t* v0 = reinterpret_cast<const uint32_t*>(&vv[0][h]);
            const uint32_t* v1 = reinterpret_cast<const uint32_t*>(&vv[1][h]);
            const uint32_t* v2 = reinterpret_cast<const uint32_t*>(&vv[2][h]);
            const uint32_t* v3 = reinterpret_cast<const uint32_t*>(&vv[3][h]);
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const uint32_t b0 = __byte_perm(v0[t], v1[t], 0x5410), b1 = __byte_perm(v2[t], v3[t], 0x5410);
                const uint32_t b2 = __byte_perm(v0[t], v1[t], 0x7632), b3 = __byte_perm(v2[t], v3[t], 0x7632);
                if constexpr (kSmall) {
                    mma16816(o[h * 4 + t], b0, b2, b1, b3, pa[0], pa[1]);
                } else {
                    mma16816(o[h * 8 + 2 * t], pa[0], pa[1], pa[2], pa[3], b0, b1);
                    mma16816(o[h * 8 + 2 * t + 1], pa[0], pa[1], pa[2], pa[3], b2, b3);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int h = 0; h < kHalves; ++h) vv[j][h] = vn[j][h];
    }

    // the warps' results
#pragma unroll
    for (int d = kSmall ? 4 : 1; d < (kSmall ? 32 : 4); d *= 2) {
        l0 += __shfl_xor_sync(0xffffffffu, l0, d);
        l1 += __shfl_xor_sync(0xffffffffu, l1, d);
    }
    if (kSmall ? g == 0 : c == 0) {
        const int r0 = kSmall ? 2 * c : g, r1 = kSmall ? 2 * c + 1 : g + 8;
        sh.m[warp][r0] = m0, sh.m[warp][r1] = m1;
        sh.l[warp][r0] = l0, sh.l[warp][r1] = l1;
    }
#pragma unroll
    for (int h = 0; h < kHalves; ++h) {
        if constexpr (kSmall) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = 2 * c + i;
                if (r < rows) {
                    float4* d4 = reinterpret_cast<float4*>(&sh.o[warp][r][h * 64 + g * 8]);
                    d4[0] = make_float4(o[h * 4][i], o[h * 4][i + 2], o[h * 4 + 1][i], o[h * 4 + 1][i + 2]);
                    d4[1] = make_float4(o[h * 4 + 2][i], o[h * 4 + 2][i + 2], o[h * 4 + 3][i],
                                        o[h * 4 + 3][i + 2]);
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = g + (i >> 1) * 8;
                if (r < rows) {
                    float4* d4 =
                        reinterpret_cast<float4*>(&sh.o[warp][r][h * 64 + c * 16 + (i & 1) * 8]);
                    d4[0] = make_float4(o[h * 8][i], o[h * 8 + 1][i], o[h * 8 + 2][i], o[h * 8 + 3][i]);
                    d4[1] = make_float4(o[h * 8 + 4][i], o[h * 8 + 5][i], o[h * 8 + 6][i], o[h * 8 + 7][i]);
                }
            }
        }
    }
    __syncthreads();
    const float ln2 = 0.69314718055994531f;
    const size_t slot_f = few_slot_floats(D);
    float* mine = p.partial + blockIdx.x * slot_f;
    // joins: four columns of a row to a thread
    constexpr int kCols = D / 4;
    constexpr int kRowStep = kFewThreads / kCols;
    const int d = threadIdx.x % kCols * 4;
    auto put = [&](int r, const float4& acc, float M, float L) {
        const bool none = L == 0.f;   // a row without keys: 0 and -inf
        const float inv = none ? 0.f : 1.0f / L;
        const size_t tok = (size_t)st.out_tok0 + row0 + r;
        *reinterpret_cast<uint2*>(p.out + (tok * p.heads + head) * D + d) =
            make_uint2(few_pack(acc.x * inv, acc.y * inv), few_pack(acc.z * inv, acc.w * inv));
        if (d == 0 && p.lse)
            p.lse[tok * p.heads + head] = none ? -INFINITY : (M + __log2f(L)) * ln2;
    };
    auto add = [](float4& acc, float w, const float4& v) {
        acc.x = fmaf(w, v.x, acc.x), acc.y = fmaf(w, v.y, acc.y);
        acc.z = fmaf(w, v.z, acc.z), acc.w = fmaf(w, v.w, acc.w);
    };
    for (int r = threadIdx.x / kCols; r < rows; r += kRowStep) {
        float M = sh.m[0][r], L = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 1; w < kFewWarps; ++w) M = fmaxf(M, sh.m[w][r]);
#pragma unroll
        for (int w = 0; w < kFewWarps; ++w) {
            const float a = few_ex2(sh.m[w][r] - M);
            L = fmaf(a, sh.l[w][r], L);
            add(acc, a, *reinterpret_cast<const float4*>(&sh.o[w][r][d]));
        }
        if (st.splits == 1) {
            put(r, acc, M, L);
        } else {
            __stcg(reinterpret_cast<float4*>(mine + r * D + d), acc);
            if (d == 0) {
                __stcg(mine + kRows * D + r, M);
                __stcg(mine + kRows * D + kRows + r, L);
            }
        }
    }
    if (st.splits == 1) return;
    __threadfence();     // this CTA's part is visible before its arrival
    __syncthreads();
    if (threadIdx.x == 0) {
        int* cnt = p.counters + st.item0 + item;
        const int last = atomicAdd(cnt, 1) == st.splits - 1;
        if (last) *cnt = 0;    // ready for the next launch
        sh.last = last;
    }
    __syncthreads();
    if (!sh.last) return;
    __threadfence();
    const float* parts = p.partial + (size_t)(blockIdx.x - split) * slot_f;
    for (int r = threadIdx.x / kCols; r < rows; r += kRowStep) {
        float M = kFewEmpty, L = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        constexpr int kBatch = 16;   // parts in flight
        for (int k0 = 0; k0 < st.splits; k0 += kBatch) {
            float mk[kBatch], lk[kBatch];
            float4 ok[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const bool in = k0 + k < st.splits;
                const float* pk = parts + (size_t)(k0 + k) * slot_f;
                mk[k] = in ? __ldcg(pk + kRows * D + r) : kFewEmpty;
                lk[k] = in ? __ldcg(pk + kRows * D + kRows + r) : 0.f;
                ok[k] = in ? __ldcg(reinterpret_cast<const float4*>(pk + r * D + d))
                           : make_float4(0.f, 0.f, 0.f, 0.f);
            }
            float Mn = M;
#pragma unroll
            for (int k = 0; k < kBatch; ++k) Mn = fmaxf(Mn, mk[k]);
            const float a = few_ex2(M - Mn);
            L *= a;
            acc = make_float4(acc.x * a, acc.y * a, acc.z * a, acc.w * a);
            M = Mn;
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const float w = few_ex2(mk[k] - M);
                L = fmaf(w, lk[k], L);
                add(acc, w, ok[k]);
            }
        }
        put(r, acc, M, L);
    }
}

template <typename Pages>
cudaError_t launch_few_any(const FewArgs<Pages>& a, int head_dim, int ctas, cudaStream_t s) {
    if (head_dim == 128)
        return a.rows == 8 ? launch_early(few_kernel<128, 8, Pages>, ctas, kFewThreads, 0, 1, s, a)
                           : launch_early(few_kernel<128, 16, Pages>, ctas, kFewThreads, 0, 1, s, a);
    return a.rows == 8 ? launch_early(few_kernel<64, 8, Pages>, ctas, kFewThreads, 0, 1, s, a)
                       : launch_early(few_kernel<64, 16, Pages>, ctas, kFewThreads, 0, 1, s, a);
}

static_assert(sizeof(FewArgs<PageTable>) <= 32000, "kernel parameters too large");

}  // namespace

cudaError_t launch_few(const FewArgs<FixedRows>& a, int head_dim, int ctas, cudaStream_t s) {
    return launch_few_any(a, head_dim, ctas, s);
}
cudaError_t launch_few(const FewArgs<PageTable>& a, int head_dim, int ctas, cudaStream_t s) {
    return launch_few_any(a, head_dim, ctas, s);
}

bool plan_few(FewStream* st, int n_streams, int heads, int head_dim, int n_sm, size_t part_floats,
              int n_counters, int* rows, int* ctas) {
    int most = 0;
    for (int i = 0; i < n_streams; ++i) most = std::max(most, st[i].n_q);
    *rows = most <= 8 ? 8 : kFewRows;
    auto tiles = [&](int i) { return (long long)heads * ((st[i].n_q + *rows - 1) / *rows); };
    long long units = 0, blocks = 0, groups = 0;
    for (int i = 0; i < n_streams; ++i) {
        units += tiles(i) * 2 * st[i].n_sel;
        blocks += (long long)heads * st[i].n_sel;
        groups += heads;
    }
    // Microseconds of this kernel and of the tcgen05 one (whose split items
    // cost a join that grows with their parts).  24 heads of 128, one query:
    // 8 blocks 6.7 against 12.7, 32 blocks 13.8 against 20.1, 128 blocks 50.2
    // against 45.2; 24 queries, 8 blocks 11.7 against 12.9, 32 blocks 22.8
    // against 20.3; one head, 24 queries over 300 blocks 25.4 against 34.6.
    const double unit = head_dim == 128 ? (*rows == 8 ? 0.0079 : 0.0097) : (*rows == 8 ? 0.0045 : 0.0055);
    const double tile = head_dim == 128 ? 0.0109 : 0.0095;
    const double few = 4.0 + unit * units;
    const double many = 10.5 + tile * blocks + 0.16 * std::min<double>(n_sm, (double)blocks) / groups;
    if (few > many) return false;
    // one wave of resident CTAs, shared out by keys
    const long long wave = (long long)n_sm * few_resident(head_dim, *rows);
    const long long per = std::max(1LL, (units + wave - 1) / wave);
    long long cta = 0, item = 0;
    for (int i = 0; i < n_streams; ++i) {
        FewStream& s = st[i];
        const long long items = tiles(i);
        // one CTA joins an item's parts: the more rows, the fewer parts (one head,
        // 128 blocks: one query 10 us with 60 parts, 16 with 256; 16 queries 16
        // with 32, 46 with 256)
        s.splits = (int)std::min((2LL * s.n_sel + per - 1) / per,
                                 1024LL / (kFewRows + std::min(*rows, s.n_q)));
        s.cta0 = (int)cta;
        s.item0 = (int)item;
        cta += items * s.splits;
        item += items;
        if (cta >= (1LL << 31) || item > n_counters) return false;
    }
    if ((size_t)cta * few_slot_floats(head_dim) > part_floats) return false;
    *ctas = (int)cta;
    return true;
}

}  // namespace pv
