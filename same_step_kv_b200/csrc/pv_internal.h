// Internal declarations shared by the host API and the kernels of libpv.
// Nothing here is part of the C ABI (include/pv.h is).
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>

#include "../../include/pv.h"

namespace pv {

using bf16 = __nv_bfloat16;

constexpr int kMaxSteps = 8;              // denoising steps per chunk a handle may hold
constexpr int kQRows = 128;               // query rows per tensor-core tile (MMA M)
constexpr int kQTilesPerCta = 2;          // two query tiles share each K/V tile
constexpr int kOutRows = 32;               // output rows of one TMA store (one softmax warp)
constexpr int kQBlock = kQRows * kQTilesPerCta;
constexpr int kKeyTile = 128;             // keys per K/V tile (MMA N of Q K^T)
constexpr int kMaxGrid = 160;             // CTAs of one attention launch at most (>= SMs)

// ---------------------------------------------------------------- early launches
// A launch that may start while the one before it in the stream still runs,
// so that its launch and set-up overlap that one's end.  Its kernel calls
// wait_for_stream in every thread before it touches global memory: nothing of
// it is seen to happen early, and it cannot end before the launch it follows.
// Chunk of 880 queries over 37 blocks, two launches a call: 72.9 -> 70.5 us;
// four streams of 64-wide heads: 91.3 -> 88.7 us.
#ifdef __CUDACC__
__device__ __forceinline__ void wait_for_stream() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
}
template <typename K, typename... A>
cudaError_t launch_early(K kernel, dim3 grid, unsigned threads, size_t smem, unsigned cluster,
                         cudaStream_t s, const A&... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[2]{};
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = cluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}
#endif

// ---------------------------------------------------------------- RoPE + append
struct RopeStreamDesc {
    int in_tok0;                     // first token of this stream in the packed input
    int n_tok;                       // tokens of the chunk
    int frame0;                      // latent frame of token 0
    int n_dst;                       // K/V destinations (0: none, 1: a step, steps: sink pass)
    long long qrot_row0;             // q_rot row (of D elements) of head 0, token 0
    long long dst_row0[kMaxSteps];   // K/V-region row of head 0, token 0, per destination
};

struct RopeParams {
    const bf16* q;
    const bf16* k;
    const bf16* v;
    bf16* q_rot;
    bf16* k_dst;            // K region base (store) or k_rot (dense)
    bf16* v_dst;            // V region base (store) or v head-major (dense)
    const float2* table;    // cos, sin per (axis, position, pair)
    int heads, head_dim, frame_w, frame_h;
    int pairs_t, pairs_h, pairs_w;
    int tab_h0, tab_w0;     // table offsets of the height and width blocks
    long long dst_head_stride;  // destination rows between heads
    // projection input instead of q, k, v (pv_qkv_rope_append): y f32
    // [tokens][3 * dim], ss the q / k sums of squares per token, gains g_q, g_k
    const float* y;
    const float* ss;
    const float* g_q;
    const float* g_k;
    float eps;
    int n_streams;
    RopeStreamDesc st[PV_MAX_STREAMS];
};

cudaError_t launch_rope(const RopeParams& p, int max_tok, cudaStream_t s);

// ----------------------------------------------------------------- attention
struct AttnStreamDesc {
    int n_q;             // queries of this stream (per head)
    int n_k;             // keys (per head)
    int q_row0;          // q_rot row of head 0, query 0 (per head + n_q)
    int kv_row0;         // K/V row of head 0, key 0
    int kv_head_stride;  // K/V rows between heads
    int out_tok0;        // first token row of out / lse
    int n_qb;            // query blocks of kQBlock rows
    int n_kt;            // key tiles
    int item0;           // global index of this stream's first (head, query block) item
    int id;              // position in the caller's list (the planner may reorder streams)
    long long cost0;     // key tiles of all items before this stream's first
};

// One launch is a list of items (head, query block) of all streams, each
// costing n_kt key tiles, laid end to end.  Under stream-K, CTA c of `grid`
// processes one contiguous range of that list; otherwise the CTAs take whole
// items one at a time (pv_plan.cu chooses).  The whole struct plus four
// tensor maps stays under 4 KB of kernel parameters.
struct AttnParams {
    bf16* out;
    float* lse;
    float* partial;      // split-KV partial results, 4 slots per CTA (unnormalised O, m, l)
    int* counters;       // arrivals per (item, query tile); the last arriver resets to 0
    int* err;            // device error word (bounded waits that gave up)
    int heads;
    int head_dim;
    float scale_log2;    // log2(e) / sqrt(D)
    int n_streams;
    int grid;            // CTAs of the launch
    int item_aligned;    // 0: stream-K; 1: whole items handed out at run time, in
                         // list order, from counters[0] (no partial results)
    int n_items;         // items of all streams
    long long total;     // key tiles of all items
    AttnStreamDesc st[PV_MAX_STREAMS];
};

// Bytes of one partial-result slot for head dimension D.
__host__ __device__ inline size_t partial_slot_floats(int D) { return (size_t)kQRows * D + 2 * kQRows; }

cudaError_t launch_attn(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                        const CUtensorMap& to, const AttnParams& p, cudaStream_t s);

// ------------------------------------------------- key blocks and pages
// Keys of a (plane, head) lie in segments of seg_len rows: the latent frames
// of a store (seg_len = T), or the one segment of an explicit buffer.  A
// segment holds bps = ceil(seg_len / 128) blocks of 128 keys, the last one
// with `tail` keys.  Block b of a sequence is block b % bps of its segment
// b / bps.  Where segment s lies in memory is its physical segment
// seg0 + head * head_segs + page(s): page(s) = s in fixed rows, the stream's
// page table in a paged store.
struct KeyBlocks {
    int seg_len, bps, tail;
    unsigned long long bps_inv;    // ceil(2^64 / bps), for ends_segment
    int head_segs;       // physical segments between heads
    int first;           // segments of the sink run (paged store)
    int seg0[PV_MAX_STREAMS];      // physical segment of head 0, page 0
    int n_blocks[PV_MAX_STREAMS];
};
// Whether block b is the last of its segment: (b + 1) is a multiple of bps,
// tested without a division (Lemire, Kaser, Kurz, "Faster remainder by direct
// computation", 2019: d divides n iff n * ceil(2^64 / d) mod 2^64 is below
// ceil(2^64 / d), for 32-bit n and d).
__host__ __device__ inline bool ends_segment(const KeyBlocks& k, int b) {
    return (unsigned long long)(unsigned)(b + 1) * k.bps_inv <= k.bps_inv - 1;
}
// Segment of block b, likewise (quotient of b by bps).
__host__ __device__ inline int segment_of(const KeyBlocks& k, int b) {
#ifdef __CUDA_ARCH__
    return k.bps == 1 ? b : (int)__umul64hi(k.bps_inv, (unsigned long long)(unsigned)b);
#else
    return b / k.bps;
#endif
}
inline void set_blocks(KeyBlocks* k, int seg_len) {
    k->seg_len = seg_len;
    k->bps = (seg_len + kKeyTile - 1) / kKeyTile;
    k->tail = seg_len - (k->bps - 1) * kKeyTile;
    k->bps_inv = ~0ull / (unsigned)k->bps + 1;   // 0, that is 2^64, for one block
}
struct FixedRows {
    __host__ __device__ static int page(const KeyBlocks&, int, int seg) { return seg; }
};
// Pages of the listed streams: the sink's first page (its pages are
// consecutive), then one page per ring slot.
struct PageTable {
    int sink[PV_MAX_STREAMS];
    int ring[PV_MAX_STREAMS][PV_MAX_RING];
    __host__ __device__ int page(const KeyBlocks& k, int stream, int seg) const {
        return seg < k.first ? sink[stream] + seg : ring[stream][seg - k.first];
    }
};

// Attention over listed blocks: every (head, query block) item reads the
// blocks of its list row, list_row0 + head * n_qb + query block, of `keep`
// entries; without a list it reads its stream's blocks 0 .. n_kt - 1.
template <typename Pages>
struct BlockArgs {
    static constexpr bool kBlocks = true;
    const int* list;
    int keep;
    int list_row0[PV_MAX_STREAMS];
    KeyBlocks kb;
    Pages pages;
};
struct NoBlocks {  // contiguous keys
    static constexpr bool kBlocks = false;
};

// tk, tv: 3D maps (D, seg_len, segments) of encode_seg_map; n_kt of a stream
// is the number of listed blocks.
cudaError_t launch_block_attn(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                              const CUtensorMap& to, const AttnParams& p,
                              const BlockArgs<FixedRows>& b, cudaStream_t s);
cudaError_t launch_block_attn(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                              const CUtensorMap& to, const AttnParams& p,
                              const BlockArgs<PageTable>& b, cudaStream_t s);
// Attention of few queries over listed blocks (pv_few.cu): items (stream,
// head, 16 queries), each cut into `splits` even parts of its units of 64 keys.
constexpr int kFewRows = 16;
constexpr int kFewUnit = 64;
// Most queries of a stream that the kernel is used for.
constexpr int kFewQueries = 32;
struct FewStream {
    int n_q, q_row0, out_tok0;
    int n_sel;           // listed blocks
    int splits;          // CTAs of an item
    int cta0, item0;     // first CTA and first item
};
template <typename Pages>
struct FewArgs {
    const bf16* q;
    const bf16* k;
    const bf16* v;
    bf16* out;
    float* lse;
    float* partial;      // few_slot_floats per CTA
    int* counters;       // arrivals per item; the last arriver resets to 0
    int heads, n_streams;
    int rows;            // queries of an item: 8 or 16
    float scale_log2;
    const int* list;     // NULL: blocks 0 .. n_sel - 1
    int keep;
    int list_row0[PV_MAX_STREAMS];
    FewStream st[PV_MAX_STREAMS];
    KeyBlocks kb;
    Pages pages;
};
__host__ __device__ inline size_t few_slot_floats(int D) { return (size_t)kFewRows * D + 2 * kFewRows; }
// Lays out the streams (n_q and n_sel set; splits, cta0, item0 filled in) on
// n_sm SMs, in items of *rows queries.  False when the parts or counters do
// not fit, or the tcgen05 kernel is expected to take less time.
bool plan_few(FewStream* st, int n_streams, int heads, int head_dim, int n_sm, size_t part_floats,
              int n_counters, int* rows, int* ctas);
cudaError_t launch_few(const FewArgs<FixedRows>& a, int head_dim, int ctas, cudaStream_t s);
cudaError_t launch_few(const FewArgs<PageTable>& a, int head_dim, int ctas, cudaStream_t s);
// K or V rows as segments: a box is 128 rows x 64 columns of one segment,
// and rows past the segment's end read as zeros.
bool encode_seg_map(CUtensorMap* map, const void* base, int seg_len, long long segs, int D,
                    char* err, size_t errlen);

// Means of key blocks (pv_blocks.cu): runs of n_segs[i] physical segments
// from seg0[i] (head 0), for every head and `planes` planes that lie
// plane_segs segments apart.
struct SummaryParams {
    const bf16* k;
    float* means;        // f32 [physical segment][bps][D]
    int head_dim, heads;
    int seg_len, bps, head_segs;
    int planes;
    long long plane_segs;
    int n_runs;
    int seg0[PV_MAX_STREAMS];
    int n_segs[PV_MAX_STREAMS];
    int item0[PV_MAX_STREAMS];   // blocks of all runs before run i
    int n_items;                 // blocks of all runs
};
cudaError_t launch_summary(const SummaryParams& p, cudaStream_t s);

// Block selection (pv_blocks.cu): one item per (stream, head, query group).
constexpr int kMaxSelectBlocks = 16384;   // blocks of one sequence
struct SelectParams {
    const bf16* q;
    const float* means;
    int* blocks;
    int head_dim, heads, keep;
    int n_streams;
    int n_items;
    int max_blocks;
    int n_q[PV_MAX_STREAMS];
    int item0[PV_MAX_STREAMS];            // also the first list row
    long long q_row0[PV_MAX_STREAMS];     // row of head 0, query 0
    int force0[PV_MAX_STREAMS][2];        // first forced block of two ranges
    int force1[PV_MAX_STREAMS][2];        // one past the last
    KeyBlocks kb;
};
cudaError_t launch_select(const SelectParams& p, const PageTable* pages, cudaStream_t s);

// Page copies (pv_blocks.cu): physical segments moved in every plane and head
// of up to three regions (K, V, block means).  fan: the run of len segments
// from src[0] goes to each of dst[0..n); otherwise segment src[i] goes to
// dst[i] in the order given, with dst[i] < src[i] and src ascending.
constexpr int kMaxMoves = 480;
struct CopyParams {
    char* base[3];
    long long seg_bytes[3];
    int n_regions;
    int heads, head_segs, planes;
    long long plane_segs;
    int fan, len, n;
    int src[kMaxMoves], dst[kMaxMoves];
};
cudaError_t launch_copy(const CopyParams& p, cudaStream_t s);

// One bounded device wait that runs out (failure-path self-test).
cudaError_t launch_wait_timeout_probe(int* err, cudaStream_t s);

// ----------------------------------------------------------------- Euler
// q, k, v projection (pv_gemm.cu): y = x w^T + b in f32 and the q / k sums of
// squares per token; tiles of 256 tokens x qkv_gemm_tile_n(dim) features.
int qkv_gemm_tile_n(int dim);
cudaError_t launch_qkv_gemm(const CUtensorMap& tx, const CUtensorMap& tw, const CUtensorMap& ty,
                            const float* bias, float* ss, int tokens, int dim, int* err,
                            cudaStream_t s);
// Destinations of the fused epilogue's TMA stores, each [rows][head_dim]
// bf16 with boxes of 32 rows x 64 features (128-byte swizzle): q_rot, the K
// region and the V region.
struct QkvOutMaps {
    CUtensorMap q, k, v;
};
// The same GEMM with the QK-Norm, RoPE and append in its epilogue (one
// cooperative launch).  ss [tokens][2][dim / tile width] takes one partial
// sum of squares per feature tile (no need to clear it); CTA c sets
// flags[c] = epoch once its partial sums are written, and the CTAs of a
// token block read them once all of its tiles' flags hold epoch (flags of
// earlier calls hold smaller values: the epoch is a 64-bit call count).  cudaErrorCooperativeLaunchTooLarge when
// its tiles cannot all be resident, there are more than kQkvFlags of them,
// or the RoPE table does not fit in shared memory beside them.
constexpr int kQkvFlags = 1024;
cudaError_t launch_qkv_fused(const CUtensorMap& tx, const CUtensorMap& tw, const float* bias,
                             float* ss, unsigned long long* flags, unsigned long long epoch,
                             int tokens, int dim, int* err, const RopeParams& rp,
                             const QkvOutMaps& om, cudaStream_t s);
bool encode_2d_map(CUtensorMap* map, const void* base, CUtensorMapDataType type, int elem_bytes,
                   long long cols, long long rows, int box_cols, int box_rows, char* err,
                   size_t errlen);
cudaError_t launch_euler(float* x, const float* v, size_t n, float dsigma, cudaStream_t s);
cudaError_t launch_euler_cfg(float* x, const float* vc, const float* vu, size_t n, float w,
                             float dsigma, cudaStream_t s);
cudaError_t launch_x0(float* x0, const float* x, const float* v, size_t n, float sigma,
                      cudaStream_t s);

// ----------------------------------------------------------------- host helpers
// Encodes a 2D bf16 tensor map over `rows` rows of `D` elements with a
// 64-element x 128-row box and the 128-byte swizzle.
bool encode_out_map(CUtensorMap* map, void* out, long long tokens, int heads, int D, char* err,
                    size_t errlen);
bool encode_rows_map(CUtensorMap* map, const void* base, long long rows, int D, char* err,
                     size_t errlen);

// Raises `kernel`'s dynamic shared-memory limit to `bytes` on the current
// device.  The attribute belongs to a device, so it is set once per device:
// `done` holds one bit per device ordinal below 64 (others set it on every
// call).  Two host threads that race here both set the same value.
template <typename K>
cudaError_t smem_limit_once(K kernel, int bytes, std::atomic<unsigned long long>& done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = (dev >= 0 && dev < 64) ? 1ull << dev : 0ull;
    if (bit && (done.load(std::memory_order_acquire) & bit)) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    if (bit) done.fetch_or(bit, std::memory_order_release);
    return cudaSuccess;
}

// Device address, on the current device, of the fixed scratch array of
// pv_attn_dense_noalloc (its first 256 bytes hold the device error word).
cudaError_t noalloc_scratch_address(void** out);

// Records a failure for pv_last_error() and returns code.
pv_status report_error(pv_status code, const char* msg);

// Work plan for one attention launch: fills n_qb, n_kt, item0, cost0 of
// every stream and grid, total, n_items, item_aligned of p (and may reorder
// p.st).  Returns the number of CTAs, or -1 when the counters (one per item,
// at least two) do not fit.  Long items run stream-K; short items, or a
// workspace without room for the partial slots (4 per CTA), get whole items
// handed out at run time instead.
// blocks: a launch over listed blocks, whose split items a second launch joins.
int plan_attention(AttnParams& p, int n_sm, int part_capacity, int cnt_capacity,
                   bool blocks = false);

}  // namespace pv
