// Stand-in for the CUDA runtime and for the kernel launches of libpv, so that the host API
// (csrc/pv_api.cu, csrc/pv_plan.cu) runs without a device: every call that would touch one is written
// to a log instead, and a launch can be made to fail.  Device addresses are never read or written.
#include <cudaTypedefs.h>

#include <cstdarg>
#include <cstdio>
#include <string>
#include <vector>

#include "../same_step_kv_b200/csrc/pv_internal.h"

namespace {
std::string g_log;
int g_copies = 0;            // page-copy launches since fake_reset
int g_fail_copy = -1;        // the one that fails
cudaError_t g_last = cudaSuccess;   // what a failed call leaves behind for cudaGetLastError
std::vector<int> g_moves;    // (src, dst) pairs of the launches that went through

void note(const char* fmt, ...) {
    char line[160];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(line, sizeof line, fmt, ap);
    va_end(ap);
    g_log += line;
    g_log += '\n';
}
CUresult fake_encode(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                     const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                     CUtensorMapL2promotion, CUtensorMapFloatOOBfill) {
    return CUDA_SUCCESS;
}
cudaError_t launched(const char* what) {
    note("launch %s", what);
    return cudaSuccess;
}
}  // namespace

// ------------------------------------------------------------------ CUDA runtime
extern "C" {
cudaError_t cudaGetDevice(int* dev) {
    *dev = 0;
    return cudaSuccess;
}
// addresses from 2^50 on lie on device 1
cudaError_t cudaPointerGetAttributes(cudaPointerAttributes* a, const void* p) {
    *a = cudaPointerAttributes{};
    a->type = cudaMemoryTypeDevice;
    a->device = ((uintptr_t)p >> 50) != 0;
    return cudaSuccess;
}
cudaError_t cudaDeviceGetAttribute(int* value, cudaDeviceAttr attr, int) {
    *value = attr == cudaDevAttrComputeCapabilityMajor ? 10 : attr == cudaDevAttrMultiProcessorCount ? 148 : 0;
    return cudaSuccess;
}
cudaError_t cudaGetDriverEntryPointByVersion(const char*, void** fn, unsigned, unsigned long long,
                                             cudaDriverEntryPointQueryResult* q) {
    *fn = (void*)fake_encode;
    *q = cudaDriverEntryPointSuccess;
    return cudaSuccess;
}
const char* cudaGetErrorString(cudaError_t) { return "made up"; }
cudaError_t cudaGetLastError(void) {
    const cudaError_t e = g_last;
    g_last = cudaSuccess;
    return e;
}
cudaError_t cudaMemset(void*, int, size_t) { return note("memset"), cudaSuccess; }
cudaError_t cudaMemsetAsync(void*, int, size_t, cudaStream_t) { return note("memset async"), cudaSuccess; }
cudaError_t cudaMemcpy(void*, const void*, size_t, cudaMemcpyKind) { return note("memcpy"), cudaSuccess; }
cudaError_t cudaStreamSynchronize(cudaStream_t s) { return note("wait %p", (void*)s), cudaSuccess; }
cudaError_t cudaDeviceSynchronize(void) { return note("wait all"), cudaSuccess; }
}

// ------------------------------------------------------------------ launches
namespace pv {
cudaError_t launch_rope(const RopeParams&, int, cudaStream_t) { return launched("rope"); }
cudaError_t launch_attn(const CUtensorMap&, const CUtensorMap&, const CUtensorMap&, const CUtensorMap&,
                        const AttnParams&, cudaStream_t) {
    return launched("attention");
}
cudaError_t launch_block_attn(const CUtensorMap&, const CUtensorMap&, const CUtensorMap&, const CUtensorMap&,
                              const AttnParams&, const BlockArgs<FixedRows>&, cudaStream_t) {
    return launched("block attention");
}
cudaError_t launch_block_attn(const CUtensorMap&, const CUtensorMap&, const CUtensorMap&, const CUtensorMap&,
                              const AttnParams&, const BlockArgs<PageTable>&, cudaStream_t) {
    return launched("block attention");
}
bool plan_few(FewStream*, int, int, int, int, size_t, int, int*, int*) { return false; }
cudaError_t launch_few(const FewArgs<FixedRows>&, int, int, cudaStream_t) { return launched("few"); }
cudaError_t launch_few(const FewArgs<PageTable>&, int, int, cudaStream_t) { return launched("few"); }
cudaError_t launch_summary(const SummaryParams&, cudaStream_t) { return launched("means"); }
cudaError_t launch_select(const SelectParams&, const PageTable*, cudaStream_t) { return launched("selection"); }
cudaError_t launch_copy(const CopyParams& p, cudaStream_t) {
    if (g_copies++ == g_fail_copy) return g_last = cudaErrorLaunchOutOfResources;
    for (int i = 0; i < p.n; ++i) {
        g_moves.push_back(p.fan ? p.src[0] : p.src[i]);
        g_moves.push_back(p.dst[i]);
    }
    return launched("copy");
}
cudaError_t launch_wait_timeout_probe(int*, cudaStream_t) { return launched("probe"); }
int qkv_gemm_tile_n(int) { return 64; }
cudaError_t launch_qkv_gemm(const CUtensorMap&, const CUtensorMap&, const CUtensorMap&, const float*, float*, int,
                            int, int*, cudaStream_t) {
    return launched("gemm");
}
cudaError_t launch_qkv_fused(const CUtensorMap&, const CUtensorMap&, const float*, float*, unsigned long long*,
                             unsigned long long, int, int, int*, const RopeParams&, const QkvOutMaps&,
                             cudaStream_t) {
    return launched("fused gemm");
}
cudaError_t launch_euler(float*, const float*, size_t, float, cudaStream_t) { return launched("euler"); }
cudaError_t launch_euler_cfg(float*, const float*, const float*, size_t, float, float, cudaStream_t) {
    return launched("euler");
}
cudaError_t launch_x0(float*, const float*, const float*, size_t, float, cudaStream_t) { return launched("x0"); }
cudaError_t noalloc_scratch_address(void**) { return cudaErrorNotSupported; }
}  // namespace pv

// ------------------------------------------------------------------ for the tests
extern "C" {
PV_API void fake_reset(int fail_copy) {
    g_log.clear();
    g_moves.clear();
    g_copies = 0;
    g_fail_copy = fail_copy;
}
PV_API const char* fake_log(void) { return g_log.c_str(); }
PV_API int fake_moves(int* out, int room) {
    for (int i = 0; i < (int)g_moves.size() && i < room; ++i) out[i] = g_moves[i];
    return (int)g_moves.size();
}
}
