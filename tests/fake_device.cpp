// Two devices that are not there: the CUDA runtime calls and the launches that
// the C entry points of csrc/mx4_api.cu make, so that their host logic runs
// without a GPU (linked with the compiled object in place of the runtime and
// the kernels).  Bits 40-43 of an address are its device + 1 (0: host memory),
// bit 44 marks managed memory.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../expert_routed_ffn_gemm_gb300/csrc/mx4.cuh"
#include "../expert_routed_ffn_gemm_gb300/csrc/norm.cuh"

namespace {
int g_device = 0;
uint64_t g_next = (1ull << 40) + (1ull << 39);

CUresult fake_encode(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                     const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                     CUtensorMapL2promotion, CUtensorMapFloatOOBfill) {
  return CUDA_SUCCESS;
}
}  // namespace

extern "C" {

// What was launched: how often in all, on which device the last time, and of
// the last product its token tile and whether its K steps were dealt out.
int fake_launches = 0, fake_launch_device = -1, fake_tile = 0, fake_balanced = -1;

cudaError_t cudaGetDevice(int* d) {
  *d = g_device;
  return cudaSuccess;
}
cudaError_t cudaSetDevice(int d) {
  g_device = d;
  return cudaSuccess;
}
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr a, int) {
  *v = a == cudaDevAttrComputeCapabilityMajor ? 10 : a == cudaDevAttrComputeCapabilityMinor ? 3 : 152;
  return cudaSuccess;
}
cudaError_t cudaPointerGetAttributes(cudaPointerAttributes* at, const void* p) {
  const uint64_t a = reinterpret_cast<uint64_t>(p);
  const int dev = static_cast<int>((a >> 40) & 15) - 1;
  at->device = dev;
  at->type = dev < 0 ? cudaMemoryTypeUnregistered : (a >> 44) & 1 ? cudaMemoryTypeManaged : cudaMemoryTypeDevice;
  return cudaSuccess;
}
cudaError_t cudaMalloc(void** p, size_t n) {
  *p = reinterpret_cast<void*>(g_next + (static_cast<uint64_t>(g_device) << 40));
  g_next += (n + 255) / 256 * 256;
  return cudaSuccess;
}
cudaError_t cudaFree(void*) { return cudaSuccess; }
cudaError_t cudaMemset(void*, int, size_t) { return cudaSuccess; }
cudaError_t cudaMemsetAsync(void*, int, size_t, cudaStream_t) {
  ++fake_launches;
  fake_launch_device = g_device;
  return cudaSuccess;
}
cudaError_t cudaMemcpyAsync(void*, const void*, size_t, cudaMemcpyKind, cudaStream_t) { return cudaSuccess; }
cudaError_t cudaDeviceSynchronize() { return cudaSuccess; }
cudaError_t cudaStreamSynchronize(cudaStream_t) { return cudaSuccess; }
cudaError_t cudaGetLastError() { return cudaSuccess; }
const char* cudaGetErrorName(cudaError_t) { return "fake"; }
cudaError_t cudaGetDriverEntryPointByVersion(const char*, void** fn, unsigned, unsigned long long,
                                             cudaDriverEntryPointQueryResult* q) {
  *fn = reinterpret_cast<void*>(fake_encode);
  *q = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}
void** __cudaRegisterFatBinary(void*) {
  static void* handle = nullptr;
  return &handle;
}
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}

}  // extern "C"

namespace moe {

static cudaError_t launched() {
  ++fake_launches;
  fake_launch_device = g_device;
  return cudaSuccess;
}

cudaError_t launch_mx4_quantize(int, Mx4QuantizeArgs, cudaStream_t) { return launched(); }
cudaError_t launch_mx4_gather(const Mx4GatherArgs&, cudaStream_t) { return launched(); }
cudaError_t launch_mx4_tile_scales(const uint8_t*, int, int, bool, int, int, int, int, uint8_t*, cudaStream_t) {
  return cudaSuccess;
}
cudaError_t mx4_gemm_prepare() { return cudaSuccess; }
cudaError_t launch_mx4_gemm(bool, int tile_n, const CUtensorMap*, const CUtensorMap*, const CUtensorMap*,
                            const Mx4GemmArgs& a, int, cudaStream_t) {
  fake_tile = tile_n;
  fake_balanced = a.balanced;
  return launched();
}
bool norm_types_ok(int s, int b) { return s >= 0 && s < 3 && b >= 0 && b < 3 && (s == b || s == 2); }
cudaError_t launch_norm(int, int, const NormArgs&, int, cudaStream_t) { return launched(); }
int norm_bwd_parts(int, int, int) { return 1; }
cudaError_t launch_norm_bwd(int, int, const NormBwdArgs&, int, cudaStream_t) { return launched(); }

}  // namespace moe
