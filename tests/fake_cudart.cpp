// A stand-in for the CUDA runtime beneath one object file of the library
// (attention over runs): every call succeeds and is written to a log, nothing
// runs.  Lets host code be checked without a GPU: the order of its calls, the
// device they ask about, the grid that they launch.
#include <cuda.h>
#include <cuda_runtime_api.h>

#include <cstdint>
#include <string>

namespace {
std::string g_log;
int g_device = 0, g_sms[2] = {152, 152}, g_error_word = 0;
cudaError_t note(const std::string& what) {
  g_log += (g_log.empty() ? "" : " ") + what;
  return cudaSuccess;
}
}  // namespace

// what the object file takes from the rest of the library
namespace pf {
void set_op_error(const std::string&) {}
bool encode_fp16_sw128(CUtensorMap*, const void*, int, const uint64_t*, const uint64_t*, const uint32_t*, std::string*) {
  return true;
}
bool encode_fp16_sw64(CUtensorMap*, const void*, int, const uint64_t*, const uint64_t*, const uint32_t*, std::string*) {
  return true;
}
}  // namespace pf

extern "C" {
const char* fake_log() { return g_log.c_str(); }
void fake_reset(int device, int sms0, int sms1, int error_word) {
  g_log.clear();
  g_device = device, g_sms[0] = sms0, g_sms[1] = sms1, g_error_word = error_word;
}

cudaError_t cudaGetDevice(int* device) {
  *device = g_device;
  return cudaSuccess;
}
cudaError_t cudaDeviceGetAttribute(int* value, cudaDeviceAttr, int device) {
  *value = g_sms[device];
  return cudaSuccess;
}
cudaError_t cudaMemcpyAsync(void* dst, const void*, size_t n, cudaMemcpyKind kind, cudaStream_t) {
  if (kind == cudaMemcpyDeviceToHost && n == sizeof(int)) *static_cast<int*>(dst) = g_error_word;
  return note("copy");
}
cudaError_t cudaMemsetAsync(void*, int value, size_t n, cudaStream_t) {
  return note("set:" + std::to_string(value) + "x" + std::to_string(n));
}
cudaError_t cudaStreamSynchronize(cudaStream_t) { return note("sync"); }
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void*, void**) {
  return note("launch:" + std::to_string(c->gridDim.x) + "x" + std::to_string(c->blockDim.x));
}
cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute, int) { return cudaSuccess; }
cudaError_t cudaGetLastError() { return cudaSuccess; }
const char* cudaGetErrorString(cudaError_t) { return "fake"; }

// registration of the object's kernels at load time
void** __cudaRegisterFatBinary(void*) {
  static void* handle = nullptr;
  return &handle;
}
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
void __cudaRegisterFunction(void**, const char*, char*, const char*, int, void*, void*, void*, void*, int*) {}
unsigned __cudaPopCallConfiguration(void*, void*, size_t*, void*) { return 1; }
cudaError_t __cudaGetKernel(void**, const void*) { return cudaErrorNotSupported; }
cudaError_t __cudaLaunchKernel(void*, dim3, dim3, void**, size_t, cudaStream_t) { return cudaErrorNotSupported; }
}
