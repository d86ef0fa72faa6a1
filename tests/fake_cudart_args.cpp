// fake_cudart.cpp, with the first argument of a launch kept for a look.
#define cudaLaunchKernelExC fake_plain_launch
#include "fake_cudart.cpp"
#undef cudaLaunchKernelExC

#include <cstring>

extern "C" {
static unsigned char g_arg[112];
const unsigned char* fake_first_arg() { return g_arg; }
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* kernel, void** args) {
  std::memcpy(g_arg, args[0], sizeof(g_arg));
  return fake_plain_launch(c, kernel, args);
}
}
