// A stand-in for the CUDA runtime, for host tests of what the library does when a launch fails: the C
// API (api.cu) and the launch code under test are linked against this file instead of libcudart. Nothing
// runs; every launch is recorded by its kernel's name, and one of them, the n-th, is refused.
#include <cstring>
#include <map>
#include <string>
#include <vector>

namespace {
// (used by other files' static initialisers)
std::map<const void*, std::string>& names() {
  static std::map<const void*, std::string> n;
  return n;
}
std::vector<std::string> launches;
int fail_at = -1, fail_code = 0, refused_attributes = 0, last_error = 0, ctas_per_sm = 32;
char memory[64];

int launch(const void* f) {
  if ((int)launches.size() == fail_at) {
    fail_at = -1;
    return last_error = fail_code;
  }
  launches.push_back(names()[f]);
  return 0;
}
}  // namespace

extern "C" {
// ------------------------------------------------------------ for the tests
void fake_reset(int nth, int code) {
  launches.clear();
  fail_at = nth;
  fail_code = code;
  last_error = 0;
}
// the next question for a kernel's attributes fails
void fake_refuse_attributes(int code) { refused_attributes = code; }
void fake_set_ctas_per_sm(int n) { ctas_per_sm = n; }
int fake_launches() { return (int)launches.size(); }
const char* fake_launch(int i) { return launches[i].c_str(); }
int fake_last_error() { return last_error; }
void fake_set_last_error(int e) { last_error = e; }

// ------------------------------------------------------------ what nvcc's host code registers
void** __cudaRegisterFatBinary(void*) {
  static void* handle;
  return &handle;
}
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
void __cudaRegisterFunction(void**, const char* host, char*, const char* name, int, void*, void*, void*, void*, int*) {
  names()[host] = name;
}
void __cudaRegisterVar(void**, char*, char*, const char*, int, size_t, int, int) {}
int __cudaGetKernel(void** kernel, const void* f) {
  *kernel = const_cast<void*>(f);
  return 0;
}
unsigned __cudaPushCallConfiguration(...) { return 0; }
int __cudaPopCallConfiguration(...) { return 0; }

// ------------------------------------------------------------ the runtime
int __cudaLaunchKernel(const void* f, ...) { return launch(f); }
int cudaLaunchKernelExC(const void*, const void* f, void**) { return launch(f); }
int cudaGetDevice(int* d) {
  *d = 0;
  return 0;
}
int cudaGetLastError() {
  const int e = last_error;
  last_error = 0;
  return e;
}
const char* cudaGetErrorString(int) { return "an error of the test's"; }
int cudaGetSymbolAddress(void** p, const void*) {
  *p = memory;
  return 0;
}
int cudaOccupancyMaxActiveBlocksPerMultiprocessor(int* n, const void*, int, size_t) {
  *n = ctas_per_sm;
  return 0;
}
int cudaOccupancyMaxActiveBlocksPerMultiprocessorWithFlags(int* n, const void*, int, size_t, unsigned) {
  *n = ctas_per_sm;
  return 0;
}
int cudaFuncSetAttribute(const void*, int, int) { return 0; }
int cudaMemcpy(void* dst, const void* src, size_t n, int) {
  std::memcpy(dst, src, n);
  return 0;
}
int cudaMemset(void* p, int v, size_t n) {
  std::memset(p, v, n);
  return 0;
}
int cudaMemcpyAsync(void*, const void*, size_t, int, void*) { return 0; }
int cudaDeviceSynchronize() { return 0; }
int cudaPointerGetAttributes(void*, const void*) { return 1; }
int cudaDeviceGetAttribute(int* v, int, int) {
  *v = 152;
  return 0;
}
// of the attributes only the registers per thread, behind three sizes and the largest block
int cudaFuncGetAttributes(void* at, const void*) {
  if (refused_attributes) {
    last_error = refused_attributes;
    refused_attributes = 0;
    return last_error;
  }
  static_cast<int*>(at)[7] = 168;
  return 0;
}
// the one driver function that is looked up: encodes a tensor map
int fake_encode(...) { return 0; }
int cudaGetDriverEntryPointByVersion(const char*, void** f, unsigned, unsigned long long, int* found) {
  *f = reinterpret_cast<void*>(&fake_encode);
  *found = 0;
  return 0;
}
}

namespace sparda {
__attribute__((weak)) int sm_count() { return 152; }      // (attn.cu's, where that is linked)
}  // namespace sparda
