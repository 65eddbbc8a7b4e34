// A stand-in for the calls of the HIP runtime that libbst.so makes, preloaded into a
// process without a GPU: kernels are registered under their names, and a launch is a line
// in a list instead of work.  The device has 256 CUs.
#include <cstdint>
#include <cstdio>
#include <map>
#include <string>

namespace {
struct Dim {
  uint32_t x, y, z;
};
Dim g_grid, g_block;
size_t g_shared;
void* g_stream;
std::map<const void*, std::string>& names() {
  static std::map<const void*, std::string> n;
  return n;
}
}  // namespace

extern "C" {
// file that launches are written to: kernel, workgroups, threads of a workgroup
FILE* record_to = nullptr;
void record_launches(const char* path) { record_to = fopen(path, "w"); }
void record_end() { fclose(record_to); }

void** __hipRegisterFatBinary(const void*) {
  static void* module;
  return &module;
}
void __hipUnregisterFatBinary(void**) {}
void __hipRegisterFunction(void**, const void* host, char*, const char* name, unsigned, void*, void*, void*, void*,
                           int*) {
  names()[host] = name;
}
void __hipRegisterVar(void**, void*, char*, const char*, int, size_t, int, int) {}
int __hipPushCallConfiguration(Dim grid, Dim block, size_t shared, void* stream) {
  g_grid = grid;
  g_block = block;
  g_shared = shared;
  g_stream = stream;
  return 0;
}
int __hipPopCallConfiguration(Dim* grid, Dim* block, size_t* shared, void** stream) {
  *grid = g_grid;
  *block = g_block;
  *shared = g_shared;
  *stream = g_stream;
  return 0;
}
int hipLaunchKernel(const void* f, Dim grid, Dim block, void**, size_t, void*) {
  if (record_to)
    fprintf(record_to, "%s %llu %llu\n", names().count(f) ? names()[f].c_str() : "?",
            (unsigned long long)grid.x * grid.y * grid.z, (unsigned long long)block.x * block.y * block.z);
  return 0;
}
int hipGetLastError() { return 0; }
const char* hipGetErrorString(int) { return ""; }
int hipGetDevice(int* d) {
  *d = 0;
  return 0;
}
int hipDeviceGetAttribute(int* v, int, int) {
  *v = 256;
  return 0;
}
int hipGetSymbolAddress(void** p, const void*) {
  *p = nullptr;
  return 1;
}
int hipOccupancyMaxActiveBlocksPerMultiprocessor(int* n, const void*, int, size_t) {
  *n = 1;
  return 0;
}
}
