// Calls one function of the library on a machine without a GPU and prints the
// kernel launches it makes.  The program's own definitions of the HIP calls the
// library imports come first in symbol lookup; the launch takes what HIP
// documents (threads per grid dimension below 2^32) and refuses the rest, as the
// runtime does.
//   launch_probe library function args...      (integers; pointers are integers)
// prints "launch kernel gx gy gz bx by bz" per launch and "status n" at the end; for
// kernels with the text of PROBE_WORDS in their name, whose first argument has to
// be a struct of 144 bytes or more, also that struct's first 18 words.
#include <dlfcn.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <map>
#include <string>

struct Dim {
  uint32_t x, y, z;
};
static std::map<const void*, std::string> names;
static Dim grid_, block_;
static size_t shmem_;
static void* stream_;
static int last;

extern "C" {
void** __hipRegisterFatBinary(const void*) {
  static void* module;
  return &module;
}
void __hipUnregisterFatBinary(void**) {}
void __hipRegisterFunction(void**, const void* host, char*, const char* name, unsigned, void*,
                           void*, void*, void*, int*) {
  names[host] = name;
}
void __hipRegisterVar(void**, void*, char*, char*, int, size_t, int, int) {}
int __hipPushCallConfiguration(Dim grid, Dim block, size_t shmem, void* stream) {
  grid_ = grid;
  block_ = block;
  shmem_ = shmem;
  stream_ = stream;
  return 0;
}
int __hipPopCallConfiguration(Dim* grid, Dim* block, size_t* shmem, void** stream) {
  *grid = grid_;
  *block = block_;
  *shmem = shmem_;
  *stream = stream_;
  return 0;
}
int hipGetDevice(int* dev) {
  *dev = 0;
  return 0;
}
int hipFuncSetAttribute(const void*, int, int) { return 0; }
int hipDeviceGetAttribute(int* v, int, int) {
  *v = 256;
  return 0;
}
int hipGetLastError() {
  const int e = last;
  last = 0;
  return e;
}
int hipLaunchKernel(const void* f, Dim g, Dim b, void** args, size_t, void*) {
  const uint64_t most = (uint64_t)1 << 32;
  const bool ok = g.x && g.y && g.z && b.x && b.y && b.z && (uint64_t)g.x * b.x < most &&
                  (uint64_t)g.y * b.y < most && (uint64_t)g.z * b.z < most && g.y < 65536 &&
                  g.z < 65536 && (uint64_t)b.x * b.y * b.z <= 1024;
  if (!ok) {
    last = 9;   // hipErrorInvalidConfiguration
    printf("refused %s %u %u %u %u %u %u\n", names[f].c_str(), g.x, g.y, g.z, b.x, b.y, b.z);
    return last;
  }
  printf("launch %s %u %u %u %u %u %u", names[f].c_str(), g.x, g.y, g.z, b.x, b.y, b.z);
  const char* with = getenv("PROBE_WORDS");
  if (with && names[f].find(with) != std::string::npos) {
    uint64_t w[18];
    memcpy(w, args[0], sizeof(w));
    for (uint64_t v : w) printf(" %llu", (unsigned long long)v);
  }
  printf("\n");
  return 0;
}
}

int main(int argc, char** argv) {
  void* lib = argc > 2 ? dlopen(argv[1], RTLD_NOW) : nullptr;
  void* f = lib ? dlsym(lib, argv[2]) : nullptr;
  if (!f) {
    fprintf(stderr, "%s\n", dlerror());
    return 2;
  }
  long long a[20] = {};
  for (int i = 3; i < argc && i < 23; ++i) a[i - 3] = strtoll(argv[i], nullptr, 0);
  typedef int (*Fn)(long long, long long, long long, long long, long long, long long, long long,
                    long long, long long, long long, long long, long long, long long, long long,
                    long long, long long, long long, long long, long long, long long);
  const int st = ((Fn)f)(a[0], a[1], a[2], a[3], a[4], a[5], a[6], a[7], a[8], a[9], a[10], a[11],
                         a[12], a[13], a[14], a[15], a[16], a[17], a[18], a[19]);
  printf("status %d\n", st);
  return 0;
}
