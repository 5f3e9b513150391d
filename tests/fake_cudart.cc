// The CUDA runtime calls that the library's host code makes, as a recorder: nothing runs on a
// GPU.  Linked with the library's objects in place of the runtime, it lets tests look at what
// the entry points do on the host: which kernels they launch, in which order, from which
// thread, on which device, and whether a kernel was set up on that device first.
//
// Device 0 has 152 SMs and room for 76 clusters, device 1 has 20 and 10 (or what a test says for
// clusters of a size).  As in CUDA, a kernel's
// shared-memory attribute belongs to one device, and a launch that asks for more than 48 KB
// without it fails.
#include <unistd.h>

#include <atomic>
#include <cstddef>
#include <cstdint>
#include <cstring>
#include <map>
#include <mutex>
#include <string>
#include <utility>
#include <vector>

namespace {

enum { kLookup = 0, kLaunch = 1, kMalloc = 2, kFree = 3 };
struct Event {
  int kind, thread, device;
  int64_t value;   // a launch's blocks, an allocation's address
  int cluster;     // blocks of a launch's clusters
  std::string name;
};
struct Dim3 {
  unsigned x, y, z;
};
struct Config {
  Dim3 grid, block;
  size_t smem;
  void* stream;
};
// cudaLaunchConfig_t
struct LaunchConfig {
  Dim3 grid, block;
  size_t smem;
  void* stream;
  void* attrs;
  unsigned num_attrs;
};

// cudaLaunchAttribute
struct LaunchAttribute {
  int id, pad;
  union {
    Dim3 dim;
    char bytes[64];
  };
};
int cluster_of(const LaunchConfig* c) {
  const LaunchAttribute* a = static_cast<const LaunchAttribute*>(c->attrs);
  for (unsigned i = 0; i < c->num_attrs; ++i)
    if (a[i].id == 4) return static_cast<int>(a[i].dim.x);   // cudaLaunchAttributeClusterDimension
  return 1;
}

struct State {
  std::mutex mu;
  std::map<std::pair<int, int>, int> clusters;       // (device, blocks) -> room for them
  std::map<const void*, std::string> names;
  std::map<std::pair<int, const void*>, int> smem;   // (device, kernel) -> attribute
  std::vector<Event> log;
  uintptr_t next = uintptr_t(1) << 40;
};
State& state() {
  static State s;
  return s;
}
std::atomic<int> g_threads{0}, g_delay_us{0};
thread_local int t_thread = g_threads++, t_device = 0, t_error = 0;
thread_local Config t_config;

constexpr int kSms[2] = {152, 20};

int fail(int e) {
  t_error = e;
  return e;
}
void pause_thread() {
  if (g_delay_us) usleep(g_delay_us);
}
void record(int kind, int64_t value, const std::string& name, int cluster = 1) {
  State& s = state();
  std::lock_guard<std::mutex> lk(s.mu);
  s.log.push_back(Event{kind, t_thread, t_device, value, cluster, name});
}
bool set_up(const void* f, size_t smem) {
  State& s = state();
  std::lock_guard<std::mutex> lk(s.mu);
  const auto it = s.smem.find({t_device, f});
  return smem <= 48 * 1024 || (it != s.smem.end() && static_cast<size_t>(it->second) >= smem);
}
int launch(const void* f, Dim3 grid, size_t smem, int cluster = 1) {
  if (!set_up(f, smem)) return fail(1);
  std::string name;
  {
    State& s = state();
    std::lock_guard<std::mutex> lk(s.mu);
    name = s.names[f];
  }
  record(kLaunch, grid.x, name, cluster);
  pause_thread();
  return 0;
}
int encode_tiled(...) { return 0; }

}  // namespace

extern "C" {

// ---- for the tests
void fake_set_device(int d) { t_device = d; }
void fake_set_delay_us(int us) { g_delay_us = us; }
int fake_thread() { return t_thread; }
void fake_set_clusters(int device, int blocks, int n) {
  State& s = state();
  std::lock_guard<std::mutex> lk(s.mu);
  s.clusters[{device, blocks}] = n;
}
int fake_event_cluster(int i) { return state().log[i].cluster; }
void fake_clear() {
  State& s = state();
  std::lock_guard<std::mutex> lk(s.mu);
  s.log.clear();
}
int fake_events() { return static_cast<int>(state().log.size()); }
int fake_event(int i, int* thread, int* device, int64_t* value, char* name, int n) {
  const Event& e = state().log[i];
  *thread = e.thread;
  *device = e.device;
  *value = e.value;
  std::strncpy(name, e.name.c_str(), n - 1);
  name[n - 1] = 0;
  return e.kind;
}

// ---- what compiled kernels' host stubs call
void** __cudaRegisterFatBinary(void*) {
  static void* handle;
  return &handle;
}
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
void __cudaRegisterVar(void**, char*, char*, const char*, int, size_t, int, int) {}
void __cudaRegisterFunction(void**, const char* host, char*, const char* name, int, void*, void*, void*,
                            void*, int*) {
  State& s = state();
  std::lock_guard<std::mutex> lk(s.mu);
  s.names[host] = name;
}
unsigned __cudaPushCallConfiguration(Dim3 grid, Dim3 block, size_t smem, void* stream) {
  t_config = Config{grid, block, smem, stream};
  return 0;
}
int __cudaPopCallConfiguration(Dim3* grid, Dim3* block, size_t* smem, void* stream) {
  *grid = t_config.grid;
  *block = t_config.block;
  *smem = t_config.smem;
  *static_cast<void**>(stream) = t_config.stream;
  return 0;
}
int __cudaGetKernel(const void** kernel, const void* f) {
  *kernel = f;
  return 0;
}
int __cudaLaunchKernel(const void* f, Dim3 grid, Dim3, void**, size_t smem, void*) {
  return launch(f, grid, smem);
}

// ---- the runtime
int cudaLaunchKernelExC(const LaunchConfig* c, const void* f, void**) {
  return launch(f, c->grid, c->smem, cluster_of(c));
}
int cudaGetLastError() {
  const int e = t_error;
  t_error = 0;
  return e;
}
int cudaGetDevice(int* d) {
  *d = t_device;
  return 0;
}
int cudaDeviceGetAttribute(int* v, int, int device) {
  *v = kSms[device];
  return 0;
}
int cudaFuncSetAttribute(const void* f, int, int value) {
  State& s = state();
  std::lock_guard<std::mutex> lk(s.mu);
  s.smem[{t_device, f}] = value;
  return 0;
}
int cudaOccupancyMaxActiveClusters(int* n, const void* f, const LaunchConfig* c) {
  if (!set_up(f, c->smem)) return fail(1);
  State& s = state();
  std::lock_guard<std::mutex> lk(s.mu);
  const auto it = s.clusters.find({t_device, cluster_of(c)});
  *n = it != s.clusters.end() ? it->second : kSms[t_device] / 2;
  return 0;
}
int cudaOccupancyMaxActiveBlocksPerMultiprocessorWithFlags(int* n, const void* f, int, size_t smem,
                                                           unsigned) {
  if (!set_up(f, smem)) return fail(1);
  *n = 1;
  return 0;
}
int cudaGetDriverEntryPointByVersion(const char*, void** fn, unsigned, unsigned long long, int* found) {
  *fn = reinterpret_cast<void*>(&encode_tiled);
  *found = 0;
  return 0;
}
int cudaGetSymbolAddress(void** p, const void*) {
  *p = reinterpret_cast<void*>(uintptr_t(1) << 32);
  return 0;
}
int cudaStreamIsCapturing(void*, int* status) {
  *status = 0;
  record(kLookup, 0, "");
  pause_thread();
  return 0;
}
int cudaMalloc(void** p, size_t n) {
  {
    State& s = state();
    std::lock_guard<std::mutex> lk(s.mu);
    *p = reinterpret_cast<void*>(s.next);
    s.next += (n + 4095) / 4096 * 4096;
  }
  record(kMalloc, reinterpret_cast<intptr_t>(*p), "");
  return 0;
}
int cudaFree(void* p) {
  record(kFree, reinterpret_cast<intptr_t>(p), "");
  return 0;
}
int cudaMemcpy(void* dst, const void* src, size_t n, int kind) {
  if (kind == 2) std::memset(dst, 0, n);   // device to host
  (void)src;
  return 0;
}
int cudaMemset(void*, int, size_t) { return 0; }
int cudaMemsetAsync(void*, int, size_t, void*) { return 0; }
int cudaStreamSynchronize(void*) { return 0; }
int cudaDeviceSynchronize() { return 0; }
int cudaEventCreate(void** e) {
  *e = nullptr;
  return 0;
}
int cudaEventDestroy(void*) { return 0; }
int cudaEventRecord(void*, void*) { return 0; }
int cudaEventSynchronize(void*) { return 0; }
int cudaEventElapsedTime(float* ms, void*, void*) {
  *ms = 1.f;
  return 0;
}

}  // extern "C"
