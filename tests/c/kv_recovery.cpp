// What ltk_kv_status does after an error, run on the host: the CUDA calls that kv_api.cu makes are
// stand-ins with "device" memory on the heap.  Work on a stream happens when that stream is
// synchronised; work on the legacy stream, which other streams do not wait for, only when the
// device is.
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <functional>
#include <map>
#include <vector>

#include <cuda_runtime_api.h>

#include "ltk.h"

namespace ltk {
struct AppendParams;
struct AttnParams;
}  // namespace ltk

static std::map<cudaStream_t, std::vector<std::function<void()>>> queued;
static std::map<size_t, void*> by_size;
static const int kCounters = 11;

static void run(cudaStream_t s) {
  for (auto& f : queued[s]) f();
  queued[s].clear();
}

extern "C" {
void** __cudaRegisterFatBinary(void*) { static void* h; return &h; }
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
cudaError_t CUDARTAPI cudaGetDevice(int* d) { *d = 0; return cudaSuccess; }
cudaError_t CUDARTAPI cudaDeviceGetAttribute(int* v, enum cudaDeviceAttr, int) { *v = 4; return cudaSuccess; }
cudaError_t CUDARTAPI cudaGetLastError(void) { return cudaSuccess; }
const char* CUDARTAPI cudaGetErrorString(cudaError_t) { return ""; }
cudaError_t CUDARTAPI cudaMalloc(void** p, size_t n) { *p = by_size[n] = std::malloc(n); return cudaSuccess; }
cudaError_t CUDARTAPI cudaFree(void* p) { std::free(p); return cudaSuccess; }
cudaError_t CUDARTAPI cudaMemset(void* p, int v, size_t n) {
  queued[nullptr].push_back([=] { std::memset(p, v, n); });
  return cudaSuccess;
}
cudaError_t CUDARTAPI cudaMemsetAsync(void* p, int v, size_t n, cudaStream_t s) {
  queued[s].push_back([=] { std::memset(p, v, n); });
  return cudaSuccess;
}
cudaError_t CUDARTAPI cudaMemcpyAsync(void* d, const void* a, size_t n, enum cudaMemcpyKind, cudaStream_t s) {
  queued[s].push_back([=] { std::memcpy(d, a, n); });
  return cudaSuccess;
}
cudaError_t CUDARTAPI cudaStreamSynchronize(cudaStream_t s) { run(s); return cudaSuccess; }
cudaError_t CUDARTAPI cudaDeviceSynchronize(void) {
  for (auto& q : queued) run(q.first);
  return cudaSuccess;
}
}

namespace ltk {
std::size_t kv_rows_part_floats(int) { return 100; }
std::size_t kv_tile_part_floats(int) { return 100; }
std::size_t kv_list_part_floats(int) { return 100; }
int kv_rows_counters(int) { return kCounters; }
int kv_tile_counters(int) { return kCounters; }
int kv_list_counters(int) { return kCounters; }
cudaError_t kv_rows_init() { return cudaSuccess; }
cudaError_t kv_tile_init() { return cudaSuccess; }
cudaError_t kv_list_init() { return cudaSuccess; }
bool kv_tile_pairs(const AttnParams&, int, int) { return false; }
cudaError_t launch_kv_append(const AppendParams&, int, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_kv_rows(const AttnParams&, int, int, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_kv_tile(const AttnParams&, int, int, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_kv_list(const AttnParams&, int, cudaStream_t) { return cudaSuccess; }
}  // namespace ltk

int main() {
  ltk_kv_config cfg{4, 2, 128, 64, 0, std::aligned_alloc(16, 16), std::aligned_alloc(16, 16),
                    static_cast<float*>(std::aligned_alloc(16, 16)), static_cast<float*>(std::aligned_alloc(16, 16))};
  ltk_kv* h = nullptr;
  if (ltk_kv_create(&cfg, &h) != LTK_OK) return std::puts("create"), 1;
  int* counters = static_cast<int*>(by_size[kCounters * 4]);
  int* status = static_cast<int*>(by_size[4]);
  for (int i = 0; i < kCounters; ++i)
    if (counters[i] != 0) return std::puts("counters at first"), 1;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(0x10);
  for (int error : {LTK_ERR_TIMEOUT, LTK_ERR_ARG, LTK_OK}) {
    for (int i = 0; i < kCounters; ++i) counters[i] = error == LTK_OK ? 0 : 7;
    *status = error;
    int value = -1;
    if (ltk_kv_status(h, &value, st) != LTK_OK || value != error) return std::printf("status %d\n", error), 1;
    // a call on the same stream may begin here
    if (*status != 0) return std::printf("status word after %d\n", error), 1;
    for (int i = 0; i < kCounters; ++i)
      if (counters[i] != 0) return std::printf("counters after %d\n", error), 1;
    if (!queued[nullptr].empty()) return std::printf("legacy stream after %d\n", error), 1;
  }
  ltk_kv_destroy(h);
  std::puts("recovery ok");
  return 0;
}
