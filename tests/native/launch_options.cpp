// Host-only check of launch_allowed against a stand-in for the CUDA runtime: what a kernel is
// allowed is kept per device, launches fail that ask for more.  One scenario per run; prints
// "ok" or what went wrong.
#include <cstdio>
#include <cstring>
#include <functional>
#include <future>
#include <map>
#include <mutex>
#include <thread>

#include "../../moe_expert_ffn_top_gb300/csrc/options.h"

namespace {

struct Allowed {
  int smem = 48 * 1024;
  bool wide = false;
};
std::mutex mu;
std::map<std::pair<int, const void*>, Allowed> allowed;
thread_local int device = 0;
// Called at this thread's next change of a memory limit, to make it at a time of its own.
thread_local std::function<void(const std::function<void()>& set)> at_set;
int failed_launches = 0, sets = 0, fail_sets = 0;
constexpr int kStatic = 9 * 1024, kOptIn = 227 * 1024;

void kernel_a(int) {}
void kernel_b(int) {}
cudaError_t launch(void (*k)(int), int smem, int cluster = 1) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = cluster;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  cfg.dynamicSmemBytes = smem;
  return moelora::launch_allowed(cfg, cluster > 8, k, 1);
}

}  // namespace

extern "C" {
cudaError_t cudaGetDevice(int* d) { return *d = device, cudaSuccess; }
cudaError_t cudaGetLastError() { return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr, int) { return *v = kOptIn, cudaSuccess; }
cudaError_t cudaFuncGetAttributes(cudaFuncAttributes* a, const void*) {
  *a = cudaFuncAttributes{};
  a->sharedSizeBytes = kStatic;
  return cudaSuccess;
}
cudaError_t cudaFuncSetAttribute(const void* f, cudaFuncAttribute what, int v) {
  const auto set_memory = [&] {
    std::lock_guard<std::mutex> l(mu);
    allowed[{device, f}].smem = v;
  };
  if (what == cudaFuncAttributeMaxDynamicSharedMemorySize && at_set) {
    const auto hook = std::move(at_set);
    at_set = nullptr;
    hook(set_memory);
    return cudaSuccess;
  }
  {
    std::lock_guard<std::mutex> l(mu);
    ++sets;
    if (fail_sets && fail_sets--) return cudaErrorInvalidValue;
    if (what == cudaFuncAttributeNonPortableClusterSizeAllowed) return allowed[{device, f}].wide = v, cudaSuccess;
    if (v + kStatic > kOptIn) return cudaErrorInvalidValue;
  }
  set_memory();
  return cudaSuccess;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* f, void**) {
  std::lock_guard<std::mutex> l(mu);
  const Allowed a = allowed[{device, f}];
  if ((int)c->dynamicSmemBytes <= a.smem && (c->attrs[0].val.clusterDim.x <= 8 || a.wide)) return cudaSuccess;
  ++failed_launches;
  return cudaErrorInvalidValue;
}
}

#define CHECK(x) \
  if (!(x)) return std::printf("%s\n", #x), 1

// Two threads at a kernel's first use, one with 180 KB and one with 100: the second comes in
// while the first is about to ask, and what it asks for takes effect last.
static int race() {
  using Set = const std::function<void()>&;
  std::promise<void> arrived, done;
  std::thread other;
  cudaError_t theirs = cudaErrorUnknown;
  at_set = [&](Set set) {
    other = std::thread([&] {
      at_set = [&](Set their_set) {
        arrived.set_value();
        done.get_future().wait();
        their_set();
      };
      theirs = launch(kernel_a, 100 << 10);
    });
    arrived.get_future().wait();
    set();
    done.set_value();
    other.join();
  };
  const cudaError_t mine = launch(kernel_a, 180 << 10);
  CHECK(theirs == cudaSuccess);
  CHECK(mine == cudaSuccess);
  CHECK(failed_launches == 0);
  return 0;
}

// A smaller launch, or one in a wide cluster, leaves a larger one what it needs.
static int no_lowering() {
  CHECK(launch(kernel_a, 200 << 10) == cudaSuccess);
  CHECK(launch(kernel_a, 100 << 10) == cudaSuccess);
  CHECK(launch(kernel_a, 64 << 10, 16) == cudaSuccess);
  CHECK(launch(kernel_a, 200 << 10) == cudaSuccess);
  CHECK(launch(kernel_b, 50 << 10) == cudaSuccess && launch(kernel_b, 1 << 10, 16) == cudaSuccess);
  CHECK(failed_launches == 0);
  const int before = sets;
  for (int i = 0; i < 5; ++i) CHECK(launch(kernel_a, (60 + 20 * i) << 10, 16) == cudaSuccess);
  CHECK(sets == before);  // asked once
  return 0;
}

// Every device is asked for by itself: no launch fails on the second one.
static int devices() {
  for (device = 0; device < 3; ++device) CHECK(launch(kernel_a, 150 << 10, 16) == cudaSuccess);
  CHECK(failed_launches == 0);
  return 0;
}

// A refusal is reported and not noted; a device that forgot (a reset) is asked again.
static int again() {
  fail_sets = 2;  // the launch asks twice
  CHECK(launch(kernel_a, 150 << 10) != cudaSuccess);
  CHECK(launch(kernel_a, 150 << 10) == cudaSuccess && failed_launches == 0);
  allowed.clear();
  CHECK(launch(kernel_a, 150 << 10) == cudaSuccess && failed_launches == 1);
  CHECK(launch(kernel_a, kOptIn) != cudaSuccess);  // more than there is
  return 0;
}

int main(int, char** v) {
  const int bad = !std::strcmp(v[1], "race")          ? race()
                  : !std::strcmp(v[1], "no_lowering") ? no_lowering()
                  : !std::strcmp(v[1], "devices")     ? devices()
                                                      : again();
  if (!bad) std::puts("ok");
  return bad;
}
