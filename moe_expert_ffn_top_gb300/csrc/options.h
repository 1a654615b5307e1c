#pragma once
#include <cuda_runtime.h>

namespace moelora {

// Launches that need more than 48 KB of shared memory, or clusters of more than eight
// blocks, which a kernel has to be allowed once per device (some calls of about a
// microsecond).  allow_options allows a kernel all that the current device
// has, the same whatever the launch: no thread's call can take back what another thread's
// launch needs.  It notes the device once that has succeeded and does nothing there from
// then on, unless `again`: a launch that fails all the same (the device was reset) allows
// it again and is repeated.
cudaError_t allow_options(const void* kernel, bool again);
template <class... P, class... Args>
cudaError_t launch_allowed(const cudaLaunchConfig_t& cfg, bool wide_cluster, void (*kernel)(P...), Args... args) {
  // with 16 KB of static memory at most, up to 32 KB need no leave
  const bool ask = cfg.dynamicSmemBytes > 32 * 1024 || wide_cluster;
  const void* k = reinterpret_cast<const void*>(kernel);
  cudaError_t e = ask ? allow_options(k, false) : cudaSuccess;
  if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, kernel, P(args)...);
  if (e != cudaSuccess && ask) {
    (void)cudaGetLastError();
    e = allow_options(k, true);
    if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, kernel, P(args)...);
  }
  return e;
}

}  // namespace moelora
