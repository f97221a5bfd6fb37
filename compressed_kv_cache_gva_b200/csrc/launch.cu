// Record of the function attributes already applied, per kernel and CUDA context.
//
// cudaFuncSetAttribute changes per-context state of a kernel; setting it on every
// launch costs host time on the eager path.  The launchers ask here first and
// apply an attribute only when the current context has not yet received an equal
// or larger value for that kernel.  The record is keyed by the context, so after
// cudaDeviceReset (a new primary context) the attributes are applied again.
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdlib.h>

#include <map>
#include <mutex>
#include <tuple>

#include "launch.h"

namespace gva {

namespace {
std::mutex g_mu;
std::map<std::tuple<const void*, const void*, int>, long long> g_applied;   // (kernel, ctx, attr)

typedef CUresult (*CtxGetCurrentFn)(CUcontext*);

// The current context (the runtime makes the device's primary context current).
const void* current_context() {
  static CtxGetCurrentFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuCtxGetCurrent", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<CtxGetCurrentFn>(p);
  });
  CUcontext c = nullptr;
  if (!fn || fn(&c) != CUDA_SUCCESS) return nullptr;
  return c;
}
}  // namespace

bool attr_applied(const void* kernel, int attr, long long value) {
  const void* ctx = current_context();
  if (!ctx) return false;
  std::lock_guard<std::mutex> lk(g_mu);
  const auto it = g_applied.find(std::make_tuple(kernel, ctx, attr));
  return it != g_applied.end() && it->second >= value;
}

void attr_record(const void* kernel, int attr, long long value) {
  const void* ctx = current_context();
  if (!ctx) return;
  std::lock_guard<std::mutex> lk(g_mu);
  long long& v = g_applied[std::make_tuple(kernel, ctx, attr)];
  if (value > v) v = value;
}

int cluster_that_fits(const void* kernel, int want, int threads, size_t smem) {
#ifdef GVA_TEST_CLUSTER_LIMIT   // test builds only: larger clusters count as not fitting
  const char* limit = getenv("GVA_TEST_CLUSTER_LIMIT");
  while (limit && want > atoi(limit) && want > 1) want >>= 1;
#endif
  static std::mutex mu;
  static std::map<std::tuple<const void*, const void*, int, int>, int> found;   // (kernel, ctx, threads, want)
  const auto key = std::make_tuple(kernel, current_context(), threads, want);
  std::lock_guard<std::mutex> lk(mu);
  const auto it = found.find(key);
  if (it != found.end()) return it->second;
  int cl = want;
  for (; cl > 1; cl >>= 1) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cl;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(cl);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) == cudaSuccess && n > 0) break;
    cudaGetLastError();   // "does not fit" is an answer here
  }
  if (std::get<1>(key)) found[key] = cl;
  return cl;
}

}  // namespace gva
