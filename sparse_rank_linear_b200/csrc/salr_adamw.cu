// salr_adamw.cu - host side of salr_adamw: argument checks, the tensor tables that travel
// in the kernels' parameters, and the launches.
#include "salr_adamw.cuh"

#include <algorithm>
#include <cmath>
#include <cstring>

#include "salr_host.h"

using namespace salr;

namespace {

// Tables of two sizes: the parameters of a launch are copied whole, and a step over a few
// tensors should not carry the 32 KB of a whole model's, which is as long as the kernel
// parameters may be.
constexpr size_t kParameterBytes = 32764;
constexpr int kFewTensors = 24;
constexpr int kManyTensors = 1 + static_cast<int>((kParameterBytes - sizeof(AdamTable<1>)) /
                                                  (sizeof(AdamTensor) + sizeof(int)));
static_assert(sizeof(AdamTable<kManyTensors>) <= kParameterBytes, "kernel parameter space");
static_assert(kManyTensors == 480, "salr.h gives the count");
static_assert(sizeof(AdamTensor) == sizeof(salr_adamw_tensor), "same table entry");

template <int MAXT, typename PT, typename GT, bool MASTER, bool EIGHT>
int launch(const AdamTable<MAXT>& tab, int dev, cudaStream_t st) {
  const auto kern = salr_adamw_kernel<MAXT, PT, GT, MASTER, EIGHT>;
  static std::atomic<int> resident[64];  // CTAs per SM; zero-initialised: not looked up yet
  if (!resident[dev]) {
    int n = 0;
    SALR_TRY(cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, kAdamThreads, 0));
    resident[dev] = n > 0 ? n : 1;
  }
  // One block a warp while all CTAs are resident; then up to four times as many CTAs as are,
  // of 64 blocks or more, so that the SMs even out at the end.
  const int total = tab.start[tab.count], slots = device_sms(dev) * resident[dev].load();
  const int grid = std::max(1, std::min((total + 7) / 8, std::max(slots, std::min(4 * slots, total / 64))));
  kern<<<grid, kAdamThreads, 0, st>>>(tab);
  SALR_TRY(cudaGetLastError());
  return SALR_OK;
}

template <int MAXT, typename PT, bool MASTER, bool EIGHT>
int launch_grad(const AdamTable<MAXT>& tab, int grad_type, int dev, cudaStream_t st) {
  return grad_type == SALR_BF16 ? launch<MAXT, PT, __nv_bfloat16, MASTER, EIGHT>(tab, dev, st)
                                : launch<MAXT, PT, float, MASTER, EIGHT>(tab, dev, st);
}
template <int MAXT, typename PT, bool MASTER>
int launch_state(const AdamTable<MAXT>& tab, const salr_adamw_config* c, int dev, cudaStream_t st) {
  return c->state_bits == 8 ? launch_grad<MAXT, PT, MASTER, true>(tab, c->grad_type, dev, st)
                            : launch_grad<MAXT, PT, MASTER, false>(tab, c->grad_type, dev, st);
}
template <int MAXT>
int launch_param(const AdamTable<MAXT>& tab, const salr_adamw_config* c, int dev, cudaStream_t st) {
  if (c->param_type == SALR_FP32) return launch_state<MAXT, float, false>(tab, c, dev, st);
  return c->master ? launch_state<MAXT, __nv_bfloat16, true>(tab, c, dev, st)
                   : launch_state<MAXT, __nv_bfloat16, false>(tab, c, dev, st);
}

AdamScalars scalars(const salr_adamw_config* c) {
  AdamScalars s;
  s.lr = c->lr;
  s.beta1 = c->beta1;
  s.beta2 = c->beta2;
  s.weight_decay = c->weight_decay;
  s.eps = static_cast<float>(c->eps);
  s.b1 = static_cast<float>(c->beta1);
  s.ob1 = static_cast<float>(1.0 - c->beta1);
  s.b2 = static_cast<float>(c->beta2);
  s.ob2 = static_cast<float>(1.0 - c->beta2);
  s.lr_dev = static_cast<const float*>(c->lr_dev);
  s.grad_scale = static_cast<const float*>(c->grad_scale);
  s.step = static_cast<long long*>(c->step);
  s.last = 0;
  return s;
}

bool skipped(const salr_adamw_tensor& t) { return t.n == 0 || !t.grad; }

// Launches over tensors [0, count): as many tensors at a time as a table holds.
template <int MAXT>
int run(const salr_adamw_tensor* tensors, int64_t count, const salr_adamw_config* c, int dev,
        cudaStream_t st) {
  AdamTable<MAXT> tab;
  tab.s = scalars(c);
  int64_t i = 0;
  do {
    tab.count = 0;
    int64_t blocks = 0;
    for (; i < count && tab.count < MAXT; ++i) {
      if (skipped(tensors[i])) continue;
      const int64_t add = (tensors[i].n + kAdamBlock - 1) / kAdamBlock;
      if (blocks + add > (1ll << 30)) break;  // block numbers are 32 bits
      tab.start[tab.count] = static_cast<int>(blocks);
      std::memcpy(&tab.t[tab.count++], &tensors[i], sizeof(AdamTensor));
      blocks += add;
    }
    while (i < count && skipped(tensors[i])) ++i;
    tab.start[tab.count] = static_cast<int>(blocks);
    tab.s.last = i == count;
    const int rc = launch_param(tab, c, dev, st);
    if (rc != SALR_OK) return rc;
  } while (i < count);
  return SALR_OK;
}

bool misaligned(const void* p, uintptr_t bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0;
}

int check(const salr_adamw_tensor* tensors, int64_t count, const salr_adamw_config* c) {
  if (!c || count < 0 || (count > 0 && !tensors) || !c->step) return SALR_ERR_INVALID;
  if ((c->param_type != SALR_BF16 && c->param_type != SALR_FP32) ||
      (c->grad_type != SALR_BF16 && c->grad_type != SALR_FP32))
    return SALR_ERR_INVALID;
  if (c->state_bits != 8 && c->state_bits != 32) return SALR_ERR_INVALID;
  if (c->master && c->param_type != SALR_BF16) return SALR_ERR_INVALID;
  if (!std::isfinite(c->lr) || !(c->beta1 >= 0 && c->beta1 < 1) || !(c->beta2 >= 0 && c->beta2 < 1) ||
      !(c->eps >= 0) || !std::isfinite(c->eps) || !std::isfinite(c->weight_decay))
    return SALR_ERR_INVALID;
  const uintptr_t pb = c->param_type == SALR_BF16 ? 2 : 4, gb = c->grad_type == SALR_BF16 ? 2 : 4;
  if (misaligned(c->step, 8) || misaligned(c->lr_dev, 4) || misaligned(c->grad_scale, 4))
    return SALR_ERR_UNSUPPORTED;
  for (int64_t i = 0; i < count; ++i) {
    const salr_adamw_tensor& t = tensors[i];
    if (t.n < 0) return SALR_ERR_INVALID;
    if (skipped(t)) continue;
    if (!t.param || !t.exp_avg || !t.exp_avg_sq || (c->master && !t.master)) return SALR_ERR_INVALID;
    if (c->state_bits == 8 && (!t.exp_avg_scale || !t.exp_avg_sq_scale)) return SALR_ERR_INVALID;
    if (t.n > (1ll << 38)) return SALR_ERR_UNSUPPORTED;
    if (misaligned(t.param, pb) || misaligned(t.grad, gb) || misaligned(t.exp_avg, 16) ||
        misaligned(t.exp_avg_sq, 16) || (c->master && misaligned(t.master, 16)) ||
        misaligned(t.exp_avg_scale, 4) || misaligned(t.exp_avg_sq_scale, 4))
      return SALR_ERR_UNSUPPORTED;
  }
  return SALR_OK;
}

}  // namespace

extern "C" int salr_adamw(const salr_adamw_tensor* tensors, int64_t count,
                          const salr_adamw_config* config, void* stream) {
  const int rc = check(tensors, count, config);
  if (rc != SALR_OK) return rc;
  int dev = 0;
  SALR_TRY(cudaGetDevice(&dev));
  if (dev < 0 || dev >= 64) return SALR_ERR_UNSUPPORTED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return count <= kFewTensors ? run<kFewTensors>(tensors, count, config, dev, st)
                              : run<kManyTensors>(tensors, count, config, dev, st);
}
