// balance.cu -- nslm_moe_balance and nslm_moe_balance_grad: the experts' counts
// and the load-balance loss of a router, and the loss's gradient.
#include <algorithm>

#include "common.cuh"

namespace nslm {
namespace {

constexpr int kMaxE = 1024;
constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxCtas = 296;
constexpr int kOneLaunchT = 1024;  // up to here one CTA, and no workspace

struct BalanceParams {
  const float *logits;
  const int32_t *ids;
  const uint8_t *mask;
  int32_t T, E, k;
  float coef;
  int32_t *counts, *offsets;
  float *mean_p, *loss;
  float *part_p;    // [CTAs][E]
  int32_t *part_c;  // [CTAs][E + 1]
};

__device__ __forceinline__ float warp_max(float v) {
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float warp_add(float v) {
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Every warp adds the softmax of its tokens to a shared row of its own.
__device__ void count_tokens(const BalanceParams &p, float *s_p, int32_t *s_c) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  for (int i = tid; i < kWarps * p.E; i += kThreads) s_p[i] = 0.f;
  for (int i = tid; i <= p.E; i += kThreads) s_c[i] = 0;
  __syncthreads();
  for (int t = blockIdx.x * kWarps + warp; t < p.T; t += gridDim.x * kWarps) {
    if (p.mask && p.mask[t] == 0) continue;
    const float *z = p.logits + (size_t)t * p.E;
    float m = -INFINITY, d = 0.f;
    bool nan = false;
    for (int e = lane; e < p.E; e += 32) m = fmaxf(m, z[e]), nan |= z[e] != z[e];
    m = warp_max(m);
    if (__any_sync(0xffffffffu, nan)) m = NAN;
    if (m != -INFINITY) {
      for (int e = lane; e < p.E; e += 32) d += expf(z[e] - m);
      d = warp_add(d);
      for (int e = lane; e < p.E; e += 32) s_p[warp * p.E + e] += expf(z[e] - m) / d;
    }
    if (lane < p.k) {
      const int e = p.ids[(size_t)t * p.k + lane];
      if (e >= 0 && e < p.E) atomicAdd(&s_c[e], 1);
    }
    if (lane == 0) atomicAdd(&s_c[p.E], 1);
  }
  __syncthreads();
}

__device__ void finish(const BalanceParams &p, int ctas) {
  __shared__ int32_t s_n;
  __shared__ double s_sum[kThreads];
  const int tid = threadIdx.x;
  for (int e = tid; e <= p.E; e += kThreads) {
    int c = 0;
    for (int g = 0; g < ctas; ++g) c += p.part_c[(size_t)g * (p.E + 1) + e];
    p.counts[e] = c;
    if (e == p.E) s_n = c;
  }
  __syncthreads();
  const double n = max(1, s_n);
  double sum = 0;
  for (int e = tid; e < p.E; e += kThreads) {
    double q = 0;
    for (int g = 0; g < ctas; ++g) q += p.part_p[(size_t)g * p.E + e];
    q /= n;
    if (p.mean_p) p.mean_p[e] = (float)q;
    sum += q * p.counts[e];
  }
  s_sum[tid] = sum;
  __syncthreads();
  if (tid == 0) {
    for (int i = 1; i < kThreads; ++i) sum += s_sum[i];
    p.loss[0] = (float)(sum * p.coef * p.E / (p.k * n));
    if (p.offsets) {
      int c = 0;
      for (int e = 0; e <= p.E; ++e) {
        p.offsets[e] = c;
        if (e < p.E) c += p.counts[e];
      }
    }
  }
}

// Few tokens: one CTA does it all, with the sums in shared memory.
__global__ void __launch_bounds__(kThreads) balance_one_kernel(BalanceParams p) {
  extern __shared__ float s_p[];
  int32_t *s_c = reinterpret_cast<int32_t *>(s_p + kWarps * p.E);
  count_tokens(p, s_p, s_c);
  for (int e = threadIdx.x; e < p.E; e += kThreads)
    for (int w = 1; w < kWarps; ++w) s_p[e] += s_p[w * p.E + e];
  __syncthreads();
  p.part_p = s_p;
  p.part_c = s_c;
  finish(p, 1);
}

__global__ void __launch_bounds__(kThreads) balance_part_kernel(const BalanceParams p) {
  extern __shared__ float s_p[];
  int32_t *s_c = reinterpret_cast<int32_t *>(s_p + kWarps * p.E);
  count_tokens(p, s_p, s_c);
  for (int e = threadIdx.x; e < p.E; e += kThreads) {
    float q = 0;
    for (int w = 0; w < kWarps; ++w) q += s_p[w * p.E + e];
    p.part_p[(size_t)blockIdx.x * p.E + e] = q;
  }
  for (int e = threadIdx.x; e <= p.E; e += kThreads) p.part_c[(size_t)blockIdx.x * (p.E + 1) + e] = s_c[e];
}

__global__ void __launch_bounds__(kThreads) balance_finish_kernel(const BalanceParams p, int ctas) { finish(p, ctas); }

__global__ void __launch_bounds__(kThreads) balance_grad_kernel(const float *logits, const int32_t *counts,
                                                                const uint8_t *mask, int T, int E, int k, float coef,
                                                                const float *dloss, float *dlogits) {
  extern __shared__ float s_f[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  long long total = 0;
  for (int e = 0; e < E; ++e) total += counts[e];
  const double n = max(1, counts[E]);
  for (int e = tid; e < E; e += kThreads) s_f[e] = (float)(((double)counts[e] - (double)total / E) / (k * n));
  __syncthreads();
  const float scale = (float)((dloss ? (double)dloss[0] : 1.0) * coef * E / n);
  for (int t = blockIdx.x * kWarps + warp; t < T; t += gridDim.x * kWarps) {
    const float *z = logits + (size_t)t * E;
    float *d = dlogits + (size_t)t * E;
    float m = -INFINITY, sum = 0.f, dot = 0.f;
    bool nan = false;
    const bool live = !mask || mask[t] != 0;
    if (live) {
      for (int e = lane; e < E; e += 32) m = fmaxf(m, z[e]), nan |= z[e] != z[e];
      m = warp_max(m);
      if (__any_sync(0xffffffffu, nan)) m = NAN;
    }
    if (m == -INFINITY) {
      for (int e = lane; e < E; e += 32) d[e] = 0.f;
      continue;
    }
    for (int e = lane; e < E; e += 32) {
      const float x = expf(z[e] - m);
      sum += x;
      dot += x * s_f[e];
    }
    sum = warp_add(sum);
    dot = warp_add(dot) / sum;
    for (int e = lane; e < E; e += 32) d[e] = scale * (expf(z[e] - m) / sum) * (s_f[e] - dot);
  }
}

int32_t check_sizes(int32_t T, int32_t E, int32_t k) {
  return T < 0 || k < 1 || k > 8 || E < k || E > kMaxE ? NSLM_ERR_SHAPE : NSLM_OK;
}

}  // namespace

size_t balance_ws_bytes(int32_t T, int32_t E) {
  if (T <= kOneLaunchT) return 0;
  return (size_t)kMaxCtas * (2 * (size_t)E + 1) * 4;
}

}  // namespace nslm

using namespace nslm;

extern "C" int32_t nslm_moe_balance(const float *logits, const int32_t *ids, const uint8_t *mask, int32_t T,
                                    int32_t E, int32_t k, float coef, int32_t *counts, int32_t *offsets,
                                    float *mean_p, float *loss, void *ws, size_t ws_bytes, nslm_stream_t stream) {
  g_launches = 0;
  if (!counts || !loss || (T > 0 && (!logits || !ids))) return NSLM_ERR_ARG;
  int32_t st = check_sizes(T, E, k);
  if (st) return st;
  if (!aligned16(logits) || !aligned16(ids) || !aligned16(mask) || !aligned16(counts) || !aligned16(offsets) ||
      !aligned16(mean_p) || !aligned16(loss))
    return NSLM_ERR_ALIGN;
  const size_t need = balance_ws_bytes(T, E);
  if (need && (!ws || ws_bytes < need)) return NSLM_ERR_WORKSPACE;
  if (need && !aligned16(ws)) return NSLM_ERR_ALIGN;
  if ((st = check_device())) return st;
  BalanceParams p{logits, ids, mask, T, E, k, coef, counts, offsets, mean_p, loss, nullptr, nullptr};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const size_t smem = ((size_t)kWarps * E + E + 1) * 4;
  if (T <= kOneLaunchT) {
    if ((st = ensure_smem((const void *)balance_one_kernel, smem))) return st;
    balance_one_kernel<<<1, kThreads, smem, s>>>(p);
    st = launch_status();
    if (st == NSLM_OK) g_launches = 1;
    return st;
  }
  p.part_p = reinterpret_cast<float *>(ws);
  p.part_c = reinterpret_cast<int32_t *>(p.part_p + (size_t)kMaxCtas * E);
  if ((st = ensure_smem((const void *)balance_part_kernel, smem))) return st;
  const int ctas = std::max(1, std::min((T + kWarps - 1) / kWarps, kMaxCtas));
  balance_part_kernel<<<ctas, kThreads, smem, s>>>(p);
  balance_finish_kernel<<<1, kThreads, 0, s>>>(p, ctas);
  st = launch_status();
  if (st == NSLM_OK) g_launches = 2;
  return st;
}

extern "C" int32_t nslm_moe_balance_grad(const float *logits, const int32_t *counts, const uint8_t *mask, int32_t T,
                                         int32_t E, int32_t k, float coef, const float *dloss, float *dlogits,
                                         nslm_stream_t stream) {
  g_launches = 0;
  if (!counts || (T > 0 && (!logits || !dlogits))) return NSLM_ERR_ARG;
  int32_t st = check_sizes(T, E, k);
  if (st) return st;
  if (!aligned16(logits) || !aligned16(counts) || !aligned16(mask) || !aligned16(dloss) || !aligned16(dlogits))
    return NSLM_ERR_ALIGN;
  if ((st = check_device())) return st;
  if (T == 0) return NSLM_OK;
  const int ctas = std::min((T + kWarps - 1) / kWarps, 8 * num_sms());
  balance_grad_kernel<<<ctas, kThreads, E * 4, reinterpret_cast<cudaStream_t>(stream)>>>(logits, counts, mask, T, E, k,
                                                                                        coef, dloss, dlogits);
  st = launch_status();
  if (st == NSLM_OK) g_launches = 1;
  return st;
}
