// sample.cu -- nslm_sample: one token a row from logits, with temperature,
// top-k, top-p and min-p, at given random numbers.
#include <cuda_bf16.h>

#include "common.cuh"

namespace nslm {
namespace {

constexpr int kMaxV = 1 << 18;
constexpr int kThreads = 1024;
constexpr double kOne = 17592186044416.0;  // 2^44: w as 64-bit fixed point; 2^18 of them stay below 2^62

struct SampleParams {
  const void *logits;
  int64_t ld;
  int32_t V;
  const float *temperature, *top_p, *min_p;
  const int32_t *top_k;
  const float *u;
  int32_t *token;
  float *prob;
};

// fp32 in the order of its values as an unsigned integer (-0 counts as 0).
__device__ __forceinline__ uint32_t key_of(float v) {
  const uint32_t b = __float_as_uint(v + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// f summed over the tokens [0, V) of the row, in every thread.
template <class F>
__device__ uint64_t row_sum(int V, F f) {
  __shared__ uint64_t s_part[kThreads / 32];
  uint64_t v = 0;
  for (int i = threadIdx.x; i < V; i += kThreads) v += f(i);
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s_part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0;
  for (int w = 0; w < kThreads / 32; ++w) v += s_part[w];
  return v;
}

// The smallest x in [0, 2^bits) whose running sum over the tokens up to x is at least need.
template <class F>
__device__ int first_index(int V, uint64_t need, F f) {
  int x = 0;
  for (int bit = 1 << 17; bit > 0; bit >>= 1) {
    const int y = x + bit;
    if (row_sum(min(V, y), f) < need) x = y;
  }
  return min(x, V - 1);
}

template <class T>
__global__ void __launch_bounds__(kThreads) sample_kernel(const SampleParams p) {
  const int row = blockIdx.x, V = p.V;
  const T *l = reinterpret_cast<const T *>(p.logits) + (size_t)row * p.ld;
  __shared__ float s_max[kThreads / 32];
  float m = -INFINITY;
  for (int i = threadIdx.x; i < V; i += kThreads) m = fmaxf(m, (float)l[i]);
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = m;
  __syncthreads();
  for (int w = 0; w < kThreads / 32; ++w) m = fmaxf(m, s_max[w]);
  if (m == -INFINITY) {
    if (threadIdx.x == 0) {
      p.token[row] = -1;
      if (p.prob) p.prob[row] = 0.f;
    }
    return;
  }
  const float temp = p.temperature ? p.temperature[row] : 1.f;
  const bool greedy = !(temp > 0.f);
  auto w_of = [&](float v) -> double {
    if (!(v <= m)) return 0.;
    if (greedy || m == INFINITY) return v == m ? 1. : 0.;
    return exp(((double)v - (double)m) / (double)temp);
  };
  auto fixed = [&](float v) -> uint64_t { return (uint64_t)__double2ll_rn(w_of(v) * kOne); };

  // the last token that stays, in (logit descending, index ascending) order
  uint32_t last_key = 0;
  int last_idx = V;
  auto kept = [&](int i) {
    const uint32_t k = key_of((float)l[i]);
    return fixed((float)l[i]) > 0 && (k > last_key || (k == last_key && i <= last_idx));
  };
  auto cut = [&](uint64_t need, auto value) {
    uint32_t key = 0;
    for (uint32_t bit = 0x80000000u; bit > 0; bit >>= 1) {
      const uint32_t k = key | bit;
      if (row_sum(V, [&](int i) { return kept(i) && key_of((float)l[i]) >= k ? value(i) : 0; }) >= need) key = k;
    }
    const uint64_t above = row_sum(V, [&](int i) { return kept(i) && key_of((float)l[i]) > key ? value(i) : 0; });
    const int idx = first_index(V, need - above, [&](int i) { return kept(i) && key_of((float)l[i]) == key ? value(i) : 0; });
    last_key = key;
    last_idx = idx;
  };
  auto one = [&](int) -> uint64_t { return 1; };
  auto mass = [&](int i) -> uint64_t { return fixed((float)l[i]); };
  if (greedy) {
    cut(1, one);
  } else {
    const int top_k = p.top_k ? p.top_k[row] : 0;
    if (top_k > 0 && (uint64_t)top_k < row_sum(V, [&](int i) { return kept(i) ? 1 : 0; })) cut(top_k, one);
    const float top_p = p.top_p ? p.top_p[row] : 1.f;
    if (top_p < 1.f) {
      const uint64_t all = row_sum(V, [&](int i) { return kept(i) ? mass(i) : 0; });
      cut(max(1ll, __double2ll_ru((double)top_p * (double)all)), mass);
    }
  }
  const float q = p.min_p ? p.min_p[row] : 0.f;
  const double min_p = q > 0.f ? fmin((double)q, 1.) : 0.;
  auto final_mass = [&](int i) -> uint64_t { return kept(i) && !(w_of((float)l[i]) < min_p) ? mass(i) : 0; };
  const uint64_t Z = row_sum(V, final_mass);
  const float u = p.u[row];
  uint64_t t = u > 0.f ? (uint64_t)((double)u * (double)Z) : 0;
  if (!(u < 1.f) && u == u) t = Z;
  const int i = first_index(V, min(t, Z - 1) + 1, final_mass);
  if (threadIdx.x == 0) {
    p.token[row] = i;
    if (p.prob) p.prob[row] = (float)(w_of((float)l[i]) * kOne / (double)Z);
  }
}

}  // namespace
}  // namespace nslm

using namespace nslm;

extern "C" int32_t nslm_sample(const void *logits, int32_t type, int32_t B, int32_t V, int64_t ld,
                               const nslm_sample_params *params, const float *u, int32_t *token, float *prob,
                               nslm_stream_t stream) {
  g_launches = 0;
  if (type != NSLM_TYPE_F32 && type != NSLM_TYPE_BF16) return NSLM_ERR_ARG;
  if (B < 0 || V < 1 || V > kMaxV || ld < V) return NSLM_ERR_SHAPE;
  if (B > 0 && (!logits || !u || !token)) return NSLM_ERR_ARG;
  if (!aligned16(logits) || !aligned16(u) || !aligned16(token) || !aligned16(prob)) return NSLM_ERR_ALIGN;
  SampleParams p{logits, ld, V, nullptr, nullptr, nullptr, nullptr, u, token, prob};
  if (params) {
    p.temperature = params->temperature;
    p.top_k = params->top_k;
    p.top_p = params->top_p;
    p.min_p = params->min_p;
    if (!aligned16(p.temperature) || !aligned16(p.top_k) || !aligned16(p.top_p) || !aligned16(p.min_p))
      return NSLM_ERR_ALIGN;
  }
  int32_t st = check_device();
  if (st) return st;
  if (B == 0) return NSLM_OK;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (type == NSLM_TYPE_BF16) sample_kernel<__nv_bfloat16><<<B, kThreads, 0, s>>>(p);
  else sample_kernel<float><<<B, kThreads, 0, s>>>(p);
  st = launch_status();
  if (st == NSLM_OK) g_launches = 1;
  return st;
}
