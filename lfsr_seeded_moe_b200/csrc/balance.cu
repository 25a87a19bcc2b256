// balance.cu -- nslm_moe_balance and nslm_moe_balance_grad: the experts' counts
// and the load-balance loss of a router, and the loss's gradient.
#include <algorithm>
#include <type_traits>

#include <cooperative_groups.h>

#include "common.cuh"

namespace nslm {
namespace {

namespace cg = cooperative_groups;

constexpr int kMaxE = 1024;
constexpr int kThreads = 512;
constexpr int kCluster = 8;
// Up to here one cluster does it all, and a caller needs no workspace.  One
// launch and two, measured at 1024 tokens: 100 experts 5.6 and 6.3 us, 256 7.4
// and 6.6, 512 11.2 and 7.8, 1024 15.3 and 10.8.
constexpr int kOneLaunchT = 1024;
constexpr int kPartThreads = 768;  // leaves the CTAs of the end their registers, so that they wait on their SMs
constexpr int kMaxCtas = 148;      // CTAs that leave parts in the workspace

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
  int32_t parts;
};

// 2 steps off at most; results below 2^-126 are 0.
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// LANES neighbouring lanes have a token, NV of its logits each: fours of
// neighbours where E is a multiple of 4 (VEC), else every LANES-th.  A token's
// softmax is then a few shuffles away, and a lane keeps its columns' sums in
// registers over all its tokens.
template <int LANES, int NV, bool VEC> struct Token {
  static constexpr int kNV = NV;
  static constexpr int kTokens = 32 / LANES;  // of a warp

  static __device__ __forceinline__ int lane() { return threadIdx.x & (LANES - 1); }
  static __device__ __forceinline__ int column(int j) {
    return VEC ? (lane() + LANES * (j / 4)) * 4 + j % 4 : lane() + LANES * j;
  }
  // -inf past the end
  static __device__ __forceinline__ void load(float (&z)[NV], const float *row, int E) {
    if constexpr (VEC) {
#pragma unroll
      for (int j = 0; j < NV; j += 4) {
        float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        if (column(j) < E) v = *reinterpret_cast<const float4 *>(row + column(j));
        z[j] = v.x, z[j + 1] = v.y, z[j + 2] = v.z, z[j + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < NV; ++j) z[j] = column(j) < E ? row[column(j)] : -INFINITY;
    }
  }
  static __device__ __forceinline__ void store(float *row, const float (&z)[NV], int E) {
    if constexpr (VEC) {
#pragma unroll
      for (int j = 0; j < NV; j += 4)
        if (column(j) < E) *reinterpret_cast<float4 *>(row + column(j)) = make_float4(z[j], z[j + 1], z[j + 2], z[j + 3]);
    } else {
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (column(j) < E) row[column(j)] = z[j];
    }
  }
  static __device__ __forceinline__ float sum(float v) {
#pragma unroll
    for (int o = 1; o < LANES; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  }
  // exp(z - max), in place; a token whose logits are all -inf has zeros, NaN stays NaN
  static __device__ __forceinline__ void exps(float (&z)[NV]) {
    float m = z[0];
#pragma unroll
    for (int j = 1; j < NV; ++j) m = fmaxf(m, z[j]);
#pragma unroll
    for (int o = 1; o < LANES; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float from = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int j = 0; j < NV; ++j) z[j] = exp2_fast((z[j] - from) * 1.44269504089f);
  }
};

// One pass over the logits with the running sums in registers.  65536 tokens of
// 128 experts take 13.4 us in two launches, 3 of them the second and its wait;
// the logits' 32 MB take 4.9 at the copy rate, and the exponentials, shuffles
// and the ids' shared-memory atomics are the rest.  64 tokens of 100 experts
// take 4.1 us, all latency.
//
// The CTA's tokens of a grid of `ctas`: the probabilities' sums to s_p[E], the
// counts and the number of tokens to s_c[E + 1].  s_w: a row of E for each warp.
//
// A lane adds kBlock probabilities in fp32, the warps join theirs (2 + 24 more
// additions), and blocks add up in fp64: equal probabilities are rounded the
// same way again and again, which in one fp32 sum of the thousands of tokens
// that a lane may have would be 1e-4 and more of it.  65536 tokens are one block.
// SUM: float where one block is all there is, else double.
constexpr int kBlock = 64;

template <class Tok, int THREADS, class SUM>
__device__ __forceinline__ void count_tokens(const BalanceParams &p, int cta, int ctas, float *s_w, SUM *s_p, int32_t *s_c) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int kWarps = THREADS / 32, kRows = Tok::kTokens * kWarps;
  float z[Tok::kNV];
  auto fetch = [&](int t) {
    const bool live = t < p.T && (!p.mask || p.mask[t] != 0);
#pragma unroll
    for (int j = 0; j < Tok::kNV; ++j) z[j] = -INFINITY;
    if (live && in_bounds((size_t)t * p.E + p.E - 1, (size_t)p.T * p.E, 30)) Tok::load(z, p.logits + (size_t)t * p.E, p.E);
  };
  // the first token's pairs and logits, on their way while the counts are cleared
  int ids[8];
  bool live = false;
  auto pairs = [&](int t) {
    live = t < p.T && (!p.mask || p.mask[t] != 0);
    if (live && !in_bounds((size_t)t * p.k + p.k - 1, (size_t)p.T * p.k, 31)) live = false;
    if (p.k % 4 == 0) {
#pragma unroll
      for (int q = 0; q < 8; q += 4) {
        int4 v = make_int4(-1, -1, -1, -1);
        if (live && q < p.k) v = *reinterpret_cast<const int4 *>(p.ids + (size_t)t * p.k + q);
        ids[q] = v.x, ids[q + 1] = v.y, ids[q + 2] = v.z, ids[q + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q) ids[q] = live && q < p.k ? p.ids[(size_t)t * p.k + q] : -1;
    }
  };
  pairs(cta * THREADS + tid);
  const int mine = tid / (32 / Tok::kTokens);
  fetch(cta * kRows + mine);
  for (int i = tid; i <= p.E; i += THREADS) s_c[i] = 0;
  __syncthreads();
  int n = 0;
  for (int t = cta * THREADS + tid; t < p.T;) {
    n += live;
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (ids[q] >= 0 && ids[q] < p.E) atomicAdd(&s_c[ids[q]], 1);
    t += ctas * THREADS;
    if (t < p.T) pairs(t);
  }
  n = __reduce_add_sync(0xffffffffu, n);
  if (lane == 0 && n) atomicAdd(&s_c[p.E], n);
  constexpr bool kOne = std::is_same<SUM, float>::value;
  static_assert(!kOne || kOneLaunchT <= kBlock * kWarps);
  for (int t0 = cta * kRows, block = 0;; ++block) {
    float acc[Tok::kNV] = {};
    for (int i = 0; (kOne || i < kBlock) && t0 < p.T; ++i) {
      Tok::exps(z);
      float d = 0.f;
#pragma unroll
      for (int j = 0; j < Tok::kNV; ++j) d += z[j];
      d = Tok::sum(d);
      const float r = d == 0.f ? 0.f : 1.f / d;  // nothing left in the row: nothing to add
#pragma unroll
      for (int j = 0; j < Tok::kNV; ++j) acc[j] = fmaf(z[j], r, acc[j]);
      t0 += ctas * kRows;
      if (t0 < p.T) fetch(t0 + mine);
    }
    // over the warp's tokens: each halving leaves a lane half of the columns
    int keep = Tok::kNV, from = 0;
#pragma unroll
    for (int o = 16; o >= 32 / Tok::kTokens; o >>= 1) {
      keep /= 2;
      const bool up = lane & o;
#pragma unroll
      for (int j = 0; j < Tok::kNV / 2; ++j) {
        if (j >= keep) break;
        const float other = __shfl_xor_sync(0xffffffffu, up ? acc[j] : acc[j + keep], o);
        acc[j] = (up ? acc[j + keep] : acc[j]) + other;
      }
      from += up ? keep : 0;
    }
#pragma unroll
    for (int j = 0; j < Tok::kNV / Tok::kTokens; ++j)
      if (Tok::column(from + j) < p.E && in_bounds(warp * p.E + Tok::column(from + j), (size_t)kWarps * p.E, 32))
        s_w[warp * p.E + Tok::column(from + j)] = acc[j];
    __syncthreads();
    for (int e = tid; e < p.E; e += THREADS) {
      float q = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) q += s_w[w * p.E + e];
      s_p[e] = kOne || block == 0 ? q : s_p[e] + q;
    }
    if (kOne || t0 >= p.T) break;
    __syncthreads();  // s_w is written again
  }
}

__device__ __forceinline__ void sync_cluster(int ctas) {
  if (ctas == 1) __syncthreads();
  else cg::this_cluster().sync();
}

struct Finish {
  double sum[kThreads];
  int32_t count[kThreads];
  double total[kMaxE + 1];
  int32_t slice[kMaxE + 1];
  double loss[kCluster];
  int32_t base[kCluster];
};

// The end, by a cluster whose CTAs have a slice of the experts each: part(g, e)
// and tokens(g, e) give the sums and counts of g's tokens, e = E their number.
// All CTAs of the cluster have to run by then: it stores into their shared memory.
template <class P, class C> __device__ void finish(const BalanceParams &p, Finish &s, int parts, P part, C tokens) {
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, rank = (int)cluster.block_rank(), ctas = (int)cluster.num_blocks();
  const int e0 = p.E * rank / ctas, len = p.E * (rank + 1) / ctas - e0;
  // a column for each expert of the slice, and one for the number of tokens
  const int cols = len + 1, sets = min(kThreads / cols, parts), set = tid / cols, c = tid - set * cols;
  const int e = c < len ? e0 + c : p.E;
  double q = 0;
  int n = 0;
  if (set < sets) {
    // eight parts' loads in flight
    for (int g = set; g < parts; g += 8 * sets) {
      float x[8];
      int y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const bool there = g + i * sets < parts;
        x[i] = there && c < len ? part(g + i * sets, e) : 0.f;
        y[i] = there ? tokens(g + i * sets, e) : 0;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) q += x[i], n += y[i];
    }
    s.sum[tid] = q;
    s.count[tid] = n;
  }
  __syncthreads();
  if (set == 0) {
#pragma unroll 8
    for (int i = 1; i < sets; ++i) q += s.sum[i * cols + c], n += s.count[i * cols + c];
    s.slice[c] = n;
    s.total[c] = q;
  }
  __syncthreads();
  const int live = s.slice[len];
  const double share = 1. / max(1, live);
  if (set == 0 && c < len && in_bounds(e, p.E, 33)) {
    p.counts[e] = n;
    if (p.mean_p) p.mean_p[e] = (float)(q * share);
  }
  if (tid < 32) {  // the slice's part of the loss, and its number of pairs
    double x = 0;
    int b = 0;
    for (int i = tid; i < len; i += 32) x += s.total[i] * s.slice[i], b += s.slice[i];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    b = __reduce_add_sync(0xffffffffu, b);
    if (tid < ctas) {
      cluster.map_shared_rank(s.loss, tid)[rank] = x;
      cluster.map_shared_rank(s.base, tid)[rank] = b;
    }
  }
  const double scale = share * share * p.coef * p.E / p.k;
  sync_cluster(ctas);  // and no CTA leaves before the others have read its parts
  if (rank == 0 && tid == 32) {
    p.counts[p.E] = live;
    double x = 0;
    for (int i = 0; i < ctas; ++i) x += s.loss[i];
    p.loss[0] = (float)(x * scale);
  }
  if (p.offsets && tid < 32) {
    int b = 0;
    for (int i = 0; i < rank; ++i) b += s.base[i];
    for (int i0 = 0; i0 < len; i0 += 32) {
      const int own = i0 + tid < len ? s.slice[i0 + tid] : 0;
      int upto = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, upto, o);
        if (tid >= o) upto += y;
      }
      if (i0 + tid < len && in_bounds(e0 + i0 + tid, p.E, 33)) p.offsets[e0 + i0 + tid] = b + upto - own;
      b += __shfl_sync(0xffffffffu, upto, 31);
    }
    if (rank == ctas - 1 && tid == 0) p.offsets[p.E] = b;
  }
}

// Shared memory: a row of E sums for each warp, then [E] (of SUM, which an even
// number of warps aligns) and [E + 1] of the CTA.
template <class SUM> size_t balance_smem(int E, int threads) {
  return (size_t)threads / 32 * E * 4 + E * sizeof(SUM) + ((size_t)E + 1) * 4;
}
static_assert(kThreads / 32 % 2 == 0 && kPartThreads / 32 % 2 == 0);

// Few tokens: one cluster does it all.
template <class Tok> __global__ void __launch_bounds__(kThreads) balance_one_kernel(const BalanceParams p) {
  extern __shared__ double smem[];
  Finish &s = *reinterpret_cast<Finish *>(smem);
  float *s_w = reinterpret_cast<float *>(&s + 1);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  cg::cluster_group cluster = cg::this_cluster();
  float *s_p = s_w + kThreads / 32 * p.E;
  int32_t *s_c = reinterpret_cast<int32_t *>(s_p + p.E);
  const int ctas = (int)cluster.num_blocks();
  count_tokens<Tok, kThreads, float>(p, (int)cluster.block_rank(), ctas, s_w, s_p, s_c);
  sync_cluster(ctas);
  finish(
      p, s, ctas, [&](int g, int e) { return cluster.map_shared_rank(s_p, g)[e]; },
      [&](int g, int e) { return cluster.map_shared_rank(s_c, g)[e]; });
}

template <class Tok> __global__ void __launch_bounds__(kPartThreads) balance_part_kernel(const BalanceParams p) {
  extern __shared__ double smem[];
  float *s_w = reinterpret_cast<float *>(smem);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  double *s_p = reinterpret_cast<double *>(s_w + kPartThreads / 32 * p.E);
  int32_t *s_c = reinterpret_cast<int32_t *>(s_p + p.E);
  count_tokens<Tok, kPartThreads, double>(p, blockIdx.x, gridDim.x, s_w, s_p, s_c);
  __syncthreads();
  if (!in_bounds(blockIdx.x, kMaxCtas, 33)) return;
  for (int e = threadIdx.x; e < p.E; e += kPartThreads) p.part_p[(size_t)blockIdx.x * p.E + e] = (float)s_p[e];
  for (int e = threadIdx.x; e <= p.E; e += kPartThreads) p.part_c[(size_t)blockIdx.x * (p.E + 1) + e] = s_c[e];
}

__global__ void __launch_bounds__(kThreads) balance_finish_kernel(const BalanceParams p) {
  extern __shared__ double smem[];
  Finish &s = *reinterpret_cast<Finish *>(smem);
  cluster_arrive();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  cluster_wait();  // finish() stores into the others
  finish(
      p, s, p.parts, [&](int g, int e) { return p.part_p[(size_t)g * p.E + e]; },
      [&](int g, int e) { return p.part_c[(size_t)g * (p.E + 1) + e]; });
}

// The gradient: a pass that reads and writes each logit once, with the next
// token's on their way: 65536 x 128 takes 12.8 us, 76% of the copy rate.
// f is f_e less its mean: a softmax's gradient does not see a constant, and a
// difference of two nearly equal sums would lose what f's differences hold.
// dlogits may be logits: a token's lanes have read it before they write it.
constexpr int kGradThreads = 128;

template <class Tok>
__global__ void __launch_bounds__(kGradThreads)
    balance_grad_kernel(const float *logits, const int32_t *counts, const uint8_t *mask, int T, int E, int k, float coef,
                        const float *dloss, float *dlogits) {
  __shared__ uint32_t s_total[2][kGradThreads / 32];
  const int tid = threadIdx.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr int kRows = Tok::kTokens * (kGradThreads / 32);
  float z[Tok::kNV], ahead[Tok::kNV];  // a token's logits, and the next one's on their way
  auto fetch = [&](int t) {
    const bool live = t < T && (!mask || mask[t] != 0);
#pragma unroll
    for (int j = 0; j < Tok::kNV; ++j) ahead[j] = -INFINITY;
    if (live && in_bounds((size_t)t * E + E - 1, (size_t)T * E, 30)) Tok::load(ahead, logits + (size_t)t * E, E);
  };
  int t = blockIdx.x * kRows + tid / (32 / Tok::kTokens);
  fetch(t);
  // counts summed over ranks fit 32 bits, their total need not: halves of 16 bits, a total of each
  uint32_t low = 0, high = 0;
  for (int e = tid; e < E; e += kGradThreads) low += counts[e] & 0xffff, high += counts[e] >> 16;
  low = __reduce_add_sync(0xffffffffu, low), high = __reduce_add_sync(0xffffffffu, high);
  if ((tid & 31) == 0) s_total[0][tid >> 5] = low, s_total[1][tid >> 5] = high;
  const double n = max(1, counts[E]);
  const float scale = (float)((dloss ? (double)dloss[0] : 1.0) * coef * E / n);
  __syncthreads();
  low = high = 0;
#pragma unroll
  for (int w = 0; w < kGradThreads / 32; ++w) low += s_total[0][w], high += s_total[1][w];
  const double mean = (high * 65536. + low) / E, share = 1. / (k * n);
  float f[Tok::kNV];
#pragma unroll
  for (int j = 0; j < Tok::kNV; ++j) f[j] = Tok::column(j) < E ? (float)((counts[Tok::column(j)] - mean) * share) : 0.f;
  for (; t - tid / (32 / Tok::kTokens) < T; t += gridDim.x * kRows) {
#pragma unroll
    for (int j = 0; j < Tok::kNV; ++j) z[j] = ahead[j];
    fetch(t + gridDim.x * kRows);
    Tok::exps(z);
    float d = 0.f, dot = 0.f;
#pragma unroll
    for (int j = 0; j < Tok::kNV; ++j) d += z[j], dot = fmaf(z[j], f[j], dot);
    d = Tok::sum(d);
    dot = Tok::sum(dot);
    const float r = d == 0.f ? 0.f : 1.f / d;
    dot *= r;
    const float by = d == 0.f ? 0.f : scale * r;
#pragma unroll
    for (int j = 0; j < Tok::kNV; ++j) z[j] = by * z[j] * (f[j] - dot);
    if (t < T && in_bounds((size_t)t * E + E - 1, (size_t)T * E, 34)) Tok::store(dlogits + (size_t)t * E, z, E);
  }
}

// The kernels for E: lanes of a token, logits of a lane.
template <class F> int32_t with_token(int E, F f) {
  auto pick = [&](auto vec) {
    constexpr bool V = decltype(vec)::value;
    if (E <= 32) return f(Token<8, 4, V>{});
    if (E <= 64) return f(Token<8, 8, V>{});
    if (E <= 128) return f(Token<8, 16, V>{});
    if (E <= 256) return f(Token<16, 16, V>{});
    if (E <= 512) return f(Token<32, 16, V>{});
    return f(Token<32, 32, V>{});
  };
  return E % 4 == 0 ? pick(std::true_type{}) : pick(std::false_type{});
}

template <class K, class... Args>
int32_t launch(K k, int ctas, int cluster, int threads, size_t smem, cudaStream_t s, Args... args) {
  if (int32_t st = ensure_smem((const void *)k, smem)) return st;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  if (int32_t st = cuda_status(cudaLaunchKernelEx(&cfg, k, args...))) return st;
  return launch_status();
}

int32_t check_sizes(int32_t T, int32_t E, int32_t k) {
  if (T < 0 || T > (1 << 28) || k < 1 || k > 8 || E < k || E > kMaxE) return NSLM_ERR_SHAPE;
  return (int64_t)T * k > INT32_MAX ? NSLM_ERR_SHAPE : NSLM_OK;  // the counts are int32
}

}  // namespace

NSLM_BOUNDS_ACCESSOR(balance)

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
  BalanceParams p{logits, ids, mask, T, E, k, coef, counts, offsets, mean_p, loss, nullptr, nullptr, 0};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (T <= kOneLaunchT) {
    // a cluster's barriers cost about what 64 tokens do; and in the end a CTA has
    // a thread for each column of its slice and one more
    int ctas = 1;
    while (ctas < kCluster && (T > 64 * ctas || ceil_div(E, ctas) + 1 > kThreads)) ctas *= 2;
    st = with_token(E, [&](auto tok) {
      return launch(balance_one_kernel<decltype(tok)>, ctas, ctas, kThreads, sizeof(Finish) + balance_smem<float>(E, kThreads), s, p);
    });
    if (st == NSLM_OK) g_launches = 1;
    return st;
  }
  p.part_p = reinterpret_cast<float *>(ws);
  p.part_c = reinterpret_cast<int32_t *>(p.part_p + (size_t)kMaxCtas * E);
  st = with_token(E, [&](auto tok) {
    using Tok = decltype(tok);
    p.parts = std::min({ceil_div(T, Tok::kTokens * kPartThreads / 32), num_sms(), kMaxCtas});
    return launch(balance_part_kernel<Tok>, p.parts, 1, kPartThreads, balance_smem<double>(E, kPartThreads), s, p);
  });
  if (st == NSLM_OK) st = launch(balance_finish_kernel, kCluster, kCluster, kThreads, sizeof(Finish), s, p);
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
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  st = with_token(E, [&](auto tok) {
    using Tok = decltype(tok);
    auto k_grad = balance_grad_kernel<Tok>;
    // one wave, and CTAs with equal numbers of rounds
    const int rounds = ceil_div(T, Tok::kTokens * (kGradThreads / 32));
    const int most = max_active_ctas((const void *)k_grad, kGradThreads, 0) * num_sms();
    const int ctas = ceil_div(rounds, ceil_div(rounds, most));
    return launch(k_grad, ctas, 1, kGradThreads, 0, s, logits, counts, mask, T, E, k, coef, dloss, dlogits);
  });
  if (st == NSLM_OK) g_launches = 1;
  return st;
}
