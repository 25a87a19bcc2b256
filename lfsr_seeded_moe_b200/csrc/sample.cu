// sample.cu -- nslm_sample: one token a row from logits, with temperature,
// top-k, top-p and min-p, at given random numbers.
#include <algorithm>
#include <cfloat>

#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include "common.cuh"

namespace nslm {
namespace {

namespace cg = cooperative_groups;

constexpr int kMaxV = 1 << 18;
constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kBins = 512;
constexpr int kList = 256;
constexpr int kLevels = 6;  // and all as the last

struct SampleParams {
  const void *logits;
  int64_t ld;
  int32_t V;
  int32_t len;  // logits of a CTA, a multiple of 8
  const float *temperature, *top_p, *min_p;
  const int32_t *top_k;
  const float *u;
  int32_t *token;
  float *prob;
};

// A cluster of up to 8 CTAs has one row, each CTA a part of it, which it reads
// once and keeps in shared memory as fp32.  w is 64-bit fixed point with 44 bits
// behind the point, at most 2^18 of them, so sums stay below 2^62 and are
// exact: whatever order threads and CTAs add in, the same u gives the same
// token.

// Weights in units of 2^-44.  exp(x) = 2^(k/16) e^r, |r| <= ln 2 / 32, with the
// 16 powers from a table and e^r by its series to r^5 (the table method of
// P. T. P. Tang, "Table-driven implementation of the exponential function in
// IEEE floating-point arithmetic", ACM TOMS 15, 1989): off by at most
// r^6 / 720 = 2^-43 of itself.  A 16-entry table lies in 32 banks, so lanes
// never wait for one another.
struct Weight {
  float m;       // the row's largest logit
  float low;     // 40 temperatures below, where weights have long been 0: what is lower is not looked at
  double step;   // 16 / (temperature ln 2)
  const double *pow16;  // shared: 2^(44 + j/16)

  __device__ __forceinline__ double operator()(float v) const {
    const double t = ((double)v - (double)m) * step;
    const double kd = t + 0x1.8p52;  // t to the nearest integer, in the low bits
    const int k = __double2loint(kd);
    const double r = t - (kd - 0x1.8p52);
    // (ln 2 / 16)^i / i!
    double e = 0x1.5d87fe78a6731p-30;
    e = fma(e, r, 0x1.3b2ab6fba4e77p-23);
    e = fma(e, r, 0x1.c6b08d704a0c0p-17);
    e = fma(e, r, 0x1.ebfbdff82c58fp-11);
    e = fma(e, r, 0x1.62e42fefa39efp-5);
    e = fma(e, r, 1.);
    const double w = e * pow16[k & 15];
    return v >= low ? __hiloint2double(__double2hiint(w) + ((k >> 4) << 20), __double2loint(w)) : 0.;
  }
  __device__ __forceinline__ uint64_t fixed(float v) const { return to_fixed((*this)(v)); }
  // to the nearest integer: below 2^51 it stands in the low bits of w + 2^52
  static __device__ __forceinline__ uint64_t to_fixed(double w) {
    return (uint64_t)__double_as_longlong(w + 0x1p52) & 0xfffffffffffffull;
  }
};

struct Candidate {
  uint64_t w;
  float v;
  int32_t i;
};

struct Shared {
  double pow16[16];
  // what every warp of the row tells every CTA, by turns
  uint64_t slot[2][kLevels + 1][kMaxCluster * kWarps];
  uint64_t warp_mass[kWarps];
  uint32_t warp_count[kWarps];
  int32_t list_n;
  int32_t found;
  uint64_t found_mass;
  uint32_t found_count, found_in;
  union {
    struct {
      uint32_t count[kBins], lo[kBins], hi[kBins];
    } hist;
    Candidate list[kList];
  };
};

template <class T> __device__ __forceinline__ T warp_sum_of(T v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
template <class T> __device__ __forceinline__ T warp_scan_of(T v, int lane) {  // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  return v;
}

// The tokens between two logits, in the order of their logits.
struct Range {
  float lo, top;   // lo <= v < top
  float hi;        // the largest v there, or a bound
  int bin = -1;    // of those, the ones in this bin of [lo, hi], or all
  uint64_t above_mass = 0;
  uint32_t above_count = 0;

  // Falls from 0 at hi to kBins - 1 at lo, for any lo < hi.
  __device__ __forceinline__ int bin_of(float v) const {
    const float h = hi - lo < INFINITY ? 1.f : 0.5f;
    return min(kBins - 1, (int)((hi * h - v * h) / (hi * h - lo * h) * kBins));
  }
  __device__ __forceinline__ bool has(float v) const { return v >= lo && v < top && (bin < 0 || bin_of(v) == bin); }
};

// Counts, and masses, of the tokens with logits from m down to some levels below, and of all.
struct Levels {
  uint64_t mass[kLevels + 1];
  uint32_t count[kLevels + 1];
};

struct Row {
  Shared &s;
  const float *l;  // shared: this CTA's logits
  int n;           // how many
  int first;       // the index of the first
  int rank, ctas;  // in the cluster
  int warp, lane;
  int parity = 0;
  float temp = 1.f, lowest = 0.f;
  Weight w{};
  // the last token that stays, in the order of descending logits and ascending indexes
  float last_v = -INFINITY;
  int last_i = kMaxV;

  __device__ __forceinline__ bool kept(int i, float v) const {
    return v > last_v || (v == last_v && first + i <= last_i);
  }

  // A warp's share of the CTA's logits: contiguous, so that sums over warps are sums over indexes.
  __device__ __forceinline__ int share() const { return ((n + kWarps - 1) / kWarps + 31) & ~31; }

  // f(i, logit) for this thread's logits, four at a time so that their
  // latencies overlap; i of a place past the end is meaningless, its logit -inf.
  template <class F> __device__ __forceinline__ void each(F f) const {
    for (int i = threadIdx.x; i < n; i += 4 * kThreads) {
      float v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = i + j * kThreads < n ? l[i + j * kThreads] : -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) f(i + j * kThreads, v[j]);
    }
  }

  __device__ void sync_row() {
    if (ctas == 1) __syncthreads();
    else cg::this_cluster().sync();
  }

  // Every warp's values (the same in all its lanes) to every CTA.  Two sets of
  // slots by turns: who writes one again has passed the barrier after which
  // the others had read it.
  using Slots = const uint64_t (*)[kMaxCluster * kWarps];
  template <int V> __device__ __forceinline__ Slots publish(const uint64_t (&v)[V]) {
    auto slot = s.slot[parity];
    parity ^= 1;
    if (lane < ctas) {
      uint64_t *to = ctas == 1 ? &slot[0][0] : cg::this_cluster().map_shared_rank(&slot[0][0], lane);
#pragma unroll
      for (int j = 0; j < V; ++j) to[j * kMaxCluster * kWarps + rank * kWarps + warp] = v[j];
    }
    sync_row();
    return slot;
  }

  // Smallest and largest over the row.
  __device__ void extremes(float &lo, float &hi) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
      hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    const uint64_t v[1] = {(uint64_t)__float_as_uint(hi) << 32 | __float_as_uint(lo)};
    const auto slot = publish(v);
    for (int k = lane; k < ctas * kWarps; k += 32) {
      lo = fminf(lo, __uint_as_float((uint32_t)slot[0][k]));
      hi = fmaxf(hi, __uint_as_float((uint32_t)(slot[0][k] >> 32)));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
      hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
  }

  // The lowest index for which the sum of f up to it exceeds target(the whole
  // sum all), as the position in the CTA that has it, valid in one warp of
  // that CTA; -1 everywhere else.
  template <class F, class G> __device__ int find(F f, G target, uint64_t &all) {
    const int per = share();
    auto sum = [&](int lo, int hi) {
      uint64_t a = 0;
      for (int i = lo + lane; i < hi; i += 128) {
#pragma unroll
        for (int j = 0; j < 4; ++j) a += f(i + 32 * j, i + 32 * j < hi ? l[i + 32 * j] : -INFINITY);
      }
      return warp_sum_of(a);
    };
    const uint64_t v[1] = {sum(warp * per, min(n, (warp + 1) * per))};
    const auto slot = publish(v);
    // the warp of the row that has it
    uint64_t x[kMaxCluster * kWarps / 32];
    all = 0;
#pragma unroll
    for (int j = 0; j < kMaxCluster * kWarps / 32; ++j) {
      x[j] = 32 * j + lane < ctas * kWarps ? slot[0][32 * j + lane] : 0;
      all += x[j];
    }
    all = warp_sum_of(all);
    uint64_t left = target(all);
    int at = -1;
#pragma unroll
    for (int j = 0; j < kMaxCluster * kWarps / 32; ++j) {
      const uint64_t upto = warp_scan_of(x[j], lane);
      const uint32_t over = __ballot_sync(0xffffffffu, upto > left);
      if (at >= 0) continue;
      if (over) {
        const int k = __ffs(over) - 1;
        at = 32 * j + k;
        left -= __shfl_sync(0xffffffffu, upto - x[j], k);
      } else {
        left -= __shfl_sync(0xffffffffu, upto, 31);
      }
    }
    if (at < 0 || at / kWarps != rank) return -1;
    at %= kWarps;
    int lo = at * per, hi = min(n, lo + per);
    if (per > 256) {  // all warps on that warp's logits
      const int sub = (per / kWarps + 31) & ~31;
      const uint64_t c = sum(lo + warp * sub, min(hi, lo + (warp + 1) * sub));
      if (lane == 0) s.warp_mass[warp] = c;
      __syncthreads();
      at = 0;
      while (at < kWarps - 1 && left >= s.warp_mass[at]) left -= s.warp_mass[at++];
      lo += at * sub;
      hi = min(hi, lo + sub);
    }
    if (warp != at) return -1;
    for (int i = lo; i < hi; i += 32) {
      const uint64_t upto = warp_scan_of(f(i + lane, i + lane < hi ? l[i + lane] : -INFINITY), lane);
      const uint32_t over = __ballot_sync(0xffffffffu, upto > left);
      if (over) return i + __ffs(over) - 1;
      left -= __shfl_sync(0xffffffffu, upto, 31);
    }
    return -1;
  }

  // The levels, in temperatures below m.
  __device__ __forceinline__ float level(int j) const {
    constexpr float below[kLevels] = {2.f, 4.f, 6.f, 8.f, 11.f, 15.f};
    float c = below[0];
#pragma unroll
    for (int i = 1; i < kLevels; ++i) c = j == i ? below[i] : c;
    return __fmaf_rn(-temp, c, w.m);
  }
  template <bool MASS> __device__ Levels levels() {
    float at[kLevels];
#pragma unroll
    for (int j = 0; j < kLevels; ++j) at[j] = level(j);
    // a thread has at most 64 logits: its counts stand in bytes, or above bit 51 of its mass, which needs 51
    uint64_t sum[kLevels + 1] = {};
    uint32_t bytes[2] = {};
    each([&](int i, float v) {
      if (!(v > -INFINITY && kept(i, v))) return;
      if (MASS) {
        const uint64_t x = w.fixed(v) | 1ull << 52;
        sum[kLevels] += x;
#pragma unroll
        for (int j = 0; j < kLevels; ++j)
          if (v >= at[j]) sum[j] += x;
      } else {
        bytes[kLevels / 4] += 1u << (8 * (kLevels % 4));
#pragma unroll
        for (int j = 0; j < kLevels; ++j)
          if (v >= at[j]) bytes[j / 4] += 1u << (8 * (j % 4));
      }
    });
    Levels t{};
    auto add = [&](Slots slot, auto put) {
#pragma unroll
      for (int j = 0; j <= kLevels; ++j) {
        uint64_t a = 0;
        for (int k = lane; k < ctas * kWarps; k += 32) a += slot[j][k];
        put(j, warp_sum_of(a));
      }
    };
    if (MASS) {
      uint64_t v[kLevels + 1];
#pragma unroll
      for (int j = 0; j <= kLevels; ++j) {
        v[j] = warp_sum_of(sum[j] & 0xfffffffffffffull);
        sum[j] = warp_sum_of((uint32_t)(sum[j] >> 52));
      }
      add(publish(v), [&](int j, uint64_t a) { t.mass[j] = a; });
    } else {
#pragma unroll
      for (int j = 0; j <= kLevels; ++j) sum[j] = warp_sum_of(bytes[j / 4] >> (8 * (j % 4)) & 255u);
    }
    add(publish(sum), [&](int j, uint64_t a) { t.count[j] = (uint32_t)a; });
    return t;
  }
  // The tokens of level j that are not of the one before.
  __device__ Range range_of(int j, const Levels &t) const {
    Range r;
    r.lo = j < kLevels ? fmaxf(level(j), lowest) : lowest;
    r.top = j > 0 ? level(j - 1) : INFINITY;
    r.hi = fminf(r.top, w.m);
    r.above_mass = j > 0 ? t.mass[j - 1] : 0;
    r.above_count = j > 0 ? t.count[j - 1] : 0;
    return r;
  }

  // The kept tokens of a range, at most kList, in CTA 0's list.
  __device__ void gather(const Range &r) {
    if (threadIdx.x == 0) s.list_n = 0;
    sync_row();
    Shared *o = ctas == 1 ? &s : cg::this_cluster().map_shared_rank(&s, 0);
    each([&](int i, float v) {
      if (r.has(v) && kept(i, v)) o->list[atomicAdd(&o->list_n, 1)] = Candidate{w.fixed(v), v, first + i};
    });
    sync_row();
  }
  // The sum of f over the list, in each of `per` threads.
  template <class F> __device__ __forceinline__ uint64_t over_list(int n, int per, F f) {
    uint64_t a = 0;
#pragma unroll 4
    for (int j = threadIdx.x & (per - 1); j < n; j += per) a += f(s.list[j]);
    for (int o = 1; o < per; o <<= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
    return a;
  }
  // threads for each of n candidates
  __device__ __forceinline__ static int threads_each(int n) { return n <= 64 ? 8 : n <= 128 ? 4 : 2; }

  // Sets the last token that stays to the one at which the kept tokens' count
  // (by_mass: their mass), in their order, first reaches `need`, which is in
  // the range of `in` tokens.
  __device__ void cut(uint64_t need, bool by_mass, Range r, uint32_t in) {
    auto inside = [&](int i, float v) { return r.has(v) && kept(i, v); };
    while (in > kList && r.lo < r.hi) {
      // a histogram of the range; the bin that has the token is the next range
      __syncthreads();
      for (int b = threadIdx.x; b < kBins; b += kThreads) s.hist.count[b] = s.hist.lo[b] = s.hist.hi[b] = 0;
      __syncthreads();
      each([&](int i, float v) {
        if (!inside(i, v)) return;
        const int b = r.bin_of(v);
        atomicAdd(&s.hist.count[b], 1u);
        if (by_mass) {
          const uint64_t x = w.fixed(v);
          const uint32_t lo = (uint32_t)x, old = atomicAdd(&s.hist.lo[b], lo);
          atomicAdd(&s.hist.hi[b], (uint32_t)(x >> 32) + (old + lo < lo ? 1u : 0u));
        }
      });
      sync_row();
      // every CTA adds all histograms and finds the bin
      constexpr int kPer = kBins / kThreads;
      uint64_t mass[kPer], m = 0;
      uint32_t count[kPer], c = 0;
#pragma unroll
      for (int q = 0; q < kPer; ++q) {
        const int b = threadIdx.x * kPer + q;
        mass[q] = 0, count[q] = 0;
        for (int k = 0; k < ctas; ++k) {
          const Shared *o = ctas == 1 ? &s : cg::this_cluster().map_shared_rank(&s, k);
          count[q] += o->hist.count[b];
          if (by_mass) mass[q] += ((uint64_t)o->hist.hi[b] << 32) + o->hist.lo[b];
        }
        m += mass[q], c += count[q];
      }
      uint64_t ms = warp_scan_of(m, lane);
      uint32_t cs = warp_scan_of(c, lane);
      if (lane == 31) s.warp_mass[warp] = ms, s.warp_count[warp] = cs;
      __syncthreads();
      ms += r.above_mass - m, cs += r.above_count - c;
      for (int k = 0; k < warp; ++k) ms += s.warp_mass[k], cs += s.warp_count[k];
#pragma unroll
      for (int q = 0; q < kPer; ++q) {
        const uint64_t from = by_mass ? ms : cs, to = from + (by_mass ? mass[q] : count[q]);
        if (from < need && need <= to)
          s.found = threadIdx.x * kPer + q, s.found_mass = ms, s.found_count = cs, s.found_in = count[q];
        ms += mass[q], cs += count[q];
      }
      __syncthreads();
      r.bin = s.found;
      r.above_mass = s.found_mass;
      r.above_count = s.found_count;
      in = s.found_in;
      if (in <= kList) break;
      // its logits' smallest and largest
      float lo = INFINITY, hi = -INFINITY;
      each([&](int i, float v) {
        if (inside(i, v)) lo = fminf(lo, v), hi = fmaxf(hi, v);
      });
      extremes(lo, hi);
      r.lo = lo, r.hi = hi, r.bin = -1;
      r.top = nextafterf(hi, INFINITY);
    }
    uint64_t found[1] = {0};  // the token's index and logit
    if (in <= kList) {
      gather(r);
      if (rank == 0) {  // few enough: CTA 0 orders them
        const int len = s.list_n, per = threads_each(len), c = threadIdx.x / per;
        const Candidate x = s.list[min(c, len - 1)];
        const uint64_t before = (by_mass ? r.above_mass : r.above_count) + over_list(len, per, [&](const Candidate &y) {
          return y.v > x.v || (y.v == x.v && y.i < x.i) ? (by_mass ? y.w : 1) : 0;
        });
        if (c < len && before < need && need <= before + (by_mass ? x.w : 1))
          s.found_mass = (uint64_t)__float_as_uint(x.v) << 32 | (uint32_t)x.i;
        __syncthreads();
        found[0] = s.found_mass;
      }
      const uint64_t x = publish(found)[0][0];
      last_v = __uint_as_float((uint32_t)(x >> 32));
      last_i = (int)(uint32_t)x;
    } else {
      // equal logits: by their indexes
      const float v = r.lo;
      uint64_t rest = need - (by_mass ? r.above_mass : r.above_count);
      if (by_mass) {
        const uint64_t x = w.fixed(v);
        rest = (rest + x - 1) / x;
      }
      uint64_t all;
      const int at = find([&](int i, float y) -> uint64_t { return y == v && kept(i, y); },
                          [&](uint64_t) { return rest - 1; }, all);
      found[0] = at >= 0 ? first + at + 1 : 0;  // in one warp of the row
      const auto slot = publish(found);
      uint64_t a = 0;
      for (int k = lane; k < ctas * kWarps; k += 32) a += slot[0][k];
      last_v = v;
      last_i = (int)warp_sum_of(a) - 1;
    }
  }
};

// NaN is never drawn.
__device__ __forceinline__ float logit_of(float v) { return v == v ? v : -INFINITY; }
__device__ __forceinline__ float logit_of(__nv_bfloat16 v) { return logit_of(__bfloat162float(v)); }

template <class T>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleParams p) {
  extern __shared__ float4 s_logits[];
  __shared__ Shared s;
  cg::cluster_group cluster = cg::this_cluster();
  const int ctas = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int row = blockIdx.x / ctas, tid = threadIdx.x;
  const int first = min(p.V, rank * p.len), n = min(p.V - first, p.len);
  if (tid < 16) s.pow16[tid] = exp2((double)tid / 16.) * 0x1p44;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // 16-byte loads from the first aligned address on; the shared copy is shifted so that its stores are aligned too
  const T *src = reinterpret_cast<const T *>(p.logits) + (size_t)row * p.ld + first;
  constexpr int kVec = 16 / sizeof(T);
  const int head = min(n, (int)((-(uintptr_t)src & 15) / sizeof(T)));
  float *l = reinterpret_cast<float *>(s_logits) + (-head & 3);
  float lo = INFINITY, hi = -INFINITY;
  auto put = [&](float v) {
    hi = fmaxf(hi, v);
    if (v > -INFINITY) lo = fminf(lo, v);
    return v;
  };
  const int vecs = (n - head) / kVec;
#pragma unroll 4
  for (int i = tid; i < vecs; i += kThreads) {
    const uint4 q = __ldcs(reinterpret_cast<const uint4 *>(src + head) + i);
    float4 *dst = reinterpret_cast<float4 *>(l + head) + i * (kVec / 4);
    const uint32_t x[4] = {q.x, q.y, q.z, q.w};
    if constexpr (sizeof(T) == 4) {
      float f[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) f[j] = put(logit_of(__uint_as_float(x[j])));
      dst[0] = make_float4(f[0], f[1], f[2], f[3]);
    } else {
      float f[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        f[2 * j] = put(logit_of(__uint_as_float(x[j] << 16)));
        f[2 * j + 1] = put(logit_of(__uint_as_float(x[j] & 0xffff0000u)));
      }
      dst[0] = make_float4(f[0], f[1], f[2], f[3]);
      dst[1] = make_float4(f[4], f[5], f[6], f[7]);
    }
  }
  if (tid < head) l[tid] = put(logit_of(src[tid]));
  if (tid < n - head - vecs * kVec) {
    const int i = head + vecs * kVec + tid;
    l[i] = put(logit_of(src[i]));
  }

  const float temp = p.temperature ? p.temperature[row] : 1.f;
  const int top_k = p.top_k ? p.top_k[row] : 0;
  const float top_p = p.top_p ? p.top_p[row] : 1.f, u = p.u[row], q = p.min_p ? p.min_p[row] : 0.f;
  const bool greedy = !(temp > 0.f);
  Row r{s, l, n, first, rank, ctas, tid >> 5, tid & 31};
  r.extremes(lo, hi);
  auto put_out = [&](int token, float prob) {
    p.token[row] = token;
    if (p.prob) p.prob[row] = prob;
  };
  if (hi == -INFINITY) {
    if (rank == 0 && tid == 0) put_out(-1, 0.f);
    return;
  }
  if (hi == INFINITY) {  // only those are left, all alike
    for (int i = tid; i < n; i += kThreads) l[i] = l[i] == INFINITY ? 0.f : -INFINITY;
    __syncthreads();
    lo = hi = 0.f;
  }
  r.temp = temp;
  r.lowest = lo;
  r.w = Weight{hi, fmaxf(__fmaf_rn(-40.f, temp, hi), -FLT_MAX), 16. / (0.69314718055994530942 * (double)temp), s.pow16};
  const double min_w = q > 0.f ? fmin((double)q, 1.) * 0x1p44 : 0.;
  auto target = [&](uint64_t all) -> uint64_t {
    if (greedy || !(u > 0.f)) return 0;
    return u < 1.f ? min((uint64_t)((double)u * (double)all), all - 1) : all - 1;
  };
  auto need_of = [&](uint64_t all) -> uint64_t {
    return (uint64_t)max(__double2ll_ru((double)top_p * (double)all), 1ll);
  };

  // Where the tokens that stay are few and at the top, CTA 0 does the rest from
  // a list of them: k first tokens, of these those whose mass before them is
  // below need (0: top_p of the k's), of these what min-p leaves.
  auto finish = [&](int j, const Levels &t, int k, uint64_t need) {
    Range top = r.range_of(j, t);
    top.top = INFINITY;
    r.gather(top);
    if (rank != 0) return;
    const int len = s.list_n, per = Row::threads_each(len), c = tid / per;
    const Candidate x = s.list[min(c, len - 1)];
    // the tokens before it, their count above bit 53 (at most 2^8 weights of at most 2^44)
    const uint64_t ahead = r.over_list(len, per, [&](const Candidate &y) {
      return y.v > x.v || (y.v == x.v && y.i < x.i) ? y.w | 1ull << 53 : 0;
    });
    const uint64_t order = ahead >> 53, before = ahead & ((1ull << 53) - 1);
    if (c < len && (int)order == min(k, len) - 1) s.found_mass = before + x.w;
    __syncthreads();
    if (need == 0) need = top_p < 1.f ? need_of(s.found_mass) : s.found_mass + 1;
    const bool stays = (int)order < k && before < need && (order == 0 || r.w(x.v) >= min_w);
    if (c < len && tid % per == 0) s.list[c].w = stays ? x.w : 0;
    __syncthreads();
    const uint64_t Z = r.over_list(len, per, [&](const Candidate &y) { return y.w; });
    const uint64_t below = r.over_list(len, per, [&](const Candidate &y) { return y.i < x.i ? y.w : 0; });
    const uint64_t at = target(Z);
    if (c < len && tid % per == 0 && stays && below <= at && at < below + x.w) put_out(x.i, (float)(r.w(x.v) / (double)Z));
  };

  if (!greedy && top_k > 0 && top_k < p.V) {
    const Levels t = r.levels<false>();
    if ((uint32_t)top_k < t.count[kLevels]) {
      int j = 0;
      while (t.count[j] < (uint32_t)top_k) ++j;
      if (t.count[j] <= kList) {
        finish(j, t, top_k, 0);
        return;
      }
      const Range range = r.range_of(j, t);
      r.cut(top_k, false, range, t.count[j] - range.above_count);
    }
  }
  if (!greedy && top_p < 1.f) {
    const Levels t = r.levels<true>();
    const uint64_t need = need_of(t.mass[kLevels]);
    int j = 0;
    while (t.mass[j] < need) ++j;
    if (t.count[j] <= kList) {
      finish(j, t, kMaxV, need);
      return;
    }
    const Range range = r.range_of(j, t);
    r.cut(need, true, range, t.count[j] - range.above_count);
  }
  uint64_t Z;
  int at;
  if (greedy) {
    at = r.find([&](int, float v) -> uint64_t { return v == hi; }, target, Z);
  } else if (min_w > 0. || r.last_v > -INFINITY) {
    // few are kept: the others are seen by their logits, min-p's a little above its bound
    const float low = min_w > 0. ? fmaxf(r.last_v, __fmaf_rn(temp, logf(fminf(q, 1.f)) * 1.0001f - 1e-4f, hi)) : r.last_v;
    at = r.find(
        [&](int i, float v) -> uint64_t {
          if (!(v >= low && r.kept(i, v))) return 0;
          const double x = r.w(v);
          return x >= min_w ? Weight::to_fixed(x) : 0;
        },
        target, Z);
  } else {
    at = r.find([&](int, float v) { return r.w.fixed(v); }, target, Z);
  }
  if (at >= 0 && r.lane == 0) put_out(first + at, greedy ? 1.f : (float)(r.w(l[at]) / (double)Z));
}

template <class T>
int32_t launch_sample(SampleParams p, int32_t B, cudaStream_t s) {
  // CTAs of a row: at most 16384 logits each where that is possible, and more
  // of them while SMs are left and a CTA keeps 2048 logits
  int ctas = 1;
  while (ctas < kMaxCluster && (ceil_div(p.V, ctas) > 16384 ||
                                ((int64_t)B * ctas * 2 <= 2 * num_sms() && p.V / (2 * ctas) >= 2048)))
    ctas *= 2;
  p.len = ceil_div(ceil_div(p.V, ctas), 8) * 8;
  const size_t smem = (size_t)(p.len + 8) * 4;
  auto k = sample_kernel<T>;
  if (int32_t st = ensure_smem((const void *)k, smem)) return st;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(B * ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)ctas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (int32_t st = cuda_status(cudaLaunchKernelEx(&cfg, k, p))) return st;
  return launch_status();
}

}  // namespace
}  // namespace nslm

using namespace nslm;

extern "C" int32_t nslm_sample(const void *logits, int32_t type, int32_t B, int32_t V, int64_t ld,
                               const nslm_sample_params *params, const float *u, int32_t *token, float *prob,
                               nslm_stream_t stream) {
  g_launches = 0;
  if (type != NSLM_TYPE_F32 && type != NSLM_TYPE_BF16) return NSLM_ERR_ARG;
  if (B < 0 || B > (1 << 24) || V < 1 || V > kMaxV || ld < V) return NSLM_ERR_SHAPE;
  if (B > 0 && (!logits || !u || !token)) return NSLM_ERR_ARG;
  if (!aligned16(logits) || !aligned16(u) || !aligned16(token) || !aligned16(prob)) return NSLM_ERR_ALIGN;
  SampleParams p{logits, ld, V, 0, nullptr, nullptr, nullptr, nullptr, u, token, prob};
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
  st = type == NSLM_TYPE_BF16 ? launch_sample<__nv_bfloat16>(p, B, s) : launch_sample<float>(p, B, s);
  if (st == NSLM_OK) g_launches = 1;
  return st;
}
