// sample.cu -- nslm_sample: one token a row from logits, with temperature,
// top-k, top-p and min-p, at given random numbers.
#include <algorithm>

#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include "common.cuh"

namespace nslm {
namespace {

namespace cg = cooperative_groups;

constexpr int kMaxV = 1 << 18;
constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kBins = 512;
constexpr int kList = 256;
constexpr int kLevels = 4;

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
  bool greedy;   // only the logits equal to m have a weight, and it is 1
  double step;   // 16 / (temperature ln 2)
  const double *pow16;  // shared: 2^(44 + j/16)

  __device__ __forceinline__ double operator()(float v) const {
    if (greedy) return v == m ? 0x1p44 : 0.;
    const double t = ((double)v - (double)m) * step;
    if (!(t >= -16. * 46.)) return 0.;  // below 2^-45, and what is not to be drawn (v = -inf)
    const double kd = t + 0x1.8p52;     // t to the nearest integer, in the low bits
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
    return __hiloint2double(__double2hiint(w) + ((k >> 4) << 20), __double2loint(w));
  }
  __device__ __forceinline__ uint64_t fixed(float v) const { return to_fixed((*this)(v)); }
  // to the nearest integer: below 2^51 it stands in the low bits of w + 2^52
  static __device__ __forceinline__ uint64_t to_fixed(double w) {
    return (uint64_t)__double_as_longlong(w + 0x1p52) & 0xfffffffffffffull;
  }
};

// What the CTAs of a row tell one another.
struct Part {
  uint64_t mass[kLevels + 1];
  uint32_t count[kLevels + 1];
  float lo, hi;
};

struct Candidate {
  uint64_t w;
  float v;
  int32_t i;
};

struct Shared {
  double pow16[16];
  Part part[2][kMaxCluster];
  uint64_t warp_mass[kWarps][kLevels + 1];
  uint32_t warp_count[kWarps][kLevels + 1];
  float warp_lo[kWarps], warp_hi[kWarps];
  int32_t list_n;
  int32_t found;
  uint64_t found_before;
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

struct Row {
  const SampleParams &p;
  Shared &s;
  const float *l;   // shared: this CTA's logits
  int n;            // how many
  int first;        // the index of the first
  int rank, ctas;   // in the cluster
  int parity = 0;
  Weight w;
  // the last token that stays, in the order of descending logits and ascending indexes
  float last_v = -INFINITY;
  int last_i = kMaxV;

  __device__ __forceinline__ bool kept(int i, float v) const {
    return v > last_v || (v == last_v && first + i <= last_i);
  }

  // A warp's share of the CTA's logits: contiguous, so that sums over warps are sums over indexes.
  __device__ __forceinline__ int share() const { return ((n + kWarps - 1) / kWarps + 31) & ~31; }

  // Every CTA's part in every CTA; `mine` is taken from thread 0.
  __device__ const Part *exchange(const Part &mine) {
    Part *slots = s.part[parity];
    parity ^= 1;
    if (ctas == 1) {
      if (threadIdx.x == 0) slots[0] = mine;
      __syncthreads();
      return slots;
    }
    cg::cluster_group cluster = cg::this_cluster();
    if (threadIdx.x == 0)
      for (int r = 0; r < ctas; ++r) *cluster.map_shared_rank(&slots[rank], r) = mine;
    cluster.sync();
    return slots;
  }

  __device__ void sync_row() {
    if (ctas == 1) __syncthreads();
    else cg::this_cluster().sync();
  }

  // Sums of `parts` masses and counts over the row.
  __device__ Part sum_row(uint64_t (&mass)[kLevels + 1], uint32_t (&count)[kLevels + 1], int parts) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int j = 0; j < parts; ++j) {
      const uint64_t a = warp_sum_of(mass[j]);
      const uint32_t c = warp_sum_of(count[j]);
      if (lane == 0) s.warp_mass[warp][j] = a, s.warp_count[warp][j] = c;
    }
    __syncthreads();
    Part t{};
    if (threadIdx.x == 0)
      for (int k = 0; k < kWarps; ++k)
        for (int j = 0; j < parts; ++j) t.mass[j] += s.warp_mass[k][j], t.count[j] += s.warp_count[k][j];
    const Part *all = exchange(t);
    t = Part{};
    for (int r = 0; r < ctas; ++r)
      for (int j = 0; j < parts; ++j) t.mass[j] += all[r].mass[j], t.count[j] += all[r].count[j];
    return t;
  }

  // The lowest index for which the sum of f up to it exceeds target(the whole
  // sum), as the position in the CTA that has it, -1 in the others; before:
  // the sum below that index; all: the whole sum.
  template <class F, class G>
  __device__ int find(F f, G target, uint64_t &all) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int per = share();
    auto sum = [&](int lo, int hi) {
      uint64_t a = 0;
      for (int i = lo + lane; i < hi; i += 32) a += f(i, l[i]);
      return warp_sum_of(a);
    };
    __syncthreads();
    const uint64_t a = sum(warp * per, min(n, (warp + 1) * per));
    if (lane == 0) s.warp_mass[warp][0] = a;
    __syncthreads();
    Part mine{};
    if (threadIdx.x == 0)
      for (int k = 0; k < kWarps; ++k) mine.mass[0] += s.warp_mass[k][0];
    const Part *parts = exchange(mine);
    uint64_t before = 0, own = parts[rank].mass[0];
    all = 0;
    for (int r = 0; r < ctas; ++r) {
      if (r < rank) before += parts[r].mass[0];
      all += parts[r].mass[0];
    }
    const uint64_t t = target(all);
    if (t < before || t - before >= own) return -1;
    // the warp that has it, then the same over that warp's logits
    uint64_t left = t - before;
    int at = 0;
    while (at < kWarps - 1 && left >= s.warp_mass[at][0]) left -= s.warp_mass[at++][0];
    __syncthreads();
    const int lo = at * per, hi = min(n, lo + per), sub = (per / kWarps + 31) & ~31;
    const uint64_t c = sum(lo + warp * sub, min(hi, lo + (warp + 1) * sub));
    if (lane == 0) s.warp_mass[warp][0] = c;
    __syncthreads();
    at = 0;
    while (at < kWarps - 1 && left >= s.warp_mass[at][0]) left -= s.warp_mass[at++][0];
    if (warp == 0) {
      for (int i = lo + at * sub + lane; i - lane < hi; i += 32) {
        uint64_t x = i < hi ? f(i, l[i]) : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint64_t y = __shfl_up_sync(0xffffffffu, x, o);
          if (lane >= o) x += y;
        }
        const uint32_t over = __ballot_sync(0xffffffffu, x > left);
        if (over) {
          if (lane == 0) s.found = i + __ffs(over) - 1;
          break;
        }
        left -= __shfl_sync(0xffffffffu, x, 31);
      }
    }
    __syncthreads();
    return s.found;
  }

  // Sets the last token that stays to the one at which the kept tokens' count
  // (by_mass: their mass), in their order, first reaches `need`; all of them
  // together reach it.
  __device__ void cut(uint64_t need, bool by_mass, Range r, uint32_t in) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto inside = [&](int i) { return kept(i, l[i]) && r.has(l[i]); };
    while (in > kList && r.lo < r.hi) {
      // a histogram of the range; the bin that has the token is the next range
      for (int b = threadIdx.x; b < kBins; b += kThreads) s.hist.count[b] = s.hist.lo[b] = s.hist.hi[b] = 0;
      __syncthreads();
      for (int i = threadIdx.x; i < n; i += kThreads) {
        if (!inside(i)) continue;
        const int b = r.bin_of(l[i]);
        atomicAdd(&s.hist.count[b], 1u);
        if (by_mass) {
          const uint64_t x = w.fixed(l[i]);
          const uint32_t lo = (uint32_t)x, old = atomicAdd(&s.hist.lo[b], lo);
          atomicAdd(&s.hist.hi[b], (uint32_t)(x >> 32) + (old + lo < lo ? 1u : 0u));
        }
      }
      sync_row();
      // every CTA adds all histograms and finds the bin
      constexpr int kPer = kBins / kThreads;
      uint64_t mass[kPer];
      uint32_t count[kPer];
      uint64_t m = 0;
      uint32_t c = 0;
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
      // running sums over the threads
      uint64_t ms = m;
      uint32_t cs = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint64_t y = __shfl_up_sync(0xffffffffu, ms, o);
        const uint32_t z = __shfl_up_sync(0xffffffffu, cs, o);
        if (lane >= o) ms += y, cs += z;
      }
      if (lane == 31) s.warp_mass[warp][0] = ms, s.warp_count[warp][0] = cs;
      __syncthreads();
      ms += r.above_mass - m, cs += r.above_count - c;
      for (int k = 0; k < warp; ++k) ms += s.warp_mass[k][0], cs += s.warp_count[k][0];
#pragma unroll
      for (int q = 0; q < kPer; ++q) {
        const uint64_t from = by_mass ? ms : cs, to = from + (by_mass ? mass[q] : count[q]);
        if (from < need && need <= to) {
          s.found = threadIdx.x * kPer + q;
          s.found_before = ms;
          s.list_n = (int32_t)cs;
          s.warp_count[0][1] = count[q];
        }
        ms += mass[q], cs += count[q];
      }
      __syncthreads();
      r.bin = s.found;
      r.above_mass = s.found_before;
      r.above_count = (uint32_t)s.list_n;
      in = s.warp_count[0][1];
      if (in <= kList) break;
      // its logits' smallest and largest
      float lo = INFINITY, hi = -INFINITY;
      for (int i = threadIdx.x; i < n; i += kThreads)
        if (inside(i)) lo = fminf(lo, l[i]), hi = fmaxf(hi, l[i]);
      extremes(lo, hi);
      r.lo = lo, r.hi = hi, r.bin = -1;
      r.top = nextafterf(hi, INFINITY);
    }
    Part found{};
    if (in <= kList) {
      // few enough: CTA 0 orders them
      __syncthreads();
      if (threadIdx.x == 0) s.list_n = 0;
      sync_row();
      Shared *o = ctas == 1 ? &s : cg::this_cluster().map_shared_rank(&s, 0);
      for (int i = threadIdx.x; i < n; i += kThreads)
        if (inside(i)) o->list[atomicAdd(&o->list_n, 1)] = Candidate{w.fixed(l[i]), l[i], first + i};
      sync_row();
      if (rank == 0) {
        const int c = threadIdx.x;
        if (c < s.list_n) {
          const Candidate x = s.list[c];
          uint64_t before = by_mass ? r.above_mass : r.above_count;
          for (int j = 0; j < s.list_n; ++j) {
            const Candidate y = s.list[j];
            if (y.v > x.v || (y.v == x.v && y.i < x.i)) before += by_mass ? y.w : 1;
          }
          if (before < need && need <= before + (by_mass ? x.w : 1)) s.warp_lo[0] = x.v, s.found = x.i;
        }
        __syncthreads();
        found.lo = s.warp_lo[0];
        found.count[0] = s.found;
      }
      const Part *all = exchange(found);
      last_v = all[0].lo;
      last_i = (int)all[0].count[0];
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
      found.count[0] = at >= 0 ? first + at + 1 : 0;
      const Part *parts = exchange(found);
      last_v = v;
      for (int k = 0; k < ctas; ++k)
        if (parts[k].count[0]) last_i = (int)parts[k].count[0] - 1;
    }
  }

  // Smallest and largest over the row.
  __device__ void extremes(float &lo, float &hi) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
      hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    if (lane == 0) s.warp_lo[warp] = lo, s.warp_hi[warp] = hi;
    __syncthreads();
    Part t{};
    t.lo = INFINITY, t.hi = -INFINITY;
    if (threadIdx.x == 0)
      for (int k = 0; k < kWarps; ++k) t.lo = fminf(t.lo, s.warp_lo[k]), t.hi = fmaxf(t.hi, s.warp_hi[k]);
    const Part *all = exchange(t);
    lo = INFINITY, hi = -INFINITY;
    for (int r = 0; r < ctas; ++r) lo = fminf(lo, all[r].lo), hi = fmaxf(hi, all[r].hi);
  }

  // The tokens with logits from m down to 3, 7, 12 and 20 temperatures below,
  // and all: how many they are, and their mass.
  __device__ __forceinline__ float level(int j, float temp) const {
    return __fmaf_rn(-temp, j == 0 ? 3.f : j == 1 ? 7.f : j == 2 ? 12.f : 20.f, w.m);
  }
  __device__ Part levels(float temp, bool by_mass) {
    uint64_t mass[kLevels + 1] = {};
    uint32_t count[kLevels + 1] = {};
    float at[kLevels];
#pragma unroll
    for (int j = 0; j < kLevels; ++j) at[j] = level(j, temp);
    for (int i = threadIdx.x; i < n; i += kThreads) {
      const float v = l[i];
      if (v == -INFINITY || !kept(i, v)) continue;
      const uint64_t x = by_mass ? w.fixed(v) : 0;
      mass[kLevels] += x, ++count[kLevels];
#pragma unroll
      for (int j = 0; j < kLevels; ++j)
        if (v >= at[j]) mass[j] += x, ++count[j];
    }
    return sum_row(mass, count, kLevels + 1);
  }
  __device__ void cut_level(uint64_t need, bool by_mass, float temp, float lowest, const Part &t) {
    int j = 0;
    while (j < kLevels && (by_mass ? t.mass[j] : t.count[j]) < need) ++j;
    Range r;
    r.lo = j < kLevels ? fmaxf(level(j, temp), lowest) : lowest;
    r.top = j > 0 ? level(j - 1, temp) : INFINITY;
    r.hi = fminf(r.top, w.m);
    r.above_mass = j > 0 ? t.mass[j - 1] : 0;
    r.above_count = j > 0 ? t.count[j - 1] : 0;
    cut(need, by_mass, r, t.count[j] - r.above_count);
  }
};

// NaN is never drawn.
__device__ __forceinline__ float logit_of(float v) { return v == v ? v : -INFINITY; }
__device__ __forceinline__ float logit_of(__nv_bfloat16 v) { return logit_of(__bfloat162float(v)); }

template <class T>
__global__ void __launch_bounds__(kThreads) sample_kernel(const SampleParams p) {
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
  for (int i = tid; i < n; i += kThreads)
    if (i < head || i >= head + vecs * kVec) l[i] = put(logit_of(src[i]));

  Row r{p, s, l, n, first, rank, ctas};
  r.extremes(lo, hi);
  const float temp = p.temperature ? p.temperature[row] : 1.f;
  const bool greedy = !(temp > 0.f);
  if (hi == INFINITY) {  // only those are left, all alike
    for (int i = tid; i < n; i += kThreads) l[i] = l[i] == INFINITY ? 0.f : -INFINITY;
    __syncthreads();
    lo = hi = 0.f;
  }
  r.w = Weight{hi, greedy, 16. / (0.69314718055994530942 * (double)temp), s.pow16};
  if (hi == -INFINITY) {
    if (rank == 0 && tid == 0) {
      p.token[row] = -1;
      if (p.prob) p.prob[row] = 0.f;
    }
    return;
  }
  if (!greedy) {
    const int top_k = p.top_k ? p.top_k[row] : 0;
    if (top_k > 0 && top_k < p.V) {
      const Part t = r.levels(temp, false);
      if ((uint32_t)top_k < t.count[kLevels]) r.cut_level(top_k, false, temp, lo, t);
    }
    const float top_p = p.top_p ? p.top_p[row] : 1.f;
    if (top_p < 1.f) {
      const Part t = r.levels(temp, true);
      const int64_t need = __double2ll_ru((double)top_p * (double)t.mass[kLevels]);
      r.cut_level((uint64_t)max(need, (int64_t)1), true, temp, lo, t);
    }
  }
  const float q = p.min_p ? p.min_p[row] : 0.f;
  const double min_w = q > 0.f ? fmin((double)q, 1.) * 0x1p44 : 0.;
  const float u = p.u[row];
  uint64_t Z;
  const int at = r.find(
      [&](int i, float v) -> uint64_t {
        if (!r.kept(i, v)) return 0;
        const double x = r.w(v);
        return x >= min_w ? Weight::to_fixed(x) : 0;
      },
      [&](uint64_t all) -> uint64_t {
        if (greedy || !(u > 0.f)) return 0;
        return u < 1.f ? min((uint64_t)((double)u * (double)all), all - 1) : all - 1;
      },
      Z);
  if (at >= 0 && tid == 0) {
    p.token[row] = first + at;
    if (p.prob) p.prob[row] = greedy ? 1.f : (float)(r.w(l[at]) / (double)Z);
  }
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
