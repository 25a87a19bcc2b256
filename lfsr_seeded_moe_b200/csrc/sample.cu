// sample.cu -- nslm_sample: one token a row from logits, with temperature,
// top-k, top-p and min-p, at given random numbers.
#include <algorithm>
#include <cfloat>
#include <type_traits>

#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include "common.cuh"

namespace nslm {
namespace {

namespace cg = cooperative_groups;

constexpr int kMaxV = 1 << 18;
constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kBins = 4096;
constexpr int kList = 2 * kThreads;       // candidates that are sorted
constexpr int kFew = kThreads / 8;        // up to here they are compared with one another
constexpr int kAll = 256;                 // a row of so few logits is one list
constexpr int kCountBins = 2 * kThreads;  // that find where a long list begins
constexpr int kGroups = 128;              // parts of a row whose largest logits are known
constexpr int kListAt = 96;               // the last of those, in descending order, from which a top-k's list begins
// The one from which on a list is made for top-p: 266 tokens on average.  At 96
// (177) it costs 1 to 3% less, at 120 (355) as much more; a row whose top-p is
// past its list costs 20 us and more.  Of rows of 32000 with some tens of likely
// tokens 45, 39 and 35% are past the three with top-p 0.9; of 131072 92, 92 and 91%.
constexpr int kListMass = 112;

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

// A cluster of up to 8 CTAs has one row, each CTA a part of it.  While there are
// SMs for more CTAs, a CTA reads its part once and keeps it in shared memory as
// fp32 (RES).  Of a larger batch it takes a longer part, which passes through
// small rings of its warps each time it is needed, from the L2 after the first:
// then a row's barriers, about 1 us each, are shared by more logits, and the
// whole batch runs at once (64 x 131072 with top-k 50: 34 us kept, 23 streamed).
//
// w is 64-bit fixed point with 44 bits behind the point, at most 2^18 of them,
// so sums stay below 2^62 and are exact: whatever order threads and CTAs add in,
// the same u gives the same token.
//
// One row of 32003 logits with top-k 50 and top-p takes 8.1 us, nearly all of it
// latency: its load, four exchanges, the list's sort and sums; 64 x 131072 without a filter 32 us, bound by the
// instructions of two passes (0.62 of the issue slots, DRAM at 15%).

// Weights in units of 2^-44.  exp(x) = 2^(k/16) e^r, |r| <= ln 2 / 32, with the
// 16 powers from a table and e^r by its series to r^5 (the table method of
// P. T. P. Tang, "Table-driven implementation of the exponential function in
// IEEE floating-point arithmetic", ACM TOMS 15, 1989): off by at most
// r^6 / 720 = 2^-43 of itself.  A 16-entry table lies in 32 banks, so lanes
// never wait for one another.  A pass is bound by its instructions, about 45 a
// logit: with k from fp32 beside the fp64 operations, or the series in pairs
// of terms, it takes more of them (32 us for 64 x 131072 logits, 34 and 35).
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
    return v >= low ? __hiloint2double(__double2hiint(w) + ((k & ~15) << 16), __double2loint(w)) : 0.;
  }
  __device__ __forceinline__ uint64_t fixed(float v) const { return to_fixed((*this)(v)); }
  // to the nearest integer: below 2^51 it stands in the low bits of w + 2^52
  static __device__ __forceinline__ uint64_t to_fixed(double w) {
    return (uint64_t)__double_as_longlong(w + 0x1p52) & 0xfffffffffffffull;
  }
};

// A logit's place among all fp32 values.
__device__ __forceinline__ uint32_t order_of(float v) {
  const uint32_t b = __float_as_uint(v + 0.f);  // -0 as 0
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
// A token of a list: its logit's place, then its index falling, so that of two
// the larger comes first.
__device__ __forceinline__ uint64_t key_of(float v, int i) { return (uint64_t)order_of(v) << 32 | ~(uint32_t)i; }
__device__ __forceinline__ int index_of(uint64_t key) { return (int)~(uint32_t)key; }
__device__ __forceinline__ float logit_of(uint64_t key) {
  const uint32_t k = (uint32_t)(key >> 32);
  return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

struct alignas(16) Shared {
  double pow16[16];
  // what the CTAs of a row tell one another, by turns
  uint64_t slot[2][2][kMaxCluster];
  alignas(16) float group_max[kGroups];
  uint64_t warp_mass[kWarps];
  uint32_t warp_count[kWarps];
  float warp_lo[kWarps], warp_hi[kWarps];
  float m, list_from, list_top;
  int32_t list_n;
  int32_t found;
  uint64_t found_mass;
  union {
    struct {
      uint32_t lo[kBins], hi[kBins];
    } hist;
    struct {
      uint64_t mine[kList];            // the CTA's part of a list; in CTA 0 then the whole in order, then by indexes
      union {
        uint64_t list[kList];          // in CTA 0 all parts
        struct {
          uint64_t few[kFew];          // (what a short list needs while `place` is written)
          uint16_t place[kList];       // of the sorted, by their indexes
        };
      };
      union {
        uint64_t key[kList];           // while they are sorted; then the weights by their indexes
        uint32_t count[kCountBins];    // before there is a list
      };
      uint32_t low[kList], start[kThreads + 1];
    };
  };
};

template <int LANES = 32, class T> __device__ __forceinline__ T warp_sum_of(T v) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
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

// Puts the n candidates of s.list in order, in s.mine, with their places in the
// order of their indexes.
//
// Up to kFew: each one's place is the number of those before it, counted by 8
// threads.  More: two bucket sorts at once, kThreads buckets by the logit
// (from `top` down, 1 / scale each) and by the index (2^shift each), with the
// two counts in the halves of a word; then each counts those of its buckets
// that come before it, a few unless logits are equal.  (What is above `top` has
// the first bucket: a few again, and one far outlier stretches none.)  Of 55 candidates
// the first takes 1050 cycles and the second 2600, of 177 they take 4700 and
// 3400.
__device__ __forceinline__ void sort_list(Shared &s, int n, float top, float scale, int shift) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (n <= kFew) {
    const int c = tid / 8;
    const uint64_t key = s.list[min(c, n - 1)];
    int order = 0, place = 0;
#pragma unroll 4
    for (int j = tid & 7; j < n; j += 8) {
      const uint64_t k = s.list[j];
      order += k > key;
      place += (uint32_t)k > (uint32_t)key;
    }
    order = warp_sum_of<8>(place << 16 | order);
    if (c < n && (tid & 7) == 0 && in_bounds(order & 0xffff, n, 45))
      s.mine[order & 0xffff] = key, s.place[order & 0xffff] = (uint16_t)(order >> 16);
    __syncthreads();
    return;
  }
  constexpr int kPer = kList / kThreads;
  s.start[tid] = 0;
  __syncthreads();
  uint64_t x[kPer];
  int by_logit[kPer], by_index[kPer];
  uint32_t at[kPer];
#pragma unroll
  for (int q = 0; q < kPer; ++q) {
    if (tid + q * kThreads >= n) break;
    x[q] = s.list[tid + q * kThreads];
    by_logit[q] = max(0, min(kThreads - 1, (int)((top - logit_of(x[q])) * scale)));
    by_index[q] = index_of(x[q]) >> shift;
    if (!in_bounds(by_index[q], kThreads, 44)) by_index[q] = 0;
    at[q] = atomicAdd(&s.start[by_logit[q]], 1u) & 0xffff;
    at[q] |= atomicAdd(&s.start[by_index[q]], 0x10000u) & 0xffff0000u;
  }
  __syncthreads();
  const uint32_t mine = s.start[tid];
  uint32_t before = warp_scan_of(mine, lane) - mine;
  if (lane == 31) s.warp_count[warp] = before + mine;
  __syncthreads();
  before += warp_sum_of(lane < warp ? s.warp_count[lane] : 0u);
  s.start[tid] = before;
  if (tid == kThreads - 1) s.start[kThreads] = before + mine;
  __syncthreads();
#pragma unroll
  for (int q = 0; q < kPer; ++q) {
    if (tid + q * kThreads >= n) break;
    const uint32_t to = (s.start[by_logit[q]] + at[q]) & 0xffff, to_low = (s.start[by_index[q]] + (at[q] & 0xffff0000u)) >> 16;
    if (in_bounds(to, n, 44)) s.key[to] = x[q];
    if (in_bounds(to_low, n, 44)) s.low[to_low] = (uint32_t)x[q];
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < kPer; ++q) {
    if (tid + q * kThreads >= n) break;
    const int logit0 = s.start[by_logit[q]] & 0xffff, logit1 = s.start[by_logit[q] + 1] & 0xffff;
    const int index0 = s.start[by_index[q]] >> 16, index1 = s.start[by_index[q] + 1] >> 16;
    int order = logit0, place = index0;
    for (int j = logit0; j < logit1; ++j) order += s.key[j] > x[q];
    for (int j = index0; j < index1; ++j) place += s.low[j] > (uint32_t)x[q];  // these fall with the index
    if (!in_bounds(order, n, 45)) continue;
    s.mine[order] = x[q];
    s.place[order] = (uint16_t)place;
  }
  __syncthreads();
}

// The sum of the values before this thread's, and of all, in the first `warps`
// warps; the others have none and only wait.
__device__ __forceinline__ uint64_t sum_before(Shared &s, uint64_t v, int warps, uint64_t &all) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint64_t before = 0;
  all = 0;
  if (warp < warps) {
    const uint64_t upto = warp_scan_of(v, lane);
    if (lane == 31) s.warp_mass[warp] = upto;
    before = upto - v;
  }
  __syncthreads();
  if (warp < warps) {
    for (int k = 0; k < warps; ++k) {
      const uint64_t x = s.warp_mass[k];
      before += k < warp ? x : 0;
      all += x;
    }
  }
  return before;
}
// The warps that have n candidates, two a thread.
__device__ __forceinline__ int warps_of(int n) { return (n + 63) / 64; }

// The candidate of s.list at which the count or mass in their order first
// reaches `need`: its key to s.found_mass.
__device__ __forceinline__ void find_in_list(Shared &s, int n, float top, float scale, int shift, uint64_t need, bool by_mass,
                                          Weight w) {
  sort_list(s, n, top, scale, shift);
  const int at = 2 * threadIdx.x;  // of two each thread has
  uint64_t x[2] = {0, 0}, m[2] = {0, 0}, all;
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    if (at + q >= n) break;
    x[q] = s.mine[at + q];
    m[q] = by_mass ? w.fixed(logit_of(x[q])) : 1;
  }
  uint64_t before = sum_before(s, m[0] + m[1], warps_of(n), all);
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    if (before < need && need <= before + m[q]) s.found_mass = x[q];
    before += m[q];
  }
  __syncthreads();
}

// Of a row whose kept tokens weigh `all`, the weight that the token's sum exceeds.
__device__ __forceinline__ uint64_t target_of(float u, uint64_t all) {
  if (!(u > 0.f)) return 0;
  return u < 1.f ? min((uint64_t)((double)u * (double)all), all - 1) : all - 1;
}
// The least mass that top-p keeps.
__device__ __forceinline__ uint64_t need_of(float top_p, uint64_t all) {
  return (uint64_t)max(__double2ll_ru((double)top_p * (double)all), 1ll);
}

struct ListTask {
  Weight weight;
  double min_w;
  uint64_t all;      // the row's mass, if top-p asks for it
  float top, scale;  // of the sort's buckets
  float u, top_p;
  int top_k;         // 0: off
  bool by_mass;
  int n, shift;
};

// Draws the row's token from the n candidates of s.list, if all that stay are
// among them; else false.  Their mass, or top-k's, in s.found_mass.
__device__ __forceinline__ bool draw_from_list(Shared &s, const SampleParams &p, int row, ListTask t) {
  const int tid = threadIdx.x, at = 2 * tid;  // of two tokens each thread has
  sort_list(s, t.n, t.top, t.scale, t.shift);
  const int limit = t.top_k ? min(t.top_k, t.n) : t.n, warps = warps_of(t.n);
  uint64_t x[2] = {0, 0}, m[2] = {0, 0}, Z;
  bool stays[2] = {false, false};
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    if (at + q >= t.n) break;
    x[q] = s.mine[at + q];
    const double w = t.weight(logit_of(x[q]));
    stays[q] = at + q < limit && (at + q == 0 || w >= t.min_w);
    m[q] = Weight::to_fixed(w);
    if (at + q == t.n - 1) s.found = w < t.min_w || p.V <= kAll;
  }
  const uint64_t before = sum_before(s, m[0] + m[1], warps, Z);
  if (at == limit - 1) s.found_mass = before + m[0];
  if (at + 1 == limit - 1) s.found_mass = before + m[0] + m[1];
  __syncthreads();
  // all that stays is in the list if its end is behind top-k's, top-p's or min-p's
  const uint64_t need = t.by_mass ? need_of(t.top_p, t.top_k ? s.found_mass : t.all) : s.found_mass + 1;
  if (t.top_k ? !(t.n >= t.top_k || (s.found && (!t.by_mass || p.V <= kAll))) : !(s.found || s.found_mass >= need)) return false;
  // of the first top_k, those stay with less than need before them that min-p leaves; then all by their indexes
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    if (at + q >= t.n) break;
    const int place = s.place[at + q];
    if (!in_bounds(place, t.n, 45)) continue;
    s.mine[place] = x[q];
    s.key[place] = stays[q] && before + (q ? m[0] : 0) < need ? m[q] : 0;
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < 2; ++q) m[q] = at + q < t.n ? s.key[at + q] : 0;
  const uint64_t below = sum_before(s, m[0] + m[1], warps, Z), to = target_of(t.u, Z);
  if (below <= to && to < below + m[0] + m[1]) {
    const uint64_t y = s.mine[at + (to < below + m[0] ? 0 : 1)];
    if (!in_bounds(index_of(y), p.V, 47)) return true;
    p.token[row] = index_of(y);
    if (p.prob) p.prob[row] = (float)(t.weight(logit_of(y)) / (double)Z);
  }
  return true;
}

// The tokens between two logits, in the order of their logits.
struct Range {
  float lo, top;       // lo <= v < top
  float hi;            // the largest v there, or a bound
  int bin = -1;        // of those, the ones in this bin of [lo, hi], or all
  uint64_t above = 0;  // the count or mass of the kept tokens that come before

  // A bin falls from 0 at hi to kBins - 1 at lo, for any lo < hi.  Bins are
  // equally wide in three rounds, which part all but values of many magnitudes,
  // unless hi - lo is so small that `scale` is infinite.  Then they have 2^shift
  // neighbouring fp32 values each: of 2^32 at most a bin has 2^20, 2^8 and one,
  // so another three rounds end at a single value, whatever the logits.
  static constexpr int kEvenRounds = 3;
  float half = 1.f, scale = 0.f;
  int shift = -1;  // -1: equally wide
  __device__ __forceinline__ void set_bins(int round) {
    static_assert(kBins == 1 << 12);
    half = hi - lo < INFINITY ? 1.f : 0.5f;
    scale = kBins / (hi * half - lo * half);
    shift = round < kEvenRounds && scale < INFINITY ? -1 : max(0, 32 - __clz(order_of(hi) - order_of(lo)) - 12);
    bin = -1;
  }
  template <bool EVEN> __device__ __forceinline__ int bin_as(float v) const {
    if (!EVEN) return (int)((order_of(hi) - order_of(v)) >> shift);
    return min(kBins - 1, (int)(__fmaf_rn(-half, v, hi * half) * scale));
  }
  __device__ __forceinline__ int bin_of(float v) const { return shift < 0 ? bin_as<true>(v) : bin_as<false>(v); }
  // The chosen bin's tokens lie between lo and top too; these are bounds that
  // are a little wide, to see most others without their bin.
  __device__ __forceinline__ void set_bin(int b) {
    bin = b;
    if (shift >= 0 || !(scale < 1e30f)) return;  // the bounds themselves would be rounded away
    const float eps = 0x1p-20f * (fabsf(hi) + fabsf(lo)) * half, of = hi * half, width = 1.f / scale;
    lo = fmaxf(lo, (of - ((b + 1.01f) * width + eps)) / half);
    if (b > 0) top = fminf(top, (of - ((b - 0.01f) * width - eps)) / half);
  }
  __device__ __forceinline__ bool has(float v) const { return v >= lo && v < top && (bin < 0 || bin_of(v) == bin); }
};

// NaN is never drawn.
__device__ __forceinline__ float logit_of(float v) { return fmaxf(v, -INFINITY); }
__device__ __forceinline__ float logit_of(__nv_bfloat16 v) { return logit_of(__bfloat162float(v)); }

constexpr int kRing = 4, kRingChunk = 512;  // chunks of a warp's ring, and their bytes

template <class T, bool RES> struct Row {
  Shared &s;
  const float *l;  // RES: this CTA's logits, in shared memory; else the CTA's rings
  const T *src;    // and in global memory
  int n;           // how many
  int first;       // the index of the first
  int rank, ctas;  // in the cluster
  int warp, lane;
  int parity = 0;
  int index_shift = 0;    // of an index to one of kThreads buckets
  bool infinite = false;  // +inf occurs: those are 0, all others -inf
  Weight w{};
  // the last token that stays, in the order of descending logits and ascending indexes
  float last_v = -INFINITY;
  int last_i = kMaxV;

  // the CTA's logits, and the up to 15 bytes between an aligned address and them
  __device__ __forceinline__ bool in_row(const char *at, int bytes) const {
    const char *lo = (const char *)((uintptr_t)src & ~(uintptr_t)15);
    return in_buffer(at, bytes, lo, (const char *)(src + n) - lo, 40);
  }

  __device__ __forceinline__ bool kept(int i, float v) const {
    return v > last_v || (v == last_v && first + i <= last_i);
  }

  // A warp's share of the CTA's logits: contiguous, so that sums over warps are sums over indexes.
  __device__ __forceinline__ int share() const { return ((n + kWarps - 1) / kWarps + 31) & ~31; }

  __device__ __forceinline__ float value(float v) const {
    return infinite ? (v == INFINITY ? 0.f : -INFINITY) : v;
  }
  __device__ __forceinline__ float at(int i) const {
    if (!in_bounds(i, n, RES ? 41 : 40)) return -INFINITY;
    return RES ? l[i] : value(logit_of(src[i]));
  }

  // f(i, logit) for this thread's logits, U at a time so that their latencies overlap.
  template <int U, class F> __device__ __forceinline__ void each(F f) const {
    if constexpr (RES) {
      int i = threadIdx.x;
      for (; i + (U - 1) * kThreads < n; i += U * kThreads) {
        float v[U];
#pragma unroll
        for (int j = 0; j < U; ++j) v[j] = l[i + j * kThreads];
#pragma unroll
        for (int j = 0; j < U; ++j) f(i + j * kThreads, v[j]);
      }
#pragma unroll 1
      for (; i < n; i += kThreads) f(i, l[i]);
    } else {
      // the warp's share by 16-byte copies from the last aligned address before
      // it; bytes past its end are zeros
      constexpr int kOf = kRingChunk / sizeof(T);
      static_assert(kRingChunk % 512 == 0 && kOf % (32 * U) == 0, "lanes go through a chunk in whole steps");
      const int lo = min(n, warp * share()), hi = min(n, lo + share());
      const int before = (int)(((uintptr_t)(src + lo) & 15) / sizeof(T));
      const char *from = reinterpret_cast<const char *>(src + lo - before);
      const int bytes = lo < hi ? (before + hi - lo) * (int)sizeof(T) : 0;
      const T *ring = reinterpret_cast<const T *>(l) + warp * kRing * kOf;
      const uint32_t to = (uint32_t)__cvta_generic_to_shared(ring) + lane * 16;
      auto load = [&](int c) {
#pragma unroll
        for (int j = 0; j < kRingChunk; j += 512) {
          const int off = c * kRingChunk + j + lane * 16;
          if (off < bytes && in_row(from + off, min(16, bytes - off)) &&
              in_bounds(warp * kRing * kRingChunk + c % kRing * kRingChunk + j + lane * 16 + 15,
                        kWarps * kRing * kRingChunk, 42))
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + c % kRing * kRingChunk + j),
                         "l"(from + off), "r"(min(16, bytes - off))
                         : "memory");
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
      };
      for (int c = 0; c < kRing - 1; ++c) load(c);
      for (int c = 0; c * kRingChunk < bytes; ++c) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 2) : "memory");
        __syncwarp();
        load(c + kRing - 1);
        const T *in = ring + c % kRing * kOf;
        const int i0 = lo + c * kOf - before;  // the index of its first
        if (i0 >= lo && i0 + kOf <= hi && !infinite) {
          for (int q = 2 * lane; q < kOf; q += 32 * U) {
            float v[U];
#pragma unroll
            for (int j = 0; j < U; j += 2) {
              if constexpr (sizeof(T) == 4) {
                const float2 x = *reinterpret_cast<const float2 *>(in + q + 32 * j);
                v[j] = logit_of(x.x), v[j + 1] = logit_of(x.y);
              } else {
                const uint32_t x = *reinterpret_cast<const uint32_t *>(in + q + 32 * j);
                v[j] = logit_of(__uint_as_float(x << 16)), v[j + 1] = logit_of(__uint_as_float(x & 0xffff0000u));
              }
            }
#pragma unroll
            for (int j = 0; j < U; ++j) f(i0 + q + 32 * (j & ~1) + (j & 1), v[j]);
          }
        } else {
#pragma unroll 1
          for (int i = max(i0, lo) + lane; i < min(i0 + kOf, hi); i += 32) f(i, value(logit_of(in[i - i0])));
        }
      }
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      __syncwarp();
    }
  }

  __device__ __forceinline__ void sync_row() const {
    if (ctas == 1) __syncthreads();
    else cg::this_cluster().sync();
  }

  // A CTA's values, held by its first warp's lanes, to every CTA.  Two sets of
  // slots by turns: who writes one again has passed the barrier after which
  // the others had read it.
  using Slots = const uint64_t (*)[kMaxCluster];
  template <int V> __device__ __forceinline__ Slots publish(const uint64_t (&v)[V]) {
    auto slot = s.slot[parity];
    parity ^= 1;
    if (threadIdx.x < ctas) {
      uint64_t *to = ctas == 1 ? &slot[0][0] : cg::this_cluster().map_shared_rank(&slot[0][0], threadIdx.x);
#pragma unroll
      for (int j = 0; j < V; ++j) to[j * kMaxCluster + rank] = v[j];
    }
    sync_row();
    return slot;
  }

  // Smallest and largest over the row.
  __device__ __forceinline__ void extremes(float &lo, float &hi) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
      hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    if (lane == 0) s.warp_lo[warp] = lo, s.warp_hi[warp] = hi;
    __syncthreads();
    for (int k = 0; k < kWarps; ++k) lo = fminf(lo, s.warp_lo[k]), hi = fmaxf(hi, s.warp_hi[k]);
    const uint64_t v[1] = {(uint64_t)__float_as_uint(hi) << 32 | __float_as_uint(lo)};
    const auto slot = publish(v);
    for (int k = 0; k < ctas; ++k) {
      lo = fminf(lo, __uint_as_float((uint32_t)slot[0][k]));
      hi = fmaxf(hi, __uint_as_float((uint32_t)(slot[0][k] >> 32)));
    }
  }

  // A lane's part of the sum of f over its warp's share.
  template <class F> __device__ __forceinline__ uint64_t over_share(F f) const {
    uint64_t a = 0;
    if constexpr (RES) {
      const int hi = min(n, (warp + 1) * share());
      int i = warp * share() + lane;
      for (; i + 32 < hi; i += 64) {
        const float x = l[i], y = l[i + 32];
        a += f(i, x) + f(i + 32, y);
      }
      if (i < hi) a += f(i, l[i]);
    } else {
      each<2>([&](int i, float v) { a += f(i, v); });
    }
    return a;
  }

  // The sum of the warps' values, in the first warp.
  __device__ __forceinline__ uint64_t cta_sum(const uint64_t (&v)[kWarps]) const {
    return warp == 0 ? warp_sum_of(lane < kWarps ? v[lane] : 0) : 0;
  }

  // The lowest index for which the sum of f up to it exceeds target(the whole
  // sum all), as the position in the CTA that has it, valid in one warp of
  // that CTA; -1 everywhere else.
  template <class F, class G> __device__ __forceinline__ int find(F f, G target, uint64_t &all) {
    const int per = share();
    auto sum = [&](int lo, int hi) {
      uint64_t a = 0;
      int i = lo + lane;
      for (; i + 32 < hi; i += 64) {
        const float x = at(i), y = at(i + 32);
        a += f(i, x) + f(i + 32, y);
      }
      if (i < hi) a += f(i, at(i));
      return warp_sum_of(a);
    };
    uint64_t mine = warp_sum_of(over_share(f));
    if (lane == 0) s.warp_mass[warp] = mine;
    __syncthreads();
    const uint64_t v[1] = {cta_sum(s.warp_mass)};
    const auto slot = publish(v);
    // the CTA that has it, then the warp
    uint64_t before = 0;
    all = 0;
    for (int k = 0; k < ctas; ++k) {
      if (k == rank) before = all;
      all += slot[0][k];
    }
    uint64_t left = target(all);
    if (left < before || left - before >= slot[0][rank]) return -1;
    left -= before;
    int in = 0;
    while (in < kWarps - 1 && left >= s.warp_mass[in]) left -= s.warp_mass[in++];
    int lo = in * per, hi = min(n, lo + per);
    for (int len = per; len > 256;) {  // all warps on that warp's logits, and again
      len = (len / kWarps + 31) & ~31;
      mine = sum(lo + warp * len, min(hi, lo + (warp + 1) * len));
      __syncthreads();
      if (lane == 0) s.warp_mass[warp] = mine;
      __syncthreads();
      in = 0;
      while (in < kWarps - 1 && left >= s.warp_mass[in]) left -= s.warp_mass[in++];
      lo += in * len;
      hi = min(hi, lo + len);
    }
    if (warp != in) return -1;
    for (int i = lo; i < hi; i += 32) {
      const uint64_t upto = warp_scan_of(f(i + lane, i + lane < hi ? at(i + lane) : -INFINITY), lane);
      const uint32_t over = __ballot_sync(0xffffffffu, upto > left);
      if (over) return i + __ffs(over) - 1;
      left -= __shfl_sync(0xffffffffu, upto, 31);
    }
    return -1;
  }

  // A token to the CTA's part of the list, which somebody emptied before the
  // last barrier; what is behind its end is counted only.
  __device__ __forceinline__ void add_to_list(int i, float v) const {
    const int at = atomicAdd(&s.list_n, 1);
    if (at < kList) s.mine[at] = key_of(v, first + i);
  }
  // The parts of all CTAs, of `counts` tokens, together in CTA 0: their number,
  // and the list if it has room for them.
  __device__ __forceinline__ int gather(const uint64_t (&counts)[kMaxCluster]) {
    int total = 0;
    for (int k = 0; k < ctas; ++k) total += (int)counts[k];
    if (rank != 0 || total > kList) return total;
    for (int i = threadIdx.x; i < total; i += kThreads) {
      int c = i, k = 0;
      while (c >= (int)counts[k]) c -= (int)counts[k++];
      const Shared *o = ctas == 1 ? &s : cg::this_cluster().map_shared_rank(&s, k);
      if (in_bounds(k, ctas, 43) && in_bounds(c, kList, 43)) s.list[i] = o->mine[c];
    }
    __syncthreads();
    return total;
  }
  // Sets the last token that stays to the one at which the kept tokens' count
  // (by_mass: their mass), in their order, first reaches `need`.  r: where it
  // is, from its top down to where weights are 0; kept tokens that are too few
  // to reach need all stay.
  __device__ __forceinline__ void cut(uint64_t need, bool by_mass, Range r) {
    auto inside = [&](int i, float v) { return r.has(v) && kept(i, v); };
    for (int round = 0; r.lo < r.hi; ++round) {
      // a histogram of the range; the bin that has the token is the next range
      r.set_bins(round);
      __syncthreads();
      for (int b = threadIdx.x; b < kBins; b += kThreads) s.hist.lo[b] = s.hist.hi[b] = 0;
      __syncthreads();
      auto count = [&](auto even, int i, float v) {
        if (!inside(i, v)) return;
        const int b = r.template bin_as<decltype(even)::value>(v);
        if (!in_bounds((uint32_t)b, kBins, 46)) return;
        if (by_mass) {
          const uint64_t x = w.fixed(v);
          const uint32_t lo = (uint32_t)x, old = atomicAdd(&s.hist.lo[b], lo);
          const uint32_t hi = (uint32_t)(x >> 32) + (old + lo < lo ? 1u : 0u);
          if (hi) atomicAdd(&s.hist.hi[b], hi);
        } else {
          atomicAdd(&s.hist.lo[b], 1u);
        }
      };
      if (r.shift < 0) each<2>([&](int i, float v) { count(std::true_type{}, i, v); });
      else each<2>([&](int i, float v) { count(std::false_type{}, i, v); });
      sync_row();
      // each CTA adds its part of all histograms
      // (kBins / ctas bins of all; always kPer values a thread, so that their
      // reads run at once: one after another they took 17000 cycles)
      constexpr int kPer = kBins / kThreads;
      const int log = __ffs(ctas) - 1, b0 = (rank * kThreads + threadIdx.x) * kPer >> log;
      auto value = [&](int q) {
        const Shared *o = cg::this_cluster().map_shared_rank(&s, q & (ctas - 1));
        return (uint64_t)o->hist.hi[b0 + (q >> log)] << 32 | o->hist.lo[b0 + (q >> log)];
      };
      uint64_t sum = 0;
#pragma unroll
      for (int q = 0; q < kPer; ++q) sum += value(q);
      uint64_t upto = warp_scan_of(sum, lane);
      if (lane == 31) s.warp_mass[warp] = upto;
      __syncthreads();
      const uint64_t v[1] = {cta_sum(s.warp_mass)};
      const auto part = publish(v);
      uint64_t all = 0;
      upto += r.above - sum;
      for (int k = 0; k < ctas; ++k) {
        if (k < rank) upto += part[0][k];
        all += part[0][k];
      }
      if (r.above + all < need) return;
      for (int k = 0; k < warp; ++k) upto += s.warp_mass[k];
      if (threadIdx.x == 0) s.found = -1, s.list_n = 0;
      __syncthreads();
      if (upto < need && need <= upto + sum) {  // one thread: its bins again
        for (int q = 0; q < kPer && upto < need;) {
          s.found = b0 + (q >> log), s.found_mass = upto;
          do upto += value(q); while (++q & (ctas - 1));
        }
      }
      __syncthreads();
      const uint64_t mine[2] = {(uint64_t)(s.found + 1), s.found >= 0 ? s.found_mass : 0};
      const auto found = publish(mine);
      uint64_t bin = 0, above = 0;
      for (int k = 0; k < ctas; ++k) bin += found[0][k], above += found[1][k];
      r.set_bin((int)bin - 1);
      r.above = above;
      if (order(need, by_mass, r)) return;
      // too many: from their largest to their smallest logit
      float lo = INFINITY, hi = -INFINITY;
      each<4>([&](int i, float v) {
        if (inside(i, v)) lo = fminf(lo, v), hi = fmaxf(hi, v);
      });
      extremes(lo, hi);
      r.lo = lo, r.hi = hi, r.bin = -1;
      r.top = nextafterf(hi, INFINITY);
    }
    // equal logits: by their indexes
    const float v = r.lo;
    uint64_t rest = need - r.above, all;
    if (by_mass) {
      const uint64_t x = w.fixed(v);
      rest = (rest + x - 1) / x;
    }
    const int at = find([&](int i, float y) -> uint64_t { return y == v && kept(i, y); },
                        [&](uint64_t) { return rest - 1; }, all);
    if (all < rest) return;
    __syncthreads();
    if (threadIdx.x == 0) s.found = 0;
    __syncthreads();
    if (at >= 0 && lane == 0) s.found = first + at + 1;  // in one warp of the row
    __syncthreads();
    const uint64_t found[1] = {(uint64_t)s.found};
    const auto slot = publish(found);
    last_v = v;
    last_i = -1;
    for (int k = 0; k < ctas; ++k) last_i += (int)slot[0][k];
  }

  // cut() for a range whose tokens fit the list (emptied before the last
  // barrier); false if they do not.
  __device__ __forceinline__ bool order(uint64_t need, bool by_mass, const Range &r) {
    each<4>([&](int i, float v) {
      if (r.has(v) && kept(i, v)) add_to_list(i, v);
    });
    __syncthreads();
    const uint64_t count[1] = {(uint64_t)s.list_n};
    const int len = gather(publish(count)[0]);
    uint64_t found[1] = {0};  // the token's key
    if (rank == 0 && len <= kList) {
      const float top = fminf(r.top, r.hi);
      find_in_list(s, len, top, __fdividef(kThreads, top - r.lo), index_shift, need - r.above, by_mass, w);
      found[0] = s.found_mass;
    }
    const auto slot = publish(found);
    if (!slot[0][0]) return false;
    last_v = logit_of(slot[0][0]);
    last_i = index_of(slot[0][0]);
    return true;
  }
};

// cut() apart from the code that most rows run.  The row goes by value, so that
// its caller's stays in registers.
struct Last {
  float v;
  int i, parity;
};
template <class T, bool RES> __device__ __noinline__ Last cut_row(Row<T, RES> r, uint64_t need, bool by_mass, Range range) {
  r.cut(need, by_mass, range);
  return Last{r.last_v, r.last_i, r.parity};
}

// A list of the first top_k tokens, which reach below `from`, has to begin
// lower: at the bin of a histogram of 8 temperatures below that has the k-th,
// and a little lower yet for its rounding.
template <class T, bool RES> __device__ __noinline__ float list_start(Row<T, RES> r, float from, int top_k, float temp) {
  const int tid = threadIdx.x;
  const float scale = __fdividef(kCountBins, 8.f * temp);
  r.template each<4>([&](int, float v) {
    const int b = (int)((from - v) * scale);
    if (b < kCountBins && in_bounds(max(0, b), kCountBins, 46)) atomicAdd(&r.s.count[max(0, b)], 1u);
  });
  if (tid == 0) r.s.found = -1;
  r.sync_row();
  // every CTA adds all histograms: two bins a thread
  uint2 mine = make_uint2(0, 0);
#pragma unroll
  for (int k = 0; k < kMaxCluster; ++k) {
    if (k >= r.ctas) break;
    const uint2 x = reinterpret_cast<const uint2 *>(cg::this_cluster().map_shared_rank(r.s.count, k))[tid];
    mine.x += x.x, mine.y += x.y;
  }
  int upto = warp_scan_of((int)(mine.x + mine.y), r.lane);
  if (r.lane == 31) r.s.warp_count[r.warp] = upto;
  __syncthreads();
  upto += (int)warp_sum_of(r.lane < r.warp ? r.s.warp_count[r.lane] : 0u);
  if (upto - (int)(mine.x + mine.y) < top_k && top_k <= upto) r.s.found = 2 * tid + (upto - (int)mine.y < top_k ? 1 : 0);
  __syncthreads();
  const int bin = r.s.found;
  return bin < 0 ? from : fmaxf(from - __fdividef(bin + 1.25f, scale), -FLT_MAX);
}

template <class T, bool RES>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const __grid_constant__ SampleParams p) {
  extern __shared__ float4 smem[];
  Shared &s = *reinterpret_cast<Shared *>(smem);
  cg::cluster_group cluster = cg::this_cluster();
  const int ctas = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  if (ctas > 1) cluster_arrive();
  const int row = blockIdx.x / ctas, tid = threadIdx.x;
  const int first = min(p.V, rank * p.len), n = min(p.V - first, p.len);
  if (tid < 16) s.pow16[tid] = exp2((double)tid / 16.) * 0x1p44;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  const T *src = reinterpret_cast<const T *>(p.logits) + (size_t)row * p.ld + first;
  float *l = reinterpret_cast<float *>(&s + 1);
  // the CTA's part lies in its row, and a logit's place in the shared copy
  auto inside = [&](int i, int many) {
    return in_bounds((size_t)i + many - 1, n, 40) && in_bounds((size_t)first + i + many - 1, p.V, 40) &&
           in_bounds((size_t)(l - reinterpret_cast<float *>(&s + 1)) + i + many - 1, p.len + 8, 41);
  };
  float hi = -INFINITY;
  if constexpr (RES) {
    // 16-byte loads from the first aligned address on; the shared copy is
    // shifted so that its stores are aligned too
    constexpr int kVec = 16 / sizeof(T);
    const int head = min(n, (int)((-(uintptr_t)src & 15) / sizeof(T)));
    l += -head & 3;
    auto put = [&](float v) {
      hi = fmaxf(hi, v);
      return v;
    };
    // every thread has a part in a row's maxima: of a short part it takes single logits
    const int vecs = n < kThreads * kVec ? 0 : (n - head) / kVec;
#pragma unroll 4
    for (int i = tid; i < vecs; i += kThreads) {
      if (!inside(head + i * kVec, kVec)) break;
      const uint4 q = __ldcs(reinterpret_cast<const uint4 *>(src + head) + i);
      float4 *dst = reinterpret_cast<float4 *>(l + head) + i * (kVec / 4);
      const uint32_t x[4] = {q.x, q.y, q.z, q.w};
      float f[kVec];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (sizeof(T) == 4) {
          f[j] = put(logit_of(__uint_as_float(x[j])));
        } else {
          f[2 * j] = put(logit_of(__uint_as_float(x[j] << 16)));
          f[2 * j + 1] = put(logit_of(__uint_as_float(x[j] & 0xffff0000u)));
        }
      }
#pragma unroll
      for (int j = 0; j < kVec; j += 4) dst[j / 4] = make_float4(f[j], f[j + 1], f[j + 2], f[j + 3]);
    }
    if (tid < head && inside(tid, 1)) l[tid] = put(logit_of(src[tid]));
#pragma unroll 4
    for (int i = head + vecs * kVec + tid; i < n; i += kThreads)
      if (inside(i, 1)) l[i] = put(logit_of(src[i]));
  }
  Row<T, RES> r{s, l, src, n, first, rank, ctas, tid >> 5, tid & 31};
  static_assert(kThreads == 512);
  r.index_shift = max(0, 32 - __clz(p.V - 1) - 9);
  if constexpr (!RES) r.template each<4>([&](int, float v) { hi = fmaxf(hi, v); });

  const float temp = p.temperature ? p.temperature[row] : 1.f;
  const int top_k = p.top_k ? p.top_k[row] : 0;
  const float top_p = p.top_p ? p.top_p[row] : 1.f, u = p.u[row], q = p.min_p ? p.min_p[row] : 0.f;
  const bool greedy = !(temp > 0.f), by_count = !greedy && top_k > 0 && top_k < p.V, by_mass = !greedy && top_p < 1.f;

  // The largest logits of kGroups parts of the row, in every CTA: `width` threads have one.
  const int width = kThreads / kGroups * ctas;
  for (int o = 1; o < width; o <<= 1) hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  if (ctas > 1) cluster_wait();  // all run: group_max is the first that goes to the others
  if (tid % width < ctas) {
    float *to = ctas == 1 ? s.group_max : cluster.map_shared_rank(s.group_max, tid % width);
    to[rank * (kGroups / ctas) + tid / width] = hi;
  }
  if (tid == 0) s.list_n = 0;
  s.count[tid] = s.count[tid + kThreads] = 0;
  r.sync_row();
  // k of them reach the k-th, so k tokens do, and seldom many more: a list from
  // there on has a top-k, and of most rows a top-p
  if (by_count || by_mass) {
    const int at = by_count ? min(top_k, kListAt) : kListMass;
    constexpr int kShare = kThreads / kGroups;  // neighbouring threads share a part's comparisons
    const int c = tid / kShare;
    const float x = s.group_max[c];
    int order = 0;
#pragma unroll
    for (int j = 0; j < kGroups / 4 / kShare; ++j) {
      const int at4 = (j * kShare + tid % kShare) * 4;
      const float4 y = *reinterpret_cast<const float4 *>(s.group_max + at4);
      order += (y.x > x) | ((y.x == x) & (at4 < c));
      order += (y.y > x) | ((y.y == x) & (at4 + 1 < c));
      order += (y.z > x) | ((y.z == x) & (at4 + 2 < c));
      order += (y.w > x) | ((y.w == x) & (at4 + 3 < c));
    }
#pragma unroll
    for (int o = 1; o < kShare; o <<= 1) order += __shfl_xor_sync(0xffffffffu, order, o);
    if (order == 0) s.m = x;
    if (order == at - 1) s.list_from = x;
    if (order == min(at, 8) - 1) s.list_top = x;
    __syncthreads();
    hi = s.m;
  } else {
#pragma unroll
    for (int j = 0; j < kGroups / 32; ++j) hi = fmaxf(hi, s.group_max[32 * j + r.lane]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  auto put_out = [&](int token, float prob) {
    if (!in_bounds(token + 1, p.V + 1, 47)) return;  // -1: nothing left
    p.token[row] = token;
    if (p.prob) p.prob[row] = prob;
  };
  if (hi == -INFINITY) {
    if (rank == 0 && tid == 0) put_out(-1, 0.f);
    return;
  }
  r.infinite = hi == INFINITY;
  if (r.infinite) {  // only those are left, all alike
    if constexpr (RES) {
      for (int i = tid; i < n; i += kThreads) l[i] = r.value(l[i]);
      __syncthreads();
    }
    hi = 0.f;
  }
  r.w = Weight{hi, fmaxf(__fmaf_rn(-40.f, temp, hi), -FLT_MAX), 16. / (0.69314718055994530942 * (double)temp), s.pow16};
  const double min_w = q > 0.f ? fmin((double)q, 1.) * 0x1p44 : 0.;
  auto target = [&](uint64_t all) -> uint64_t { return greedy ? 0 : target_of(u, all); };

  uint64_t all_mass = 0, list_mass = 0;  // of the row, and from list_from on
  float list_from = INFINITY;
  if (by_count || by_mass) {
    float from = p.V <= kAll || r.infinite ? -FLT_MAX : fmaxf(s.list_from, -FLT_MAX);
    if (by_count && top_k > kListAt && top_k <= kList && from > -FLT_MAX) from = list_start(r, from, top_k, temp);
    uint64_t sum[2] = {0, 0};
    if (by_count) {
      r.template each<4>([&](int i, float v) {
        if (v >= from) r.add_to_list(i, v);
      });
    } else {
      r.template each<2>([&](int i, float v) {
        sum[0] += r.w.fixed(v);
        if (v >= from) r.add_to_list(i, v);
      });
      sum[0] = warp_sum_of(sum[0]);
      if (r.lane == 0) s.warp_mass[r.warp] = sum[0];
    }
    __syncthreads();
    if (!by_count) sum[0] = r.cta_sum(s.warp_mass);
    sum[1] = (uint64_t)s.list_n;
    const auto slot = r.publish(sum);
    const int len = r.gather(slot[1]);
    for (int k = 0; k < ctas; ++k) all_mass += slot[0][k];
    // CTA 0 tells the others whether the list had the token
    uint64_t good[2] = {0, 0};
    if (rank == 0 && len <= kList) {
      // buckets down to the list's end; of a whole row to 40 temperatures, below which weights are 0
      const float top = r.infinite ? hi : s.list_top;
      const float scale = __fdividef(kThreads, from > -FLT_MAX ? top - from : 40.f * temp);
      good[0] = draw_from_list(s, p, row, ListTask{r.w, min_w, all_mass, top, scale, u, top_p, by_count ? top_k : 0, by_mass,
                                                   len, r.index_shift});
      good[1] = s.found_mass;
    }
    const auto told = r.publish(good);
    list_from = told[1][0] && !by_count ? from : INFINITY;
    list_mass = told[1][0];
    if (told[0][0]) return;
  }
  if (by_count || by_mass) {
    // the slow way: down to 32 temperatures below m, where weights are 0
    Range range;
    range.lo = fmaxf(__fmaf_rn(-32.f, temp, hi), -FLT_MAX);
    range.top = INFINITY;
    range.hi = hi;
    auto cut = [&](uint64_t need, bool mass) {
      const Last last = cut_row(r, need, mass, range);
      r.last_v = last.v, r.last_i = last.i, r.parity = last.parity;
    };
    if (by_count) {
      cut(top_k, false);
      if (by_mass) {
        uint64_t sum[1] = {0};
        r.template each<2>([&](int i, float v) {
          if (v >= r.last_v && r.kept(i, v)) sum[0] += r.w.fixed(v);
        });
        sum[0] = warp_sum_of(sum[0]);
        __syncthreads();
        if (r.lane == 0) s.warp_mass[r.warp] = sum[0];
        __syncthreads();
        sum[0] = r.cta_sum(s.warp_mass);
        const auto slot = r.publish(sum);
        all_mass = 0;
        for (int k = 0; k < ctas; ++k) all_mass += slot[0][k];
      }
    } else if (list_from < INFINITY) {  // below the list, whose mass is known
      range.top = range.hi = list_from;
      range.lo = fminf(range.lo, list_from);
      range.above = list_mass;
    }
    if (by_mass) cut(need_of(top_p, all_mass), true);
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
  if (at >= 0 && r.lane == 0) put_out(first + at, greedy ? 1.f : (float)(r.w(r.at(at)) / (double)Z));
}

template <class T, bool RES> int32_t launch_sample(const SampleParams &p, int32_t B, int ctas, size_t smem, cudaStream_t s) {
  auto k = sample_kernel<T, RES>;
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

template <class T> int32_t launch_sample(SampleParams p, int32_t B, cudaStream_t s) {
  // CTAs of a row: at most 16384 logits each where that is possible, and more
  // of them while SMs are left and a CTA keeps 2048 logits
  const int slots = 2 * num_sms();  // CTAs that run at once: 512 threads of 64 registers
  int ctas = 1;
  while (ctas < kMaxCluster && (ceil_div(p.V, ctas) > 16384 ||
                                ((int64_t)B * ctas * 2 <= slots && p.V / (2 * ctas) >= 2048)))
    ctas *= 2;
  auto part = [&] { return ceil_div(ceil_div(p.V, ctas), 8) * 8; };
  p.len = part();
  size_t smem = sizeof(Shared) + (size_t)(p.len + 8) * 4;
  const int64_t at_once = 2 * smem <= 226 * 1024 ? slots : slots / 2;
  if (B * (int64_t)ctas <= at_once) return launch_sample<T, true>(p, B, ctas, smem, s);
  // more than run at once: longer parts
  while (ctas > 1 && B * (int64_t)ctas > slots) ctas /= 2;
  p.len = part();
  smem = sizeof(Shared) + kWarps * kRing * kRingChunk;
  return launch_sample<T, false>(p, B, ctas, smem, s);
}

}  // namespace

NSLM_BOUNDS_ACCESSOR(sample)

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
