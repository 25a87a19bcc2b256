// q4.cu -- nslm_q4_gemv: the decode matrix-vector product from 4-bit weights
// with a scale (and an offset) for each group along K.
#include <algorithm>

#include <cuda_bf16.h>

#include "common.cuh"

namespace nslm {
namespace {

constexpr int kMaxVec = 8;
constexpr int kMaxMK = 65536;  // bf16 activations of one call that stay in shared memory

__device__ __forceinline__ float bf16_f32(uint32_t h) { return __uint_as_float(h << 16); }

// A tile is 16 rows, a stage 256 weights of each, with their scales and offsets.
// kw warps of a CTA share a tile, each with a range of its stages, and add their
// sums in shared memory at its end; a CTA has WARPS / kw tiles at a time and
// walks over the rows.  Stages come by cp.async into a ring of each warp's own,
// which runs ahead across tiles, so no load waits for the sums or the barrier.
// (Loads into registers would: those in flight share a few counters with the
// shared-memory loads of the products, which then wait for them.)
//
// The product runs on mma.sync m16n8k16 with the weights as A (q - 8, exact in
// bf16, straight from the packed words to the fragment's registers) and the
// vectors as B: with at most 8 vectors the tensor cores' 128-row form would
// spend its time on building operands, and a CUDA-core product would be bound
// by its fp32 multiply-adds from two vectors on.  A word holds weights 0..7 of
// a row; the pairs (0,4), (1,5), (2,6), (3,7) are what a mask takes out of it
// at once, so these are the fragment's pairs, and the staged activations are in
// the same order.  Each group gets an accumulator of its own, multiplied by the
// scale in fp32; products are exact, so nothing of a weight is rounded.  The
// rest of an affine weight, (b + 8 s) times the group's sum of x, is a product
// over the groups, [b s] times [x's sum, 8 times that], with b and s as they are
// stored (bf16) and the sums in three bf16 parts (24 bits): 3 mma a stage.
//
// 131072 x 4096 with groups of 64 takes 64 to 66 us with one vector and 68 to 76
// with 8 in bursts of 100 calls, 72 and 75 to 80 in runs of thousands (306 MB: 47
// at the copy rate); 50257 x 2048 15.5 (8.8).  Copies alone take 48 to 55 us of
// the first, computing alone 52 to 62 (the unpacking's shifts and masks on the
// ALU pipe), and they overlap but for the rest.  512 x 1024 takes 2 us, a launch
// and a load.

constexpr int kTile = 16;
constexpr int kStageK = 256;             // weights of a row in a stage
constexpr int kRow = kStageK / 2;        // and their bytes
constexpr int kStage = kTile * kRow;
constexpr int kZero = 8 * 4 * 16 * 4;    // bytes of zeros that lanes without a vector read in a stage

struct Q4Params {
  nslm_q4_matrix W;
  const uint16_t *x;
  float *y;
  int32_t M, NG, NS;  // NG, NS: groups and stages of a row
  int32_t kw;       // warps that share a tile
  int32_t steps;    // tiles / (WARPS / kw), rounded up
  int32_t spc;      // stages whose scales are copied at once
  bool ready;
};

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_bf16_k8(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t b0) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5}, {%6}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(b0));
}

// The bf16 pair (w_i - 8, w_{i+4} - 8) of a word: 0x4300 | q is 128 + q.
template <int I>
__device__ __forceinline__ uint32_t pair_of(uint32_t v) {
  uint32_t p, r;
  asm("lop3.b32 %0, %1, 0x000f000f, %2, 0xea;" : "=r"(p) : "r"(v >> (4 * I)), "r"(0x43004300u));
  asm("sub.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(p), "r"(0x43084308u));
  return r;
}

__device__ __forceinline__ uint32_t smem_addr(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ uint4 lds128(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}
template <int WORDS>
__device__ __forceinline__ void lds_words(uint32_t (&a)[WORDS], uint32_t at) {
  if constexpr (WORDS == 1) asm volatile("ld.shared.u32 %0, [%1];" : "=r"(a[0]) : "r"(at) : "memory");
  if constexpr (WORDS == 2) asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(a[0]), "=r"(a[1]) : "r"(at) : "memory");
  if constexpr (WORDS == 4)
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void copy16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// 4, 8 or 16 bytes.
template <int BYTES> __device__ __forceinline__ void copy(uint32_t dst, const void *src) {
  if constexpr (BYTES == 16) copy16(dst, src);
  else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES) : "memory");
}

template <int G> constexpr int kGroups = kStageK / G;             // of a stage: 8, 4 or 2
// Scales are copied 8 groups (16 bytes) of a row at once where whole rows and
// the warps' ranges allow it and there are rows enough for it to matter: each
// row's piece is a transaction of its own, whatever its size.  (Groups of 64 by
// 8-byte copies: 80 us at 131072 x 4096 and 8 vectors, by 16-byte ones 66.)
constexpr int kScaleRow = 16;
constexpr int kScales = kTile * kScaleRow;
template <bool AFFINE> constexpr int kSlot = kStage + kScales * (AFFINE ? 2 : 1);
// A stage's entries of sums of x: [sums, 8 times those] and zeros up to 8 at least.
template <int G> constexpr int kSums = G == 32 ? 16 : 8;

// MP: vectors in shared memory, M rounded up to 1, 2, 4 or 8 (zeros behind the last).
template <int G, int MP, int WARPS, int STAGES, bool AFFINE>
__global__ void __launch_bounds__(WARPS * 32, WARPS == 8 ? 2 : 1) q4_gemv_kernel(const Q4Params p) {
  constexpr int kWords = G / 32;       // words of a row and group for each of 4 lanes
  constexpr int kGps = kGroups<G>, kChunk = kScales * (AFFINE ? 2 : 1);
  // The 16-byte chunks of a stage's row change places by the row, so that the
  // rows that one phase of a shared-memory load reads lie in different banks.
  constexpr int kFlip = G / 2;         // in units of a group's bytes
  constexpr int kFlips = kRow / kFlip; // 8, 4 or 2
  extern __shared__ __align__(128) uint4 smem[];
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int M = p.M, K = p.W.K, N = p.W.N, NG = p.NG, NS = p.NS;
  uint4 *xs = smem + kZero / 16;  // [K / 32][MP][4], behind the zeros
  uint16_t *sx = reinterpret_cast<uint16_t *>(xs + (size_t)MP * K / 8);  // [3][MP][sx_row]
  const int sx_row = NS * kSums<G> + 8;
  // on 128 bytes: copies write whole sectors
  uint8_t *rings = reinterpret_cast<uint8_t *>(sx) + (AFFINE ? (6 * MP * sx_row + 127) & ~127 : 0);
  float *red = reinterpret_cast<float *>(rings + WARPS * STAGES * kSlot<AFFINE>);  // [2][WARPS][8][16]
  const uint32_t ring = smem_addr(rings) + warp * STAGES * kSlot<AFFINE>;

  const int sub = warp / p.kw, kp = warp - sub * p.kw, tps = WARPS / p.kw;
  // this warp's stages of a tile
  const int units = (NS + p.spc - 1) / p.spc, st0 = kp * units / p.kw * p.spc;
  const int nst = min(NS, (kp + 1) * units / p.kw * p.spc) - st0;
  const bool whole = K % kStageK == 0;  // every stage is, and its scales lie in aligned words
  const int last = p.spc - 1;           // spc is a power of two

  // the load side: which stage comes next, its two row pointers, and the
  // scales (lanes 0 to 15) or offsets (16 to 31) of one row
  const int first = sub < tps ? (int)blockIdx.x : p.steps;  // warps that are left over have no tile
  int l_step = first, l_st = 0, l_left = 0, l_group = 0;
  uint32_t l_slot = 0, l_chunk = 0;  // the next stage's place, and the next scales'
  const uint8_t *src0 = nullptr, *src1 = nullptr;
  const uint16_t *src2 = nullptr;
  auto rows_of = [&]() {
    const int row = (l_step * tps + sub) * kTile;
    const size_t pitch = (size_t)K / 2;
    const uint8_t *base = reinterpret_cast<const uint8_t *>(p.W.q) + (size_t)st0 * kRow + t * 16;
    src0 = base + (size_t)min(row + g, N - 1) * pitch;
    src1 = base + (size_t)min(row + g + 8, N - 1) * pitch;
    src2 = (AFFINE && lane >= 16 ? p.W.biases : p.W.scales) + (size_t)min(row + lane % 16, N - 1) * NG + st0 * kGps;
    l_group = st0 * kGps;
    l_left = K - st0 * kStageK - t * 32;
    l_st = nst;
  };
  // chunks t and t + 4 of rows g and g + 8 are this lane's to copy
  const uint32_t dst0 = ring + g * kRow + ((t * 16) ^ ((g % kFlips) * kFlip));
  const uint32_t dst1 = ring + g * kRow + ((t * 16 + 64) ^ ((g % kFlips) * kFlip));
  const uint32_t scales = ring + STAGES * kStage;
  const uint32_t dst2 = scales + (lane / 16) * kScales + (lane % 16) * kScaleRow;
  if (l_step < p.steps) rows_of();
  const auto weights = [&](uint32_t dst, const uint8_t *src) {
    if (in_buffer(src, 16, p.W.q, (size_t)N * K / 2, 20) && in_bounds(dst - ring + 15, STAGES * kStage, 22)) copy16(dst, src);
  };
  auto load_stage = [&]() {
    if (l_st > 0) {
      if (l_left > 0) {
        weights(dst0 + l_slot, src0);
        weights(dst0 + l_slot + 8 * kRow, src1);
      }
      if (l_left > 128) {
        weights(dst1 + l_slot, src0 + 64);
        weights(dst1 + l_slot + 8 * kRow, src1 + 64);
      }
      if (((nst - l_st) & last) == 0) {
        const int bytes = 2 * (last ? 8 : min(kGps, NG - l_group));  // of the row's scales
        if ((AFFINE || lane < 16) &&
            in_buffer(src2, bytes, AFFINE && lane >= 16 ? p.W.biases : p.W.scales, (size_t)N * NG * 2, 21) &&
            in_bounds(dst2 + l_chunk - scales + kScaleRow - 1, STAGES * kChunk, 22)) {
          if (last) {
            copy16(dst2 + l_chunk, src2);
          } else if (whole) {
            copy<kGps * 2>(dst2 + l_chunk, src2);
          } else {  // what is behind the row counts as 0
#pragma unroll
            for (int j = 0; j < kGps; ++j) {
              const uint16_t v = l_group + j < NG ? __ldg(src2 + j) : 0;
              asm volatile("st.shared.u16 [%0], %1;" ::"r"(dst2 + l_chunk + 2 * j), "h"(v) : "memory");
            }
          }
        }
        l_chunk = l_chunk == (STAGES - 1) * kChunk ? 0 : l_chunk + kChunk;
      }
      src0 += kRow, src1 += kRow, src2 += kGps;
      l_group += kGps;
      l_left -= kStageK;
      l_slot = l_slot == (STAGES - 1) * kStage ? 0 : l_slot + kStage;
      if (--l_st == 0) {
        l_step += gridDim.x;
        if (l_step < p.steps) rows_of();
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  auto prologue = [&]() {
    for (int i = 0; i < STAGES - 1; ++i) load_stage();
  };

  if (p.ready) prologue();
  for (int i = tid; i < kZero / 16; i += WARPS * 32) smem[i] = make_uint4(0, 0, 0, 0);
  if (AFFINE) {
    for (int i = tid; i < 3 * MP * sx_row / 2; i += WARPS * 32) reinterpret_cast<uint32_t *>(sx)[i] = 0;
    __syncthreads();
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (!p.ready) prologue();

  // activations: word wi of a group is what lane wi / kWords multiplies in step wi % kWords
  for (int m = 0; m < MP; ++m)
  for (int w = tid; w < K / 8; w += WARPS * 32) {
    const int gi = w / (G / 8), wi = w % (G / 8);
    const uint4 v = m < M && in_bounds((size_t)m * (K / 8) + w, (size_t)M * K / 8, 23)
                        ? __ldg(reinterpret_cast<const uint4 *>(p.x) + (size_t)m * (K / 8) + w)
                        : make_uint4(0, 0, 0, 0);
    const uint4 q = make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632),
                               __byte_perm(v.y, v.w, 0x5410), __byte_perm(v.y, v.w, 0x7632));
    const size_t place = ((size_t)(gi * kWords + wi % kWords) * MP + m) * 4 + wi / kWords;
    if (in_bounds(place, (size_t)MP * K / 8, 24)) xs[place] = q;
    if (AFFINE) {
      float s = 0.f;
      const uint32_t h[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) s += bf16_f32(h[j] & 0xffffu) + __uint_as_float(h[j] & 0xffff0000u);
      // G / 8 neighbouring lanes hold a group; groups do not straddle the end
      const int left = K / 8 - (w - lane);
      const uint32_t mask = left >= 32 ? 0xffffffffu : (1u << left) - 1;
#pragma unroll
      for (int o = 1; o < G / 8; o <<= 1) s += __shfl_xor_sync(mask, s, o);
      if (wi == 0) {
        uint16_t *at = sx + m * sx_row + gi / kGps * kSums<G> + gi % kGps;
#pragma unroll
        for (int j = 0; j < 3; ++j) {
          if (!in_bounds((size_t)(at - sx) + j * MP * sx_row + kGps, (size_t)3 * MP * sx_row, 25)) break;
          const __nv_bfloat16 b = __float2bfloat16_rn(s);
          at[j * MP * sx_row] = __bfloat16_as_ushort(b);
          at[j * MP * sx_row + kGps] = __bfloat16_as_ushort(__float2bfloat16_rn(8.f * __bfloat162float(b)));
          s -= __bfloat162float(b);
        }
      }
    }
  }
  __syncthreads();

  // lanes of columns without a vector read the zeros and stay there
  const uint32_t xb = smem_addr(smem) + (g < MP ? kZero + ((st0 * (kStageK / 32) * MP + g) * 4 + t) * 16 : 0);
  const uint32_t x_stage = g < MP ? kGps * kWords * MP * 64 : 0;
  const uint32_t sb = smem_addr(sx) + (g < MP ? (g * sx_row + st0 * kSums<G> + 2 * t) * 2 : 0);
  auto in_sums = [&](uint32_t at) { return in_bounds(at - smem_addr(sx) + 3, (size_t)6 * MP * sx_row, 25); };
  // where the lane's pair of [b s] of row g stands
  const uint32_t co = scales + g * kScaleRow +
                      (kGps == 8 || t < kGps / 2 ? kScales + t * 4 : (t - kGps / 2) * 4);
  const uint32_t a_lane = ring + g * kRow + t * 4 * kWords;
  const uint32_t flip = (g % kFlips) * kFlip;
  const uint32_t s_lane = scales + g * kScaleRow;

  uint32_t slot = 0, chunk = 0;
  int buf = 0;
  for (int step = first; step < p.steps; step += gridDim.x, buf ^= 1) {
    float acc[4] = {}, c_co[4] = {};
    uint32_t xp = xb;
    for (int st = 0; st < nst; ++st) {
      asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 2) : "memory");
      __syncwarp();
      load_stage();
      const uint32_t rp = a_lane + slot, in = chunk + (st & last) * (kGps * 2), sp = s_lane + in;
      uint32_t s0w[kGps / 2], s1w[kGps / 2];  // scales of rows g and g + 8
      lds_words<kGps / 2>(s0w, sp);
      lds_words<kGps / 2>(s1w, sp + 8 * kScaleRow);
      if (AFFINE) {
        const uint32_t at = co + in;
        uint32_t a0 = 0, a1 = 0;
        if (t < kGps) a0 = lds32(at), a1 = lds32(at + 8 * kScaleRow);
        if constexpr (kGps == 8) {
          const uint32_t a2 = lds32(at - kScales), a3 = lds32(at - kScales + 8 * kScaleRow);
#pragma unroll
          for (int j = 0; j < 3; ++j) {
            const uint32_t from = sb + (j * MP * sx_row + st * kSums<G>) * 2;
            uint32_t b0 = 0, b1 = 0;
            if (g < MP && in_sums(from + 16)) b0 = lds32(from), b1 = lds32(from + 16);
            mma_bf16(c_co, a0, a1, a2, a3, b0, b1);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 3; ++j) {
            const uint32_t from = sb + (j * MP * sx_row + st * kSums<G>) * 2;
            uint32_t b0 = 0;
            if (g < MP && in_sums(from)) b0 = lds32(from);
            mma_bf16_k8(c_co, a0, a1, b0);
          }
        }
      }
      slot = slot == (STAGES - 1) * kStage ? 0 : slot + kStage;
      if ((st & last) == last || st + 1 == nst) chunk = chunk == (STAGES - 1) * kChunk ? 0 : chunk + kChunk;
      auto group = [&](int gi) {
        uint32_t a0[kWords], a1[kWords];
        lds_words<kWords>(a0, rp + (flip ^ (gi * kFlip)));
        lds_words<kWords>(a1, rp + (flip ^ (gi * kFlip)) + 8 * kRow);
        float c[4] = {};
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
          const uint32_t from = xp + (gi * kWords + i) * MP * 64;
          const bool staged = in_bounds(from - smem_addr(smem) + 15, kZero + (size_t)2 * MP * K, 24);
          const uint4 b = staged ? lds128(from) : make_uint4(0, 0, 0, 0);
          mma_bf16(c, pair_of<0>(a0[i]), pair_of<0>(a1[i]), pair_of<1>(a0[i]), pair_of<1>(a1[i]), b.x, b.y);
          mma_bf16(c, pair_of<2>(a0[i]), pair_of<2>(a1[i]), pair_of<3>(a0[i]), pair_of<3>(a1[i]), b.z, b.w);
        }
        const float s0 = __uint_as_float(gi & 1 ? s0w[gi / 2] & 0xffff0000u : s0w[gi / 2] << 16);
        const float s1 = __uint_as_float(gi & 1 ? s1w[gi / 2] & 0xffff0000u : s1w[gi / 2] << 16);
        acc[0] = fmaf(s0, c[0], acc[0]);
        acc[1] = fmaf(s0, c[1], acc[1]);
        acc[2] = fmaf(s1, c[2], acc[2]);
        acc[3] = fmaf(s1, c[3], acc[3]);
      };
      const int ngs = NG - (st0 + st) * kGps;
      if (ngs >= kGps) {
#pragma unroll
        for (int gi = 0; gi < kGps; ++gi) group(gi);
      } else {  // the end of the row
#pragma unroll
        for (int gi = 0; gi < kGps - 1; ++gi)
          if (gi < ngs) group(gi);
      }
      xp += x_stage;
    }
    // sums over the tile's warps; only these wait for one another
    float *rb = red + (buf * WARPS + sub * p.kw) * kMaxVec * kTile;
    float *rw = rb + kp * kMaxVec * kTile + g;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int m = 2 * t + (r & 1);
      if (m < MP) rw[m * kTile + 8 * (r >> 1)] = acc[r] + (AFFINE ? c_co[r] : 0.f);
    }
    if (p.kw == 1) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(1 + sub), "r"(p.kw * 32) : "memory");
    for (int i = kp * 32 + lane; i < MP * kTile; i += p.kw * 32) {
      const int m = i / kTile, row = (step * tps + sub) * kTile + i % kTile;
      if (m >= M || row >= N || !in_bounds((size_t)m * N + row, (size_t)M * N, 26)) continue;
      float s = 0.f;
      for (int k = 0; k < p.kw; ++k) s += rb[k * kMaxVec * kTile + i];
      p.y[(size_t)m * N + row] = s;
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

int32_t check_q4(const nslm_q4_matrix *W) {
  if (!W) return NSLM_ERR_ARG;
  if (W->group != 32 && W->group != 64 && W->group != 128) return NSLM_ERR_SHAPE;
  if (W->N < 0 || W->N > (1 << 30) || W->K <= 0 || W->K % W->group != 0) return NSLM_ERR_SHAPE;
  if (W->N > 0) {
    if (!W->q || !W->scales) return NSLM_ERR_ARG;
    if (!aligned16(W->q) || !aligned16(W->scales) || !aligned16(W->biases)) return NSLM_ERR_ALIGN;
  }
  return NSLM_OK;
}

constexpr size_t kSmemPerSm = 228 * 1024, kSmemReserved = 1024;  // of an SM, and of that for each CTA

template <int G, bool AFFINE> constexpr size_t q4_smem(int mp, int K, int warps, int stages) {
  const int NS = (K + kStageK - 1) / kStageK;
  return kZero + (size_t)2 * mp * K + (AFFINE ? ((size_t)6 * mp * (NS * kSums<G> + 8) + 127) / 128 * 128 : 0) +
         (size_t)warps * stages * kSlot<AFFINE> + (size_t)2 * warps * kMaxVec * kTile * 4;
}

// Splits the work for CTAs of `warps` and gives their shared memory.
template <int G, bool AFFINE> size_t q4_plan(Q4Params &p, int mp, int warps, int stages) {
  // the split of K with the least rounds of work: stages of a warp, and what a
  // tile costs besides (sums, barrier), about one of them
  const int tiles = ceil_div(p.W.N, kTile), ctas = num_sms() * (warps == 8 ? 2 : 1);
  // scales 16 bytes at once if there is a tile for every warp
  p.spc = p.W.K % (8 * p.W.group) == 0 && tiles >= ctas * warps ? 8 / kGroups<G> : 1;
  const int units = ceil_div(p.NS, p.spc);
  int64_t best = INT64_MAX;
  for (int kw = warps; kw >= 1; --kw) {
    if (kw > units) continue;
    const int64_t rounds = ceil_div(ceil_div(tiles, warps / kw), ctas);
    const int64_t cost = rounds * (ceil_div(units, kw) * p.spc + 1);
    if (cost < best) best = cost, p.kw = kw;
  }
  p.steps = ceil_div(tiles, warps / p.kw);
  return q4_smem<G, AFFINE>(mp, p.W.K, warps, stages);
}

template <int G, int MP, int WARPS, int STAGES, bool AFFINE>
int32_t launch_q4_as(const Q4Params &p, size_t smem, cudaStream_t s) {
  auto k = q4_gemv_kernel<G, MP, WARPS, STAGES, AFFINE>;
  if (int32_t st = ensure_smem((const void *)k, smem)) return st;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)std::min(p.steps, num_sms() * (WARPS == 8 ? 2 : 1)));
  cfg.blockDim = dim3(WARPS * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (int32_t st = cuda_status(cudaLaunchKernelEx(&cfg, k, p))) return st;
  return launch_status();
}

// Two CTAs of 8 warps on an SM where the activations leave room for both, else
// one of 16, or of 14 with a shorter ring for the longest rows; of 12 where not
// even those fit, which is groups of 32 with offsets (their sums take 24 KB).
template <int G, int MP, bool AFFINE>
int32_t launch_q4(Q4Params p, cudaStream_t s) {
  size_t smem = q4_plan<G, AFFINE>(p, MP, 8, 4);
  if (2 * (smem + kSmemReserved) <= kSmemPerSm) return launch_q4_as<G, MP, 8, 4, AFFINE>(p, smem, s);
  smem = q4_plan<G, AFFINE>(p, MP, 8, 3);
  if (2 * (smem + kSmemReserved) <= kSmemPerSm) return launch_q4_as<G, MP, 8, 3, AFFINE>(p, smem, s);
  smem = q4_plan<G, AFFINE>(p, MP, 16, 3);
  if (smem + kSmemReserved <= kSmemPerSm) return launch_q4_as<G, MP, 16, 3, AFFINE>(p, smem, s);
  smem = q4_plan<G, AFFINE>(p, MP, 14, 2);
  constexpr bool kFits = q4_smem<G, AFFINE>(MP, kMaxMK / MP, 14, 2) + kSmemReserved <= kSmemPerSm;
  if constexpr (!kFits) {
    static_assert(q4_smem<G, AFFINE>(MP, kMaxMK / MP, 12, 2) + kSmemReserved <= kSmemPerSm);
    if (smem + kSmemReserved > kSmemPerSm) {
      smem = q4_plan<G, AFFINE>(p, MP, 12, 2);
      return launch_q4_as<G, MP, 12, 2, AFFINE>(p, smem, s);
    }
  }
  return launch_q4_as<G, MP, 14, 2, AFFINE>(p, smem, s);
}

template <int G, int MP>
int32_t launch_q4(const Q4Params &p, cudaStream_t s) {
  return p.W.biases ? launch_q4<G, MP, true>(p, s) : launch_q4<G, MP, false>(p, s);
}

template <int G>
int32_t launch_q4(const Q4Params &p, cudaStream_t s) {
  return p.M == 1   ? launch_q4<G, 1>(p, s)
         : p.M == 2 ? launch_q4<G, 2>(p, s)
         : p.M <= 4 ? launch_q4<G, 4>(p, s)
                    : launch_q4<G, 8>(p, s);
}

}  // namespace

NSLM_BOUNDS_ACCESSOR(q4)

}  // namespace nslm

using namespace nslm;

extern "C" int32_t nslm_q4_gemv(const nslm_q4_matrix *W, const uint16_t *x_bf16, int32_t M, float *y,
                                uint32_t flags, nslm_stream_t stream) {
  g_launches = 0;
  if (flags & ~(uint32_t)NSLM_GEMV_FIELDS_READY) return NSLM_ERR_ARG;
  int32_t st = check_q4(W);
  if (st) return st;
  if (!x_bf16 || !y) return NSLM_ERR_ARG;
  if (M < 1 || M > kMaxVec || (int64_t)(M <= 2 ? M : M <= 4 ? 4 : 8) * W->K > kMaxMK) return NSLM_ERR_SHAPE;
  if (!aligned16(x_bf16) || !aligned16(y)) return NSLM_ERR_ALIGN;
  if ((st = check_device())) return st;
  if (W->N == 0) return NSLM_OK;
  Q4Params p{*W, x_bf16, y, M, W->K / W->group, ceil_div(W->K, kStageK), 1, 0, 1, (flags & NSLM_GEMV_FIELDS_READY) != 0};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  st = W->group == 32 ? launch_q4<32>(p, s) : W->group == 64 ? launch_q4<64>(p, s) : launch_q4<128>(p, s);
  if (st == NSLM_OK) g_launches = 1;
  return st;
}
