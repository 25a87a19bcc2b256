// q4.cu -- nslm_q4_gemv: the decode matrix-vector product from 4-bit weights
// with a scale (and an offset) for each group along K.
#include <algorithm>

#include "common.cuh"

namespace nslm {
namespace {

constexpr int kMaxVec = 8;
constexpr int kMaxMK = 65536;  // bf16 activations of one call that stay in shared memory

__device__ __forceinline__ float bf16_f32(uint32_t h) { return __uint_as_float(h << 16); }

// One warp per row; a lane takes every 32nd word of 8 weights.
template <int M>
__global__ void __launch_bounds__(256) q4_gemv_kernel(const nslm_q4_matrix W, const uint16_t *__restrict__ x,
                                                      float *__restrict__ y) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const int row = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (row >= W.N) return;
  const int nw = W.K / 8, ng = W.K / W.group;
  float acc[M] = {};
  for (int j = lane; j < nw; j += 32) {
    const uint32_t v = W.q[(size_t)row * nw + j];
    const int g = 8 * j / W.group;
    const float s = bf16_f32(W.scales[(size_t)row * ng + g]);
    const float b = W.biases ? bf16_f32(W.biases[(size_t)row * ng + g]) : -8.f * s;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float w = fmaf(s, (float)((v >> (4 * i)) & 15u), b);
#pragma unroll
      for (int m = 0; m < M; ++m) acc[m] = fmaf(w, bf16_f32(x[(size_t)m * W.K + 8 * j + i]), acc[m]);
    }
  }
#pragma unroll
  for (int m = 0; m < M; ++m) {
    for (int o = 16; o > 0; o >>= 1) acc[m] += __shfl_xor_sync(0xffffffffu, acc[m], o);
    if (lane == 0) y[(size_t)m * W.N + row] = acc[m];
  }
}

int32_t check_q4(const nslm_q4_matrix *W) {
  if (!W) return NSLM_ERR_ARG;
  if (W->group != 32 && W->group != 64 && W->group != 128) return NSLM_ERR_SHAPE;
  if (W->N < 0 || W->K <= 0 || W->K % W->group != 0) return NSLM_ERR_SHAPE;
  if (W->N > 0) {
    if (!W->q || !W->scales) return NSLM_ERR_ARG;
    if (!aligned16(W->q) || !aligned16(W->scales) || !aligned16(W->biases)) return NSLM_ERR_ALIGN;
  }
  return NSLM_OK;
}

}  // namespace
}  // namespace nslm

using namespace nslm;

extern "C" int32_t nslm_q4_gemv(const nslm_q4_matrix *W, const uint16_t *x_bf16, int32_t M, float *y,
                                uint32_t flags, nslm_stream_t stream) {
  g_launches = 0;
  if (flags & ~(uint32_t)NSLM_GEMV_FIELDS_READY) return NSLM_ERR_ARG;
  int32_t st = check_q4(W);
  if (st) return st;
  if (!x_bf16 || !y) return NSLM_ERR_ARG;
  if (M < 1 || M > kMaxVec || (int64_t)M * W->K > kMaxMK) return NSLM_ERR_SHAPE;
  if (!aligned16(x_bf16) || !aligned16(y)) return NSLM_ERR_ALIGN;
  if ((st = check_device())) return st;
  if (W->N == 0) return NSLM_OK;
  void (*const kernels[])(nslm_q4_matrix, const uint16_t *, float *) = {
      q4_gemv_kernel<1>, q4_gemv_kernel<2>, q4_gemv_kernel<3>, q4_gemv_kernel<4>,
      q4_gemv_kernel<5>, q4_gemv_kernel<6>, q4_gemv_kernel<7>, q4_gemv_kernel<8>};
  kernels[M - 1]<<<(W->N + 7) / 8, 256, 0, reinterpret_cast<cudaStream_t>(stream)>>>(*W, x_bf16, y);
  st = launch_status();
  if (st == NSLM_OK) g_launches = 1;
  return st;
}
