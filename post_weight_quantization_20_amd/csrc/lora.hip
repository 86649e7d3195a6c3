// Low-rank adapters of many requests beside a shared projection.
//
// Row i of x names adapter a = index[i]:  y_i = base_i + s_a B_a (A_a x_i),  A_a [r x d], B_a [rows x r];
// a row that names none takes base_i. Two steps: T = x A^T (shrink_kernel) and y = base + s T B^T
// (expand_kernel). T and all sums are fp32; nothing is rounded to fewer bits.
#include "common.hpp"

namespace gptq {
namespace {

struct LoraArgs {
  const void* x;
  int64_t ldx;
  int64_t m, d, rows;
  const void *A, *B;
  int dtype;
  int64_t adapters;
  int rank;
  const int32_t *ranks, *index;
  const float* scales;
  const float* base;
  int64_t ldb;
  float* y;
  int64_t ldy;
  float* T;      // m x rank
};

GPTQ_DEV int rank_of(const LoraArgs& a, int64_t ad) {
  if (!a.ranks) return a.rank;
  const int r = a.ranks[ad];
  return r < 0 ? 0 : r > a.rank ? a.rank : r;
}

// One wave per (row, rank): the dot product of x_i and row k of A_a.
__global__ __launch_bounds__(256) void shrink_kernel(LoraArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t items = a.m * a.rank;
  for (int64_t it = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); it < items; it += (int64_t)gridDim.x * 4) {
    const int64_t i = it / a.rank;
    const int k = (int)(it - i * a.rank);
    const int64_t ad = a.index[i];
    if (ad < 0 || ad >= a.adapters || k >= rank_of(a, ad)) continue;
    const int64_t xo = i * a.ldx, ao = (ad * a.rank + k) * a.d;
    float s = 0.f;
    for (int64_t c = lane; c < a.d; c += 64)
      s = __builtin_fmaf(load_as_f32(a.x, a.dtype, xo + c), load_as_f32(a.A, a.dtype, ao + c), s);
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o, 64);
    if (lane == 0) a.T[it] = s;
  }
}

__global__ __launch_bounds__(256) void expand_kernel(LoraArgs a) {
  const int64_t total = a.m * a.rows;
  for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < total; e += (int64_t)gridDim.x * 256) {
    const int64_t i = e / a.rows, j = e - i * a.rows;
    const int64_t ad = a.index[i];
    float v = a.base ? a.base[i * a.ldb + j] : 0.f;
    if (ad >= 0 && ad < a.adapters) {
      const int r = rank_of(a, ad);
      const int64_t bo = (ad * a.rows + j) * a.rank;
      float s = 0.f;
      for (int k = 0; k < r; ++k) s = __builtin_fmaf(a.T[i * a.rank + k], load_as_f32(a.B, a.dtype, bo + k), s);
      if (r) v += (a.scales ? a.scales[ad] : 1.0f) * s;
    }
    a.y[i * a.ldy + j] = v;
  }
}

}  // namespace

size_t lora_workspace_bytes(int64_t m, int64_t, int64_t, int64_t, int32_t rank) { return (size_t)m * rank * 4; }

hipError_t lora_gemm(const void* x, int dtype, int64_t m, int64_t ldx, const void* A, const void* B,
                     const int32_t* ranks, const float* scales, int64_t adapters, int32_t rank, const int32_t* index,
                     int64_t rows, int64_t d, const float* base, int64_t ld_base, float* y, int64_t ldy, void* work,
                     hipStream_t s) {
  LoraArgs a{};
  a.x = x; a.ldx = ldx; a.m = m; a.d = d; a.rows = rows;
  a.A = A; a.B = B; a.dtype = dtype; a.adapters = adapters; a.rank = rank;
  a.ranks = ranks; a.index = index; a.scales = scales;
  a.base = base; a.ldb = ld_base; a.y = y; a.ldy = ldy;
  a.T = static_cast<float*>(work);
  hipLaunchKernelGGL(shrink_kernel, dim3((unsigned)std::min<int64_t>((m * rank + 3) / 4, 65536)), dim3(256), 0, s, a);
  hipLaunchKernelGGL(expand_kernel, dim3((unsigned)std::min<int64_t>((m * rows + 255) / 256, 65536)), dim3(256), 0, s,
                     a);
  return hipGetLastError();
}

}  // namespace gptq
