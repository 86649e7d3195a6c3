// y[i, r] = sx[i] sw[r] sum_k x[i, k] (w[r, k] - z[r]) for int8 rows x and 8-bit weights w.
//
// Signed weights (z absent) go to the matrix cores as they are. Unsigned codes c of a stored layer become signed
// by flipping their top bit, c - 128, and sum x (c - z) = sum x (c - 128) + (128 - z) sum x: the rows' sums are
// formed beside the product. All sums are exact whole numbers in 32 bits for d <= 131071 (each product is at most
// 2^14), so any order and any split gives the same bits.
#include "common.hpp"

namespace gptq {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));
typedef i32x4 Unit __attribute__((aligned(1)));

struct GemmI8 {
  const int8_t* x;
  const uint8_t* w;
  const float *xs, *ws;
  const int32_t* z;
  void* y;
  int64_t m, rows, ld_x, ld_w, ld_y;
  int d, y_dtype;
};

GPTQ_DEV void store(const GemmI8& a, int64_t i, int64_t r, int sum, int xsum) {
  int64_t whole = sum;
  if (a.z) whole += ((int64_t)128 - a.z[r]) * xsum;
  float v = (float)whole;
  if (a.xs) v *= a.xs[i];
  if (a.ws) v *= a.ws[r];
  const int64_t at = i * a.ld_y + r;
  if (a.y_dtype == F32) static_cast<float*>(a.y)[at] = v;
  else if (a.y_dtype == F16) static_cast<_Float16*>(a.y)[at] = (_Float16)v;
  else static_cast<__bf16*>(a.y)[at] = (__bf16)v;
}

// 16 bytes of a row from column k on, zeros past the last one.
GPTQ_DEV i32x4 bytes16(const void* row, int k, int d) {
  const uint8_t* p = static_cast<const uint8_t*>(row) + k;
  if (k + 16 <= d) return *reinterpret_cast<const Unit*>(p);
  uint32_t v[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int e = 0; e < 16; ++e)
    if (k + e < d) v[e / 4] |= (uint32_t)p[e] << (8 * (e % 4));
  return i32x4{(int)v[0], (int)v[1], (int)v[2], (int)v[3]};
}

// A wave owns 32 x 32 outputs; operands come straight from memory, 16 bytes a lane (v_mfma_i32_32x32x32_i8: lane l
// holds row l % 32, columns 16 (l / 32) .. + 15 of 32).
__global__ __launch_bounds__(256) void byte_gemm_kernel(GemmI8 a) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int col = lane & 31, half = lane >> 5;
  const int64_t i0 = (int64_t)blockIdx.x * 64 + 32 * (wave & 1), r0 = (int64_t)blockIdx.y * 64 + 32 * (wave >> 1);
  const int64_t i = min(i0 + col, a.m - 1), r = min(r0 + col, a.rows - 1);
  const int8_t* x = a.x + i * a.ld_x;
  const uint8_t* w = a.w + r * a.ld_w;
  i32x16 acc = {};
  int xsum = 0;
  const int flip = a.z ? (int)0x80808080 : 0;
  for (int k = 0; k < a.d; k += 32) {
    const i32x4 xf = bytes16(x, k + 16 * half, a.d);
    i32x4 wf = bytes16(w, k + 16 * half, a.d);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      wf[e] ^= flip;   // past the last column the row of x is zero
      xsum = __builtin_amdgcn_sdot4(xf[e], 0x01010101, xsum, false);
    }
    acc = __builtin_amdgcn_mfma_i32_32x32x32_i8(xf, wf, acc, 0, 0, 0);
  }
  xsum += __shfl_xor(xsum, 32, 64);
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const int mine = 8 * (e >> 2) + 4 * half + (e & 3);
    const int xs = __shfl(xsum, mine, 64);
    if (i0 + mine < a.m && r0 + col < a.rows) store(a, i0 + mine, r0 + col, acc[e], xs);
  }
}

}  // namespace

size_t byte_gemm_workspace_bytes(int64_t m, int64_t rows, int64_t d) { return 0; }

hipError_t byte_gemm(const int8_t* x, int64_t m, int64_t ld_x, const float* xs, const void* w, int64_t ld_w,
                     const float* ws, const int32_t* z, int64_t rows, int64_t d, void* y, int y_dtype, int64_t ld_y,
                     void* work, size_t work_bytes, hipStream_t s) {
  GemmI8 a{x, static_cast<const uint8_t*>(w), xs, ws, z, y, m, rows, ld_x, ld_w, ld_y, (int)d, y_dtype};
  // at most 2^16 row tiles a launch
  const int64_t step = (int64_t)1 << 22, rstep = (int64_t)1 << 21;
  for (int64_t r0 = 0; r0 < rows; r0 += rstep)
    for (int64_t i0 = 0; i0 < m; i0 += step) {
      GemmI8 b = a;
      b.m = std::min(step, m - i0);
      b.rows = std::min(rstep, rows - r0);
      b.x = x + i0 * ld_x;
      b.w = a.w + r0 * ld_w;
      if (xs) b.xs = xs + i0;
      if (ws) b.ws = ws + r0;
      if (z) b.z = z + r0;
      b.y = static_cast<char*>(y) + (i0 * ld_y + r0) * (y_dtype == F32 ? 4 : 2);
      hipLaunchKernelGGL(byte_gemm_kernel, dim3((unsigned)((b.m + 63) / 64), (unsigned)((b.rows + 63) / 64)), dim3(256), 0,
                         s, b);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
  return hipSuccess;
}

}  // namespace gptq
