// y[i, r] = sx[i] sw[r] sum_k x[i, k] (w[r, k] - z[r]) for int8 rows x and 8-bit weights w.
//
// Signed weights (z absent) go to the matrix cores as they are. Unsigned codes c of a stored layer become signed
// by flipping their top bit, c - 128, and sum x (c - z) = sum x (c - 128) + (128 - z) sum x: the rows' sums are
// formed beside the product. All sums are exact whole numbers in 32 bits for d <= 131071 (each product is at most
// 2^14), so any order and any split gives the same bits.
//
// Three kernels, by the number of tokens:
//   tile    256 x 256 outputs a workgroup (4 waves of 128 x 128, v_mfma_i32_32x32x32_i8), operands through LDS
//   strip   up to 128 tokens x 64 outputs a workgroup, whose waves share the sum over k and read both operands
//           straight from memory: each byte of w is used by one wave
//   token   up to 16 tokens x 16 outputs (v_mfma_i32_16x16x64_i8), eight waves sharing the sum
#include "common.hpp"

#include <atomic>

namespace gptq {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));
typedef i32x4 Unit __attribute__((aligned(1)));
#define GPTQ_LDS __attribute__((address_space(3)))

struct GemmI8 {
  const int8_t* x;
  const uint8_t* w;
  const float *xs, *ws;
  const int32_t* z;
  void* y;
  int64_t m, rows, ld_x, ld_w, ld_y;
  int d, y_dtype;
  int y_vec;              // rows of y take 16-byte stores
  uint32_t tiles_m, tiles_n;
};

// One output from its whole sum and its row's sum of x: fp32 roundings of the sum and of two products. The whole
// number is exact in a double below 2^53, which only zeros beyond 2^28 (|xsum| is below 2^24) can pass.
template <bool CODES>
GPTQ_DEV float output(int sum, int xsum, int zero, float xs, float ws) {
  const float v = CODES ? (float)__builtin_fma(128.0 - (double)zero, (double)xsum, (double)sum) : (float)sum;
  return v * xs * ws;
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

GPTQ_DEV i32x4 flip(i32x4 v) {
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] ^= (int)0x80808080;
  return v;
}

GPTQ_DEV int add_bytes(i32x4 v, int sum) {
#pragma unroll
  for (int e = 0; e < 4; ++e) sum = __builtin_amdgcn_sdot4(v[e], 0x01010101, sum, false);
  return sum;
}

GPTQ_DEV void store_one(const GemmI8& a, int64_t i, int64_t r, float v) {
  const int64_t at = i * a.ld_y + r;
  if (a.y_dtype == F32) static_cast<float*>(a.y)[at] = v;
  else if (a.y_dtype == F16) static_cast<_Float16*>(a.y)[at] = (_Float16)v;
  else static_cast<__bf16*>(a.y)[at] = (__bf16)v;
}

// ------------------------------------------------------------------ tiles
//
// Stages of 128 columns of 256 rows of each operand go to LDS by way of registers: a thread loads 16 units of 16 bytes
// of stage s + 2 while stage s is multiplied, and each is written to LDS a whole stage later, so that every load has
// that long to arrive and neither loads nor writes come in bursts that matrix instructions would queue behind (loads
// straight into LDS have to wait for their buffer: 4096 x 4096 x 65536 in 1030 us with them). Units of a row are
// XOR-swizzled so that the 16 rows of an operand read's cycle fall in distinct banks. Columns past d and rows past
// the last read as zeros through the descriptor's range; where rows are not 4-byte aligned or d is no multiple of 16
// the loads are ordinary ones with masks. Codes are flipped, and the rows of x summed, on their way through registers.
constexpr int BT = 256;                 // tile edge
constexpr int KB = 128;                 // columns of a stage
constexpr int OPB = BT * KB;            // bytes of an operand's stage
constexpr int STAGEB = 2 * OPB;
constexpr int GROUP = 8;                // row tiles that run side by side

// Tile of a workgroup: XCD b % 8 takes a contiguous run of an order in which GROUP row tiles run side by side
// through the column tiles, so that what its L2 holds is shared.
GPTQ_DEV bool tile_of(const GemmI8& a, uint32_t b, uint32_t& tm, uint32_t& tn) {
  const uint32_t total = a.tiles_m * a.tiles_n, per = (total + 7) / 8;
  const uint32_t slot = (b & 7) * per + (b >> 3);
  if ((b >> 3) >= per || slot >= total) return false;
  const uint32_t span = GROUP * a.tiles_n, grp = slot / span, in = slot - grp * span;
  const uint32_t height = min((uint32_t)GROUP, a.tiles_m - grp * GROUP);
  tm = grp * GROUP + in % height;
  tn = in / height;
  return true;
}

template <bool WHOLE, bool CODES, int YT>
__global__ __launch_bounds__(256) void tile_kernel(GemmI8 a) {
  extern __shared__ __align__(16) char smem_raw[];
  GPTQ_LDS char* lds = (GPTQ_LDS char*)smem_raw;
  uint32_t tm, tn;
  if (!tile_of(a, blockIdx.x, tm, tn)) return;
  const int64_t m0 = (int64_t)tm * BT, n0 = (int64_t)tn * BT;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1, col = lane & 31, half = lane >> 5;
  const int nst = (a.d + KB - 1) / KB;

  // staging: unit q of a thread is row 32 q + tid / 8 of the tile, LDS unit tid % 8 of that row, which holds column
  // unit (tid % 8) ^ swizzle(row)
  const int64_t mrows = min((int64_t)BT, a.m - m0), nrows = min((int64_t)BT, a.rows - n0);
  const int8_t* xb = a.x + m0 * a.ld_x;
  const uint8_t* wb = a.w + n0 * a.ld_w;
  const int srow = tid >> 3, scol = 16 * ((tid & 7) ^ ((srow >> 1) & 7));
  i32x4 st[16];                                   // 8 units of x, 8 of w
  auto fetch = [&](int s, int q) {
    const int k0 = s * KB, e = q & 7;
    const bool isx = q < 8;
    const int64_t ld = isx ? a.ld_x : a.ld_w, rows = isx ? mrows : nrows;
    const char* base = (isx ? reinterpret_cast<const char*>(xb) : reinterpret_cast<const char*>(wb)) + k0;
    if constexpr (WHOLE) {
      // past d: beyond the descriptor's range, as rows past the last are (ld >= d)
      const int bytes = s < nst ? (int)((rows - 1) * ld + a.d - k0) : 0;
      const uint32_t off = k0 + scol < a.d ? (uint32_t)((srow + 32 * e) * (int)ld + scol) : 0x80000000u;
      st[q] = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(
          __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(base), 0, bytes, 0x00020000), off, 0, 0));
    } else {
      const int row = srow + 32 * e;
      st[q] = i32x4{0, 0, 0, 0};
      if (k0 + scol < a.d && row < rows) st[q] = bytes16(base - k0 + row * ld, k0 + scol, a.d);
    }
  };
  int xsum[8] = {0, 0, 0, 0, 0, 0, 0, 0};         // of rows 32 q + tid / 8: this thread's columns
  auto put = [&](int s, int q) {
    i32x4 v = st[q];
    if constexpr (CODES) {
      if (q < 8) xsum[q] = add_bytes(v, xsum[q]);
      else v = flip(v);
    }
    *(GPTQ_LDS i32x4*)(lds + (s & 1) * STAGEB + 4096 * q + 16 * tid) = v;
  };

  // operand reads: row 32 i + col of the wave's 128, unit 2 ks + half
  const int xrow = (128 * wm + col) * KB, wrow = OPB + (128 * wn + col) * KB, sw = (col >> 1) & 7;
  struct Step {
    i32x4 x[4], w[4];
  };
  // a quarter of a step's operands: two blocks of w, the others of w, two of x, the others of x
  auto read = [&](int s, int ks, Step& o, int quarter) {
    GPTQ_LDS char* b = lds + (s & 1) * STAGEB + (((2 * ks + half) ^ sw) << 4);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int i = 2 * (quarter & 1) + e;
      if (quarter < 2) o.w[i] = *(GPTQ_LDS i32x4*)(b + wrow + 32 * KB * i);
      else o.x[i] = *(GPTQ_LDS i32x4*)(b + xrow + 32 * KB * i);
    }
  };
  i32x16 acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = i32x16{};

  // A step multiplies operands that are in registers while the next step's are read, in quarters; with each quarter a
  // unit of stage s goes to LDS and its register takes one of stage s + 1. The barrier before a stage's last step
  // says that every wave has read that stage to its end and written the next one.
  auto step = [&](Step& cur, Step& next, int s, int ks, int to, int q0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      read(s, ks, next, i);
      put(to, q0 + i);
      fetch(to + 1, q0 + i);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(cur.w[j], cur.x[i], acc[i][j], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
#pragma unroll
  for (int q = 0; q < 16; ++q) fetch(0, q);
#pragma unroll
  for (int q = 0; q < 16; ++q) {
    put(0, q);
    fetch(1, q);
  }
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    put(1, q);
    fetch(2, q);
  }
  __syncthreads();
  Step even, odd;
#pragma unroll
  for (int q = 0; q < 4; ++q) read(0, 0, even, q);
  for (int it = 0; it < nst; ++it) {
    step(even, odd, it, 1, it + 1, 4);
    step(odd, even, it, 2, it + 1, 8);
    step(even, odd, it, 3, it + 1, 12);
    // LDS reads and writes done, loads still on their way
    __builtin_amdgcn_s_waitcnt(0xC07F);
    asm volatile("s_barrier" ::: "memory");
    step(odd, even, it + 1, 0, it + 2, 0);        // what this reads after the last stage is not used
  }
  __syncthreads();

  // Register e of lane l: output 8 (e / 4) + 4 (l / 32) + e % 4 of block j, token l % 32 of block i. Outputs leave
  // through LDS, 32 tokens by the wave's 128 outputs at a time, so that a token's come side by side.
  typedef typename ElemOf<YT>::T T;
  typedef T T4 __attribute__((ext_vector_type(4)));
  constexpr int ESZ = sizeof(T), PITCH = 128 * ESZ + 16, UR = 8 * ESZ;   // UR: 16-byte units of a row
  GPTQ_LDS char* area = lds + wave * 32 * (128 * 4 + 16);
  GPTQ_LDS float* ws = (GPTQ_LDS float*)(lds + 4 * 32 * (128 * 4 + 16));
  GPTQ_LDS int32_t* zs = (GPTQ_LDS int32_t*)(ws + BT);
  GPTQ_LDS int32_t* sums = zs + BT;
  {
    const int64_t r = min(n0 + tid, a.rows - 1);
    ws[tid] = a.ws ? a.ws[r] : 1.0f;
    if constexpr (CODES) {
      zs[tid] = a.z[r];
#pragma unroll
      for (int q = 0; q < 8; ++q) {
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) xsum[q] += __shfl_xor(xsum[q], o, 64);
        if ((tid & 7) == 0) sums[32 * q + srow] = xsum[q];
      }
    }
  }
  float xs[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) xs[i] = a.xs ? a.xs[min(m0 + 128 * wm + 32 * i + col, a.m - 1)] : 1.0f;
  __syncthreads();
  const int64_t nc = n0 + 128 * wn;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t mr = m0 + 128 * wm + 32 * i;
    const int xsm = CODES ? sums[128 * wm + 32 * i + col] : 0;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int c = 32 * j + 8 * b + 4 * half;
        const floatx4 w4 = *(GPTQ_LDS floatx4*)(ws + 128 * wn + c);
        i32x4 z4 = {};
        if constexpr (CODES) z4 = *(GPTQ_LDS i32x4*)(zs + 128 * wn + c);
        T4 o;
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = (T)output<CODES>(acc[i][j][4 * b + e], xsm, z4[e], xs[i], w4[e]);
        *(GPTQ_LDS T4*)(area + col * PITCH + c * ESZ) = o;
      }
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int q = 0; q < UR / 2; ++q) {
      const int u = 64 * q + lane, row = u / UR, c = u % UR * 16 / ESZ;
      if (mr + row >= a.m || nc + c >= a.rows) continue;
      GPTQ_LDS char* o = area + row * PITCH + c * ESZ;
      T* dst = static_cast<T*>(a.y) + (mr + row) * a.ld_y + nc + c;
      if (a.y_vec && nc + c + 16 / ESZ <= a.rows) {
        *reinterpret_cast<i32x4*>(dst) = *(GPTQ_LDS i32x4*)o;
      } else {
        for (int e = 0; e < 16 / ESZ; ++e)
          if (nc + c + e < a.rows) dst[e] = ((GPTQ_LDS T*)o)[e];
      }
    }
    __builtin_amdgcn_wave_barrier();
  }
}

// ------------------------------------------------------------------ strips

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
  for (int k = 0; k < a.d; k += 32) {
    const i32x4 xf = bytes16(x, k + 16 * half, a.d);
    i32x4 wf = bytes16(w, k + 16 * half, a.d);
    if (a.z) wf = flip(wf);   // past the last column the row of x is zero
    xsum = add_bytes(xf, xsum);
    acc = __builtin_amdgcn_mfma_i32_32x32x32_i8(xf, wf, acc, 0, 0, 0);
  }
  xsum += __shfl_xor(xsum, 32, 64);
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const int mine = 8 * (e >> 2) + 4 * half + (e & 3);
    const int xsm = __shfl(xsum, mine, 64);
    if (i0 + mine < a.m && r0 + col < a.rows)
      store_one(a, i0 + mine, r0 + col, output<true>(acc[e], xsm, a.z ? a.z[r0 + col] : 128, a.xs ? a.xs[i0 + mine] : 1.0f,
                                                     a.ws ? a.ws[r0 + col] : 1.0f));
  }
}

// Asks once per device for a kernel's LDS beyond 64 KB.
template <typename K>
hipError_t ask_lds(K kernel, size_t lds, std::atomic<uint64_t>& asked) {
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  const uint64_t bit = (uint64_t)1 << (dev & 63);
  if (dev > 63 || !(asked.load() & bit)) {
    e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
    asked |= bit;
  }
  return hipSuccess;
}

template <bool WHOLE, bool CODES, int YT>
hipError_t launch_tile(const GemmI8& a, hipStream_t s) {
  static std::atomic<uint64_t> asked{0};
  constexpr size_t lds = 2 * STAGEB;
  auto f = tile_kernel<WHOLE, CODES, YT>;
  const hipError_t e = ask_lds(f, lds, asked);
  if (e != hipSuccess) return e;
  const uint32_t per = (a.tiles_m * a.tiles_n + 7) / 8;
  hipLaunchKernelGGL(f, dim3(8 * per), dim3(256), lds, s, a);
  return hipGetLastError();
}

template <bool WHOLE, bool CODES>
hipError_t tile_type(const GemmI8& a, hipStream_t s) {
  return a.y_dtype == F32   ? launch_tile<WHOLE, CODES, F32>(a, s)
         : a.y_dtype == F16 ? launch_tile<WHOLE, CODES, F16>(a, s)
                            : launch_tile<WHOLE, CODES, BF16>(a, s);
}

hipError_t one(const GemmI8& a, hipStream_t s) {
  if (a.m > 128) {
    // 16-byte units inside rows of whole words, and a tile inside 31-bit offsets
    const bool whole = a.d % 16 == 0 && reinterpret_cast<uintptr_t>(a.x) % 4 == 0 &&
                       reinterpret_cast<uintptr_t>(a.w) % 4 == 0 && a.ld_x % 4 == 0 && a.ld_w % 4 == 0 &&
                       std::max(a.ld_x, a.ld_w) < ((int64_t)1 << 22);
    if (whole) return a.z ? tile_type<true, true>(a, s) : tile_type<true, false>(a, s);
    return a.z ? tile_type<false, true>(a, s) : tile_type<false, false>(a, s);
  }
  hipLaunchKernelGGL(byte_gemm_kernel, dim3((unsigned)((a.m + 63) / 64), (unsigned)((a.rows + 63) / 64)), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace

size_t byte_gemm_workspace_bytes(int64_t m, int64_t rows, int64_t d) { return 0; }

hipError_t byte_gemm(const int8_t* x, int64_t m, int64_t ld_x, const float* xs, const void* w, int64_t ld_w,
                     const float* ws, const int32_t* z, int64_t rows, int64_t d, void* y, int y_dtype, int64_t ld_y,
                     void* work, size_t work_bytes, hipStream_t s) {
  GemmI8 a{x, static_cast<const uint8_t*>(w), xs, ws, z, y, m, rows, ld_x, ld_w, ld_y, (int)d, y_dtype, 0, 0, 0};
  const int64_t esz = y_dtype == F32 ? 4 : 2;
  a.y_vec = reinterpret_cast<uintptr_t>(y) % 16 == 0 && ld_y * esz % 16 == 0;
  // a launch takes at most 2^20 tokens by 2^18 outputs (2^22 tiles)
  const int64_t step = (int64_t)1 << 20, rstep = (int64_t)1 << 18;
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
      b.y = static_cast<char*>(y) + (i0 * ld_y + r0) * esz;
      b.tiles_m = (uint32_t)((b.m + BT - 1) / BT);
      b.tiles_n = (uint32_t)((b.rows + BT - 1) / BT);
      const hipError_t e = one(b, s);
      if (e != hipSuccess) return e;
    }
  return hipSuccess;
}

}  // namespace gptq
