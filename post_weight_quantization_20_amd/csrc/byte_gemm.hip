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
// number is exact in a double below 2^53 (|xsum| is below 2^24), and in 64 bits for any zero.
template <bool CODES>
GPTQ_DEV float output(int sum, int xsum, int zero, float xs, float ws) {
  float v = (float)sum;
  if constexpr (CODES) {
    if (__builtin_expect(zero > -(1 << 28) && zero < (1 << 28), 1))
      v = (float)__builtin_fma((double)(128 - zero), (double)xsum, (double)sum);
    else
      v = (float)((int64_t)sum + (128 - (int64_t)zero) * xsum);
  }
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

template <bool CODES>
GPTQ_DEV i32x4 as_signed(i32x4 v) {
  if constexpr (CODES) {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] ^= (int)0x80808080;
  }
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
// Stages of KB columns of 256 rows of each operand stream into LDS 16 bytes a lane (buffer_load ... lds), through a
// ring of NST stages; units of a row are XOR-swizzled so that the 32 rows of an operand read fall in distinct
// banks. Columns past d and rows past the last read as zeros through the descriptor's range. Rows that are not
// 16-byte aligned, or whose width is not a multiple of 16, are staged through registers instead.
constexpr int BT = 256;        // tile edge
constexpr int GROUP = 8;       // row tiles that run side by side

GPTQ_DEV void dma16(i32x4 rsrc, uint32_t voff, uint32_t lds_addr) {
  asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds" ::"v"(voff), "s"(rsrc), "{m0}"(lds_addr)
               : "memory");
}

// Waits until at most N of this thread's loads into LDS are in flight and all its LDS reads are done, then meets
// the workgroup. The builtin tells the compiler that no LDS read is pending; the loads it does not track.
template <int N>
GPTQ_DEV void stage_barrier() {
  __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0)
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

GPTQ_DEV i32x4 descriptor(const void* base, int64_t bytes) {
  const uint64_t b = (uint64_t)(uintptr_t)base;
  return i32x4{__builtin_amdgcn_readfirstlane((int)(uint32_t)b), __builtin_amdgcn_readfirstlane((int)(uint32_t)(b >> 32)),
               __builtin_amdgcn_readfirstlane((int)bytes), 0x00020000};
}

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

template <int KB, int NST, bool DMA, bool CODES, int YT>
__global__ __launch_bounds__(256) void tile_kernel(GemmI8 a) {
  constexpr int UN = KB / 16, KS = KB / 32;       // units of a row, products of 32 columns
  constexpr int OPB = BT * KB, STAGEB = 2 * OPB;  // bytes of an operand and of a stage
  constexpr int LOADS = OPB / 16 / 256;           // units a thread stages of each operand
  extern __shared__ __align__(16) char smem_raw[];
  GPTQ_LDS char* lds = (GPTQ_LDS char*)smem_raw;
  uint32_t tm, tn;
  if (!tile_of(a, blockIdx.x, tm, tn)) return;
  const int64_t m0 = (int64_t)tm * BT, n0 = (int64_t)tn * BT;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1, col = lane & 31, half = lane >> 5;
  const int nst = (a.d + KB - 1) / KB;

  // unit q of a thread: LDS unit 256 q + tid, row / UN, in which column unit (u ^ swizzle) of the row lies
  // (an operand read takes 16 lanes a cycle, rows r .. r + 15 of one unit, over 64 banks: 256 bytes)
  auto swizzle = [](int row) { return UN == 8 ? ((row >> 1) & 7) : ((row >> 2) & 3); };
  constexpr uint32_t OOB = 0x80000000u;           // beyond any descriptor's range: reads as zero
  const int64_t mrows = min((int64_t)BT, a.m - m0), nrows = min((int64_t)BT, a.rows - n0);
  const int8_t* xb = a.x + m0 * a.ld_x;
  const uint8_t* wb = a.w + n0 * a.ld_w;
  int srow[LOADS], scol[LOADS];
  uint32_t xo[LOADS], wo[LOADS];
#pragma unroll
  for (int q = 0; q < LOADS; ++q) {
    const int u = 256 * q + tid;
    srow[q] = u / UN;
    scol[q] = 16 * ((u % UN) ^ swizzle(u / UN));
    xo[q] = (uint32_t)(srow[q] * a.ld_x + scol[q]);
    wo[q] = (uint32_t)(srow[q] * a.ld_w + scol[q]);
    if (srow[q] >= mrows) xo[q] = OOB;
    if (srow[q] >= nrows) wo[q] = OOB;
  }
  auto issue = [&](int s) {
    const int k0 = s * KB;
    GPTQ_LDS char* dst = lds + (s % NST) * STAGEB;
    if constexpr (DMA) {
      const i32x4 xr = descriptor(xb + k0, (mrows - 1) * a.ld_x + a.d - k0),
                  wr = descriptor(wb + k0, (nrows - 1) * a.ld_w + a.d - k0);
      const uint32_t base = (uint32_t)(uintptr_t)dst + 1024 * wave;
      const bool last = k0 + KB > a.d;            // columns past d would be the next row's
#pragma unroll
      for (int q = 0; q < LOADS; ++q) dma16(xr, last && k0 + scol[q] >= a.d ? OOB : xo[q], base + 4096 * q);
#pragma unroll
      for (int q = 0; q < LOADS; ++q) dma16(wr, last && k0 + scol[q] >= a.d ? OOB : wo[q], base + OPB + 4096 * q);
    } else {
      i32x4 xv[LOADS], wv[LOADS];
#pragma unroll
      for (int q = 0; q < LOADS; ++q) {
        xv[q] = wv[q] = i32x4{0, 0, 0, 0};
        if (k0 + scol[q] < a.d) {
          if (srow[q] < mrows) xv[q] = bytes16(xb + srow[q] * a.ld_x, k0 + scol[q], a.d);
          if (srow[q] < nrows) wv[q] = bytes16(wb + srow[q] * a.ld_w, k0 + scol[q], a.d);
        }
      }
#pragma unroll
      for (int q = 0; q < LOADS; ++q) {
        *(GPTQ_LDS i32x4*)(dst + 4096 * q + 16 * tid) = xv[q];
        *(GPTQ_LDS i32x4*)(dst + OPB + 4096 * q + 16 * tid) = wv[q];
      }
    }
  };

  // operand reads: row 32 i + col of the wave's 128, unit 2 ks + half
  const int xrow = (128 * wm + col) * KB, wrow = OPB + (128 * wn + col) * KB;
  const int sw = swizzle(col);
  auto read = [&](int s, int ks, i32x4 (&xv)[4], i32x4 (&wv)[4], int i0, int i1) {
    GPTQ_LDS char* b = lds + (s % NST) * STAGEB + (((2 * ks + half) ^ sw) << 4);
#pragma unroll
    for (int i = i0; i < i1; ++i) {
      xv[i] = *(GPTQ_LDS i32x4*)(b + xrow + 32 * KB * i);
      wv[i] = *(GPTQ_LDS i32x4*)(b + wrow + 32 * KB * i);
    }
  };
  i32x16 acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = i32x16{};
  int xsum[4] = {0, 0, 0, 0};
  auto multiply = [&](const i32x4 (&xv)[4], i32x4 (&wv)[4], int i0, int i1) {   // from i0 = 0 on, in order
    if (i0 == 0) {
#pragma unroll
      for (int j = 0; j < 4; ++j) wv[j] = as_signed<CODES>(wv[j]);
    }
#pragma unroll
    for (int i = i0; i < i1; ++i) {
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(wv[j], xv[i], acc[i][j], 0, 0, 0);
      if constexpr (CODES) xsum[i] = add_bytes(xv[i], xsum[i]);
    }
  };

  if constexpr (DMA) {
    constexpr int L = 2 * LOADS;                  // loads of a thread a stage
    for (int s = 0; s < NST && s < nst; ++s) issue(s);
    if (nst >= NST) stage_barrier<(NST - 1) * L>();
    else stage_barrier<0>();
    i32x4 x0[4], w0[4], x1[4], w1[4];
    read(0, 0, x0, w0, 0, 4);
    for (int it = 0; it < nst; ++it) {
      // All steps of the stage but the last, each under the reads of the next one's operands.
#pragma unroll
      for (int ks = 0; ks + 1 < KS; ++ks) {
        __builtin_amdgcn_s_waitcnt(0xC07F);       // lgkmcnt(0): this step's operands, read a step ago
        if (ks & 1) {
          read(it, ks + 1, x0, w0, 0, 4);
          multiply(x1, w1, 0, 4);
        } else {
          read(it, ks + 1, x1, w1, 0, 4);
          multiply(x0, w0, 0, 4);
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          __builtin_amdgcn_sched_group_barrier(0x008, 2, 0);   // two MFMAs
          __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);   // one LDS read
        }
      }
      // The last step (its operands are in x1, w1): stage it is read to the end by every wave and stage it + 1 has
      // arrived behind the barrier, so the loads of stage it + NST go out and the first operands of stage it + 1
      // are read while it multiplies (after the last stage those reads are stale and not used).
      if (it + NST <= nst) stage_barrier<(NST - 2) * L>();
      else stage_barrier<0>();
      read(it + 1, 0, x0, w0, 0, 2);
      multiply(x1, w1, 0, 2);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        __builtin_amdgcn_sched_group_barrier(0x008, 2, 1);
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 1);
      }
      if (it + NST < nst) issue(it + NST);
      read(it + 1, 0, x0, w0, 2, 4);
      multiply(x1, w1, 2, 4);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        __builtin_amdgcn_sched_group_barrier(0x008, 2, 2);
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 2);
      }
    }
    stage_barrier<0>();
  } else {
    issue(0);
    for (int it = 0; it < nst; ++it) {
      __syncthreads();
      if (it + 1 < nst) issue(it + 1);
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        i32x4 xv[4], wv[4];
        read(it, ks, xv, wv, 0, 4);
        multiply(xv, wv, 0, 4);
      }
    }
    __syncthreads();
  }

  // Register e of lane l: output 8 (e / 4) + 4 (l / 32) + e % 4 of block j, token l % 32 of block i. Outputs leave
  // through LDS, 32 tokens by the wave's 128 outputs at a time, so that a token's come side by side.
  typedef typename ElemOf<YT>::T T;
  typedef T T4 __attribute__((ext_vector_type(4)));
  constexpr int ESZ = sizeof(T), PITCH = 128 * ESZ + 16, UR = 8 * ESZ;   // UR: 16-byte units of a row
  GPTQ_LDS char* area = lds + wave * 32 * (128 * 4 + 16);
  GPTQ_LDS float* ws = (GPTQ_LDS float*)(lds + 4 * 32 * (128 * 4 + 16));
  GPTQ_LDS int32_t* zs = (GPTQ_LDS int32_t*)(ws + BT);
  {
    const int64_t r = min(n0 + tid, a.rows - 1);
    ws[tid] = a.ws ? a.ws[r] : 1.0f;
    if constexpr (CODES) zs[tid] = a.z[r];
  }
  float xs[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) xs[i] = a.xs ? a.xs[min(m0 + 128 * wm + 32 * i + col, a.m - 1)] : 1.0f;
  __syncthreads();
  const int64_t nc = n0 + 128 * wn;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t mr = m0 + 128 * wm + 32 * i;
    if constexpr (CODES) xsum[i] += __shfl_xor(xsum[i], 32, 64);
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
        for (int e = 0; e < 4; ++e) o[e] = (T)output<CODES>(acc[i][j][4 * b + e], xsum[i], z4[e], xs[i], w4[e]);
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
  const int flip = a.z ? (int)0x80808080 : 0;
  for (int k = 0; k < a.d; k += 32) {
    const i32x4 xf = bytes16(x, k + 16 * half, a.d);
    i32x4 wf = bytes16(w, k + 16 * half, a.d);
#pragma unroll
    for (int e = 0; e < 4; ++e) wf[e] ^= flip;   // past the last column the row of x is zero
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

constexpr int kKB = 128, kNST = 2;

template <bool DMA, bool CODES, int YT>
hipError_t launch_tile(const GemmI8& a, hipStream_t s) {
  static std::atomic<uint64_t> asked{0};
  constexpr size_t lds = (size_t)kNST * 2 * BT * kKB;
  auto f = tile_kernel<kKB, kNST, DMA, CODES, YT>;
  const hipError_t e = ask_lds(f, lds, asked);
  if (e != hipSuccess) return e;
  const uint32_t per = (a.tiles_m * a.tiles_n + 7) / 8;
  hipLaunchKernelGGL(f, dim3(8 * per), dim3(256), lds, s, a);
  return hipGetLastError();
}

template <bool DMA, bool CODES>
hipError_t tile_type(const GemmI8& a, hipStream_t s) {
  return a.y_dtype == F32   ? launch_tile<DMA, CODES, F32>(a, s)
         : a.y_dtype == F16 ? launch_tile<DMA, CODES, F16>(a, s)
                            : launch_tile<DMA, CODES, BF16>(a, s);
}

hipError_t one(const GemmI8& a, hipStream_t s) {
  if (a.m > 128) {
    // 16-byte units inside rows, and a tile inside 31-bit offsets
    const bool dma = a.d % 16 == 0 && reinterpret_cast<uintptr_t>(a.x) % 16 == 0 && reinterpret_cast<uintptr_t>(a.w) % 16 == 0 &&
                     a.ld_x % 16 == 0 && a.ld_w % 16 == 0 && std::max(a.ld_x, a.ld_w) < ((int64_t)1 << 22);
    if (dma) return a.z ? tile_type<true, true>(a, s) : tile_type<true, false>(a, s);
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
