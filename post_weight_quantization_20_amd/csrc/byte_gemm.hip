// y[i, r] = sx[i] sw[r] sum_k x[i, k] (w[r, k] - z[r]) for int8 rows x and 8-bit weights w.
//
// Signed weights (z absent) go to the matrix cores as they are. Unsigned codes c of a stored layer become signed
// by flipping their top bit, c - 128, and sum x (c - z) = sum x (c - 128) + (128 - z) sum x: the rows' sums are
// formed beside the product. All sums are exact whole numbers in 32 bits for d <= 131071 (each product is at most
// 2^14), so any order and any split gives the same bits.
//
// Two kernels:
//   tile    256 x 256 outputs a workgroup (4 waves of 128 x 128, v_mfma_i32_32x32x32_i8), operands through LDS
//   strip   up to 128 tokens and as many outputs as give each CU a workgroup, whose waves share the sum over k and read
//           both operands straight from memory
//
// Measured, calls after one another: 8192 x 4096 x 11008 in 369 us, 2.0 POPS (random data, the board's power limit holds
// the clock at 1.73 GHz; 278 us where the data is zero), with codes 413 us; 96 x 4096 x 11008 with codes in 22 us;
// 8 x 4096 x 4096 in 5.5 us, 3.0 TB/s.
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
  uint32_t whole_tiles, cut;   // tiles of whole rounds; parts of each other tile
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
constexpr int GROUP = 8;                // row tiles that run side by side
// Up to so many tiles go to strips instead, which read x again for every strip but leave no CU idle: 256 tokens by 4096
// outputs (16 tiles) of 4096 columns take 17.0 us as strips and 19.6 as tiles, by 5120 outputs (20 tiles) 24.5 and 19.8;
// the two sides cross there with 1024 and 11008 columns and with 512 and 1024 tokens too.
constexpr uint32_t kStripTiles = 16;

// Tile `slot` of an order in which GROUP row tiles run side by side through the column tiles.
GPTQ_DEV void tile_at(const GemmI8& a, uint32_t slot, uint32_t& tm, uint32_t& tn) {
  const uint32_t span = GROUP * a.tiles_n, grp = slot / span, in = slot - grp * span;
  const uint32_t height = min((uint32_t)GROUP, a.tiles_m - grp * GROUP);
  tm = grp * GROUP + in % height;
  tn = in / height;
}

// One tile of 64 XI tokens by 64 WJ outputs from (m0, n0) on, by 2 x 2 waves of XI x WJ blocks of 32 x 32.
template <int XI, int WJ, bool WHOLE, bool CODES, int YT>
GPTQ_DEV void tile(const GemmI8& a, int64_t m0, int64_t n0, GPTQ_LDS char* lds) {
  constexpr int BM = 64 * XI, BN = 64 * WJ, STAGE = (BM + BN) * KB;
  constexpr int QX = 2 * XI, NQ = QX + 2 * WJ;    // units that a thread stages of x, and in all
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1, col = lane & 31, half = lane >> 5;
  const int nst = (a.d + KB - 1) / KB;

  // staging: unit q of a thread is row 32 q + tid / 8 of an operand's tile, LDS unit tid % 8 of that row, which holds
  // column unit (tid % 8) ^ swizzle(row)
  const int64_t mrows = min((int64_t)BM, a.m - m0), nrows = min((int64_t)BN, a.rows - n0);
  const int8_t* xb = a.x + m0 * a.ld_x;
  const uint8_t* wb = a.w + n0 * a.ld_w;
  const int srow = tid >> 3, scol = 16 * ((tid & 7) ^ ((srow >> 1) & 7));
  i32x4 st[NQ];
  auto fetch = [&](int s, int q) {
    const int k0 = s * KB, e = q < QX ? q : q - QX;
    const bool isx = q < QX;
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
  int xsum[QX] = {};                              // of rows 32 q + tid / 8: this thread's columns
  auto put = [&](int s, int q) {
    i32x4 v = st[q];
    if constexpr (CODES) {
      if (q < QX) xsum[q] = add_bytes(v, xsum[q]);
      else v = flip(v);
    }
    *(GPTQ_LDS i32x4*)(lds + (s & 1) * STAGE + 4096 * q + 16 * tid) = v;
  };

  // operand reads: row 32 i + col of the wave's, unit 2 ks + half
  const int xrow = (32 * XI * wm + col) * KB, wrow = BM * KB + (32 * WJ * wn + col) * KB, sw = (col >> 1) & 7;
  struct Step {
    i32x4 x[XI], w[WJ];
  };
  // part i of XI of a step's operands, those of w first
  auto read = [&](int s, int ks, Step& o, int i) {
    GPTQ_LDS char* b = lds + (s & 1) * STAGE + (((2 * ks + half) ^ sw) << 4);
#pragma unroll
    for (int e = i * (XI + WJ) / XI; e < (i + 1) * (XI + WJ) / XI; ++e) {
      if (e < WJ) o.w[e] = *(GPTQ_LDS i32x4*)(b + wrow + 32 * KB * e);
      else o.x[e - WJ] = *(GPTQ_LDS i32x4*)(b + xrow + 32 * KB * (e - WJ));
    }
  };
  i32x16 acc[XI][WJ];
#pragma unroll
  for (int i = 0; i < XI; ++i)
#pragma unroll
    for (int j = 0; j < WJ; ++j) acc[i][j] = i32x16{};

  // A step multiplies operands that are in registers while the next step's are read, in parts; with each part some
  // units of stage `to` go to LDS and their registers take those of stage to + 1. The barrier before a stage's last
  // step says that every wave has read that stage to its end and written the next one.
  auto step = [&](Step& cur, Step& next, int s, int ks, int to, int part0) {
#pragma unroll
    for (int i = 0; i < XI; ++i) {
      read(s, ks, next, i);
#pragma unroll
      for (int q = (part0 + i) * NQ / (4 * XI); q < (part0 + i + 1) * NQ / (4 * XI); ++q) {
        put(to, q);
        fetch(to + 1, q);
      }
#pragma unroll
      for (int j = 0; j < WJ; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(cur.w[j], cur.x[i], acc[i][j], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
#pragma unroll
  for (int q = 0; q < NQ; ++q) fetch(0, q);
#pragma unroll
  for (int q = 0; q < NQ; ++q) {
    put(0, q);
    fetch(1, q);
  }
#pragma unroll
  for (int q = 0; q < NQ / 4; ++q) {
    put(1, q);
    fetch(2, q);
  }
  __syncthreads();
  Step even, odd;
#pragma unroll
  for (int i = 0; i < XI; ++i) read(0, 0, even, i);
  for (int it = 0; it < nst; ++it) {
    step(even, odd, it, 1, it + 1, XI);
    step(odd, even, it, 2, it + 1, 2 * XI);
    step(even, odd, it, 3, it + 1, 3 * XI);
    // LDS reads and writes done, loads still on their way
    __builtin_amdgcn_s_waitcnt(0xC07F);
    asm volatile("s_barrier" ::: "memory");
    step(odd, even, it + 1, 0, it + 2, 0);        // what this reads after the last stage is not used
  }
  __syncthreads();

  // Register e of lane l: output 8 (e / 4) + 4 (l / 32) + e % 4 of block j, token l % 32 of block i. Outputs leave
  // through LDS, 32 tokens by the wave's outputs at a time, so that a token's come side by side.
  typedef typename ElemOf<YT>::T T;
  typedef T T4 __attribute__((ext_vector_type(4)));
  constexpr int ESZ = sizeof(T), WC = 32 * WJ, PITCH = WC * ESZ + 16, UR = WC * ESZ / 16;   // UR: 16-byte units of a row
  GPTQ_LDS char* area = lds + wave * 32 * PITCH;
  GPTQ_LDS float* ws = (GPTQ_LDS float*)(lds + 4 * 32 * PITCH);
  GPTQ_LDS int32_t* zs = (GPTQ_LDS int32_t*)(ws + BN);
  GPTQ_LDS int32_t* sums = zs + BN;
  if (tid < BN) {
    const int64_t r = min(n0 + tid, a.rows - 1);
    ws[tid] = a.ws ? a.ws[r] : 1.0f;
    if constexpr (CODES) zs[tid] = a.z[r];
  }
  if constexpr (CODES) {
#pragma unroll
    for (int q = 0; q < QX; ++q) {
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) xsum[q] += __shfl_xor(xsum[q], o, 64);
      if ((tid & 7) == 0) sums[32 * q + srow] = xsum[q];
    }
  }
  float xs[XI];
#pragma unroll
  for (int i = 0; i < XI; ++i) xs[i] = a.xs ? a.xs[min(m0 + 32 * (XI * wm + i) + col, a.m - 1)] : 1.0f;
  __syncthreads();
  const int64_t nc = n0 + WC * wn;
#pragma unroll
  for (int i = 0; i < XI; ++i) {
    const int64_t mr = m0 + 32 * (XI * wm + i);
    const int xsm = CODES ? sums[32 * (XI * wm + i) + col] : 0;
#pragma unroll
    for (int j = 0; j < WJ; ++j)
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int c = 32 * j + 8 * b + 4 * half;
        const floatx4 w4 = *(GPTQ_LDS floatx4*)(ws + WC * wn + c);
        i32x4 z4 = {};
        if constexpr (CODES) z4 = *(GPTQ_LDS i32x4*)(zs + WC * wn + c);
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

// Workgroups of whole rounds of the 256 CUs take a tile each, XCD b % 8 a contiguous run of them, so that what its L2
// holds is shared. The tiles of the last round are cut into `cut` parts where that many more workgroups still run at
// once: 256 x 128 (cut = 2) or 128 x 128 (cut = 4).
template <bool WHOLE, bool CODES, int YT>
__global__ __launch_bounds__(256) void tile_kernel(GemmI8 a) {
  extern __shared__ __align__(16) char smem_raw[];
  GPTQ_LDS char* lds = (GPTQ_LDS char*)smem_raw;
  const uint32_t b = blockIdx.x;
  uint32_t tm, tn;
  if (b < a.whole_tiles) {
    tile_at(a, (b & 7) * (a.whole_tiles >> 3) + (b >> 3), tm, tn);
    tile<4, 4, WHOLE, CODES, YT>(a, (int64_t)tm * BT, (int64_t)tn * BT, lds);
    return;
  }
  const uint32_t rest = b - a.whole_tiles, t = rest / a.cut, part = rest - t * a.cut;
  tile_at(a, a.whole_tiles + t, tm, tn);
  const int64_t m0 = (int64_t)tm * BT, n0 = (int64_t)tn * BT;
  if (a.cut == 1) {
    tile<4, 4, WHOLE, CODES, YT>(a, m0, n0, lds);
  } else if (a.cut == 2) {
    if (n0 + 128 * part < a.rows) tile<4, 2, WHOLE, CODES, YT>(a, m0, n0 + 128 * part, lds);
  } else {
    const int64_t m1 = m0 + 128 * (part >> 1), n1 = n0 + 128 * (part & 1);
    if (m1 < a.m && n1 < a.rows) tile<2, 2, WHOLE, CODES, YT>(a, m1, n1, lds);
  }
}

// ------------------------------------------------------------------ strips
//
// 16 MB tokens by 16 NB outputs a workgroup (v_mfma_i32_16x16x64_i8: lane l holds row l % 16 and 16 columns of each 64).
// The waves share the sum over k in blocks of 128 columns and add their sums up in LDS. Both operands come straight
// from memory, the next block's while one is multiplied: a byte of w is read by one wave. An instruction reads 64
// bytes of each of 16 rows, the first half of a line of even rows and the second of odd ones, which the cache serves
// side by side (128 x 4096 x 4096: 15.6 us against 21.9 with one half of all); the halves change places in registers. Few
// tokens are bound by reading w, more of them by reading x again for every strip.
template <int MB, int NB, int WAVES, bool CODES>
__global__ __launch_bounds__(64 * WAVES) void strip_kernel(GemmI8 a) {
  __shared__ int part[WAVES][NB][4][64];
  __shared__ int sums[WAVES][16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n = lane & 15, g = lane >> 4;
  const int64_t r0 = (int64_t)blockIdx.x * 16 * NB, i0 = (int64_t)blockIdx.y * 16 * MB;
  const uint8_t* w[NB];
  const int8_t* x[MB];
#pragma unroll
  for (int j = 0; j < NB; ++j) w[j] = a.w + min(r0 + 16 * j + n, a.rows - 1) * a.ld_w + 16 * g;
#pragma unroll
  for (int i = 0; i < MB; ++i) x[i] = a.x + min(i0 + 16 * i + n, a.m - 1) * a.ld_x + 16 * g;
  i32x4 acc[MB][NB];
  int xsum[MB];
#pragma unroll
  for (int i = 0; i < MB; ++i) {
    xsum[i] = 0;
#pragma unroll
    for (int j = 0; j < NB; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
  }
  struct Block {
    i32x4 x[2][MB], w[2][NB];
  };
  const int blocks = a.d >> 7;                    // whole ones
  const bool swap = n & 1;
  const int half[2] = {swap ? 64 : 0, swap ? 0 : 64};
  auto load = [&](int b, Block& o) {
    if (b >= blocks) return;
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e) o.w[e][j] = *reinterpret_cast<const Unit*>(w[j] + 128 * b + half[e]);
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) o.x[e][i] = *reinterpret_cast<const Unit*>(x[i] + 128 * b + half[e]);
  };
  auto multiply = [&](Block& o) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if constexpr (CODES) {
#pragma unroll
        for (int j = 0; j < NB; ++j) o.w[e][j] = flip(o.w[e][j]);
#pragma unroll
        for (int i = 0; i < MB; ++i) xsum[i] = add_bytes(o.x[e][i], xsum[i]);
      }
#pragma unroll
      for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(o.w[e][j], o.x[e][i], acc[i][j], 0, 0, 0);
    }
  };
  auto straight = [&](i32x4& first, i32x4& second) {
    const i32x4 f = first;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      first[e] = swap ? second[e] : f[e];
      second[e] = swap ? f[e] : second[e];
    }
  };
  auto whole = [&](Block& o) {
#pragma unroll
    for (int j = 0; j < NB; ++j) straight(o.w[0][j], o.w[1][j]);
#pragma unroll
    for (int i = 0; i < MB; ++i) straight(o.x[0][i], o.x[1][i]);
    multiply(o);
  };
  Block even, odd;
  load(wave, even);
  for (int b = wave; b < blocks; b += 2 * WAVES) {
    load(b + WAVES, odd);
    whole(even);
    load(b + 2 * WAVES, even);
    if (b + WAVES < blocks) whole(odd);
  }
  if ((a.d & 127) && wave == blocks % WAVES) {    // the last, partial block
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int k = 128 * blocks + 64 * e + 16 * g;
#pragma unroll
      for (int j = 0; j < NB; ++j) even.w[e][j] = k < a.d ? bytes16(w[j] - 16 * g, k, a.d) : i32x4{0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < MB; ++i) even.x[e][i] = k < a.d ? bytes16(x[i] - 16 * g, k, a.d) : i32x4{0, 0, 0, 0};
    }
    multiply(even);
  }
  // register e of lane l: output 4 (l / 16) + e of block j, token l % 16
#pragma unroll
  for (int i = 0; i < MB; ++i) {
    if (i) __syncthreads();
    if constexpr (CODES) {
      xsum[i] += __shfl_xor(xsum[i], 16, 64);
      xsum[i] += __shfl_xor(xsum[i], 32, 64);
      if (g == 0) sums[wave][n] = xsum[i];
    }
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) part[wave][j][e][lane] = acc[i][j][e];
    __syncthreads();
    const int64_t t = i0 + 16 * i + n;
    for (int j = wave; j < NB; j += WAVES) {
      const int64_t r = r0 + 16 * j + 4 * g;
      if (t >= a.m || r >= a.rows) continue;
      int sum[4] = {0, 0, 0, 0}, xsm = 0;
#pragma unroll
      for (int v = 0; v < WAVES; ++v) {
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[e] += part[v][j][e][lane];
        if constexpr (CODES) xsm += sums[v][n];
      }
      const float xs = a.xs ? a.xs[t] : 1.0f;
      float o[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int64_t c = min(r + e, a.rows - 1);
        o[e] = output<CODES>(sum[e], xsm, CODES ? a.z[c] : 0, xs, a.ws ? a.ws[c] : 1.0f);
      }
      auto put = [&](auto* y) {
        typedef typename std::remove_pointer<decltype(y)>::type T;
        typedef T T4 __attribute__((ext_vector_type(4), aligned(sizeof(T))));
        y += t * a.ld_y + r;
        if (r + 4 <= a.rows) {
          *reinterpret_cast<T4*>(y) = T4{(T)o[0], (T)o[1], (T)o[2], (T)o[3]};
        } else {
          for (int e = 0; e < 3; ++e)
            if (r + e < a.rows) y[e] = (T)o[e];
        }
      };
      if (a.y_dtype == F32) put(static_cast<float*>(a.y));
      else if (a.y_dtype == F16) put(static_cast<_Float16*>(a.y));
      else put(static_cast<__bf16*>(a.y));
    }
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
  constexpr size_t lds = 2 * 2 * BT * KB;   // two stages; the epilogue takes at most 69 KB of it
  auto f = tile_kernel<WHOLE, CODES, YT>;
  const hipError_t e = ask_lds(f, lds, asked);
  if (e != hipSuccess) return e;
  const uint32_t rest = a.tiles_m * a.tiles_n - a.whole_tiles;
  hipLaunchKernelGGL(f, dim3(a.whole_tiles + rest * a.cut), dim3(256), lds, s, a);
  return hipGetLastError();
}

template <bool WHOLE, bool CODES>
hipError_t tile_type(const GemmI8& a, hipStream_t s) {
  return a.y_dtype == F32   ? launch_tile<WHOLE, CODES, F32>(a, s)
         : a.y_dtype == F16 ? launch_tile<WHOLE, CODES, F16>(a, s)
                            : launch_tile<WHOLE, CODES, BF16>(a, s);
}

template <int MB, int NB>
hipError_t launch_strip(const GemmI8& a, hipStream_t s) {
  constexpr int WAVES = MB * NB <= 4 ? 8 : 4;
  const dim3 grid((unsigned)((a.rows + 16 * NB - 1) / (16 * NB)), (unsigned)((a.m + 16 * MB - 1) / (16 * MB)));
  if (a.z) hipLaunchKernelGGL((strip_kernel<MB, NB, WAVES, true>), grid, dim3(64 * WAVES), 0, s, a);
  else hipLaunchKernelGGL((strip_kernel<MB, NB, WAVES, false>), grid, dim3(64 * WAVES), 0, s, a);
  return hipGetLastError();
}

template <int MB>
hipError_t strip(const GemmI8& a, int nb, hipStream_t s) {
  switch (nb) {
    case 1: return launch_strip<MB, 1>(a, s);
    case 2: return launch_strip<MB, 2>(a, s);
    case 3: return launch_strip<MB, 3>(a, s);
    default: return launch_strip<MB, 4>(a, s);
  }
}

hipError_t one(GemmI8 a, hipStream_t s) {
  // Whole rounds of 256 tiles, and the last round's tiles cut as long as it stays one round.
  const uint32_t tiles = a.tiles_m * a.tiles_n;
  a.whole_tiles = tiles / 256 * 256;
  const uint32_t rest = tiles - a.whole_tiles;
  a.cut = rest > 128 ? 1 : rest > 64 ? 2 : 4;
  if (a.m > 128 && tiles > kStripTiles) {
    // 16-byte units inside rows of whole words, and a tile inside 31-bit offsets
    const bool whole = a.d % 16 == 0 && reinterpret_cast<uintptr_t>(a.x) % 4 == 0 &&
                       reinterpret_cast<uintptr_t>(a.w) % 4 == 0 && a.ld_x % 4 == 0 && a.ld_w % 4 == 0 &&
                       std::max(a.ld_x, a.ld_w) < ((int64_t)1 << 22);
    if (whole) return a.z ? tile_type<true, true>(a, s) : tile_type<true, false>(a, s);
    return a.z ? tile_type<false, true>(a, s) : tile_type<false, false>(a, s);
  }
  // Strips as wide as leaves a workgroup to each CU: 16 NB outputs. Of as many blocks of 16 tokens as hold the call's, or
  // the next of 1, 2, 4, 6 and 8: with 4096 outputs of 4096 columns 48 tokens take the 10.5 us of 64, and 112 the 20 of
  // 128, so blocks of 3 and 7 would gain little; 96 take 14.0 in blocks of 6 and 20.1 in blocks of 8.
  const int64_t mb = (std::min<int64_t>(a.m, 128) + 15) / 16, chunks = (a.m + 127) / 128;
  const int nb = (int)std::min<int64_t>(4, std::max<int64_t>(1, ((a.rows + 15) / 16 * chunks + 255) / 256));
  if (mb <= 1) return strip<1>(a, nb, s);
  if (mb <= 2) return strip<2>(a, nb, s);
  if (mb <= 4) return strip<4>(a, nb, s);
  if (mb <= 6) return strip<6>(a, nb, s);
  return strip<8>(a, nb, s);
}

}  // namespace

hipError_t byte_gemm(const int8_t* x, int64_t m, int64_t ld_x, const float* xs, const void* w, int64_t ld_w,
                     const float* ws, const int32_t* z, int64_t rows, int64_t d, void* y, int y_dtype, int64_t ld_y,
                     hipStream_t s) {
  GemmI8 a{x, static_cast<const uint8_t*>(w), xs, ws, z, y, m, rows, ld_x, ld_w, ld_y, (int)d, y_dtype, 0, 0, 0, 0, 0};
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
