// Low-rank adapters of many requests beside a shared projection.
//
// Row i of x names adapter a = index[i]:  y_i = base_i + s_a B_a (A_a x_i),  A_a [r x d], B_a [rows x r];
// a row that names none takes base_i. Two launches: T = x A^T (shrink_kernel), y = base + s T B^T
// (expand_kernel). What the pass has to move is x, the adapters in use, base and y; at 2 r (d + rows) flops
// a row it is bound by those bytes, or by the two launches' latency for a few rows.
//
// Rows stay in their order (no sort): a workgroup takes 16 or more consecutive rows, lists the distinct
// adapters they name (its slots, in order of first row) and forms each slot's product for all its rows,
// keeping it for the rows that name the slot. Rows of one prompt share an adapter, so a tile has one or two
// slots; a batch of single tokens has up to 16, whose products are bound by reading the adapters and are
// shared out over waves (expand) and workgroups (shrink).
//
// shrink: 16-bit products on v_mfma_f32_16x16x32 (exact products, fp32 sums), fp32 ones on
// v_mfma_f32_16x16x4, operands straight from memory (both run along d). The d axis is split over the waves
// of a workgroup (joined in LDS in wave order) and, while there are few workgroups, over the grid; expand
// adds the grid's partial sums in order. expand: fp32 MFMA, so T is never rounded to 16 bits: with r <= 256
// the product is small beside y's bytes. Nothing depends on scheduling.
//
// Measured: 4096 bf16 rows of rank 64, 4096 x 11008, in 59 (shrink) + 50 us (expand), against 48 for the
// bytes: A, T and B come from L2 once per tile. 64 rows over 48 adapters of rank 16, 11008 x 4096, 5 + 13 us;
// 4 rows on 4 adapters, 4096 x 4096, 4 + 4 us.
#include "common.hpp"

namespace gptq {
namespace {

constexpr int EW = 4;   // waves of an expand workgroup

typedef short v8s __attribute__((ext_vector_type(8)));

struct LoraArgs {
  const void* x;
  int64_t ldx;
  int64_t m, d, rows;
  const void *A, *B;
  int64_t adapters;
  int rank;
  const int32_t *ranks, *index;
  const float* scales;
  const float* base;
  int64_t ldb;
  float* y;
  int64_t ldy;
  float* T;          // [ksplit][m][rp]
  int rp;            // rank rounded up to 16
  int ksplit;        // ranges of d over the grid
  int64_t kper;      // columns of a range, a multiple of 32
  int slot_groups;   // workgroups that share out a tile's slots (shrink)
  int64_t tile0;     // first row tile of the launch (expand)
  int xvec, bvec, yvec;
};

constexpr int64_t kPiece = (int64_t)1 << 19;   // rows taken at a time: the workspace holds one piece's T

GPTQ_DEV int rank_of(const LoraArgs& a, int64_t ad) {
  if (!a.ranks) return a.rank;
  const int r = a.ranks[ad];
  return r < 0 ? 0 : r > a.rank ? a.rank : r;
}

// The adapter of row i0 + lane, or -1 (past the tile or the rows, or none).
GPTQ_DEV int adapter_of(const LoraArgs& a, int64_t i0, int tile, int lane) {
  if (lane >= tile || i0 + lane >= a.m) return -1;
  const int ad = a.index[i0 + lane];
  return ad < 0 || ad >= a.adapters ? -1 : ad;
}

// Calls f(slot, adapter, rows) for the distinct adapters of a wave's lanes in order of first lane.
template <typename F>
GPTQ_DEV void each_slot(int ad, F&& f) {
  uint64_t left = __ballot(ad >= 0);
  for (int s = 0; left; ++s) {
    const int a = __builtin_amdgcn_readlane(ad, __builtin_ctzll(left));
    const uint64_t mine = __ballot(ad == a);
    f(s, a, mine);
    left &= ~mine;
  }
}

// Eight (16-bit types) or four (fp32) consecutive elements from column k of a row of n columns.
template <int DT> struct Frag;
template <> struct Frag<F16> { typedef v8s T; static constexpr int N = 8; };
template <> struct Frag<BF16> { typedef v8s T; static constexpr int N = 8; };
template <> struct Frag<F32> { typedef floatx4 T; static constexpr int N = 4; };

template <int DT, bool VEC>
GPTQ_DEV typename Frag<DT>::T load_frag(const void* row, int64_t k, int64_t n, bool ok) {
  typedef typename Frag<DT>::T V;
  typedef typename std::conditional<DT == F32, float, short>::type E;
  const E* p = static_cast<const E*>(row);
  V v = {};
  if (!ok) return v;
  if (VEC) {
    if (k < n) v = *reinterpret_cast<const V*>(p + k);
  } else {
#pragma unroll
    for (int e = 0; e < Frag<DT>::N; ++e)
      if (k + e < n) v[e] = p[k + e];
  }
  return v;
}

template <int DT>
GPTQ_DEV floatx4 dot_step(typename Frag<DT>::T a, typename Frag<DT>::T b, floatx4 c) {
  if constexpr (DT == F16) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8, a), __builtin_bit_cast(half8, b), c, 0, 0, 0);
  } else if constexpr (DT == BF16) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0,
                                                   0);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], b[e], c, 0, 0, 0);
    return c;
  }
}

// T of 16 MT rows for slots blockIdx.z, blockIdx.z + slot_groups, ... and range blockIdx.y of d; 16 NR ranks
// at a time. Lane l of the MFMA holds row l % 16 of x (and rank l % 16 of A) at 8 (or 4) columns of its
// quarter l / 16; it gets T of rank l % 16 and rows 4 (l / 16) .. + 3.
template <int DT, int MT, int NR, bool VEC>
__global__ __launch_bounds__(256) void shrink_kernel(LoraArgs a) {
  constexpr int KS = 4 * Frag<DT>::N;     // columns of a step
  __shared__ floatx4 part[3][MT][NR][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  // neighbouring tiles, which share adapters, on one XCD (workgroups go to the eight in turn)
  const int64_t per = gridDim.x >> 3;
  const int64_t tile = blockIdx.x < 8 * per ? (blockIdx.x & 7) * per + (blockIdx.x >> 3) : blockIdx.x;
  const int64_t i0 = tile * 16 * MT;
  const int ad = adapter_of(a, i0, 16 * MT, lane);
  const int esz = DT == F32 ? 4 : 2;
  const int l16 = lane & 15, quarter = lane >> 4;
  const char* xrow[MT];
  bool xok[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    const int64_t i = i0 + 16 * t + l16;
    xok[t] = i < a.m;
    xrow[t] = static_cast<const char*>(a.x) + (xok[t] ? i : 0) * a.ldx * esz;
  }
  // U steps' loads in flight at a time; the waves take such pieces of the range in turn, so that the
  // workgroup reads each row in long runs
  constexpr int U = 4, STEP = U * KS;
  const int64_t k0 = blockIdx.y * a.kper + wave * STEP;
  const int64_t k1 = min(a.d, (int64_t)(blockIdx.y + 1) * a.kper);
  float* T = a.T + (int64_t)blockIdx.y * a.m * a.rp;
  each_slot(ad, [&](int slot, int adapter, uint64_t mine) {
    if (slot % a.slot_groups != (int)blockIdx.z) return;
    const int r = rank_of(a, adapter);
    for (int n0 = 0; n0 < a.rank; n0 += 16 * NR) {
      floatx4 acc[MT][NR];
      const char* arow[NR];
      bool aok[NR];
#pragma unroll
      for (int n = 0; n < NR; ++n) {
        const int k = n0 + 16 * n + l16;
        aok[n] = k < r;
        arow[n] = static_cast<const char*>(a.A) + ((int64_t)adapter * a.rank + (aok[n] ? k : 0)) * a.d * esz;
#pragma unroll
        for (int t = 0; t < MT; ++t) acc[t][n] = floatx4{0.f, 0.f, 0.f, 0.f};
      }
      for (int64_t k = k0; k < k1; k += 4 * STEP) {
        typename Frag<DT>::T xf[U][MT], af[U][NR];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int64_t kk = k + u * KS + quarter * Frag<DT>::N;
#pragma unroll
          for (int t = 0; t < MT; ++t) xf[u][t] = load_frag<DT, VEC>(xrow[t], kk, k1, xok[t]);
#pragma unroll
          for (int n = 0; n < NR; ++n) af[u][n] = load_frag<DT, VEC>(arow[n], kk, k1, aok[n]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int n = 0; n < NR; ++n) acc[t][n] = dot_step<DT>(xf[u][t], af[u][n], acc[t][n]);
      }
      __syncthreads();   // the last partial sums have been read
      if (wave) {
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
          for (int n = 0; n < NR; ++n) part[wave - 1][t][n][lane] = acc[t][n];
      }
      __syncthreads();
      if (wave == 0) {
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
          for (int n = 0; n < NR; ++n) {
            floatx4 s = acc[t][n];
#pragma unroll
            for (int w = 0; w < 3; ++w) {
              const floatx4 o = part[w][t][n][lane];
#pragma unroll
              for (int e = 0; e < 4; ++e) s[e] += o[e];
            }
            // ranks past the adapter's are zero whatever x holds: an infinity times A's zeros is NaN here
            const int k = n0 + 16 * n + l16;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int row = 16 * t + 4 * quarter + e;
              if (k < a.rp && ((mine >> row) & 1)) T[(i0 + row) * a.rp + k] = aok[n] ? s[e] : 0.f;
            }
          }
      }
    }
  });
}

// N consecutive elements of a row of B, zeros from column r on.
template <int DT, int N>
using Piece = typename ElemOf<DT>::T __attribute__((ext_vector_type(N)));

template <int DT, int N>
GPTQ_DEV Piece<DT, N> load_b(const void* B, int64_t at, int k, int r, bool vec) {
  typedef typename ElemOf<DT>::T T;
  const T* p = static_cast<const T*>(B) + at + k;
  Piece<DT, N> v = {};
  if (vec && k + N <= r) {
    v = *reinterpret_cast<const Piece<DT, N>*>(p);
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (k + e < r) v[e] = p[e];
  }
  return v;
}

// y of 16 MT rows. SLOTS: the four waves share 16 NJ columns and take the tile's slots in turn (each row is
// written by the wave of its slot); otherwise each wave takes 16 NJ columns of its own and every slot. The
// MFMA's lane l holds B row (column of y) l % 16 and T row l % 16 at ranks 4 (l / 16) .. + 3, and gets four
// consecutive columns of y of row l % 16. AHEAD (SLOTS, B's rows one piece a lane, as ranks up to 16 or 32 are):
// B of all the wave's slots is loaded while T is formed, so that the slots' latencies are paid once (64 requests
// over 48 adapters of rank 16: 13.5 against 16 us).
template <int DT, int MT, int NJ, int KN, bool SLOTS, bool AHEAD>
__global__ __launch_bounds__(64 * EW) void expand_kernel(LoraArgs a) {
  extern __shared__ __align__(16) float ts[];   // [16 MT][rp + 4]
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int l16 = lane & 15, quarter = lane >> 4;
  const int64_t i0 = (a.tile0 + blockIdx.y) * 16 * MT;
  const int ad = adapter_of(a, i0, 16 * MT, lane);
  const floatx4 zero = {0.f, 0.f, 0.f, 0.f};
  const uint64_t with = __ballot(ad >= 0);   // rows with an adapter
  // base of this lane's rows and columns
  constexpr int64_t COLS = (SLOTS ? 1 : EW) * 16 * NJ;
  const int64_t j0 = blockIdx.x * COLS + (SLOTS ? 0 : wave * 16 * NJ);
  // base of the rows this wave writes, on its way while T is formed
  floatx4 o[MT][NJ];
  {
    int64_t owner = 0;   // the wave of this lane's row: its slot's, the first for rows without an adapter
    if (SLOTS)
      each_slot(ad, [&](int slot, int, uint64_t mine) {
        if ((mine >> l16) & 1) owner = slot % EW;
      });
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      const int64_t i = i0 + 16 * t + l16;
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const int64_t c = j0 + 16 * j + 4 * quarter;
        o[t][j] = zero;
        if (!a.base || i >= a.m || c >= a.rows || (SLOTS && owner != wave)) continue;
        const float* bp = a.base + i * a.ldb + c;
        if (a.yvec && c + 4 <= a.rows) {
          o[t][j] = *reinterpret_cast<const floatx4*>(bp);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (c + e < a.rows) o[t][j][e] = bp[e];
        }
      }
    }
  }
  // AHEAD: B of all the wave's slots is on its way too
  constexpr int MINE = AHEAD ? 16 * MT / EW : 1;   // slots of a wave at most
  int own[MINE];
  uint64_t own_rows[MINE];
  Piece<DT, KN> ahead_b[MINE][NJ];
  if constexpr (AHEAD) {
#pragma unroll
    for (int q = 0; q < MINE; ++q) own[q] = -1;
    each_slot(ad, [&](int slot, int adapter, uint64_t mine) {
#pragma unroll
      for (int q = 0; q < MINE; ++q)
        if (slot == EW * q + wave) {
          own[q] = adapter;
          own_rows[q] = mine;
        }
    });
#pragma unroll
    for (int q = 0; q < MINE; ++q)
      if (own[q] >= 0) {
        const int r = rank_of(a, own[q]);
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          const int64_t jr = min(j0 + 16 * j + l16, a.rows - 1);
          ahead_b[q][j] = load_b<DT, KN>(a.B, ((int64_t)own[q] * a.rows + jr) * a.rank, KN * quarter, r, a.bvec);
        }
      }
  }
  // T of the tile's rows, the ranges of d added in order, four ranks a thread and eight ranges at a time;
  // rows without an adapter (whose T is not written) are zero
  const int rp = a.rp, pitch = rp + 4, q4 = rp >> 2, pieces = 16 * MT * q4;
  for (int e = threadIdx.x; e < pieces; e += 64 * EW) {
    const int row = e / q4, k = 4 * (e - row * q4);
    floatx4 s = zero;
    if ((with >> row) & 1) {
      const float* p = a.T + (i0 + row) * rp + k;
      for (int z0 = 0; z0 < a.ksplit; z0 += 8) {
        floatx4 v[8];
#pragma unroll
        for (int z = 0; z < 8; ++z)
          v[z] = z0 + z < a.ksplit ? *reinterpret_cast<const floatx4*>(p + (int64_t)(z0 + z) * a.m * rp) : zero;
#pragma unroll
        for (int z = 0; z < 8; ++z)
#pragma unroll
          for (int c = 0; c < 4; ++c) s[c] += v[z][c];
      }
    }
    *reinterpret_cast<floatx4*>(ts + row * pitch + k) = s;
  }
  __syncthreads();

  if (j0 >= a.rows) return;
  auto store = [&](int t, int j, const floatx4& v, float scale, int64_t i) {
    const int64_t c = j0 + 16 * j + 4 * quarter;
    float* yp = a.y + i * a.ldy + c;
    floatx4 r = o[t][j];
#pragma unroll
    for (int e = 0; e < 4; ++e) r[e] = __builtin_fmaf(scale, v[e], r[e]);
    if (a.yvec && c + 4 <= a.rows) {
      *reinterpret_cast<floatx4*>(yp) = r;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (c + e < a.rows) yp[e] = r[e];
    }
  };

  if constexpr (AHEAD) {
    floatx4 t4[KN / 4];
#pragma unroll
    for (int c = 0; c < KN / 4; ++c) t4[c] = *reinterpret_cast<const floatx4*>(ts + l16 * pitch + KN * quarter + 4 * c);
#pragma unroll
    for (int q = 0; q < MINE; ++q)
      if (own[q] >= 0) {
        const float scale = rank_of(a, own[q]) == 0 ? 0.f : a.scales ? a.scales[own[q]] : 1.0f;
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          floatx4 s = zero;
#pragma unroll
          for (int e = 0; e < KN; ++e)
            s = __builtin_amdgcn_mfma_f32_16x16x4f32((float)ahead_b[q][j][e], t4[e / 4][e % 4], s, 0, 0, 0);
          if ((own_rows[q] >> l16) & 1) store(0, j, s, scale, i0 + l16);
        }
      }
  } else each_slot(ad, [&](int slot, int adapter, uint64_t mine) {
    if (SLOTS && slot % EW != wave) return;
    const int r = rank_of(a, adapter);
    const float scale = a.scales ? a.scales[adapter] : 1.0f;
    floatx4 acc[MT][NJ];
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int j = 0; j < NJ; ++j) acc[t][j] = zero;
    for (int k0 = 0; k0 < r; k0 += 4 * KN) {
      const int k = k0 + KN * quarter;
      Piece<DT, KN> b[NJ];
      floatx4 t4[MT][KN / 4];
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const int64_t jr = min(j0 + 16 * j + l16, a.rows - 1);
        b[j] = load_b<DT, KN>(a.B, ((int64_t)adapter * a.rows + jr) * a.rank, k, r, a.bvec);
      }
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int c = 0; c < KN / 4; ++c)
          t4[t][c] = *reinterpret_cast<const floatx4*>(ts + (16 * t + l16) * pitch + k + 4 * c);
#pragma unroll
      for (int e = 0; e < KN; ++e)
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
          for (int j = 0; j < NJ; ++j)
            acc[t][j] = __builtin_amdgcn_mfma_f32_16x16x4f32((float)b[j][e], t4[t][e / 4][e % 4], acc[t][j], 0, 0, 0);
    }
#pragma unroll
    for (int t = 0; t < MT; ++t)
      if ((mine >> (16 * t + l16)) & 1) {
#pragma unroll
        for (int j = 0; j < NJ; ++j) store(t, j, acc[t][j], r ? scale : 0.f, i0 + 16 * t + l16);
      }
  });
  // rows without an adapter
  if (SLOTS && wave != 0) return;
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    const int64_t i = i0 + 16 * t + l16;
    if (i < a.m && !((with >> (16 * t + l16)) & 1)) {
#pragma unroll
      for (int j = 0; j < NJ; ++j) store(t, j, zero, 0.f, i);
    }
  }
}

int padded_rank(int rank) { return (rank + 15) / 16 * 16; }

// How the call is laid out, from its sizes alone.
struct Plan {
  int mt_shrink, slot_groups, ksplit;
  int64_t kper;
};

Plan plan(int64_t m, int64_t d, int64_t adapters) {
  Plan p{};
  // Rows of a shrink tile: an adapter is read once per tile, so long runs take 32.
  p.mt_shrink = m >= 1024 ? 2 : 1;
  const int64_t tile = 16 * p.mt_shrink, tiles = (m + tile - 1) / tile;
  // Few tiles: a workgroup for each slot. Then d is split until there are about 512 workgroups, in ranges
  // of at least 512 columns (128 a wave).
  // Long inputs: workgroups for two slots of a tile, so that a tile where two prompts meet takes no longer.
  p.slot_groups = (int)std::min<int64_t>(tiles >= 64 ? 2 : std::min(tile, m), std::max<int64_t>(1, adapters));
  // A tile's slots are not known here and rows mostly share adapters: of the loaded ones at most four a tile count
  // as work, so that a prompt does not pay for adapters that no row names (1024 rows of one of 64 adapters, rank 64,
  // 11008 x 4096: 36 us, 76 with all of them counted and 33 with one loaded; single tokens over all 64 take
  // 386 and 380). Counting one a tile costs them more (429).
  const int64_t wgs = tiles >= 64 ? tiles : tiles * std::min(p.slot_groups, 4);
  p.ksplit = (int)std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(16, (512 + wgs - 1) / wgs), d / 512));
  p.kper = ((d + p.ksplit - 1) / p.ksplit + 127) / 128 * 128;
  p.ksplit = (int)((d + p.kper - 1) / p.kper);
  return p;
}

template <int DT, bool VEC>
hipError_t shrink(const LoraArgs& a, const Plan& p, hipStream_t s) {
  const int64_t tile = 16 * p.mt_shrink;
  const dim3 grid((unsigned)((a.m + tile - 1) / tile), (unsigned)a.ksplit, (unsigned)a.slot_groups);
  const int nr = a.rank <= 16 ? 1 : a.rank <= 32 ? 2 : 4;
#define GPTQ_SHRINK(MT, NR) hipLaunchKernelGGL((shrink_kernel<DT, MT, NR, VEC>), grid, dim3(256), 0, s, a)
  if (p.mt_shrink == 1) {
    if (nr == 1) GPTQ_SHRINK(1, 1);
    else if (nr == 2) GPTQ_SHRINK(1, 2);
    else GPTQ_SHRINK(1, 4);
  } else {
    if (nr == 1) GPTQ_SHRINK(2, 1);
    else if (nr == 2) GPTQ_SHRINK(2, 2);
    else GPTQ_SHRINK(2, 4);
  }
#undef GPTQ_SHRINK
  return hipGetLastError();
}

template <int DT, int MT, int NJ, int KN, bool SLOTS, bool AHEAD>
hipError_t launch_expand_k(const LoraArgs& a, hipStream_t s) {
  const int64_t cols = (SLOTS ? 1 : EW) * 16 * NJ;
  const size_t lds = (size_t)16 * MT * (a.rp + 4) * sizeof(float);
  // a grid holds fewer than 2^32 threads: very wide outputs take their row tiles in several launches
  const int64_t xs = (a.rows + cols - 1) / cols, tiles = (a.m + 16 * MT - 1) / (16 * MT);
  const int64_t step = std::min<int64_t>(65535, std::max<int64_t>(1, ((int64_t)1 << 23) / xs));
  for (int64_t t0 = 0; t0 < tiles; t0 += step) {
    LoraArgs b = a;
    b.tile0 = t0;
    hipLaunchKernelGGL((expand_kernel<DT, MT, NJ, KN, SLOTS, AHEAD>), dim3((unsigned)xs, (unsigned)std::min(step, tiles - t0)),
                       dim3(64 * EW), lds, s, b);
  }
  return hipGetLastError();
}

template <int DT, int MT, int NJ, bool SLOTS>
hipError_t launch_expand(const LoraArgs& a, hipStream_t s) {
  // B's rows 16 bytes a lane at a time where the padded rank is whole pieces of four lanes
  if constexpr (SLOTS) {
    // one piece a lane is the whole rank: a wave's slots are loaded at once
    if (a.rp == 16) return launch_expand_k<DT, MT, NJ, 4, true, true>(a, s);
    if constexpr (DT != F32)
      if (a.rp == 32) return launch_expand_k<DT, MT, NJ, 8, true, true>(a, s);
  }
  if constexpr (DT != F32)
    if (a.rp % 32 == 0) return launch_expand_k<DT, MT, NJ, 8, SLOTS, false>(a, s);
  return launch_expand_k<DT, MT, NJ, 4, SLOTS, false>(a, s);
}

template <int DT>
hipError_t run(const LoraArgs& a, const Plan& p, hipStream_t s) {
  hipError_t e = a.adapters == 0 ? hipSuccess : a.xvec ? shrink<DT, true>(a, p, s) : shrink<DT, false>(a, p, s);
  if (e != hipSuccess) return e;
  // Long inputs: 32 rows and 128 columns a workgroup. 4096 x 4096 outputs of rank 64 took 55 us with them (50
  // now), 62 with 64 rows (half B's reads, fewer waves a CU) and 66 with 256 columns (half T's reads). Few
  // rows: 16, slots over the waves, and narrow columns while a launch of wide ones has fewer than 512
  // workgroups (4 rows on 4096 columns: 4.2 us against 4.9; 64 on 11008: 21 against 13). The two meet near 256
  // rows (rank 16): runs of 60 on 4096 columns take 5.7 us in long tiles and 8.0 in short ones, single tokens
  // over 48 adapters on 11008 columns 40 and 37, 128 of them 28 and 21.
  if (a.m >= 256) return launch_expand<DT, 2, 2, false>(a, s);
  const int64_t wide = (a.rows + 63) / 64 * ((a.m + 15) / 16);
  return wide >= 512 ? launch_expand<DT, 1, 4, true>(a, s) : launch_expand<DT, 1, 1, true>(a, s);
}

}  // namespace

size_t lora_workspace_bytes(int64_t m, int64_t d, int64_t, int64_t adapters, int32_t rank) {
  m = std::min(m, kPiece);
  return (size_t)plan(m, d, adapters).ksplit * m * padded_rank(rank) * 4;
}

hipError_t lora_gemm(const void* x, int dtype, int64_t m, int64_t ldx, const void* A, const void* B,
                     const int32_t* ranks, const float* scales, int64_t adapters, int32_t rank, const int32_t* index,
                     int64_t rows, int64_t d, const float* base, int64_t ld_base, float* y, int64_t ldy, void* work,
                     hipStream_t s) {
  const Plan p = plan(std::min(m, kPiece), d, adapters);
  LoraArgs a{};
  a.x = x; a.ldx = ldx; a.m = m; a.d = d; a.rows = rows;
  a.A = A; a.B = B; a.adapters = adapters; a.rank = rank;
  a.rp = padded_rank(rank);
  a.ranks = ranks; a.index = index; a.scales = scales;
  a.base = base; a.ldb = ld_base; a.y = y; a.ldy = ldy;
  a.T = static_cast<float*>(work);
  a.ksplit = p.ksplit; a.kper = p.kper; a.slot_groups = p.slot_groups;
  // 16-byte loads of x and A, four or eight elements of B at a time, 16-byte accesses of base and y
  const int64_t esz = dtype == F32 ? 4 : 2, n = 16 / esz;
  auto at = [](const void* q, int64_t to) { return reinterpret_cast<uintptr_t>(q) % to == 0; };
  a.xvec = d % n == 0 && ldx % n == 0 && at(x, 16) && at(A, 16);
  const int64_t kn = dtype != F32 && a.rp % 32 == 0 ? 8 : 4;
  a.bvec = rank % kn == 0 && at(B, kn * esz);
  a.yvec = ldy % 4 == 0 && at(y, 16) && (!base || (ld_base % 4 == 0 && at(base, 16)));
  for (int64_t i0 = 0; i0 < m; i0 += kPiece) {
    LoraArgs b = a;
    b.m = std::min(kPiece, m - i0);
    b.x = static_cast<const char*>(x) + i0 * ldx * esz;
    b.index = index + i0;
    b.base = base ? base + i0 * ld_base : nullptr;
    b.y = y + i0 * ldy;
    const hipError_t e = dtype == F32 ? run<F32>(b, p, s) : dtype == F16 ? run<F16>(b, p, s) : run<BF16>(b, p, s);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace gptq
