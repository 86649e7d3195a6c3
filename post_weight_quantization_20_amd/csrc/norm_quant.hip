// Residual addition, root-mean-square norm and int8 rows in one pass.
//
// For one row of d elements:
//   h_c = round_T(x_c + r_c)                                   (r optional; h is what the next layer adds to)
//   p_c = h_c w_c,   rho = 1 / sqrt(mean(h^2) + eps),   y_c = p_c rho
//   a = max |p|,   scale = a rho / 127,   q_c = rint(127 p_c / a)
// The norm's root cancels in q: a code is decided by products of inputs alone.
//
// The pass is bound by HBM: x and r are read once, h, q and a scale written once (7 bytes an element in 16 bits).
// A row stays in the registers of its lanes between the two sums and the rounding. The sum of squares is taken in 64
// bits, where squares of finite fp32 numbers neither overflow nor vanish. Products of 16-bit elements and weights are
// exact in fp32 within its range; others, and quotients that fp32 finds near a half, are formed in 64 bits, so that a
// code is the rounding of the exact quotient.
//
// Measured: 8192 rows of 4096 bf16 elements in 54 us, 4.3 TB/s (a copy: 5.1); 5003 fp32 rows of 11008 in 111 us, held up
// by the 64-bit products; 8 rows in 5.
#include "common.hpp"

namespace gptq {
namespace {

struct NormArgs {
  const void *x, *r, *w;
  void *sum, *y;
  int8_t* q;
  float* scales;
  int64_t n, x_ld, r_ld, sum_ld, y_ld, q_ld;
  int d, w_dtype;
  double eps;
};

constexpr int64_t kNormGroups = 2048;   // workgroups of 256 lanes

// The nearest whole number to 127 p / top, ties to even, for |p| <= top with inv near 127 / top: of the whole numbers k and
// k + 1 around the quotient, the nearer one by the sign of 254 |p| - (2 k + 1) top.
GPTQ_DEV int exact_code(double p, double top, double inv) {
  const double k = floor(fabs(p) * inv);
  const double side = __builtin_fma(-(2.0 * k + 1.0), top, 254.0 * fabs(p));
  const bool up = side > 0.0 || (side == 0.0 && ((int)k & 1));
  const int c = min((int)k + (up ? 1 : 0), 127);
  return p < 0.0 ? -c : c;
}

// Hides where a value comes from, so that what was formed from it before is not kept for later.
#define GPTQ_OPAQUE(x) \
  if constexpr (sizeof(x) >= 8) asm volatile("" : "+v"(x))

// A 64-bit number rounded to E once. For 16 bits it goes through fp32, where a result that is not exact takes the one of
// its two neighbours whose last bit is set (rounding to odd): that lies on no border of the shorter type.
template <typename E>
GPTQ_DEV E rounded(double v) {
  float f = (float)v;
  if constexpr (sizeof(E) < 4) {
    if ((double)f != v) {
      uint32_t b = __builtin_bit_cast(uint32_t, f);
      if (fabs((double)f) > fabs(v)) --b;
      f = __builtin_bit_cast(float, b | 1u);
    }
  }
  return (E)f;
}

// A weight in 64 bits, formed where it is used.
GPTQ_DEV double wide(float w) {
  asm volatile("" : "+v"(w));
  return (double)w;
}

// Weights of V columns from c on.
template <int V>
GPTQ_DEV void load_weights(const NormArgs& a, int c, float (&w)[V]) {
  auto read = [&](const auto* p) {
    typedef typename std::remove_cv<typename std::remove_pointer<decltype(p)>::type>::type E;
    typedef E Vec __attribute__((ext_vector_type(V), aligned(sizeof(E))));
    const Vec v = *reinterpret_cast<const Vec*>(p + c);
#pragma unroll
    for (int e = 0; e < V; ++e) w[e] = (float)v[e];
  };
  if (!a.w) {
#pragma unroll
    for (int e = 0; e < V; ++e) w[e] = 1.0f;
  } else if (a.w_dtype == F32) {
    read(static_cast<const float*>(a.w));
  } else if (a.w_dtype == F16) {
    read(static_cast<const _Float16*>(a.w));
  } else {
    read(static_cast<const __bf16*>(a.w));
  }
}

// T lanes take a row (256 / T rows a workgroup of 256 lanes), a lane C chunks of V elements. A workgroup goes through
// rows gridDim.x apart and loads the next one's while it works on one. A chunk that passes the row's end (d >= V) is
// read V columns before it, and its first elements, which the chunk before holds, count as zeros. KEEP: the weights stay in registers between
// rows; else they are read again, from the caches, for each sum and each rounding. SHORT: 16-bit weights with 16-bit
// elements, whose products fp32 holds exactly within its range.
template <int DT, int V, int T, int C, bool KEEP, bool SHORT>
__global__ __launch_bounds__(T < 256 ? 256 : T) void norm_quant_kernel(NormArgs a) {
  typedef typename ElemOf<DT>::T E;
  // accesses need no more than the element's alignment
  typedef E Vec __attribute__((ext_vector_type(V), aligned(sizeof(E))));
  typedef int8_t Codes __attribute__((ext_vector_type(V), aligned(1)));
  constexpr int RPW = T < 256 ? 256 / T : 1, WAVES = T / 64;
  const int sub = threadIdx.x % T;
  const int64_t step = (int64_t)gridDim.x * RPW;
  int64_t row = (int64_t)blockIdx.x * RPW + threadIdx.x / T;
  if (T < 256 && row >= a.n) return;   // no barrier follows for T = 64

  Vec xv[C], rv[C];
  auto column = [&](int i) { return min(V * (sub + i * T), a.d - V); };   // the first that is read
  auto load = [&](int64_t at) {
    const E* x = static_cast<const E*>(a.x) + at * a.x_ld;
    const E* r = a.r ? static_cast<const E*>(a.r) + at * a.r_ld : x;
#pragma unroll
    for (int i = 0; i < C; ++i) {
      xv[i] = *reinterpret_cast<const Vec*>(x + column(i));
      rv[i] = *reinterpret_cast<const Vec*>(r + column(i));
    }
  };
  // stores chunk i of a row: whole, or the elements that no other chunk holds
  auto store = [&](auto* row_p, int i, const auto& v) {
    int skip = V * (sub + i * T) - column(i);
    if (skip == 0) {
      __builtin_memcpy(row_p + column(i), &v, V * sizeof(*row_p));
    } else if (skip < V) {
      asm volatile("" : "+v"(skip));   // its comparisons belong here, not in registers over all rows
#pragma unroll
      for (int e = 1; e < V; ++e)
        if (e >= skip) row_p[column(i) + e] = v[e];
    }
  };
  float w[KEEP ? C : 1][V];
  load(row);
  if constexpr (KEEP) {
#pragma unroll
    for (int i = 0; i < C; ++i) load_weights<V>(a, column(i), w[i]);
  }
  __shared__ double part[3][2][WAVES];   // by rows in turn: one barrier a row
  int turn = 0;
  for (; row < a.n; row += step) {
    E* sum = a.sum ? static_cast<E*>(a.sum) + row * a.sum_ld : nullptr;
    Vec h[C];
    double ss = 0.0, top = 0.0, odd = 0.0;   // odd: zero, unless a product is not finite
    float top32 = 0.f, odd32 = 0.f;
#pragma unroll
    for (int i = 0; i < C; ++i) {
      if constexpr (!KEEP) load_weights<V>(a, column(i), w[0]);
      const float(&wi)[V] = w[KEEP ? i : 0];
#pragma unroll
      for (int e = 0; e < V; ++e) h[i][e] = a.r ? (E)((float)xv[i][e] + (float)rv[i][e]) : xv[i][e];
      if (sum) store(sum, i, h[i]);
      int skip = V * (sub + i * T) - column(i);
      if (skip) {
        asm volatile("" : "+v"(skip));
#pragma unroll
        for (int e = 0; e < V; ++e)
          if (e < skip) h[i][e] = (E)0.0f;
      }
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float hf = (float)h[i][e];
        const double hd = (double)hf;
        ss = __builtin_fma(hd, hd, ss);
        if constexpr (SHORT) {
          const float p = hf * wi[e];
          top32 = fmaxf(top32, fabsf(p));
          odd32 = __builtin_fmaf(p, 0.f, odd32);
        } else {
          const double p = hd * wide(wi[e]);
          top = fmax(top, fabs(p));
          odd = __builtin_fma(p, 0.0, odd);
        }
      }
    }
    if (row + step < a.n) load(row + step);
    // the row's sum and maximum
    auto reduce = [&](double& sum2, double& most) {
#pragma unroll
      for (int o = 32; o > 0; o >>= 1) {
        sum2 += __shfl_xor(sum2, o, 64);
        most = fmax(most, __shfl_xor(most, o, 64));
      }
      if constexpr (WAVES > 1) {
        if ((threadIdx.x & 63) == 0) {
          part[turn][0][threadIdx.x >> 6] = sum2;
          part[turn][1][threadIdx.x >> 6] = most;
        }
        // LDS alone: the next row's loads stay on their way
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        sum2 = part[turn][0][0];
        most = part[turn][1][0];
#pragma unroll
        for (int v = 1; v < WAVES; ++v) {
          sum2 += part[turn][0][v];
          most = fmax(most, part[turn][1][v]);
        }
        turn = turn == 2 ? 0 : turn + 1;
      }
    };
    if (SHORT ? !(odd32 == 0.f) : !(odd == 0.0)) top = INFINITY;
    else if (SHORT) top = (double)top32;
    reduce(ss, top);
    bool fast = top >= 0x1p-60 && top <= 0x1p60;   // products and quotients in fp32's range
    if (SHORT && !fast) {
      // products that fp32 does not hold, a row of zeros, or one that is not finite
      double none = 0.0;
      top = odd = 0.0;
#pragma unroll
      for (int i = 0; i < C; ++i) GPTQ_OPAQUE(h[i]);
#pragma unroll
      for (int i = 0; i < C; ++i) {
        if constexpr (!KEEP) load_weights<V>(a, column(i), w[0]);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const double p = (double)(float)h[i][e] * wide(w[KEEP ? i : 0][e]);
          top = fmax(top, fabs(p));
          odd = __builtin_fma(p, 0.0, odd);
        }
      }
      if (!(odd == 0.0)) top = INFINITY;
      reduce(none, top);
    }
    // what follows forms its products anew: kept from above they would fill the registers
#pragma unroll
    for (int i = 0; i < C; ++i) GPTQ_OPAQUE(h[i]);
    const bool finite = ss < INFINITY && top < INFINITY;   // false for NaN
    const double ms = ss / a.d + a.eps;
    const double rho = ms == 0.0 ? 0.0 : 1.0 / sqrt(ms);
    const bool some = finite && top > 0.0;
    const double inv = some ? 127.0 / top : 0.0;
    const float inv32 = (float)inv;
    if (a.q && sub == 0) a.scales[row] = finite ? (float)(top * rho / 127.0) : NAN;
    E* y = a.y ? static_cast<E*>(a.y) + row * a.y_ld : nullptr;
    int8_t* q = a.q ? a.q + row * a.q_ld : nullptr;
#pragma unroll
    for (int i = 0; i < C; ++i) {
      if constexpr (!KEEP) load_weights<V>(a, column(i), w[0]);
      const float(&wi)[V] = w[KEEP ? i : 0];
      // in fp32, whose three roundings are within 2.3e-5 of the quotient; exactly where that is near a half
      Codes k = {};
      bool near = some && !fast;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float t = (float)h[i][e] * wi[e] * inv32, n = rintf(t);
        near |= fabsf(t - n) > 0.4999f;
        k[e] = (int8_t)(int)(fast ? n : 0.f);
      }
      if (near) {
        GPTQ_OPAQUE(h[i]);
#pragma unroll
        for (int e = 0; e < V; ++e) k[e] = (int8_t)exact_code((double)(float)h[i][e] * wide(wi[e]), top, inv);
      }
      if (q) store(q, i, k);
      if (y) {
        Vec yv;
#pragma unroll
        for (int e = 0; e < V; ++e) yv[e] = rounded<E>((double)(float)h[i][e] * wide(wi[e]) * rho);
        store(y, i, yv);
      }
    }
  }
}

template <int DT, int V, int T, int C>
hipError_t launch(const NormArgs& a, hipStream_t s) {
  constexpr int RPW = T < 256 ? 256 / T : 1;
  // as many workgroups as run at once
  const int64_t groups = (a.n + RPW - 1) / RPW, most = kNormGroups * 256 / (T < 256 ? 256 : T);
  const dim3 grid((unsigned)std::min(groups, most)), wg(T < 256 ? 256 : T);
  constexpr bool KEEP = C * V <= 16;
  if (DT != F32 && (!a.w || a.w_dtype != F32))
    hipLaunchKernelGGL((norm_quant_kernel<DT, V, T, C, KEEP, DT != F32>), grid, wg, 0, s, a);
  else
    hipLaunchKernelGGL((norm_quant_kernel<DT, V, T, C, KEEP, false>), grid, wg, 0, s, a);
  return hipGetLastError();
}

// A wave a row up to 16 elements a lane (8 in fp32), then 256, 512 and 1024 lanes a row.
template <int DT>
hipError_t by_width(const NormArgs& a, hipStream_t s) {
  constexpr int V = DT == F32 ? 4 : 8;
  const int chunks = (a.d + V - 1) / V;
  if (a.d < V) return launch<DT, 1, 64, 1>(a, s);
  if (chunks <= 64) return launch<DT, V, 64, 1>(a, s);
  if (chunks <= 128) return launch<DT, V, 64, 2>(a, s);
  if (chunks <= 256) return launch<DT, V, 256, 1>(a, s);
  if (chunks <= 512) return launch<DT, V, 256, 2>(a, s);
  if (chunks <= 2 * 512) return launch<DT, V, 512, 2>(a, s);
  if (chunks <= 2 * 1024) return launch<DT, V, 1024, 2>(a, s);
  if (chunks <= 3 * 1024) return launch<DT, V, 1024, 3>(a, s);
  if (chunks <= 4 * 1024) return launch<DT, V, 1024, 4>(a, s);
  if constexpr (DT == F32)
    if (chunks > 8 * 1024) return launch<DT, V, 1024, 16>(a, s);
  return launch<DT, V, 1024, 8>(a, s);
}

}  // namespace

hipError_t norm_quant(const gptq_norm_quant_t& t, const void* x, const void* r, const void* w, void* sum, void* y,
                      int8_t* q, float* scales, hipStream_t s) {
  NormArgs a{};
  a.x = x; a.r = r; a.w = w; a.sum = sum; a.y = y; a.q = q; a.scales = scales;
  a.n = t.n; a.x_ld = t.x_ld; a.r_ld = t.r_ld; a.sum_ld = t.sum_ld; a.y_ld = t.y_ld; a.q_ld = t.q_ld;
  a.d = (int)t.d; a.w_dtype = t.w_dtype; a.eps = t.eps;
  return t.dtype == F32 ? by_width<F32>(a, s) : t.dtype == F16 ? by_width<F16>(a, s) : by_width<BF16>(a, s);
}

}  // namespace gptq
