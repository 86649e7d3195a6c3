// Residual addition, root-mean-square norm and int8 rows in one pass.
//
// For one row of d elements:
//   h_c = round_T(x_c + r_c)                                   (r optional; h is what the next layer adds to)
//   p_c = h_c w_c,   rho = 1 / sqrt(mean(h^2) + eps),   y_c = p_c rho
//   a = max |p|,   scale = a rho / 127,   q_c = rint(127 p_c / a)
// The norm's root cancels in q: a code is decided by products of inputs alone.
//
// The pass is bound by HBM: x and r are read once, h, q and a scale written once (7 bytes an element in 16 bits).
// A row stays in the registers of its lanes between the two sums and the rounding. Sums, the maximum and the
// products are taken in 64 bits, whose rate is that of unpacked fp32 here: squares and products of finite fp32
// numbers neither overflow nor vanish there, and a code is the rounding of the exact quotient.
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

// The nearest whole number to 127 p / a, ties to even, for |p| <= a, with inv = 127 / a. The product with inv is
// within 2^-50 of the quotient, so only quotients that near a half are formed exactly.
GPTQ_DEV int code_of(double p, double a, double inv) {
  const double t = p * inv;
  double k = rint(t);
  if (__builtin_expect(fabs(fabs(t - k) - 0.5) < 1e-12, 0)) k = rint(p * 127.0 / a);
  return (int)k;
}

// Weights of V columns from c on; ones past the last.
template <int V>
GPTQ_DEV void load_weights(const NormArgs& a, int c, float (&w)[V]) {
  auto read = [&](const auto* p) {
    typedef typename std::remove_cv<typename std::remove_pointer<decltype(p)>::type>::type E;
    typedef E Vec __attribute__((ext_vector_type(V), aligned(sizeof(E))));
    if (c + V <= a.d) {
      const Vec v = *reinterpret_cast<const Vec*>(p + c);
#pragma unroll
      for (int e = 0; e < V; ++e) w[e] = (float)v[e];
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e) w[e] = c + e < a.d ? (float)p[c + e] : 1.0f;
    }
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

// T lanes take a row (256 / T rows a workgroup of 256 lanes, one of 1024), a lane C chunks of V elements.
template <int DT, int V, int T, int C>
__global__ __launch_bounds__(T < 256 ? 256 : T) void norm_quant_kernel(NormArgs a) {
  typedef typename ElemOf<DT>::T E;
  // accesses need no more than the element's alignment
  typedef E Vec __attribute__((ext_vector_type(V), aligned(sizeof(E))));
  typedef int8_t Codes __attribute__((ext_vector_type(V), aligned(1)));
  constexpr int RPW = T < 256 ? 256 / T : 1, WAVES = T / 64;
  const int sub = threadIdx.x % T;
  const int64_t row = (int64_t)blockIdx.x * RPW + threadIdx.x / T;
  if (T < 256 && row >= a.n) return;   // no barrier follows for T = 64
  const E* x = static_cast<const E*>(a.x) + row * a.x_ld;
  const E* r = a.r ? static_cast<const E*>(a.r) + row * a.r_ld : nullptr;
  E* sum = a.sum ? static_cast<E*>(a.sum) + row * a.sum_ld : nullptr;

  float h[C][V];
  Vec xv[C], rv[C];
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int c = V * (sub + i * T);
    xv[i] = Vec{};
    rv[i] = Vec{};
    if (c + V <= a.d) {
      xv[i] = *reinterpret_cast<const Vec*>(x + c);
      if (r) rv[i] = *reinterpret_cast<const Vec*>(r + c);
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e)
        if (c + e < a.d) {
          xv[i][e] = x[c + e];
          if (r) rv[i][e] = r[c + e];
        }
    }
  }
  double ss = 0.0, top = 0.0, odd = 0.0;   // odd: zero, unless a product is not finite
  float w[C][V];
#pragma unroll
  for (int i = 0; i < C; ++i) load_weights<V>(a, V * (sub + i * T), w[i]);
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int c = V * (sub + i * T);
    Vec s;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      s[e] = r ? (E)((float)xv[i][e] + (float)rv[i][e]) : xv[i][e];
      h[i][e] = (float)s[e];
      const double p = (double)h[i][e] * (double)w[i][e];
      ss = __builtin_fma((double)h[i][e], (double)h[i][e], ss);
      top = fmax(top, fabs(p));
      odd = __builtin_fma(p, 0.0, odd);
    }
    if (sum) {
      if (c + V <= a.d) {
        *reinterpret_cast<Vec*>(sum + c) = s;
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e)
          if (c + e < a.d) sum[c + e] = s[e];
      }
    }
  }
  if (!(odd == 0.0)) top = INFINITY;
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    ss += __shfl_xor(ss, o, 64);
    top = fmax(top, __shfl_xor(top, o, 64));
  }
  if constexpr (WAVES > 1) {
    __shared__ double part[2][WAVES];
    if ((threadIdx.x & 63) == 0) {
      part[0][threadIdx.x >> 6] = ss;
      part[1][threadIdx.x >> 6] = top;
    }
    __syncthreads();
    ss = part[0][0];
    top = part[1][0];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) {
      ss += part[0][w];
      top = fmax(top, part[1][w]);
    }
  }
  const bool finite = ss < INFINITY && top < INFINITY;   // false for NaN
  const double ms = ss / a.d + a.eps;
  const double rho = ms == 0.0 ? 0.0 : 1.0 / sqrt(ms);
  const bool some = finite && top > 0.0;
  const double inv = some ? 127.0 / top : 0.0;
  if (a.q && sub == 0) a.scales[row] = finite ? (float)(top * rho / 127.0) : NAN;
  E* y = a.y ? static_cast<E*>(a.y) + row * a.y_ld : nullptr;
  int8_t* q = a.q ? a.q + row * a.q_ld : nullptr;
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int c = V * (sub + i * T);
    Codes k;
    Vec yv;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const double p = (double)h[i][e] * (double)w[i][e];
      k[e] = (int8_t)(some ? code_of(p, top, inv) : 0);
      yv[e] = (E)(float)(p * rho);
    }
    if (c + V <= a.d) {
      if (q) *reinterpret_cast<Codes*>(q + c) = k;
      if (y) *reinterpret_cast<Vec*>(y + c) = yv;
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e)
        if (c + e < a.d) {
          if (q) q[c + e] = k[e];
          if (y) y[c + e] = yv[e];
        }
    }
  }
}

template <int DT, int V, int T, int C>
hipError_t launch(const NormArgs& a, hipStream_t s) {
  constexpr int RPW = T < 256 ? 256 / T : 1;
  // a launch takes at most 2^20 workgroups
  const int64_t step = (int64_t)RPW << 20;
  for (int64_t t = 0; t < a.n; t += step) {
    NormArgs b = a;
    b.n = std::min(step, a.n - t);
    constexpr int64_t esz = DT == F32 ? 4 : 2;
    b.x = static_cast<const char*>(a.x) + t * a.x_ld * esz;
    if (a.r) b.r = static_cast<const char*>(a.r) + t * a.r_ld * esz;
    if (a.sum) b.sum = static_cast<char*>(a.sum) + t * a.sum_ld * esz;
    if (a.y) b.y = static_cast<char*>(a.y) + t * a.y_ld * esz;
    if (a.q) {
      b.q = a.q + t * a.q_ld;
      b.scales = a.scales + t;
    }
    hipLaunchKernelGGL((norm_quant_kernel<DT, V, T, C>), dim3((unsigned)((b.n + RPW - 1) / RPW)),
                       dim3(T < 256 ? 256 : T), 0, s, b);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// A wave a row up to 16 elements a lane, then 256 lanes up to 32, then 1024.
template <int DT>
hipError_t by_width(const NormArgs& a, hipStream_t s) {
  constexpr int V = DT == F32 ? 4 : 8;
  const int chunks = (a.d + V - 1) / V;
  if (chunks <= 64) return launch<DT, V, 64, 1>(a, s);
  if (chunks <= 128) return launch<DT, V, 64, 2>(a, s);
  if (chunks <= 256) return launch<DT, V, 256, 1>(a, s);
  if (chunks <= 512) return launch<DT, V, 256, 2>(a, s);
  if (chunks <= 1024) return launch<DT, V, 256, 4>(a, s);
  if (chunks <= 2048) return launch<DT, V, 1024, 2>(a, s);
  if (chunks <= 4096) return launch<DT, V, 1024, 4>(a, s);
  if (chunks <= 8192) return launch<DT, V, 1024, 8>(a, s);
  return launch<DT, V, 1024, 64 / V>(a, s);
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
