// Per-head RMS norm of queries and keys with the position rotation in the same pass.
//
// For one head x of dh elements of one token:
//   y_c = x_c w_c / sqrt(mean(x^2) + eps)                     (the norm, optional; w optional)
//   pair i of the first rd columns, (a, b) = (i, i + rd/2) or (2i, 2i + 1):
//   out_a = y_a cos t - y_b sin t,  out_b = y_b cos t + y_a sin t,  t = pos[axis(i)][token] f_i
// and the columns from rd on are y itself. Sums, angles and products are fp32 or wider; the result
// is rounded once, to the type of x.
//
// The pass is bound by HBM: every element is read once and written once (about 7 flops each). A head
// is taken by a group of G lanes, and a lane holds a chunk of V elements from each side of V pairs, so
// that the norm's sum is a butterfly over G lanes and the rotation needs no exchange between lanes.
// The angles of a token are shared by all its heads: a workgroup takes a few whole tokens and keeps
// their (cos, sin) in LDS.
//
// A far position times a frequency loses its fraction of a turn in 32 bits (at 2^20 the product's
// rounding alone is 0.06 rad), so the angle is formed in 64 bits, in quarter turns, and only the
// remainder in [-1/2, 1/2] goes to fp32: half a step of it is at most 2^-26 quarter turns.
//
// Measured: 8192 tokens of 32 + 32 fp32 heads of 128 in 105 us, 65536 tokens of 32 + 8 bf16 heads in 276 us,
// 5.1 and 4.9 TB/s, which is what a copy of 2 GiB reaches; 8 tokens in 4.7 us.
#include "common.hpp"

namespace gptq {
namespace {

constexpr int kMaxChunks = 8;   // chunks of pairs a lane can hold: 1024-wide heads at V = 1, G = 64

struct RotArgs {
  const void *q, *k;
  void *qo, *ko;
  int64_t q_ld, k_ld, qo_ld, ko_ld, q_hp, k_hp, qo_hp, ko_hp;
  int64_t n;
  int hq, hk, dh, rd;
  int rot_chunks, chunks;      // chunks of V pairs among the rotated columns, and in all
  int interleaved, norm;
  float eps;
  const void *qw, *kw;
  int w_dtype;
  const int32_t* pos;          // axes rows of pitch pos_ld
  int64_t pos_ld;
  int axes;
  const float* inv_freq;       // rd / 2
  const int32_t* pair_axis;    // rd / 2, or null: axis 0
  int tokens_per_wg, heads_per_wg;
};

// cos and sin of pos * f
GPTQ_DEV float2 turn(int32_t pos, float f) {
  const double t = (double)pos * (double)f * 0.63661977236758134308;   // 2 / pi: quarter turns
  const double k = rint(t);
  const float r = (float)(t - k) * 0.5f;                               // half turns, in [-1/4, 1/4]
  float s = sinpif(r), c = cospif(r);
  const int quadrant = (int)((int64_t)k & 3);
  if (quadrant & 1) {
    const float o = s;
    s = c;
    c = -o;
  }
  if (quadrant & 2) {
    s = -s;
    c = -c;
  }
  return make_float2(c, s);
}

// Squares of fp32 overflow above 2^64 and lose their bits below 2^-63, in heads that are themselves finite and
// normal (bf16 has the same range). Where the mean with eps is below 2^-80 (from there on, what at most 1024
// squares lose, half of 2^-149 each, is under 2^-59 of it) or is not finite, the head is scaled first, by the
// power of two that takes the larger of its largest element and sqrt(eps) to 1..2: exact, and y = x / rms is
// the same for both. Returns the mean of the scaled squares plus the scaled eps. A head that holds an infinity or
// NaN, or nothing but zeros with eps = 0, is left as it was. The group's lanes come here together.
constexpr float kSmallMean = 0x1p-80f;

template <int G, int MC, int V>
GPTQ_DEV float rescale(float (&u)[MC][V], float (&v)[MC][V], float eps, float dh, float mean) {
  float top = sqrtf(eps);
#pragma unroll
  for (int m = 0; m < MC; ++m)
#pragma unroll
    for (int e = 0; e < V; ++e) top = fmaxf(top, fmaxf(fabsf(u[m][e]), fabsf(v[m][e])));
#pragma unroll
  for (int s = 1; s < G; s <<= 1) top = fmaxf(top, __shfl_xor(top, s, G));
  if (!(top > 0.f && top < INFINITY)) return mean;
  // within the exponents of normal fp32 numbers; elements below 2^-100 have squares in range at 2^100 times
  const int e = min(max(ilogbf(top), -100), 126);
  const float scale = ldexpf(1.0f, -e);
  float ss = 0.f;
#pragma unroll
  for (int m = 0; m < MC; ++m)
#pragma unroll
    for (int i = 0; i < V; ++i) {
      u[m][i] *= scale;
      v[m][i] *= scale;
      ss = __builtin_fmaf(u[m][i], u[m][i], ss);
      ss = __builtin_fmaf(v[m][i], v[m][i], ss);
    }
#pragma unroll
  for (int s = 1; s < G; s <<= 1) ss += __shfl_xor(ss, s, G);
  return ss / dh + eps * scale * scale;
}

// The workgroup takes tokens_per_wg tokens and heads_per_wg of their hq + hk heads (queries first).
// MC: chunks per lane.
template <int DT, int V, int G, int MC, bool WEIGHTS>
__global__ __launch_bounds__(256) void norm_rotate_kernel(RotArgs a) {
  typedef typename ElemOf<DT>::T T;
  typedef T Vec __attribute__((ext_vector_type(V)));
  extern __shared__ __align__(16) float smem[];
  // the weights of a query's and a key's columns, then the angles [tokens_per_wg][rd / 2]
  float* wl = smem;
  float2* cs = reinterpret_cast<float2*>(smem + (WEIGHTS ? 2 * ((a.dh + 3) & ~3) : 0));
  const int half = a.rd >> 1;
  const int64_t t0 = (int64_t)blockIdx.x * a.tokens_per_wg;
  const int nt = (int)min((int64_t)a.tokens_per_wg, a.n - t0);
  for (int i = threadIdx.x; i < nt * half; i += 256) {
    const int t = i / half, p = i - t * half;
    int ax = a.pair_axis ? a.pair_axis[p] : 0;
    ax = ax < 0 ? 0 : ax >= a.axes ? a.axes - 1 : ax;
    cs[i] = turn(a.pos[(int64_t)ax * a.pos_ld + t0 + t], a.inv_freq[p]);
  }
  if constexpr (WEIGHTS) {
    const int kb = (a.dh + 3) & ~3;
    for (int i = threadIdx.x; i < a.dh; i += 256) {
      wl[i] = a.qw ? load_as_f32(a.qw, a.w_dtype, i) : 1.0f;
      wl[kb + i] = a.kw ? load_as_f32(a.kw, a.w_dtype, i) : 1.0f;
    }
  }
  __syncthreads();

  const int sub = threadIdx.x % G;
  const int h0 = (int)blockIdx.y * a.heads_per_wg;
  const int nh = min(a.heads_per_wg, a.hq + a.hk - h0);
  const int items = nt * nh;
  int t = 0, hl = threadIdx.x / G;   // the item's token and head
  for (int it = hl; it < items; it += 256 / G, hl += 256 / G) {
    while (hl >= nh) {
      hl -= nh;
      ++t;
    }
    const int h = h0 + hl;
    const bool isq = h < a.hq;
    const int64_t tok = t0 + t;
    const T* x = isq ? static_cast<const T*>(a.q) + tok * a.q_ld + h * a.q_hp
                     : static_cast<const T*>(a.k) + tok * a.k_ld + (h - a.hq) * a.k_hp;
    T* o = isq ? static_cast<T*>(a.qo) + tok * a.qo_ld + h * a.qo_hp
               : static_cast<T*>(a.ko) + tok * a.ko_ld + (h - a.hq) * a.ko_hp;
    const float* w = wl + (isq ? 0 : (a.dh + 3) & ~3);
    float u[MC][V], v[MC][V];   // the two sides of the lane's pairs
    int ca[MC], cb[MC];         // their first columns (cb = dh: none)
    float ss = 0.f;
#pragma unroll
    for (int m = 0; m < MC; ++m) {
      const int c = sub + m * G;
      ca[m] = cb[m] = a.dh;
      if (c < a.chunks) {
        if (c < a.rot_chunks) {
          ca[m] = a.interleaved ? 2 * V * c : V * c;
          cb[m] = a.interleaved ? ca[m] + V : ca[m] + half;
        } else {
          ca[m] = a.rd + 2 * V * (c - a.rot_chunks);
          cb[m] = ca[m] + V;   // dh for the last column of an odd tail
        }
      }
      Vec xa = {}, xb = {};
      if (ca[m] < a.dh) xa = *reinterpret_cast<const Vec*>(x + ca[m]);
      if (cb[m] < a.dh) xb = *reinterpret_cast<const Vec*>(x + cb[m]);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        u[m][e] = (float)xa[e];
        v[m][e] = (float)xb[e];
        ss = __builtin_fmaf(u[m][e], u[m][e], ss);
        ss = __builtin_fmaf(v[m][e], v[m][e], ss);
      }
    }
    if (a.norm) {
#pragma unroll
      for (int s = 1; s < G; s <<= 1) ss += __shfl_xor(ss, s, G);
      float mean = ss / (float)a.dh + a.eps;
      if (!(mean >= kSmallMean && mean < INFINITY)) mean = rescale<G, MC, V>(u, v, a.eps, (float)a.dh, mean);
      const float r = 1.0f / sqrtf(mean);
#pragma unroll
      for (int m = 0; m < MC; ++m)
#pragma unroll
        for (int e = 0; e < V; ++e) {
          u[m][e] *= r;
          v[m][e] *= r;
          if constexpr (WEIGHTS) {
            if (ca[m] < a.dh) u[m][e] *= w[ca[m] + e];
            if (cb[m] < a.dh) v[m][e] *= w[cb[m] + e];
          }
        }
    }
#pragma unroll
    for (int m = 0; m < MC; ++m) {
      const int c = sub + m * G;
      if (c < a.rot_chunks) {
        const float2* r = cs + t * half + c * V;
        if (a.interleaved && V > 1) {
          // elements 2e, 2e + 1 of the lane's 2 V columns form a pair
#pragma unroll
          for (int e = 0; e < V; e += 2) {
            const float2 r0 = r[e / 2], r1 = r[V / 2 + e / 2];
            const float a0 = u[m][e], b0 = u[m][e + 1 < V ? e + 1 : e], a1 = v[m][e], b1 = v[m][e + 1 < V ? e + 1 : e];
            u[m][e] = a0 * r0.x - b0 * r0.y;
            u[m][e + 1 < V ? e + 1 : e] = b0 * r0.x + a0 * r0.y;
            v[m][e] = a1 * r1.x - b1 * r1.y;
            v[m][e + 1 < V ? e + 1 : e] = b1 * r1.x + a1 * r1.y;
          }
        } else {
#pragma unroll
          for (int e = 0; e < V; ++e) {
            const float2 rr = r[e];
            const float p = u[m][e], s = v[m][e];
            u[m][e] = p * rr.x - s * rr.y;
            v[m][e] = s * rr.x + p * rr.y;
          }
        }
      }
      Vec oa, ob;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        oa[e] = (T)u[m][e];
        ob[e] = (T)v[m][e];
      }
      if (ca[m] < a.dh) *reinterpret_cast<Vec*>(o + ca[m]) = oa;
      if (cb[m] < a.dh) *reinterpret_cast<Vec*>(o + cb[m]) = ob;
    }
  }
}

template <int DT, int V, int G, int MC>
hipError_t launch(const RotArgs& a, dim3 grid, hipStream_t s) {
  const size_t angles = (size_t)a.tokens_per_wg * (a.rd / 2) * sizeof(float2);
  if (a.qw || a.kw)
    hipLaunchKernelGGL((norm_rotate_kernel<DT, V, G, MC, true>), grid, dim3(256),
                       angles + 2 * ((a.dh + 3) & ~3) * sizeof(float), s, a);
  else
    hipLaunchKernelGGL((norm_rotate_kernel<DT, V, G, MC, false>), grid, dim3(256), angles, s, a);
  return hipGetLastError();
}

// The group: the smallest power of two of lanes, 2 .. 64, that covers the chunks, and more chunks a
// lane beyond 64 lanes.
template <int DT, int V>
hipError_t dispatch(RotArgs a, hipStream_t s) {
  a.rot_chunks = a.rd / (2 * V);
  a.chunks = a.rot_chunks + (a.dh - a.rd + 2 * V - 1) / (2 * V);
  int g = 2;
  while (g < a.chunks && g < 64) g *= 2;
  // Whole tokens for a workgroup, so that their angles are formed once; below 512 workgroups the
  // heads of a token are shared out instead (each workgroup then forms the angles it needs again; 8 tokens of
  // 40 heads: 5.0 us against 6.2).
  const int heads = a.hq + a.hk, slots = 256 / g;
  int tokens = std::max(1, (8 * slots) / heads);
  tokens = (int)std::min<int64_t>(tokens, std::max<int64_t>(1, a.n / 1024));
  tokens = std::max(1, std::min(tokens, 8192 / std::max(1, a.rd)));   // at most 32 KB of angles
  a.tokens_per_wg = tokens;
  a.heads_per_wg = heads;
  const int64_t wgs = (a.n + tokens - 1) / tokens;
  if (wgs < 512) a.heads_per_wg = std::min(heads, slots);
  const dim3 grid((unsigned)wgs, (unsigned)((heads + a.heads_per_wg - 1) / a.heads_per_wg));
  if (a.chunks <= 64) {
    switch (g) {
      case 2: return launch<DT, V, 2, 1>(a, grid, s);
      case 4: return launch<DT, V, 4, 1>(a, grid, s);
      case 8: return launch<DT, V, 8, 1>(a, grid, s);
      case 16: return launch<DT, V, 16, 1>(a, grid, s);
      case 32: return launch<DT, V, 32, 1>(a, grid, s);
      default: return launch<DT, V, 64, 1>(a, grid, s);
    }
  }
  if constexpr (V <= 4) return launch<DT, V, 64, kMaxChunks>(a, grid, s);   // 1024 / (2 * 64 * V) <= 8
  return hipErrorInvalidValue;
}

// The widest chunk that the columns, the pitches and the pointers allow.
template <int DT>
hipError_t by_width(const RotArgs& a, hipStream_t s) {
  constexpr int esz = DT == F32 ? 4 : 2, vmax = 16 / esz;
  auto fits = [&](int v) {
    if (a.rd % (2 * v) || (a.dh - a.rd) % (2 * v)) return false;
    auto ok = [&](const void* p, int64_t ld, int64_t hp) {
      return reinterpret_cast<uintptr_t>(p) % (v * esz) == 0 && ld % v == 0 && hp % v == 0;
    };
    if (a.hq && !(ok(a.q, a.q_ld, a.q_hp) && ok(a.qo, a.qo_ld, a.qo_hp))) return false;
    return !a.hk || (ok(a.k, a.k_ld, a.k_hp) && ok(a.ko, a.ko_ld, a.ko_hp));
  };
  if constexpr (vmax == 8)
    if (fits(8)) return dispatch<DT, 8>(a, s);
  if (fits(4)) return dispatch<DT, 4>(a, s);
  if (fits(2)) return dispatch<DT, 2>(a, s);
  return dispatch<DT, 1>(a, s);
}

}  // namespace

hipError_t norm_rotate(const gptq_norm_rotate_t& r, const void* q, const void* k, const void* qw, const void* kw,
                       const int32_t* pos, const float* inv_freq, const int32_t* pair_axis, void* qo, void* ko,
                       hipStream_t s) {
  RotArgs a{};
  a.q = q; a.k = k; a.qo = qo; a.ko = ko;
  a.q_ld = r.q_ld; a.k_ld = r.k_ld; a.qo_ld = r.q_out_ld; a.ko_ld = r.k_out_ld;
  a.q_hp = r.q_hp; a.k_hp = r.k_hp; a.qo_hp = r.q_out_hp; a.ko_hp = r.k_out_hp;
  a.n = r.n; a.hq = r.q_heads; a.hk = r.k_heads; a.dh = r.head_dim; a.rd = r.rotary_dim;
  a.interleaved = r.interleaved; a.norm = r.norm; a.eps = (float)r.eps;
  a.qw = qw; a.kw = kw; a.w_dtype = r.w_dtype;
  a.pos = pos; a.pos_ld = r.n; a.axes = r.axes; a.inv_freq = inv_freq; a.pair_axis = pair_axis;
  // a launch takes at most 2^22 tokens (a grid holds fewer than 2^32 threads)
  const int64_t esz = r.dtype == F32 ? 4 : 2, step = (int64_t)1 << 22;
  for (int64_t t0 = 0; t0 < r.n; t0 += step) {
    RotArgs b = a;
    b.n = std::min(step, r.n - t0);
    b.q = static_cast<const char*>(q) + t0 * a.q_ld * esz;
    b.qo = static_cast<char*>(qo) + t0 * a.qo_ld * esz;
    if (a.hk) {
      b.k = static_cast<const char*>(k) + t0 * a.k_ld * esz;
      b.ko = static_cast<char*>(ko) + t0 * a.ko_ld * esz;
    }
    if (pos) b.pos = pos + t0;
    const hipError_t e = r.dtype == F32 ? by_width<F32>(b, s) : r.dtype == F16 ? by_width<F16>(b, s) : by_width<BF16>(b, s);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace gptq
