// Keys, rotated by position, and values appended to a paged cache of 8-bit codes with one scale for each page
// and head.
//
// For the new tokens x_t of one (page, head), rotated as in rotate.hip where they are keys:
//   m = max |x|,  new scale s' = m / 127, or the larger of that and the scale s of tokens the page holds already
//   new codes rint(x / s') in [-127, 127];  earlier codes c become rint(c s / s') where s' > s
// so a page's codes always stand on one scale, and appending the same tokens again changes nothing.
//
// One wave owns a (page, head) of keys or of values: its two passes (maximum, rounding) need no exchange beyond
// the wave, and no other wave touches its codes or its scale. Angles of a page's tokens are formed once for the
// heads of a workgroup, in LDS. Angles and rotation are computed in 64 bits, and so is a quotient that fp32 finds near a
// half, so the code is the rounding of the exact quotient but for the last bits of 64.
//
// Measured: 8 bf16 prompts of 10.7 thousand tokens, 8 heads of 128, into pages of 16 in 61 us (71 MB: 14 us at a copy's
// rate), bound by about 50 vector instructions an element; one token of each of 32 sequences in 9 us.
#include "common.hpp"

namespace gptq {
namespace {

struct AppendArgs {
  gptq_kv_cache_t c;
  const void *k, *v;
  int64_t k_ld, k_hp, v_ld, v_hp;
  int64_t seqs, n, n_even;
  int rd, interleaved, axes;
  const int32_t *start, *past, *table, *pos, *pair_axis;
  const float* inv_freq;
  int ang_tokens;         // tokens whose angles LDS holds at a time
  int tasks_per_wg;       // of a unit's 2 kv_heads tasks, heads of keys and then of values
  int64_t unit0;          // first unit of the launch
};

constexpr int kWaves = 4;
constexpr int kKeep = 2;    // batches of 64 items that stay in registers between the passes

// Unit u of the call: the page `page` of sequence seq, and the sequence's rows in it.
struct Unit {
  int64_t page;      // in the pool, or -1
  int64_t row0;      // first new row of k and v
  int64_t t0;        // and its token
  int slot0, count;  // its slot, and the new tokens of the page
};

GPTQ_DEV int64_t clamp64(int64_t v, int64_t lo, int64_t hi) { return v < lo ? lo : v > hi ? hi : v; }

GPTQ_DEV Unit find_unit(const AppendArgs& a, int64_t u, int lane) {
  Unit r{-1, 0, 0, 0, 0};
  const int64_t cap = min((int64_t)a.c.max_pages * a.c.page_size, (int64_t)0x7ffffc00);
  int64_t before = 0;
  for (int64_t s0 = 0; s0 < a.seqs; s0 += 64) {
    const int64_t s = s0 + lane;
    int64_t row = 0, len = 0, past = 0;
    if (s < a.seqs) {
      if (a.start) {
        row = clamp64(a.start[s], 0, a.n);
        len = clamp64(a.start[s + 1], row, a.n) - row;
      } else {
        len = a.n_even;
        row = s * len;
      }
      past = clamp64(a.past[s], 0, cap);
      len = min(len, cap - past);
    }
    const int first = (int)(past / a.c.page_size);
    const int pages = len > 0 ? (int)((past + len - 1) / a.c.page_size) - first + 1 : 0;
    int64_t sum = pages;   // inclusive prefix sum over the lanes
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int64_t v = __shfl_up(sum, o, 64);
      if (lane >= o) sum += v;
    }
    const uint64_t at = __ballot(before + sum > u);
    if (at) {
      const int l = __builtin_ctzll(at);
      const int64_t mine = u - before - (__shfl(sum, l, 64) - __shfl(pages, l, 64));
      row = __shfl(row, l, 64);
      len = __shfl(len, l, 64);
      past = __shfl(past, l, 64);
      const int64_t b = __shfl(first, l, 64) + mine;
      const int64_t lo = max(past, b * a.c.page_size), hi = min(past + len, (b + 1) * a.c.page_size);
      r.page = a.table[(s0 + l) * a.c.max_pages + b];
      if (r.page < 0 || r.page >= a.c.pages) r.page = -1;
      r.row0 = row + (lo - past);
      r.t0 = lo;
      r.slot0 = (int)(lo - b * a.c.page_size);
      r.count = (int)(hi - lo);
      return r;
    }
    before += __shfl(sum, 63, 64);
  }
  return r;
}

// cos and sin of pos * f, to the last bits of 64: the angle less a whole number of quarter turns (pi / 2 in two
// parts, as Cody and Waite reduce it; products inside an fma are exact), then Taylor's polynomials on
// [-pi / 4, pi / 4], whose first terms left out are below 2^-58.
GPTQ_DEV double2 turn(int32_t pos, float f) {
  const double t = (double)pos * (double)f;
  const double k = rint(t * 0.63661977236758134308);   // 2 / pi
  const double r = __builtin_fma(-k, 6.123233995736766e-17, __builtin_fma(-k, 1.5707963267948966, t));
  const double z = r * r;
  double s = 1.0 / 355687428096000.0, c = 1.0 / 20922789888000.0;   // 1 / 17!, 1 / 16!
  s = __builtin_fma(s, z, -1.0 / 1307674368000.0);
  c = __builtin_fma(c, z, -1.0 / 87178291200.0);
  s = __builtin_fma(s, z, 1.0 / 6227020800.0);
  c = __builtin_fma(c, z, 1.0 / 479001600.0);
  s = __builtin_fma(s, z, -1.0 / 39916800.0);
  c = __builtin_fma(c, z, -1.0 / 3628800.0);
  s = __builtin_fma(s, z, 1.0 / 362880.0);
  c = __builtin_fma(c, z, 1.0 / 40320.0);
  s = __builtin_fma(s, z, -1.0 / 5040.0);
  c = __builtin_fma(c, z, -1.0 / 720.0);
  s = __builtin_fma(s, z, 1.0 / 120.0);
  c = __builtin_fma(c, z, 1.0 / 24.0);
  s = __builtin_fma(s, z, -1.0 / 6.0);
  c = __builtin_fma(c, z, -0.5);
  s = __builtin_fma(s * z, r, r);
  c = __builtin_fma(c, z, 1.0);
  const int quadrant = (int)((int64_t)k & 3);
  if (quadrant & 1) {
    const double o = s;
    s = c;
    c = -o;
  }
  if (quadrant & 2) {
    s = -s;
    c = -c;
  }
  return make_double2(c, s);
}

// Angles of nt tokens of the page from its tb-th new one on, by the whole workgroup.
GPTQ_DEV void make_angles(const AppendArgs& a, const Unit& u, int tb, int nt, double2* angles) {
  const int half = a.rd >> 1;
  __syncthreads();
  for (int i = threadIdx.x; i < nt * half; i += 64 * kWaves) {
    const int t = i / half, pr = i - t * half;
    int ax = a.pair_axis ? a.pair_axis[pr] : 0;
    ax = ax < 0 ? 0 : ax >= a.axes ? a.axes - 1 : ax;
    const int32_t ps = a.pos ? a.pos[(int64_t)ax * a.n + u.row0 + tb + t] : (int32_t)(u.t0 + tb + t);
    angles[i] = turn(ps, a.inv_freq[pr]);
  }
  __syncthreads();
}

// The nearest whole number to x / s, ties to even, in [-127, 127], with inv near 1 / s: of the whole numbers k and k + 1
// around the quotient, the nearer one by the sign of 2 |x| - (2 k + 1) s.
GPTQ_DEV int exact_code(double x, double s, double inv) {
  const double k = floor(fabs(x) * inv);
  const double side = __builtin_fma(-(2.0 * k + 1.0), s, 2.0 * fabs(x));
  const bool up = side > 0.0 || (side == 0.0 && ((int)k & 1));
  const int c = min((int)fmin(k, 127.0) + (up ? 1 : 0), 127);
  return x < 0.0 ? -c : c;
}

// Writes the new tokens of one (page, head). V: elements of a chunk on each side of V pairs. ready: LDS holds the angles
// of all the page's new tokens; else of ang_tokens at a time, and the workgroup's waves come here together (h past the
// last head: for the angles only).
template <int DT, int V, bool KEYS>
GPTQ_DEV void append_head(const AppendArgs& a, const Unit& u, int h, int lane, bool ready, double2* angles) {
  typedef typename ElemOf<DT>::T T;
  typedef T Vec __attribute__((ext_vector_type(V), aligned(sizeof(T))));
  typedef int8_t Codes __attribute__((ext_vector_type(V), aligned(1)));
  const int dh = a.c.head_dim, rd = KEYS ? a.rd : 0, half = rd >> 1;
  const int rot_chunks = rd / (2 * V), chunks = rot_chunks + (dh - rd + 2 * V - 1) / (2 * V);
  const int64_t ld = KEYS ? a.k_ld : a.v_ld;
  const T* x = static_cast<const T*>(KEYS ? a.k : a.v) + u.row0 * ld + h * (KEYS ? a.k_hp : a.v_hp);
  const int64_t tok = KEYS ? a.c.k_tok : a.c.v_tok;
  int8_t* cache = (KEYS ? a.c.k : a.c.v) + u.page * (KEYS ? a.c.k_page : a.c.v_page) + h * (KEYS ? a.c.k_hp : a.c.v_hp);
  float* scale = (KEYS ? a.c.k_scales : a.c.v_scales) + u.page * a.c.kv_heads + h;
  const bool mine = h < a.c.kv_heads;

  auto columns = [&](int c, int& ca, int& cb) {
    if (c < rot_chunks) {
      ca = a.interleaved ? 2 * V * c : V * c;
      cb = a.interleaved ? ca + V : ca + half;
    } else {
      ca = rd + 2 * V * (c - rot_chunks);
      cb = ca + V;   // dh for the last column of an odd tail
    }
  };
  // the two sides of chunk c of token t, rotated
  auto values = [&](int t, int c, double (&y)[V], double (&z)[V]) {
    int ca, cb;
    columns(c, ca, cb);
    const T* xr = x + t * ld;
    const Vec xa = *reinterpret_cast<const Vec*>(xr + ca);
    Vec xb = {};
    if (cb < dh) xb = *reinterpret_cast<const Vec*>(xr + cb);
    double p[V], q[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      y[e] = p[e] = (double)(float)xa[e];
      z[e] = q[e] = (double)(float)xb[e];
    }
    if (!KEYS || c >= rot_chunks) return;
    const double2* r = angles + (t % a.ang_tokens) * half + c * V;
    if (a.interleaved && V > 1) {
#pragma unroll
      for (int e = 0; e + 1 < V; e += 2) {
        const double2 r0 = r[e / 2], r1 = r[V / 2 + e / 2];
        y[e] = p[e] * r0.x - p[e + 1] * r0.y;
        y[e + 1] = p[e + 1] * r0.x + p[e] * r0.y;
        z[e] = q[e] * r1.x - q[e + 1] * r1.y;
        z[e + 1] = q[e + 1] * r1.x + q[e] * r1.y;
      }
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        y[e] = p[e] * r[e].x - q[e] * r[e].y;
        z[e] = q[e] * r[e].x + p[e] * r[e].y;
      }
    }
  };
  // Calls f(batch, token, chunk) for the lane's items. Values of up to kKeep batches stay in registers between the
  // passes, in fp32.
  const bool kept = u.count * chunks <= 64 * kKeep && (!KEYS || !rd || u.count <= a.ang_tokens);
  auto each = [&](bool again, auto&& f) {
    const int most = KEYS && rd ? a.ang_tokens : u.count;
    for (int tb = 0; tb < u.count; tb += most) {
      const int nt = min(most, u.count - tb);
      if (KEYS && rd && !ready && !(again && kept)) make_angles(a, u, tb, nt, angles);
      if (!mine) continue;
      if (kept) {
#pragma unroll
        for (int b = 0; b < kKeep; ++b) {
          const int it = 64 * b + lane;
          if (it < nt * chunks) f(b, it / chunks, it % chunks);
        }
      } else {
        for (int it = lane; it < nt * chunks; it += 64) f(0, tb + it / chunks, it % chunks);
      }
    }
  };

  float ky[kKeep][V], kz[kKeep][V];
  double top = 0.0;
  bool bad = false;   // a value is not finite
  each(false, [&](int b, int t, int c) {
    double y[V], z[V];
    values(t, c, y, z);
    float odd = 0.f;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      top = fmax(top, fmax(fabs(y[e]), fabs(z[e])));
      ky[b][e] = (float)y[e];
      kz[b][e] = (float)z[e];
      odd = __builtin_fmaf(ky[b][e], 0.f, __builtin_fmaf(kz[b][e], 0.f, odd));
    }
    if (!(odd == 0.f)) {   // rotated beyond fp32's largest number, or not finite at all
#pragma unroll
      for (int e = 0; e < V; ++e) bad |= !(fabs(y[e]) < INFINITY && fabs(z[e]) < INFINITY);
    }
  });
  if (bad) top = INFINITY;
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) top = fmax(top, __shfl_xor(top, o, 64));

  float sn = 0.f, so = 0.f;
  if (mine) {
    sn = top < INFINITY ? (float)(top / 127.0) : NAN;
    if (u.slot0 > 0) {
      so = *scale;
      if (!(so <= sn)) sn = sn != sn ? sn : so;   // the larger; NaN where either is
    }
  }
  const bool some = sn > 0.f && sn < INFINITY;
  const double sd = some ? (double)sn : 1.0, inv = some ? 1.0 / sd : 0.0;
  const float inv32 = (float)inv;
  const bool fast = sn >= 0x1p-100f && sn <= 0x1p100f;   // quotients in fp32's range
  each(true, [&](int b, int t, int c) {
    double y[V], z[V];
    if (!kept) {
      values(t, c, y, z);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        ky[b][e] = (float)y[e];
        kz[b][e] = (float)z[e];
      }
    }
    // in fp32, whose three roundings are within 2.3e-5 of the quotient; exactly where that is near a half
    Codes ka = {}, kb = {};
    bool near = some && !fast;
    if (fast) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float p = ky[b][e] * inv32, q = kz[b][e] * inv32, m = rintf(p), n = rintf(q);
        near |= fabsf(p - m) > 0.4999f || fabsf(q - n) > 0.4999f;
        ka[e] = (int8_t)(int)fminf(fmaxf(m, -127.f), 127.f);
        kb[e] = (int8_t)(int)fminf(fmaxf(n, -127.f), 127.f);
      }
    }
    if (near) {
      values(t, c, y, z);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        ka[e] = (int8_t)exact_code(y[e], sd, inv);
        kb[e] = (int8_t)exact_code(z[e], sd, inv);
      }
    }
    int ca, cb;
    columns(c, ca, cb);
    int8_t* o = cache + (u.slot0 + t) * tok;
    *reinterpret_cast<Codes*>(o + ca) = ka;
    if (cb < dh) *reinterpret_cast<Codes*>(o + cb) = kb;
  });
  if (!mine) return;
  if (u.slot0 > 0 && some && sn > so) {
    // four codes a lane where the head's width allows it
    if (dh % 4 == 0) {
      typedef int8_t C4 __attribute__((ext_vector_type(4), aligned(1)));
      const int quads = dh >> 2;
      for (int it = lane; it < u.slot0 * quads; it += 64) {
        C4* o = reinterpret_cast<C4*>(cache + (it / quads) * tok + 4 * (it % quads));
        C4 k = *o;
#pragma unroll
        for (int e = 0; e < 4; ++e) k[e] = (int8_t)exact_code((double)k[e] * (double)so, sd, inv);
        *o = k;
      }
    } else {
      for (int it = lane; it < u.slot0 * dh; it += 64) {
        int8_t* o = cache + (it / dh) * tok + it % dh;
        *o = (int8_t)exact_code((double)*o * (double)so, sd, inv);
      }
    }
  }
  if (lane == 0 && !(u.slot0 > 0 && sn == so)) *scale = sn;
}

// blockIdx.x: unit; blockIdx.y: a range of its tasks, heads of keys and then of values.
template <int DT, int VK, int VV>
__global__ __launch_bounds__(64 * kWaves) void append_kernel(AppendArgs a) {
  extern __shared__ __align__(16) double2 angles[];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, hk = a.c.kv_heads;
  const Unit u = find_unit(a, a.unit0 + blockIdx.x, lane);
  if (u.page < 0) return;   // the same for every wave
  const int t0 = blockIdx.y * a.tasks_per_wg, t1 = min(t0 + a.tasks_per_wg, 2 * hk);
  const bool ready = u.count <= a.ang_tokens || !a.rd;
  if (t0 < hk && !ready) {
    for (int h = t0; h < min(t1, hk); h += kWaves)
      append_head<DT, VK, true>(a, u, h + wave < min(t1, hk) ? h + wave : hk, lane, false, angles);
  } else if (t0 < hk && a.rd) {
    make_angles(a, u, 0, u.count, angles);
  }
  for (int t = (ready ? t0 : max(t0, hk)) + wave; t < t1; t += kWaves) {
    if (t < hk) append_head<DT, VK, true>(a, u, t, lane, true, angles);
    else append_head<DT, VV, false>(a, u, t - hk, lane, true, angles);
  }
}

template <int DT, int VK, int VV>
hipError_t launch(AppendArgs a, hipStream_t s) {
  const int64_t ps = a.c.page_size;
  // a sequence's rows touch at most one page each, and rows / page_size + 2 in all
  const int64_t units = std::min(a.n, a.n / ps + 2 * a.seqs);
  const int half = a.rd / 2;
  a.ang_tokens = half ? (int)std::max<int64_t>(1, std::min<int64_t>(ps, 4096 / half)) : (int)ps;   // 64 KB at most
  // All heads of a page in one workgroup, which finds its place and forms the angles once; with fewer pages than fill
  // the card they are shared out, down to a head of keys or values for each wave.
  const int tasks = 2 * a.c.kv_heads;
  const int64_t share = std::max<int64_t>(1, std::min<int64_t>((tasks + kWaves - 1) / kWaves, (1024 + units - 1) / units));
  a.tasks_per_wg = (int)((((tasks + kWaves - 1) / kWaves + share - 1) / share) * kWaves);
  const unsigned groups = (unsigned)((tasks + a.tasks_per_wg - 1) / a.tasks_per_wg);
  const size_t lds = std::max<size_t>(16, (size_t)(half ? a.ang_tokens * half : 0) * sizeof(double2));
  // a grid holds fewer than 2^32 threads along x
  const int64_t step = (int64_t)1 << 23;
  for (a.unit0 = 0; a.unit0 < units; a.unit0 += step) {
    hipLaunchKernelGGL((append_kernel<DT, VK, VV>), dim3((unsigned)std::min(step, units - a.unit0), groups),
                       dim3(64 * kWaves), lds, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// The widest chunks that the columns allow.
template <int DT, int VK>
hipError_t by_value(const AppendArgs& a, hipStream_t s) {
  const int dh = a.c.head_dim;
  if constexpr (DT != F32)
    if (dh % 16 == 0) return launch<DT, VK, 8>(a, s);
  if (dh % 8 == 0) return launch<DT, VK, 4>(a, s);
  return launch<DT, VK, 1>(a, s);
}

template <int DT>
hipError_t by_key(const AppendArgs& a, hipStream_t s) {
  const int dh = a.c.head_dim;
  auto fits = [&](int v) { return a.rd % (2 * v) == 0 && (dh - a.rd) % (2 * v) == 0; };
  if constexpr (DT != F32)
    if (fits(8)) return by_value<DT, 8>(a, s);
  if (fits(4)) return by_value<DT, 4>(a, s);
  return by_value<DT, 1>(a, s);
}

}  // namespace

hipError_t kv_append(const gptq_kv_append_t& t, const gptq_kv_cache_t& c, const void* k, const void* v,
                     const int32_t* start, const int32_t* past, const int32_t* table, const int32_t* pos,
                     const float* inv_freq, const int32_t* pair_axis, hipStream_t s) {
  AppendArgs a{};
  a.c = c; a.k = k; a.v = v;
  a.k_ld = t.k_ld; a.k_hp = t.k_hp; a.v_ld = t.v_ld; a.v_hp = t.v_hp;
  a.seqs = t.seqs; a.n = t.n; a.n_even = t.n / t.seqs;
  a.rd = t.rotary_dim; a.interleaved = t.interleaved; a.axes = t.axes;
  a.start = start; a.past = past; a.table = table; a.pos = pos; a.pair_axis = pair_axis; a.inv_freq = inv_freq;
  return t.dtype == F32 ? by_key<F32>(a, s) : t.dtype == F16 ? by_key<F16>(a, s) : by_key<BF16>(a, s);
}

}  // namespace gptq
