// Softmax attention over a paged cache of 8-bit keys and values.
//
// Query i of a sequence with lq queries and len cached tokens stands at position p = i + len - lq. Key j lies in
// slot j % page_size of page table[j / page_size]; with the scales ks, vs of that page and key head
//   s_j = scale ks q . kc_j;  with a cap c: s_j = c tanh(s_j / c);  with a slope: s_j -= slope_h |p - j|
//   seen_j = (j <= p or not causal) and (p - j < window or no window) and the page is in the pool
//   o = sum over seen j of exp(s_j - M) vs vc_j / sum of exp(s_j - M),  M = max of the seen s_j
// and o = 0 for a query that sees nothing.
#include "common.hpp"

#include <cmath>

namespace gptq {
namespace {

constexpr int kMaxHead = 1024;

struct KvArgs {
  gptq_kv_cache_t c;
  const void* q;
  void* out;
  int64_t q_ld, q_hp, o_ld, o_hp;
  int64_t seqs, nq, lq_even;
  int hq, hk, group, dh, ps;
  int causal, window;
  float scale, cap;
  const int32_t *q_start, *lens, *table;
  const float* slopes;
};

struct Seq {
  int64_t q0, lq;
  int64_t len;
};

GPTQ_DEV int64_t clamp64(int64_t v, int64_t lo, int64_t hi) { return v < lo ? lo : v > hi ? hi : v; }

GPTQ_DEV Seq sequence(const KvArgs& a, int64_t s) {
  Seq r;
  if (a.q_start) {
    r.q0 = clamp64(a.q_start[s], 0, a.nq);
    r.lq = clamp64(a.q_start[s + 1], r.q0, a.nq) - r.q0;
  } else {
    r.lq = a.lq_even;
    r.q0 = s * r.lq;
  }
  r.len = clamp64(a.lens[s], 0, min((int64_t)a.c.max_pages * a.ps, (int64_t)0x7fffffff));
  return r;
}

GPTQ_DEV float wave_max(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o, 64));
  return v;
}

GPTQ_DEV float wave_add(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

// One query and head by one wave, 64 keys at a time: a lane takes a key for the scores and columns lane,
// lane + 64, ... of the output. Heads of any width and pitch. acc is the average of the values so far.
template <int DT>
__global__ __launch_bounds__(256) void kv_row_kernel(KvArgs a) {
  typedef typename ElemOf<DT>::T T;
  constexpr int NC = kMaxHead / 64;
  const int lane = threadIdx.x & 63;
  for (int64_t s = blockIdx.y; s < a.seqs; s += gridDim.y) {
    const Seq sq = sequence(a, s);
    const int32_t* table = a.table + s * a.c.max_pages;
    const int64_t items = sq.lq * a.hq;
    for (int64_t it = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); it < items; it += (int64_t)gridDim.x * 4) {
      const int64_t i = it / a.hq;
      const int h = (int)(it - i * a.hq), g = h / a.group;
      const int64_t p = i + sq.len - sq.lq;
      const T* q = static_cast<const T*>(a.q) + (sq.q0 + i) * a.q_ld + h * a.q_hp;
      const int64_t j1 = a.causal ? min(sq.len, p + 1) : sq.len;
      const int64_t j0 = a.window ? max((int64_t)0, p - a.window + 1) : 0;
      const float slope = a.slopes ? a.slopes[h] : 0.f;
      float acc[NC], m = -INFINITY, l = 0.f;
#pragma unroll
      for (int c = 0; c < NC; ++c) acc[c] = 0.f;
      for (int64_t jb = j0; jb < j1; jb += 64) {
        const int64_t j = jb + lane;
        bool seen = j < j1;
        int64_t page = 0;
        if (seen) {
          page = table[j / a.ps];
          seen = page >= 0 && page < a.c.pages;
        }
        float sc = -INFINITY, vs = 0.f;
        int64_t vat = 0;
        if (seen) {
          const int8_t* k = a.c.k + page * a.c.k_page + (j % a.ps) * a.c.k_tok + g * a.c.k_hp;
          float dot = 0.f;
          for (int c = 0; c < a.dh; ++c) dot = __builtin_fmaf((float)q[c], (float)k[c], dot);
          sc = dot * a.c.k_scales[page * a.hk + g] * a.scale;
          if (a.cap > 0.f) sc = a.cap * tanhf(sc / a.cap);
          if (a.slopes) sc -= slope * fabsf((float)(p - j));
          vs = a.c.v_scales[page * a.hk + g];
          vat = page * a.c.v_page + (j % a.ps) * a.c.v_tok;
        }
        if (!__ballot(seen && !(sc == -INFINITY))) continue;
        const float mn = fmaxf(m, wave_max(sc));
        const float w = seen ? expf(sc - mn) : 0.f;
        const float before = l * expf(m - mn);
        m = mn;
        l = before + wave_add(w);
        const float keep = before / l, share = w / l;
#pragma unroll
        for (int c = 0; c < NC; ++c) acc[c] *= keep;
        const uint64_t vis = __ballot(seen);
        for (int e = 0; e < 64; ++e) {
          if (!((vis >> e) & 1)) continue;
          const float we = __shfl(share, e, 64), ve = __shfl(vs, e, 64);
          const int8_t* v = a.c.v + __shfl(vat, e, 64) + g * a.c.v_hp;
#pragma unroll
          for (int c = 0; c < NC; ++c)
            if (c * 64 + lane < a.dh) acc[c] = __builtin_fmaf(we, ve * (float)v[c * 64 + lane], acc[c]);
        }
      }
      T* o = static_cast<T*>(a.out) + (sq.q0 + i) * a.o_ld + h * a.o_hp;
#pragma unroll
      for (int c = 0; c < NC; ++c)
        if (c * 64 + lane < a.dh) o[c * 64 + lane] = (T)(l == 0.f ? 0.f : acc[c]);
    }
  }
}

}  // namespace

size_t kv_attention_workspace_bytes(const gptq_kv_attention_t& t, const gptq_kv_cache_t& c) { return 0; }

hipError_t kv_attention(const gptq_kv_attention_t& t, const gptq_kv_cache_t& c, const void* q, const int32_t* q_start,
                        const int32_t* lens, const int32_t* table, const float* slopes, void* out, void* work,
                        size_t work_bytes, hipStream_t s) {
  KvArgs a{};
  a.c = c; a.q = q; a.out = out;
  a.q_ld = t.q_ld; a.q_hp = t.q_hp; a.o_ld = t.out_ld; a.o_hp = t.out_hp;
  a.seqs = t.seqs; a.nq = t.n_q; a.lq_even = t.n_q / t.seqs;
  a.hq = t.q_heads; a.hk = c.kv_heads; a.group = a.hq / a.hk; a.dh = c.head_dim; a.ps = c.page_size;
  a.causal = t.causal; a.window = t.window; a.scale = (float)t.scale; a.cap = (float)t.softcap;
  a.q_start = q_start; a.lens = lens; a.table = table; a.slopes = slopes;
  const int64_t waves = a.nq * a.hq;
  const dim3 grid((unsigned)std::min<int64_t>((waves + 3) / 4, 4096), (unsigned)std::min<int64_t>(t.seqs, 4096));
  if (t.dtype == F32) hipLaunchKernelGGL(kv_row_kernel<F32>, grid, dim3(256), 0, s, a);
  else if (t.dtype == F16) hipLaunchKernelGGL(kv_row_kernel<F16>, grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL(kv_row_kernel<BF16>, grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace gptq
