// Softmax attention over packed sequences.
//
// Query i of a sequence with lq queries and lk keys stands at position p = i + lk - lq (the queries are
// the sequence's last tokens). Head h reads key and value head h / (hq / hk). For key j
//   s_j = scale q . k_j;  with a cap c: s_j = c tanh(s_j / c);  with a slope: s_j -= slope_h |p - j|
//   seen_j = (document of the query == document of j, and it is >= 0) and (j < prefix or not causal or j <= p)
//   o = sum over seen j of exp(s_j - M) v_j / sum of exp(s_j - M),  M = max of the seen s_j
// and o = 0 for a query that sees nothing. The running maximum, sum and output are fp32. A key that is
// not seen takes no part: whatever its k and v hold (infinities and NaN too) leaves o as it is.
#include "common.hpp"

#include <cmath>

namespace gptq {
namespace {

constexpr int kMaxHead = 1024;

struct AttnArgs {
  const void *q, *k, *v;
  void* out;
  int64_t q_ld, k_ld, v_ld, o_ld, q_hp, k_hp, v_hp, o_hp;
  int64_t seqs, nq, nk;
  int hq, hk, group, dh;
  int causal;
  float scale, cap;
  const int32_t *q_start, *kv_start, *q_doc, *kv_doc, *prefix;
  const float* slopes;
};

// The query and key ranges of a sequence. Offsets are clamped to the tokens there are.
struct Seq {
  int64_t q0, k0;
  int64_t lq, lk;
};

GPTQ_DEV int64_t clamp64(int64_t v, int64_t lo, int64_t hi) { return v < lo ? lo : v > hi ? hi : v; }

GPTQ_DEV Seq sequence(const AttnArgs& a, int64_t s) {
  Seq r;
  if (a.q_start) {
    r.q0 = clamp64(a.q_start[s], 0, a.nq);
    r.lq = clamp64(a.q_start[s + 1], r.q0, a.nq) - r.q0;
  } else {
    r.lq = a.nq / a.seqs;
    r.q0 = s * r.lq;
  }
  if (a.kv_start) {
    r.k0 = clamp64(a.kv_start[s], 0, a.nk);
    r.lk = clamp64(a.kv_start[s + 1], r.k0, a.nk) - r.k0;
  } else {
    r.lk = a.nk / a.seqs;
    r.k0 = s * r.lk;
  }
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

// One query and head by one wave, 64 keys at a time: a lane takes a key for the scores and columns
// lane, lane + 64, ... for the output. Only keys that are seen are read into the output.
template <int DT>
GPTQ_DEV void attn_row(const AttnArgs& a, const Seq& sq, int64_t s, int64_t i, int h, int lane) {
  typedef typename ElemOf<DT>::T T;
  const T* q = static_cast<const T*>(a.q) + (sq.q0 + i) * a.q_ld + h * a.q_hp;
  const T* kb = static_cast<const T*>(a.k) + sq.k0 * a.k_ld + (h / a.group) * a.k_hp;
  const T* vb = static_cast<const T*>(a.v) + sq.k0 * a.v_ld + (h / a.group) * a.v_hp;
  const int64_t p = i + sq.lk - sq.lq;
  const int64_t pre = a.prefix ? (int64_t)a.prefix[s] : 0;
  const int32_t doc = a.q_doc ? a.q_doc[sq.q0 + i] : 0;
  const float slope = a.slopes ? a.slopes[h] : 0.f;
  float m = -INFINITY, l = 0.f, acc[kMaxHead / 64];
#pragma unroll
  for (int c = 0; c < kMaxHead / 64; ++c) acc[c] = 0.f;
  int64_t end = a.causal ? (p + 1 > pre ? p + 1 : pre) : sq.lk;
  end = end > sq.lk ? sq.lk : end;
  for (int64_t j0 = 0; j0 < end; j0 += 64) {
    const int64_t j = j0 + lane;
    bool seen = j < end && (!a.causal || j <= p || j < pre);
    if (seen && a.q_doc) seen = doc >= 0 && a.kv_doc[sq.k0 + j] == doc;
    float sc = -INFINITY;
    if (seen) {
      float dot = 0.f;
      for (int c = 0; c < a.dh; ++c) dot = __builtin_fmaf((float)q[c], (float)kb[j * a.k_ld + c], dot);
      sc = dot * a.scale;
      if (a.cap > 0.f) sc = a.cap * tanhf(sc / a.cap);
      if (a.slopes) sc -= slope * fabsf((float)(p - j));
    }
    const float mn = fmaxf(m, wave_max(sc));
    const uint64_t any = __ballot(seen && !(sc == -INFINITY));
    if (!any) continue;
    const float w = seen ? expf(sc - mn) : 0.f;
    const float f = expf(m - mn);
    m = mn;
    l = l * f + wave_add(w);
#pragma unroll
    for (int c = 0; c < kMaxHead / 64; ++c) acc[c] *= f;
    const uint64_t vis = __ballot(seen);
    for (int e = 0; e < 64; ++e) {
      if (!((vis >> e) & 1)) continue;
      const float we = __shfl(w, e, 64);
      const T* vr = vb + (j0 + e) * a.v_ld;
#pragma unroll
      for (int c = 0; c < kMaxHead / 64; ++c)
        if (c * 64 + lane < a.dh) acc[c] = __builtin_fmaf(we, (float)vr[c * 64 + lane], acc[c]);
    }
  }
  T* o = static_cast<T*>(a.out) + (sq.q0 + i) * a.o_ld + h * a.o_hp;
#pragma unroll
  for (int c = 0; c < kMaxHead / 64; ++c)
    if (c * 64 + lane < a.dh) o[c * 64 + lane] = (T)(l == 0.f ? 0.f : acc[c] / l);
}

// Waves over (sequence, query, head).
template <int DT>
__global__ __launch_bounds__(256) void attn_row_kernel(AttnArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t s = blockIdx.y;
  const Seq sq = sequence(a, s);
  const int64_t items = sq.lq * a.hq;
  for (int64_t it = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); it < items; it += (int64_t)gridDim.x * 4)
    attn_row<DT>(a, sq, s, it / a.hq, (int)(it % a.hq), lane);
}

}  // namespace

size_t attention_workspace_bytes(const gptq_attention_t&) { return 0; }

hipError_t attention(const gptq_attention_t& t, const void* q, const void* k, const void* v, const int32_t* q_start,
                     const int32_t* kv_start, const float* slopes, const int32_t* q_doc, const int32_t* kv_doc,
                     const int32_t* prefix, void* out, void* work, size_t work_bytes, hipStream_t s) {
  (void)work;
  (void)work_bytes;
  AttnArgs a{};
  a.q = q; a.k = k; a.v = v; a.out = out;
  a.q_ld = t.q_ld; a.k_ld = t.k_ld; a.v_ld = t.v_ld; a.o_ld = t.out_ld;
  a.q_hp = t.q_hp; a.k_hp = t.k_hp; a.v_hp = t.v_hp; a.o_hp = t.out_hp;
  a.seqs = t.seqs; a.nq = t.n_q; a.nk = t.n_kv;
  a.hq = t.q_heads; a.hk = t.kv_heads; a.group = t.q_heads / t.kv_heads; a.dh = t.head_dim;
  a.causal = t.causal; a.scale = (float)t.scale; a.cap = (float)t.softcap;
  a.q_start = q_start; a.kv_start = kv_start; a.q_doc = q_doc; a.kv_doc = kv_doc; a.prefix = prefix;
  a.slopes = slopes;
  const int64_t waves = a.nq * a.hq;
  const dim3 grid((unsigned)std::min<int64_t>((waves + 3) / 4, 4096), (unsigned)t.seqs);
  if (t.dtype == F32) hipLaunchKernelGGL(attn_row_kernel<F32>, grid, dim3(256), 0, s, a);
  else if (t.dtype == F16) hipLaunchKernelGGL(attn_row_kernel<F16>, grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL(attn_row_kernel<BF16>, grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace gptq
