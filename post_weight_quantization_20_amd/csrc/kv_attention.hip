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
constexpr int64_t kMaxTokens = 0x7ffffc00;   // of a sequence: positions and tile ends stay in 32 bits

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
  r.len = clamp64(a.lens[s], 0, min((int64_t)a.c.max_pages * a.ps, kMaxTokens));
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

// ------------------------------------------------------------------ few queries: one pass over the cache
//
// The query heads that share a key head are packed rows of one tile: packed row r of a sequence is query
// r / group and head r % group, 16 rows a tile. A wave takes 32 keys at a time, straight from memory to its
// registers, and nothing but its own rows' statistics crosses lanes:
//   S^T = K Q^T          v_mfma_f32_16x16x32_f16, A = K (row l % 16 of 16 keys, bytes of its head widened to fp16),
//                        B = Q^T (column l % 16: a packed row); lane l then holds the scores of row l % 16 with
//                        keys 4 (l / 16) .. + 3 of each 16
//   O^T += V^T P^T       the same instruction over 32 keys: the probabilities are the B operand as they lie, and lane
//                        l reads V of the 8 keys that it holds scores of, VB bytes of each, whose columns become
//                        rows of VB products: bytes of two keys are put side by side while they are widened.
// A code c becomes fp16 exactly: byte c ^ 128 under the exponent of 1024 is 1152 + c, and 1152 is subtracted.
// Queries are scaled to [1, 2) by a power of two (fp16 ones are taken as they are); fp32 ones are two fp16 terms, and
// their probabilities too. A key block's scale multiplies its scores, a value block's its probabilities; those are
// kept in fp16's range by a power of two common to the wave that bounds all value scales seen so far.
//
// Workgroups share the work by keys: the tiles of 32 keys of all (sequence, key head, 16 rows) are one list, of which
// each takes an equal, contiguous part, whatever the lengths are. A part begins and ends anywhere; where it holds
// a whole unit the result is written at once, else a partial one, and a second kernel joins these in order.

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef _Float16 half2v __attribute__((ext_vector_type(2)));

constexpr int kRowTile = 16, kKeyTile = 32;
constexpr int kParts = 512;        // workgroups: two a CU
constexpr int kMinTiles = 8;       // key tiles that a workgroup takes at least
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kShift = 7.0f, kRaise = 8.0f;

struct FewArgs {
  KvArgs a;
  int parts;                       // > 0: workgroups that share the list by key tiles; 0: by whole units
  int64_t each;                    // parts = 0: units of a workgroup
  float *part_ml, *part_o;         // [parts][2][16][2] and [parts][2][16][dh]
};

GPTQ_DEV int32_t uniform(int32_t v) { return __builtin_amdgcn_readfirstlane(v); }
GPTQ_DEV int64_t uniform(int64_t v) {
  return (int64_t)((uint64_t)(uint32_t)uniform((int32_t)v) | (uint64_t)(uint32_t)uniform((int32_t)(v >> 32)) << 32);
}

// What a sequence contributes to the list: row tiles, its first key tile, key tiles of a unit.
struct Span {
  int64_t rows, units, tiles, tlo;
  GPTQ_DEV int64_t work(bool whole) const { return whole ? units : units * tiles; }
};

GPTQ_DEV Span span_of(const KvArgs& a, const Seq& q) {
  Span r;
  r.rows = (q.lq * a.group + kRowTile - 1) / kRowTile;
  r.units = r.rows * a.hk;
  const int64_t first = q.len - q.lq;   // the first query's position
  r.tlo = a.window ? clamp64(first - a.window + 1, 0, q.len) / kKeyTile : 0;
  r.tiles = (q.len + kKeyTile - 1) / kKeyTile - r.tlo;
  if (r.tiles < 1) r.tiles = 1;         // a unit without keys is there all the same: its rows are zeros
  return r;
}

// Sum of the list's entries before sequence s, for s given or, with at >= 0, for the sequence that holds entry
// `at` (s = -1: none does). One lane a sequence, 64 at a time.
GPTQ_DEV int64_t before_seq(const KvArgs& a, bool whole, int64_t at, int64_t& s, int lane) {
  int64_t before = 0;
  const int64_t stop = s;
  for (int64_t s0 = 0; s0 < a.seqs; s0 += 64) {
    const int64_t mine = s0 + lane;
    int64_t w = 0;
    if (mine < a.seqs && (at >= 0 || mine < stop)) w = span_of(a, sequence(a, mine)).work(whole);
    int64_t sum = w;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int64_t v = __shfl_up(sum, o, 64);
      if (lane >= o) sum += v;
    }
    if (at >= 0) {
      const uint64_t past = __ballot(before + sum > at);
      if (past) {
        const int l = __builtin_ctzll(past);
        s = s0 + l;
        return before + uniform(__shfl(sum, l, 64) - __shfl(w, l, 64));
      }
    } else if (s0 + 64 >= stop) {
      return before + uniform(__shfl(sum, 63, 64));
    }
    before += uniform(__shfl(sum, 63, 64));
  }
  if (at >= 0) s = -1;
  return before;
}

// Entries of each workgroup's part.
GPTQ_DEV int64_t part_size(int64_t total, int parts) {
  const int64_t n = (total + parts - 1) / parts;
  return n < kMinTiles ? kMinTiles : n;
}

GPTQ_DEV float load_q(const KvArgs& a, int dtype, int64_t at) { return load_as_f32(a.q, dtype, at); }

GPTQ_DEV half2v widen(uint32_t pair) {   // bytes c ^ 128 under the exponent of 1024
  return __builtin_bit_cast(half2v, pair) - half2v{(_Float16)1152.0f, (_Float16)1152.0f};
}

// Eight codes of consecutive columns.
GPTQ_DEV half8 widen8(uint32_t w0, uint32_t w1) {
  w0 ^= 0x80808080u;
  w1 ^= 0x80808080u;
  const half2v a = widen(__builtin_amdgcn_perm(0x64646464u, w0, 0x04010400u)),
               b = widen(__builtin_amdgcn_perm(0x64646464u, w0, 0x04030402u)),
               c = widen(__builtin_amdgcn_perm(0x64646464u, w1, 0x04010400u)),
               d = widen(__builtin_amdgcn_perm(0x64646464u, w1, 0x04030402u));
  return half8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// Byte b of two words side by side.
template <int B>
GPTQ_DEV half2v widen_pair(uint32_t x0, uint32_t x1) {
  return widen(__builtin_amdgcn_perm(x1, x0, 0x0c000c00u | (uint32_t)(4 + B) << 16 | (uint32_t)B) ^ 0x64806480u);
}

GPTQ_DEV floatx4 mfma32(half8 a, half8 b, floatx4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }

GPTQ_DEV float read_lane(float v, int l) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), l));
}

// DHP: the head padded to 64, 128 or 256 columns. KB: bytes a lane reads of a key at once. TERMS: fp16 terms of a
// query and a probability (two for fp32). ANY: caps and slopes.
template <int DHP, int KB, int TERMS, bool ANY>
__global__ __launch_bounds__(256, DHP <= 128 ? 2 : 1) void kv_few_kernel(FewArgs f, int dtype) {
  constexpr int NK = DHP / 32;                    // products of 32 columns
  constexpr int KL = DHP / (4 * KB);              // loads of a key tile's row of 16
  constexpr int VB = DHP == 64 ? 4 : 8, NU = DHP == 256 ? 2 : 1, NT = VB * NU;
  typedef uint32_t KUnit __attribute__((ext_vector_type(KB / 4), aligned(1)));
  typedef uint32_t VUnit __attribute__((ext_vector_type(VB / 4), aligned(1)));
  __shared__ float merge[2][4 * NT + 3][64];
  const KvArgs& a = f.a;
  const int lane = threadIdx.x & 63, wave = uniform((int32_t)(threadIdx.x >> 6));
  const int n = lane & 15, g = lane >> 4;
  const bool whole = f.parts == 0;
  const int dh = a.dh;

  int64_t s = a.seqs, pos, end;
  if (whole) {
    pos = (int64_t)blockIdx.x * f.each;
    end = pos + f.each;
  } else {
    const int64_t total = before_seq(a, false, -1, s, lane);
    const int64_t size = part_size(total, f.parts);
    pos = (int64_t)blockIdx.x * size;
    end = min(total, pos + size);
  }
  if (pos >= end) return;
  int64_t before = before_seq(a, whole, pos, s, lane);
  if (s < 0) return;

  // the lane's place in a key tile and in its rows
  const int kcol = KB * g;                        // of 4 KB columns a load
  const int64_t k_lane = n * a.c.k_tok + kcol, v_lane = 4 * g * a.c.v_tok + VB * n;

  while (true) {
    const Seq sq = sequence(a, s);
    const Span sp = span_of(a, sq);
    const int64_t at = pos - before;              // within the sequence's entries
    const int64_t unit = whole ? at : at / sp.tiles;
    const int64_t t0 = whole ? 0 : at - unit * sp.tiles;
    const int64_t t1 = whole ? sp.tiles : min(sp.tiles, t0 + (end - pos));
    const int kvh = uniform((int32_t)(unit / sp.rows));
    const int64_t row0 = uniform((unit - kvh * sp.rows) * kRowTile);

    // this lane's packed row
    const int64_t r = row0 + n;
    const bool live = r < sq.lq * a.group;
    const int64_t qi = live ? r / a.group : 0;
    const int h = kvh * a.group + (live ? (int)(r - qi * a.group) : 0);
    const int64_t p = qi + sq.len - sq.lq;
    const int32_t lim = !live ? 0x7fffffff : (int32_t)(a.causal ? clamp64(p + 1, 0, sq.len) : sq.len);
    const int32_t lo = live && a.window ? (int32_t)clamp64(p - a.window + 1, 0, sq.len) : 0;
    int32_t lim_min = lim, lo_max = lo, lim_max = live ? lim : 0;
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) {
      lim_min = min(lim_min, __shfl_xor(lim_min, o, 64));
      lim_max = max(lim_max, __shfl_xor(lim_max, o, 64));
      lo_max = max(lo_max, __shfl_xor(lo_max, o, 64));
    }
    lim_min = uniform(lim_min);
    lim_max = uniform(lim_max);
    lo_max = uniform(lo_max);

    // Q^T: 8 columns of the row for each product, in the order in which the keys' bytes lie
    half8 q[TERMS][NK];
    int qe = 0;                                   // queries are 2^qe larger than q
    {
      const int64_t q_at = (sq.q0 + qi) * a.q_ld + h * a.q_hp;
      float v[NK][8], top = 0.f;
#pragma unroll
      for (int ks = 0; ks < NK; ++ks) {
        const int c0 = KB == 16 ? 64 * (ks / 2) + 16 * g + 8 * (ks & 1) : 32 * ks + 8 * g;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          v[ks][e] = live && c0 + e < dh ? load_q(a, dtype, q_at + c0 + e) : 0.f;
          top = fmaxf(top, fabsf(v[ks][e]));
        }
      }
      if (dtype != F16) {
        top = fmaxf(top, __shfl_xor(top, 16, 64));
        top = fmaxf(top, __shfl_xor(top, 32, 64));
        if (top > 0.f && top < INFINITY) {
          qe = ilogbf(top);
#pragma unroll
          for (int ks = 0; ks < NK; ++ks)
#pragma unroll
            for (int i = 0; i < 8; ++i) v[ks][i] = ldexpf(v[ks][i], -qe);
        }
      }
#pragma unroll
      for (int ks = 0; ks < NK; ++ks)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          q[0][ks][i] = (_Float16)v[ks][i];
          if constexpr (TERMS == 2) q[1][ks][i] = (_Float16)(v[ks][i] - (float)q[0][ks][i]);
        }
    }
    const float slope = ANY && a.slopes ? a.slopes[h] : 0.f;

    floatx4 acc[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[t] = floatx4{0.f, 0.f, 0.f, 0.f};
    float m = -INFINITY, l = 0.f;
    int ve = -200;                                // value scales are below 2^ve

    // this wave's tiles: t0 + wave, + 4, ..., of which 32 at a time have their pages and scales in lanes
    const int64_t tfirst = sp.tlo + t0 + wave, tend = min(sp.tlo + t1, (int64_t)(lim_max + kKeyTile - 1) / kKeyTile);
    const int per_page = a.ps >> 4;
    for (int64_t tb = tfirst; tb < tend; tb += 4 * 32) {
      // lane 2 i + e: subtile e (16 keys) of the batch's tile i
      const int64_t sub = 2 * (tb + 4 * (lane >> 1)) + (lane & 1);
      int64_t page = -1;
      if (tb + 4 * (lane >> 1) < tend && 16 * sub < sq.len) {
        page = a.table[s * a.c.max_pages + sub / per_page];
        if (page >= a.c.pages) page = -1;
      }
      const uint64_t valid = __ballot(page >= 0);
      float ks = 0.f, vs = 0.f;
      if (page >= 0) {
        ks = a.c.k_scales[page * a.hk + kvh];
        vs = a.c.v_scales[page * a.hk + kvh];
      }
      const int32_t slot = (int32_t)(sub % per_page) * 16;
      {
        float top = fabsf(vs) < INFINITY ? fabsf(vs) : 0.f;
        top = wave_max(top);
        if (top > 0.f) {
          const int e = uniform((int32_t)ilogbf(top)) + 1;
          if (e > ve) {
            const float d = ldexpf(1.0f, max(ve - e, -200));
#pragma unroll
            for (int t = 0; t < NT; ++t) acc[t] *= d;
            ve = e;
          }
        }
        if (fabsf(vs) < INFINITY) vs = ldexpf(vs, -ve);
      }
      const int count = (int)min((int64_t)32, (tend - tb + 3) / 4);

      KUnit kx[2][KL];
      VUnit vx[8][NU];
      auto load = [&](int i) {
        // where one half of a tile has no page, the other's is read in its place; without both there is no tile
        const int both = (int)(valid >> (2 * i)) & 3;
        if (!both) return;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int from = 2 * i + ((both >> e) & 1 ? e : 1 - e);
          const int64_t pg = __builtin_amdgcn_readlane((int)page, from);
          const int64_t sl = __builtin_amdgcn_readlane(slot, from);
          const int8_t* kp = a.c.k + (pg * a.c.k_page + sl * a.c.k_tok + kvh * a.c.k_hp) + k_lane;
          const int8_t* vp = a.c.v + (pg * a.c.v_page + sl * a.c.v_tok + kvh * a.c.v_hp) + v_lane;
#pragma unroll
          for (int j = 0; j < KL; ++j)
            kx[e][j] = 4 * KB * j + kcol < dh ? *reinterpret_cast<const KUnit*>(kp + 4 * KB * j) : KUnit{};
#pragma unroll
          for (int b = 0; b < 4; ++b)
#pragma unroll
            for (int u = 0; u < NU; ++u)
              vx[4 * e + b][u] = 128 * u + VB * n < dh
                                     ? *reinterpret_cast<const VUnit*>(vp + b * a.c.v_tok + 128 * u)
                                     : VUnit{};
        }
      };
      load(0);
      for (int i = 0; i < count; ++i) {
        const int both = (int)(valid >> (2 * i)) & 3;
        if (!both) {
          if (i + 1 < count) load(i + 1);
          continue;
        }
        // this tile's operands out of the way of the next one's loads
        floatx4 S[2];
        uint32_t vw[8][NU][VB / 4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          S[e] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int k = 0; k < NK; ++k) {
            const half8 kf = KB == 16 ? widen8(kx[e][k / 2][2 * (k & 1)], kx[e][k / 2][2 * (k & 1) + 1])
                                      : widen8(kx[e][k][0], kx[e][k][1]);
#pragma unroll
            for (int t = 0; t < TERMS; ++t) S[e] = mfma32(kf, q[t][k], S[e]);
          }
        }
#pragma unroll
        for (int b = 0; b < 8; ++b)
#pragma unroll
          for (int u = 0; u < NU; ++u)
#pragma unroll
            for (int c = 0; c < VB / 4; ++c) vw[b][u][c] = vx[b][u][c];
        if (i + 1 < count) load(i + 1);

        const int32_t j0 = (int32_t)((tb + 4 * i) * kKeyTile);
        const int32_t jl = j0 + 4 * g;            // the key of register c of half e: jl + 16 e + c
        float mx = -INFINITY;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float fk = ldexpf(read_lane(ks, 2 * i + e) * (ANY ? a.scale : a.scale * kLog2e), qe);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            float x = S[e][c] * fk;
            if constexpr (ANY) {
              if (a.cap > 0.f) x = a.cap * tanhf(x / a.cap);
              x = __builtin_fmaf(-slope, fabsf((float)((int32_t)p - (jl + 16 * e + c))), x) * kLog2e;
            }
            S[e][c] = x;
          }
        }
        if (both != 3 || j0 + kKeyTile > lim_min || j0 < lo_max) {
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const int32_t j = jl + 16 * e + c;
              if (!((both >> e) & 1) || j >= lim || j < lo) S[e][c] = -INFINITY;
            }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int c = 0; c < 4; ++c) mx = fmaxf(mx, S[e][c]);
        if (__ballot(!(mx <= m + kRaise))) {
          mx = fmaxf(mx, __shfl_xor(mx, 16, 64));
          mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
          const float m2 = fmaxf(m, mx);
          const float d = m2 == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m - m2);
          m = m2;
          l *= d;
#pragma unroll
          for (int t = 0; t < NT; ++t) acc[t] *= d;
        }
        const float off = kShift - (m == -INFINITY ? 0.f : m);
        half8 w[TERMS];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float sv = read_lane(vs, 2 * i + e);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const float pr = __builtin_amdgcn_exp2f(S[e][c] + off);
            l += pr;
            const float x = S[e][c] == -INFINITY ? 0.f : pr * sv;   // a scale that is not a number stays unseen
            w[0][4 * e + c] = (_Float16)x;
            if constexpr (TERMS == 2) w[1][4 * e + c] = (_Float16)(x - (float)w[0][4 * e + c]);
          }
        }
#pragma unroll
        for (int u = 0; u < NU; ++u)
          static_for<0, VB>([&](auto bb) {
            constexpr int B = decltype(bb)::value;
            half8 vf;
#pragma unroll
            for (int pr = 0; pr < 4; ++pr) {
              const half2v x = widen_pair<B % 4>(vw[2 * pr][u][B / 4], vw[2 * pr + 1][u][B / 4]);
              vf[2 * pr] = x[0];
              vf[2 * pr + 1] = x[1];
            }
#pragma unroll
            for (int t = 0; t < TERMS; ++t) acc[u * VB + B] = mfma32(vf, w[t], acc[u * VB + B]);
          });
      }
    }
    l += __shfl_xor(l, 16, 64);
    l += __shfl_xor(l, 32, 64);

    // the four waves' results into the first: 2 and 3 into 0 and 1, then 1 into 0
    __syncthreads();                              // the area may still be read from the segment before
#pragma unroll
    for (int step = 0; step < 2; ++step) {
      const int from = 2 >> step;                 // waves from .. 2 from - 1 give
      if (wave >= from && wave < 2 * from) {
        float(*o)[64] = merge[wave - from];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int c = 0; c < 4; ++c) o[4 * t + c][lane] = acc[t][c];
        o[4 * NT][lane] = m;
        o[4 * NT + 1][lane] = l;
        o[4 * NT + 2][lane] = __builtin_bit_cast(float, ve);
      }
      __syncthreads();
      if (wave < from) {
        float(*o)[64] = merge[wave];
        const float m1 = o[4 * NT][lane], m2 = fmaxf(m, m1);
        const int e1 = __builtin_bit_cast(int, o[4 * NT + 2][lane]), e2 = max(ve, e1);
        const float f0 = m == -INFINITY && l == 0.f ? 0.f : __builtin_amdgcn_exp2f(m - m2);
        const float f1 = m1 == -INFINITY && o[4 * NT + 1][lane] == 0.f ? 0.f : __builtin_amdgcn_exp2f(m1 - m2);
        const float g0 = f0 * ldexpf(1.0f, max(ve - e2, -200)), g1 = f1 * ldexpf(1.0f, max(e1 - e2, -200));
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int c = 0; c < 4; ++c) acc[t][c] = acc[t][c] * g0 + o[4 * t + c][lane] * g1;
        l = l * f0 + o[4 * NT + 1][lane] * f1;
        m = m2;
        ve = e2;
      }
      if (step == 0) __syncthreads();
    }
    if (wave == 0 && live) {
      const float inv = l == 0.f ? 0.f : 1.0f / l;
      const bool complete = t0 == 0 && t1 == sp.tiles;
      float* po = nullptr;
      if (!complete) {
        // one part has at most one unit that it did not begin, and one more that it does not end
        const int64_t slot = ((int64_t)blockIdx.x * 2 + (t0 == 0 ? 1 : 0)) * kRowTile + n;
        if (g == 0) {
          f.part_ml[2 * slot] = m;
          f.part_ml[2 * slot + 1] = l;
        }
        po = f.part_o + slot * dh;
      }
      const int64_t o_at = (sq.q0 + qi) * a.o_ld + h * a.o_hp;
#pragma unroll
      for (int u = 0; u < NU; ++u)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int c0 = 128 * u + VB * (4 * g + c);
          if (c0 >= dh) continue;
          float o[VB];
#pragma unroll
          for (int b = 0; b < VB; ++b) o[b] = ldexpf(acc[u * VB + b][c] * inv, ve);
          auto put = [&](auto* dst) {
            typedef typename std::remove_pointer<decltype(dst)>::type T;
            typedef T Vec __attribute__((ext_vector_type(VB), aligned(sizeof(T))));
            Vec x;
#pragma unroll
            for (int b = 0; b < VB; ++b) x[b] = (T)o[b];
            *reinterpret_cast<Vec*>(dst) = x;
          };
          if (po) put(po + c0);
          else if (dtype == F32) put(static_cast<float*>(a.out) + o_at + c0);
          else if (dtype == F16) put(static_cast<_Float16*>(a.out) + o_at + c0);
          else put(static_cast<__bf16*>(a.out) + o_at + c0);
        }
    }
    // on to the next unit, in this sequence or the next that has any
    pos += whole ? 1 : t1 - t0;
    if (pos >= end) break;
    if (pos >= before + sp.work(whole)) {
      before += sp.work(whole);
      do {
        ++s;
      } while (s < a.seqs && span_of(a, sequence(a, s)).units == 0);
      if (s >= a.seqs) break;
    }
  }
}

// Joins the partial results of each unit that several workgroups shared: a workgroup a (query, head).
__global__ __launch_bounds__(256) void kv_join_kernel(FewArgs f, int dtype) {
  const KvArgs& a = f.a;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  __shared__ float part[4][256];
  int64_t all = a.seqs;
  const int64_t size = part_size(before_seq(a, false, -1, all, lane), f.parts);
  const int64_t total = a.nq * a.hq;
  for (int64_t it = blockIdx.x; it < total; it += gridDim.x) {
    const int64_t row = it / a.hq;
    const int h = (int)(it - row * a.hq), kvh = h / a.group;
    // the sequence that holds the row
    int64_t s = -1;
    if (!a.q_start) {
      s = row / a.lq_even;
    } else {
      for (int64_t s0 = 0; s0 < a.seqs && s < 0; s0 += 64) {
        bool in = false;
        if (s0 + lane < a.seqs) {
          const Seq q = sequence(a, s0 + lane);
          in = row >= q.q0 && row < q.q0 + q.lq;
        }
        const uint64_t b = __ballot(in);
        if (b) s = s0 + __builtin_ctzll(b);
      }
    }
    if (s < 0) continue;
    const Seq sq = sequence(a, s);
    const Span sp = span_of(a, sq);
    const int64_t before = before_seq(a, false, -1, s, lane);
    const int64_t r = (row - sq.q0) * a.group + (h - kvh * a.group);
    const int64_t u0 = before + (kvh * sp.rows + r / kRowTile) * sp.tiles, u1 = u0 + sp.tiles;
    const int64_t w0 = u0 / size, w1 = (u1 - 1) / size;
    if (w0 == w1) continue;                       // written by its one workgroup
    const int n = (int)(r % kRowTile);
    auto slot = [&](int64_t w) { return (2 * w + (w == w0 ? 1 : 0)) * kRowTile + n; };
    float m = -INFINITY;
    for (int64_t w = w0 + lane; w <= w1; w += 64)
      if (f.part_ml[2 * slot(w) + 1] != 0.f) m = fmaxf(m, f.part_ml[2 * slot(w)]);
    m = wave_max(m);
    float l = 0.f;
    for (int64_t w = w0 + lane; w <= w1; w += 64) {
      const float lw = f.part_ml[2 * slot(w) + 1];
      if (lw != 0.f) l += lw * __builtin_amdgcn_exp2f(f.part_ml[2 * slot(w)] - m);
    }
    l = wave_add(l);
    float o[4] = {0.f, 0.f, 0.f, 0.f};
    for (int64_t w = w0 + wave; w <= w1; w += 4) {
      const float lw = f.part_ml[2 * slot(w) + 1];
      if (lw == 0.f) continue;
      const float share = lw * __builtin_amdgcn_exp2f(f.part_ml[2 * slot(w)] - m) / l;
      const float* po = f.part_o + slot(w) * a.dh;
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (64 * c + lane < a.dh) o[c] = __builtin_fmaf(po[64 * c + lane], share, o[c]);
    }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < 4; ++c) part[wave][64 * c + lane] = o[c];
    __syncthreads();
    const int c = threadIdx.x;
    if (c < a.dh) {
      const float v = (part[0][c] + part[1][c]) + (part[2][c] + part[3][c]);
      const int64_t o_at = row * a.o_ld + h * a.o_hp + c;
      if (dtype == F32) static_cast<float*>(a.out)[o_at] = v;
      else if (dtype == F16) static_cast<_Float16*>(a.out)[o_at] = (_Float16)v;
      else static_cast<__bf16*>(a.out)[o_at] = (__bf16)v;
    }
  }
}

template <int DHP, int TERMS>
hipError_t launch_few(const FewArgs& f, int dtype, unsigned grid, hipStream_t s) {
  const bool any = f.a.cap > 0.f || f.a.slopes;
  if (f.a.dh % 16 != 0) hipLaunchKernelGGL((kv_few_kernel<DHP, 8, TERMS, true>), dim3(grid), dim3(256), 0, s, f, dtype);
  else if (any) hipLaunchKernelGGL((kv_few_kernel<DHP, 16, TERMS, true>), dim3(grid), dim3(256), 0, s, f, dtype);
  else hipLaunchKernelGGL((kv_few_kernel<DHP, 16, TERMS, false>), dim3(grid), dim3(256), 0, s, f, dtype);
  return hipGetLastError();
}

// The call's plan. Units: an upper bound on (sequence, key head, row tile).
struct Plan {
  bool few;
  int64_t units;
  int parts;
};

Plan plan(const gptq_kv_attention_t& t, const gptq_kv_cache_t& c) {
  Plan p{};
  p.few = c.head_dim <= 256 && c.head_dim % 8 == 0;
  if (!p.few) return p;
  const int64_t group = t.q_heads / c.kv_heads;
  p.units = (t.n_q * group / kRowTile + t.seqs) * c.kv_heads;
  // with four units a CU or more, a workgroup a unit fills the card by itself
  const int64_t most = std::min<int64_t>(t.seqs * (((int64_t)c.max_pages * c.page_size + kKeyTile - 1) / kKeyTile), (int64_t)1 << 40);
  p.parts = p.units >= 1024 || most <= kMinTiles ? 0 : kParts;
  return p;
}

}  // namespace

size_t kv_attention_workspace_bytes(const gptq_kv_attention_t& t, const gptq_kv_cache_t& c) {
  const Plan p = plan(t, c);
  return (size_t)p.parts * 2 * kRowTile * (c.head_dim + 2) * sizeof(float);
}

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
  const Plan p = plan(t, c);
  if (p.few) {
    FewArgs f{a, 0, 1, nullptr, nullptr};
    if (p.parts && work && work_bytes >= kv_attention_workspace_bytes(t, c)) {
      f.parts = p.parts;
      f.part_ml = static_cast<float*>(work);
      f.part_o = f.part_ml + (size_t)p.parts * 2 * kRowTile * 2;
    }
    // a grid holds fewer than 2^32 threads
    const int64_t most = (int64_t)1 << 22;
    f.each = (p.units + most - 1) / most;
    const unsigned grid = f.parts ? (unsigned)f.parts : (unsigned)((p.units + f.each - 1) / f.each);
    const bool two = t.dtype == F32;
    hipError_t e = a.dh <= 64    ? (two ? launch_few<64, 2>(f, t.dtype, grid, s) : launch_few<64, 1>(f, t.dtype, grid, s))
                   : a.dh <= 128 ? (two ? launch_few<128, 2>(f, t.dtype, grid, s) : launch_few<128, 1>(f, t.dtype, grid, s))
                                 : (two ? launch_few<256, 2>(f, t.dtype, grid, s) : launch_few<256, 1>(f, t.dtype, grid, s));
    if (e != hipSuccess || !f.parts) return e;
    hipLaunchKernelGGL(kv_join_kernel, dim3((unsigned)std::min<int64_t>(a.nq * a.hq, 65536)), dim3(256), 0, s, f, t.dtype);
    return hipGetLastError();
  }
  const int64_t waves = a.nq * a.hq;
  const dim3 grid((unsigned)std::min<int64_t>((waves + 3) / 4, 4096), (unsigned)std::min<int64_t>(t.seqs, 4096));
  if (t.dtype == F32) hipLaunchKernelGGL(kv_row_kernel<F32>, grid, dim3(256), 0, s, a);
  else if (t.dtype == F16) hipLaunchKernelGGL(kv_row_kernel<F16>, grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL(kv_row_kernel<BF16>, grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace gptq
