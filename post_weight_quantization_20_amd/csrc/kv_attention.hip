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
// A query's row is scaled by a power of two that brings its largest element to fp16's last but one octave (fp16 ones are
// taken as they are), so that its smaller elements stay above fp16's smallest steps: bf16 ones are exact down to 2^-31 of
// the largest. fp32 ones are two fp16 terms.
// Probabilities are two terms for every type: one of 11 bits moves an output by up to 2^-11 of sum p |v|, which is as
// much as its own rounding to fp16 and shows wherever values cancel. The second product costs 1 % for 16 tokens against
// caches of up to 8192, and 7 % for four chunks of 512 against up to 4096.
// A key block's scale multiplies its scores, a value block's its probabilities. The products are kept in fp16's range by
// a power of two a row, which bounds those of the keys that the row has seen, probability and scale together: neither a
// scale that a row does not see nor one that its probabilities make small takes bits from the others. (One power for
// the wave, of all scales that it loads, would save 4 % for the chunks, and loses rows whose scales are small.)
//
// Workgroups share the work by keys: the tiles of 32 keys of all (sequence, key head, 16 rows) are one list, of which
// each takes an equal, contiguous part, whatever the lengths are. A part begins and ends anywhere; where it holds
// a whole unit the result is written at once, else a partial one, and a second kernel joins these in order. A part costs
// about 8 us before its first key (lengths, pages, keys, one after another), so there are no more of them than run at
// once: 16 tokens against caches of up to 8192 take 54 us with 512 parts, 61 with 768, 81 with 2048.
//
// Measured there: 168 MB in 48 us with start and end, 3.5 TB/s, and the join 5; one token against 100003 keys 49 + 9; four
// chunks of 512 against up to 4096 in 419 us after one another, 384 with pauses, where every 16 rows read and widen K and
// V again.

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 half2v __attribute__((ext_vector_type(2)));

constexpr int kRowTile = 16, kKeyTile = 32;
constexpr int kParts = 512;        // workgroups: two a CU
constexpr int kMinTiles = 4;       // key tiles that a workgroup takes at least
constexpr float kLog2e = 1.44269504088896340736f;
// exp2(score - m + kShift), and its product with a value's scale in units of 2^ve, stay below 2^15 while a score passes m by
// no more than kRaise: kShift - m may round up by one where m is large.
constexpr float kShift = 7.0f, kRaise = 7.0f;
constexpr int kQueryExp = 14;      // a scaled row's largest element is in [2^14, 2^15)
constexpr int kNoExp = -1000;      // the exponent of a scale that is zero or not finite

struct FewArgs {
  KvArgs a;
  int parts;                       // > 0: workgroups that share the list by key tiles; 0: by whole units
  int64_t each;                    // parts = 0: units of a workgroup
  struct Head* head;               // [parts]: the unit that a part leaves to the next ones
  float *part_ml, *part_o;         // [parts][2][16][2] and [parts][2][16][dh]
};

// A unit that part w began and part `last` ends: its sequence's queries, its rows and key head.
struct Head {
  int64_t q0, lq, row0;
  int32_t kvh, last;               // last: -1 where part w leaves no unit
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

// The list's total, and for an entry the sequence that holds it (at.s = -1: none does) with the entries before it.
// One lane a sequence, 64 at a time.
struct At {
  int64_t s, before;
  Seq sq;
};

GPTQ_DEV int64_t prefix_sum(int64_t v, int lane) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int64_t x = __shfl_up(v, o, 64);
    if (lane >= o) v += x;
  }
  return v;
}

GPTQ_DEV int64_t lane_value(int64_t v, int l) {
  return (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)v, l) |
                   (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(v >> 32), l) << 32);
}

// entry(total) names the entry.
template <typename F>
GPTQ_DEV At find_entry(const KvArgs& a, bool whole, int lane, F&& entry) {
  At r{-1, 0, {}};
  Seq q{};
  int64_t w = 0, sum = 0, total = 0;
  for (int64_t s0 = 0; s0 < a.seqs; s0 += 64) {
    q = Seq{};
    w = 0;
    if (s0 + lane < a.seqs) {
      q = sequence(a, s0 + lane);
      w = span_of(a, q).work(whole);
    }
    sum = prefix_sum(w, lane);
    total += lane_value(sum, 63);
  }
  const int64_t at = entry(total);
  if (at < 0 || at >= total) return r;
  for (int64_t s0 = 0; s0 < a.seqs; s0 += 64) {
    if (a.seqs > 64) {   // else what the lanes hold is the list
      q = Seq{};
      w = 0;
      if (s0 + lane < a.seqs) {
        q = sequence(a, s0 + lane);
        w = span_of(a, q).work(whole);
      }
      sum = prefix_sum(w, lane);
    }
    const uint64_t past = __ballot(r.before + sum > at);
    if (past) {
      const int l = __builtin_ctzll(past);
      r.s = s0 + l;
      r.before += lane_value(sum, l) - lane_value(w, l);
      r.sq = Seq{lane_value(q.q0, l), lane_value(q.lq, l), lane_value(q.len, l)};
      return r;
    }
    r.before += lane_value(sum, 63);
  }
  return r;
}

// Entries of each workgroup's part.
GPTQ_DEV int64_t part_size(int64_t total, int parts) {
  const int64_t n = (total + parts - 1) / parts;
  return n < kMinTiles ? kMinTiles : n;
}

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
// query (two for fp32). ANY: caps and slopes.
template <int DHP, int KB, int TERMS, bool ANY>
__global__ __launch_bounds__(256, DHP <= 128 ? 2 : 1) void kv_few_kernel(FewArgs f, int dtype) {
  constexpr int NK = DHP / 32;                    // products of 32 columns
  constexpr int KL = DHP / (4 * KB);              // loads of a key tile's row of 16
  constexpr int VB = DHP == 64 ? 4 : 8, NU = DHP == 256 ? 2 : 1, NT = VB * NU;
  typedef uint32_t KUnit __attribute__((ext_vector_type(KB / 4), aligned(1)));
  typedef uint32_t VUnit __attribute__((ext_vector_type(VB / 4), aligned(1)));
  __shared__ float merge[4][4][VB][64], stats[4][3][64];
  const KvArgs& a = f.a;
  const int lane = threadIdx.x & 63, wave = uniform((int32_t)(threadIdx.x >> 6));
  const int n = lane & 15, g = lane >> 4;
  const bool whole = f.parts == 0;
  const int dh = a.dh;

  int64_t pos = 0, end = 0, size = 0;
  At at = find_entry(a, whole, lane, [&](int64_t total) {
    size = whole ? f.each : part_size(total, f.parts);
    pos = (int64_t)blockIdx.x * size;
    end = min(total, pos + size);
    return pos;
  });
  Head left{0, 0, 0, 0, -1};

  // the lane's columns in a key tile's rows (those past the head read the first ones, which meet zeros in Q)
  int64_t k_lane[KL];
#pragma unroll
  for (int j = 0; j < KL; ++j) {
    const int c = 4 * KB * j + KB * g;
    k_lane[j] = n * a.c.k_tok + (c < dh ? c : 0);
  }
  int64_t v_lane[NU];
#pragma unroll
  for (int u = 0; u < NU; ++u) {
    const int c = 128 * u + VB * n;               // past the head: columns of the output that are not stored
    v_lane[u] = 4 * g * a.c.v_tok + (c < dh ? c : 0);
  }

  while (at.s >= 0) {
    const int64_t s = at.s;
    const Seq sq = at.sq;
    const Span sp = span_of(a, sq);
    const int64_t in = pos - at.before;           // within the sequence's entries
    const int64_t unit = whole ? in : in / sp.tiles;
    const int64_t t0 = whole ? 0 : in - unit * sp.tiles;
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

    // Q^T: 8 columns of the row for each product, in the order in which the keys' bytes lie. Its loads, the pages'
    // and the first tile's are on their way together.
    constexpr int QW = TERMS == 2 ? 8 : 4;        // words of 8 columns: two terms are for fp32 alone
    typedef uint32_t QWords __attribute__((ext_vector_type(QW), aligned(TERMS == 2 ? 4 : 2)));
    QWords qw[NK];
    auto q_column = [&](int ks) { return KB == 16 ? 64 * (ks / 2) + 16 * g + 8 * (ks & 1) : 32 * ks + 8 * g; };
    {
      const char* base = static_cast<const char*>(a.q) + ((sq.q0 + qi) * a.q_ld + h * a.q_hp) * (QW / 2);
#pragma unroll
      for (int ks = 0; ks < NK; ++ks) {
        const int c0 = q_column(ks);
        qw[ks] = *reinterpret_cast<const QWords*>(base + (c0 < dh ? c0 : 0) * (QW / 2));
      }
    }
    const float slope = ANY && a.slopes ? a.slopes[h] : 0.f;

    // this wave's tiles: t0 + wave, + 4, ..., of which 32 at a time have their pages and scales in lanes
    const int32_t tfirst = (int32_t)(sp.tlo + t0) + wave,
                  tend = min((int32_t)(sp.tlo + t1), (int32_t)(((int64_t)lim_max + kKeyTile - 1) / kKeyTile));
    const uint32_t per_page = (uint32_t)a.ps >> 4;
    uint64_t valid = 0;
    int64_t k_at = 0, v_at = 0;
    float ks = 0.f, vm = 0.f;                     // value scale vm 2^vx, |vm| in [1/2, 1)
    int vx = kNoExp, count = 0;
    auto open = [&](int32_t tb) {
      // lane 2 i + e: subtile e (16 keys) of the batch's tile i
      const int32_t tile = tb + 4 * (lane >> 1);
      const uint32_t sub = 2 * (uint32_t)tile + (lane & 1), at_page = sub / per_page;
      int64_t page = -1;
      if (tile < tend && 16 * (int64_t)sub < sq.len) {
        page = a.table[s * a.c.max_pages + at_page];
        if (page >= a.c.pages) page = -1;
      }
      valid = __ballot(page >= 0);
      ks = vm = 0.f;
      if (page >= 0) {
        ks = a.c.k_scales[page * a.hk + kvh];
        vm = a.c.v_scales[page * a.hk + kvh];
      }
      // where one half of a tile has no page, the other's is read in its place; without both there is no tile
      const int64_t slot = (sub - at_page * per_page) * 16;
      k_at = page * a.c.k_page + slot * a.c.k_tok + kvh * a.c.k_hp;
      v_at = page * a.c.v_page + slot * a.c.v_tok + kvh * a.c.v_hp;
      const int64_t ko = __shfl_xor(k_at, 1, 64), vo = __shfl_xor(v_at, 1, 64);
      if (page < 0) {
        k_at = ko;
        v_at = vo;
      }
      count = min(32, (tend - tb + 3) / 4);
    };
    // Two tiles' bytes in registers: one on its way while the other is used.
    struct Tile {
      KUnit k[2][KL];
      VUnit v[8][NU];
    };
    auto load = [&](int i, Tile& x) {
      if (i >= count || !((int)(valid >> (2 * i)) & 3)) return;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int8_t* kp = a.c.k + lane_value(k_at, 2 * i + e);
        const int8_t* vp = a.c.v + lane_value(v_at, 2 * i + e);
#pragma unroll
        for (int j = 0; j < KL; ++j) x.k[e][j] = *reinterpret_cast<const KUnit*>(kp + k_lane[j]);
#pragma unroll
        for (int u = 0; u < NU; ++u)
#pragma unroll
          for (int b = 0; b < 4; ++b) x.v[4 * e + b][u] = *reinterpret_cast<const VUnit*>(vp + b * a.c.v_tok + v_lane[u]);
      }
    };
    Tile even, odd;
    if (tfirst < tend) {
      open(tfirst);
      load(0, even);
    }

    half8 q[TERMS][NK];
    int qe = 0;                                   // the row is q times 2^qe
    {
      float v[NK][8], top = 0.f;
#pragma unroll
      for (int k = 0; k < NK; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float x;
          if constexpr (TERMS == 2) {
            x = __builtin_bit_cast(float, (uint32_t)qw[k][e]);
          } else {
            const uint16_t w = (uint16_t)(qw[k][e / 2] >> (16 * (e & 1)));
            x = dtype == F16 ? (float)__builtin_bit_cast(_Float16, w) : bf16_bits_to_f32(w);
          }
          v[k][e] = live && q_column(k) < dh ? x : 0.f;
          top = fmaxf(top, fabsf(v[k][e]));
        }
      if (TERMS == 2 || dtype != F16) {
        top = fmaxf(top, __shfl_xor(top, 16, 64));
        top = fmaxf(top, __shfl_xor(top, 32, 64));
        if (top > 0.f && top < INFINITY) {
          qe = ilogbf(top) - kQueryExp;
#pragma unroll
          for (int k = 0; k < NK; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i) v[k][i] = ldexpf(v[k][i], -qe);
        }
      }
#pragma unroll
      for (int k = 0; k < NK; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          q[0][k][i] = (_Float16)v[k][i];
          if constexpr (TERMS == 2) q[1][k][i] = (_Float16)(v[k][i] - (float)q[0][k][i]);
        }
    }

    floatx4 acc[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[t] = floatx4{0.f, 0.f, 0.f, 0.f};
    float m = -INFINITY, l = 0.f;                 // of the row: the scores' maximum and sum
    float mt = -INFINITY;                         // and that of score - m + exponent of the value's scale
    int ve = 0;                                   // ceil(mt): acc is in units of 2^ve

    for (int32_t tb = tfirst; tb < tend;) {
      vx = kNoExp;
      if (vm != 0.f && fabsf(vm) < INFINITY) {
        vx = ilogbf(vm) + 1;
        vm = ldexpf(vm, -vx);
      }
      auto compute = [&](int i, const Tile& x) {
        const int both = (int)(valid >> (2 * i)) & 3;
        if (i >= count || !both) return;
        floatx4 S[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          S[e] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int k = 0; k < NK; ++k) {
            const half8 kf = KB == 16 ? widen8(x.k[e][k / 2][2 * (k & 1)], x.k[e][k / 2][2 * (k & 1) + 1])
                                      : widen8(x.k[e][k][0], x.k[e][k][1]);
#pragma unroll
            for (int t = 0; t < TERMS; ++t) S[e] = mfma32(kf, q[t][k], S[e]);
          }
        }
        const int32_t j0 = (int32_t)((tb + 4 * i) * kKeyTile);
        const int32_t jl = j0 + 4 * g;            // the key of register c of half e: jl + 16 e + c
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
        int sx[2];
        float ms[2], mx = -INFINITY, tx = -INFINITY;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          sx[e] = __builtin_amdgcn_readlane(vx, 2 * i + e);
          ms[e] = fmaxf(fmaxf(S[e][0], S[e][1]), fmaxf(S[e][2], S[e][3]));
          mx = fmaxf(mx, ms[e]);
          tx = fmaxf(tx, (ms[e] - m) + (float)sx[e]);   // in this order: a large score has no room for an exponent
        }
        if (__ballot(!(mx <= m + kRaise && tx <= mt + kRaise))) {
          mx = fmaxf(mx, __shfl_xor(mx, 16, 64));
          mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
          const float m2 = fmaxf(m, mx);
          tx = fmaxf((ms[0] - m2) + (float)sx[0], (ms[1] - m2) + (float)sx[1]);
          tx = fmaxf(tx, __shfl_xor(tx, 16, 64));
          tx = fmaxf(tx, __shfl_xor(tx, 32, 64));
          if (m2 != -INFINITY) {
            const float dm = m - m2;
            mt = fmaxf(mt + dm, tx);
            const int ve2 = (int)ceilf(fminf(fmaxf(mt, -2000.f), 2000.f));
            const float d = __builtin_amdgcn_exp2f(dm + (float)(ve - ve2));
            l *= __builtin_amdgcn_exp2f(dm);
#pragma unroll
            for (int t = 0; t < NT; ++t) acc[t] *= d;
            m = m2;
            ve = ve2;
          }
        }
        const float off = kShift - (m == -INFINITY ? 0.f : m);
        half8 w[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          // capped where the probability is too small for fp32, so that it is not zero times infinity
          const float sv = ldexpf(read_lane(vm, 2 * i + e), min(sx[e] - ve, 120));
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const float pr = __builtin_amdgcn_exp2f(S[e][c] + off);
            l += pr;
            const float y = S[e][c] == -INFINITY ? 0.f : pr * sv;   // a scale that is not a number stays unseen
            w[0][4 * e + c] = (_Float16)y;
            w[1][4 * e + c] = (_Float16)(y - (float)w[0][4 * e + c]);
          }
        }
#pragma unroll
        for (int u = 0; u < NU; ++u)
          static_for<0, VB>([&](auto bb) {
            constexpr int B = decltype(bb)::value;
            half8 vf;
#pragma unroll
            for (int pr = 0; pr < 4; ++pr) {
              const half2v y = widen_pair<B % 4>(x.v[2 * pr][u][B / 4], x.v[2 * pr + 1][u][B / 4]);
              vf[2 * pr] = y[0];
              vf[2 * pr + 1] = y[1];
            }
#pragma unroll
            for (int t = 0; t < 2; ++t) acc[u * VB + B] = mfma32(vf, w[t], acc[u * VB + B]);
          });
      };
      for (int i = 0; i < count; i += 2) {
        load(i + 1, odd);
        compute(i, even);
        load(i + 2, even);
        compute(i + 1, odd);
      }
      tb += 4 * 32;
      if (tb < tend) {
        open(tb);
        load(0, even);
      }
    }
    l += __shfl_xor(l, 16, 64);
    l += __shfl_xor(l, 32, 64);

    // The four waves' results together, wave c taking register c of every product: columns VB (4 g + c) .. + VB - 1
    // of the lane's row.
    __syncthreads();                              // the area may still be read from the segment before
    stats[wave][0][lane] = m;
    stats[wave][1][lane] = l;
    stats[wave][2][lane] = __builtin_bit_cast(float, ve);
    float part[NT], give[4], lsum = 0.f;
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      if (u) __syncthreads();
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int b = 0; b < VB; ++b) merge[wave][c][b][lane] = acc[u * VB + b][c];
      __syncthreads();
      if (u == 0) {
        float mw[4], lw[4];
        int ew[4];
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          mw[w] = stats[w][0][lane];
          lw[w] = stats[w][1][lane];
          ew[w] = __builtin_bit_cast(int, stats[w][2][lane]);
        }
        m = fmaxf(fmaxf(mw[0], mw[1]), fmaxf(mw[2], mw[3]));
        ve = -4000;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          mw[w] -= m;
          if (lw[w] != 0.f) ve = max(ve, ew[w] + (int)ceilf(fmaxf(mw[w], -2000.f)));
        }
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          lsum += lw[w] == 0.f ? 0.f : lw[w] * __builtin_amdgcn_exp2f(mw[w]);
          give[w] = lw[w] == 0.f ? 0.f : __builtin_amdgcn_exp2f(mw[w] + (float)(ew[w] - ve));
        }
      }
#pragma unroll
      for (int b = 0; b < VB; ++b) {
        part[u * VB + b] = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w)
          part[u * VB + b] = __builtin_fmaf(merge[w][wave][b][lane], give[w], part[u * VB + b]);
      }
    }
    if (live) {
      const float inv = lsum == 0.f ? 0.f : 1.0f / lsum;
      float* po = nullptr;
      if (t0 != 0 || t1 != sp.tiles) {
        // one part has at most one unit that it did not begin, and one more that it does not end
        const int64_t slot = ((int64_t)blockIdx.x * 2 + (t0 == 0 ? 1 : 0)) * kRowTile + n;
        if (g == 0 && wave == 0) {
          f.part_ml[2 * slot] = m;
          f.part_ml[2 * slot + 1] = lsum;
        }
        po = f.part_o + slot * dh;
      }
      const int64_t o_at = (sq.q0 + qi) * a.o_ld + h * a.o_hp;
#pragma unroll
      for (int u = 0; u < NU; ++u) {
        const int c0 = 128 * u + VB * (4 * g + wave);
        if (c0 >= dh) continue;
        auto put = [&](auto* dst) {
          typedef typename std::remove_pointer<decltype(dst)>::type T;
          typedef T Vec __attribute__((ext_vector_type(VB), aligned(sizeof(T))));
          Vec x;
#pragma unroll
          for (int b = 0; b < VB; ++b) x[b] = (T)ldexpf(part[u * VB + b] * inv, ve);
          *reinterpret_cast<Vec*>(dst) = x;
        };
        if (po) put(po + c0);
        else if (dtype == F32) put(static_cast<float*>(a.out) + o_at + c0);
        else if (dtype == F16) put(static_cast<_Float16*>(a.out) + o_at + c0);
        else put(static_cast<__bf16*>(a.out) + o_at + c0);
      }
    }
    if (t0 == 0 && t1 < sp.tiles) left = Head{sq.q0, sq.lq, row0, kvh, (int32_t)((pos + sp.tiles - 1) / size)};

    // on to the next unit, in this sequence or the next that has any
    pos += whole ? 1 : t1 - t0;
    if (pos >= end) break;
    if (pos >= at.before + sp.work(whole)) {
      at.before += sp.work(whole);
      do {
        ++at.s;
        if (at.s < a.seqs) at.sq = sequence(a, at.s);
      } while (at.s < a.seqs && span_of(a, at.sq).units == 0);
      if (at.s >= a.seqs) break;
    }
  }
  if (!whole && threadIdx.x == 0) f.head[blockIdx.x] = left;
}

// Joins the partial results of a row of a unit that several workgroups shared, in their order: workgroup (w, n) row n of
// the unit that part w began and did not end.
__global__ __launch_bounds__(256) void kv_join_kernel(FewArgs f, int dtype) {
  const KvArgs& a = f.a;
  const int lane = threadIdx.x & 63, w0 = blockIdx.x, n = blockIdx.y;
  const Head hd = f.head[w0];
  if (hd.last < 0 || hd.row0 + n >= hd.lq * a.group) return;
  const int parts = hd.last - w0 + 1, dh = a.dh;
  __shared__ float share[kParts];
  __shared__ floatx4 sums[256];
  auto slot = [&](int w) { return ((int64_t)2 * (w0 + w) + (w == 0 ? 1 : 0)) * kRowTile + n; };
  if (threadIdx.x < 64) {
    float m = -INFINITY, l = 0.f, mw[kParts / 64], lw[kParts / 64];
#pragma unroll
    for (int i = 0; i < kParts / 64; ++i) {
      const int w = 64 * i + lane;
      mw[i] = -INFINITY;
      lw[i] = 0.f;
      if (w < parts) {
        const float2 ml = *reinterpret_cast<const float2*>(f.part_ml + 2 * slot(w));
        lw[i] = ml.y;
        if (ml.y != 0.f) mw[i] = ml.x;
      }
      m = fmaxf(m, mw[i]);
    }
    m = wave_max(m);
#pragma unroll
    for (int i = 0; i < kParts / 64; ++i) {
      lw[i] = lw[i] == 0.f ? 0.f : lw[i] * __builtin_amdgcn_exp2f(mw[i] - m);
      l += lw[i];
    }
    l = wave_add(l);
#pragma unroll
    for (int i = 0; i < kParts / 64; ++i)
      if (64 * i + lane < parts) share[64 * i + lane] = lw[i] == 0.f ? 0.f : lw[i] / l;
  }
  __syncthreads();
  // four columns a thread (dh <= 256: at most 64 of them), and the parts shared among the threads that leaves over
  const int quads = dh >> 2, split = 256 / quads;
  const int z = (int)threadIdx.x / quads, c = 4 * ((int)threadIdx.x - z * quads);
  floatx4 o = {0.f, 0.f, 0.f, 0.f};
  if (z < split) {
    for (int w = z; w < parts; w += 4 * split) {
      floatx4 x[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int u = w + e * split;
        x[e] = floatx4{0.f, 0.f, 0.f, 0.f};
        if (u < parts && share[u] != 0.f)
          x[e] = *reinterpret_cast<const floatx4*>(f.part_o + slot(u) * dh + c) * share[u];
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) o += x[e];
    }
  }
  sums[threadIdx.x] = o;
  __syncthreads();
  if (z != 0) return;
  for (int e = 1; e < split; ++e) o += sums[threadIdx.x + e * quads];
  const int64_t r = hd.row0 + n, qi = r / a.group;
  const int64_t o_at = (hd.q0 + qi) * a.o_ld + (hd.kvh * a.group + (r - qi * a.group)) * a.o_hp + c;
  auto put = [&](auto* dst) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      dst[e] = (typename std::remove_reference<decltype(*dst)>::type)o[e];
  };
  if (dtype == F32) put(static_cast<float*>(a.out) + o_at);
  else if (dtype == F16) put(static_cast<_Float16*>(a.out) + o_at);
  else put(static_cast<__bf16*>(a.out) + o_at);
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
  return (size_t)p.parts * (2 * kRowTile * (c.head_dim + 2) * sizeof(float) + sizeof(Head));
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
    FewArgs f{a, 0, 1, nullptr, nullptr, nullptr};
    if (p.parts && work && work_bytes >= kv_attention_workspace_bytes(t, c)) {
      f.parts = p.parts;
      f.head = static_cast<Head*>(work);
      f.part_ml = reinterpret_cast<float*>(f.head + p.parts);
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
    hipLaunchKernelGGL(kv_join_kernel, dim3((unsigned)f.parts, kRowTile), dim3(256), 0, s, f, t.dtype);
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
