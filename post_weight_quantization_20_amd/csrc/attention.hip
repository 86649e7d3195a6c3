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

#include <atomic>
#include <cmath>

namespace gptq {
namespace {

constexpr int kMaxHead = 1024;
constexpr int64_t kRows = 128;   // packed rows of a tile

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
  int o_vec, o_rows;           // out takes stores of four elements; of 16 bytes
  int64_t lq_even, lk_even;    // sequence lengths without offsets
  uint32_t seq_tiles;          // and their row tiles
  int64_t tiles;               // row tiles of one key head, over all sequences (an upper bound)
  int nsplit;                  // ranges that a sequence's keys are split into
  float *part_ml, *part_o;     // nsplit > 1: [nsplit][nq][hq][2] and [nsplit][nq][hq][dh]
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
    r.lq = a.lq_even;
    r.q0 = s * r.lq;
  }
  if (a.kv_start) {
    r.k0 = clamp64(a.kv_start[s], 0, a.nk);
    r.lk = clamp64(a.kv_start[s + 1], r.k0, a.nk) - r.k0;
  } else {
    r.lk = a.lk_even;
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

// The keys a query may see end at this index: its own position or the prefix, whichever is later, and
// nothing for a padding document.
GPTQ_DEV int32_t key_limit_nodoc(const AttnArgs& a, const Seq& sq, int32_t prefix, int64_t i) {
  if (!a.causal) return (int32_t)sq.lk;
  const int64_t p = i + sq.lk - sq.lq + 1;
  return (int32_t)clamp64(p > prefix ? p : prefix, 0, sq.lk);
}

GPTQ_DEV int64_t key_limit(const AttnArgs& a, const Seq& sq, int64_t s, int64_t i) {
  if (a.q_doc && a.q_doc[sq.q0 + i] < 0) return 0;
  return key_limit_nodoc(a, sq, a.prefix ? a.prefix[s] : 0, i);
}

// Whether a sequence holds this row of q.
GPTQ_DEV bool in_a_sequence(const AttnArgs& a, int64_t row, int lane) {
  if (!a.q_start) return true;
  for (int64_t s0 = 0; s0 < a.seqs; s0 += 64) {
    const int64_t s = s0 + lane;
    bool in = false;
    if (s < a.seqs) {
      const int64_t q0 = clamp64(a.q_start[s], 0, a.nq);
      in = row >= q0 && row < clamp64(a.q_start[s + 1], q0, a.nq);
    }
    if (__ballot(in)) return true;
  }
  return false;
}

// The XOR of a 16-byte unit's place in row `row` of a staged tile, for rows of UN units. K: eight rows in
// a row put one unit in eight distinct places; V: four rows put a pair of units in four.
template <int UN>
GPTQ_DEV int swz_k(int row) {
  return UN % 8 == 0 ? (row & 7) : ((row >> 1) & 3);
}
template <int UN>
GPTQ_DEV int swz_v(int row) {
  return UN % 8 == 0 ? 2 * (row & 3) : (row & 2);
}

GPTQ_DEV uint64_t uniform64(uint64_t v) {
  return (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)v) |
         (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(v >> 32)) << 32;
}

// One query and head by one wave over keys [j0, j1), 64 at a time: a lane takes a key for the scores and
// columns lane, lane + 64, ... of the output. Only keys that are seen are read into the output, so this is
// also the exact path for a row whose tile held infinities or NaN that it may not see. acc is the average of
// the values so far, not their weighted sum, which can pass fp32's range where the average does not: a sum
// of weights up to l times values above 2^128 / l. NC: columns a lane.
template <int DT, int NC>
GPTQ_DEV void attn_row(const AttnArgs& a, const Seq& sq, int64_t s, int64_t i, int h, int lane, int64_t j0, int64_t j1,
                       float (&acc)[NC], float& m, float& l) {
  typedef typename ElemOf<DT>::T T;
  const T* q = static_cast<const T*>(a.q) + (sq.q0 + i) * a.q_ld + h * a.q_hp;
  const T* kb = static_cast<const T*>(a.k) + sq.k0 * a.k_ld + (h / a.group) * a.k_hp;
  const T* vb = static_cast<const T*>(a.v) + sq.k0 * a.v_ld + (h / a.group) * a.v_hp;
  const int64_t p = i + sq.lk - sq.lq;
  const int32_t doc = a.q_doc ? a.q_doc[sq.q0 + i] : 0;
  const float slope = a.slopes ? a.slopes[h] : 0.f;
  m = -INFINITY;
  l = 0.f;
#pragma unroll
  for (int c = 0; c < NC; ++c) acc[c] = 0.f;
  const int64_t lim = key_limit(a, sq, s, i);
  const int64_t end = lim < j1 ? lim : j1;
  for (int64_t jb = j0; jb < end; jb += 64) {
    const int64_t j = jb + lane;
    bool seen = j < end;
    if (seen && a.q_doc) seen = a.kv_doc[sq.k0 + j] == doc;
    float sc = -INFINITY;
    if (seen) {
      float dot = 0.f;
      for (int c = 0; c < a.dh; ++c) dot = __builtin_fmaf((float)q[c], (float)kb[j * a.k_ld + c], dot);
      sc = dot * a.scale;
      if (a.cap > 0.f) sc = a.cap * tanhf(sc / a.cap);
      if (a.slopes) sc -= slope * fabsf((float)(p - j));
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
      const float we = __shfl(share, e, 64);
      const T* vr = vb + (jb + e) * a.v_ld;
#pragma unroll
      for (int c = 0; c < NC; ++c)
        if (c * 64 + lane < a.dh) acc[c] = __builtin_fmaf(we, (float)vr[c * 64 + lane], acc[c]);
    }
  }
}

template <int DT, int NC>
GPTQ_DEV void store_row(const AttnArgs& a, int64_t row, int h, int lane, const float (&acc)[NC], float l) {
  typedef typename ElemOf<DT>::T T;
  T* o = static_cast<T*>(a.out) + row * a.o_ld + h * a.o_hp;
#pragma unroll
  for (int c = 0; c < NC; ++c)
    if (c * 64 + lane < a.dh) o[c * 64 + lane] = (T)(l == 0.f ? 0.f : acc[c]);
}

// Heads wider than the matrix-core kernels take: waves over (sequence, query, head).
template <int DT>
__global__ __launch_bounds__(256) void attn_row_kernel(AttnArgs a) {
  const int lane = threadIdx.x & 63;
  for (int64_t s = blockIdx.y; s < a.seqs; s += gridDim.y) {
    const Seq sq = sequence(a, s);
    const int64_t items = sq.lq * a.hq;
    for (int64_t it = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); it < items; it += (int64_t)gridDim.x * 4) {
      float acc[kMaxHead / 64], m, l;
      const int64_t i = it / a.hq;
      const int h = (int)(it - i * a.hq);
      attn_row<DT>(a, sq, s, i, h, lane, 0, sq.lk, acc, m, l);
      store_row<DT>(a, sq.q0 + i, h, lane, acc, l);
    }
  }
}

// ------------------------------------------------------------------ matrix cores
//
// The query heads that share a key head are rows of one tile: packed row r of a sequence is query
// r / group and head r % group, so a key tile is read once for all of them, and a single new token still
// gives `group` rows. A wave owns 32 packed rows. Scores are formed transposed, S^T = K Q^T
// (v_mfma_f32_32x32x16: lane l holds row l % 32 and, of each 8 keys, the four of its half l / 32), so that
// the softmax of a row runs inside a lane and its mirror lane, and the probabilities, rounded to the 16-bit
// type, are the next product's operand O^T += V^T P^T as they lie: the contraction takes the keys in the
// order the lanes hold them, and the transposing LDS reads of V follow that order.
//
// Keys and values stream into LDS in 16-byte units (buffer_load ... lds), double-buffered; units of a row
// are XOR-swizzled so that the operand reads of K (one unit of 32 rows) and the transposing reads of V
// (four rows of two units) fall in distinct banks. Units beyond the head or the keys read as zero through
// the descriptor's range. Tensors that are not 16-byte aligned are staged through registers instead.
//
// The four waves of a workgroup hold 128 rows and share tiles of 64 keys (fp32: 32). With few queries only the
// first waves have rows to work for, which reading the keys leaves them time to do.
//
// The maximum is raised only when a score exceeds it by 8 (in powers of two); probabilities are kept 2^7
// larger, so they stay below 2^15 and small ones keep their bits in fp16. A masked key's probability is
// an exact zero, but zero times an infinity or NaN in V is NaN: a row whose result is not finite is
// computed again by attn_row, which reads the keys that are seen and no others. So is a row whose weighted sum
// passes fp32's range (values above about 2^113, at weights up to 2^15). It is a wave a row and many times
// slower.
//
// Long inputs are bound by the matrix cores and the softmax's vector instructions beside them (2 x 8192 causal
// bf16 tokens, 32 / 8 heads of 128: 1.21 ms, 0.91 PFLOP/s of the pairs seen; 4 x 2048 fp32 tokens of 32 heads:
// 1.12 ms, 0.12 PFLOP/s), few queries by reading K and V (16 against 4915 keys each: 67 us, 4.9 TB/s).

typedef short v4s __attribute__((ext_vector_type(4)));
typedef short v8s __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
#define GPTQ_LDS __attribute__((address_space(3)))

GPTQ_DEV void dma16(i32x4 rsrc, uint32_t voff, uint32_t lds_addr) {
  asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds" ::"v"(voff), "s"(rsrc), "{m0}"(lds_addr)
               : "memory");
}

GPTQ_DEV void dma4(i32x4 rsrc, uint32_t voff, uint32_t lds_addr) {
  asm volatile("s_nop 0\n\tbuffer_load_dword %0, %1, 0 offen lds" ::"v"(voff), "s"(rsrc), "{m0}"(lds_addr)
               : "memory");
}

// Buffer descriptor of `bytes` bytes from a wave-uniform address.
GPTQ_DEV i32x4 descriptor(uint64_t base, int64_t bytes) {
  const uint64_t b = uniform64(base);
  return i32x4{(int)(uint32_t)b, (int)(uint32_t)(b >> 32), __builtin_amdgcn_readfirstlane((int)bytes), 0x00020000};
}

// Keys of a tile, double-buffered within 160 KB of LDS: two workgroups a CU up to 128-wide heads.
template <int DT, int DHP>
struct Tile {
  static constexpr int ESZ = DT == F32 ? 4 : 2;
  static constexpr int KT = DT == F32 ? 32 : 64;
  static constexpr int TILEB = KT * DHP * ESZ;
  static constexpr int LDS = 2 * 2 * TILEB + 2048 + 128;
};

template <int DT>
GPTQ_DEV floatx16 mfma16(v8s a, v8s b, floatx16 c) {
  if constexpr (DT == F16)
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(half8, a), __builtin_bit_cast(half8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0,
                                                   0);
}

template <int DT>
GPTQ_DEV v8s round8(const float* p) {
  if constexpr (DT == F16) {
    half8 r;
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = (_Float16)p[i];
    return __builtin_bit_cast(v8s, r);
  } else {
    bf16x8 r;
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = (__bf16)p[i];
    return __builtin_bit_cast(v8s, r);
  }
}

// The maximum and the sum with the lane 32 away: the swap of two copies leaves the lower half's values in
// both halves of one and the upper half's in the other. Written out with the wait states that a just
// written operand needs: the builtin with one value for both operands gives its first result twice.
GPTQ_DEV void mirror(float v, float& lo, float& hi) {
  lo = v;
  hi = v;
  asm("s_nop 1\n\tv_permlane32_swap_b32 %0, %1\n\ts_nop 1" : "+v"(lo), "+v"(hi));
}
GPTQ_DEV float mirror_max(float v) {
  float lo, hi;
  mirror(v, lo, hi);
  return fmaxf(lo, hi);
}
GPTQ_DEV float mirror_sum(float v) {
  float lo, hi;
  mirror(v, lo, hi);
  return lo + hi;
}

// Row tile t of a key head: its sequence, the tile's place in it (seq = -1: past the last tile) and the
// sequence's ranges and prefix, uniform over the wave.
struct TileAt {
  int64_t seq;
  uint32_t tile;
  Seq sq;
  int32_t prefix;
};

GPTQ_DEV int32_t lane_value(int32_t v, int lane) { return __builtin_amdgcn_readlane(v, lane); }

GPTQ_DEV TileAt find_tile(const AttnArgs& a, int64_t t, int lane) {
  TileAt r{-1, 0, {}, 0};
  if (!a.q_start) {
    const uint32_t per = a.seq_tiles, u = (uint32_t)t;   // a grid holds fewer than 2^24 tiles
    if (per > 0 && u / per < a.seqs) {
      r.seq = u / per;
      r.tile = u % per;
      r.sq = sequence(a, r.seq);
      if (a.prefix) r.prefix = a.prefix[r.seq];
    }
    return r;
  }
  // a lane takes a sequence; the counts of one group of 64 stay below 2^30 tiles and are summed in 64 bits
  int64_t before = 0;
  for (int64_t s0 = 0; s0 < a.seqs; s0 += 64) {
    const int64_t s = s0 + lane;
    Seq q{};
    int32_t pre = 0, n = 0;
    if (s < a.seqs) {
      q = sequence(a, s);
      if (a.prefix) pre = a.prefix[s];
      // at most 2^30 rows of q: a sequence with more tiles than a grid has is never reached
      n = (int32_t)min((q.lq * a.group + kRows - 1) / kRows, (int64_t)1 << 24);
    }
    int32_t sum = n;   // inclusive prefix sum over the lanes
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int32_t v = __shfl_up(sum, o, 64);
      if (lane >= o) sum += v;
    }
    const uint64_t past = __ballot(before + sum > t);
    if (past) {
      const int at = __builtin_ctzll(past);
      r.seq = s0 + at;
      r.tile = (uint32_t)(t - before - lane_value(sum, at) + lane_value(n, at));
      r.sq = Seq{lane_value((int32_t)q.q0, at), lane_value((int32_t)q.k0, at), lane_value((int32_t)q.lq, at),
                 lane_value((int32_t)q.lk, at)};
      r.prefix = lane_value(pre, at);
      return r;
    }
    before += lane_value(sum, 63);
  }
  return r;
}

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kShift = 7.0f, kRaise = 8.0f;
// Caps up to this are formed from 1 / (e^2y + 1), whose 2^-24 the cap multiplies: at most 6e-5 of a score,
// under an eighth of fp16's half step once it weighs a key. Larger ones take tanhf.
constexpr float kSmallCap = 256.0f;

// DHP: head width padded to 32. DMA: 16-byte aligned tensors. MODE 0: scores only scaled, 1: capped, 2: any
// (a bias, both, scaled by zero; caps in fp32 and large ones).
template <int DT, int DHP, bool DMA, int MODE>
__global__ __launch_bounds__(256, DHP <= 128 ? 2 : 1) void attn_mfma_kernel(AttnArgs a) {
  typedef typename ElemOf<DT>::T T;
  typedef Tile<DT, DHP> C;
  constexpr int KT = C::KT;                     // keys of a tile
  constexpr int NT = KT / 32, NF = DHP / 32;
  constexpr int ESZ = C::ESZ, EPU = 16 / ESZ;   // elements of a 16-byte unit
  constexpr int NK = DHP / (2 * EPU);           // unit pairs of a row: one unit of a pair to each half wave
  constexpr int UN = DHP / EPU;                 // units of a row
  constexpr int ROWB = DHP * ESZ, TILEB = C::TILEB, BUFB = 2 * TILEB;
  constexpr int LOADS = KT * UN / 256;          // units a lane stages of K (and of V)
  constexpr int ROWS = (int)kRows;
  typedef typename std::conditional<DT == F32, floatx4, v8s>::type Unit;
  extern __shared__ char smem_raw[];
  GPTQ_LDS char* smem = (GPTQ_LDS char*)smem_raw;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 31, half = lane >> 5;
  // small LDS area behind the tiles: documents of a tile per wave, what the tiles of a block hold
  GPTQ_LDS char* tail = smem + 2 * BUFB;
  GPTQ_LDS int32_t* docs = (GPTQ_LDS int32_t*)tail + 128 * wave;   // two tiles' worth

  // the workgroup's key head, tile of rows and range of keys
  uint32_t kvh, rem;
  if (a.hk % 8 == 0) {
    // Workgroups go to the 8 XCDs in turn: each takes an eighth of the heads, which its L2 keeps, tile by
    // tile (head by head, an XCD's last head would run alone: 4 x 2048 fp32 tokens took a quarter longer).
    const uint32_t mine = (uint32_t)a.hk >> 3, at = blockIdx.x >> 3;
    rem = at / mine;
    kvh = (blockIdx.x & 7) * mine + (at - rem * mine);
  } else {
    rem = blockIdx.x / (uint32_t)a.hk;
    kvh = blockIdx.x - rem * a.hk;
  }
  const uint32_t tord = rem / (uint32_t)a.nsplit;
  const int z = (int)(rem - tord * a.nsplit);
  const TileAt at = find_tile(a, a.tiles - 1 - tord, lane);   // long (late) tiles first
  if (at.seq < 0) return;
  const Seq sq = at.sq;
  const int64_t nrows = sq.lq * a.group, row0 = (int64_t)at.tile * ROWS;

  // this lane's row
  const int64_t r = row0 + 32 * wave + col;
  const bool live = r < nrows;
  // packed rows of one sequence stay below 2^24 tiles of at most 128
  const int64_t qi = live ? (uint32_t)r / (uint32_t)a.group : 0;
  const int g = live ? (int)((uint32_t)r - (uint32_t)qi * a.group) : 0;
  const int h = (int)kvh * a.group + g;
  const int32_t qdoc = live && a.q_doc ? a.q_doc[sq.q0 + qi] : 0;

  // keys: the workgroup's range [kb, ke)
  const int64_t last_row = (row0 + ROWS < nrows ? row0 + ROWS : nrows) - 1;
  int64_t ke = key_limit_nodoc(a, sq, at.prefix, (uint32_t)last_row / (uint32_t)a.group);
  int64_t kb = 0;
  if (a.nsplit > 1) {
    const uint32_t nt = (uint32_t)((ke + KT - 1) / KT), per = (nt + a.nsplit - 1) / (uint32_t)a.nsplit;
    kb = (int64_t)z * per * KT;
    if (ke > kb + (int64_t)per * KT) ke = kb + (int64_t)per * KT;
  }
  // the documents of a block of 64 tiles, a quarter tile a thread, loaded ahead of their use
  constexpr int QK = KT / 4;
  typedef int32_t I4 __attribute__((ext_vector_type(4), aligned(4)));
  I4 bd[QK / 4];
  auto fetch_docs = [&](int64_t b0) {
    const int64_t j0 = b0 + QK * (int64_t)threadIdx.x;
    const int32_t* dp = a.kv_doc + sq.k0 + j0;
    if (j0 + QK <= ke) {
#pragma unroll
      for (int e = 0; e < QK / 4; ++e) bd[e] = *reinterpret_cast<const I4*>(dp + 4 * e);
    } else {
#pragma unroll
      for (int e = 0; e < QK; ++e) bd[e / 4][e % 4] = j0 + e < ke ? dp[e] : 0;
    }
  };
  if (a.q_doc && kb < ke) fetch_docs(kb);

  // Q^T operand: row col, unit 2 ks + half of it (on its way while the ranges are found). Loaded like that, a
  // row at a time, the 32 bytes of a row that an instruction reads come from L2 over and over: 16-bit tiles go
  // through the second buffer in whole rows.
  typedef typename std::conditional<DT == F32, float, short>::type E;   // an element's bits
  constexpr bool QLDS = DMA && DT != F32;
  Unit qf[NK];
  GPTQ_LDS char* qarea = smem + BUFB + wave * 32 * ROWB;
  if constexpr (QLDS) {
    const int64_t q0 = (uint32_t)row0 / (uint32_t)a.group;
    const uint32_t span = (uint32_t)(((ROWS + a.group - 1) / a.group + 1) * a.q_ld + a.group * a.q_hp + a.dh) * ESZ;
    const i32x4 qr = descriptor((uint64_t)(uintptr_t)(static_cast<const E*>(a.q) + (sq.q0 + q0) * a.q_ld +
                                                      kvh * a.group * a.q_hp), span);
    const uint32_t mine = live ? (uint32_t)(((qi - q0) * a.q_ld + g * a.q_hp) * ESZ) : 0x80000000u;
#pragma unroll
    for (int i = 0; i < UN / 2; ++i) {
      const int unit = 64 * i + lane, row = unit / UN, u = (unit - row * UN) ^ swz_k<UN>(row);
      const uint32_t off = (uint32_t)__shfl((int)mine, row, 64);
      dma16(qr, u * EPU < a.dh ? off + 16 * u : 0x80000000u, (uint32_t)(uintptr_t)(qarea + 1024 * i));
    }
  } else {
    const E* qp = static_cast<const E*>(a.q) + (sq.q0 + qi) * a.q_ld + h * a.q_hp;
#pragma unroll
    for (int ks = 0; ks < NK; ++ks) {
      const int c0 = EPU * (2 * ks + half);
      Unit f = {};
      if (DMA) {
        // Past the head K is zero and any finite value will do (a row that holds others is computed again);
        // lanes past the last row hold the sequence's first.
        f = *reinterpret_cast<const Unit*>(qp + (c0 < a.dh ? c0 : 0));
      } else {
#pragma unroll
        for (int e = 0; e < EPU; ++e)
          if (c0 + e < a.dh) f[e] = qp[c0 + e];
      }
      qf[ks] = f;
    }
  }
  const int32_t lim = live && qdoc >= 0 ? key_limit_nodoc(a, sq, at.prefix, qi) : 0;
  const int32_t pos = (int32_t)(qi + sq.lk - sq.lq);
  float slope = 0.f;
  if (MODE == 2 && a.slopes) slope = a.slopes[h];

  // Where masking starts and ends for the wave. Limits rise with the row (padding aside, which sees
  // nothing): the first row's and the last one's.
  const uint32_t seeing = (uint32_t)__ballot(live && qdoc >= 0);
  const bool all_see = seeing == (uint32_t)__ballot(live);
  const int32_t wmin = seeing && all_see ? lane_value(lim, 0) : 0;
  const int32_t wmax = seeing ? lane_value(lim, 31 - __builtin_clz(seeing)) : 0;
  // the documents of the wave's rows: mostly one
  int32_t dmin = 0x7fffffff, dmax = -1;
  bool one_doc = true;
  if (a.q_doc && seeing) {
    dmin = dmax = lane_value(qdoc, __builtin_ctz(seeing));
    one_doc = __ballot(live && qdoc >= 0 && qdoc != dmin) == 0;
    if (!one_doc) {
      dmin = live && qdoc >= 0 ? qdoc : 0x7fffffff;
      dmax = live ? qdoc : -1;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        dmin = min(dmin, __shfl_xor(dmin, o, 64));
        dmax = max(dmax, __shfl_xor(dmax, o, 64));
      }
    }
  }
  if (a.q_doc) {   // the workgroup's range of documents
    if (lane == 0) {
      docs[0] = dmin;
      docs[1] = dmax;
    }
    __syncthreads();
    for (int w = 0; w < 4; ++w) {
      dmin = min(dmin, ((GPTQ_LDS int32_t*)tail)[128 * w]);
      dmax = max(dmax, ((GPTQ_LDS int32_t*)tail)[128 * w + 1]);
    }
    __syncthreads();
  }
  dmin = __builtin_amdgcn_readfirstlane(dmin);
  dmax = __builtin_amdgcn_readfirstlane(dmax);

  const E* kp = static_cast<const E*>(a.k) + sq.k0 * a.k_ld + kvh * a.k_hp;
  const E* vp = static_cast<const E*>(a.v) + sq.k0 * a.v_ld + kvh * a.v_hp;
  auto negate_q = [&]() {   // for a negative scale: the largest score is the largest product of -q
    if (MODE == 0 && a.scale < 0.f) {
#pragma unroll
      for (int ks = 0; ks < NK; ++ks)
#pragma unroll
        for (int e = 0; e < EPU; ++e) {
          if constexpr (DT == F32) qf[ks][e] = -qf[ks][e];
          else qf[ks][e] ^= (short)0x8000;
        }
    }
  };
  bool have_q = !QLDS;
  if (!QLDS) negate_q();

  // staging: load q of this wave fills 16-byte units 64 (q + LOADS wave') + lane of a tile
  int srow[LOADS], ku[LOADS], vu[LOADS];
#pragma unroll
  for (int i = 0; i < LOADS; ++i) {
    const int unit = 64 * (LOADS * wave + i) + lane;
    const int row = unit / UN, up = unit - row * UN;
    srow[i] = row;
    ku[i] = up ^ swz_k<UN>(row);
    vu[i] = DT == F32 ? up : up ^ swz_v<UN>(row);
  }
  constexpr uint32_t OOB = 0x80000000u;   // beyond any descriptor's range: reads as zero
  uint32_t kvo[LOADS], vvo[LOADS];
  if (DMA) {
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
      kvo[i] = ku[i] * EPU < a.dh ? (uint32_t)((srow[i] * a.k_ld + ku[i] * EPU) * ESZ) : OOB;
      vvo[i] = vu[i] * EPU < a.dh ? (uint32_t)((srow[i] * a.v_ld + vu[i] * EPU) * ESZ) : OOB;
    }
  }
  // whole: every key of the tile has the document of all rows, so their documents are not needed
  auto stage = [&](int64_t j0, int buf, bool whole) {
    const int64_t left = sq.lk - j0;
    const int rows = left < KT ? (int)left : KT;
    GPTQ_LDS char* kd = smem + buf * BUFB + LOADS * wave * 1024;
    GPTQ_LDS char* vd = kd + TILEB;
    if (DMA) {
      const uint64_t ka = (uint64_t)(uintptr_t)(kp + j0 * a.k_ld), va = (uint64_t)(uintptr_t)(vp + j0 * a.v_ld);
      const i32x4 kr = descriptor(ka, ((rows - 1) * a.k_ld + a.dh) * ESZ),
                  vr = descriptor(va, ((rows - 1) * a.v_ld + a.dh) * ESZ);
      const uint32_t k32 = (uint32_t)(uintptr_t)kd, v32 = (uint32_t)(uintptr_t)vd;
#pragma unroll
      for (int i = 0; i < LOADS; ++i) dma16(kr, kvo[i], k32 + 1024 * i);
#pragma unroll
      for (int i = 0; i < LOADS; ++i) dma16(vr, vvo[i], v32 + 1024 * i);
      if (a.q_doc && !(whole && one_doc))   // keys past the last one read as document 0 and are past every limit
        dma4(descriptor((uint64_t)(uintptr_t)(a.kv_doc + sq.k0 + j0), 4 * rows), 4 * lane,
             (uint32_t)(uintptr_t)(docs + 64 * buf));
    } else {
      if (a.q_doc) docs[64 * buf + lane] = lane < rows ? a.kv_doc[sq.k0 + j0 + lane] : -1;
#pragma unroll
      for (int i = 0; i < LOADS; ++i) {
        Unit kx = {}, vx = {};
        if (srow[i] < rows) {
          const E* ks = kp + (j0 + srow[i]) * a.k_ld;
          const E* vs = vp + (j0 + srow[i]) * a.v_ld;
#pragma unroll
          for (int e = 0; e < EPU; ++e) {
            if (ku[i] * EPU + e < a.dh) kx[e] = ks[ku[i] * EPU + e];
            if (vu[i] * EPU + e < a.dh) vx[e] = vs[vu[i] * EPU + e];
          }
        }
        *(GPTQ_LDS Unit*)(kd + 1024 * i + 16 * lane) = kx;
        *(GPTQ_LDS Unit*)(vd + 1024 * i + 16 * lane) = vx;
      }
    }
  };

  // operand addresses inside a tile
  int koff[4], voff[2] = {4 * half * ROWB + 4 * col, 0};
#pragma unroll
  for (int i = 0; i < 4; ++i) koff[i] = col * ROWB + (((2 * i + half) ^ swz_k<UN>(col)) << 4);
  if constexpr (DT != F32) {
    const int s = lane & 15, trow = 4 * half + (s >> 2);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      voff[i] = trow * ROWB + (((4 * i + 2 * ((lane >> 4) & 1) + ((s & 3) >> 1)) ^ swz_v<UN>(trow)) << 4) + 8 * (s & 1);
  }

  floatx16 acc[NF];
#pragma unroll
  for (int f = 0; f < NF; ++f) acc[f] = floatx16{};
  float m = -INFINITY, l = 0.f;
  // a key's weight is 2^(c S): S is the product (MODE 0), -1 / (e^2y + 1) with y = scale q.k / cap, which
  // is (tanh y - 1) / 2 (MODE 1), or the finished score (MODE 2)
  const float c = MODE == 0 ? fabsf(a.scale) * kLog2e : MODE == 1 ? 2.0f * a.cap * kLog2e : kLog2e;
  const float raise = kRaise / c;
  const float inv_cap = a.cap > 0.f ? 1.0f / a.cap : 0.f;
  const float to_cap = 2.0f * kLog2e * inv_cap;

  auto compute = [&](int64_t j0, int buf, bool whole) {
    GPTQ_LDS char* kt = smem + buf * BUFB;
    GPTQ_LDS char* vt = kt + TILEB;
    floatx16 S[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      S[t] = floatx16{};
#pragma unroll
      for (int ks = 0; ks < NK; ++ks) {
        const Unit kf = *(GPTQ_LDS Unit*)(kt + 32 * t * ROWB + koff[ks & 3] + 128 * (ks >> 2));
        if constexpr (DT == F32) {
#pragma unroll
          for (int e = 0; e < 4; ++e) S[t] = __builtin_amdgcn_mfma_f32_32x32x2f32(kf[e], qf[ks][e], S[t], 0, 0, 0);
        } else {
          S[t] = mfma16<DT>(kf, qf[ks], S[t]);
        }
      }
    }
    const int32_t jb = (int32_t)j0 + 4 * half;   // the key of register i of subtile t: jb + 32 t + 8 (i / 4) + i % 4
    if constexpr (MODE == 1) {
      const float k = a.scale * to_cap;
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          S[t][i] = -__builtin_amdgcn_rcpf(__builtin_amdgcn_exp2f(S[t][i] * k) + 1.0f);
    }
    if constexpr (MODE == 2) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) S[t][i] *= a.scale;
      if (a.cap > 0.f) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            if (DT == F32 || a.cap > kSmallCap)
              S[t][i] = a.cap * tanhf(S[t][i] * inv_cap);
            else   // tanh y = 1 - 2 / (e^2y + 1)
              S[t][i] = a.cap - 2.0f * a.cap * __builtin_amdgcn_rcpf(__builtin_amdgcn_exp2f(S[t][i] * to_cap) + 1.0f);
          }
      }
      if (a.slopes) {
        const float d0 = (float)(pos - jb);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int i = 0; i < 16; ++i)
            S[t][i] = __builtin_fmaf(-slope, fabsf(d0 - (float)(32 * t + 8 * (i / 4) + i % 4)), S[t][i]);
      }
    }
    const bool doc_mask = a.q_doc && !(whole && one_doc);
    if (j0 + KT > wmin || doc_mask) {
      if (doc_mask) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            const i32x4 kd = *(GPTQ_LDS i32x4*)(docs + 64 * buf + 32 * t + 8 * b + 4 * half);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (kd[e] != qdoc) S[t][4 * b + e] = -INFINITY;
          }
      }
      const int32_t rel = lim - jb;
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) S[t][i] = rel > 32 * t + 8 * (i / 4) + i % 4 ? S[t][i] : -INFINITY;
    }
    float mx = -INFINITY;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i) mx = fmaxf(mx, S[t][i]);
    mx = mirror_max(mx);
    if (__ballot(!(mx <= m + raise))) {
      const float m2 = fmaxf(m, mx);
      const float f = m2 == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f((m - m2) * c);
      m = m2;
      l *= f;
#pragma unroll
      for (int ft = 0; ft < NF; ++ft)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[ft][i] *= f;
    }
    const float off = kShift - (m == -INFINITY ? 0.f : m * c);
    float p[NT][16], sum[4] = {0.f, 0.f, 0.f, 0.f};   // a tile's sum apart, so that long sums stay short chains
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        p[t][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(S[t][i], c, off));
        sum[i & 3] += p[t][i];
      }
    l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
    if constexpr (DT == F32) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i)
#pragma unroll
          for (int ft = 0; ft < NF; ++ft) {
            const float vf = *(GPTQ_LDS float*)(vt + (32 * t + 8 * (i / 4) + i % 4) * ROWB + voff[0] + 128 * ft);
            acc[ft] = __builtin_amdgcn_mfma_f32_32x32x2f32(vf, p[t][i], acc[ft], 0, 0, 0);
          }
      return;
    } else {
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const v8s pf = round8<DT>(&p[t][8 * e]);
#pragma unroll
        for (int ft = 0; ft < NF; ++ft) {
          GPTQ_LDS char* va = vt + (32 * t + 16 * e) * ROWB + voff[ft & 1] + 128 * (ft >> 1);
          const v4s v0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((GPTQ_LDS v4s*)va);
          const v4s v1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((GPTQ_LDS v4s*)(va + 8 * ROWB));
          acc[ft] = mfma16<DT>(__builtin_shufflevector(v0, v1, 0, 1, 2, 3, 4, 5, 6, 7), pf, acc[ft]);
        }
      }
    }
  };

  auto ready = [&]() {   // the staged tile is in LDS, and the other buffer is no longer read
    if (DMA) asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    else __syncthreads();
  };

  // Tiles in order, 64 at a time (a block): with documents, the block's tiles that hold a document of the
  // rows' range are found first, a quarter tile a thread.
  int parity = 0;
  for (int64_t b0 = kb; b0 < ke; b0 += 64 * KT) {
    uint64_t active = ~0ull, whole = 0;
    const int64_t left = (ke - b0 + KT - 1) / KT;
    if (left < 64) active = (1ull << left) - 1;
    if (a.q_doc) {
      const int64_t j0 = b0 + QK * (int64_t)threadIdx.x;
      int32_t lo = 0x7fffffff, hi = (int32_t)0x80000000;
#pragma unroll
      for (int e = 0; e < QK; ++e)
        if (j0 + e < ke) {
          lo = min(lo, bd[e / 4][e % 4]);
          hi = max(hi, bd[e / 4][e % 4]);
        }
      if (b0 + 64 * KT < ke) fetch_docs(b0 + 64 * KT);
      lo = min(lo, __shfl_xor(lo, 1, 64));
      hi = max(hi, __shfl_xor(hi, 1, 64));
      lo = min(lo, __shfl_xor(lo, 2, 64));
      hi = max(hi, __shfl_xor(hi, 2, 64));
      // bit 0: holds a document of the range, bit 1: nothing but the one document of all rows. Two areas in
      // turn: a wave may still read the last block's.
      GPTQ_LDS uint8_t* state = (GPTQ_LDS uint8_t*)(tail + 2048) + 64 * parity;
      parity ^= 1;
      if ((lane & 3) == 0)
        state[threadIdx.x >> 2] = (lo <= dmax && hi >= dmin ? 1 : 0) | (lo == hi && lo == dmin && dmin == dmax ? 2 : 0);
      __syncthreads();
      const uint32_t st = state[lane];
      active &= __ballot(st & 1);
      whole = __ballot(st & 2);
    }
    active = uniform64(active);
    whole = uniform64(whole);
    if (!active) continue;
    auto tile_of = [&](int t) { return b0 + (int64_t)t * KT; };
    int t = __builtin_ctzll(active), buf = 0;
    __syncthreads();   // every wave is done with both buffers (of the block before)
    stage(tile_of(t), 0, (whole >> t) & 1);
    while (true) {
      const int64_t j0 = tile_of(t);
      const bool full = (whole >> t) & 1;
      active &= active - 1;
      ready();
      if (QLDS && !have_q) {
#pragma unroll
        for (int ks = 0; ks < NK; ++ks) qf[ks] = *(GPTQ_LDS Unit*)(qarea + koff[ks & 3] + 128 * (ks >> 2));
        negate_q();
        have_q = true;
        __syncthreads();   // the second buffer is free
      }
      if (active) {
        t = __builtin_ctzll(active);
        stage(tile_of(t), buf ^ 1, (whole >> t) & 1);
      }
      if (j0 < wmax) compute(j0, buf, full);
      if (!active) break;
      buf ^= 1;
    }
  }
  if (QLDS) asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // also where no tile was active
  l = mirror_sum(l);

  // rows whose sum is not finite: computed again without the keys they do not see
  float nothing = l * 0.f;   // zero, unless a value is not finite
#pragma unroll
  for (int ft = 0; ft < NF; ++ft)
#pragma unroll
    for (int i = 0; i < 16; ++i) nothing = __builtin_fmaf(acc[ft][i], 0.f, nothing);
  const bool odd = !(nothing == 0.f);
  uint32_t redo = 0;
  {
    const uint64_t o = __ballot(odd && live);
    redo = (uint32_t)o | (uint32_t)(o >> 32);
  }
  if (DMA && a.nsplit == 1 && a.o_rows) {
    // Rows leave through LDS, 16 bytes a lane along each (a lane's own pieces are 8 bytes of every 16): the
    // tiles' area is free when every wave is here.
    __syncthreads();
    GPTQ_LDS char* area = smem + wave * 32 * ROWB;
    const float inv = l == 0.f ? 0.f : 1.0f / l;
    typedef T T4 __attribute__((ext_vector_type(4)));
#pragma unroll
    for (int ft = 0; ft < NF; ++ft)
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        T4 o;
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = (T)(acc[ft][4 * b + e] * inv);
        const int at16 = (32 * ft + 8 * b + 4 * half) * ESZ;
        *(GPTQ_LDS T4*)(area + col * ROWB + (((at16 >> 4) ^ swz_k<UN>(col)) << 4) + (at16 & 15)) = o;
      }
    __builtin_amdgcn_wave_barrier();
    const int64_t to = live && !((redo >> col) & 1) ? (sq.q0 + qi) * a.o_ld + h * a.o_hp : -1;
#pragma unroll
    for (int i = 0; i < UN / 2; ++i) {
      const int unit = 64 * i + lane, row = unit / UN, u = (unit - row * UN) ^ swz_k<UN>(row);
      const int64_t row_to = __shfl(to, row, 64);
      const Unit v = *(GPTQ_LDS Unit*)(area + 1024 * i + 16 * lane);
      if (row_to >= 0 && u * EPU < a.dh)
        *reinterpret_cast<Unit*>(static_cast<E*>(a.out) + row_to + u * EPU) = v;
    }
  } else if (live && !((redo >> col) & 1)) {
    const int64_t row = sq.q0 + qi;
    if (a.nsplit > 1) {
      // O and l are in units of 2^mexp
      const float mexp = m == -INFINITY ? -INFINITY : m * c + (MODE == 1 ? a.cap * kLog2e : 0.f) - kShift;
      const int64_t pr = ((int64_t)z * a.nq + row) * a.hq + h;
      if (half == 0) {
        a.part_ml[2 * pr] = mexp;
        a.part_ml[2 * pr + 1] = l;
      }
      float* po = a.part_o + pr * a.dh;
#pragma unroll
      for (int ft = 0; ft < NF; ++ft)
#pragma unroll
        for (int b = 0; b < 4; ++b)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int f = 32 * ft + 8 * b + 4 * half + e;
            if (f < a.dh) po[f] = acc[ft][4 * b + e];
          }
    } else {
      T* po = static_cast<T*>(a.out) + row * a.o_ld + h * a.o_hp;
      const float inv = l == 0.f ? 0.f : 1.0f / l;
      const bool vec = DMA && a.o_vec;
#pragma unroll
      for (int ft = 0; ft < NF; ++ft)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const int f = 32 * ft + 8 * b + 4 * half;
          typedef T T4 __attribute__((ext_vector_type(4)));
          T4 o;
#pragma unroll
          for (int e = 0; e < 4; ++e) o[e] = (T)(acc[ft][4 * b + e] * inv);
          if (vec) {
            if (f < a.dh) *reinterpret_cast<T4*>(po + f) = o;
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (f + e < a.dh) po[f + e] = o[e];
          }
        }
    }
  }
  while (redo) {
    const int rr = __builtin_ctz(redo);
    redo &= redo - 1;
    const int64_t rw = __shfl(r, rr, 64);
    const int64_t i2 = rw / a.group;
    const int h2 = (int)kvh * a.group + (int)(rw - i2 * a.group);
    constexpr int NC = (DHP + 63) / 64;
    float ar[NC], m2, l2;
    attn_row<DT>(a, sq, at.seq, i2, h2, lane, kb, ke, ar, m2, l2);
    if (a.nsplit > 1) {
      const int64_t pr = ((int64_t)z * a.nq + sq.q0 + i2) * a.hq + h2;
      int e2;   // the sum as a fraction below one, so that the average times it stays in range
      const float lf = frexpf(l2, &e2);
      if (lane == 0) {
        a.part_ml[2 * pr] = l2 == 0.f ? m2 : m2 * kLog2e + (float)e2;
        a.part_ml[2 * pr + 1] = lf;
      }
#pragma unroll
      for (int cc = 0; cc < NC; ++cc)
        if (64 * cc + lane < a.dh) a.part_o[pr * a.dh + 64 * cc + lane] = ar[cc] * lf;
    } else {
      store_row<DT>(a, sq.q0 + i2, h2, lane, ar, l2);
    }
  }
}

// Joins the key ranges of each row, in order: one wave per (query, head), columns over the lanes.
template <int DT>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs a) {
  typedef typename ElemOf<DT>::T T;
  const int lane = threadIdx.x & 63;
  const int64_t total = a.nq * a.hq;
  for (int64_t it = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); it < total; it += (int64_t)gridDim.x * 4) {
    const int64_t row = it / a.hq;
    if (!in_a_sequence(a, row, lane)) continue;
    const int h = (int)(it - row * a.hq);
    // lane z holds range z's maximum and sum (at most 64 ranges)
    const bool mine = lane < a.nsplit;
    float mz = -INFINITY, lz = 0.f;
    if (mine) {
      const float2 ml = *reinterpret_cast<const float2*>(a.part_ml + 2 * ((int64_t)lane * total + it));
      mz = ml.x;
      lz = ml.y;
    }
    const float m = wave_max(mz);
    // a range that the row does not see takes no part
    const float f = mz == -INFINITY && lz == 0.f ? 0.f : __builtin_amdgcn_exp2f(mz - m);
    const float l = wave_add(lz * f);
    const float part = l == 0.f ? 0.f : f / l;   // weights of the average: the sum itself may pass fp32's range
    constexpr int NC = 4;
    float acc[NC] = {};
    for (int z0 = 0; z0 < a.nsplit; z0 += 8) {
      float v[8][NC];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        // zeros past the last range: zero times what another range holds would be NaN for an infinity
        const float* po = a.part_o + ((int64_t)(z0 + e) * total + it) * a.dh;
#pragma unroll
        for (int c = 0; c < NC; ++c) v[e][c] = z0 + e < a.nsplit && 64 * c + lane < a.dh ? po[64 * c + lane] : 0.f;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {   // lanes past the last range hold a factor of zero
        const float fz = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, part), z0 + e));
#pragma unroll
        for (int c = 0; c < NC; ++c) acc[c] = __builtin_fmaf(v[e][c], fz, acc[c]);
      }
    }
    T* o = static_cast<T*>(a.out) + row * a.o_ld + h * a.o_hp;
#pragma unroll
    for (int c = 0; c < NC; ++c)
      if (64 * c + lane < a.dh) o[64 * c + lane] = (T)acc[c];
  }
}

template <int DT, int DHP, bool DMA, int MODE>
hipError_t launch_mfma(const AttnArgs& a, hipStream_t s) {
  constexpr size_t lds = Tile<DT, DHP>::LDS;
  auto f = attn_mfma_kernel<DT, DHP, DMA, MODE>;
  // the LDS beyond 64 KB is asked for once per device
  static std::atomic<uint64_t> asked{0};
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  const uint64_t bit = (uint64_t)1 << (dev & 63);
  if (lds > 65536 && (dev > 63 || !(asked.load() & bit))) {
    e = hipFuncSetAttribute(reinterpret_cast<const void*>(f), hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
    asked |= bit;
  }
  hipLaunchKernelGGL(f, dim3((unsigned)(a.tiles * a.hk * a.nsplit)), dim3(256), lds, s, a);
  return hipGetLastError();
}

template <int DT, int DHP>
hipError_t by_mode(const AttnArgs& a, bool dma, hipStream_t s) {
  if (!dma) return launch_mfma<DT, DHP, false, 2>(a, s);
  if (a.slopes || a.scale == 0.f) return launch_mfma<DT, DHP, true, 2>(a, s);
  if (a.cap == 0.f) return launch_mfma<DT, DHP, true, 0>(a, s);
  if constexpr (DT != F32)
    if (a.cap <= kSmallCap) return launch_mfma<DT, DHP, true, 1>(a, s);
  return launch_mfma<DT, DHP, true, 2>(a, s);
}

template <int DT>
hipError_t by_head(const AttnArgs& a, bool dma, hipStream_t s) {
  if (a.dh <= 64) return by_mode<DT, 64>(a, dma, s);
  if (a.dh <= 96) return by_mode<DT, 96>(a, dma, s);
  if (a.dh <= 128) return by_mode<DT, 128>(a, dma, s);
  return by_mode<DT, 256>(a, dma, s);
}

// The launch's plan: tiles of rows, ranges that keys are split into.
struct Plan {
  bool mfma;
  int64_t tiles;
  int nsplit;
};

Plan plan(const gptq_attention_t& t) {
  Plan p{};
  p.mfma = t.head_dim <= 256;
  if (!p.mfma) return p;
  const int64_t group = t.q_heads / t.kv_heads;
  p.tiles = t.n_q * group / kRows + t.seqs;
  // Fewer than two workgroups a CU: split the keys until there are two, in ranges of at least 256 keys (of
  // the average sequence). More ranges cost more than they fill: 16 tokens against 4915 keys each take 67 us
  // with 512 workgroups and 71 with 768.
  const int64_t items = p.tiles * t.kv_heads, keys = t.n_kv / t.seqs;
  p.nsplit = 1;
  if (items < 512)
    p.nsplit = (int)std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(64, (512 + items - 1) / items), keys / 256));
  return p;
}

}  // namespace

// A grid holds fewer than 2^32 threads; keys are split only far below that.
bool attention_fits(const gptq_attention_t& t) {
  const Plan p = plan(t);
  return !p.mfma || p.tiles * t.kv_heads < (int64_t)1 << 24;
}

size_t attention_workspace_bytes(const gptq_attention_t& t) {
  const Plan p = plan(t);
  if (!p.mfma || p.nsplit <= 1) return 0;
  return (size_t)p.nsplit * t.n_q * t.q_heads * (t.head_dim + 2) * sizeof(float);
}

hipError_t attention(const gptq_attention_t& t, const void* q, const void* k, const void* v, const int32_t* q_start,
                     const int32_t* kv_start, const float* slopes, const int32_t* q_doc, const int32_t* kv_doc,
                     const int32_t* prefix, void* out, void* work, size_t work_bytes, hipStream_t s) {
  AttnArgs a{};
  a.q = q; a.k = k; a.v = v; a.out = out;
  a.q_ld = t.q_ld; a.k_ld = t.k_ld; a.v_ld = t.v_ld; a.o_ld = t.out_ld;
  a.q_hp = t.q_hp; a.k_hp = t.k_hp; a.v_hp = t.v_hp; a.o_hp = t.out_hp;
  a.seqs = t.seqs; a.nq = t.n_q; a.nk = t.n_kv;
  a.hq = t.q_heads; a.hk = t.kv_heads; a.group = t.q_heads / t.kv_heads; a.dh = t.head_dim;
  a.causal = t.causal; a.scale = (float)t.scale; a.cap = (float)t.softcap;
  a.q_start = q_start; a.kv_start = kv_start; a.q_doc = q_doc; a.kv_doc = kv_doc; a.prefix = prefix;
  a.slopes = slopes;
  a.lq_even = a.nq / a.seqs;
  a.lk_even = a.nk / a.seqs;
  Plan p = plan(t);
  if (!p.mfma) {
    const int64_t waves = a.nq * a.hq;
    const dim3 grid((unsigned)std::min<int64_t>((waves + 3) / 4, 4096), (unsigned)std::min<int64_t>(t.seqs, 4096));
    if (t.dtype == F32) hipLaunchKernelGGL(attn_row_kernel<F32>, grid, dim3(256), 0, s, a);
    else if (t.dtype == F16) hipLaunchKernelGGL(attn_row_kernel<F16>, grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL(attn_row_kernel<BF16>, grid, dim3(256), 0, s, a);
    return hipGetLastError();
  }
  const size_t need = attention_workspace_bytes(t);
  if (!work || work_bytes < need) p.nsplit = 1;
  a.tiles = p.tiles;
  a.nsplit = p.nsplit;
  a.seq_tiles = (uint32_t)std::min<int64_t>(1 << 24, (a.lq_even * a.group + kRows - 1) / kRows);
  if (p.nsplit > 1) {
    a.part_ml = static_cast<float*>(work);
    a.part_o = a.part_ml + (int64_t)p.nsplit * a.nq * a.hq * 2;
  }
  // 16-byte units: pointers, pitches and head width multiples of 16 bytes, and a tile inside 31-bit offsets
  const int unit = t.dtype == F32 ? 4 : 8;
  auto al = [&](const void* ptr, int64_t ld, int64_t hp) {
    return reinterpret_cast<uintptr_t>(ptr) % 16 == 0 && ld % unit == 0 && hp % unit == 0;
  };
  const bool dma = a.dh % unit == 0 && al(q, a.q_ld, a.q_hp) && al(k, a.k_ld, a.k_hp) && al(v, a.v_ld, a.v_hp) &&
                   std::max(a.k_ld, a.v_ld) < ((int64_t)1 << 23) &&
                   (128 / a.group + 2) * a.q_ld + a.group * a.q_hp < ((int64_t)1 << 28);
  a.o_rows = reinterpret_cast<uintptr_t>(out) % 16 == 0 && a.o_ld % unit == 0 && a.o_hp % unit == 0;
  a.o_vec = reinterpret_cast<uintptr_t>(out) % (t.dtype == F32 ? 16 : 8) == 0 && a.o_ld % 4 == 0 && a.o_hp % 4 == 0;
  hipError_t e = t.dtype == F32   ? by_head<F32>(a, dma, s)
                 : t.dtype == F16 ? by_head<F16>(a, dma, s)
                                  : by_head<BF16>(a, dma, s);
  if (e != hipSuccess || p.nsplit <= 1) return e;
  const dim3 grid((unsigned)std::min<int64_t>((a.nq * a.hq + 3) / 4, 65536));
  if (t.dtype == F32) hipLaunchKernelGGL(attn_join_kernel<F32>, grid, dim3(256), 0, s, a);
  else if (t.dtype == F16) hipLaunchKernelGGL(attn_join_kernel<F16>, grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL(attn_join_kernel<BF16>, grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace gptq
