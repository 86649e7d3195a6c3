// C-ABI entry points: host-side argument checks, then launches on the caller's stream.
#include <cmath>
#include <cstring>

#include "../../include/gptq.h"
#include "common.hpp"


namespace {

constexpr int64_t kMaxDim = (int64_t)1 << 31;  // d * d and rows * d stay far inside int64

bool dtype_ok(int32_t t) { return t == GPTQ_F32 || t == GPTQ_F16 || t == GPTQ_BF16; }

// Validates the settings shared by factor and quantize. Returns GPTQ_OK or the error.
gptq_status_t check_params(const gptq_params_t* p, int64_t d, bool quant) {
  if (!p) return GPTQ_EINVAL;
  if ((p->sym != 0 && p->sym != 1) || (p->static_groups != 0 && p->static_groups != 1) ||
      (p->compact_meta != 0 && p->compact_meta != 1))
    return GPTQ_EINVAL;
  if (p->act_order != 0 && p->act_order != 1) return GPTQ_EINVAL;
  if (!(p->damp >= 0.0) || !std::isfinite(p->damp)) return GPTQ_EINVAL;
  if (!quant) return GPTQ_OK;
  if (p->bits < 2 || p->bits > 8) return GPTQ_EINVAL;
  if (p->block_size < 1) return GPTQ_EINVAL;
  if (p->block_size > 128) return GPTQ_EUNSUPPORTED;
  const int64_t g = p->group_size <= 0 ? d : p->group_size;
  if (g == 1) return GPTQ_EINVAL;
  if (g < d && !(p->block_size % g == 0 || g % p->block_size == 0)) return GPTQ_EINVAL;
  return GPTQ_OK;
}

gptq_status_t hip_status(hipError_t e) { return e == hipSuccess ? GPTQ_OK : GPTQ_EHIP; }

}  // namespace

extern "C" {

const char* gptq_status_string(gptq_status_t s) {
  switch (s) {
    case GPTQ_OK: return "ok";
    case GPTQ_EINVAL: return "invalid argument";
    case GPTQ_ENOTPD: return "damped Hessian is not positive definite";
    case GPTQ_EUNSUPPORTED: return "unsupported setting";
    case GPTQ_EHIP: return "HIP runtime error";
    case GPTQ_ENOMEM: return "workspace too small";
    default: return "unknown status";
  }
}

size_t gptq_workspace_bytes(int32_t kind, int64_t a, int64_t d, const gptq_params_t* p) {
  if (d <= 0 || d > kMaxDim || a < 0 || a > kMaxDim) return 0;
  switch (kind) {
    case GPTQ_WS_HESSIAN: return gptq::hessian_workspace_bytes(a, d);
    case GPTQ_WS_FACTOR: return gptq::factor_workspace_bytes(d);
    case GPTQ_WS_QUANTIZE: {
      if (!p || p->block_size < 1 || p->block_size > 128) return 0;
      return gptq::quant_layout(a, d, p->block_size).total;
    }
    default: return 0;
  }
}

}  // extern "C"

namespace {

// gptq_hessian_accumulate (H += 2 X^T X) and gptq_hessian_compute (H = 2 X^T X)
gptq_status_t hessian_call(float* H, int64_t d, const void* X, int32_t x_dtype, int64_t n_tok, int64_t ld_x,
                           void* work, size_t work_bytes, void* stream, bool overwrite) {
  if (!H || d <= 0 || d > kMaxDim || n_tok < 0 || n_tok > kMaxDim || !dtype_ok(x_dtype)) return GPTQ_EINVAL;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (n_tok == 0) return overwrite ? hip_status(gptq::zero_matrix(H, d * d, s)) : GPTQ_OK;
  if (!X || ld_x < d) return GPTQ_EINVAL;
  if (x_dtype == GPTQ_F32) {
    gptq::GemmArgs a{};
    a.M = d; a.N = d; a.K = n_tok;
    a.A = static_cast<const float*>(X); a.lda = ld_x; a.transA = 1;
    a.B = static_cast<const float*>(X); a.ldb = ld_x; a.transB = 0;
    a.C = H; a.ldc = d;
    a.alpha = 2.0f; a.beta = overwrite ? 0.0f : 1.0f; a.tri = 2;
    return hip_status(gptq::gemm_f32(a, s));
  }
  return hip_status(gptq::hessian_f16(H, d, X, x_dtype, n_tok, ld_x, work, work_bytes, s, overwrite));
}

}  // namespace

extern "C" {

gptq_status_t gptq_hessian_accumulate(float* H, int64_t d, const void* X, int32_t x_dtype, int64_t n_tok,
                                      int64_t ld_x, void* work, size_t work_bytes, void* stream) {
  return hessian_call(H, d, X, x_dtype, n_tok, ld_x, work, work_bytes, stream, false);
}

gptq_status_t gptq_hessian_compute(float* H, int64_t d, const void* X, int32_t x_dtype, int64_t n_tok,
                                   int64_t ld_x, void* work, size_t work_bytes, void* stream) {
  return hessian_call(H, d, X, x_dtype, n_tok, ld_x, work, work_bytes, stream, true);
}

}  // extern "C"

namespace {

// The checks and the call shared by gptq_factor and gptq_factor_noalloc: work is the workspace (the
// caller's, or the static scratch), one_stream keeps every launch on the caller's stream.
gptq_status_t factor_call(const float* H, int64_t d, int64_t n_total, const gptq_params_t* p, float* U,
                          int32_t* perm, void* work, int64_t* info, hipStream_t s, bool one_stream) {
  int* status_dev = nullptr;
  int64_t* info_dev = nullptr;
  hipError_t e = gptq::factor(H, d, n_total, p->damp, p->act_order, U, perm, work, s, &status_dev, &info_dev,
                              one_stream);
  if (e != hipSuccess) return GPTQ_EHIP;
  int64_t dev_info = 0;
  int dev_status = 0;
  if (hipMemcpyAsync(&dev_info, info_dev, sizeof(dev_info), hipMemcpyDeviceToHost, s) != hipSuccess) return GPTQ_EHIP;
  if (hipMemcpyAsync(&dev_status, status_dev, sizeof(dev_status), hipMemcpyDeviceToHost, s) != hipSuccess)
    return GPTQ_EHIP;
  if (hipStreamSynchronize(s) != hipSuccess) return GPTQ_EHIP;
  // the factorization runs on the reversed order; report the processing-order column (1-based)
  *info = dev_info > 0 ? d - dev_info + 1 : 0;
  if (dev_status != 0) return GPTQ_EINVAL;
  return dev_info != 0 ? GPTQ_ENOTPD : GPTQ_OK;
}

gptq_status_t factor_args(const float* H, int64_t d, int64_t n_total, const gptq_params_t* p, const float* U,
                          const int32_t* perm, const int64_t* info) {
  if (!H || !U || !perm || !info || d <= 0 || d > kMaxDim || n_total <= 0) return GPTQ_EINVAL;
  gptq_status_t st = check_params(p, d, false);
  if (st != GPTQ_OK) return st;
  const char* h0 = reinterpret_cast<const char*>(H);
  const char* u0 = reinterpret_cast<const char*>(U);
  const size_t bytes = (size_t)d * d * sizeof(float);
  if (h0 != u0 && h0 < u0 + bytes && u0 < h0 + bytes) return GPTQ_EINVAL;   // in place, or apart
  return GPTQ_OK;
}

}  // namespace

extern "C" {

gptq_status_t gptq_factor(const float* H, int64_t d, int64_t n_total, const gptq_params_t* p, float* U,
                          int32_t* perm, void* work, size_t work_bytes, int64_t* info, void* stream) {
  gptq_status_t st = factor_args(H, d, n_total, p, U, perm, info);
  if (st != GPTQ_OK) return st;
  if (!work) return GPTQ_EINVAL;
  if (work_bytes < gptq::factor_workspace_bytes(d)) return GPTQ_ENOMEM;
  return factor_call(H, d, n_total, p, U, perm, work, info, static_cast<hipStream_t>(stream), false);
}

gptq_status_t gptq_factor_noalloc(const float* H, int64_t d, int64_t n_total, const gptq_params_t* p, float* U,
                                  int32_t* perm, int64_t* info, void* stream) {
  gptq_status_t st = factor_args(H, d, n_total, p, U, perm, info);
  if (st != GPTQ_OK) return st;
  if (d > GPTQ_FACTOR_NOALLOC_MAX_D) return GPTQ_EUNSUPPORTED;
  static_assert(GPTQ_FACTOR_NOALLOC_MAX_D == gptq::kNoallocMaxD, "scratch sized for another maximum");
  if (gptq::factor_workspace_bytes(d) > gptq::kNoallocScratchBytes) return GPTQ_EUNSUPPORTED;
  void* scratch = nullptr;
  if (gptq::noalloc_scratch(&scratch) != hipSuccess) return GPTQ_EHIP;
  return factor_call(H, d, n_total, p, U, perm, scratch, info, static_cast<hipStream_t>(stream), true);
}

}  // extern "C"

namespace {

gptq_status_t quantize_call(const void* W, int32_t w_dtype, int64_t rows, int64_t d, int64_t ld_w, const float* U,
                            const int32_t* perm, const gptq_params_t* p, uint8_t* codes, float* scales,
                            int32_t* zeros, int32_t* g_idx, double* loss, void* work, size_t work_bytes,
                            void* stream, double* part_ms) {
  if (rows < 0 || rows > kMaxDim || d <= 0 || d > kMaxDim || !dtype_ok(w_dtype)) return GPTQ_EINVAL;
  if (!U || !perm || !g_idx || !loss || !work) return GPTQ_EINVAL;
  if (rows > 0 && (!W || !codes || !scales || !zeros || ld_w < d)) return GPTQ_EINVAL;
  gptq_status_t st = check_params(p, d, true);
  if (st != GPTQ_OK) return st;
  if (work_bytes < gptq::quant_layout(rows, d, p->block_size).total) return GPTQ_ENOMEM;
  const int64_t g = p->group_size <= 0 ? d : p->group_size;
  hipStream_t s = static_cast<hipStream_t>(stream);
  return hip_status(gptq::quantize(W, w_dtype, rows, d, ld_w, U, perm, p->bits, g, p->block_size, p->sym,
                                   p->static_groups, p->compact_meta, codes, scales, zeros, g_idx, loss, work, s,
                                   part_ms));
}

}  // namespace

extern "C" {

gptq_status_t gptq_quantize_layer(const void* W, int32_t w_dtype, int64_t rows, int64_t d, int64_t ld_w,
                                  const float* U, const int32_t* perm, const gptq_params_t* p, uint8_t* codes,
                                  float* scales, int32_t* zeros, int32_t* g_idx, double* loss, void* work,
                                  size_t work_bytes, void* stream) {
  return quantize_call(W, w_dtype, rows, d, ld_w, U, perm, p, codes, scales, zeros, g_idx, loss, work, work_bytes,
                       stream, nullptr);
}

gptq_status_t gptq_quantize_layer_timed(const void* W, int32_t w_dtype, int64_t rows, int64_t d, int64_t ld_w,
                                        const float* U, const int32_t* perm, const gptq_params_t* p, uint8_t* codes,
                                        float* scales, int32_t* zeros, int32_t* g_idx, double* loss, void* work,
                                        size_t work_bytes, double* part_ms, void* stream) {
  if (!part_ms) return GPTQ_EINVAL;
  return quantize_call(W, w_dtype, rows, d, ld_w, U, perm, p, codes, scales, zeros, g_idx, loss, work, work_bytes,
                       stream, part_ms);
}

gptq_status_t gptq_pack(const uint8_t* codes, int64_t rows, int64_t d, int32_t bits, int32_t* packed, void* stream) {
  if (rows < 0 || rows > kMaxDim || d < 8 || d > kMaxDim || d % 8 != 0 || bits < 1 || bits > 8) return GPTQ_EINVAL;
  if (rows == 0) return GPTQ_OK;
  if (!codes || !packed) return GPTQ_EINVAL;
  return hip_status(gptq::pack(codes, rows, d, bits, packed, static_cast<hipStream_t>(stream)));
}

gptq_status_t gptq_pack_dense(const uint8_t* codes, int64_t rows, int64_t d, int32_t bits, int32_t* packed,
                              void* stream) {
  if (rows < 0 || rows > kMaxDim || d < 1 || d > kMaxDim || bits < 1 || bits > 8 || (d * bits) % 32 != 0)
    return GPTQ_EINVAL;
  if (rows == 0) return GPTQ_OK;
  if (!codes || !packed) return GPTQ_EINVAL;
  return hip_status(gptq::pack_dense(codes, rows, d, bits, packed, static_cast<hipStream_t>(stream)));
}

gptq_status_t gptq_pack_ordered(const uint8_t* codes, int64_t rows, int64_t d, int32_t bits, const int32_t* order,
                                int32_t* packed, void* stream) {
  if (rows < 0 || rows > kMaxDim || d < 8 || d > kMaxDim || d % 8 != 0 || bits < 1 || bits > 8) return GPTQ_EINVAL;
  if (rows == 0) return GPTQ_OK;
  if (!codes || !order || !packed) return GPTQ_EINVAL;
  return hip_status(gptq::pack_ordered(codes, rows, d, order, bits, packed, static_cast<hipStream_t>(stream)));
}

gptq_status_t gptq_permute_columns(const void* in, int32_t dtype, int64_t m, int64_t d, int64_t ld_in,
                                   const int32_t* order, void* out, int64_t ld_out, void* stream) {
  if (m < 0 || m > kMaxDim || d < 1 || d > kMaxDim || !dtype_ok(dtype) || ld_in < d || ld_out < d) return GPTQ_EINVAL;
  if (m == 0) return GPTQ_OK;
  if (!in || !order || !out) return GPTQ_EINVAL;
  const int esz = dtype == GPTQ_F32 ? 4 : 2;
  const char* i0 = static_cast<const char*>(in);
  const char* o0 = static_cast<const char*>(out);
  const int64_t in_bytes = ((m - 1) * ld_in + d) * esz, out_bytes = ((m - 1) * ld_out + d) * esz;
  if (i0 < o0 + out_bytes && o0 < i0 + in_bytes) return GPTQ_EINVAL;   // in place would race
  return hip_status(gptq::permute_columns(in, m, d, ld_in, order, esz, out, ld_out, static_cast<hipStream_t>(stream)));
}

gptq_status_t gptq_dequant_gemm(const void* x, int32_t x_dtype, int64_t m, int64_t ld_x, const int32_t* packed,
                                int32_t bits, int32_t layout, const float* scales, const int32_t* zeros,
                                const int32_t* g_idx, int64_t rows, int64_t d, int32_t group_size, float* y,
                                int64_t ld_y, void* stream) {
  if (m < 0 || m > kMaxDim || rows < 0 || rows > kMaxDim || d < 8 || d > kMaxDim || d % 8 != 0) return GPTQ_EINVAL;
  if (!dtype_ok(x_dtype) || ld_x < d || ld_x > kMaxDim || ld_y < rows || ld_y > kMaxDim) return GPTQ_EINVAL;
  if (bits < 1 || bits > 8) return GPTQ_EINVAL;
  if (layout != GPTQ_LAYOUT_FIELDS && layout != GPTQ_LAYOUT_DENSE) return GPTQ_EINVAL;
  if (layout == GPTQ_LAYOUT_DENSE && (d * bits) % 32 != 0) return GPTQ_EINVAL;
  if (m == 0 || rows == 0) return GPTQ_OK;
  if (!x || !packed || !scales || !zeros || !y) return GPTQ_EINVAL;
  const int64_t g = group_size <= 0 ? d : group_size;
  return hip_status(gptq::dequant_gemm(x, x_dtype, m, ld_x, packed, bits, layout == GPTQ_LAYOUT_DENSE, scales, zeros,
                                       g_idx, rows, d, g, y, ld_y, static_cast<hipStream_t>(stream)));
}

namespace {

// A strided [tokens x heads x width] array of esz-byte elements.
struct Tensor3 {
  const void* p;
  int64_t n, heads, width, ld, hp;
  int64_t esz;
  const char* begin() const { return static_cast<const char*>(p); }
  int64_t bytes() const {
    return n <= 0 || heads <= 0 ? 0 : ((n - 1) * ld + (heads - 1) * hp + width) * esz;
  }
};

// Pitches are not negative, and the array's bytes stay far inside int64.
bool pitches_ok(const Tensor3& t) {
  constexpr int64_t most = (int64_t)1 << 56;
  if (t.ld < 0 || t.ld > most || t.hp < 0 || t.hp > most) return false;
  const __int128 span = (__int128)t.n * t.ld + (__int128)t.heads * t.hp + t.width;
  return span * t.esz <= most;
}

// No two elements of an output share an address: tokens outside heads or heads outside tokens.
bool elements_apart(const Tensor3& t) {
  if (t.heads > 1 && t.hp < t.width) return false;
  if (t.n > 1 && t.ld < t.width) return false;
  if (t.heads <= 1 || t.n <= 1) return true;
  return t.ld >= (t.heads - 1) * t.hp + t.width || t.hp >= (t.n - 1) * t.ld + t.width;
}

// True when the arrays can be seen to share no element: address ranges apart, or column ranges of
// rows with one pitch that do not meet.
bool apart(const Tensor3& a, const Tensor3& b) {
  if (!a.bytes() || !b.bytes()) return true;
  if (a.begin() + a.bytes() <= b.begin() || b.begin() + b.bytes() <= a.begin()) return true;
  if (a.ld != b.ld || a.esz != b.esz || a.ld <= 0) return false;
  const int64_t row = a.ld * a.esz, ra = ((a.heads - 1) * a.hp + a.width) * a.esz,
                rb = ((b.heads - 1) * b.hp + b.width) * b.esz;
  int64_t off = (b.begin() - a.begin()) % row;
  if (off < 0) off += row;
  return off >= ra && off + rb <= row;
}

bool same(const Tensor3& a, const Tensor3& b) {
  return a.p == b.p && (a.ld == b.ld || a.n <= 1) && (a.hp == b.hp || a.heads <= 1);
}

int64_t elem_bytes(int32_t t) { return t == GPTQ_F32 ? 4 : 2; }

bool norm_rotate_ok(const gptq_norm_rotate_t* a) {
  if (!a || !dtype_ok(a->dtype) || !dtype_ok(a->w_dtype) || a->n < 0 || a->n >= kMaxDim) return false;
  if (a->q_heads < 1 || a->q_heads > 65535 || a->k_heads < 0 || a->k_heads > 65535) return false;
  if (a->head_dim < 1 || a->head_dim > 1024 || a->rotary_dim < 0 || a->rotary_dim > a->head_dim || a->rotary_dim % 2)
    return false;
  if ((a->interleaved != 0 && a->interleaved != 1) || (a->norm != 0 && a->norm != 1) || a->axes < 1 || a->axes > 64)
    return false;
  return std::isfinite(a->eps) && a->eps >= 0.0;
}

bool attention_ok(const gptq_attention_t* a) {
  if (!a || !dtype_ok(a->dtype) || a->seqs < 0 || a->seqs >= kMaxDim) return false;
  if (a->n_q < 0 || a->n_q > kMaxDim / 2 || a->n_kv < 0 || a->n_kv > kMaxDim / 2) return false;
  if (a->q_heads < 1 || a->q_heads > 65535 || a->kv_heads < 1 || a->kv_heads > a->q_heads ||
      a->q_heads % a->kv_heads != 0 || a->head_dim < 1 || a->head_dim > 1024)
    return false;
  if (a->causal != 0 && a->causal != 1) return false;
  // both as fp32: finite, and a cap not lost to zero
  const float scale = (float)a->scale, cap = (float)a->softcap;
  return std::isfinite(scale) && std::isfinite(cap) && a->softcap >= 0.0 && (a->softcap == 0.0 || cap >= 1e-37f);
}

}  // namespace

static constexpr int64_t kMaxRows = (int64_t)1 << 24;   // gptq_lora_gemm's outputs

size_t gptq_lora_workspace_bytes(int64_t m, int64_t d, int64_t rows, int64_t adapters, int32_t rank) {
  if (m <= 0 || m > kMaxDim || d < 1 || d > kMaxDim || rows <= 0 || rows > kMaxRows || adapters <= 0 ||
      adapters > kMaxDim || rank < 1 || rank > 256)
    return 0;
  return gptq::lora_workspace_bytes(m, d, rows, adapters, rank);
}

gptq_status_t gptq_lora_gemm(const void* x, int32_t dtype, int64_t m, int64_t ld_x, const void* A, const void* B,
                             const int32_t* ranks, const float* scales, int64_t adapters, int32_t rank,
                             const int32_t* index, int64_t rows, int64_t d, const float* base, int64_t ld_base,
                             float* y, int64_t ld_y, void* work, size_t work_bytes, void* stream) {
  if (m < 0 || m > kMaxDim || rows < 0 || rows > kMaxRows || d < 1 || d > kMaxDim || !dtype_ok(dtype)) return GPTQ_EINVAL;
  if (adapters < 0 || adapters > kMaxDim || rank < 1 || rank > 256) return GPTQ_EINVAL;
  if (ld_x < d || ld_x > kMaxDim || ld_y < rows || ld_y > kMaxDim) return GPTQ_EINVAL;
  if (base && (ld_base < rows || ld_base > kMaxDim)) return GPTQ_EINVAL;
  if (m == 0 || rows == 0) return GPTQ_OK;
  if (!x || !index || !y || (adapters > 0 && (!A || !B || !work))) return GPTQ_EINVAL;
  const Tensor3 tx{x, m, 1, d, ld_x, 0, elem_bytes(dtype)}, ty{y, m, 1, rows, ld_y, 0, 4},
      tb{base, m, 1, rows, ld_base, 0, 4};
  if (!pitches_ok(tx) || !pitches_ok(ty) || (base && !pitches_ok(tb))) return GPTQ_EINVAL;
  if (base && !same(ty, tb) && !apart(ty, tb)) return GPTQ_EINVAL;
  if (reinterpret_cast<uintptr_t>(work) % 16 != 0) return GPTQ_EINVAL;
  if (adapters > 0 && work_bytes < gptq::lora_workspace_bytes(m, d, rows, adapters, rank)) return GPTQ_ENOMEM;
  return hip_status(gptq::lora_gemm(x, dtype, m, ld_x, A, B, ranks, scales, adapters, rank, index, rows, d, base,
                                    ld_base, y, ld_y, work, static_cast<hipStream_t>(stream)));
}

gptq_status_t gptq_norm_rotate(const gptq_norm_rotate_t* a, const void* q, const void* k, const void* q_weight,
                               const void* k_weight, const int32_t* positions, const float* inv_freq,
                               const int32_t* pair_axis, void* q_out, void* k_out, void* stream) {
  if (!norm_rotate_ok(a) || (!a->norm && (q_weight || k_weight))) return GPTQ_EINVAL;
  const int64_t esz = elem_bytes(a->dtype), hk = a->k_heads, dh = a->head_dim;
  const Tensor3 q3{q, a->n, a->q_heads, dh, a->q_ld, a->q_hp, esz}, k3{k, a->n, hk, dh, a->k_ld, a->k_hp, esz},
      qo{q_out, a->n, a->q_heads, dh, a->q_out_ld, a->q_out_hp, esz},
      ko{k_out, a->n, hk, dh, a->k_out_ld, a->k_out_hp, esz};
  if (!pitches_ok(q3) || !pitches_ok(qo) || (hk && (!pitches_ok(k3) || !pitches_ok(ko)))) return GPTQ_EINVAL;
  if (a->n == 0) return GPTQ_OK;
  if (!q || !q_out || (hk && (!k || !k_out))) return GPTQ_EINVAL;
  if (a->rotary_dim && (!positions || !inv_freq)) return GPTQ_EINVAL;
  if (!elements_apart(qo) || (!same(qo, q3) && !apart(qo, q3))) return GPTQ_EINVAL;
  if (hk && (!elements_apart(ko) || (!same(ko, k3) && !apart(ko, k3)) || !apart(qo, ko) || !apart(qo, k3) ||
             !apart(ko, q3)))
    return GPTQ_EINVAL;
  return hip_status(gptq::norm_rotate(*a, q, k, q_weight, k_weight, positions, inv_freq, pair_axis, q_out, k_out,
                                      static_cast<hipStream_t>(stream)));
}

size_t gptq_attention_workspace_bytes(const gptq_attention_t* a) {
  if (!attention_ok(a) || a->seqs == 0 || a->n_q == 0) return 0;
  return gptq::attention_workspace_bytes(*a);
}

gptq_status_t gptq_attention(const gptq_attention_t* a, const void* q, const void* k, const void* v,
                             const int32_t* q_start, const int32_t* kv_start, const float* slopes,
                             const int32_t* q_doc, const int32_t* kv_doc, const int32_t* prefix, void* out, void* work,
                             size_t work_bytes, void* stream) {
  if (!attention_ok(a)) return GPTQ_EINVAL;
  if ((q_doc == nullptr) != (kv_doc == nullptr) && a->n_kv > 0) return GPTQ_EINVAL;
  const int64_t esz = elem_bytes(a->dtype), dh = a->head_dim;
  const Tensor3 q3{q, a->n_q, a->q_heads, dh, a->q_ld, a->q_hp, esz},
      k3{k, a->n_kv, a->kv_heads, dh, a->k_ld, a->k_hp, esz}, v3{v, a->n_kv, a->kv_heads, dh, a->v_ld, a->v_hp, esz},
      o3{out, a->n_q, a->q_heads, dh, a->out_ld, a->out_hp, esz};
  if (!pitches_ok(q3) || !pitches_ok(k3) || !pitches_ok(v3) || !pitches_ok(o3)) return GPTQ_EINVAL;
  if (a->seqs == 0 || a->n_q == 0) return GPTQ_OK;
  if (!q_start && a->n_q % a->seqs != 0) return GPTQ_EINVAL;
  if (!kv_start && a->n_kv % a->seqs != 0) return GPTQ_EINVAL;
  if (!q || !out || (a->n_kv > 0 && (!k || !v))) return GPTQ_EINVAL;
  if (!elements_apart(o3) || !apart(o3, q3) || !apart(o3, k3) || !apart(o3, v3)) return GPTQ_EINVAL;
  if (reinterpret_cast<uintptr_t>(work) % 16 != 0) return GPTQ_EINVAL;
  if (!gptq::attention_fits(*a)) return GPTQ_EUNSUPPORTED;
  return hip_status(gptq::attention(*a, q, k, v, q_start, kv_start, slopes, q_doc, kv_doc, prefix, out, work,
                                    work ? work_bytes : 0, static_cast<hipStream_t>(stream)));
}

namespace {

bool block_shape_ok(const gptq_block_shape_t* sh) {
  if (!sh) return false;
  if (sh->hidden < 8 || sh->hidden > kMaxDim || sh->inter < 8 || sh->inter > kMaxDim) return false;
  if (sh->heads < 1 || sh->heads > 65535 || sh->hidden % sh->heads != 0) return false;
  if (sh->seqs < 1 || sh->seq_len < 1 || sh->seq_len > kMaxDim || sh->seqs > kMaxDim / sh->seq_len) return false;
  if (sh->heads * sh->seq_len > kMaxDim) return false;   // softmax rows of one sequence, one workgroup each
  return std::isfinite(sh->eps) && sh->eps >= 0.0;
}

bool block_attn_ok(const gptq_block_shape_t& sh, const gptq_block_attn_t* at) {
  if (!at || at->kv_heads < 1 || at->kv_heads > sh.heads || sh.heads % at->kv_heads != 0) return false;
  const gptq_norm_rotate_t r = gptq::block_rotate(sh, *at);
  const gptq_attention_t t = gptq::block_attention(sh, *at);
  if (!norm_rotate_ok(&r) || !attention_ok(&t)) return false;
  if (!at->qk_norm && (at->q_norm || at->k_norm)) return false;
  return !at->rotary_dim || (at->inv_freq && at->positions);
}

// gptq_quantize_block and gptq_quantize_block_attn (attn not null)
gptq_status_t block_call(const gptq_block_shape_t* shape, const gptq_block_attn_t* attn, const void* X, int32_t x_dtype,
                         const gptq_params_t* p, int32_t true_sequential, const gptq_block_layer_t* layers, float* Y,
                         float* const* hess, void* work, size_t work_bytes, int64_t* info, void* stream) {
  if (!X || !dtype_ok(x_dtype) || !layers || !Y || !work || !info) return GPTQ_EINVAL;
  if (true_sequential != 0 && true_sequential != 1) return GPTQ_EINVAL;
  gptq_status_t st = check_params(p, std::min(shape->hidden, shape->inter), true);
  if (st != GPTQ_OK) return st;
  if ((st = check_params(p, std::max(shape->hidden, shape->inter), true)) != GPTQ_OK) return st;
  for (int i = 0; i < 7; ++i) {
    const gptq_block_layer_t& l = layers[i];
    if (!l.W || !l.codes || !l.scales || !l.zeros || !l.g_idx || !l.perm || !l.loss || !dtype_ok(l.w_dtype))
      return GPTQ_EINVAL;
  }
  if (attn && !gptq::attention_fits(gptq::block_attention(*shape, *attn))) return GPTQ_EUNSUPPORTED;
  if (work_bytes < gptq::block_layout(*shape, attn, *p).total) return GPTQ_ENOMEM;
  return gptq::quantize_block(*shape, attn, X, x_dtype, *p, true_sequential, layers, Y, hess,
                              static_cast<char*>(work), info, static_cast<hipStream_t>(stream));
}

}  // namespace

size_t gptq_block_workspace_bytes(const gptq_block_shape_t* shape, const gptq_params_t* p) {
  if (!block_shape_ok(shape) || !p || p->block_size < 1 || p->block_size > 128) return 0;
  return gptq::block_layout(*shape, nullptr, *p).total;
}

size_t gptq_block_attn_workspace_bytes(const gptq_block_shape_t* shape, const gptq_block_attn_t* attn,
                                       const gptq_params_t* p) {
  if (!block_shape_ok(shape) || !block_attn_ok(*shape, attn) || !p || p->block_size < 1 || p->block_size > 128) return 0;
  if (!gptq::attention_fits(gptq::block_attention(*shape, *attn))) return 0;
  return gptq::block_layout(*shape, attn, *p).total;
}

gptq_status_t gptq_quantize_block(const gptq_block_shape_t* shape, const void* X, int32_t x_dtype,
                                  const gptq_params_t* p, int32_t true_sequential, const gptq_block_layer_t* layers,
                                  float* Y, float* const* hess, void* work, size_t work_bytes, int64_t* info,
                                  void* stream) {
  if (info) info[0] = -1, info[1] = 0;
  if (!block_shape_ok(shape)) return GPTQ_EINVAL;
  return block_call(shape, nullptr, X, x_dtype, p, true_sequential, layers, Y, hess, work, work_bytes, info, stream);
}

gptq_status_t gptq_quantize_block_attn(const gptq_block_shape_t* shape, const gptq_block_attn_t* attn, const void* X,
                                       int32_t x_dtype, const gptq_params_t* p, int32_t true_sequential,
                                       const gptq_block_layer_t* layers, float* Y, float* const* hess, void* work,
                                       size_t work_bytes, int64_t* info, void* stream) {
  if (info) info[0] = -1, info[1] = 0;
  if (!block_shape_ok(shape) || !block_attn_ok(*shape, attn)) return GPTQ_EINVAL;
  return block_call(shape, attn, X, x_dtype, p, true_sequential, layers, Y, hess, work, work_bytes, info, stream);
}

}  // extern "C"
