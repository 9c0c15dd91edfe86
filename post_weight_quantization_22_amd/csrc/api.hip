// extern "C" entry points: argument validation, workspace sizing, launches.
// Every check here runs on the host before anything is enqueued.
#include <cmath>

#include "kernels.hpp"

using namespace gptq;

namespace {

constexpr int64_t kMaxDim = int64_t(1) << 24;  // sanity bound on m, n

inline bool bad_dim(int64_t v) { return v < 0 || v > kMaxDim; }

inline gptq_status hip_status(hipError_t e) { return e == hipSuccess ? GPTQ_OK : GPTQ_ERR_HIP; }

inline bool valid_dtype(int dt) { return dt == GPTQ_F32 || dt == GPTQ_BF16; }

inline bool quant_group_ok(int32_t g) {
  return g == -1 || g == 8 || g == 16 || g == 32 || g == 64 || g == 128 || g == 256 || g == 512;
}

gptq_status check_ws(void* ws, size_t ws_bytes, size_t need) {
  if (need == 0) return GPTQ_OK;
  if (ws == nullptr || ws_bytes < need) return GPTQ_ERR_WORKSPACE;
  return GPTQ_OK;
}

// a tile's rows are addressed by a 24-bit product with the row stride, which for
// fp8_linear's own codes is n rounded up to 128
constexpr int64_t kFp8MaxStride = (int64_t(1) << 24) - 128;

// what fp8_gemm and fp8_linear share; GPTQ_OK also where there is nothing to do
gptq_status fp8_operands_ok(int64_t tokens, int64_t n, const void* W, int64_t m, int64_t ldw,
                            const float* wscales, int64_t ldws, const void* Y, int ydt,
                            int64_t ldy) {
  if (bad_dim(tokens) || bad_dim(m) || n <= 0 || bad_dim(n) || !valid_dtype(ydt))
    return GPTQ_ERR_INVALID_ARG;
  if (n % 16 != 0) return GPTQ_ERR_UNSUPPORTED;
  if (tokens == 0 || m == 0) return GPTQ_OK;
  if (!W || !wscales || !Y || ldw < n || ldw % 16 != 0 || ldy < m ||
      (reinterpret_cast<uintptr_t>(W) & 15) != 0 || ldws < ceil_div(n, int64_t(128)))
    return GPTQ_ERR_INVALID_ARG;
  return ldw > kFp8MaxStride ? GPTQ_ERR_UNSUPPORTED : GPTQ_OK;
}

gptq_status kv_cache_ok(const gptq_kv_cache* c, int64_t tokens) {
  if (!c || !c->codes || !c->scales || c->pages <= 0 || c->page_size <= 0 || c->heads <= 0 ||
      c->head_dim <= 0)
    return GPTQ_ERR_INVALID_ARG;
  if (c->format != GPTQ_KV_INT4 && c->format != GPTQ_KV_INT8 && c->format != GPTQ_KV_E4M3)
    return GPTQ_ERR_INVALID_ARG;
  const int32_t g = c->group_size;
  if (g != -1 && (g < 16 || g > 512 || (g & (g - 1)) != 0)) return GPTQ_ERR_INVALID_ARG;
  // (the lanes of a token are counted in 22 bits, slots in 31)
  if (c->head_dim % 8 != 0 || c->head_dim > 1024 || (g == -1 && c->head_dim > 512) ||
      int64_t(c->heads) * (c->head_dim / 8) > (int64_t(1) << 20) ||
      c->pages > INT32_MAX / c->page_size)
    return GPTQ_ERR_UNSUPPORTED;
  // an expanded dimension would have two places share their bytes
  if ((c->pages > 1 && (c->page_stride == 0 || c->param_page_stride == 0)) ||
      (c->page_size > 1 && (c->slot_stride == 0 || c->param_slot_stride == 0)) ||
      (c->heads > 1 && (c->head_stride == 0 || c->param_head_stride == 0)))
    return GPTQ_ERR_INVALID_ARG;
  const int a = c->format == GPTQ_KV_INT4 ? 4 : 8;
  if ((reinterpret_cast<uintptr_t>(c->codes) % a) != 0 || c->page_stride % a != 0 ||
      c->slot_stride % a != 0 || c->head_stride % a != 0)
    return GPTQ_ERR_INVALID_ARG;
  // a token's lanes: at most twice its 8-value chunks (a short last group)
  if (tokens * c->heads * (c->head_dim / 8) * 2 >= (int64_t(1) << 31)) return GPTQ_ERR_UNSUPPORTED;
  return GPTQ_OK;
}

gptq_status kv_call_ok(const void* K, const void* V, int dt, int64_t tokens, const int64_t* slots,
                       const gptq_kv_cache* kc, const gptq_kv_cache* vc) {
  if (bad_dim(tokens) || !valid_dtype(dt) || (!kc && !vc)) return GPTQ_ERR_INVALID_ARG;
  for (const gptq_kv_cache* c : {kc, vc})
    if (c) {
      const gptq_status ok = kv_cache_ok(c, tokens);
      if (ok != GPTQ_OK) return ok;
    }
  if (kc && vc && (kc->pages != vc->pages || kc->page_size != vc->page_size))
    return GPTQ_ERR_INVALID_ARG;
  if (tokens == 0) return GPTQ_OK;
  if (!slots || (K != nullptr) != (kc != nullptr) || (V != nullptr) != (vc != nullptr))
    return GPTQ_ERR_INVALID_ARG;
  return GPTQ_OK;
}

}  // namespace

extern "C" {

uint32_t gptq_abi_version(void) { return GPTQ_ABI_VERSION; }

const char* gptq_status_str(int32_t status) {
  switch (status) {
    case GPTQ_OK: return "ok";
    case GPTQ_ERR_INVALID_ARG: return "invalid argument";
    case GPTQ_ERR_NOT_PD: return "damped Hessian is not positive definite (raise perc_damp)";
    case GPTQ_ERR_NONFINITE: return "non-finite value in the input";
    case GPTQ_ERR_EMPTY: return "no calibration tokens";
    case GPTQ_ERR_WORKSPACE: return "workspace missing or too small";
    case GPTQ_ERR_HIP: return "HIP runtime error";
    case GPTQ_ERR_UNSUPPORTED: return "configuration not supported by this library";
    default: return "unknown status";
  }
}

gptq_status gptq_hessian_workspace_size(int64_t n, int64_t tokens, size_t* bytes) {
  if (!bytes || n <= 0 || bad_dim(n) || tokens < 0) return GPTQ_ERR_INVALID_ARG;
  *bytes = hessian_ws_bytes(n, tokens, GPTQ_BF16);
  return GPTQ_OK;
}

gptq_status gptq_hessian_accumulate(float* S, int64_t n, int64_t lds, const void* X,
                                    gptq_dtype xdt, int64_t tokens, int64_t ldx, void* ws,
                                    size_t ws_bytes, hipStream_t stream) {
  if (!S || n <= 0 || bad_dim(n) || lds < n || tokens < 0 || !valid_dtype(xdt))
    return GPTQ_ERR_INVALID_ARG;
  if (tokens == 0) return GPTQ_OK;
  if (!X || ldx < n) return GPTQ_ERR_INVALID_ARG;
  const gptq_status w = check_ws(ws, ws_bytes, hessian_ws_bytes(n, tokens, xdt));
  if (w != GPTQ_OK) return w;
  return hip_status(launch_hessian(S, n, lds, X, xdt, tokens, ldx, ws, ws_bytes, stream));
}

gptq_status gptq_prepare_workspace_size(int64_t n, size_t* bytes) {
  if (!bytes || n <= 0 || bad_dim(n)) return GPTQ_ERR_INVALID_ARG;
  *bytes = prepare_ws_bytes(n);
  return GPTQ_OK;
}

gptq_status gptq_prepare(const float* S, int64_t n, int64_t lds, int64_t tokens, float perc_damp,
                         int32_t desc_act, float* U, int64_t ldu, int32_t* perm, uint8_t* dead,
                         float* lambda_out, int32_t* info, void* ws, size_t ws_bytes,
                         hipStream_t stream) {
  if (!S || !U || !info || n <= 0 || bad_dim(n) || lds < n || ldu < n || tokens < 0 ||
      !(perc_damp >= 0.0f) || !std::isfinite(perc_damp) || (desc_act != 0 && desc_act != 1))
    return GPTQ_ERR_INVALID_ARG;
  if (U == S && ldu != lds) return GPTQ_ERR_INVALID_ARG;
  if (tokens == 0) return GPTQ_ERR_EMPTY;
  const gptq_status w = check_ws(ws, ws_bytes, prepare_ws_bytes(n));
  if (w != GPTQ_OK) return w;
  return hip_status(launch_prepare(S, n, lds, perc_damp, desc_act, U, ldu, perm, dead, lambda_out,
                                   info, ws, stream));
}

gptq_status gptq_quantize_workspace_size(int64_t m, int64_t n, const gptq_config* cfg,
                                         size_t* bytes) {
  if (!bytes || !cfg || bad_dim(m) || bad_dim(n)) return GPTQ_ERR_INVALID_ARG;
  *bytes = quantize_ws_bytes(m, n, cfg->desc_act);
  return GPTQ_OK;
}

gptq_status gptq_quantize_layer(const void* W, gptq_dtype wdt, int64_t m, int64_t n, int64_t ldw,
                                const float* U, int64_t ldu, const int32_t* perm,
                                const uint8_t* dead, const gptq_config* cfg, uint8_t* codes,
                                float* scales, float* zeros, int32_t* g_idx, float* row_err,
                                int32_t* info, void* ws, size_t ws_bytes, hipStream_t stream) {
  return quantize_layer_checked(W, wdt, m, n, ldw, U, ldu, perm, dead, cfg, codes, scales, zeros,
                                g_idx, row_err, info, ws, ws_bytes, stream);
}

gptq_status gptq_pack(const uint8_t* codes, int64_t m, int64_t n, int32_t bits, uint32_t* packed,
                      hipStream_t stream) {
  if (bad_dim(m) || bad_dim(n) || bits < 1 || bits > 8) return GPTQ_ERR_INVALID_ARG;
  if (m == 0 || n == 0) return GPTQ_OK;
  if (!codes || !packed) return GPTQ_ERR_INVALID_ARG;
  return hip_status(launch_pack(codes, m, n, bits, nullptr, packed, stream));
}

gptq_status gptq_pack_ordered(const uint8_t* codes, int64_t m, int64_t n, int32_t bits,
                              const int32_t* perm, uint32_t* packed, hipStream_t stream) {
  if (bad_dim(m) || bad_dim(n) || bits < 1 || bits > 8) return GPTQ_ERR_INVALID_ARG;
  if (m == 0 || n == 0) return GPTQ_OK;
  if (!codes || !packed) return GPTQ_ERR_INVALID_ARG;
  return hip_status(launch_pack(codes, m, n, bits, perm, packed, stream));
}

gptq_status gptq_dequant_gemm_workspace_size(int64_t tokens, int64_t m, int64_t n,
                                             int32_t has_perm, size_t* bytes) {
  if (!bytes || tokens < 0 || bad_dim(tokens) || bad_dim(m) || bad_dim(n) ||
      (has_perm != 0 && has_perm != 1))
    return GPTQ_ERR_INVALID_ARG;
  *bytes = (tokens == 0 || m == 0 || n == 0) ? 0 : dequant_gemm_ws_bytes(tokens, m, n, has_perm);
  return GPTQ_OK;
}

gptq_status gptq_dequantize(const uint32_t* packed, int64_t ldp, int32_t bits,
                            int32_t group_size, const float* scales, const float* zeros,
                            int64_t m, int64_t n, void* W, int64_t ldw, hipStream_t stream) {
  if (bad_dim(m) || n <= 0 || bad_dim(n) || bits < 2 || bits > 8 ||
      !(group_size == -1 || (group_size >= 8 && group_size % 8 == 0)))
    return GPTQ_ERR_INVALID_ARG;
  if (n % 8 != 0) return GPTQ_ERR_UNSUPPORTED;
  if (m == 0) return GPTQ_OK;
  if (!packed || !scales || !zeros || !W || ldp < ceil_div(n * bits, 32) || ldw < n ||
      ldw % 8 != 0 || (reinterpret_cast<uintptr_t>(W) & 15) != 0)
    return GPTQ_ERR_INVALID_ARG;
  return hip_status(launch_dequantize(packed, ldp, bits, m, n, scales, zeros, group_size,
                                      static_cast<uint16_t*>(W), ldw, stream));
}

gptq_status gptq_gemm_bf16(const void* X, int64_t tokens, int64_t n, int64_t ldx, const void* W,
                           int64_t m, int64_t ldw, void* Y, gptq_dtype ydt, int64_t ldy,
                           hipStream_t stream) {
  if (tokens < 0 || bad_dim(tokens) || bad_dim(m) || n <= 0 || bad_dim(n) || !valid_dtype(ydt))
    return GPTQ_ERR_INVALID_ARG;
  if (n % 8 != 0) return GPTQ_ERR_UNSUPPORTED;
  if (tokens == 0 || m == 0) return GPTQ_OK;
  if (!X || !W || !Y || ldx < n || ldw < n || ldy < m || ldx % 8 != 0 || ldw % 8 != 0 ||
      (reinterpret_cast<uintptr_t>(X) & 15) != 0 || (reinterpret_cast<uintptr_t>(W) & 15) != 0)
    return GPTQ_ERR_INVALID_ARG;
  // the DMA offsets within a tile are 32-bit
  if (ldx >= (int64_t(1) << 23) || ldw >= (int64_t(1) << 23)) return GPTQ_ERR_UNSUPPORTED;
  return hip_status(launch_dense_gemm(static_cast<const uint16_t*>(X), ldx, tokens, n,
                                      static_cast<const uint16_t*>(W), ldw, m, Y, ldy,
                                      ydt == GPTQ_BF16 ? 1 : 0, stream));
}

gptq_status gptq_gather_columns(const void* X, gptq_dtype xdt, int64_t tokens, int64_t n,
                                int64_t ldx, const int32_t* perm, void* Xp, int64_t ldxp,
                                hipStream_t stream) {
  if (tokens < 0 || bad_dim(tokens) || n <= 0 || bad_dim(n) || !valid_dtype(xdt))
    return GPTQ_ERR_INVALID_ARG;
  if (xdt != GPTQ_BF16) return GPTQ_ERR_UNSUPPORTED;
  if (tokens == 0) return GPTQ_OK;
  if (!X || !perm || !Xp || ldx < n || ldxp < n || ldxp % 8 != 0 ||
      (reinterpret_cast<uintptr_t>(Xp) & 15) != 0)
    return GPTQ_ERR_INVALID_ARG;
  launch_gather(static_cast<const uint16_t*>(X), ldx, perm, tokens, n, ldxp,
                static_cast<uint16_t*>(Xp), stream);
  return hip_status(hipGetLastError());
}

gptq_status gptq_dequant_gemm(const void* X, gptq_dtype xdt, int64_t tokens, int64_t n,
                              int64_t ldx, const uint32_t* packed, int64_t ldp, int32_t bits,
                              int32_t group_size, const float* scales, const float* zeros,
                              const int32_t* perm, int64_t m, void* Y, gptq_dtype ydt,
                              int64_t ldy, void* ws, size_t ws_bytes, hipStream_t stream) {
  if (tokens < 0 || bad_dim(tokens) || bad_dim(m) || n <= 0 || bad_dim(n) || bits < 2 ||
      bits > 8 || !valid_dtype(xdt) || !valid_dtype(ydt) ||
      !(group_size == -1 || (group_size >= 8 && group_size % 8 == 0)))
    return GPTQ_ERR_INVALID_ARG;
  if (xdt != GPTQ_BF16) return GPTQ_ERR_UNSUPPORTED;
  if (tokens == 0 || m == 0) return GPTQ_OK;
  if (!X || !packed || !scales || !zeros || !Y || ldx < n || ldp < ceil_div(n * bits, 32) ||
      ldy < m)
    return GPTQ_ERR_INVALID_ARG;
  // X is read with 16-byte loads unless the permutation gathers it first
  if (!perm && (ldx % 8 != 0 || (reinterpret_cast<uintptr_t>(X) & 15) != 0))
    return GPTQ_ERR_INVALID_ARG;
  const gptq_status w =
      check_ws(ws, ws_bytes, dequant_gemm_ws_bytes(tokens, m, n, perm != nullptr ? 1 : 0));
  if (w != GPTQ_OK) return w;
  DequantArgs d;
  d.X = X;
  d.tokens = tokens;
  d.n = n;
  d.ldx = ldx;
  d.packed = packed;
  d.ldp = ldp;
  d.bits = bits;
  d.group_size = group_size;
  d.scales = scales;
  d.zeros = zeros;
  d.perm = perm;
  d.m = m;
  d.Y = Y;
  d.ydt = ydt;
  d.ldy = ldy;
  d.ws = ws;
  return hip_status(launch_dequant_gemm(d, stream));
}

gptq_status gptq_swiglu(const float* gate, int64_t ldg, const float* up, int64_t ldu,
                        int64_t tokens, int64_t n, void* h, int64_t ldh, hipStream_t stream) {
  if (tokens < 0 || bad_dim(tokens) || n < 0 || bad_dim(n)) return GPTQ_ERR_INVALID_ARG;
  if (tokens == 0 || n == 0) return GPTQ_OK;
  if (!gate || !up || !h || ldg < n || ldu < n || ldh < n) return GPTQ_ERR_INVALID_ARG;
  return hip_status(launch_swiglu(gate, ldg, up, ldu, tokens, n, h, ldh, stream));
}

gptq_status gptq_residual_add(const void* x, int64_t ldx, const float* y, int64_t ldy,
                              int64_t tokens, int64_t n, void* out, int64_t ldo,
                              hipStream_t stream) {
  if (tokens < 0 || bad_dim(tokens) || n < 0 || bad_dim(n)) return GPTQ_ERR_INVALID_ARG;
  if (tokens == 0 || n == 0) return GPTQ_OK;
  if (!x || !y || !out || ldx < n || ldy < n || ldo < n) return GPTQ_ERR_INVALID_ARG;
  return hip_status(launch_residual_add(x, ldx, y, ldy, tokens, n, out, ldo, stream));
}

gptq_status awq_absum_workspace_size(int64_t n, int64_t tokens, size_t* bytes) {
  if (!bytes || n <= 0 || bad_dim(n) || tokens < 0) return GPTQ_ERR_INVALID_ARG;
  *bytes = awq_absum_ws_bytes(n, tokens);
  return GPTQ_OK;
}

gptq_status awq_activation_absum(const void* X, gptq_dtype xdt, int64_t tokens, int64_t n,
                                 int64_t ldx, float* absum, void* ws, size_t ws_bytes,
                                 hipStream_t stream) {
  if (!absum || n <= 0 || bad_dim(n) || tokens < 0 || !valid_dtype(xdt))
    return GPTQ_ERR_INVALID_ARG;
  if (tokens == 0) return GPTQ_OK;
  if (!X || ldx < n) return GPTQ_ERR_INVALID_ARG;
  const gptq_status w = check_ws(ws, ws_bytes, awq_absum_ws_bytes(n, tokens));
  if (w != GPTQ_OK) return w;
  return hip_status(launch_awq_absum(X, xdt, tokens, n, ldx, absum, ws, stream));
}

gptq_status awq_lite_workspace_size(int64_t m, int64_t n, size_t* bytes) {
  if (!bytes || m <= 0 || n <= 0 || bad_dim(m) || bad_dim(n)) return GPTQ_ERR_INVALID_ARG;
  *bytes = awq_lite_ws_bytes(m, n);
  return GPTQ_OK;
}

gptq_status awq_lite(const void* W, gptq_dtype wdt, int64_t m, int64_t n, int64_t ldw,
                     const float* S, int64_t lds, const float* absum, int64_t tokens,
                     int32_t bits, int32_t group_size, int32_t sym, int32_t n_alpha,
                     float* s_out, float* alpha_out, float* losses, void* ws, size_t ws_bytes,
                     hipStream_t stream) {
  if (!W || !S || !absum || !s_out || !alpha_out || !losses || m <= 0 || n <= 0 ||
      bad_dim(m) || bad_dim(n) || ldw < n || lds < n || !valid_dtype(wdt) || bits < 2 ||
      bits > 8 || group_size == 0 || group_size < -1 || (sym != 0 && sym != 1) ||
      n_alpha < 2 || n_alpha > 101)
    return GPTQ_ERR_INVALID_ARG;
  if (tokens <= 0) return GPTQ_ERR_EMPTY;
  const gptq_status w = check_ws(ws, ws_bytes, awq_lite_ws_bytes(m, n));
  if (w != GPTQ_OK) return w;
  return hip_status(launch_awq_lite(W, wdt, m, n, ldw, S, lds, absum, tokens, bits, group_size,
                                    sym, n_alpha, s_out, alpha_out, losses, ws, stream));
}

gptq_status gptq_layer_error_workspace_size(int64_t m, int64_t n, size_t* bytes) {
  if (!bytes || bad_dim(m) || n <= 0 || bad_dim(n)) return GPTQ_ERR_INVALID_ARG;
  *bytes = layer_error_ws_bytes(m, n);
  return GPTQ_OK;
}

gptq_status gptq_layer_error(const void* W, gptq_dtype wdt, int64_t m, int64_t n, int64_t ldw,
                             const uint8_t* codes, const float* scales, const float* zeros,
                             int64_t ngroups, const int32_t* g_idx, const float* S, int64_t lds,
                             double* err, void* ws, size_t ws_bytes, hipStream_t stream) {
  if (!W || !codes || !scales || !zeros || !g_idx || !S || !err || bad_dim(m) || n <= 0 ||
      bad_dim(n) || ldw < n || lds < n || ngroups < 1 || ngroups > n || !valid_dtype(wdt))
    return GPTQ_ERR_INVALID_ARG;
  if (m == 0) return GPTQ_OK;
  const gptq_status w = check_ws(ws, ws_bytes, layer_error_ws_bytes(m, n));
  if (w != GPTQ_OK) return w;
  return hip_status(launch_layer_error(W, wdt, m, n, ldw, codes, scales, zeros, ngroups, g_idx, S,
                                       lds, err, ws, stream));
}

gptq_status awq_clip_quantize(const void* W, gptq_dtype wdt, int64_t m, int64_t n, int64_t ldw,
                              const float* S, int64_t lds, const float* s, int32_t bits,
                              int32_t group_size, int32_t sym, int32_t n_steps, uint8_t* codes,
                              float* scales, float* zeros, uint8_t* clip_idx,
                              hipStream_t stream) {
  if (!W || !S || !codes || !scales || !zeros || m < 0 || n <= 0 || bad_dim(m) || bad_dim(n) ||
      ldw < n || lds < n || !valid_dtype(wdt) || bits < 2 || bits > 8 || group_size < 1 ||
      (sym != 0 && sym != 1) || n_steps < 1 || n_steps > 11)
    return GPTQ_ERR_INVALID_ARG;
  if (group_size > 128) return GPTQ_ERR_UNSUPPORTED;
  if (m == 0) return GPTQ_OK;
  return hip_status(launch_awq_clip(W, wdt, m, n, ldw, S, lds, s, bits, group_size, sym, n_steps,
                                    codes, scales, zeros, clip_idx, stream));
}

gptq_status rtn_minmax(const void* W, gptq_dtype wdt, int64_t m, int64_t n, int64_t ldw,
                       int32_t bits, int32_t group_size, int32_t sym, uint8_t* codes,
                       float* scales, float* zeros, hipStream_t stream) {
  if (bad_dim(m) || bad_dim(n) || !valid_dtype(wdt) || bits < 2 || bits > 8 ||
      group_size == 0 || group_size < -1 || (sym != 0 && sym != 1))
    return GPTQ_ERR_INVALID_ARG;
  if (m == 0 || n == 0) return GPTQ_OK;
  if (!W || !codes || !scales || !zeros || ldw < n) return GPTQ_ERR_INVALID_ARG;
  return hip_status(launch_rtn(W, wdt, m, n, ldw, bits, group_size, sym, codes, scales, zeros,
                               stream));
}

gptq_status fp8_quantize_rows(const void* X, gptq_dtype xdt, int64_t tokens, int64_t n,
                              int64_t ldx, uint8_t* codes, int64_t ldc, float* scales,
                              int64_t lds, hipStream_t stream) {
  if (tokens < 0 || bad_dim(tokens) || n <= 0 || bad_dim(n) || !valid_dtype(xdt))
    return GPTQ_ERR_INVALID_ARG;
  if (tokens == 0) return GPTQ_OK;
  if (!X || !codes || !scales || ldx < n || ldc < n || lds < tokens || codes == X)
    return GPTQ_ERR_INVALID_ARG;
  return hip_status(launch_fp8_rows(X, ldx, nullptr, 0, xdt, tokens, n, codes, ldc, scales, lds,
                                    stream));
}

gptq_status fp8_swiglu_quantize(const void* gate, int64_t ldg, const void* up, int64_t ldu,
                                gptq_dtype dt, int64_t tokens, int64_t n, uint8_t* codes,
                                int64_t ldc, float* scales, int64_t lds, hipStream_t stream) {
  if (tokens < 0 || bad_dim(tokens) || n <= 0 || bad_dim(n) || !valid_dtype(dt))
    return GPTQ_ERR_INVALID_ARG;
  if (tokens == 0) return GPTQ_OK;
  if (!gate || !up || !codes || !scales || ldg < n || ldu < n || ldc < n || lds < tokens ||
      codes == gate || codes == up)
    return GPTQ_ERR_INVALID_ARG;
  return hip_status(launch_fp8_rows(gate, ldg, up, ldu, dt, tokens, n, codes, ldc, scales, lds,
                                    stream));
}

gptq_status fp8_quantize_blocks(const void* W, gptq_dtype wdt, int64_t m, int64_t n, int64_t ldw,
                                uint8_t* codes, int64_t ldc, float* scales, int64_t lds,
                                hipStream_t stream) {
  if (m < 0 || bad_dim(m) || n <= 0 || bad_dim(n) || !valid_dtype(wdt))
    return GPTQ_ERR_INVALID_ARG;
  if (m == 0) return GPTQ_OK;
  if (!W || !codes || !scales || ldw < n || ldc < n || lds < ceil_div(n, int64_t(128)) ||
      codes == W)
    return GPTQ_ERR_INVALID_ARG;
  return hip_status(launch_fp8_blocks(W, wdt, m, n, ldw, codes, ldc, scales, lds, stream));
}

gptq_status fp8_gemm_workspace_size(int64_t tokens, int64_t m, int64_t n, size_t* bytes) {
  if (!bytes || tokens < 0 || bad_dim(tokens) || m < 0 || bad_dim(m) || n <= 0 || bad_dim(n))
    return GPTQ_ERR_INVALID_ARG;
  *bytes = tokens == 0 || m == 0 ? 0 : fp8_gemm_ws_bytes(tokens, m, n);
  return GPTQ_OK;
}

gptq_status fp8_linear_workspace_size(int64_t tokens, int64_t m, int64_t n, size_t* bytes) {
  if (!bytes || tokens < 0 || bad_dim(tokens) || m < 0 || bad_dim(m) || n <= 0 || bad_dim(n))
    return GPTQ_ERR_INVALID_ARG;
  *bytes = tokens == 0 || m == 0 ? 0 : fp8_linear_ws_bytes(tokens, m, n);
  return GPTQ_OK;
}

gptq_status fp8_gemm(const uint8_t* X, int64_t tokens, int64_t n, int64_t ldx, const float* xs,
                     int64_t ldxs, const uint8_t* W, int64_t m, int64_t ldw, const float* wscales,
                     int64_t ldws, const void* R, int64_t ldr, void* Y, gptq_dtype ydt,
                     int64_t ldy, void* ws, size_t ws_bytes, hipStream_t stream) {
  const gptq_status ok = fp8_operands_ok(tokens, n, W, m, ldw, wscales, ldws, Y, ydt, ldy);
  if (ok != GPTQ_OK || tokens == 0 || m == 0) return ok;
  if (!X || !xs || ldx < n || ldx % 16 != 0 || (reinterpret_cast<uintptr_t>(X) & 15) != 0 ||
      ldxs < tokens || (R && ldr < m) || (R == Y && ldr != ldy))
    return GPTQ_ERR_INVALID_ARG;
  if (ldx > kFp8MaxStride) return GPTQ_ERR_UNSUPPORTED;
  const gptq_status w = check_ws(ws, ws_bytes, fp8_gemm_ws_bytes(tokens, m, n));
  if (w != GPTQ_OK) return w;
  if ((reinterpret_cast<uintptr_t>(ws) & 15) != 0 || X == Y) return GPTQ_ERR_INVALID_ARG;
  Fp8GemmArgs g{X, ldx, tokens, n, xs, ldxs, W, ldw, m, wscales, ldws, Y, ydt, ldy, R, ldr, ws};
  return hip_status(launch_fp8_gemm(g, stream));
}

gptq_status fp8_linear(const void* X, gptq_dtype xdt, int64_t tokens, int64_t n, int64_t ldx,
                       const uint8_t* W, int64_t m, int64_t ldw, const float* wscales,
                       int64_t ldws, void* Y, gptq_dtype ydt, int64_t ldy, void* ws,
                       size_t ws_bytes, hipStream_t stream) {
  const gptq_status ok = fp8_operands_ok(tokens, n, W, m, ldw, wscales, ldws, Y, ydt, ldy);
  if (ok != GPTQ_OK) return ok;
  if (!valid_dtype(xdt)) return GPTQ_ERR_INVALID_ARG;
  if (tokens == 0 || m == 0) return GPTQ_OK;
  if (!X || ldx < n) return GPTQ_ERR_INVALID_ARG;
  const gptq_status w = check_ws(ws, ws_bytes, fp8_linear_ws_bytes(tokens, m, n));
  if (w != GPTQ_OK) return w;
  // the codes lie at the workspace's start and are read 16 bytes at a time; a small
  // batch's workgroups read X while others write Y
  if ((reinterpret_cast<uintptr_t>(ws) & 15) != 0 || X == Y) return GPTQ_ERR_INVALID_ARG;
  Fp8GemmArgs g{nullptr, 0, tokens, n, nullptr, 0, W, ldw, m, wscales, ldws, Y, ydt, ldy,
                nullptr, 0, nullptr};
  return hip_status(launch_fp8_linear(X, xdt, ldx, g, ws, stream));
}

gptq_status fp8_gated_gemm_workspace_size(int64_t tokens, int64_t m, int64_t n, size_t* bytes) {
  if (!bytes || tokens < 0 || bad_dim(tokens) || m < 0 || bad_dim(m) || n <= 0 || bad_dim(n))
    return GPTQ_ERR_INVALID_ARG;
  *bytes = tokens == 0 || m == 0 ? 0 : fp8_gated_ws_bytes(tokens, m, n);
  return GPTQ_OK;
}

gptq_status fp8_gated_gemm(const uint8_t* X, int64_t tokens, int64_t n, int64_t ldx,
                           const float* xs, int64_t ldxs, const uint8_t* Wg, int64_t m,
                           int64_t ldwg, const float* gscales, int64_t ldgs, const uint8_t* Wu,
                           int64_t ldwu, const float* uscales, int64_t ldus, uint8_t* codes,
                           int64_t ldc, float* scales, int64_t lds, void* ws, size_t ws_bytes,
                           hipStream_t stream) {
  for (int up = 0; up < 2; ++up) {
    const gptq_status ok =
        fp8_operands_ok(tokens, n, up ? Wu : Wg, m, up ? ldwu : ldwg, up ? uscales : gscales,
                        up ? ldus : ldgs, codes, GPTQ_BF16, m);
    if (ok != GPTQ_OK) return ok;
  }
  if (tokens == 0 || m == 0) return GPTQ_OK;
  if (!X || !xs || ldx < n || ldx % 16 != 0 || (reinterpret_cast<uintptr_t>(X) & 15) != 0 ||
      ldxs < tokens || !scales || ldc < m || lds < tokens)
    return GPTQ_ERR_INVALID_ARG;
  if (ldx > kFp8MaxStride) return GPTQ_ERR_UNSUPPORTED;
  const gptq_status w = check_ws(ws, ws_bytes, fp8_gated_ws_bytes(tokens, m, n));
  if (w != GPTQ_OK) return w;
  // in one kernel, workgroups read X while others write codes
  if ((reinterpret_cast<uintptr_t>(ws) & 15) != 0 || codes == X) return GPTQ_ERR_INVALID_ARG;
  Fp8GemmArgs g{X,    ldx,     tokens, n,       xs, ldxs, Wg,      ldwg, m, gscales,
                ldgs, nullptr, GPTQ_BF16, 0, nullptr, 0, ws};
  return hip_status(launch_fp8_gated(g, Wu, ldwu, uscales, ldus, codes, ldc, scales, lds, stream));
}

gptq_status kv_cache_write_workspace_size(int64_t tokens, const gptq_kv_cache* cache,
                                          size_t* bytes) {
  if (!bytes || tokens < 0 || bad_dim(tokens)) return GPTQ_ERR_INVALID_ARG;
  const gptq_status ok = kv_cache_ok(cache, tokens);
  if (ok != GPTQ_OK) return ok;
  *bytes = kv_write_ws_bytes(tokens, cache->pages * cache->page_size);
  return GPTQ_OK;
}

gptq_status kv_cache_write(const void* K, int64_t k_token_stride, int64_t k_head_stride,
                           const void* V, int64_t v_token_stride, int64_t v_head_stride,
                           gptq_dtype dt, int64_t tokens, const int64_t* slots,
                           const gptq_kv_cache* kc, const gptq_kv_cache* vc, int32_t* info,
                           void* ws, size_t ws_bytes, hipStream_t stream) {
  const gptq_status ok = kv_call_ok(K, V, dt, tokens, slots, kc, vc);
  if (ok != GPTQ_OK || tokens == 0) return ok;
  const gptq_kv_cache* c = kc ? kc : vc;
  const gptq_status w = check_ws(ws, ws_bytes, kv_write_ws_bytes(tokens, c->pages * c->page_size));
  if (w != GPTQ_OK) return w;
  // (one cache for both: keys and values would race for its slots)
  if ((reinterpret_cast<uintptr_t>(ws) & 3) != 0 ||
      (kc && vc && (kc->codes == vc->codes || kc->scales == vc->scales ||
                    (kc->zeros && kc->zeros == vc->zeros))))
    return GPTQ_ERR_INVALID_ARG;
  const KvRows k{const_cast<void*>(K), k_token_stride, k_head_stride};
  const KvRows v{const_cast<void*>(V), v_token_stride, v_head_stride};
  return hip_status(launch_kv_write(k, v, dt, tokens, slots, kc, vc, info, ws, stream));
}

gptq_status kv_cache_read(const gptq_kv_cache* kc, const gptq_kv_cache* vc, const int64_t* slots,
                          int64_t tokens, void* K, int64_t k_token_stride, int64_t k_head_stride,
                          void* V, int64_t v_token_stride, int64_t v_head_stride, gptq_dtype dt,
                          int32_t* info, hipStream_t stream) {
  const gptq_status ok = kv_call_ok(K, V, dt, tokens, slots, kc, vc);
  if (ok != GPTQ_OK || tokens == 0) return ok;
  // rows that are written share no place
  if ((kc && ((tokens > 1 && k_token_stride == 0) || (kc->heads > 1 && k_head_stride == 0))) ||
      (vc && ((tokens > 1 && v_token_stride == 0) || (vc->heads > 1 && v_head_stride == 0))) ||
      (kc && vc && K == V))
    return GPTQ_ERR_INVALID_ARG;
  const KvRows k{K, k_token_stride, k_head_stride}, v{V, v_token_stride, v_head_stride};
  return hip_status(launch_kv_read(kc, vc, slots, tokens, k, v, dt, info, stream));
}

gptq_status token_logprobs_workspace_size(int64_t tokens, int64_t vocab, int32_t top,
                                          size_t* bytes) {
  if (!bytes || tokens < 0 || bad_dim(tokens) || vocab <= 0 || bad_dim(vocab) || top < 0 ||
      top > 32 || top > vocab)
    return GPTQ_ERR_INVALID_ARG;
  *bytes = tokens == 0 ? 0 : logprobs_ws_bytes(tokens, vocab, top);
  return GPTQ_OK;
}

gptq_status token_logprobs(const void* logits, gptq_dtype dt, int64_t tokens, int64_t vocab,
                           int64_t ldl, const int64_t* ids, float* logprob, float* entropy,
                           int32_t top, int32_t* top_ids, float* top_logprobs, void* ws,
                           size_t ws_bytes, hipStream_t stream) {
  if (tokens < 0 || bad_dim(tokens) || vocab <= 0 || bad_dim(vocab) || !valid_dtype(dt) ||
      top < 0 || top > 32 || top > vocab)
    return GPTQ_ERR_INVALID_ARG;
  if (tokens == 0) return GPTQ_OK;
  if (!logits || ldl < vocab || (ids != nullptr) != (logprob != nullptr) ||
      (top > 0 && (!top_ids || !top_logprobs)))
    return GPTQ_ERR_INVALID_ARG;
  const gptq_status w = check_ws(ws, ws_bytes, logprobs_ws_bytes(tokens, vocab, top));
  if (w != GPTQ_OK) return w;
  if ((reinterpret_cast<uintptr_t>(ws) & 15) != 0) return GPTQ_ERR_INVALID_ARG;
  return hip_status(launch_logprobs(logits, dt, tokens, vocab, ldl, ids, logprob, entropy, top,
                                    top_ids, top_logprobs, ws, stream));
}

}  // extern "C"

// Argument checks and launch of gptq_quantize_layer, shared with its
// no-allocation variant (which passes its static scratch as the workspace).
gptq_status gptq::quantize_layer_checked(const void* W, gptq_dtype wdt, int64_t m, int64_t n, int64_t ldw,
                                const float* U, int64_t ldu, const int32_t* perm,
                                const uint8_t* dead, const gptq_config* cfg, uint8_t* codes,
                                float* scales, float* zeros, int32_t* g_idx, float* row_err,
                                int32_t* info, void* ws, size_t ws_bytes, hipStream_t stream) {
  if (!cfg || bad_dim(m) || bad_dim(n) || !valid_dtype(wdt)) return GPTQ_ERR_INVALID_ARG;
  if (cfg->bits < 2 || cfg->bits > 8 || cfg->block_size <= 0 || cfg->group_size == 0 ||
      cfg->group_size < -1 ||
      (cfg->group_size > 0 && cfg->block_size % cfg->group_size != 0 &&
       cfg->group_size % cfg->block_size != 0) ||
      (cfg->desc_act != 0 && cfg->desc_act != 1) || (cfg->sym != 0 && cfg->sym != 1) ||
      (cfg->static_groups != 0 && cfg->static_groups != 1))
    return GPTQ_ERR_INVALID_ARG;
  if (cfg->block_size != 128 || !quant_group_ok(cfg->group_size)) return GPTQ_ERR_UNSUPPORTED;
  if (m == 0 || n == 0) return GPTQ_OK;
  if (!W || !U || !codes || !scales || !zeros || ldw < n || ldu < n) return GPTQ_ERR_INVALID_ARG;
  if (cfg->desc_act && !perm) return GPTQ_ERR_INVALID_ARG;
  const gptq_status w = check_ws(ws, ws_bytes, quantize_ws_bytes(m, n, cfg->desc_act));
  if (w != GPTQ_OK) return w;
  QuantArgs a;
  a.W = W;
  a.wdt = wdt;
  a.m = m;
  a.n = n;
  a.ldw = ldw;
  a.U = U;
  a.ldu = ldu;
  a.perm = perm;
  a.dead = dead;
  a.bits = cfg->bits;
  a.group_size = cfg->group_size;
  a.block_size = cfg->block_size;
  a.desc_act = cfg->desc_act;
  a.sym = cfg->sym;
  a.static_groups = cfg->group_size > 0 ? cfg->static_groups : 0;
  a.codes = codes;
  a.scales = scales;
  a.zeros = zeros;
  a.g_idx = g_idx;
  a.row_err = row_err;
  a.info = info;
  a.ws = ws;
  return hip_status(launch_quantize(a, stream));
}
