// Entry points of the paged key/value cache: argument checks, then the kernels of
// cache_append.cu and cache_attn.cu.  The contract is in include/dsa.h, section 5.
#include <math.h>
#include <stdarg.h>
#include <stdio.h>

#include "cache.cuh"
#include "checks.h"
#include "kernels.h"

namespace {

dsa_status fail(dsa_status st, const char* fmt, ...) {
  char buf[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  dsa::set_last_error(buf);
  return st;
}

#define REQUIRE(cond, st, ...)                 \
  do {                                         \
    if (!(cond)) return fail(st, __VA_ARGS__); \
  } while (0)

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

dsa_status cuda_status(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return DSA_OK;
  if (e == cudaErrorNotSupported)
    return fail(DSA_ERR_UNSUPPORTED, "%s: no kernel for this shape", what);
  return fail(DSA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

bool dims_ok(int DQK, int DV) {
  return (DQK == 64 || DQK == 128 || DQK == 192) && (DV == 64 || DV == 128);
}

// What the workspace sizes go by too (no pointers).
dsa_status check_shape(const dsa_cache* c, int B, int S) {
  REQUIRE(c != nullptr, DSA_ERR_INVALID_ARG, "null cache");
  REQUIRE(c->format == DSA_CACHE_BF16 || c->format == DSA_CACHE_E2M1, DSA_ERR_INVALID_ARG,
          "unknown cache format %d", (int)c->format);
  REQUIRE(B > 0 && S > 0 && c->n_pages > 0 && c->page_size > 0 && c->max_pages > 0 && c->HKV > 0 &&
              c->DQK > 0 && c->DV > 0,
          DSA_ERR_INVALID_ARG, "sizes must be positive");
  REQUIRE(dims_ok(c->DQK, c->DV), DSA_ERR_UNSUPPORTED,
          "the cache needs DQK in {64,128,192} and DV in {64,128} (DQK=%d DV=%d)", c->DQK, c->DV);
  REQUIRE(c->HKV <= 64, DSA_ERR_UNSUPPORTED, "HKV=%d > 64", c->HKV);
  REQUIRE((long long)c->max_pages * c->page_size <= (1LL << 30), DSA_ERR_UNSUPPORTED,
          "max_pages * page_size must be at most 2^30");
  REQUIRE((long long)c->n_pages * c->page_size < (1LL << 31), DSA_ERR_UNSUPPORTED,
          "n_pages * page_size must be below 2^31");
  REQUIRE((long long)B * S <= (1LL << 24), DSA_ERR_UNSUPPORTED, "B*S=%lld > 2^24",
          (long long)B * S);
  return DSA_OK;
}

dsa_status check_cache(const dsa_cache* c, const int32_t* pos, int B, int S) {
  const dsa_status st = check_shape(c, B, S);
  if (st != DSA_OK) return st;
  REQUIRE(c->pages && c->table && pos, DSA_ERR_INVALID_ARG, "null pointer argument");
  REQUIRE(isfinite(c->k_scale) && c->k_scale > 0.f && isfinite(c->v_scale) && c->v_scale > 0.f,
          DSA_ERR_INVALID_ARG, "k_scale and v_scale must be finite and > 0");
  REQUIRE(c->format == DSA_CACHE_E2M1 || (c->k_scale == 1.f && c->v_scale == 1.f),
          DSA_ERR_INVALID_ARG, "k_scale and v_scale belong to the 4-bit format");
  REQUIRE(aligned16(c->pages), DSA_ERR_UNSUPPORTED, "pages must be 16-byte aligned");
  REQUIRE(aligned4(c->table) && aligned4(pos), DSA_ERR_UNSUPPORTED,
          "table and pos must be 4-byte aligned");
  return DSA_OK;
}

dsa::CacheView view(const dsa_cache* c) {
  dsa::CacheView v{};
  v.pages = static_cast<uint8_t*>(c->pages);
  v.table = c->table;
  v.format = (int)c->format;
  v.n_pages = c->n_pages; v.page_size = c->page_size; v.max_pages = c->max_pages;
  v.HKV = c->HKV; v.DQK = c->DQK; v.DV = c->DV;
  v.k_scale = c->k_scale; v.v_scale = c->v_scale;
  v.row_bytes = dsa::cache_row_bytes(v.format, v.HKV, v.DQK, v.DV);
  v.cap = c->max_pages * c->page_size;
  dsa::set_page_divisor(&v);
  return v;
}

dsa_status check_heads(const dsa_cache* c, int H) {
  REQUIRE(H > 0 && H % c->HKV == 0, DSA_ERR_INVALID_ARG, "H=%d not a multiple of HKV=%d", H,
          c->HKV);
  REQUIRE(H <= 64, DSA_ERR_UNSUPPORTED, "H=%d > 64", H);
  return DSA_OK;
}

dsa_status check_window(int window, int n_first) {
  REQUIRE(window >= 0 && n_first >= 0, DSA_ERR_INVALID_ARG,
          "window and n_first must not be negative");
  REQUIRE(window > 0 || n_first == 0, DSA_ERR_INVALID_ARG,
          "n_first goes with a window (window 0 sees every key)");
  return DSA_OK;
}

// Both attention forms: idx with K > 0, or the window form with idx == NULL.
dsa_status run_attn(const char* what, const dsa_cache* c, const void* q, const int32_t* pos,
                    const int32_t* idx, int K, int window, int n_first, const void* gate,
                    dsa_gate_mode gm, float sm_scale, int B, int S, int H, void* out, void* ws,
                    size_t ws_bytes, cudaStream_t st) {
  dsa_status e = check_cache(c, pos, B, S);
  if (e != DSA_OK) return e;
  if ((e = check_heads(c, H)) != DSA_OK) return e;
  REQUIRE(q && out, DSA_ERR_INVALID_ARG, "null pointer argument");
  REQUIRE(gm >= DSA_GATE_OFF && gm <= DSA_GATE_SILU, DSA_ERR_INVALID_ARG,
          "unknown gate mode %d (only sigmoid and silu exist)", (int)gm);
  REQUIRE((gm == DSA_GATE_OFF) == (gate == nullptr), DSA_ERR_INVALID_ARG,
          "gate pointer must be given exactly when the gate is on");
  REQUIRE(!isnan(sm_scale) && !isinf(sm_scale), DSA_ERR_INVALID_ARG, "sm_scale not finite");
  REQUIRE(aligned16(q) && aligned16(out) && aligned16(gate), DSA_ERR_UNSUPPORTED,
          "pointers must be 16-byte aligned");
  REQUIRE(dsa::cache_attn_supported((int)c->format, H, c->HKV, c->DQK, c->DV), DSA_ERR_UNSUPPORTED,
          "no kernel for H=%d HKV=%d", H, c->HKV);
  const dsa::CacheView v = view(c);
  dsa::CacheAttnProblem p{v, q, pos, idx, K, window, n_first, gate, (int)gm,
                          sm_scale > 0.f ? sm_scale : 1.0f / sqrtf((float)c->DQK), B, S, H, out};
  const size_t need = dsa::cache_attn_workspace_bytes(p);
  REQUIRE(need == 0 || (ws != nullptr && ws_bytes >= need), DSA_ERR_INVALID_ARG,
          "workspace too small: %zu bytes given, %zu needed", ws ? ws_bytes : (size_t)0, need);
  REQUIRE(need == 0 || aligned16(ws), DSA_ERR_UNSUPPORTED, "workspace must be 16-byte aligned");
  return cuda_status(dsa::launch_cache_attn(p, ws, ws_bytes, st), what);
}

size_t attn_workspace(const dsa_cache* c, int B, int S, int H, const int32_t* idx, int K,
                      int window, int n_first) {
  if (check_shape(c, B, S) != DSA_OK || check_heads(c, H) != DSA_OK) return 0;
  const dsa::CacheView v = view(c);
  const dsa::CacheAttnProblem p{v, nullptr, nullptr, idx, K, window, n_first, nullptr, 0, 1.f,
                                B, S, H, nullptr};
  return dsa::cache_attn_workspace_bytes(p);
}

}  // namespace

extern "C" {

size_t dsa_cache_row_bytes(dsa_cache_format format, int HKV, int DQK, int DV) {
  if ((format != DSA_CACHE_BF16 && format != DSA_CACHE_E2M1) || HKV <= 0 || HKV > 64 ||
      !dims_ok(DQK, DV))
    return 0;
  return (size_t)dsa::cache_row_bytes((int)format, HKV, DQK, DV);
}

dsa_status dsa_cache_append(const dsa_cache* cache, const int32_t* pos, const void* k,
                            const void* v, dsa_rope_mode rope_mode, int rope_dim,
                            const float* inv_freq, int B, int S, int H, const void* q, void* q_out,
                            void* k_out, dsa_stream_t stream) {
  dsa_status st = check_cache(cache, pos, B, S);
  if (st != DSA_OK) return st;
  REQUIRE(k && v, DSA_ERR_INVALID_ARG, "null pointer argument");
  REQUIRE(rope_mode >= DSA_ROPE_OFF && rope_mode <= DSA_ROPE_HALF, DSA_ERR_INVALID_ARG,
          "unknown rope mode %d", (int)rope_mode);
  if (rope_mode == DSA_ROPE_OFF) {
    REQUIRE(rope_dim == 0 && !inv_freq && !q && !q_out, DSA_ERR_INVALID_ARG,
            "rope_dim, inv_freq, q and q_out go with a rotation");
  } else {
    REQUIRE(rope_dim > 0 && inv_freq, DSA_ERR_INVALID_ARG,
            "a rotation needs rope_dim > 0 and inv_freq");
    REQUIRE(rope_dim % 32 == 0 && rope_dim <= cache->DQK, DSA_ERR_UNSUPPORTED,
            "rope_dim=%d must be a multiple of 32, at most DQK=%d", rope_dim, cache->DQK);
    REQUIRE(aligned4(inv_freq), DSA_ERR_UNSUPPORTED, "inv_freq must be 4-byte aligned");
    REQUIRE((q == nullptr) == (q_out == nullptr), DSA_ERR_INVALID_ARG,
            "q and q_out must be given together");
    if (q && (st = check_heads(cache, H)) != DSA_OK) return st;
  }
  REQUIRE(aligned16(k) && aligned16(v) && aligned16(q) && aligned16(q_out) && aligned16(k_out),
          DSA_ERR_UNSUPPORTED, "pointers must be 16-byte aligned");
  const dsa::CacheView c = view(cache);
  const dsa::CacheAppendProblem p{c, q, k, v, pos, (int)rope_mode, rope_dim, inv_freq, B, S, H,
                                  q_out, k_out};
  return cuda_status(dsa::launch_cache_append(p, (cudaStream_t)stream), "dsa_cache_append");
}

dsa_status dsa_cache_read(const dsa_cache* cache, const int32_t* pos, int B, int S, void* k,
                          void* v, dsa_stream_t stream) {
  const dsa_status st = check_cache(cache, pos, B, S);
  if (st != DSA_OK) return st;
  REQUIRE(k && v, DSA_ERR_INVALID_ARG, "null pointer argument");
  REQUIRE(aligned16(k) && aligned16(v), DSA_ERR_UNSUPPORTED, "pointers must be 16-byte aligned");
  return cuda_status(dsa::launch_cache_read(view(cache), pos, B, S, k, v, (cudaStream_t)stream),
                     "dsa_cache_read");
}

size_t dsa_cache_attn_workspace_bytes(const dsa_cache* cache, int B, int S, int H, int window,
                                      int n_first) {
  if (check_window(window, n_first) != DSA_OK) return 0;
  return attn_workspace(cache, B, S, H, nullptr, 0, window, n_first);
}

dsa_status dsa_cache_attn(const dsa_cache* cache, const void* q, const int32_t* pos, int window,
                          int n_first, const void* gate, dsa_gate_mode gate_mode, float sm_scale,
                          int B, int S, int H, void* out, void* ws, size_t ws_bytes,
                          dsa_stream_t stream) {
  const dsa_status st = check_window(window, n_first);
  if (st != DSA_OK) return st;
  return run_attn("dsa_cache_attn", cache, q, pos, nullptr, 0, window, n_first, gate, gate_mode,
                  sm_scale, B, S, H, out, ws, ws_bytes, (cudaStream_t)stream);
}

size_t dsa_cache_sparse_attn_workspace_bytes(const dsa_cache* cache, int B, int S, int H, int K) {
  if (K <= 0) return 0;
  static const int32_t some = 0;  // the selected form; not read
  return attn_workspace(cache, B, S, H, &some, K, 0, 0);
}

dsa_status dsa_cache_sparse_attn(const dsa_cache* cache, const void* q, const int32_t* pos,
                                 const int32_t* idx, int K, const void* gate,
                                 dsa_gate_mode gate_mode, float sm_scale, int B, int S, int H,
                                 void* out, void* ws, size_t ws_bytes, dsa_stream_t stream) {
  const dsa_status st = dsa::check_idx_args(idx, K);
  if (st != DSA_OK) return st;
  REQUIRE(K <= (1 << 30), DSA_ERR_UNSUPPORTED, "K=%d > 2^30", K);
  return run_attn("dsa_cache_sparse_attn", cache, q, pos, idx, K, 0, 0, gate, gate_mode, sm_scale,
                  B, S, H, out, ws, ws_bytes, (cudaStream_t)stream);
}

}  // extern "C"
