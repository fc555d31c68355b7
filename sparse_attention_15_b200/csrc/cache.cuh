// The paged key/value cache: its row layout and the lookups shared by the cache kernels.
#pragma once

#include <stdint.h>

#include "common.cuh"

namespace dsa {

// Device view of a cache (dsa_cache in include/dsa.h): page `table[b][t / page_size]` holds token
// t of sequence b in its row t % page_size.
struct CacheView {
  uint8_t* pages;
  const int32_t* table;  // [B, max_pages]
  int format;            // 0 bf16, 1 e2m1
  int n_pages, page_size, max_pages;
  int HKV, DQK, DV;
  float k_scale, v_scale;
  long long row_bytes;
  int cap;               // max_pages * page_size: keys a sequence can hold, at most 2^30
  uint32_t page_mul;     // t / page_size = (t * page_mul) >> 32 >> page_shift for t < 2^31
  int page_shift;        // (page_size 1: page_mul 0)
};

// The divisor's multiplier: ceil(2^(31 + L) / d) with L = ceil(log2 d), which fits 32 bits and
// rounds every quotient of a 31-bit number down correctly.
inline void set_page_divisor(CacheView* c) {
  int L = 0;
  while ((1LL << L) < c->page_size) ++L;
  c->page_shift = L > 0 ? L - 1 : 0;
  c->page_mul =
      L > 0 ? (uint32_t)(((1ULL << (31 + L)) + c->page_size - 1) / (unsigned long long)c->page_size)
            : 0;
}

// Byte offsets inside a row.  bf16: [K | V]; e2m1: [K codes | V codes | K scales | V scales],
// two codes to a byte (even element low), one e4m3 scale for 16 elements of a head.
__host__ __device__ inline long long cache_row_bytes(int format, int HKV, int DQK, int DV) {
  const long long n = (long long)HKV * (DQK + DV);
  return format == 0 ? 2 * n : (n / 2 + n / 16 + 15) / 16 * 16;
}
__host__ __device__ inline int cache_v_off(int format, int HKV, int DQK) {
  return format == 0 ? 2 * HKV * DQK : HKV * DQK / 2;
}
__host__ __device__ inline int cache_ks_off(int HKV, int DQK, int DV) {
  return HKV * (DQK + DV) / 2;
}
__host__ __device__ inline int cache_vs_off(int HKV, int DQK, int DV) {
  return HKV * (DQK + DV) / 2 + HKV * DQK / 16;
}

// The physical row (page * page_size + slot, below 2^31) of token t of a sequence with this table
// row, or -1 if the cache has none: t out of range, or a table entry that names no page.
__device__ __forceinline__ int cache_row(const CacheView& c, const int32_t* table_row, int t) {
  if ((uint32_t)t >= (uint32_t)c.cap) return -1;
  const int p = c.page_mul ? (int)(__umulhi((uint32_t)t, c.page_mul) >> c.page_shift) : t;
  const int page = __ldg(table_row + p);
  if ((uint32_t)page >= (uint32_t)c.n_pages) return -1;
  return page * c.page_size + (t - p * c.page_size);
}

// Four e2m1 pairs (the bytes of w, low element first) as f16 pairs; exact.
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&r)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
}
// Two e4m3 values (low byte first) as an f16 pair; exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16(uint32_t v) {
  uint32_t r;
  asm("{\n\t.reg .b16 t, u;\n\tmov.b32 {t, u}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}"
      : "=r"(r)
      : "r"(v));
  return r;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

}  // namespace dsa
