// Appending tokens to the paged key/value cache with the rotary rotation applied on the way, and
// reading tokens back.
//
// A token at position p has the last 2J dims of each key head (and query head) rotated pairwise,
//   (u, w) -> (u cos a - w sin a, w cos a + u sin a),   a = p * inv_freq[j], j < J,
// pairs (2j, 2j + 1) of the rotated part, or (j, j + J) in the half-split form.  The angle, its
// sine and cosine and the rotation are float64: p * inv_freq is then exact (31 + 24 bits), where
// float32 would be off by radians at far positions, and the result is rounded to bf16 as the
// exact one is but for one case in 2^40.  It is far from being the bound (one sine and cosine per
// token and pair, shared by the heads; four float64 operations per pair and head).
//
// 4-bit rows: 16 consecutive values of a head share an e4m3 scale s = max|y| / 6 (rounded to
// nearest, saturated at 448), y = x / (the tensor's scale); a value is the e2m1 code of y / s
// (rounded to nearest even, saturated at 6).  Keys are taken as bf16 holds them, so a 4-bit cache
// holds the quantised rows of the bf16 cache.  Every operation is one correctly rounded float32
// operation, so codes and scales are reproducible to the bit.  4 bits hold no infinity or NaN: a
// group with one gets a NaN scale and reads back as NaN.
//
// Memory-bound: a thread takes a group of 16 values (32 bytes in, 8 + 1 out, or 32), so a group's
// maximum needs no exchange; a half-split thread takes both groups of its pairs.
#include <float.h>

#include "cache.cuh"
#include "kernels.h"

namespace dsa {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = 96;    // J: half of the largest head dim
constexpr int kMaxTokens = 8;    // tokens per CTA

struct AppendArgs {
  CacheView c;
  const __nv_bfloat16* q;  // [B,S,H,DQK] or NULL
  const __nv_bfloat16* k;  // [B,S,HKV,DQK]
  const __nv_bfloat16* v;  // [B,S,HKV,DV]
  const int32_t* pos;      // [B,S]
  const float* inv_freq;   // [J]
  __nv_bfloat16* q_out;
  __nv_bfloat16* k_out;    // or NULL
  int S, H, mode, J, per_cta;
  long long tokens;
};

struct Group {
  uint4 w[2];  // 16 bf16
};
__device__ __forceinline__ Group load_group(const __nv_bfloat16* p) {
  Group x;
  x.w[0] = *reinterpret_cast<const uint4*>(p);
  x.w[1] = *reinterpret_cast<const uint4*>(p + 8);
  return x;
}
__device__ __forceinline__ void store_group(void* p, const Group& x) {
  reinterpret_cast<uint4*>(p)[0] = x.w[0];
  reinterpret_cast<uint4*>(p)[1] = x.w[1];
}
__device__ __forceinline__ uint32_t word(const Group& x, int i) {
  return (&x.w[i >> 2].x)[i & 3];
}
__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack_bf16(double a, double b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(__double2float_rn(a), __double2float_rn(b));
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Pairs (2i, 2i + 1) of the group, cs[i] = (cos, sin).
__device__ __forceinline__ void rotate_interleaved(Group& x, const double2* cs) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    uint32_t& w = (&x.w[i >> 2].x)[i & 3];
    const double u = lo_f(w), t = hi_f(w);
    w = pack_bf16(u * cs[i].x - t * cs[i].y, t * cs[i].x + u * cs[i].y);
  }
}
// Pairs (x[i], y[i]), cs[i] = (cos, sin).
__device__ __forceinline__ void rotate_halves(Group& x, Group& y, const double2* cs) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    uint32_t &a = (&x.w[i >> 2].x)[i & 3], &b = (&y.w[i >> 2].x)[i & 3];
    const double u0 = lo_f(a), u1 = hi_f(a), t0 = lo_f(b), t1 = hi_f(b);
    const double2 c0 = cs[2 * i], c1 = cs[2 * i + 1];
    a = pack_bf16(u0 * c0.x - t0 * c0.y, u1 * c1.x - t1 * c1.y);
    b = pack_bf16(t0 * c0.x + u0 * c0.y, t1 * c1.x + u1 * c1.y);
  }
}

// The codes (8 bytes) and the scale of 16 values x / tensor_scale.
__device__ __forceinline__ void encode_group(const Group& x, float tensor_scale, uint2* codes,
                                             uint8_t* scale) {
  float y[16];
  float top = 0.f;
  bool finite = true;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    y[2 * i] = __fdiv_rn(lo_f(word(x, i)), tensor_scale);
    y[2 * i + 1] = __fdiv_rn(hi_f(word(x, i)), tensor_scale);
    top = fmaxf(top, fmaxf(fabsf(y[2 * i]), fabsf(y[2 * i + 1])));
    finite = finite && fabsf(y[2 * i]) <= FLT_MAX && fabsf(y[2 * i + 1]) <= FLT_MAX;
  }
  if (!finite) {
    *codes = make_uint2(0u, 0u);
    *scale = 0x7f;
    return;
  }
  uint32_t s8;
  asm("{\n\t.reg .b16 t;\n\tcvt.rn.satfinite.e4m3x2.f32 t, %1, %2;\n\tcvt.u32.u16 %0, t;\n\t}"
      : "=r"(s8)
      : "f"(0.f), "f"(__fdiv_rn(top, 6.0f)));
  const uint32_t sh = e4m3x2_to_f16(s8);
  float s;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.f32.f16 %0, l;\n\t}" : "=f"(s) : "r"(sh));
  uint32_t w[2] = {0u, 0u};
  if (s > 0.f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t b;
      asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n\tcvt.u32.u8 %0, t;\n\t}"
          : "=r"(b)
          : "f"(__fdiv_rn(y[2 * i + 1], s)), "f"(__fdiv_rn(y[2 * i], s)));
      w[i >> 2] |= b << (8 * (i & 3));
    }
  }
  *codes = make_uint2(w[0], w[1]);
  *scale = (uint8_t)s8;
}

// One group into a cache row: `code_off` and `scale_off` are the head arrays' byte offsets in the
// row (bf16: code_off alone), `at` the first value's index in that array.
template <int FMT>
__device__ __forceinline__ void put_group(const CacheView& c, uint8_t* row, int code_off,
                                          int scale_off, int at, const Group& x,
                                          float tensor_scale) {
  if (FMT == 0) {
    store_group(row + code_off + 2 * at, x);
  } else {
    uint2 codes;
    uint8_t s;
    encode_group(x, tensor_scale, &codes, &s);
    *reinterpret_cast<uint2*>(row + code_off + at / 2) = codes;
    row[scale_off + at / 16] = s;
  }
}

template <int FMT>
__global__ void __launch_bounds__(kThreads) cache_append_kernel(const AppendArgs a) {
  extern __shared__ double2 cs_all[];  // [token][J]
  const CacheView& c = a.c;
  const long long tok0 = (long long)blockIdx.x * a.per_cta;
  const int nt = (int)min((long long)a.per_cta, a.tokens - tok0);
  for (int i = threadIdx.x; i < nt * a.J; i += kThreads) {
    const int p = __ldg(a.pos + tok0 + i / a.J);
    double sn = 0.0, cn = 1.0;
    if (p >= 0) sincos((double)p * (double)__ldg(a.inv_freq + i % a.J), &sn, &cn);
    cs_all[i] = make_double2(cn, sn);
  }
  __syncthreads();
  const int rot0 = c.DQK - 2 * a.J;  // the first rotated dim
  const bool halves = a.mode == 2;
  // threads' units of a head: groups of 16, in the half-split form two groups for the pairs
  const int ud = halves ? rot0 / 16 + a.J / 16 : c.DQK / 16;
  const int uq = a.q ? a.H * ud : 0, uk = c.HKV * ud, uv = c.HKV * (c.DV / 16);
  const int per = uq + uk + uv;
  const Group zero = {{make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)}};
  for (int i = threadIdx.x; i < nt * per; i += kThreads) {
    const int ti = i / per;
    int u = i - ti * per;
    const long long tok = tok0 + ti;
    const int p = __ldg(a.pos + tok);
    const int b = (int)(tok / a.S);
    const long long r = u < uq ? -1 : cache_row(c, c.table + (size_t)b * c.max_pages, p);
    uint8_t* row = r >= 0 ? c.pages + r * c.row_bytes : nullptr;
    if (u >= uq + uk) {  // a group of V
      u -= uq + uk;
      if (row)
        put_group<FMT>(c, row, cache_v_off(FMT, c.HKV, c.DQK), cache_vs_off(c.HKV, c.DQK, c.DV),
                       u * 16, load_group(a.v + tok * c.HKV * c.DV + u * 16), c.v_scale);
      continue;
    }
    const bool is_q = u < uq;
    if (!is_q) u -= uq;
    const int h = u / ud, e = u - h * ud;
    const size_t base = ((size_t)tok * (is_q ? a.H : c.HKV) + h) * c.DQK;
    const __nv_bfloat16* src = (is_q ? a.q : a.k) + base;
    __nv_bfloat16* dst = is_q ? a.q_out + base : (a.k_out ? a.k_out + base : nullptr);
    const double2* cs = cs_all + ti * a.J;
    const int d = e * 16;  // this unit's first dim, and its partner's
    Group x = load_group(src + d), y;
    const bool pair = halves && d >= rot0;
    if (pair) {
      y = load_group(src + d + a.J);
      rotate_halves(x, y, cs + (d - rot0));
    } else if (a.mode == 1 && d >= rot0) {
      rotate_interleaved(x, cs + (d - rot0) / 2);
    }
    if (dst) {  // padded tokens (p < 0) give zeros
      store_group(dst + d, p >= 0 ? x : zero);
      if (pair) store_group(dst + d + a.J, p >= 0 ? y : zero);
    }
    if (row) {
      const int so = cache_ks_off(c.HKV, c.DQK, c.DV);
      put_group<FMT>(c, row, 0, so, h * c.DQK + d, x, c.k_scale);
      if (pair) put_group<FMT>(c, row, 0, so, h * c.DQK + d + a.J, y, c.k_scale);
    }
  }
}

// 16 values of a cache row as bf16: exact for bf16 rows, code * scale * tensor scale (the first
// product exact, the second float32) rounded to bf16 for 4-bit rows.
template <int FMT>
__device__ __forceinline__ Group get_group(const uint8_t* row, int code_off, int scale_off, int at,
                                           float tensor_scale) {
  Group x;
  if (FMT == 0) return load_group(reinterpret_cast<const __nv_bfloat16*>(row + code_off) + at);
  const uint2 codes = *reinterpret_cast<const uint2*>(row + code_off + at / 2);
  const uint32_t s = e4m3x2_to_f16((uint32_t)row[scale_off + at / 16] * 0x0101u);
#pragma unroll
  for (int hf = 0; hf < 2; ++hf) {
    uint32_t f[4];
    e2m1x8_to_f16(hf ? codes.y : codes.x, f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t m = mul_f16x2(f[i], s);
      float a, b;
      asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\t"
          "cvt.f32.f16 %1, h;\n\t}"
          : "=f"(a), "=f"(b)
          : "r"(m));
      const __nv_bfloat162 h2 = __floats2bfloat162_rn(a * tensor_scale, b * tensor_scale);
      (&x.w[hf].x)[i] = *reinterpret_cast<const uint32_t*>(&h2);
    }
  }
  return x;
}

// Tokens read back: k [B,S,HKV,DQK], v [B,S,HKV,DV]; zeros where the cache has no row.
template <int FMT>
__global__ void __launch_bounds__(kThreads)
    cache_read_kernel(const CacheView c, const int32_t* __restrict__ pos, int S, long long tokens,
                      __nv_bfloat16* k, __nv_bfloat16* v) {
  const int uk = c.HKV * (c.DQK / 16), uv = c.HKV * (c.DV / 16), per = uk + uv;
  const long long total = tokens * per;
  const Group zero = {{make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)}};
  for (long long i = (long long)blockIdx.x * kThreads + threadIdx.x; i < total;
       i += (long long)gridDim.x * kThreads) {
    const long long tok = i / per;
    const int u = (int)(i - tok * per);
    const int b = (int)(tok / S);
    const long long r = cache_row(c, c.table + (size_t)b * c.max_pages, __ldg(pos + tok));
    const uint8_t* row = c.pages + (r >= 0 ? r : 0) * c.row_bytes;
    if (u < uk) {
      store_group(k + (size_t)tok * uk * 16 + u * 16,
                  r < 0 ? zero
                        : get_group<FMT>(row, 0, cache_ks_off(c.HKV, c.DQK, c.DV), u * 16,
                                         c.k_scale));
    } else {
      const int w = u - uk;
      store_group(v + (size_t)tok * uv * 16 + w * 16,
                  r < 0 ? zero
                        : get_group<FMT>(row, cache_v_off(FMT, c.HKV, c.DQK),
                                         cache_vs_off(c.HKV, c.DQK, c.DV), w * 16, c.v_scale));
    }
  }
}

}  // namespace

cudaError_t launch_cache_append(const CacheAppendProblem& p, cudaStream_t st) {
  AppendArgs a{};
  a.c = p.cache;
  a.q = static_cast<const __nv_bfloat16*>(p.q);
  a.k = static_cast<const __nv_bfloat16*>(p.k);
  a.v = static_cast<const __nv_bfloat16*>(p.v);
  a.pos = p.pos; a.inv_freq = p.inv_freq;
  a.q_out = static_cast<__nv_bfloat16*>(p.q_out);
  a.k_out = static_cast<__nv_bfloat16*>(p.k_out);
  a.S = p.S; a.H = p.H; a.mode = p.rope_mode;
  a.J = p.rope_mode == 0 ? 0 : p.rope_dim / 2;
  a.tokens = (long long)p.B * p.S;
  // enough CTAs to fill the GPU first, then several tokens per CTA (their sines in one go)
  long long per = a.tokens / (148 * 8);
  a.per_cta = (int)(per < 1 ? 1 : (per > kMaxTokens ? kMaxTokens : per));
  const unsigned grid = (unsigned)((a.tokens + a.per_cta - 1) / a.per_cta);
  const size_t smem = (size_t)a.per_cta * a.J * sizeof(double2);
  if (a.J > kMaxPairs) return cudaErrorNotSupported;
  if (p.cache.format == 0)
    cache_append_kernel<0><<<grid, kThreads, smem, st>>>(a);
  else
    cache_append_kernel<1><<<grid, kThreads, smem, st>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_cache_read(const CacheView& c, const int32_t* pos, int B, int S, void* k,
                              void* v, cudaStream_t st) {
  const long long tokens = (long long)B * S;
  const long long total = tokens * (c.HKV * ((c.DQK + c.DV) / 16));
  const long long want = (total + kThreads - 1) / kThreads;
  const unsigned grid = (unsigned)(want < 148 * 16 ? want : 148 * 16);
  if (c.format == 0)
    cache_read_kernel<0><<<grid, kThreads, 0, st>>>(c, pos, S, tokens,
                                                    static_cast<__nv_bfloat16*>(k),
                                                    static_cast<__nv_bfloat16*>(v));
  else
    cache_read_kernel<1><<<grid, kThreads, 0, st>>>(c, pos, S, tokens,
                                                    static_cast<__nv_bfloat16*>(k),
                                                    static_cast<__nv_bfloat16*>(v));
  return cudaGetLastError();
}

}  // namespace dsa
