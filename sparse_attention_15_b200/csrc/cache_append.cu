// Appending tokens to the paged key/value cache with the rotary rotation applied on the way, and
// reading tokens back.
//
// A token at position p has the last 2J dims of each key head (and query head) rotated pairwise,
//   (u, w) -> (u cos a - w sin a, w cos a + u sin a),   a = p * inv_freq[j], j < J,
// pairs (2j, 2j + 1) of the rotated part, or (j, j + J) in the half-split form.  The angle and its
// sine and cosine are float64 -- p * inv_freq is then exact (31 + 24 bits), where float32 would be
// off by radians at far positions -- once per token and pair, for all heads.  The rotation gives
// what float64 rounded to float32 and then to bf16 gives, but for one result in 2^30 or so, in
// float32 arithmetic (float64 conversions would bound the kernel: 8 clocks a warp each): cos a =
// ch + cl with 16 bits in ch, so that u ch, of 8 + 16 bits, is exact, and the difference of the two
// exact products keeps its rounding error (a two-sum).
//
// 4-bit rows: 16 consecutive values of a head share an e4m3 scale s = max|y| / 6 (rounded to
// nearest, saturated at 448), y = x / (the tensor's scale); a value is the e2m1 code of y / s
// (rounded to nearest even, saturated at 6).  Keys are taken as bf16 holds them, so a 4-bit cache
// holds the quantised rows of the bf16 cache.  Every operation is one correctly rounded float32
// operation, so codes and scales are reproducible to the bit.  4 bits hold no infinity or NaN: a
// group with one among its x gets a NaN scale and reads back as NaN.  (A finite x whose y is past
// float32's range saturates like any other.)
//
// Memory-bound in bf16 (8192 tokens of 32 heads, 537 MB: 95 us, 5.7 TB/s; reading back, 335 MB: 56
// us, 6.0 TB/s).  In 4 bits (2 x 4001 tokens of 8 heads, 249 MB: 60 us, 4.1 TB/s; reading back, 52 MB:
// 12.5 us, 4.2 TB/s) latency and the encoding's instructions show, and with them the registers: at 64
// a thread the half-split kernels spill 150 bytes, the interleaved ones 24, and the encoding by
// division, a call of its own, keeps its group on the stack.  A thread takes a group of 16 values (32
// bytes in, 8 + 1 out, or 32), so a group's maximum needs no exchange; a half-split thread takes both
// groups of its pairs.
#include <math.h>

#include "cache.cuh"
#include "kernels.h"

namespace dsa {

namespace {

constexpr int kThreads = 256;    // of a CTA that reads
// Threads of a CTA that appends: a CTA starts with its sines, which the other CTAs of its SM cover,
// the better the more there are.  4-bit rows are smaller (2 x 4001 tokens of 8 heads, keys and
// values only: 22 us by 128 threads, 28 by 256, 36 by 512); of 8192 bf16 tokens with queries the
// rotated rows alone keep 256 busy (94 us; 128: 95, 512: 109).
__host__ __device__ constexpr int append_threads(int format) { return format == 1 ? 128 : 256; }
constexpr int kMaxTokens = 4;    // tokens per CTA

// x / d for 0 <= x < 2^31, by a multiplier as in CacheView.
struct Divisor {
  uint32_t d, mul;
  int shift;
  __device__ __forceinline__ int of(int x) const {
    return mul ? (int)(__umulhi((uint32_t)x, mul) >> shift) : x;
  }
};
Divisor divisor(int d) {
  CacheView v{};
  v.page_size = d;
  set_page_divisor(&v);
  return Divisor{(uint32_t)d, v.page_mul, v.page_shift};
}

// A tensor's scale, and its reciprocal where the scale is a power of two (else 0).
struct TensorScale {
  float scale, inv;
};

struct AppendArgs {
  CacheView c;
  const __nv_bfloat16* q;  // [B,S,H,DQK] or NULL
  const __nv_bfloat16* k;  // [B,S,HKV,DQK]
  const __nv_bfloat16* v;  // [B,S,HKV,DV]
  const int32_t* pos;      // [B,S]
  const float* inv_freq;   // [J]
  __nv_bfloat16* q_out;
  __nv_bfloat16* k_out;    // or NULL
  int S, H, J, per_cta;
  // units of a token (a thread takes one at a time): of q's and k's plain dims and rotated dims, and
  // of v; and of a head's
  Divisor q_plain, q_rot, k_plain, k_rot, uv, plain, rot;
  TensorScale k_scale, v_scale;
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
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// cos a and sin a as sums of two floats, the first of 16 bits.
struct Turn {
  float ch, cl, sh, sl;
};
__device__ __forceinline__ Turn turn_of(double c, double s) {
  Turn t;
  t.ch = __uint_as_float(__float_as_uint((float)c) & 0xffffff00u);
  t.sh = __uint_as_float(__float_as_uint((float)s) & 0xffffff00u);
  t.cl = (float)(c - (double)t.ch);
  t.sl = (float)(s - (double)t.sh);
  return t;
}
// A pair (u, v) turned, as float32 pairs: p = (u, v) ch and q = (-v, u) sh are exact; their sum d and
// its rounding error, then the small products.  (Past float32's range, and for infinities, the
// rounding error is NaN: d alone then.)
__device__ __forceinline__ unsigned long long mul2(unsigned long long a, unsigned long long b) {
  unsigned long long d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ void turn_pair(float& u, float& v, const Turn& t) {
  const unsigned long long x = pack2(u, v), y = pack2(-v, u);
  const unsigned long long p = mul2(x, pack2(t.ch, t.ch)), q = mul2(y, pack2(t.sh, t.sh));
  const unsigned long long d = add2(p, q), b = sub2(d, p);
  const unsigned long long e = add2(sub2(p, sub2(d, b)), sub2(q, b));
  const unsigned long long r =
      add2(d, add2(e, fma2(x, pack2(t.cl, t.cl), mul2(y, pack2(t.sl, t.sl)))));
  float d0, d1, r0, r1;
  unpack2(d, d0, d1);
  unpack2(r, r0, r1);
  u = r0 == r0 ? r0 : d0;
  v = r1 == r1 ? r1 : d1;
}
// Turns are kept with one empty place after each 8, so that the groups of a warp meet no bank twice.
__device__ __forceinline__ int turn_at(int j) { return j + (j >> 3); }

// Pairs (2i, 2i + 1) of the group; its first turn is number j of the token's.
__device__ __forceinline__ void rotate_interleaved(Group& x, const Turn* turns, int j) {
  const Turn* t = turns + turn_at(j);  // j is a multiple of 8
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    uint32_t& w = (&x.w[i >> 2].x)[i & 3];
    float u = lo_f(w), v = hi_f(w);
    turn_pair(u, v, t[i]);
    w = pack_bf16(u, v);
  }
}
// Pairs (x[i], y[i]); j as above.
__device__ __forceinline__ void rotate_halves(Group& x, Group& y, const Turn* turns, int j) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    uint32_t &a = (&x.w[i >> 2].x)[i & 3], &b = (&y.w[i >> 2].x)[i & 3];
    float u0 = lo_f(a), u1 = hi_f(a), v0 = lo_f(b), v1 = hi_f(b);
    const Turn* t = turns + turn_at(j + 8 * (i >> 2)) + 2 * (i & 3);
    turn_pair(u0, v0, t[0]);
    turn_pair(u1, v1, t[1]);
    a = pack_bf16(u0, u1);
    b = pack_bf16(v0, v1);
  }
}

// The codes (8 bytes) and the scale of 16 values x / tensor scale.
//
// With a scale that is a power of two the divisions are products.  x / 2^k is one either way; and a
// value y / s has 8 bits over 4, so it is a border of two codes (2 or 3 bits) exactly, or at least
// 2^-9 of itself away from it: y * fl(1/s) falls on the same side, and where y / s is a border, it
// is that border or the next float above (checked for each of the 8 significands of s), which
// clearing the last 4 bits takes back.
__device__ __forceinline__ uint32_t e4m3_of(float v, float* value) {  // v >= 0
  uint32_t s8;
  asm("{\n\t.reg .b16 t;\n\tcvt.rn.satfinite.e4m3x2.f32 t, %1, %2;\n\tcvt.u32.u16 %0, t;\n\t}"
      : "=r"(s8)
      : "f"(0.f), "f"(v));
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.f32.f16 %0, l;\n\t}"
      : "=f"(*value)
      : "r"(e4m3x2_to_f16(s8)));
  return s8;
}
__device__ __forceinline__ uint32_t e2m1x2_of(float lo, float hi) {
  uint32_t b;
  asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n\tcvt.u32.u8 %0, t;\n\t}"
      : "=r"(b)
      : "f"(hi), "f"(lo));
  return b;
}
struct Encoded {
  uint2 codes;
  uint32_t scale;
};
// Whether no value of the group is an infinity or NaN (an exponent field of ones).
__device__ __forceinline__ bool all_finite(const Group& x) {
  bool finite = true;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    finite = finite && (word(x, i) & 0x7f800000u) != 0x7f800000u &&
             (word(x, i) & 0x7f80u) != 0x7f80u;
  return finite;
}
// `inv` the reciprocal of a scale that is a power of two.
__device__ __forceinline__ Encoded encode_group(const Group& x, float inv) {
  float y[16], top = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    y[2 * i] = lo_f(word(x, i)) * inv;
    y[2 * i + 1] = hi_f(word(x, i)) * inv;
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) top = fmaxf(top, fabsf(y[i]));
  const bool finite = all_finite(x);
  float s;
  Encoded e;
  e.scale = e4m3_of(__fdiv_rn(top, 6.0f), &s);
  const float r = s > 0.f ? __frcp_rn(s) : 0.f;
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    w[i >> 2] |= e2m1x2_of(__uint_as_float(__float_as_uint(y[2 * i] * r) & 0xfffffff0u),
                           __uint_as_float(__float_as_uint(y[2 * i + 1] * r) & 0xfffffff0u))
                 << (8 * (i & 3));
  e.codes = s > 0.f && finite ? make_uint2(w[0], w[1]) : make_uint2(0u, 0u);
  if (!finite) e.scale = 0x7f;
  return e;
}
// Any scale: true divisions, out of the way (32 of them).
__device__ __noinline__ Encoded encode_group_by_division(const Group& x, float tensor_scale) {
  float top = 0.f;
  for (int i = 0; i < 8; ++i) {
    const float a = __fdiv_rn(lo_f(word(x, i)), tensor_scale);
    const float b = __fdiv_rn(hi_f(word(x, i)), tensor_scale);
    top = fmaxf(top, fmaxf(fabsf(a), fabsf(b)));
  }
  const bool finite = all_finite(x);
  float s;
  Encoded e;
  e.scale = e4m3_of(__fdiv_rn(top, 6.0f), &s);
  uint32_t w[2] = {0u, 0u};
  if (s > 0.f && finite)
    for (int i = 0; i < 8; ++i)
      w[i >> 2] |= e2m1x2_of(__fdiv_rn(__fdiv_rn(lo_f(word(x, i)), tensor_scale), s),
                             __fdiv_rn(__fdiv_rn(hi_f(word(x, i)), tensor_scale), s))
                   << (8 * (i & 3));
  e.codes = make_uint2(w[0], w[1]);
  if (!finite) e.scale = 0x7f;
  return e;
}

// One group into a cache row: `code_off` and `scale_off` are the head arrays' byte offsets in the
// row (bf16: code_off alone), `at` the first value's index in that array.
template <int FMT>
__device__ __forceinline__ void put_group(uint8_t* row, int code_off, int scale_off, int at,
                                          const Group& x, TensorScale tensor_scale) {
  if (FMT == 0) {
    store_group(row + code_off + 2 * at, x);
  } else {
    const Encoded e = tensor_scale.inv != 0.f ? encode_group(x, tensor_scale.inv)
                                              : encode_group_by_division(x, tensor_scale.scale);
    *reinterpret_cast<uint2*>(row + code_off + at / 2) = e.codes;
    row[scale_off + at / 16] = (uint8_t)e.scale;
  }
}

// Where the tokens of a CTA go: the row's address, or NULL.
__device__ __forceinline__ uint8_t* row_address(const CacheView& c, const int32_t* pos, int S,
                                                long long tok) {
  const int r = cache_row(c, c.table + (size_t)(tok / S) * c.max_pages, __ldg(pos + tok));
  return r >= 0 ? c.pages + (long long)r * c.row_bytes : nullptr;
}

// One unit of q or k: a group of 16 values, in the rotated part of the half-split form (MODE 2) the
// two groups of 16 pairs.
template <int MODE, bool ROTATED>
struct Unit {
  static constexpr bool kPair = MODE == 2 && ROTATED;
  Group x, y;  // y: the second group, J dims further
  int token, head, d;  // d: x's first dim
  // unit i of the CTA's: plain ones before the rotated part, or those of the rotated part
  __device__ __forceinline__ void place(int i, const Divisor& per_token, const Divisor& per_head,
                                        int first_dim) {
    token = per_token.of(i);
    const int e = i - token * (int)per_token.d;
    head = per_head.of(e);
    d = first_dim + 16 * (e - head * (int)per_head.d);
  }
  __device__ __forceinline__ void load(const __nv_bfloat16* p, int J) {
    x = load_group(p + d);
    if (kPair) y = load_group(p + d + J);
  }
  __device__ __forceinline__ void rotate(const Turn* turns, int first_dim) {
    if (kPair) rotate_halves(x, y, turns, d - first_dim);
    else if (ROTATED) rotate_interleaved(x, turns, (d - first_dim) / 2);
  }
  __device__ __forceinline__ void store(__nv_bfloat16* p, int J) const {
    store_group(p + d, x);
    if (kPair) store_group(p + d + J, y);
  }
  __device__ __forceinline__ void clear() {
    x.w[0] = x.w[1] = make_uint4(0, 0, 0, 0);
    if (kPair) y = x;
  }
};

// 64 units (number `chunk`) of q, or of k, of one kind, by one warp: two a lane, both loads ahead of
// the arithmetic.
template <int FMT, int MODE, bool ROTATED, bool IS_K>
__device__ __forceinline__ void take_units(const AppendArgs& a, long long tok0, int nt, int chunk,
                                           const Turn* turns, int per_turns, uint8_t* const* row_of,
                                           const bool* padding) {
  const Divisor& per_token = IS_K ? (ROTATED ? a.k_rot : a.k_plain) : (ROTATED ? a.q_rot : a.q_plain);
  const Divisor& per_head = ROTATED ? a.rot : a.plain;
  const CacheView& c = a.c;
  const int first = ROTATED ? c.DQK - 2 * a.J : 0;
  const int H = IS_K ? c.HKV : a.H, n = nt * (int)per_token.d;
  const __nv_bfloat16* src = IS_K ? a.k : a.q;
  __nv_bfloat16* dst = IS_K ? a.k_out : a.q_out;
  const int i0 = chunk * 64 + (threadIdx.x & 31);
  Unit<MODE, ROTATED> u[2];
#pragma unroll
  for (int z = 0; z < 2; ++z) {
    u[z].place(min(i0 + 32 * z, n - 1), per_token, per_head, first);
    u[z].load(src + ((size_t)(tok0 + u[z].token) * H + u[z].head) * c.DQK, a.J);
  }
#pragma unroll
  for (int z = 0; z < 2; ++z) {
    Unit<MODE, ROTATED>& w = u[z];
    w.rotate(turns + w.token * per_turns, first);
    if (padding[w.token]) w.clear();
    if (i0 + 32 * z >= n) continue;
    if (dst) w.store(dst + ((size_t)(tok0 + w.token) * H + w.head) * c.DQK, a.J);
    uint8_t* row = IS_K ? row_of[w.token] : nullptr;
    if (IS_K && row) {
      const int so = cache_ks_off(c.HKV, c.DQK, c.DV), at = w.head * c.DQK + w.d;
      put_group<FMT>(row, 0, so, at, w.x, a.k_scale);
      if (w.kPair) put_group<FMT>(row, 0, so, at + a.J, w.y, a.k_scale);
    }
  }
}
__device__ __forceinline__ int chunks_of(const Divisor& per_token, int nt) {
  return (nt * (int)per_token.d + 63) / 64;
}

template <int FMT, int MODE>
__global__ void __launch_bounds__(append_threads(FMT), 1024 / append_threads(FMT))
    cache_append_kernel(const AppendArgs a) {
  constexpr int kThreads = append_threads(FMT);
  extern __shared__ Turn turns[];  // [token][turn_at(J)]
  __shared__ uint8_t* row_of[kMaxTokens];
  __shared__ bool padding[kMaxTokens];
  const CacheView& c = a.c;
  const int per_turns = turn_at(a.J);
  const long long tok0 = (long long)blockIdx.x * a.per_cta;
  const int nt = (int)min((long long)a.per_cta, a.tokens - tok0);
  if ((int)threadIdx.x < nt) {
    row_of[threadIdx.x] = row_address(c, a.pos, a.S, tok0 + threadIdx.x);
    padding[threadIdx.x] = __ldg(a.pos + tok0 + threadIdx.x) < 0;
  }
  if (MODE != 0)
    for (int i = threadIdx.x; i < nt * a.J; i += kThreads) {
      const int p = __ldg(a.pos + tok0 + i / a.J);
      double sn = 0.0, cn = 1.0;
      if (p >= 0) sincos((double)p * (double)__ldg(a.inv_freq + i % a.J), &sn, &cn);
      turns[i / a.J * per_turns + turn_at(i % a.J)] = turn_of(cn, sn);
    }
  __syncthreads();
  // Chunks of one kind after another, the dearest first; a warp takes one at a time and so one path.
  const int kr = MODE != 0 ? chunks_of(a.k_rot, nt) : 0, kp = kr + chunks_of(a.k_plain, nt);
  const int vv = kp + chunks_of(a.uv, nt);
  const int qr = vv + (MODE != 0 && a.q ? chunks_of(a.q_rot, nt) : 0);
  const int qp = qr + (MODE != 0 && a.q ? chunks_of(a.q_plain, nt) : 0);
  for (int w = threadIdx.x >> 5; w < qp; w += kThreads / 32) {
    if (MODE != 0 && w < kr) {
      take_units<FMT, MODE, true, true>(a, tok0, nt, w, turns, per_turns, row_of, padding);
    } else if (w < kp) {
      take_units<FMT, MODE, false, true>(a, tok0, nt, w - kr, turns, per_turns, row_of, padding);
    } else if (w < vv) {
      const int n = nt * (int)a.uv.d, i0 = (w - kp) * 64 + (threadIdx.x & 31);
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        const int i = i0 + 32 * z;
        if (i >= n) break;
        const int t = a.uv.of(i), e = i - t * (int)a.uv.d;
        const Group x = load_group(a.v + (size_t)(tok0 + t) * c.HKV * c.DV + e * 16);
        if (uint8_t* row = row_of[t])
          put_group<FMT>(row, cache_v_off(FMT, c.HKV, c.DQK), cache_vs_off(c.HKV, c.DQK, c.DV),
                         e * 16, x, a.v_scale);
      }
    } else if (MODE != 0 && w < qr) {
      take_units<FMT, MODE, true, false>(a, tok0, nt, w - vv, turns, per_turns, row_of, padding);
    } else if (MODE != 0) {
      take_units<FMT, MODE, false, false>(a, tok0, nt, w - qr, turns, per_turns, row_of, padding);
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
                      int per_cta, Divisor uk, Divisor uv, __nv_bfloat16* __restrict__ k,
                      __nv_bfloat16* __restrict__ v) {
  __shared__ const uint8_t* row_of[kMaxTokens];
  const long long tok0 = (long long)blockIdx.x * per_cta;
  const int nt = (int)min((long long)per_cta, tokens - tok0);
  if ((int)threadIdx.x < nt) row_of[threadIdx.x] = row_address(c, pos, S, tok0 + threadIdx.x);
  __syncthreads();
  const Group zero = {{make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)}};
  const int nk = nt * (int)uk.d, n = nk + nt * (int)uv.d;
#pragma unroll 2
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const bool is_k = i < nk;
    const int t = is_k ? uk.of(i) : uv.of(i - nk);
    const int e = is_k ? i - t * (int)uk.d : i - nk - t * (int)uv.d;
    const uint8_t* row = row_of[t];
    __nv_bfloat16* to = (is_k ? k : v) + ((size_t)(tok0 + t) * (is_k ? uk.d : uv.d) + e) * 16;
    Group x = zero;
    if (row)
      x = get_group<FMT>(row, is_k ? 0 : cache_v_off(FMT, c.HKV, c.DQK),
                         is_k ? cache_ks_off(c.HKV, c.DQK, c.DV)
                              : cache_vs_off(c.HKV, c.DQK, c.DV),
                         e * 16, is_k ? c.k_scale : c.v_scale);
    store_group(to, x);
  }
}

TensorScale tensor_scale(float scale) {
  int e;
  const bool exact = frexpf(scale, &e) == 0.5f && e > -100 && e < 100;
  return TensorScale{scale, exact ? 1.0f / scale : 0.f};
}

// Tokens per CTA: enough CTAs to fill the GPU first, then several tokens each (their sines in one
// go, and their units spread over the warps).  Appending with queries of 32 heads, in us for one, two,
// three and four tokens a CTA (interleaved pairs): 4 bits, 8 heads, 4736 tokens 41, 37, 39, 34; 8002
// tokens 66, 62, 60, 57; 24000 tokens 185, 166, 163, 158: four.  bf16, 32 heads, 8002 tokens 100, 91,
// 92, 94 and reading back 52, 54, 56, 57; 24000 tokens 286, 258, 259, 259 and 146, 149, 152, 154: two
// (8 heads would take four: 24000 tokens 184, 165, 151, 150).  The last, partly filled round of CTAs
// moves any one size by up to 10% either way (4 bits, 6000 tokens: 50, 46, 45, 48).
int tokens_per_cta(long long tokens, int format) {
  const long long per = tokens / (148 * 8), most = format == 1 ? 4 : 2;
  return (int)(per < 1 ? 1 : (per > most ? most : per));
}

template <int FMT>
void launch_append(const AppendArgs& a, int mode, unsigned grid, size_t smem, cudaStream_t st) {
  constexpr int threads = append_threads(FMT);
  if (mode == 0) cache_append_kernel<FMT, 0><<<grid, threads, smem, st>>>(a);
  if (mode == 1) cache_append_kernel<FMT, 1><<<grid, threads, smem, st>>>(a);
  if (mode == 2) cache_append_kernel<FMT, 2><<<grid, threads, smem, st>>>(a);
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
  a.S = p.S; a.H = p.H;
  a.J = p.rope_mode == 0 ? 0 : p.rope_dim / 2;
  a.tokens = (long long)p.B * p.S;
  a.per_cta = tokens_per_cta(a.tokens, a.c.format);
  const int plain = (a.c.DQK - 2 * a.J) / 16, rot = p.rope_mode == 2 ? a.J / 16 : a.J / 8;
  a.plain = divisor(plain > 0 ? plain : 1);
  a.rot = divisor(rot > 0 ? rot : 1);
  a.q_plain = divisor(a.H * plain);
  a.q_rot = divisor(a.H * rot);
  a.k_plain = divisor(a.c.HKV * plain);
  a.k_rot = divisor(a.c.HKV * rot);
  a.uv = divisor(a.c.HKV * a.c.DV / 16);
  const unsigned grid = (unsigned)((a.tokens + a.per_cta - 1) / a.per_cta);
  a.k_scale = tensor_scale(a.c.k_scale);
  a.v_scale = tensor_scale(a.c.v_scale);
  const size_t smem = (size_t)a.per_cta * (a.J + a.J / 8) * sizeof(Turn);
  if (a.c.format == 0)
    launch_append<0>(a, p.rope_mode, grid, smem, st);
  else
    launch_append<1>(a, p.rope_mode, grid, smem, st);
  return cudaGetLastError();
}

cudaError_t launch_cache_read(const CacheView& c, const int32_t* pos, int B, int S, void* k,
                              void* v, cudaStream_t st) {
  const long long tokens = (long long)B * S;
  const int per = tokens_per_cta(tokens, c.format);
  const unsigned grid = (unsigned)((tokens + per - 1) / per);
  const Divisor uk = divisor(c.HKV * c.DQK / 16), uv = divisor(c.HKV * c.DV / 16);
  __nv_bfloat16 *kt = static_cast<__nv_bfloat16*>(k), *vt = static_cast<__nv_bfloat16*>(v);
  if (c.format == 0)
    cache_read_kernel<0><<<grid, kThreads, 0, st>>>(c, pos, S, tokens, per, uk, uv, kt, vt);
  else
    cache_read_kernel<1><<<grid, kThreads, 0, st>>>(c, pos, S, tokens, per, uk, uv, kt, vt);
  return cudaGetLastError();
}

}  // namespace dsa
