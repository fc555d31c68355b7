// Attention over the paged cache: what the bf16 kernel (cache_attn.cu) and the 4-bit kernel
// (cache_attn_q4.cu) share.
#pragma once

#include "cache.cuh"
#include "kernels.h"

namespace dsa {

struct CacheAttnArgs {
  CacheView c;
  const __nv_bfloat16* q;  // [B,S,H,DQK]
  const int32_t* pos;      // [B,S]
  const int32_t* idx;      // [B,S,K] or NULL
  const __nv_bfloat16* gate;
  __nv_bfloat16* out;      // [B,S,H,DV]
  float* part_o;           // [rows, nsplit, H, DV] (nsplit > 1)
  float* part_ml;          // [rows, nsplit, H, 2]
  int gate_mode, S, H, G, K, window, n_first;
  float qk_scale;          // sm_scale * log2(e) * k_scale
  int nsplit, hc, nhg;     // key slices, KV heads per CTA, CTAs per (token, slice)
  int nsub, kw;            // warps per KV head (8 query heads each), 16-key groups side by side
  int nstages, pitch;      // bf16: ring depth, bytes between the rows in shared memory
};

// Launches the 4-bit kernel over `grid` CTAs (cache_attn_q4.cu).
cudaError_t launch_cache_attn_q4(const CacheAttnArgs& a, unsigned grid, cudaStream_t st);
// Its CTA: warps, all of them consumers.
constexpr int kQ4Warps = 8;

namespace {

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3},{%4,%5,%6,%7},{%8,%9},"
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The same with C = 0.
__device__ __forceinline__ void mma_f16_zero(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                             uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3},{%4,%5,%6,%7},{%8,%9},"
      "{%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3},{%4,%5,%6,%7},{%8,%9},"
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// The keys of a query at position `pos`: n of them, key e being at(e).
struct KeyList {
  const int32_t* idx;
  int n, nf, low;
  __device__ __forceinline__ int at(int e) const {
    return idx ? __ldg(idx + e) : (e < nf ? e : low + (e - nf));
  }
};
__device__ __forceinline__ KeyList key_list(const CacheAttnArgs& a, int row, int pos) {
  KeyList l;
  l.idx = a.idx ? a.idx + (size_t)row * a.K : nullptr;
  l.nf = l.low = 0;
  if (pos < 0) {
    l.n = 0;
  } else if (a.idx) {
    l.n = a.K;
  } else {
    const int hi = min(pos, a.c.cap - 1);
    l.low = a.window > 0 && pos >= a.window ? pos - a.window + 1 : 0;
    l.nf = min(min(a.n_first, l.low), a.c.cap);
    l.n = l.nf + max(0, hi - l.low + 1);
  }
  return l;
}

// This CTA's slice [j0, j1) of the list: equal slices, whole groups of 16 keys.
__device__ __forceinline__ void key_slice(const KeyList& l, int nsplit, int split, int* j0,
                                          int* j1) {
  const int per = ((l.n + nsplit - 1) / nsplit + 15) & ~15;
  const long long j = (long long)split * per;
  *j0 = (int)min(j, (long long)l.n);
  *j1 = (int)min(j + per, (long long)l.n);
}

// One 16-key step of the online softmax for the columns 2t, 2t + 1 (heads) of this thread's rows:
// x = (key g: two columns, key g + 8: two columns) in log2 units, -inf for keys not there.  The
// running maximum m sits 2^TOP above 1 and is raised once a score passes it by 2^8; p, l and o
// follow it.
template <int TOP, int MT>
__device__ __forceinline__ void softmax_step(const float (&x)[4], float (&m)[2], float (&l)[2],
                                             float (&o)[MT][4], float (&p)[4]) {
  float y0 = fmaxf(x[0], x[2]), y1 = fmaxf(x[1], x[3]);
  if (__any_sync(0xffffffffu, y0 > m[0] + (TOP + 8.0f) || y1 > m[1] + (TOP + 8.0f))) {
#pragma unroll
    for (int d = 4; d < 32; d <<= 1) {
      y0 = fmaxf(y0, __shfl_xor_sync(0xffffffffu, y0, d));
      y1 = fmaxf(y1, __shfl_xor_sync(0xffffffffu, y1, d));
    }
    const float n0 = fmaxf(m[0], y0 - TOP), n1 = fmaxf(m[1], y1 - TOP);
    const float a0 = m[0] == -INFINITY ? 0.f : ex2_ftz(m[0] - n0);
    const float a1 = m[1] == -INFINITY ? 0.f : ex2_ftz(m[1] - n1);
    l[0] *= a0;
    l[1] *= a1;
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      o[i][0] *= a0; o[i][1] *= a1; o[i][2] *= a0; o[i][3] *= a1;
    }
    m[0] = n0;
    m[1] = n1;
  }
  // a column without a score above -inf so far has m = -inf: its p must be 0, not NaN
  const float u0 = m[0] == -INFINITY ? 0.f : m[0], u1 = m[1] == -INFINITY ? 0.f : m[1];
  p[0] = ex2_ftz(x[0] - u0);
  p[1] = ex2_ftz(x[1] - u1);
  p[2] = ex2_ftz(x[2] - u0);
  p[3] = ex2_ftz(x[3] - u1);
  l[0] += p[0] + p[2];
  l[1] += p[1] + p[3];
}

// The end of a CTA's slice: the warps' (m, l) in ml [warp][8][2] and O in ob [warp][8][DV] are
// merged over the key groups in order (warp = group * nhw + head warp), into the output row or
// this slice's part of it.
template <int DV>
__device__ __forceinline__ void merge_groups(const CacheAttnArgs& a, const float* ml,
                                             const float* ob, int nhw, int row, int split,
                                             int kv0) {
  for (int i = threadIdx.x; i < a.hc * a.G * (DV / 4); i += blockDim.x) {
    const int hl = i / (DV / 4), d = (i % (DV / 4)) * 4;
    const int hh = hl % a.G;
    const int hw = (hl / a.G) * a.nsub + (hh >> 3), col = hh & 7;
    float M = -INFINITY;
    for (int k = 0; k < a.kw; ++k) M = fmaxf(M, ml[(k * nhw + hw) * 16 + col * 2]);
    float L = 0.f, x[4] = {0.f, 0.f, 0.f, 0.f};
    for (int k = 0; k < a.kw; ++k) {
      const int w = k * nhw + hw;
      const float mk = ml[w * 16 + col * 2];
      const float f = mk == -INFINITY ? 0.f : ex2_ftz(mk - M);
      L = fmaf(ml[w * 16 + col * 2 + 1], f, L);
      const float4 v = *reinterpret_cast<const float4*>(ob + (size_t)(w * 8 + col) * DV + d);
      x[0] = fmaf(v.x, f, x[0]); x[1] = fmaf(v.y, f, x[1]);
      x[2] = fmaf(v.z, f, x[2]); x[3] = fmaf(v.w, f, x[3]);
    }
    const int h = kv0 * a.G + hl;
    if (a.nsplit == 1) {
      float f = L > 0.f ? a.c.v_scale / L : 0.f;
      if (a.gate) f *= gate_act(__bfloat162float(a.gate[(size_t)row * a.H + h]), a.gate_mode);
      const __nv_bfloat162 y0 = __floats2bfloat162_rn(x[0] * f, x[1] * f);
      const __nv_bfloat162 y1 = __floats2bfloat162_rn(x[2] * f, x[3] * f);
      uint2 y;
      y.x = *reinterpret_cast<const uint32_t*>(&y0);
      y.y = *reinterpret_cast<const uint32_t*>(&y1);
      *reinterpret_cast<uint2*>(a.out + ((size_t)row * a.H + h) * DV + d) = y;
    } else {
      const size_t base = ((size_t)row * a.nsplit + split) * a.H + h;
      const float f = a.c.v_scale;
      *reinterpret_cast<float4*>(a.part_o + base * DV + d) =
          make_float4(x[0] * f, x[1] * f, x[2] * f, x[3] * f);
      if (d == 0) {
        a.part_ml[base * 2] = M;
        a.part_ml[base * 2 + 1] = L;
      }
    }
  }
}

}  // namespace

}  // namespace dsa
