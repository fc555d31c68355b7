// Attention of single query tokens over the paged key/value cache (bf16 rows, or rows held in 4
// bits), with a sliding window and visible first tokens, over whole contexts, or over selected
// keys; the headwise gate fused.
//
//   o[h,:] = sum_t p_t v[t,h/G,:],  p = softmax_t(sm_scale * q[h,:] . k[t,h/G,:]),  G = H/HKV
//
// over the query's keys: idx[b,s,:], or t <= pos with t > pos - window or t < n_first.  Every
// query token has its own key list, so masked keys are never read and what they hold (NaN, a
// page of another sequence, nothing yet) does not matter.
//
// Work split.  One CTA takes a query token, a group of KV heads and a slice of its keys; a
// producer warp turns keys into cache rows through the page table and streams them into a ring of
// shared-memory slots (1-D bulk copies, mbarrier transaction counts, no multicast); each consumer
// warp owns one KV head (8 of its query heads) and 16 keys of a stage.  Slices of one query are
// merged by launch_split_combine in a fixed order.
//
// Products.  Both run on mma.sync m16n8k16 with the cache as the 16-row operand and the up to 8
// query heads of a KV head as the 8 columns: S^T = K Q^T [16 keys x 8 heads], O^T += V^T P^T
// [dims x 8 heads], float32 accumulation.  (A tcgen05 tile would need 128 rows that share an
// operand, and the operand in shared memory in its final type; here 4-bit rows are widened in
// registers on their way into the product, for 1 to 8 rows.)  The contraction order is free, so
// each thread takes the 16 consecutive dims that share a scale: one 8-byte load, one scale.
//
// 4-bit rows are widened to f16, exactly: an e2m1 value times an e4m3 scale has 6 significant
// bits and stays in f16's normal range.  Queries become f16 after a scaling of each head by a
// power of two (its largest element to [2^13, 2^14)): exact for every element within 2^-30 of
// the largest (8 bits into 11), and off by 2^-38 of it at most otherwise.  Probabilities
// are f16 with the running maximum at 2^6 (so terms down to 2^-30 of the largest stay): half a
// step is 2^-11 each, below the rounding of the output.  bf16 rows are used as they are, with
// probabilities as a bf16 pair hi + lo.
#include <cuda_fp16.h>

#include "cache.cuh"
#include "kernels.h"

namespace dsa {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kMaxWarps = 16;     // consumer warps of a CTA
constexpr int kMaxStages = 8;
constexpr int kMaxSplit = 64;     // launch_split_combine's limit

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
  int nsub, kw;            // warps per KV head (8 query heads each), 16-key groups per stage
  int nstages, pitch;      // ring depth, bytes between the rows in shared memory
};

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3},{%4,%5,%6,%7},{%8,%9},"
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
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
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// 4 or 8 consecutive bytes of a slot (aligned to their size).
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[1]) {
  w[0] = *reinterpret_cast<const uint32_t*>(p);
}
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[2]) {
  const uint2 v = *reinterpret_cast<const uint2*>(p);
  w[0] = v.x;
  w[1] = v.y;
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
    const int hi = (long long)pos < a.c.cap ? pos : (int)(a.c.cap - 1);  // cap <= 2^30
    l.low = a.window > 0 && pos >= a.window ? pos - a.window + 1 : 0;
    l.nf = (int)min((long long)min(a.n_first, l.low), a.c.cap);
    l.n = l.nf + max(0, hi - l.low + 1);
  }
  return l;
}

// Consumer row order.  Row m of the 16-row operands is key kappa(m) of the group (m and m + 8
// alike): with rows 32 bytes (mod 128) apart, both the K loads (rows g = 0..3 and 4..7 of a half
// warp) and the V loads (rows 2t, or 2t + 1) then touch four different 32-byte bank groups.
template <int FMT>
__device__ __forceinline__ int kappa(int g) {
  return FMT == 1 ? (g ^ ((g >> 2) & 1)) : g;
}

template <int FMT, int DQK, int DV>
__global__ void __maxnreg__(112) cache_attn_kernel(const CacheAttnArgs a) {
  constexpr int QC = DQK / 64;       // 64-dim chunks: 16 dims per thread each
  constexpr int MT = DV / 16;        // 16-row tiles of O^T
  constexpr int VPT = DV / 8;        // e2m1: value dims per thread row
  extern __shared__ __align__(128) uint8_t smem[];
  uint64_t* full = reinterpret_cast<uint64_t*>(smem);
  uint64_t* empty = full + kMaxStages;
  int* meta = reinterpret_cast<int*>(empty + kMaxStages);  // [stage][8]: -1 = end, 4 mask words
  float* ml = reinterpret_cast<float*>(smem + 512);        // [warp][8][2]
  uint8_t* ring = smem + 512 + kMaxWarps * 64;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t4 = lane & 3;
  const int nw = (blockDim.x >> 5) - 1;
  const int nhw = nw / a.kw;                 // warps that share a key group
  const int split = blockIdx.x % a.nsplit;
  const int hg = (blockIdx.x / a.nsplit) % a.nhg;
  const int row = blockIdx.x / (a.nsplit * a.nhg);
  const int hc = a.hc, kv0 = hg * hc;
  const int ks = a.kw * 16;                  // keys per stage
  const int pos = __ldg(a.pos + row);

  if (threadIdx.x == 0) {
    for (int i = 0; i < a.nstages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], nw);
    }
    fence_mbar_init();
  }
  __syncthreads();

  // byte offsets of this CTA's heads inside a slot: K, V, K scales, V scales
  const int kb = FMT == 0 ? hc * DQK * 2 : hc * DQK / 2;
  const int vb = FMT == 0 ? hc * DV * 2 : hc * DV / 2;
  const int ksb = hc * DQK / 16, vsb = hc * DV / 16;

  if (warp == nw) {
    // ------------------------------------------------------------- producer
    const KeyList l = key_list(a, row, pos);
    const int per = ((l.n + a.nsplit - 1) / a.nsplit + 15) & ~15;
    const long long j0l = (long long)split * per;
    const int j0 = (int)min(j0l, (long long)l.n);
    const int j1 = (int)min(j0l + per, (long long)l.n);
    const int b = row / a.S;
    const bool whole = a.nhg == 1;  // one copy of the row, else its parts for these heads
    const uint32_t bytes = whole ? (uint32_t)a.c.row_bytes
                                 : (uint32_t)(kb + vb + (FMT == 1 ? ksb + vsb : 0));
    int fills = 0;
    bool ok = true;
    for (int j = j0; ok && j < j1;) {
      long long r[4];
      uint32_t m[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        r[i] = -1;
        m[i] = 0;
        if (32 * i < ks) {  // warp-uniform
          const int e = j + 32 * i + lane;
          if (32 * i + lane < ks && e < j1) {
            const int t = l.at(e);
            if (t <= pos) r[i] = cache_row(a.c, b, t);
          }
          m[i] = __ballot_sync(0xffffffffu, r[i] >= 0);
        }
      }
      j = j1 - j > ks ? j + ks : j1;
      const int nvalid = __popc(m[0]) + __popc(m[1]) + __popc(m[2]) + __popc(m[3]);
      if (nvalid == 0) continue;
      const int st = fills % a.nstages;
      if (fills >= a.nstages)
        ok = warp_wait(&empty[st], (uint32_t)(fills / a.nstages - 1) & 1u);
      if (!ok) break;
      if (lane == 0) {
        meta[st * 8] = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) meta[st * 8 + 1 + i] = (int)m[i];
        mbar_arrive_expect_tx(&full[st], (uint32_t)nvalid * bytes);
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (r[i] < 0) continue;
        uint8_t* dst = ring + (size_t)(st * ks + 32 * i + lane) * a.pitch;
        const uint8_t* src = a.c.pages + r[i] * a.c.row_bytes;
        if (whole) {
          bulk_g2s(dst, src, bytes, &full[st]);
        } else {
          bulk_g2s(dst, src + (size_t)kv0 * (kb / hc), kb, &full[st]);
          bulk_g2s(dst + kb, src + cache_v_off(FMT, a.c.HKV, DQK) + (size_t)kv0 * (vb / hc), vb,
                   &full[st]);
          if (FMT == 1) {
            bulk_g2s(dst + kb + vb, src + cache_ks_off(a.c.HKV, DQK, DV) + kv0 * (DQK / 16), ksb,
                     &full[st]);
            bulk_g2s(dst + kb + vb + ksb, src + cache_vs_off(a.c.HKV, DQK, DV) + kv0 * (DV / 16),
                     vsb, &full[st]);
          }
        }
      }
      ++fills;
    }
    // the end mark takes a stage of its own
    const int st = fills % a.nstages;
    if (ok && fills >= a.nstages)
      ok = warp_wait(&empty[st], (uint32_t)(fills / a.nstages - 1) & 1u);
    if (ok && lane == 0) {
      meta[st * 8] = -1;
      mbar_arrive(&full[st]);
    }
    // Copies in flight land before the ring is used again or the CTA exits: the last fill of
    // every stage but the end mark's (whose stage was empty), or of all when a wait gave up.
    if (lane == 0)
      for (int f = fills - 1; f >= 0 && f >= fills - a.nstages + (ok ? 1 : 0); --f)
        drain_wait(&full[f % a.nstages], (uint32_t)(f / a.nstages) & 1u);
    __syncwarp();
  } else {
    // ------------------------------------------------------------- consumers
    const int kg = warp / nhw, hw = warp % nhw;
    const int kvl = hw / a.nsub, sub = hw % a.nsub;  // local KV head, block of 8 query heads
    const int ncol = min(8, a.G - sub * 8);          // query heads in the 8 columns
    const int h0 = (kv0 + kvl) * a.G + sub * 8;

    // Q^T fragments: column g, dims 64c + 16t .. + 15 of the head
    uint32_t qf[QC][8];
    float cs[2];  // score scale of columns 2t, 2t + 1
    {
      const bool has = g < ncol;
      const uint4* qp = reinterpret_cast<const uint4*>(
          a.q + ((size_t)row * a.H + (has ? h0 + g : 0)) * DQK + 16 * t4);
#pragma unroll
      for (int c = 0; c < QC; ++c)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint4 x = has ? __ldg(qp + c * 8 + i) : make_uint4(0, 0, 0, 0);
          qf[c][4 * i + 0] = x.x; qf[c][4 * i + 1] = x.y;
          qf[c][4 * i + 2] = x.z; qf[c][4 * i + 3] = x.w;
        }
      float scale = a.qk_scale;
      if (FMT == 1) {
        uint32_t top = 0;  // the largest exponent field: of |q|, as bits
#pragma unroll
        for (int c = 0; c < QC; ++c)
#pragma unroll
          for (int i = 0; i < 8; ++i)
            top = max(top, max((qf[c][i] << 16) & 0x7f800000u, qf[c][i] & 0x7f800000u));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int ex = max((int)(top >> 23) - 127, -100);  // 2^ex <= max|q| (or less)
        const float up = __int_as_float((13 - ex + 127) << 23);
        scale *= __int_as_float((ex - 13 + 127) << 23);
#pragma unroll
        for (int c = 0; c < QC; ++c)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float x0 = __uint_as_float(qf[c][i] << 16) * up;
            const float x1 = __uint_as_float(qf[c][i] & 0xffff0000u) * up;
            const __half2 h = __floats2half2_rn(x0, x1);
            qf[c][i] = *reinterpret_cast<const uint32_t*>(&h);
          }
      }
      cs[0] = __shfl_sync(0xffffffffu, scale, (2 * t4) * 4);
      cs[1] = __shfl_sync(0xffffffffu, scale, (2 * t4 + 1) * 4);
    }
    // the running maximum sits at 2^kTop (f16 probabilities), raised past 2^8 above it
    constexpr float kTop = FMT == 1 ? 6.0f : 0.0f;
    constexpr float kRaise = kTop + 8.0f;
    float o[MT][4];
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] = 0.f;

    const int key_a = kg * 16 + kappa<FMT>(g);  // rows g and g + 8 of the K operand
    const int key_v0 = kg * 16 + kappa<FMT>(2 * t4), key_v1 = kg * 16 + kappa<FMT>(2 * t4 + 1);
    int st = 0;
    uint32_t phase = 0;
    while (warp_wait(&full[st], phase)) {
      if (meta[st * 8] < 0) break;
      const uint32_t mask = ((uint32_t)meta[st * 8 + 1 + (kg >> 1)] >> ((kg & 1) * 16)) & 0xffffu;
      if (mask != 0u) {
        const uint8_t* slot = ring + (size_t)st * ks * a.pitch;
        float s[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[i][e] = 0.f;
        const uint8_t* ra = slot + (size_t)key_a * a.pitch;
        const uint8_t* rb = ra + (size_t)8 * a.pitch;
        if constexpr (FMT == 1) {
          const int co = kvl * (DQK / 2) + t4 * 8;
          const int so = kb + vb + kvl * (DQK / 16) + t4;
#pragma unroll
          for (int c = 0; c < QC; ++c) {
            const uint2 wa = *reinterpret_cast<const uint2*>(ra + co + c * 32);
            const uint2 wb = *reinterpret_cast<const uint2*>(rb + co + c * 32);
            const uint32_t sa = e4m3x2_to_f16((uint32_t)ra[so + c * 4] * 0x0101u);
            const uint32_t sb = e4m3x2_to_f16((uint32_t)rb[so + c * 4] * 0x0101u);
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              uint32_t xa[4], xb[4];
              e2m1x8_to_f16(hf ? wa.y : wa.x, xa);
              e2m1x8_to_f16(hf ? wb.y : wb.x, xb);
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const uint32_t f[4] = {mul_f16x2(xa[2 * i], sa), mul_f16x2(xb[2 * i], sb),
                                       mul_f16x2(xa[2 * i + 1], sa), mul_f16x2(xb[2 * i + 1], sb)};
                mma_f16(s[i], f, qf[c][4 * hf + 2 * i], qf[c][4 * hf + 2 * i + 1]);
              }
            }
          }
        } else {
          const int co = kvl * (DQK * 2) + t4 * 32;
#pragma unroll
          for (int c = 0; c < QC; ++c)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              const uint4 xa = *reinterpret_cast<const uint4*>(ra + co + c * 128 + hf * 16);
              const uint4 xb = *reinterpret_cast<const uint4*>(rb + co + c * 128 + hf * 16);
              const uint32_t f0[4] = {xa.x, xb.x, xa.y, xb.y};
              const uint32_t f1[4] = {xa.z, xb.z, xa.w, xb.w};
              mma_bf16(s[0], f0, qf[c][4 * hf], qf[c][4 * hf + 1]);
              mma_bf16(s[1], f1, qf[c][4 * hf + 2], qf[c][4 * hf + 3]);
            }
        }
        // scores in log2 units: (key a, columns 2t, 2t + 1), (key a + 8, the same)
        const bool va = (mask >> (key_a & 15)) & 1u, vbk = (mask >> ((key_a & 15) + 8)) & 1u;
        const float x0 = va ? (s[0][0] + s[1][0]) * cs[0] : -INFINITY;
        const float x1 = va ? (s[0][1] + s[1][1]) * cs[1] : -INFINITY;
        const float x2 = vbk ? (s[0][2] + s[1][2]) * cs[0] : -INFINITY;
        const float x3 = vbk ? (s[0][3] + s[1][3]) * cs[1] : -INFINITY;
        float y0 = fmaxf(x0, x2), y1 = fmaxf(x1, x3);
        if (__any_sync(0xffffffffu, y0 > m0 + kRaise || y1 > m1 + kRaise)) {
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) {
            y0 = fmaxf(y0, __shfl_xor_sync(0xffffffffu, y0, d));
            y1 = fmaxf(y1, __shfl_xor_sync(0xffffffffu, y1, d));
          }
          const float n0 = fmaxf(m0, y0 - kTop), n1 = fmaxf(m1, y1 - kTop);
          const float a0 = m0 == -INFINITY ? 0.f : ex2_ftz(m0 - n0);
          const float a1 = m1 == -INFINITY ? 0.f : ex2_ftz(m1 - n1);
          // a sum that is already NaN stays so; one of no keys is 0 either way
          l0 *= a0;
          l1 *= a1;
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            o[i][0] *= a0; o[i][1] *= a1; o[i][2] *= a0; o[i][3] *= a1;
          }
          m0 = n0;
          m1 = n1;
        }
        // a column whose scores are all -inf so far has m = -inf: its p must be 0, not NaN
        const float u0 = m0 == -INFINITY ? 0.f : m0, u1 = m1 == -INFINITY ? 0.f : m1;
        const float p0 = ex2_ftz(x0 - u0), p1 = ex2_ftz(x1 - u1);
        const float p2 = ex2_ftz(x2 - u0), p3 = ex2_ftz(x3 - u1);
        l0 += p0 + p2;
        l1 += p1 + p3;
        if constexpr (FMT == 1) {
          const __half2 h0_ = __floats2half2_rn(p0, p1), h1_ = __floats2half2_rn(p2, p3);
          const uint32_t b0 = transpose8x8(*reinterpret_cast<const uint32_t*>(&h0_));
          const uint32_t b1 = transpose8x8(*reinterpret_cast<const uint32_t*>(&h1_));
          const uint8_t* v0 = slot + (size_t)key_v0 * a.pitch;
          const uint8_t* v1 = slot + (size_t)key_v1 * a.pitch;
          const uint8_t* v2 = v0 + (size_t)8 * a.pitch;
          const uint8_t* v3 = v1 + (size_t)8 * a.pitch;
          const int so = kb + vb + ksb + kvl * (DV / 16) + (g * VPT) / 16;
          uint32_t sc0 = v0[so] | ((uint32_t)v1[so] << 8), sc1 = v2[so] | ((uint32_t)v3[so] << 8);
          if (mask != 0xffffu) {  // a slot that was not filled may hold a NaN scale
            const uint32_t k0 = key_v0 & 15, k1 = key_v1 & 15;
            sc0 &= (((mask >> k0) & 1u) * 0xffu) | (((mask >> k1) & 1u) * 0xff00u);
            sc1 &= (((mask >> (k0 + 8)) & 1u) * 0xffu) | (((mask >> (k1 + 8)) & 1u) * 0xff00u);
          }
          const uint32_t s01 = e4m3x2_to_f16(sc0), s23 = e4m3x2_to_f16(sc1);
          const int co = kb + kvl * (DV / 2) + g * (VPT / 2);
          uint32_t vw[4][VPT / 8];
          load_words(v0 + co, vw[0]);
          load_words(v1 + co, vw[1]);
          load_words(v2 + co, vw[2]);
          load_words(v3 + co, vw[3]);
#pragma unroll
          for (int wd = 0; wd < VPT / 8; ++wd) {
            const uint32_t w0 = vw[0][wd], w1 = vw[1][wd], w2 = vw[2][wd], w3 = vw[3][wd];
            constexpr uint32_t kLo = 0x0f0f0f0fu;
            uint32_t e01[4], o01[4], e23[4], o23[4];  // even and odd dims of two keys each
            e2m1x8_to_f16((w0 & kLo) | ((w1 << 4) & ~kLo), e01);
            e2m1x8_to_f16(((w0 >> 4) & kLo) | (w1 & ~kLo), o01);
            e2m1x8_to_f16((w2 & kLo) | ((w3 << 4) & ~kLo), e23);
            e2m1x8_to_f16(((w2 >> 4) & kLo) | (w3 & ~kLo), o23);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t f[4] = {mul_f16x2(e01[i], s01), mul_f16x2(o01[i], s01),
                                     mul_f16x2(e23[i], s23), mul_f16x2(o23[i], s23)};
              mma_f16(o[4 * wd + i], f, b0, b1);
            }
          }
        } else {
          const __nv_bfloat162 h01 = __floats2bfloat162_rn(p0, p1);
          const __nv_bfloat162 h23 = __floats2bfloat162_rn(p2, p3);
          const __nv_bfloat162 r01 = __floats2bfloat162_rn(p0 - __low2float(h01),
                                                           p1 - __high2float(h01));
          const __nv_bfloat162 r23 = __floats2bfloat162_rn(p2 - __low2float(h23),
                                                           p3 - __high2float(h23));
          const uint32_t b0 = transpose8x8(*reinterpret_cast<const uint32_t*>(&h01));
          const uint32_t b1 = transpose8x8(*reinterpret_cast<const uint32_t*>(&h23));
          const uint32_t c0 = transpose8x8(*reinterpret_cast<const uint32_t*>(&r01));
          const uint32_t c1 = transpose8x8(*reinterpret_cast<const uint32_t*>(&r23));
          uint32_t k01 = 0xffffffffu, k23 = 0xffffffffu;
          if (mask != 0xffffu) {  // a slot that was not filled may hold anything
            k01 = (((mask >> (2 * t4)) & 1u) * 0xffffu) |
                  (((mask >> (2 * t4 + 1)) & 1u) * 0xffff0000u);
            k23 = (((mask >> (2 * t4 + 8)) & 1u) * 0xffffu) |
                  (((mask >> (2 * t4 + 9)) & 1u) * 0xffff0000u);
          }
          const uint32_t va_ = smem_u32(slot) +
                               (uint32_t)((kg * 16 + (lane & 7) + ((lane >> 4) << 3)) * a.pitch +
                                          kb + kvl * (DV * 2) + ((lane >> 3) & 1) * 16);
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            uint32_t f[4];
            ldmatrix_x4_trans(f, va_ + i * 32);
            f[0] &= k01; f[1] &= k01; f[2] &= k23; f[3] &= k23;
            mma_bf16(o[i], f, b0, b1);
            mma_bf16(o[i], f, c0, c1);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[st]);
      if (++st == a.nstages) {
        st = 0;
        phase ^= 1u;
      }
    }
    // this warp's (m, l, O) for the merge
#pragma unroll
    for (int d = 4; d < 32; d <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, d);
      l1 += __shfl_xor_sync(0xffffffffu, l1, d);
    }
    __syncthreads();  // every warp is done with the ring, and its copies have landed
    if (g == 0) {
      float* w = ml + warp * 16 + 4 * t4;
      w[0] = m0; w[1] = l0; w[2] = m1; w[3] = l1;
    }
    float* ow = reinterpret_cast<float*>(ring) + (size_t)warp * 8 * DV;
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      float* c0 = ow + (2 * t4) * DV;
      float* c1 = c0 + DV;
      if constexpr (FMT == 1) {
        const int d = g * VPT + 2 * i;
        *reinterpret_cast<float2*>(c0 + d) = make_float2(o[i][0], o[i][2]);
        *reinterpret_cast<float2*>(c1 + d) = make_float2(o[i][1], o[i][3]);
      } else {
        const int d = 16 * i + g;
        c0[d] = o[i][0]; c1[d] = o[i][1]; c0[d + 8] = o[i][2]; c1[d + 8] = o[i][3];
      }
    }
  }
  if (warp == nw) __syncthreads();  // the producer's part of the barrier above
  __syncthreads();

  // merge of the key groups, in order; then the output row, or this slice's part of it
  const float* ob = reinterpret_cast<const float*>(ring);
  for (int i = threadIdx.x; i < hc * a.G * (DV / 4); i += blockDim.x) {
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

// How a call is laid out over CTAs: KV heads per CTA, warps, stages, key slices.
struct Plan {
  int hc, nhg, nsub, kw, nw, nstages, pitch, nsplit;
  size_t smem;
};

constexpr size_t kHeadBytes = 512 + kMaxWarps * 64;  // barriers, stage marks, (m, l) of the warps

// Ring of `hc` KV heads per CTA; false if two stages do not fit.
bool plan_ring(int format, int hc, int HKV, int DQK, int DV, Plan* p) {
  p->hc = hc;
  p->nhg = HKV / hc;
  const int nhw = hc * p->nsub;
  p->kw = nhw >= 8 ? 1 : 8 / nhw;
  p->nw = nhw * p->kw;
  const long long part = cache_row_bytes(format, hc, DQK, DV);
  // rows 32 or 96 bytes (4 bits) or 16 bytes (bf16) past a multiple of 128 apart: the loads of
  // the consumer warps then meet no bank twice
  const int step = format == 1 ? 64 : 128, want = format == 1 ? 32 : 16;
  p->pitch = (int)((part - want + step - 1) / step * step + want);
  const size_t stage = (size_t)p->kw * 16 * p->pitch;
  const size_t merge = (size_t)p->nw * 8 * DV * 4;
  // two CTAs per SM where two stages fit in half of its 227 KB, else one
  size_t budget = p->nw <= 8 ? 113 * 1024 : 226 * 1024;
  if (kHeadBytes + 2 * stage > budget) budget = 226 * 1024;
  if (kHeadBytes + 2 * stage > budget || kHeadBytes + merge > budget) return false;
  const int ns = (int)((budget - kHeadBytes) / stage);
  p->nstages = ns > kMaxStages ? kMaxStages : ns;
  const size_t ring = p->nstages * stage;
  p->smem = kHeadBytes + (ring > merge ? ring : merge);
  return true;
}

// Shapes only (no device query), so that workspace sizes are reproducible.
bool make_plan(int format, int rows, int H, int HKV, int DQK, int DV, long long max_keys, Plan* p) {
  const int G = H / HKV;
  p->nsub = (G + 7) / 8;
  // KV heads per CTA: up to 8 warps of them where they divide evenly and the parts of a row stay
  // multiples of 16 bytes (4-bit scales: 4 heads, or 2 with both dims 128); heads that do not
  // divide so share one CTA of up to 16 warps
  const int unit = format == 0 ? 1 : (DQK == 128 && DV == 128 ? 2 : 4);
  bool fits = false;
  if (HKV * p->nsub <= 8) {
    fits = plan_ring(format, HKV, HKV, DQK, DV, p);
  } else {
    int h = 8 / p->nsub;
    while (h > 0 && (HKV % h != 0 || h % unit != 0)) --h;
    if (h * p->nsub < 4 && HKV * p->nsub <= kMaxWarps)
      fits = plan_ring(format, HKV, HKV, DQK, DV, p);
    if (!fits && h > 0) fits = plan_ring(format, h, HKV, DQK, DV, p);
  }
  if (!fits) return false;
  // key slices: fill the resident CTAs in whole waves, 64 keys a slice at least
  const int resident = 148 * (p->smem <= 113 * 1024 && p->nw <= 8 ? 2 : 1);
  const long long ctas = (long long)rows * p->nhg;
  int best = 1;
  if (ctas < resident && max_keys > 128) {
    long long most = (max_keys + 63) / 64;
    if (most > kMaxSplit) most = kMaxSplit;
    double best_eff = -1.0;
    for (int n = 1; n <= (int)most; ++n) {
      const long long items = ctas * n, waves = (items + resident - 1) / resident;
      const double eff = (double)items / (double)(waves * resident);
      if (eff >= 0.95) {
        best = n;
        break;
      }
      if (eff > best_eff + 1e-9) {
        best_eff = eff;
        best = n;
      }
    }
  }
  p->nsplit = best;
  return true;
}

long long max_keys_of(const CacheAttnProblem& p) {
  const long long cap = (long long)p.cache.max_pages * p.cache.page_size;
  if (p.idx) return p.K;
  if (p.window > 0) {
    const long long n = (long long)p.window + p.n_first;
    return n < cap ? n : cap;
  }
  return cap;
}

template <int FMT, int DQK, int DV>
cudaError_t launch(const CacheAttnArgs& a, const Plan& p, int rows, cudaStream_t st) {
  auto kern = cache_attn_kernel<FMT, DQK, DV>;
  cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)p.smem);
  if (e != cudaSuccess) return e;
  const unsigned grid = (unsigned)rows * (unsigned)(p.nhg * p.nsplit);
  kern<<<grid, 32 * (p.nw + 1), p.smem, st>>>(a);
  return cudaGetLastError();
}

template <int FMT>
cudaError_t launch_dims(const CacheAttnArgs& a, const Plan& p, int rows, cudaStream_t st) {
  const int dqk = a.c.DQK, dv = a.c.DV;
  if (dqk == 64 && dv == 64) return launch<FMT, 64, 64>(a, p, rows, st);
  if (dqk == 64 && dv == 128) return launch<FMT, 64, 128>(a, p, rows, st);
  if (dqk == 128 && dv == 64) return launch<FMT, 128, 64>(a, p, rows, st);
  if (dqk == 128 && dv == 128) return launch<FMT, 128, 128>(a, p, rows, st);
  if (dqk == 192 && dv == 64) return launch<FMT, 192, 64>(a, p, rows, st);
  if (dqk == 192 && dv == 128) return launch<FMT, 192, 128>(a, p, rows, st);
  return cudaErrorNotSupported;
}

}  // namespace

bool cache_attn_supported(int format, int H, int HKV, int DQK, int DV) {
  Plan p;
  return make_plan(format, 1, H, HKV, DQK, DV, 1, &p);
}

size_t cache_attn_workspace_bytes(const CacheAttnProblem& p) {
  Plan pl;
  const int rows = p.B * p.S;
  if (!make_plan(p.cache.format, rows, p.H, p.cache.HKV, p.cache.DQK, p.cache.DV, max_keys_of(p),
                 &pl) ||
      pl.nsplit == 1)
    return 0;
  return (size_t)rows * pl.nsplit * p.H * (p.cache.DV + 2) * sizeof(float);
}

cudaError_t launch_cache_attn(const CacheAttnProblem& p, void* ws, size_t ws_bytes,
                              cudaStream_t st) {
  Plan pl;
  const int rows = p.B * p.S;
  if (!make_plan(p.cache.format, rows, p.H, p.cache.HKV, p.cache.DQK, p.cache.DV, max_keys_of(p),
                 &pl))
    return cudaErrorNotSupported;
  CacheAttnArgs a{};
  a.c = p.cache;
  a.q = static_cast<const __nv_bfloat16*>(p.q);
  a.pos = p.pos; a.idx = p.idx; a.K = p.K; a.window = p.window; a.n_first = p.n_first;
  a.gate = static_cast<const __nv_bfloat16*>(p.gate); a.gate_mode = p.gate_mode;
  a.out = static_cast<__nv_bfloat16*>(p.out);
  a.S = p.S; a.H = p.H; a.G = p.H / p.cache.HKV;
  a.qk_scale = p.sm_scale * kLog2e * p.cache.k_scale;
  a.nsplit = pl.nsplit; a.hc = pl.hc; a.nhg = pl.nhg; a.nsub = pl.nsub; a.kw = pl.kw;
  a.nstages = pl.nstages; a.pitch = pl.pitch;
  if (pl.nsplit > 1) {
    const size_t need = (size_t)rows * pl.nsplit * p.H * (p.cache.DV + 2) * sizeof(float);
    if (ws == nullptr || ws_bytes < need) return cudaErrorInvalidValue;
    a.part_o = static_cast<float*>(ws);
    a.part_ml = a.part_o + (size_t)rows * pl.nsplit * p.H * p.cache.DV;
  }
  cudaError_t e = p.cache.format == 0 ? launch_dims<0>(a, pl, rows, st)
                                      : launch_dims<1>(a, pl, rows, st);
  if (e != cudaSuccess || pl.nsplit == 1) return e;
  return launch_split_combine(1, a.part_o, a.part_ml, rows, pl.nsplit, p.H, p.cache.DV, p.gate,
                              p.gate_mode, p.out, st);
}

}  // namespace dsa
