// Attention of single query tokens over cache rows held in 4 bits.  The formula and the split over
// CTAs are those of cache_attn.cu; a warp takes one KV head (8 of its query heads as the 8 columns
// of both products) and every kw-th group of 16 keys of the CTA's slice.
//
// What bounds it: 9/16 byte a value, so at 6.5 TB/s 41 values arrive per clock and SM, and each has
// to be widened to f16 before the tensor cores take it.  Widening costs about 22 instructions per
// 256 values (16 bytes of codes a thread become 16 f16 pairs by 16 conversions and 16 products
// with the group's scale), so the issue slots are as scarce as the bandwidth, and everything else
// is kept short.  Each warp works alone: it copies its own head's part of 16 keys at a time into
// its own ring (cp.async, 16 bytes a lane, two steps ahead), so there is no barrier and no producer
// in the loop.  A thread takes 16 consecutive dims of a key (the contraction order is free): 8
// bytes of codes and one scale.  The V operand needs two keys in a register: the nibbles of two
// keys are interleaved before the conversion, which makes pairs of nibbles.
//
// Widening is exact: an e2m1 value times an e4m3 scale has 6 significant bits and stays in f16's
// normal range.  Queries become f16 after a scaling of each head by a power of two (its largest
// element to [2^13, 2^14)): exact for every element within 2^-30 of the largest (8 bits into 11),
// and off by 2^-38 of it at most otherwise.  Probabilities are f16 with the running maximum at 2^6
// (so terms down to 2^-30 of the largest stay): half a step is 2^-11 each, below the rounding of
// the output.
#include <cuda_fp16.h>

#include "cache_attn.cuh"

namespace dsa {

namespace {

constexpr int kAhead = 2;           // steps of 16 keys copied ahead
constexpr int kStages = kAhead + 1;

// A key in a warp's ring: K codes, V codes, then the pieces of 16 bytes that hold the K scales and
// the V scales (4, 8 or 12 bytes anywhere in one or two pieces).
template <int DQK, int DV>
struct Slot {
  static constexpr int V = DQK / 2, KS = V + DV / 2, VS = KS + 32;
  static constexpr int PIECES = (VS + 32) / 16;
  // lanes that copy one key, and keys that a warp copies at once
  static constexpr int LANES = PIECES <= 8 ? 8 : 16, KEYS = 32 / LANES;
  static_assert(PIECES <= LANES, "one piece per lane");
  // 32 or 96 bytes past a multiple of 128: no bank conflicts (kappa)
  static constexpr int PITCH = (VS + 32 - 32 + 63) / 64 * 64 + 32;
  static constexpr int STEP = 16 * PITCH;  // a step of 16 keys
};

// Asynchronous 16-byte copy to shared memory; a group of them; all but the last N groups landed.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// N words of a slot (aligned to 4N bytes), by their shared-memory address; a byte of one.
__device__ __forceinline__ void load_words(uint32_t at, uint32_t (&w)[1]) {
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(at));
}
__device__ __forceinline__ void load_words(uint32_t at, uint32_t (&w)[2]) {
  asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(at));
}
__device__ __forceinline__ void load_words4(uint32_t at, uint32_t& a, uint32_t& b, uint32_t& c,
                                            uint32_t& d) {
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(a), "=r"(b), "=r"(c), "=r"(d)
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ uint32_t load_byte(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(at));
  return v;
}

// Row m of the 16-row operands is key kappa(m) of the group (m and m + 8 alike): with rows 32 or 96
// bytes past a multiple of 128 apart, the K loads (rows g = 0..3 and 4..7 of a half warp) and the V
// loads (rows 2t, or 2t + 1) both touch four different groups of 8 banks.
__device__ __forceinline__ int kappa(int g) { return g ^ ((g >> 2) & 1); }

template <int DQK, int DV>
__global__ void __launch_bounds__(32 * kQ4Warps, 2) cache_attn_q4_kernel(const CacheAttnArgs a) {
  using S = Slot<DQK, DV>;
  constexpr int QC = DQK / 64;       // 64-dim chunks: 16 dims per thread each
  constexpr int MT = DV / 16;        // 16-row tiles of O^T
  constexpr int VPT = DV / 8;        // value dims per thread row
  constexpr int TOP = 6;
  extern __shared__ __align__(128) uint8_t smem[];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t4 = lane & 3;
  const int nhw = a.hc * a.nsub;
  const int split = blockIdx.x % a.nsplit;
  const int hg = (blockIdx.x / a.nsplit) % a.nhg;
  const int row = blockIdx.x / (a.nsplit * a.nhg);
  const int32_t* table = a.c.table + (size_t)(row / a.S) * a.c.max_pages;
  const int kv0 = hg * a.hc;
  const int kg = warp / nhw, hw = warp % nhw;
  const int kv = kv0 + hw / a.nsub, sub = hw % a.nsub;
  const int ncol = min(8, a.G - sub * 8);  // query heads in the 8 columns
  const int h0 = kv * a.G + sub * 8;

  const int pos = __ldg(a.pos + row);
  const KeyList list = key_list(a, row, pos);
  int j0, j1;
  key_slice(list, a.nsplit, split, &j0, &j1);
  // this warp's steps of 16 keys: every kw-th, from kg.  Steps come in pairs: lane l looks after key
  // l & 15 of step l >> 4 of a pair, reads it two pairs ahead and looks its row up one ahead.
  const int steps = (((j1 - j0 + 15) >> 4) - kg + a.kw - 1) / a.kw;
  const int my_j = j0 + 16 * (kg + a.kw * (lane >> 4)) + (lane & 15);
  auto read_key = [&](int pair) {  // (below j1 + 2^10: no overflow)
    const int e = my_j + 32 * a.kw * pair;
    return e < j1 ? list.at(e) : -1;
  };
  auto look_up = [&](int t) { return t <= pos ? cache_row(a.c, table, t) : -1; };
  int rn = look_up(read_key(0)), tn = read_key(1);

  // ---- copies: lane = piece `at` of key `at_key` (of KEYS) in row 0 and in the step's first slots
  const int at_key = lane / S::LANES, at = lane % S::LANES;
  const int ks0 = cache_ks_off(a.c.HKV, DQK, DV) + kv * (DQK / 16);  // this head's scales
  const int vs0 = cache_vs_off(a.c.HKV, DQK, DV) + kv * (DV / 16);
  int piece = 16 * at;
  bool has_piece = true;
  if (piece < S::V) {
    piece += kv * (DQK / 2);
  } else if (piece < S::KS) {
    piece += cache_v_off(1, a.c.HKV, DQK) + kv * (DV / 2) - S::V;
  } else if (piece < S::VS) {
    piece += (ks0 & ~15) - S::KS;
    has_piece = piece < ks0 + DQK / 16;
  } else {
    piece += (vs0 & ~15) - S::VS;
    has_piece = at < S::PIECES && piece < vs0 + DV / 16;
  }
  const uint8_t* from = a.c.pages + (has_piece ? piece : 0);
  const uint32_t row_bytes = (uint32_t)a.c.row_bytes;
  const uint32_t ring = smem_u32(smem) + warp * (kStages * S::STEP);
  const uint32_t fill_at = ring + at_key * S::PITCH + 16 * at;
  // A pair's rows, as a thread needs them: its keys at_key, at_key + KEYS, ... of a step in a row of
  // `rows` (key 0 of the pair in its word 0); a key without a row reads row 0.
  uint32_t* rows = reinterpret_cast<uint32_t*>(smem + kQ4Warps * kStages * S::STEP) + 32 * warp;
  const int my_word = (lane & 16) + (lane & (S::KEYS - 1)) * (16 / S::KEYS) + (lane & 15) / S::KEYS;
  const uint32_t rows_at = smem_u32(rows) + at_key * (4 * 16 / S::KEYS);
  auto fill = [&](uint32_t stage, int half) {
    uint32_t rk[16 / S::KEYS];
#pragma unroll
    for (int i = 0; i < 16 / S::KEYS; i += 4)
      load_words4(rows_at + 64 * half + 4 * i, rk[i], rk[i + 1], rk[i + 2], rk[i + 3]);
    if (has_piece) {
#pragma unroll
      for (int i = 0; i < 16 / S::KEYS; ++i)
        cp_async16(fill_at + stage + i * S::KEYS * S::PITCH,
                   from + (unsigned long long)rk[i] * row_bytes);
    }
  };

  // ---- Q^T fragments, column g: dims 64c + 16t .. + 15 of the head
  uint32_t qf[QC][8];
  float cs[2];  // score scale of columns 2t, 2t + 1
  {
    const bool has = g < ncol;
    const uint4* qp = reinterpret_cast<const uint4*>(
        a.q + ((size_t)row * a.H + (has ? h0 + g : 0)) * DQK + 16 * t4);
    uint32_t top = 0;  // the largest exponent field of |q|
#pragma unroll
    for (int c = 0; c < QC; ++c)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint4 x = has ? __ldg(qp + c * 8 + i) : make_uint4(0, 0, 0, 0);
        qf[c][4 * i + 0] = x.x; qf[c][4 * i + 1] = x.y;
        qf[c][4 * i + 2] = x.z; qf[c][4 * i + 3] = x.w;
      }
#pragma unroll
    for (int c = 0; c < QC; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        top = max(top, max((qf[c][i] << 16) & 0x7f800000u, qf[c][i] & 0x7f800000u));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const int ex = max((int)(top >> 23) - 127, -100);  // 2^ex <= max|q| (or less)
    const float up = __int_as_float((13 - ex + 127) << 23);
    const float scale = a.qk_scale * __int_as_float((ex - 13 + 127) << 23);
#pragma unroll
    for (int c = 0; c < QC; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const __half2 h = __floats2half2_rn(__uint_as_float(qf[c][i] << 16) * up,
                                            __uint_as_float(qf[c][i] & 0xffff0000u) * up);
        qf[c][i] = *reinterpret_cast<const uint32_t*>(&h);
      }
    cs[0] = __shfl_sync(0xffffffffu, scale, (2 * t4) * 4);
    cs[1] = __shfl_sync(0xffffffffu, scale, (2 * t4 + 1) * 4);
  }

  float o[MT][4];
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[i][e] = 0.f;

  // ---- main loop
  const int ka = kappa(g), k0 = kappa(2 * t4), k1 = kappa(2 * t4 + 1);
  // this thread's places in a step: key ka's codes and scales, keys k0's and k1's values
  const uint32_t k_at = ring + ka * S::PITCH + t4 * 8;
  const uint32_t ks_at = ring + ka * S::PITCH + S::KS + (ks0 & 15) + t4;
  const uint32_t v_at0 = ring + k0 * S::PITCH + S::V + g * (VPT / 2);
  const uint32_t v_at1 = ring + k1 * S::PITCH + S::V + g * (VPT / 2);
  const uint32_t vs_off = S::VS - S::V + (vs0 & 15) + (g * VPT) / 16 - g * (VPT / 2);
  // one step: the 16 keys in slots `base` .., of which `mask` have a row
  auto step = [&](uint32_t base, uint32_t mask) {
    // S^T = K Q^T, two accumulators
    float s[2][4];
    const uint32_t ra = k_at + base, rb = ra + 8 * S::PITCH;
    const uint32_t rsa = ks_at + base, rsb = rsa + 8 * S::PITCH;
#pragma unroll
    for (int c = 0; c < QC; ++c) {
      uint32_t wa[2], wb[2];
      load_words(ra + c * 32, wa);
      load_words(rb + c * 32, wb);
      const uint32_t sa = e4m3x2_to_f16(load_byte(rsa + c * 4) * 0x0101u);
      const uint32_t sb = e4m3x2_to_f16(load_byte(rsb + c * 4) * 0x0101u);
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        uint32_t xa[4], xb[4];
        e2m1x8_to_f16(wa[hf], xa);
        e2m1x8_to_f16(wb[hf], xb);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t f[4] = {mul_f16x2(xa[2 * i], sa), mul_f16x2(xb[2 * i], sb),
                                 mul_f16x2(xa[2 * i + 1], sa), mul_f16x2(xb[2 * i + 1], sb)};
          if (c == 0 && hf == 0)
            mma_f16_zero(s[i], f, qf[c][4 * hf + 2 * i], qf[c][4 * hf + 2 * i + 1]);
          else
            mma_f16(s[i], f, qf[c][4 * hf + 2 * i], qf[c][4 * hf + 2 * i + 1]);
        }
      }
    }
    // this thread's values, on their way while the softmax runs
    const uint32_t v0 = v_at0 + base, v1 = v_at1 + base, v2 = v0 + 8 * S::PITCH,
                   v3 = v1 + 8 * S::PITCH;
    uint32_t vw[4][VPT / 8];
    load_words(v0, vw[0]);
    load_words(v1, vw[1]);
    load_words(v2, vw[2]);
    load_words(v3, vw[3]);
    uint32_t sc0 = load_byte(v0 + vs_off) | (load_byte(v1 + vs_off) << 8);
    uint32_t sc1 = load_byte(v2 + vs_off) | (load_byte(v3 + vs_off) << 8);

    float x[4] = {(s[0][0] + s[1][0]) * cs[0], (s[0][1] + s[1][1]) * cs[1],
                  (s[0][2] + s[1][2]) * cs[0], (s[0][3] + s[1][3]) * cs[1]};
    if (mask != 0xffffu) {  // row 0 stands in for a missing key: its scale may be NaN
      if (!((mask >> ka) & 1u)) x[0] = x[1] = -INFINITY;
      if (!((mask >> (ka + 8)) & 1u)) x[2] = x[3] = -INFINITY;
      sc0 &= (((mask >> k0) & 1u) * 0xffu) | (((mask >> k1) & 1u) * 0xff00u);
      sc1 &= (((mask >> (k0 + 8)) & 1u) * 0xffu) | (((mask >> (k1 + 8)) & 1u) * 0xff00u);
    }
    float p[4];
    softmax_step<TOP, MT>(x, m, l, o, p);
    const __half2 p01 = __floats2half2_rn(p[0], p[1]), p23 = __floats2half2_rn(p[2], p[3]);
    const uint32_t b0 = transpose8x8(*reinterpret_cast<const uint32_t*>(&p01));
    const uint32_t b1 = transpose8x8(*reinterpret_cast<const uint32_t*>(&p23));
    const uint32_t s01 = e4m3x2_to_f16(sc0), s23 = e4m3x2_to_f16(sc1);
    // O^T += V^T P^T
#pragma unroll
    for (int w = 0; w < VPT / 8; ++w) {
      constexpr uint32_t kLo = 0x0f0f0f0fu;
      uint32_t e01[4], o01[4], e23[4], o23[4];  // even and odd dims, two keys each
      e2m1x8_to_f16((vw[0][w] & kLo) | ((vw[1][w] << 4) & ~kLo), e01);
      e2m1x8_to_f16(((vw[0][w] >> 4) & kLo) | (vw[1][w] & ~kLo), o01);
      e2m1x8_to_f16((vw[2][w] & kLo) | ((vw[3][w] << 4) & ~kLo), e23);
      e2m1x8_to_f16(((vw[2][w] >> 4) & kLo) | (vw[3][w] & ~kLo), o23);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t f[4] = {mul_f16x2(e01[i], s01), mul_f16x2(o01[i], s01),
                               mul_f16x2(e23[i], s23), mul_f16x2(o23[i], s23)};
        mma_f16(o[4 * w + i], f, b0, b1);
      }
    }
  };

  static_assert(kAhead == 2, "a pair of steps is copied while the pair before is worked on");
  uint32_t masks, masks_n = __ballot_sync(0xffffffffu, rn >= 0);  // keys with a row, of a pair
  rows[my_word] = max(rn, 0);
  rn = look_up(tn);
  tn = read_key(2);
  __syncwarp();
  fill(0, 0);
  cp_async_commit();
  fill(S::STEP, 1);
  cp_async_commit();
  uint32_t at_step = 0;                   // the slots of the step worked on,
  uint32_t at_fill = kAhead * S::STEP;    // and of the step copied
  auto advance = [](uint32_t x) { return x == kAhead * S::STEP ? 0u : x + S::STEP; };
  for (int n = 0; n < steps; n += 2) {
    __syncwarp();  // the rows of the pair before have been read
    masks = masks_n;
    masks_n = __ballot_sync(0xffffffffu, rn >= 0);
    rows[my_word] = max(rn, 0);
    rn = look_up(tn);
    tn = read_key((n >> 1) + 3);
    __syncwarp();
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      if (masks_n != 0u) fill(at_fill, half);
      cp_async_commit();
      cp_async_wait<kAhead>();  // this step's copies have landed
      __syncwarp();
      const uint32_t mask = half ? masks >> 16 : masks & 0xffffu;
      if (mask != 0u) step(at_step, mask);
      __syncwarp();  // its slots may be filled again
      at_step = advance(at_step);
      at_fill = advance(at_fill);
    }
  }
  cp_async_wait<0>();  // copies in flight land before the ring is used again

  // this warp's (m, l, O) for the merge
#pragma unroll
  for (int d = 4; d < 32; d <<= 1) {
    l[0] += __shfl_xor_sync(0xffffffffu, l[0], d);
    l[1] += __shfl_xor_sync(0xffffffffu, l[1], d);
  }
  __syncthreads();
  float* ml = reinterpret_cast<float*>(smem);    // [warp][8][2]
  float* ob = ml + kQ4Warps * 16;                // [warp][8][DV]
  if (g == 0)
    *reinterpret_cast<float4*>(ml + warp * 16 + 4 * t4) = make_float4(m[0], l[0], m[1], l[1]);
  float* c0 = ob + (size_t)(warp * 8 + 2 * t4) * DV + g * VPT;
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    *reinterpret_cast<float2*>(c0 + 2 * i) = make_float2(o[i][0], o[i][2]);
    *reinterpret_cast<float2*>(c0 + DV + 2 * i) = make_float2(o[i][1], o[i][3]);
  }
  __syncthreads();
  merge_groups<DV>(a, ml, ob, nhw, row, split, kv0);
}

template <int DQK, int DV>
cudaError_t launch(const CacheAttnArgs& a, unsigned grid, cudaStream_t st) {
  const int nw = a.hc * a.nsub * a.kw;
  constexpr size_t ring = (size_t)kQ4Warps * kStages * Slot<DQK, DV>::STEP;
  constexpr size_t merge = (size_t)kQ4Warps * (16 + 8 * DV) * sizeof(float);
  constexpr size_t rows = kQ4Warps * 32 * sizeof(uint32_t);
  constexpr size_t smem = ring + rows > merge ? ring + rows : merge;
  static_assert(smem <= 112 * 1024, "two CTAs per SM");
  auto kern = cache_attn_q4_kernel<DQK, DV>;
  cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  // all of the SM's shared memory, or a second CTA would find too little of it
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout,
                             cudaSharedmemCarveoutMaxShared);
  if (e != cudaSuccess) return e;
  kern<<<grid, 32 * nw, smem, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_attn_q4(const CacheAttnArgs& a, unsigned grid, cudaStream_t st) {
  const int dqk = a.c.DQK, dv = a.c.DV;
  if (dqk == 64 && dv == 64) return launch<64, 64>(a, grid, st);
  if (dqk == 64 && dv == 128) return launch<64, 128>(a, grid, st);
  if (dqk == 128 && dv == 64) return launch<128, 64>(a, grid, st);
  if (dqk == 128 && dv == 128) return launch<128, 128>(a, grid, st);
  if (dqk == 192 && dv == 64) return launch<192, 64>(a, grid, st);
  if (dqk == 192 && dv == 128) return launch<192, 128>(a, grid, st);
  return cudaErrorNotSupported;
}

}  // namespace dsa
