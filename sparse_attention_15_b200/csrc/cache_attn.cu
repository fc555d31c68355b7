// Attention of single query tokens over the paged key/value cache (bf16 rows, or rows held in 4
// bits), with a sliding window and visible first tokens, over whole contexts, or over selected
// keys; the headwise gate fused.
//
//   o[h,:] = sum_t p_t v[t,h/G,:],  p = softmax_t(sm_scale * q[h,:] . k[t,h/G,:]),  G = H/HKV
//
// over the query's keys: idx[b,s,:], or t <= pos with t > pos - window or t < n_first.  Every
// query token has its own key list, so masked keys are never looked at and what they hold (NaN, a
// page of another sequence, nothing yet) does not matter.
//
// Products.  Both run on mma.sync m16n8k16 with the cache as the 16-row operand and the up to 8
// query heads of a KV head as the 8 columns: S^T = K Q^T [16 keys x 8 heads], O^T += V^T P^T
// [dims x 8 heads], float32 accumulation.  (A tcgen05 tile wants 128 rows that share an operand;
// here 1 to 8 do, and 4-bit rows have to be widened on their way into the product.)  The
// contraction order over the dims is free, so a thread takes 16 consecutive dims of a key.
//
// Work.  The (query token, group of KV heads) rows, laid end to end in steps of 16 keys, are cut
// into equal pieces, one per resident CTA, whatever their lengths; a row in several pieces is
// merged by a second kernel, in order.  Inside a CTA (of 4 warps for 4 bits, so that four fit an SM
// and fewer wait for one) each warp works alone on one KV head (8 of its query heads): it copies its
// own head's part of 16 keys at a time into its own ring (cp.async, 16 bytes a lane, a step or two
// ahead), so the loop has no barrier and no producer.
//
// What bounds the 4-bit form: latency, with neither limit reached (64 x 2048 keys: issue slots 62%
// used, DRAM 50%).  A step (16 keys of a head, 5120 values of 9/16 byte) takes 450 instructions, the
// pieces' starts and ends counted in: 160 widen (a conversion and a product with the group's scale for
// each f16 pair, 8 per 256 values), 20 are MMAs, 85 copy and look up, the rest are the softmax, the
// masks, addresses and the probabilities' pairs.  At 6.5 TB/s 41 values arrive per clock and SM, which
// would take 3.6 of its 4 issue slots; four warps a scheduler do not cover the widening's chains well
// enough for that (stalls per issue: fixed latencies 1.6, busy half-rate pipes 0.7).  So everything
// else is kept short.  The V operand needs two keys in a register: the nibbles of two keys are interleaved
// before the conversion, which makes pairs of nibbles.  Widening is exact: an e2m1 value times an
// e4m3 scale has 6 significant bits and stays in f16's normal range.  Queries become f16 after a
// scaling of each head by a power of two (its largest element to [2^13, 2^14)): exact for every
// element within 2^-30 of the largest (8 bits into 11), and off by 2^-38 of it at most otherwise.
// Probabilities are f16 pairs hi + lo with the running maximum at 2^6 (so terms down to 2^-30 of the
// largest stay): 22 bits, as one f16's 11 would show wherever the values cancel.  Warps of up to 4
// query heads have them twice, in the columns 0..3 and 4..7, and the second four take lo: the pair
// costs no product (64 x 2048 keys: 206 us, one f16 201 us, two products 219 us).  Warps of 5 to 8
// heads take two products, as bf16 rows do.
//
// Measured, a call among others: 64 x 2048 selected keys of 32 heads (755 MB) in 199-211 us, 3.7 TB/s;
// eight contexts of up to 131072 tokens and 8 heads (1.13 GB) in 282-333 us (by the machine and
// where the pages lie), 3.4-4.0 TB/s.  (The figures of the layouts below, taken in a graph on one set of pages, compare with
// 250-260 us there.)
//
// bf16 rows are bound by the bandwidth (16 x 2048 keys of 32 heads, 671 MB: 122-128 us, 5.4 TB/s).  They
// are used as they are; probabilities are a bf16 pair, as one bf16 would be no more exact than the
// output.
#include <cuda_fp16.h>

#include <atomic>
#include <type_traits>

#include "cache.cuh"
#include "kernels.h"

namespace dsa {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kWarps = 8;         // most warps of a CTA

struct CacheAttnArgs {
  CacheView c;
  const __nv_bfloat16* q;  // [B,S,H,DQK]
  const int32_t* pos;      // [B,S]
  const int32_t* idx;      // [B,S,K] or NULL
  const __nv_bfloat16* gate;
  __nv_bfloat16* out;      // [B,S,H,DV]
  float* part_o;           // [piece, heads of a CTA, DV] (pieces)
  float* part_ml;          // [piece, heads of a CTA, 2]
  int gate_mode, S, H, G, K, window, n_first;
  float qk_scale;          // sm_scale * log2(e)
  int rows, hc, nhg;       // query tokens, KV heads per CTA, CTAs per token and step
  int nsub, kw;            // warps per KV head (8 query heads each), 16-key groups side by side
  int grid;                // CTAs that share the steps in pieces; 0: one CTA per token and group
  int least_log;           // log2 of the steps of the least piece
};

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

__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

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
__device__ __forceinline__ void load_words(uint32_t at, uint32_t (&w)[4]) {
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ uint32_t load_byte(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(at));
  return v;
}

// 4 bits: row m of the 16-row operands is key kappa(m) of the step (m and m + 8 alike).  With rows
// 32 or 96 bytes past a multiple of 128 apart, the K loads (rows g = 0..3 and 4..7 of a half warp)
// and the V loads (rows 2t, or 2t + 1) both touch four different groups of 8 banks.
__device__ __forceinline__ int kappa(int g) { return g ^ ((g >> 2) & 1); }

// A key in a warp's ring, and how its pieces of 16 bytes are copied: lane l takes pieces l, l + 32,
// ... of CYCLE keys' pieces laid end to end, in ROUNDS rounds.
template <int FMT, int DQK, int DV>
struct Slot;
// bf16: K, V.  Rows 16 bytes past a multiple of 128 apart: no bank conflicts.
template <int DQK, int DV>
struct Slot<0, DQK, DV> {
  static constexpr int V = DQK * 2, PIECES = (DQK + DV) / 8;
  static constexpr int CYCLE = PIECES == 16 ? 2 : PIECES == 32 ? 1 : 4;
  static constexpr int PITCH = (DQK + DV) * 2 + 16;
};
// 4 bits: K codes, V codes, then the pieces that hold the K scales and the V scales (4, 8 or 12
// bytes anywhere in one or two pieces); lanes past the pieces idle.
template <int DQK, int DV>
struct Slot<1, DQK, DV> {
  static constexpr int V = DQK / 2, KS = V + DV / 2, VS = KS + 32;
  static constexpr int PIECES = (VS + 32) / 16 <= 8 ? 8 : 16;
  static constexpr int CYCLE = 32 / PIECES;
  static constexpr int PITCH = (VS + 63) / 64 * 64 + 32;
  static_assert((VS + 32) / 16 <= 16 && PITCH >= VS + 32, "a key's pieces");
};
template <int FMT, int DQK, int DV>
struct Ring {
  using S = Slot<FMT, DQK, DV>;
  static constexpr int STEP = 16 * S::PITCH;  // a step of 16 keys
  static constexpr int ROUNDS = S::CYCLE * S::PIECES / 32;
  static constexpr int ROWS = kWarps * 64 * 4;  // a warp's rows of two pairs of steps
  static constexpr int fits(int stages, int warps) { return ROWS + warps * stages * STEP; }
  // Warps that a CTA should have, and steps in a warp's ring (one worked on).  4 bits: 4 warps, four
  // CTAs per SM (eight contexts: 254 us; 8 warps: 262; 2 warps: 290).  bf16: two CTAs per SM, of 8
  // warps if that leaves two steps or more, else of 4 (64 windows: 44 us; 2 warps: 55).  (An SM has
  // 228 KB, 1 KB of them for each CTA's own use.)
  static constexpr int HALF = 113 * 1024, WHOLE = 226 * 1024;
  static constexpr int WARPS = FMT == 1 ? 4 : fits(2, 8) <= HALF ? 8 : 4;
  static constexpr int STAGES = fits(3, WARPS) <= HALF ? 3 : 2;
  static constexpr int smem(int warps) {
    const int merge = warps * (16 + 8 * DV) * 4;
    return fits(STAGES, warps) > merge ? fits(STAGES, warps) : merge;
  }
  static_assert(smem(WARPS) <= HALF && smem(kWarps) <= WHOLE && S::CYCLE * S::PIECES % 32 == 0,
                "ring");
};

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
// Its steps of kw groups of 16 keys.
__device__ __forceinline__ int row_steps(const CacheAttnArgs& a, int row) {
  const int n = key_list(a, row, __ldg(a.pos + row)).n;
  return (n + 16 * a.kw - 1) / (16 * a.kw);
}

// Pieces.  The steps of all rows (query tokens), once for each group of heads, are numbered end to
// end, `each` for a group; share c of g has numbers [c * all / g, (c + 1) * all / g).  Piece numbers
// grow by one with each CTA and with each row: row r of group hg in share c is piece c + hg * R + r.
__device__ __forceinline__ int ctas_of(const CacheAttnArgs& a, long long all) {
  const long long most = all >> a.least_log;
  return (int)(most < 1 ? 1 : most < a.grid ? most : a.grid);
}
// a / b for a >= 0, b > 0: by a 32-bit division (a fifth of the time) where both fit, as they nearly
// always do.
__device__ __forceinline__ long long quotient(long long a, long long b) {
  if (((unsigned long long)(a | b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
  return a / b;
}
// The share that has step number s.
__device__ __forceinline__ int cta_of(long long s, long long all, int g) {
  return (int)quotient((s + 1) * g - 1, all);
}

// Sum over the block of `mine`, and of the threads before this one (blockDim <= 1024).
__device__ __forceinline__ long long block_scan(long long mine, long long* warp_sums,
                                                long long* before) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  long long x = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  long long base = 0, total = 0;
  for (int w = 0; w < nw; ++w) {
    if (w < warp) base += warp_sums[w];
    total += warp_sums[w];
  }
  __syncthreads();
  *before = base + x - mine;
  return total;
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

// Two float32 values in f16; with `rest`, what their f16 values `h` leave of them.
__device__ __forceinline__ __half2 without(const float* p, __half2 h, bool rest) {
  uint32_t w = *reinterpret_cast<const uint32_t*>(&h);
  w &= rest ? 0xffffffffu : 0u;
  h = *reinterpret_cast<const __half2*>(&w);
  return __floats2half2_rn(p[0] - __low2float(h), p[1] - __high2float(h));
}

// FEW (4 bits): at most 4 query heads to a warp, which the columns 4..7 hold a second time for the
// lo halves of the probabilities.
template <int FMT, int DQK, int DV, bool FEW>
__global__ void __launch_bounds__(32 * kWarps, (FMT == 1 || Ring<FMT, DQK, DV>::WARPS == 8 ? 2 : 1))
    cache_attn_kernel(const CacheAttnArgs a) {
  using S = Slot<FMT, DQK, DV>;
  using R = Ring<FMT, DQK, DV>;
  constexpr int QC = DQK / 64;       // 64-dim chunks: 16 dims per thread each
  constexpr int MT = DV / 16;        // 16-row tiles of O^T
  constexpr int VPT = DV / 8;        // 4 bits: value dims per thread row
  constexpr int TOP = FMT == 1 ? 6 : 0;
  constexpr int AHEAD = R::STAGES - 1;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ long long warp_sums[kWarps];
  __shared__ int first_row, first_step;
  __shared__ uint32_t first_piece;  // the share's number: of its piece of row 0 in group 0

  // the merge kernel may start: it waits for this grid's end before it reads the pieces
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t4 = lane & 3;
  const int nhw = a.hc * a.nsub;
  const int kg = warp / nhw, hw = warp % nhw;
  const int sub = hw % a.nsub;
  const int ncol = min(8, a.G - sub * 8);  // query heads in the 8 columns

  // ---- this CTA's steps
  int row, hg, u0;      // the row, head group and step it starts with
  long long left;       // its steps
  if (a.grid == 0) {
    row = blockIdx.x / a.nhg;
    hg = blockIdx.x % a.nhg;
    u0 = 0;
    left = row_steps(a, row);
    if (left == 0) left = 1;  // a row without keys gets its zeros from an empty step
  } else {
    const int per = (a.rows + blockDim.x - 1) / blockDim.x;
    const int r0 = min((int)threadIdx.x * per, a.rows), r1 = min(r0 + per, a.rows);
    long long mine = 0, before;
    for (int i = r0; i < r1; ++i) mine += row_steps(a, i);
    const long long each = block_scan(mine, warp_sums, &before);
    const long long all = each * a.nhg;
    const int ctas = ctas_of(a, all);
    // with groups of heads along x, neighbours read the same keys (make_plan says when)
    const uint32_t share = blockIdx.x * gridDim.y + blockIdx.y;
    if ((int)share >= ctas || all == 0) return;
    const long long begin = quotient(share * all, ctas);
    left = quotient((share + 1) * all, ctas) - begin;
    if (threadIdx.x == 0) first_piece = share;
    hg = (int)quotient(begin, each);
    const long long in = begin - hg * each;
    if (before <= in && in < before + mine) {
      long long s = in - before;
      int i = r0;
      for (int n; s >= (n = row_steps(a, i)); ++i) s -= n;
      first_row = i;
      first_step = (int)s;
    }
    __syncthreads();
    row = first_row;
    u0 = first_step;
  }

  const uint32_t ring = smem_u32(smem) + R::ROWS + warp * (R::STAGES * R::STEP);
  uint32_t* rows = reinterpret_cast<uint32_t*>(smem) + 64 * warp;
  const uint32_t row_bytes = (uint32_t)a.c.row_bytes;
  // this lane's pieces of a cycle of keys: the first round's in key cy0, the next rounds' 32 further
  int cy[R::ROUNDS], at[R::ROUNDS];
#pragma unroll
  for (int x = 0; x < R::ROUNDS; ++x) {
    cy[x] = (lane + 32 * x) / S::PIECES;
    at[x] = 16 * ((lane + 32 * x) % S::PIECES);
  }

  for (; left > 0; u0 = 0, hg += row + 1 == a.rows, row = row + 1 == a.rows ? 0 : row + 1) {
    const int pos = __ldg(a.pos + row);
    const KeyList list = key_list(a, row, pos);
    const int n_steps = (list.n + 16 * a.kw - 1) / (16 * a.kw);
    if (a.grid > 0 && n_steps == 0) continue;
    const int u1 = (int)min((long long)n_steps, u0 + left);
    left -= a.grid > 0 ? u1 - u0 : left;
    const bool alone = u0 == 0 && u1 == n_steps;  // the row's only piece
    const int j0 = u0 * 16 * a.kw, j1 = min(list.n, u1 * 16 * a.kw);
    const int kv = hg * a.hc + hw / a.nsub;
    const int h0 = kv * a.G + sub * 8;
    const int32_t* table = a.c.table + (size_t)(row / a.S) * a.c.max_pages;

    // ---- keys and rows.  This warp's groups of 16 keys, one per step, come in pairs: lane l looks
    // after key l & 15 of step l >> 4 of a pair, reads it two pairs ahead and looks its row up one
    // ahead.
    const int steps = u1 - u0;
    const int my_j = j0 + 16 * (kg + a.kw * (lane >> 4)) + (lane & 15);
    auto read_key = [&](int pair) {  // (below j1 + 2^11: no overflow)
      const int e = my_j + 32 * a.kw * pair;
      return e < j1 ? list.at(e) : -1;
    };
    auto look_up = [&](int t) { return t <= pos ? cache_row(a.c, table, t) : -1; };
    int rn = look_up(read_key(0)), tn = read_key(1);

    // ---- copies: where this lane's pieces lie in row 0
    const int ks0 = cache_ks_off(a.c.HKV, DQK, DV) + kv * (DQK / 16);  // 4 bits: the head's scales
    const int vs0 = cache_vs_off(a.c.HKV, DQK, DV) + kv * (DV / 16);
    const uint8_t* from[R::ROUNDS];
    bool has_piece = true;
#pragma unroll
    for (int x = 0; x < R::ROUNDS; ++x) {
      int piece = at[x];
      if constexpr (FMT == 0) {
        piece += piece < S::V ? kv * (DQK * 2)
                              : cache_v_off(0, a.c.HKV, DQK) + kv * (DV * 2) - S::V;
      } else if (piece < S::V) {
        piece += kv * (DQK / 2);
      } else if (piece < S::KS) {
        piece += cache_v_off(1, a.c.HKV, DQK) + kv * (DV / 2) - S::V;
      } else if (piece < S::VS) {
        piece += (ks0 & ~15) - S::KS;
        has_piece = piece < ks0 + DQK / 16;
      } else {
        piece += (vs0 & ~15) - S::VS;
        has_piece = at[x] < S::VS + 32 && piece < vs0 + DV / 16;
      }
      from[x] = a.c.pages + (has_piece ? piece : 0);
    }
    // A pair's rows in `rows` (two pairs in turn), a step's keys in the order that its copies take
    // them: key k of the step is word (k % CYCLE) * (16 / CYCLE) + k / CYCLE of its 16.  A key
    // without a row reads row 0.
    constexpr int PER = 16 / S::CYCLE;
    const int my_word = (lane & 16) + (lane & 15) % S::CYCLE * PER + (lane & 15) / S::CYCLE;
    auto fill = [&](uint32_t stage, int pair_half) {
#pragma unroll
      for (int x = 0; x < R::ROUNDS; ++x) {
        const uint32_t dst = ring + stage + cy[x] * S::PITCH + at[x];
        const uint32_t rows_at = smem_u32(rows) + pair_half * 64 + cy[x] * (PER * 4);
#pragma unroll
        for (int i = 0; i < PER; i += 4) {
          uint32_t rk[4];
          load_words(rows_at + 4 * i, rk);
          if (has_piece) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              cp_async16(dst + (i + k) * S::CYCLE * S::PITCH,
                         from[x] + (unsigned long long)rk[k] * row_bytes);
          }
        }
      }
    };

    // ---- the first steps' copies, on their way while the queries are read
    uint32_t masks, masks_n = __ballot_sync(0xffffffffu, rn >= 0);  // keys with a row, of a pair
    rows[my_word] = max(rn, 0);
    rn = look_up(tn);
    tn = read_key(2);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      fill(i * R::STEP, i);
      cp_async_commit();
    }

    // ---- Q^T fragments, column g: dims 64c + 16t .. + 15 of the head
    uint32_t qf[QC][8];
    float cs[2] = {a.qk_scale, a.qk_scale};  // score scale of columns 2t, 2t + 1
    {
      const int head = FEW ? g & 3 : g;
      const bool has = head < ncol;
      const uint4* qp = reinterpret_cast<const uint4*>(
          a.q + ((size_t)row * a.H + (has ? h0 + head : 0)) * DQK + 16 * t4);
#pragma unroll
      for (int c = 0; c < QC; ++c)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint4 x = has ? __ldg(qp + c * 8 + i) : make_uint4(0, 0, 0, 0);
          qf[c][4 * i + 0] = x.x; qf[c][4 * i + 1] = x.y;
          qf[c][4 * i + 2] = x.z; qf[c][4 * i + 3] = x.w;
        }
    }
    if constexpr (FMT == 1) {
      uint32_t top = 0;  // the largest exponent field of |q|
#pragma unroll
      for (int c = 0; c < QC; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i)
          top = max(top, max((qf[c][i] << 16) & 0x7f800000u, qf[c][i] & 0x7f800000u));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int ex = max((int)(top >> 23) - 127, -100);  // 2^ex <= max|q| (or less)
      const float up = __int_as_float((13 - ex + 127) << 23);
      // (in this order: the tensor's scale may be as small as q is large)
      const float scale = a.qk_scale * __int_as_float((ex - 13 + 127) << 23) * a.c.k_scale;
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

    // one step: the 16 keys in slots `base` .., of which `mask` have a row
    const int ka = kappa(g), k0 = kappa(2 * t4), k1 = kappa(2 * t4 + 1);
    auto step = [&](uint32_t base, uint32_t mask) {
      if constexpr (FMT == 1) {
        // this thread's places in a step: key ka's codes and scales, keys k0's and k1's values
        const uint32_t k_at = ring + ka * S::PITCH + t4 * 8;
        const uint32_t ks_at = ring + ka * S::PITCH + S::KS + (ks0 & 15) + t4;
        const uint32_t v_at0 = ring + k0 * S::PITCH + S::V + g * (VPT / 2);
        const uint32_t v_at1 = ring + k1 * S::PITCH + S::V + g * (VPT / 2);
        const uint32_t vs_off = S::VS - S::V + (vs0 & 15) + (g * VPT) / 16 - g * (VPT / 2);
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
        // probabilities hi + lo: in the columns 0..3 and 4..7, or in two products
        __half2 p01 = __floats2half2_rn(p[0], p[1]), p23 = __floats2half2_rn(p[2], p[3]);
        uint32_t c0, c1;
        if constexpr (FEW) {
          p01 = without(p, p01, t4 >= 2);
          p23 = without(p + 2, p23, t4 >= 2);
        } else {
          const __half2 r01 = without(p, p01, true), r23 = without(p + 2, p23, true);
          c0 = transpose8x8(*reinterpret_cast<const uint32_t*>(&r01));
          c1 = transpose8x8(*reinterpret_cast<const uint32_t*>(&r23));
        }
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
            if constexpr (!FEW) mma_f16(o[4 * w + i], f, c0, c1);
          }
        }
      } else {
        // S^T = K Q^T, two accumulators
        float s[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[i][e] = 0.f;
        const uint32_t ra = ring + base + g * S::PITCH + t4 * 32, rb = ra + 8 * S::PITCH;
#pragma unroll
        for (int c = 0; c < QC; ++c)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            uint32_t xa[4], xb[4];
            load_words(ra + c * 128 + hf * 16, xa);
            load_words(rb + c * 128 + hf * 16, xb);
            const uint32_t f0[4] = {xa[0], xb[0], xa[1], xb[1]};
            const uint32_t f1[4] = {xa[2], xb[2], xa[3], xb[3]};
            mma_bf16(s[0], f0, qf[c][4 * hf], qf[c][4 * hf + 1]);
            mma_bf16(s[1], f1, qf[c][4 * hf + 2], qf[c][4 * hf + 3]);
          }
        float x[4] = {(s[0][0] + s[1][0]) * cs[0], (s[0][1] + s[1][1]) * cs[1],
                      (s[0][2] + s[1][2]) * cs[0], (s[0][3] + s[1][3]) * cs[1]};
        uint32_t k01 = 0xffffffffu, k23 = 0xffffffffu;
        if (mask != 0xffffu) {  // row 0 stands in for a missing key: it may hold anything
          if (!((mask >> g) & 1u)) x[0] = x[1] = -INFINITY;
          if (!((mask >> (g + 8)) & 1u)) x[2] = x[3] = -INFINITY;
          const uint32_t mk = mask >> (2 * t4);
          k01 = ((mk & 1u) * 0xffffu) | (((mk >> 1) & 1u) * 0xffff0000u);
          k23 = (((mk >> 8) & 1u) * 0xffffu) | (((mk >> 9) & 1u) * 0xffff0000u);
        }
        float p[4];
        softmax_step<TOP, MT>(x, m, l, o, p);
        const __nv_bfloat162 h01 = __floats2bfloat162_rn(p[0], p[1]);
        const __nv_bfloat162 h23 = __floats2bfloat162_rn(p[2], p[3]);
        const __nv_bfloat162 r01 = __floats2bfloat162_rn(p[0] - __low2float(h01),
                                                         p[1] - __high2float(h01));
        const __nv_bfloat162 r23 = __floats2bfloat162_rn(p[2] - __low2float(h23),
                                                         p[3] - __high2float(h23));
        const uint32_t b0 = transpose8x8(*reinterpret_cast<const uint32_t*>(&h01));
        const uint32_t b1 = transpose8x8(*reinterpret_cast<const uint32_t*>(&h23));
        const uint32_t c0 = transpose8x8(*reinterpret_cast<const uint32_t*>(&r01));
        const uint32_t c1 = transpose8x8(*reinterpret_cast<const uint32_t*>(&r23));
        const uint32_t v0 = ring + base + ((lane & 7) + ((lane >> 4) << 3)) * S::PITCH + S::V +
                            ((lane >> 3) & 1) * 16;
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          uint32_t f[4];
          ldmatrix_x4_trans(f, v0 + i * 32);
          f[0] &= k01; f[1] &= k01; f[2] &= k23; f[3] &= k23;
          mma_bf16(o[i], f, b0, b1);
          mma_bf16(o[i], f, c0, c1);
        }
      }
    };

    // ---- main loop
    uint32_t at_step = 0;                   // the slots of the step worked on,
    uint32_t at_fill = AHEAD * R::STEP;     // and of the step copied
    auto advance = [](uint32_t x) { return x == AHEAD * R::STEP ? 0u : x + R::STEP; };
    int turn = 0;                           // which half of `rows` the pair worked on has
    for (int n = 0; n < steps; n += 2) {
      masks = masks_n;
      masks_n = __ballot_sync(0xffffffffu, rn >= 0);
      rows[32 * (turn ^ 1) + my_word] = max(rn, 0);
      rn = look_up(tn);
      tn = read_key((n >> 1) + 3);
      __syncwarp();
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        // step n + half + AHEAD: of this pair (one ahead, half 0), or of the next
        constexpr bool kOne = AHEAD == 1;
        const bool next = !kOne || half == 1;
        if (next ? masks_n != 0u : masks >= 0x10000u)
          fill(at_fill, 2 * (next ? turn ^ 1 : turn) + (kOne ? half ^ 1 : half));
        cp_async_commit();
        cp_async_wait<AHEAD>();  // this step's copies have landed
        __syncwarp();
        const uint32_t mask = half ? masks >> 16 : masks & 0xffffu;
        if (mask != 0u) step(at_step, mask);
        __syncwarp();  // its slots may be filled again
        at_step = advance(at_step);
        at_fill = advance(at_fill);
      }
      turn ^= 1;
    }
    cp_async_wait<0>();  // copies in flight land before the ring is used again

    // ---- this warp's (m, l, O)
#pragma unroll
    for (int d = 4; d < 32; d <<= 1) {
      l[0] += __shfl_xor_sync(0xffffffffu, l[0], d);
      l[1] += __shfl_xor_sync(0xffffffffu, l[1], d);
    }
    __syncthreads();
    float* ml = reinterpret_cast<float*>(smem);    // [warp][8][2]
    float* ob = ml + (blockDim.x >> 5) * 16;       // [warp][8][DV]
    if (g == 0)
      *reinterpret_cast<float4*>(ml + warp * 16 + 4 * t4) = make_float4(m[0], l[0], m[1], l[1]);
    float* c0 = ob + (size_t)(warp * 8 + 2 * t4) * DV;
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      if constexpr (FMT == 1) {
        const int d = g * VPT + 2 * i;
        *reinterpret_cast<float2*>(c0 + d) = make_float2(o[i][0], o[i][2]);
        *reinterpret_cast<float2*>(c0 + DV + d) = make_float2(o[i][1], o[i][3]);
      } else {
        const int d = 16 * i + g;
        c0[d] = o[i][0]; c0[DV + d] = o[i][1]; c0[d + 8] = o[i][2]; c0[DV + d + 8] = o[i][3];
      }
    }
    __syncthreads();
    // ---- merged over the key groups in order: the output row, or this piece of it
    const int heads = a.hc * a.G;
    const size_t piece = (size_t)first_piece + (size_t)hg * a.rows + row;
    for (int i = threadIdx.x; i < heads * (DV / 4); i += blockDim.x) {
      const int hl = i / (DV / 4), d = (i % (DV / 4)) * 4;
      const int hh = hl % a.G;
      const int w0 = (hl / a.G) * a.nsub + (hh >> 3), col = hh & 7;
      float M = -INFINITY;
      for (int k = 0; k < a.kw; ++k) M = fmaxf(M, ml[(k * nhw + w0) * 16 + col * 2]);
      float L = 0.f, x[4] = {0.f, 0.f, 0.f, 0.f};
      for (int k = 0; k < a.kw; ++k) {
        const int w = k * nhw + w0;
        const float mk = ml[w * 16 + col * 2];
        const float f = mk == -INFINITY ? 0.f : ex2_ftz(mk - M);
        L = fmaf(ml[w * 16 + col * 2 + 1], f, L);
        float4 v = *reinterpret_cast<const float4*>(ob + (size_t)(w * 8 + col) * DV + d);
        if constexpr (FEW) {  // the columns 4..7 hold the lo products of 0..3
          const float4 y = *reinterpret_cast<const float4*>(ob + (size_t)(w * 8 + col + 4) * DV + d);
          v.x += y.x; v.y += y.y; v.z += y.z; v.w += y.w;
        }
        x[0] = fmaf(v.x, f, x[0]); x[1] = fmaf(v.y, f, x[1]);
        x[2] = fmaf(v.z, f, x[2]); x[3] = fmaf(v.w, f, x[3]);
      }
      const int h = hg * heads + hl;
      if (alone) {
        // (the mean before the tensor's scale and the gate: their product with 1 / L may underflow)
        const float f = L > 0.f ? 1.0f / L : 0.f;
        const float gt =
            a.gate ? gate_act(__bfloat162float(a.gate[(size_t)row * a.H + h]), a.gate_mode) : 1.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = x[e] * f * a.c.v_scale * gt;
        const __nv_bfloat162 y0 = __floats2bfloat162_rn(x[0], x[1]);
        const __nv_bfloat162 y1 = __floats2bfloat162_rn(x[2], x[3]);
        uint2 y;
        y.x = *reinterpret_cast<const uint32_t*>(&y0);
        y.y = *reinterpret_cast<const uint32_t*>(&y1);
        *reinterpret_cast<uint2*>(a.out + ((size_t)row * a.H + h) * DV + d) = y;
      } else {
        const size_t at_part = piece * heads + hl;
        *reinterpret_cast<float4*>(a.part_o + at_part * DV + d) =
            make_float4(x[0], x[1], x[2], x[3]);
        if (d == 0) {
          a.part_ml[at_part * 2] = M;
          a.part_ml[at_part * 2 + 1] = L;
        }
      }
    }
    __syncthreads();  // the ring may be filled again
  }
}

// Rows in several pieces, merged in order: one CTA per (query token, head).  Rows without keys get
// their zeros here.
template <int DV>
__global__ void __launch_bounds__(DV) cache_merge_kernel(const CacheAttnArgs a) {
  __shared__ long long warp_sums[DV / 32];
  __shared__ long long s_before;
  __shared__ float2 weight[DV];   // and weighted sum
  __shared__ float warp_max[DV / 32];
  const int row = blockIdx.x / a.H, h = blockIdx.x % a.H;
  const int heads = a.hc * a.G, hg = h / heads, hl = h % heads;
  const int per = (a.rows + DV - 1) / DV;
  const int r0 = min((int)threadIdx.x * per, a.rows), r1 = min(r0 + per, a.rows);
  long long mine = 0, before;
  for (int i = r0; i < r1; ++i) mine += row_steps(a, i);
  const long long each = block_scan(mine, warp_sums, &before);
  if (r0 <= row && row < r1) {
    for (int i = r0; i < row; ++i) before += row_steps(a, i);
    s_before = before;
  }
  __syncthreads();
  const int n = row_steps(a, row);
  // the pieces are written (every CTA waits, so that this grid never ends before the one it merges)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __nv_bfloat16* out = a.out + ((size_t)row * a.H + h) * DV + threadIdx.x;
  if (n == 0) {
    *out = __float2bfloat16_rn(0.f);
    return;
  }
  const long long all = each * a.nhg, s = hg * each + s_before;
  const int ctas = ctas_of(a, all);
  const int c0 = cta_of(s, all, ctas), c1 = cta_of(s + n - 1, all, ctas);
  if (c0 == c1) return;  // one piece: written by its CTA
  const size_t p0 = (size_t)c0 + (size_t)hg * a.rows + row;
  const int np = c1 - c0 + 1;
  const float* ml = a.part_ml + (p0 * heads + hl) * 2;
  const float* po = a.part_o + (p0 * heads + hl) * DV + threadIdx.x;
  const size_t step = heads;
  // the pieces' maximum
  float M = -INFINITY;
  for (int p = threadIdx.x; p < np; p += DV) M = fmaxf(M, ml[p * step * 2]);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
  if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = M;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < DV / 32; ++w) M = fmaxf(M, warp_max[w]);
  float L = 0.f, x = 0.f;
  for (int q = 0; q < np; q += DV) {
    const int nq = min(DV, np - q);
    __syncthreads();
    if ((int)threadIdx.x < nq) {
      const float2 e = *reinterpret_cast<const float2*>(ml + (q + threadIdx.x) * step * 2);
      const float w = e.x == -INFINITY ? 0.f : ex2_ftz(e.x - M);
      weight[threadIdx.x] = make_float2(w, e.y * w);
    }
    __syncthreads();
#pragma unroll 8
    for (int p = 0; p < nq; ++p) {
      L += weight[p].y;
      x = fmaf(po[(q + p) * step * DV], weight[p].x, x);
    }
  }
  x = x * (L > 0.f ? 1.0f / L : 0.f) * a.c.v_scale;
  if (a.gate) x *= gate_act(__bfloat162float(a.gate[(size_t)row * a.H + h]), a.gate_mode);
  *out = __float2bfloat16_rn(x);
}

// How a call is laid out over CTAs.
struct Plan {
  int hc, nhg, nsub, kw, nw, grid, shares, least_log;
  size_t pieces;
};

template <typename F>
bool with_dims(int format, int DQK, int DV, F&& f) {
  auto dims = [&](auto fmt) {
    constexpr int FMT = decltype(fmt)::value;
    if (DQK == 64 && DV == 64) return f(Ring<FMT, 64, 64>{}), true;
    if (DQK == 64 && DV == 128) return f(Ring<FMT, 64, 128>{}), true;
    if (DQK == 128 && DV == 64) return f(Ring<FMT, 128, 64>{}), true;
    if (DQK == 128 && DV == 128) return f(Ring<FMT, 128, 128>{}), true;
    if (DQK == 192 && DV == 64) return f(Ring<FMT, 192, 64>{}), true;
    if (DQK == 192 && DV == 128) return f(Ring<FMT, 192, 128>{}), true;
    return false;
  };
  return format == 0 ? dims(std::integral_constant<int, 0>{})
                     : dims(std::integral_constant<int, 1>{});
}

constexpr int kPiece = 4;

// Shapes only (no device query), so that workspace sizes are reproducible.
bool make_plan(int format, int rows, int H, int HKV, int DQK, int DV, long long max_keys,
               bool selected, Plan* p) {
  *p = Plan{};
  p->nsub = (H / HKV + 7) / 8;
  int warps = 0;
  if (!with_dims(format, DQK, DV, [&](auto r) { warps = decltype(r)::WARPS; })) return false;
  if (p->nsub > warps) warps = kWarps;
  // KV heads per CTA: the most that divide HKV and keep 3 of 4 warps busy, more than one warp per
  // head taking different keys
  int hc = warps / p->nsub;
  while (HKV % hc != 0 || (hc > 1 && 4 * hc * p->nsub * (warps / (hc * p->nsub)) < 3 * warps)) --hc;
  p->hc = hc;
  p->nhg = HKV / hc;
  const int nhw = hc * p->nsub;
  p->kw = warps / nhw;
  p->nw = nhw * p->kw;
  int smem = 0;
  with_dims(format, DQK, DV, [&](auto r) { smem = decltype(r)::smem(p->nw); });
  const int resident = 148 * (format == 1 && p->nw <= 4 ? 4 : smem <= 113 * 1024 ? 2 : 1);
  // Pieces while they may fill the GPU better than the rows do: below two rounds of rows.  A piece
  // costs as much as some steps (its queries, the first copies' latency, its part of the merge): the
  // least piece has 8 steps, or 4 or 2 where that still leaves at most two CTAs, or one, per SM.  In
  // us, for 2, 4 and 8 steps: one 4-bit window of 33 steps in 2 groups 11.7, 12.7, 16.6; 16 of them
  // 18.0, 15.7, 17.5; one context of 257 steps 21.5, 15.7, 16.9; 20 tokens of 32 steps in 5 groups
  // 23.0, 22.9, 19.1; 8 contexts of 257 steps 28.7, 28.7, 27.1.
  // Over 72 shapes (both formats, 8 and 32 KV heads, 1 to 64 rows of 64 to 131072 keys) 2 steps
  // throughout are up to 18 us slower than this rule, 4 up to 14, 8 up to 4, and none is faster by more
  // than the timer's 2 us; without the whole shares below, 4 us slower at most and 2 faster.
  const long long ctas = (long long)rows * p->nhg;
  const long long steps = ctas * ((max_keys + 16 * p->kw - 1) / (16 * p->kw));
  p->least_log = steps <= 2 * 148 ? 1 : steps <= 8 * 148 ? 2 : 3;
  if (ctas < 2 * resident && (steps >> p->least_log) > ctas) {
    p->grid = (int)((steps >> p->least_log) < resident ? (steps >> p->least_log) : resident);
    // A cut inside a CTA's share costs a second piece, about kPiece steps: a grid that cuts rows of
    // one length into whole shares may be faster, although smaller (64 windows of 33 steps in 2
    // groups: 44.6 us on 256 CTAs, 47.9 us on 296; 16 rows of 128 steps in 8: 130 us on 296).
    const long long whole = ctas * (p->grid / ctas);
    if (whole > 0 && steps / whole + kPiece < steps / p->grid + 2 * kPiece) p->grid = (int)whole;
    p->pieces = (size_t)p->grid + (size_t)ctas;
    // Rows are laid out by whole tokens, so two groups' parts of a row share 64-byte lines.  Read at
    // the same time by neighbours, those come from memory once.  Eight contexts: 256 us, and 267 with
    // each group's shares together; 64 windows: 43.5 and 44.4.  Selected keys gain nothing (64 x
    // 2048: 184 us, 181).
    if (!selected && p->least_log == 3 && p->grid % p->nhg == 0) p->shares = p->grid / p->nhg;
  }
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

size_t workspace_of(const Plan& pl, const CacheAttnProblem& p) {
  return pl.pieces * pl.hc * (p.H / p.cache.HKV) * (p.cache.DV + 2) * sizeof(float);
}

bool plan_of(const CacheAttnProblem& p, Plan* pl) {
  return make_plan(p.cache.format, p.B * p.S, p.H, p.cache.HKV, p.cache.DQK, p.cache.DV,
                   max_keys_of(p), p.idx != nullptr, pl);
}

template <int FMT, int DQK, int DV>
cudaError_t launch(const CacheAttnArgs& a, const Plan& p, Ring<FMT, DQK, DV>, cudaStream_t st) {
  const int smem = Ring<FMT, DQK, DV>::smem(p.nw);
  const bool few = FMT == 1 && a.G <= 4;
  auto kern = few ? cache_attn_kernel<FMT, DQK, DV, FMT == 1> : cache_attn_kernel<FMT, DQK, DV, false>;
  const dim3 grid = p.shares > 0 ? dim3((unsigned)p.nhg, (unsigned)p.shares)
                    : p.grid > 0 ? dim3((unsigned)p.grid)
                                 : dim3((unsigned)a.rows * (unsigned)p.nhg);
  // The kernel's attributes are set once per device (each call of theirs costs a host microsecond),
  // and again if a launch finds them gone, as after a device reset.
  static std::atomic<unsigned long long> ready_of[2];
  std::atomic<unsigned long long>& ready = ready_of[few];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev < 64 ? 1ULL << dev : 0;
  for (int attempt = 0; attempt < 2; ++attempt) {
    const bool known = (ready.load(std::memory_order_relaxed) & bit) != 0 && attempt == 0;
    if (!known) {
      // the most that any call of this instantiation asks for
      e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               Ring<FMT, DQK, DV>::smem(kWarps));
      // all of the SM's shared memory, or a second CTA would find too little of it
      if (e == cudaSuccess)
        e = cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout,
                                 cudaSharedmemCarveoutMaxShared);
      if (e != cudaSuccess) return e;
      ready.fetch_or(bit, std::memory_order_relaxed);
    }
    kern<<<grid, 32 * p.nw, smem, st>>>(a);
    e = cudaGetLastError();
    if (!known || e != cudaErrorInvalidValue) break;
  }
  if (e != cudaSuccess || p.grid == 0) return e;
  // launched beside the pieces (programmatic dependence), so that its start costs no time after them
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)a.rows * a.H);
  cfg.blockDim = dim3(DV);
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, cache_merge_kernel<DV>, a);
}

}  // namespace

bool cache_attn_supported(int format, int H, int HKV, int DQK, int DV) {
  Plan p;
  return make_plan(format, 1, H, HKV, DQK, DV, 1, false, &p);
}

size_t cache_attn_workspace_bytes(const CacheAttnProblem& p) {
  Plan pl;
  return plan_of(p, &pl) ? workspace_of(pl, p) : 0;
}

cudaError_t launch_cache_attn(const CacheAttnProblem& p, void* ws, size_t ws_bytes,
                              cudaStream_t st) {
  Plan pl;
  if (!plan_of(p, &pl)) return cudaErrorNotSupported;
  CacheAttnArgs a{};
  a.c = p.cache;
  a.q = static_cast<const __nv_bfloat16*>(p.q);
  a.pos = p.pos; a.idx = p.idx; a.K = p.K; a.window = p.window; a.n_first = p.n_first;
  a.gate = static_cast<const __nv_bfloat16*>(p.gate); a.gate_mode = p.gate_mode;
  a.out = static_cast<__nv_bfloat16*>(p.out);
  a.S = p.S; a.H = p.H; a.G = p.H / p.cache.HKV; a.rows = p.B * p.S;
  a.qk_scale = p.sm_scale * kLog2e;
  a.hc = pl.hc; a.nhg = pl.nhg; a.nsub = pl.nsub; a.kw = pl.kw; a.grid = pl.grid;
  a.least_log = pl.least_log;
  if (pl.grid > 0) {
    if (ws == nullptr || ws_bytes < workspace_of(pl, p)) return cudaErrorInvalidValue;
    a.part_o = static_cast<float*>(ws);
    a.part_ml = a.part_o + pl.pieces * pl.hc * a.G * p.cache.DV;
  }
  cudaError_t e = cudaErrorNotSupported;
  with_dims(p.cache.format, p.cache.DQK, p.cache.DV,
            [&](auto ring) { e = launch(a, pl, ring, st); });
  return e;
}

}  // namespace dsa
