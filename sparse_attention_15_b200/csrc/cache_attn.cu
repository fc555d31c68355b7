// Attention of single query tokens over the paged key/value cache, the headwise gate fused: how a
// call is laid out over CTAs, and the kernel for bf16 rows (rows held in 4 bits: cache_attn_q4.cu).
//
//   o[h,:] = sum_t p_t v[t,h/G,:],  p = softmax_t(sm_scale * q[h,:] . k[t,h/G,:]),  G = H/HKV
//
// over the query's keys: idx[b,s,:], or t <= pos with t > pos - window or t < n_first.  Every
// query token has its own key list, so masked keys are never looked at and what they hold (NaN, a
// page of another sequence, nothing yet) does not matter.
//
// One CTA takes a query token, a group of KV heads and a slice of its keys; the slices of one
// query are merged by launch_split_combine in a fixed order.  Both products run on mma.sync
// m16n8k16 with the cache as the 16-row operand and the up to 8 query heads of a KV head as the 8
// columns: S^T = K Q^T [16 keys x 8 heads], O^T += V^T P^T [dims x 8 heads], float32
// accumulation.  (A tcgen05 tile wants 128 rows that share an operand; here 1 to 8 do.)
//
// bf16 rows: a producer warp turns keys into cache rows through the page table and streams them
// into a ring of shared-memory slots (1-D bulk copies, mbarrier transaction counts, no
// multicast); each consumer warp owns one KV head (8 of its query heads) and 16 keys of a stage.
// The contraction order over the dims is free, so a thread takes 16 consecutive ones of a key.
// Probabilities are a bf16 pair hi + lo, as one bf16 would be no more exact than the output.
#include "cache_attn.cuh"

namespace dsa {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kMaxWarps = 16;     // consumer warps of a CTA
constexpr int kMaxStages = 8;
constexpr int kMaxSplit = 64;     // launch_split_combine's limit

__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

template <int DQK, int DV>
__global__ void __maxnreg__(96) cache_attn_bf16_kernel(const CacheAttnArgs a) {
  constexpr int QC = DQK / 64;       // 64-dim chunks: 16 dims per thread each
  constexpr int MT = DV / 16;        // 16-row tiles of O^T
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

  if (threadIdx.x == 0) {
    for (int i = 0; i < a.nstages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], nw);
    }
    fence_mbar_init();
  }
  __syncthreads();

  const int kb = hc * DQK * 2, vb = hc * DV * 2;  // a slot: this CTA's heads' K, then V

  if (warp == nw) {
    // ------------------------------------------------------------- producer
    const int pos = __ldg(a.pos + row);
    const KeyList l = key_list(a, row, pos);
    int j0, j1;
    key_slice(l, a.nsplit, split, &j0, &j1);
    const int32_t* table = a.c.table + (size_t)(row / a.S) * a.c.max_pages;
    const uint32_t bytes = (uint32_t)(kb + vb);
    int fills = 0;
    bool ok = true;
    // The keys of a stage (lane: keys lane, lane + 32, ...) are read two stages ahead and their
    // rows looked up one stage ahead, so that neither load is waited for per stage.
    int t[4];
    long long r[4];
    auto read_keys = [&](int j) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int k = 32 * i + lane;
        t[i] = k < ks && j < j1 && k < j1 - j ? l.at(j + k) : -1;
      }
    };
    auto look_up = [&] {
#pragma unroll
      for (int i = 0; i < 4; ++i) r[i] = t[i] <= pos ? cache_row(a.c, table, t[i]) : -1;
    };
    auto after = [&](int j) { return j1 - j > ks ? j + ks : j1; };
    read_keys(j0);
    look_up();
    read_keys(after(j0));
    for (int j = j0; ok && j < j1; j = after(j)) {
      uint32_t m[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) m[i] = __ballot_sync(0xffffffffu, r[i] >= 0);
      const int nvalid = __popc(m[0]) + __popc(m[1]) + __popc(m[2]) + __popc(m[3]);
      const int st = fills % a.nstages;
      if (nvalid > 0 && fills >= a.nstages)
        ok = warp_wait(&empty[st], (uint32_t)(fills / a.nstages - 1) & 1u);
      if (!ok) break;
      if (nvalid > 0 && lane == 0) {
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
        if (a.nhg == 1) {  // all heads: the whole row
          bulk_g2s(dst, src, bytes, &full[st]);
        } else {
          bulk_g2s(dst, src + (size_t)kv0 * DQK * 2, kb, &full[st]);
          bulk_g2s(dst + kb, src + cache_v_off(0, a.c.HKV, DQK) + (size_t)kv0 * DV * 2, vb,
                   &full[st]);
        }
      }
      if (nvalid > 0) ++fills;
      look_up();
      read_keys(after(after(j)));
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
    float o[MT][4];
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] = 0.f;

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
        const uint8_t* ra = slot + (size_t)(kg * 16 + g) * a.pitch + kvl * (DQK * 2) + t4 * 32;
        const uint8_t* rb = ra + (size_t)8 * a.pitch;
#pragma unroll
        for (int c = 0; c < QC; ++c)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const uint4 xa = *reinterpret_cast<const uint4*>(ra + c * 128 + hf * 16);
            const uint4 xb = *reinterpret_cast<const uint4*>(rb + c * 128 + hf * 16);
            const uint32_t f0[4] = {xa.x, xb.x, xa.y, xb.y};
            const uint32_t f1[4] = {xa.z, xb.z, xa.w, xb.w};
            mma_bf16(s[0], f0, qf[c][4 * hf], qf[c][4 * hf + 1]);
            mma_bf16(s[1], f1, qf[c][4 * hf + 2], qf[c][4 * hf + 3]);
          }
        const bool va = (mask >> g) & 1u, vbk = (mask >> (g + 8)) & 1u;
        const float cs = a.qk_scale;
        const float x[4] = {va ? (s[0][0] + s[1][0]) * cs : -INFINITY,
                            va ? (s[0][1] + s[1][1]) * cs : -INFINITY,
                            vbk ? (s[0][2] + s[1][2]) * cs : -INFINITY,
                            vbk ? (s[0][3] + s[1][3]) * cs : -INFINITY};
        float p[4];
        softmax_step<0, MT>(x, m, l, o, p);
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
        uint32_t k01 = 0xffffffffu, k23 = 0xffffffffu;
        if (mask != 0xffffu) {  // a slot that was not filled may hold anything
          k01 = (((mask >> (2 * t4)) & 1u) * 0xffffu) |
                (((mask >> (2 * t4 + 1)) & 1u) * 0xffff0000u);
          k23 = (((mask >> (2 * t4 + 8)) & 1u) * 0xffffu) |
                (((mask >> (2 * t4 + 9)) & 1u) * 0xffff0000u);
        }
        const uint32_t v0 = smem_u32(slot) +
                            (uint32_t)((kg * 16 + (lane & 7) + ((lane >> 4) << 3)) * a.pitch + kb +
                                       kvl * (DV * 2) + ((lane >> 3) & 1) * 16);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          uint32_t f[4];
          ldmatrix_x4_trans(f, v0 + i * 32);
          f[0] &= k01; f[1] &= k01; f[2] &= k23; f[3] &= k23;
          mma_bf16(o[i], f, b0, b1);
          mma_bf16(o[i], f, c0, c1);
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
      l[0] += __shfl_xor_sync(0xffffffffu, l[0], d);
      l[1] += __shfl_xor_sync(0xffffffffu, l[1], d);
    }
    __syncthreads();  // every warp is done with the ring, and its copies have landed
    if (g == 0) *reinterpret_cast<float4*>(ml + warp * 16 + 4 * t4) = make_float4(m[0], l[0], m[1], l[1]);
    float* c0 = reinterpret_cast<float*>(ring) + (size_t)(warp * 8 + 2 * t4) * DV + g;
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      c0[16 * i] = o[i][0];
      c0[16 * i + DV] = o[i][1];
      c0[16 * i + 8] = o[i][2];
      c0[16 * i + 8 + DV] = o[i][3];
    }
  }
  if (warp == nw) __syncthreads();  // the producer's part of the barrier above
  __syncthreads();
  merge_groups<DV>(a, ml, reinterpret_cast<const float*>(ring), nhw, row, split, kv0);
}

// How a call is laid out over CTAs: KV heads per CTA, warps, stages, key slices.
struct Plan {
  int hc, nhg, nsub, kw, nw, nstages, pitch, nsplit;
  size_t smem;
};

constexpr size_t kHeadBytes = 512 + kMaxWarps * 64;  // barriers, stage marks, (m, l) of the warps

// bf16: the ring of `hc` KV heads per CTA; false if two stages do not fit.
bool plan_ring(int hc, int DQK, int DV, Plan* p) {
  // rows 16 bytes past a multiple of 128 apart: the consumers' loads then meet no bank twice
  const int part = hc * (DQK + DV) * 2;
  p->pitch = (part - 16 + 127) / 128 * 128 + 16;
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
  *p = Plan{};
  p->nsub = (H / HKV + 7) / 8;
  // KV heads per CTA: the most that divide HKV and keep 6 to 8 warps busy, more than one warp per
  // head taking different keys
  int hc = 8 / p->nsub;
  while (HKV % hc != 0 || (hc > 1 && hc * p->nsub * (8 / (hc * p->nsub)) < 6)) --hc;
  p->hc = hc;
  p->nhg = HKV / hc;
  const int nhw = hc * p->nsub;
  p->kw = 8 / nhw;
  p->nw = nhw * p->kw;
  int resident = 2 * 148;
  if (format == 0) {
    if (!plan_ring(hc, DQK, DV, p)) return false;
    if (p->smem > 113 * 1024) resident = 148;
  }
  // key slices: fill the resident CTAs in whole waves, 64 keys a slice at least
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

template <int DQK, int DV>
cudaError_t launch_bf16(const CacheAttnArgs& a, const Plan& p, unsigned grid, cudaStream_t st) {
  auto kern = cache_attn_bf16_kernel<DQK, DV>;
  cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)p.smem);
  // all of the SM's shared memory, or a second CTA would find too little of it
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout,
                             cudaSharedmemCarveoutMaxShared);
  if (e != cudaSuccess) return e;
  kern<<<grid, 32 * (p.nw + 1), p.smem, st>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_dims(const CacheAttnArgs& a, const Plan& p, int rows, cudaStream_t st) {
  const unsigned grid = (unsigned)rows * (unsigned)(p.nhg * p.nsplit);
  if (a.c.format == 1) return launch_cache_attn_q4(a, grid, st);
  const int dqk = a.c.DQK, dv = a.c.DV;
  if (dqk == 64 && dv == 64) return launch_bf16<64, 64>(a, p, grid, st);
  if (dqk == 64 && dv == 128) return launch_bf16<64, 128>(a, p, grid, st);
  if (dqk == 128 && dv == 64) return launch_bf16<128, 64>(a, p, grid, st);
  if (dqk == 128 && dv == 128) return launch_bf16<128, 128>(a, p, grid, st);
  if (dqk == 192 && dv == 64) return launch_bf16<192, 64>(a, p, grid, st);
  if (dqk == 192 && dv == 128) return launch_bf16<192, 128>(a, p, grid, st);
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
  const cudaError_t e = launch_dims(a, pl, rows, st);
  if (e != cudaSuccess || pl.nsplit == 1) return e;
  return launch_split_combine(1, a.part_o, a.part_ml, rows, pl.nsplit, p.H, p.cache.DV, p.gate,
                              p.gate_mode, p.out, st);
}

}  // namespace dsa
