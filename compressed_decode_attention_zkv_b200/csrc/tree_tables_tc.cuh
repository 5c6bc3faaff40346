// Key lookup tables of many query rows on the tensor cores (sm_100a, tcgen05): the tables of
// query_tables.cuh where one kv head has more than three blocks of 64 rows.
//
// CTA = 128 rows of one kv head (TMEM lanes) x some of its stages.  The rows are rotated once, scaled
// and split into two fp16 planes (mma_split.cuh) in shared memory, in the tensor cores' K-major,
// 128-byte-swizzled operand layout; the codewords come split from a kernel before, NB of a stage at a
// time.  Per step one thread of a warp of its own issues the three products lo hi, hi lo and hi hi (D / 16 tcgen05.mma of
// kind::f16 each, M = 128, N = NB) into one float32 accumulator of NB TMEM columns and commits them to an
// mbarrier; the cross terms come first, so that their sum, 2^-11 of the rest, is complete before it
// meets the large one.  While a step's products run, the step before is read from TMEM, scaled and
// written, and the step after is copied (d = 256 has room for one operand buffer: there the copy
// follows the products).
// 18 us at 512 rows per kv head, 8 heads, 4 stages, d = 128; 35 us at 1536 rows (mma.sync with the
// codewords split before: 25 and 67 us).  Writing the tables bounds it: 32 bytes per codeword, stage
// and row group, about 3000 cycles a step beside 2800 of products.
#pragma once

#include "query_tables.cuh"
#include "tc_util.cuh"

namespace zkv {

constexpr int kTtRows = 128;
constexpr int kTtWork = 512;                 // threads that rotate, copy and read; one more warp issues
constexpr int kTtThreads = kTtWork + 32;

template <int D>
struct TtCfg {
  static constexpr int NB = D == 64 ? 256 : D == 128 ? 128 : 64;    // codewords per step
  static constexpr int BUFS = D == 256 ? 1 : 2;                     // operand buffers
  static constexpr int P = D / 64;                                  // 128-byte panels of a row
  static constexpr int STEPS = kCodebook / NB;                      // per stage
  static constexpr int GROUPS = NB >= 128 ? 4 : 2;                  // column groups of the reading warps
};

template <int D>
struct TtSmem {
  using C = TtCfg<D>;
  __half a[2][C::P][kTtRows * 64];           // rotated queries: plane, panel
  __half b[C::BUFS][2][C::P][C::NB * 64];    // codewords: buffer, plane, panel
  float qs[kTtRows];                         // scales of the rows (softmax scale included)
  float cs[3][C::NB];                        // scales of the steps' codewords (three steps are in flight)
  uint64_t mbar[2];
  uint32_t tmem_base;
};
template <int D>
constexpr size_t tt_smem_bytes() {
  return sizeof(TtSmem<D>) + 1024;           // + alignment of the operand panels
}

// element (r, i) of a panel of 64 fp16 per row: 16-byte chunk q of row r at position q ^ (r & 7)
__device__ __forceinline__ int tt_swz(int r, int i) { return r * 64 + ((((i >> 3) ^ r) & 7) << 3) + (i & 7); }

// D float32, A and B fp16, both K-major, M = 128, N
constexpr uint32_t tt_idesc(int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(kTtRows >> 4) << 24);
}

template <int D>
__device__ __forceinline__ void tree_tables_tc(const QueryTables& a, int64_t blk, int shares, TtSmem<D>& sm,
                                               int32_t* err) {
  using C = TtCfg<D>;
  constexpr int E = D / 32, NB = C::NB;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int tiles = (int)(((int64_t)a.B * a.RP + kTtRows - 1) / kTtRows);
  const int share = (int)(blk % shares);
  const int tile = (int)(blk / shares % tiles), kvh = (int)(blk / shares / tiles);
  const int row0 = tile * kTtRows, rows = a.B * a.RP - row0;
  const uint32_t mbar[2] = {(uint32_t)__cvta_generic_to_shared(&sm.mbar[0]),
                            (uint32_t)__cvta_generic_to_shared(&sm.mbar[1])};
  if (warp == 0) {
    const uint32_t slot = (uint32_t)__cvta_generic_to_shared(&sm.tmem_base);
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot),
                 "r"((uint32_t)(2 * NB))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (tid == 0) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(mbar[0]) : "memory");
    asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(mbar[1]) : "memory");
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  // steps of this CTA: stages share, share + shares, ..., STEPS each
  const int mine = a.Sk > share ? (a.Sk - share - 1) / shares + 1 : 0, steps = mine * C::STEPS;
  auto stage_of = [&](int u) { return share + u / C::STEPS * shares; };
  auto copy = [&](int u) {       // step u's codewords (asynchronous) and their scales
    if (u < steps) {
      const int64_t first = ((int64_t)kvh * a.Sk + stage_of(u)) * kCodebook + u % C::STEPS * NB;
      auto& b = sm.b[u % C::BUFS];
      for (int f = tid; f < NB * (D / 8); f += kTtWork) {
        const int n = f / (D / 8), gc = f % (D / 8), at = tt_swz(n, (gc & 7) * 8);
        cp_async16(&b[0][gc >> 3][at], a.books.hi + (first + n) * D + gc * 8);
        cp_async16(&b[1][gc >> 3][at], a.books.lo + (first + n) * D + gc * 8);
      }
      if (tid < NB) sm.cs[u % 3][tid] = a.books.scale[first + tid];
    }
    cp_async_commit();
  };
  const bool works = tid < kTtWork;
  // rows, rotated (float32 transform): warp w takes rows w, w + 16, ...
  if (works) {
    // (short code that repeats: executed once, long straight code waits for its instructions)
#pragma unroll 1
    for (int k = 0; k < 8; k += 2) {
      float v[2][E], part[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int r = warp + 16 * (k + u), j = row0 + r;
        int b = a.by_rp.quotient(j);
        const int rho = j - b * a.RP;
        int i = a.by_g.quotient(rho), g = rho - i * a.G;
        const bool there = r < rows && rho < a.R;
        if (!there) b = i = g = 0;
        const int present = a.n_query ? a.n_query[b] : a.N;
        const __half* qr = a.q + b * a.q_sb + i * a.q_sn + ((int64_t)kvh * a.G + g) * a.q_sh + lane;
#pragma unroll
        for (int e = 0; e < E; ++e) v[u][e] = __half2float(qr[e * 32]);
        if (!there || i >= present)
#pragma unroll
          for (int e = 0; e < E; ++e) v[u][e] = 0.f;
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if (a.k_smooth) {   // the query absorbs the keys' smoothing: lambda * q
          const float* l = a.k_smooth + (int64_t)kvh * D + lane;
#pragma unroll
          for (int e = 0; e < E; ++e) v[u][e] *= l[e * 32];
        }
        fwht_warp_f32<D>(v[u], lane);
        part[u] = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) part[u] = fmaf(v[u][e], v[u][e], part[u]);
      }
      int own = 0;          // the norms of both rows at once
      const int ex = split_exponent(sqrtf(TransposeSum<2, 2, 16>::run(part, lane, own)));
      const float down_of = exp2_int(-ex);
      sm.qs[warp + 16 * (k + own)] = exp2_int(ex) * (float)(a.rot * (double)a.scale_log2);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float down = __shfl_sync(0xffffffffu, down_of, sum_owner<2>(u));
        const int r = warp + 16 * (k + u);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const int at = tt_swz(r, (e & 1) * 32 + lane);
          split(v[u][e] * down, sm.a[0][e >> 1][at], sm.a[1][e >> 1][at]);
        }
      }
    }
  }
  pdl_wait();             // (the kernel before splits the codewords)
  if (works) copy(0);
  // reading a step: row = TMEM lane 32 (warp % 4) + lane, columns of group warp / 4
  constexpr int COLS = NB / C::GROUPS;
  const int quarter = warp & 3, col0 = (warp >> 2) * COLS, r = quarter * 32 + lane;
  const bool reads = works && warp < 4 * C::GROUPS;
  const int step = a.SKP * a.RG;
  float* out = nullptr;
  if (works && r < rows) {
    const int j = row0 + r, b = a.by_rp.quotient(j), rho = j - b * a.RP, rg = a.by_rg.quotient(rho);
    out = a.lut + (((int64_t)b * a.Hkv + kvh) * (a.RP / a.RG) + rg) * ((int64_t)kCodebook * step) + (rho - rg * a.RG);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  const uint32_t taddr = tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)col0;
  const float qs = sm.qs[r & (kTtRows - 1)];
  auto put = [&](int u) {
    float* o = out + (u % C::STEPS * NB + col0) * step + stage_of(u) * a.RG;
#pragma unroll 1
    for (int c = 0; c < COLS; c += 32) {
      float v[32];
      tc_ld32(taddr + (uint32_t)((u & 1) * NB + c), v);
      if (out) {
#pragma unroll
        for (int k = 0; k < 32; ++k) o[(c + k) * step] = v[k] * sm.cs[u % 3][col0 + c + k] * qs;
      }
    }
  };
  const uint32_t a_base = (uint32_t)__cvta_generic_to_shared(&sm.a[0][0][0]);
  bool late = false;                     // (the same in a whole warp: reading TMEM takes all its lanes)
  int last = -1;                         // the last step whose products were issued
  auto wait_for = [&](int u) {
    late = __any_sync(0xffffffffu, !tc_wait(mbar[u & 1], (uint32_t)(u >> 1) & 1u));
    tc_fence_after();
  };
  for (int u = 0; u < steps; ++u) {
    cp_async_wait_all();
    // the rows and the copies must be visible to the tensor cores
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    tc_fence_before();
    if (__syncthreads_or(late)) {        // (uniform)
      late = true;
      break;
    }
    tc_fence_after();
    last = u;
    if (tid == kTtWork) {
      const uint32_t b_base = (uint32_t)__cvta_generic_to_shared(&sm.b[u % C::BUFS][0][0][0]);
      const uint32_t acc = tmem + (uint32_t)((u & 1) * NB);
#pragma unroll 1
      for (int prod = 0; prod < 3; ++prod) {       // lo hi, hi lo, hi hi
        const uint32_t ap = a_base + (prod == 0 ? C::P * kTtRows * 128u : 0u);
        const uint32_t bp = b_base + (prod == 1 ? C::P * NB * 128u : 0u);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const int p = k >> 2, o = (k & 3) * 32;  // panel, byte offset inside the 128-byte row
          const uint64_t ad = tc_desc(ap + (uint32_t)(p * kTtRows * 128 + o));
          const uint64_t bd = tc_desc(bp + (uint32_t)(p * NB * 128 + o));
          const uint32_t add = prod > 0 || k > 0 ? 1u : 0u;
          asm volatile(
              "{\n\t.reg .pred p;\n\t"
              "setp.ne.b32 p, %4, 0;\n\t"
              "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
              ::"r"(acc), "l"(ad), "l"(bd), "r"(tt_idesc(NB)), "r"(add)
              : "memory");
        }
      }
      asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(mbar[u & 1])
                   : "memory");
    }
    if (!works) continue;
    // the step that is read now: the one before, or with one operand buffer this one
    const int x = C::BUFS == 2 ? u - 1 : u;
    if (x >= 0) wait_for(x);
    copy(u + 1);                         // into the buffer that step u - 1 (or u) has left
    if (x >= 0 && !late && reads) put(x);
  }
  if (C::BUFS == 2 && steps > 0 && !late && works) {
    wait_for(steps - 1);
    if (!late && reads) put(steps - 1);
  }
  cp_async_wait_all();
  if (late && lane == 0) set_error(err, ZKV_DEVERR_TIMEOUT);
  // the padded stages' entries are zero
  if (out && share == 0)
    for (int s = a.Sk; s < a.SKP; ++s)
      for (int c = warp >> 2; c < kCodebook; c += kTtWork / 128) out[c * step + s * a.RG] = 0.f;
  tc_fence_before();
  if (__syncthreads_or(late)) {
    // products still in flight get one more bounded wait before their columns are freed
    if (last >= 0) (void)tc_wait(mbar[last & 1], (uint32_t)(last >> 1) & 1u);
    __syncthreads();
  }
  if (warp == 0) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"((uint32_t)(2 * NB))
                 : "memory");
  }
}

}  // namespace zkv
