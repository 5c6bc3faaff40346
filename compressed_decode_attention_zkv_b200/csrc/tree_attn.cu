// Attention of a tree of drafted tokens over the compressed cache (sm_100a).
//
// Passages: VQKV (gist.science summary of arXiv 2603.16435), section 2.3 "Decoding Stage"
// (on-demand reconstruction inside attention, local sliding window); VeloxQuant-MLX 0.5.1,
// "VecInfer" (the rotation is absorbed into the query); Differential-KV README, "Decode & Prefill
// Innovations" (fp32 log-sum-exp combine).  The tree of drafts has no counterpart on the pages.
//
// A (sequence, kv head) pair has R = N * G query rows rho = i * G + g, taken in groups ("items")
// of kTreeRG = 8.  Five kernels per call (programmatic dependent launches):
//   1. tree_dense_kernel    the dense part (fp16 window and the drafts that the mask names: partial
//      maximum, sum and output per row); one block computes the partition of the compressed tokens.
//      tree_tables_kernel   beside it: the key lookup tables of every row (query_tables.cuh); with
//      many rows after tree_split_kernel, which splits the codewords once for them and for 3.
//   2. tree_scan_kernel     per item and range of tokens: base-2 scores from the tables and the
//      per-codeword weight histograms W_s[c][row] = sum over the tokens with zv_s = c of
//      2^(score - ref).  Each (range, item) writes one slot.
//   3. tree_contract_kernel joins the slots of an item and contracts W_s with the value codebooks:
//      one part per (stage, half of the codewords).
//   4. tree_finish_kernel   sums the parts, rotates back, joins the dense part by log-sum-exp.
//
// Why tables and histograms here too: with R rows a (token, pair) costs R (Sk + Sv) / 32 shared-memory
// passes of 128 bytes, gathers and counter additions together.  Reconstructing its key and value for
// float32-accurate matrix products costs (Sk + Sv) d / 32 passes to gather float32 codewords and d / 16
// to write the split vectors, whatever R is, and the codebooks of more than one stage do not fit in
// shared memory.  So the histogram form is the cheaper one up to about R = d.  Wider trees take it too: the
// other form would be the cheaper one there by this count, and has not been built.
//
// Measured (B200), a call among others: 8 sequences x 32640 tokens, 32 / 8 heads, d = 128, 4 + 4 stages,
// 16 drafts 264 us (split 7, tables 20, dense 17, scan 209, contraction 27, finish 9, each alone and cold;
// partly side by side); one sequence x 130816 tokens, 28 / 4 heads, 2 + 4 stages, 25 drafts 148 us;
// 64 ragged sequences of 1024 .. 16384 tokens, 5 drafts 369 .. 382 us; one head, 960 tokens, 8 drafts 26 us,
// the latency of five dependent launches.  Rows of absent drafts are scanned and contracted like others.
#include "query_tables.cuh"
#include "tree_tables_tc.cuh"

#include <algorithm>
#include <cmath>
#include <cstddef>
#include <type_traits>

namespace zkv {

constexpr int kTreeRG = 8;           // query rows per item
constexpr int kTreeUnit = 128;       // tokens per unit of the partition
constexpr int kTreeMinUnits = 2;     // smallest range of a scan block, in units
constexpr int kTreeHalves = 2;       // codeword chunks per stage in the contraction
constexpr int kTreeCw = kCodebook / kTreeHalves;
constexpr int kTreeTK = 16;          // tokens per thread and tile
constexpr size_t kTreeSmemMax = 227 * 1024;

struct TreeArgs {
  QueryTables qt;
  int B, N, G, Hq, Hkv, Sk, Sv, R, RP, NRG, grid;
  int64_t Tcap, Wcap, max_comp;
  const int32_t* n_draft;
  const __half *dk, *dv;
  int64_t k_sb, k_sn, k_sh, v_sb, v_sn, v_sh;
  const uint8_t* mask;
  int64_t m_sb, m_sn;
  const uint8_t *k_codes, *v_codes;
  const int32_t* comp_len;
  const float* Cv;
  const __half *win_k, *win_v;
  const int32_t* win_len;
  float *out, *lse;
  int32_t* err;
  const int32_t* table;
  int64_t max_pages, n_pages;
  int pshift;
  // workspace
  int64_t* pre;            // [B + 1] units of one item of the sequences before b; then the range
  SplitBooks vbooks;       // of Cv, or null planes
  float *pw, *pm;          // slots: [slot][Sv][256][8] weights, [slot][8] references
  float *dm, *dl, *dout;   // dense part per row: maximum (log2), sum, output [D]
  float *parts;            // [Sv * halves][row][D]
  float *rm, *rl;          // [row] maximum, [halves][row] sums
};

// compressed tokens of sequence b that the call reads
__device__ __forceinline__ int64_t comp_tokens(const int32_t* comp_len, int b, int64_t Tcap,
                                               int64_t max_comp) {
  int64_t c = comp_len[b];
  c = c < 0 ? 0 : c > Tcap ? Tcap : c;
  return c < max_comp ? c : max_comp;
}

// ---------------------------------------------------------------------------------------------
// 1. Tables, dense part, partition
// ---------------------------------------------------------------------------------------------

constexpr int kTreeDenseThreads = 128;
constexpr int kTreeDenseRows = 16;    // query rows of a dense block
constexpr int kTreeDenseKeys = 64;    // keys per step, 16 per warp
constexpr float kTreeDenseUp = 32768.f;   // of the weights in the products: 2^15 is the largest, 2^-40 the last

template <int D>
struct TreeDenseSmem {
  __half q[kTreeDenseRows * D];
  __half k[kTreeDenseKeys * D];
  __half v[kTreeDenseKeys * D];
  unsigned long long see[kTreeDenseRows];   // the keys of the step that a row attends to
  float ml[4][kTreeDenseRows][2];           // maximum and sum of each warp's keys
  int odd;                                  // a draft's value holds an infinity or NaN
};

// prefix sums of the sequences' units and the range of one scan block (at least kTreeMinUnits)
__device__ __forceinline__ void tree_partition(const TreeArgs& a) {
  constexpr int T = kTreeDenseThreads;
  __shared__ int64_t ws[T / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int64_t base = 0;
  for (int b0 = 0; b0 < a.B; b0 += T) {
    const int b = b0 + tid;
    int64_t u = 0;
    if (b < a.B) {
      const int64_t c = a.comp_len[b];
      if (c < 0 || c > a.Tcap) set_error(a.err, ZKV_DEVERR_COMP_LEN);
      const int64_t w = a.win_len[b];
      if (w < 0 || w > a.Wcap) set_error(a.err, ZKV_DEVERR_WIN_LEN);
      if (a.n_draft && (a.n_draft[b] < 0 || a.n_draft[b] > a.N)) set_error(a.err, ZKV_DEVERR_DRAFT);
      u = (comp_tokens(a.comp_len, b, a.Tcap, a.max_comp) + kTreeUnit - 1) / kTreeUnit;
    }
    int64_t s = u;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += x;
    }
    if (lane == 31) ws[warp] = s;
    __syncthreads();
    int64_t before = base, all = 0;
    for (int w = 0; w < T / 32; ++w) {
      if (w < warp) before += ws[w];
      all += ws[w];
    }
    if (b < a.B) a.pre[b] = before + s - u;
    base += all;
    __syncthreads();
  }
  if (tid == 0) {
    a.pre[a.B] = base;
    const int64_t total = base * a.Hkv * a.NRG;
    const int64_t per = (total + a.grid - 1) / a.grid;
    a.pre[a.B + 1] = per < kTreeMinUnits ? kTreeMinUnits : per;
  }
}

// Dense attention of 16 rows of a pair over its window and its drafts: one pass over the keys in
// steps of 64, 16 keys per warp with running maxima and sums of the warp's own; the four warps are
// joined at the end (64 rows per block and one warp per 16 rows: 38 us instead of 15 us at 64 pairs,
// 64 rows, 144 keys: the chain of steps of one warp is what takes time).  Queries, keys and values are fp16 and their products exact; the weights, times
// 2^15, are split into two fp16 planes, and every 16 products are added up in float32.  (fp16 ends at
// 2^-25: without the factor every key lighter than that of its warp's heaviest was lost, with 4095 keys
// of 2^-25.5 and eight times its value 1.6e-4 of the output.)
template <int D>
__device__ __forceinline__ void tree_dense(const TreeArgs& a, int64_t blk, TreeDenseSmem<D>& sm) {
  constexpr int NT = D / 8;                    // output tiles of 8 columns
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t4 = lane & 3;
  const int tiles = (a.R + kTreeDenseRows - 1) / kTreeDenseRows;
  const int row0 = (int)(blk % tiles) * kTreeDenseRows;
  const int64_t pair = blk / tiles;
  const int b = (int)(pair / a.Hkv), kvh = (int)(pair % a.Hkv);
  const int nd = present_queries(a.n_draft, b, a.N);
  int64_t wl = a.win_len[b];
  wl = wl < 0 ? 0 : wl > a.Wcap ? a.Wcap : wl;
  if (row0 / a.G >= nd) return;                // no row of the block is present (block-uniform)
  const uint4 zero = make_uint4(0, 0, 0, 0);
  for (int f = tid; f < kTreeDenseRows * (D / 8); f += kTreeDenseThreads) {
    const int r = f / (D / 8), c = (f % (D / 8)) * 8, rho = row0 + r;
    __half* dst = sm.q + tile_at<D>(r, c);
    if (rho < a.R && rho / a.G < nd)
      cp_async16(dst, a.qt.q + b * a.qt.q_sb + (rho / a.G) * a.qt.q_sn +
                          ((int64_t)kvh * a.G + rho % a.G) * a.qt.q_sh + c);
    else
      *reinterpret_cast<uint4*>(dst) = zero;
  }
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};     // rows g and g + 8
  float o[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) o[n][i] = 0.f;
  const int64_t nk = wl + nd;
  for (int64_t k0 = 0; k0 < nk; k0 += kTreeDenseKeys) {
    __syncthreads();                           // the previous keys have been read
    if (tid == 0 && k0 == 0) sm.odd = 0;
    for (int f = tid; f < kTreeDenseKeys * (D / 8); f += kTreeDenseThreads) {
      const int r = f / (D / 8), c = (f % (D / 8)) * 8, at = tile_at<D>(r, c);
      const int64_t t = k0 + r;
      if (t < nk) {
        const __half *ks, *vs;
        if (t < wl) {
          ks = a.win_k + (pair * a.Wcap + t) * D;
          vs = a.win_v + (pair * a.Wcap + t) * D;
        } else {
          ks = a.dk + b * a.k_sb + (t - wl) * a.k_sn + (int64_t)kvh * a.k_sh;
          vs = a.dv + b * a.v_sb + (t - wl) * a.v_sn + (int64_t)kvh * a.v_sh;
        }
        cp_async16(sm.k + at, ks + c);
        cp_async16(sm.v + at, vs + c);
      } else {
        *reinterpret_cast<uint4*>(sm.k + at) = zero;
        *reinterpret_cast<uint4*>(sm.v + at) = zero;
      }
    }
    cp_async_commit();
    // warp w finds the keys that rows 4 w .. 4 w + 3 attend to
    bool see[4][2];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int rho = row0 + 4 * warp + r, i = rho / a.G;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int64_t t = k0 + 32 * q + lane, x = t - wl;
        see[r][q] = rho < a.R && i < nd && t < nk;
        if (see[r][q] && x >= 0) see[r][q] = a.mask ? a.mask[b * a.m_sb + i * a.m_sn + x] != 0 : x <= i;
      }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const unsigned lo = __ballot_sync(0xffffffffu, see[r][0]), hi = __ballot_sync(0xffffffffu, see[r][1]);
      if (lane == 0) sm.see[4 * warp + r] = (unsigned long long)hi << 32 | lo;
    }
    cp_async_wait_all();
    __syncthreads();
    // a draft that a row does not see must not reach it through 0 * infinity: what is not finite is
    // taken out of the products and added at the end to the rows that see it
    if (k0 + kTreeDenseKeys > wl) {
      for (int f = tid; f < kTreeDenseKeys * (D / 8); f += kTreeDenseThreads) {
        uint4& x = *reinterpret_cast<uint4*>(sm.v + tile_at<D>(f / (D / 8), (f % (D / 8)) * 8));
        uint32_t y[4] = {x.x, x.y, x.z, x.w};
        bool any = false;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if ((y[q] & 0x7c00u) == 0x7c00u) y[q] &= 0xffff0000u, any = true;
          if ((y[q] & 0x7c000000u) == 0x7c000000u) y[q] &= 0xffffu, any = true;
        }
        if (any && k0 + f / (D / 8) >= wl) {
          x = make_uint4(y[0], y[1], y[2], y[3]);
          sm.odd = 1;
        }
      }
      __syncthreads();
    }
    uint32_t bits[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) bits[q] = (uint32_t)(sm.see[g + 8 * q] >> (16 * warp)) & 0xffffu;
    if (!__any_sync(0xffffffffu, bits[0] | bits[1])) continue;
    float s[2][4];
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[n][i] = 0.f;
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      uint32_t qf[4], kf[4];
      frag_a<D>(qf, sm.q, 0, ks, lane);
      frag_b<D>(kf, sm.k, 16 * warp, ks, lane);
      mma16816_add(s[0], qf, kf[0], kf[1]);
      mma16816_add(s[1], qf, kf[2], kf[3]);
    }
    float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool sees = bits[i >> 1] >> (8 * n + 2 * t4 + (i & 1)) & 1u;
        s[n][i] = sees ? s[n][i] * a.qt.scale_log2 : -INFINITY;
        mx[i >> 1] = fmaxf(mx[i >> 1], s[n][i]);
      }
    float ref[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      mx[q] = fmaxf(mx[q], __shfl_xor_sync(0xffffffffu, mx[q], 1));
      mx[q] = fmaxf(mx[q], __shfl_xor_sync(0xffffffffu, mx[q], 2));
      const float mn = fmaxf(m[q], mx[q]);
      ref[q] = mn == -INFINITY ? 0.f : mn;
      const float corr = ex2_approx(m[q] - ref[q]);
      m[q] = mn;
      l[q] *= corr;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        o[n][2 * q] *= corr;
        o[n][2 * q + 1] *= corr;
      }
    }
    // the weights of the warp's 16 keys as an A operand: high and low plane
    uint32_t ph[4], pl[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x = ex2_approx(s[i >> 1][2 * (i & 1)] - ref[i & 1]);
      const float y = ex2_approx(s[i >> 1][2 * (i & 1) + 1] - ref[i & 1]);
      l[i & 1] += x + y;
      const float xs = x * kTreeDenseUp, ys = y * kTreeDenseUp;
      const __half2 hi = __floats2half2_rn(xs, ys);
      const float2 back = __half22float2(hi);
      const __half2 lo = __floats2half2_rn(xs - back.x, ys - back.y);
      ph[i] = *reinterpret_cast<const uint32_t*>(&hi);
      pl[i] = *reinterpret_cast<const uint32_t*>(&lo);
    }
#pragma unroll
    for (int n = 0; n < NT; n += 2) {
      uint32_t vf[4];
      frag_bt<D>(vf, sm.v, 8 * n, warp, lane);
      float t[4], u[4];
      mma16816_zero(t, pl, vf[0], vf[1]);
      mma16816_zero(u, pl, vf[2], vf[3]);
      mma16816(t, ph, vf[0], vf[1]);
      mma16816(u, ph, vf[2], vf[3]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        o[n][i] += t[i];
        o[n + 1][i] += u[i];
      }
    }
  }
  // join the warps, in their order
  float* os = reinterpret_cast<float*>(sm.k);          // [4][16][D]
  static_assert(offsetof(TreeDenseSmem<D>, v) == offsetof(TreeDenseSmem<D>, k) + sizeof(sm.k) &&
                    sizeof(sm.k) + sizeof(sm.v) >= 4 * kTreeDenseRows * D * sizeof(float), "fits");
  __syncthreads();
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int r = g + 8 * q;
    l[q] += __shfl_xor_sync(0xffffffffu, l[q], 1);
    l[q] += __shfl_xor_sync(0xffffffffu, l[q], 2);
    if (t4 == 0) {
      sm.ml[warp][r][0] = m[q];
      sm.ml[warp][r][1] = l[q];
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
      *reinterpret_cast<float2*>(os + (warp * kTreeDenseRows + r) * D + 8 * n + 2 * t4) =
          make_float2(o[n][2 * q], o[n][2 * q + 1]);
  }
  __syncthreads();
  for (int r = warp; r < kTreeDenseRows; r += 4) {
    const int rho = row0 + r, i = rho / a.G;
    if (rho >= a.R || i >= nd) break;
    float top = -INFINITY, sum = 0.f, y[D / 32];
#pragma unroll
    for (int k = 0; k < 4; ++k) top = fmaxf(top, sm.ml[k][r][0]);
#pragma unroll
    for (int e = 0; e < D / 32; ++e) y[e] = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float f = ex2_approx(sm.ml[k][r][0] - (top == -INFINITY ? 0.f : top));
      sum = fmaf(sm.ml[k][r][1], f, sum);
#pragma unroll
      for (int e = 0; e < D / 32; ++e) y[e] = fmaf(os[(k * kTreeDenseRows + r) * D + e * 32 + lane], f, y[e]);
    }
#pragma unroll
    for (int e = 0; e < D / 32; ++e) y[e] *= 1.f / kTreeDenseUp;
    // An infinity of the window has become NaN in a plane of the weights that is zero: a dimension that
    // holds such values is their sum, whatever the weights are.
#pragma unroll
    for (int e = 0; e < D / 32; ++e)
      if (!(fabsf(y[e]) < INFINITY)) {
        float all = 0.f;
        for (int64_t t = 0; t < wl; ++t) {
          const float v = __half2float(a.win_v[(pair * a.Wcap + t) * D + e * 32 + lane]);
          if (!(fabsf(v) < INFINITY)) all += v;
        }
        if (all != 0.f) y[e] = all;
      }
    if (sm.odd)
      for (int key = 0; key < nd; ++key) {
        if (a.mask ? a.mask[b * a.m_sb + i * a.m_sn + key] == 0 : key > i) continue;
        const __half* vs = a.dv + b * a.v_sb + key * a.v_sn + (int64_t)kvh * a.v_sh + lane;
#pragma unroll
        for (int e = 0; e < D / 32; ++e) {
          const float v = __half2float(vs[e * 32]);
          if (!(fabsf(v) < INFINITY)) y[e] += v;
        }
      }
    const int64_t row = pair * a.RP + rho;
    if (lane == 0) {
      a.dm[row] = top;
      a.dl[row] = sum;
    }
#pragma unroll
    for (int e = 0; e < D / 32; ++e) a.dout[row * D + e * 32 + lane] = y[e];
  }
}

template <int D>
__global__ void __launch_bounds__(kTreeDenseThreads) tree_dense_kernel(TreeArgs a) {
  extern __shared__ __align__(16) unsigned char smraw[];
  pdl_trigger();
  TreeDenseSmem<D>& sm = *reinterpret_cast<TreeDenseSmem<D>*>(smraw);
  const int64_t blk = (int64_t)blockIdx.x - 1;
  if (blk < 0) tree_partition(a);
  else tree_dense<D>(a, blk, sm);
  pdl_wait();      // (after a normal launch it returns at once)
}

// The key and value codewords split once, 64 a block, for the blocks of the tables and the contraction
template <int D>
__global__ void __launch_bounds__(kQtThreads) tree_split_kernel(TreeArgs a) {
  pdl_trigger();
  const int64_t keys = (int64_t)a.Hkv * a.Sk * (kCodebook / 64), blk = blockIdx.x;
  if (blk < keys) split_books_block<D>(a.qt.Ck, a.qt.books, blk * 64);
  else split_books_block<D>(a.Cv, a.vbooks, (blk - keys) * 64);
}

// Few rows: runs beside the dense part, which it does not read, and completes after it
template <int D>
__global__ void __launch_bounds__(kQtThreads) tree_tables_kernel(TreeArgs a) {
  extern __shared__ __align__(16) unsigned char smraw[];
  pdl_trigger();
  query_tables_block<D>(a.qt, blockIdx.x, *reinterpret_cast<QtSmem<D>*>(smraw));
  pdl_wait();
}

// Many rows, after the split kernel
template <int D>
__global__ void __launch_bounds__(kTtThreads, 1) tree_tables_tc_kernel(TreeArgs a, int shares) {
  extern __shared__ __align__(16) unsigned char smraw[];
  pdl_trigger();
  TtSmem<D>& sm = *reinterpret_cast<TtSmem<D>*>((reinterpret_cast<uintptr_t>(smraw) + 1023) & ~uintptr_t(1023));
  tree_tables_tc<D>(a.qt, blockIdx.x, shares, sm, a.err);
}

// ---------------------------------------------------------------------------------------------
// 2. Scan
// ---------------------------------------------------------------------------------------------
// Lane = (token slot h = lane / 4, row pair r = lane % 4); a thread takes kTreeTK tokens of a tile
// for rows 2 r and 2 r + 1.  Shared memory holds 256 rows (codewords) of 256 bytes: bytes [0, 128)
// the key table entries [stage][copy][row] of the codeword, bytes [128, 256) its weight counters, so
// that the address of either is one byte permutation [column | code] of the packed codes.  With 8
// stages on either side each kind has 256-byte rows of its own.  Slot h visits the stages in the
// order s = i ^ (h % 4) (fewer than four stages: copies) and slots 4 .. 7 add their odd row first, so
// the lanes of every gather phase and of every counter addition lie in distinct banks, whatever the
// codes are.
//
// Weights.  p = 2^(score - ref) with ref the row's maximum over the first tokens of the segment.  The block sums p
// per row over the tile before it adds any (one barrier), so a row's unit can be chosen: a power
// of two with the first tile's sum at 2^27 .. 2^28 units.  Counters then take u = floor(p / unit + d)
// as exact integers in any order; when the sum of a row could pass 2^32 the counters are folded
// into the slot (float32) and the unit chosen anew.  d in [0, 1) is an offset of the token's place:
// the 8 slots x NW warps of a tile have equally spaced ones, which turn from tile to tile, so that
// equal weights below a unit are counted as often as their sum asks for.  (Rounding to the nearest
// loses them all: for a first token and 32639 of 2^-28.1 of its weight each that is 1.1e-4 of the
// sum and 1.6e-4 of the output, with the offsets 2e-7 and nothing in the float32 lse; the times are
// the same.)  A weight is off by less than a unit, 2^-27 of a tile's sum, its mean over the places by
// nothing; no weight (p = 0) counts nothing.  A tile whose sum is above 2^64 is
// folded against its own maximum as the new ref.
//
// Bound: the shared-memory pipe.  At 8 x 32640 tokens, 64 rows: 209 us, 76 % of its passes used (40.5 M
// of gathers, code reads and additions, 42.7 M with the copies), 57 % of the issue slots, 2 CTAs of 12 warps
// per SM.  Steps
// measured on that case: one row per lane 275 us; two rows per lane (half the address permutations and
// code reads) with the codes copied ahead into shared memory instead of registers 185 us beside the
// tables; 8 instead of 12 warps 6 % slower; 8 instead of 16 tokens per thread 30 % slower (the exchange
// of sums per tile).
template <int SKP, int SVP>
struct TreeScan {
  static constexpr bool WIDE = SKP == 8 || SVP == 8;
  static constexpr int NW = WIDE ? 16 : 12;         // warps
  static constexpr int THREADS = NW * 32;
  static constexpr int TILE = NW * 8 * kTreeTK;     // tokens
  static constexpr int VOFF = WIDE ? 65536 : 128;   // weight counters of a codeword
  static constexpr int KR = SKP >= 4 ? 1 : 4 / SKP; // copies
  static constexpr int VR = SVP >= 4 ? 1 : 4 / SVP;
  static constexpr int TABLES = WIDE ? 131072 : 65536;
  static constexpr int SUMS = 2 * kTreeRG * NW * 4;
  static constexpr int CODES = 32 * (kTreeTK / 4) * (SKP + SVP);   // bytes of a warp's part of a tile
  static constexpr int SMEM = TABLES + SUMS + 2 * NW * CODES;
  static constexpr int KW = SKP <= 4 ? 1 : 2, VW = SVP <= 4 ? 1 : 2;   // code words per token

  // Offsets of the roundings in units of 2^-32: place (slot h, warp w) is one of 8 NW equal steps,
  // with the slots of a warp and the warps of a slot spread over all of them, too.
  static constexpr uint32_t STEP = 0x80000000u / (4 * NW);
  __device__ __forceinline__ static uint32_t place(uint32_t h, uint32_t w) {
    const uint32_t at = NW == 12 ? 4u * ((3u * h + 2u * w) % 24u) + (h >> 1) : 8u * ((2u * h + w) % 16u) + h;
    return at * STEP + STEP / 2;
  }
  // The turn from tile to tile, near the golden ratio's 0.618 and such that the steps themselves
  // move by 0.618 of one (59.618 / 96, 79.618 / 128)
  static constexpr uint32_t TURN = NW == 12 ? 2667265689u : 2671537907u;
};

// The codes of four tokens from the warp's copy (p: the first one's S bytes; 4-byte aligned).  EXACT:
// rows are SP bytes.
template <int SP, int W, bool EXACT>
__device__ __forceinline__ void read_four(const unsigned char* p, int S, uint32_t (&w)[4][W]) {
  const uint32_t* p4 = reinterpret_cast<const uint32_t*>(p);
  if constexpr (SP == 1) {
    const uint32_t x = *p4;
#pragma unroll
    for (int u = 0; u < 4; ++u) w[u][0] = (x >> (8 * u)) & 255u;
  } else if constexpr (SP == 2) {
    const uint2 x = *reinterpret_cast<const uint2*>(p);
    w[0][0] = x.x & 0xffffu; w[1][0] = x.x >> 16;
    w[2][0] = x.y & 0xffffu; w[3][0] = x.y >> 16;
  } else if constexpr (SP == 4) {
    if (EXACT || S == 4) {
      const uint4 x = *reinterpret_cast<const uint4*>(p);
      w[0][0] = x.x; w[1][0] = x.y; w[2][0] = x.z; w[3][0] = x.w;
    } else {
      const uint32_t x = p4[0], y = p4[1], z = p4[2];
      w[0][0] = x & 0xffffffu;
      w[1][0] = __funnelshift_r(x, y, 24) & 0xffffffu;
      w[2][0] = __funnelshift_r(y, z, 16) & 0xffffffu;
      w[3][0] = z >> 8;
    }
  } else if (EXACT || S == 8) {
    const uint4 x = reinterpret_cast<const uint4*>(p)[0], y = reinterpret_cast<const uint4*>(p)[1];
    w[0][0] = x.x; w[0][W - 1] = x.y; w[1][0] = x.z; w[1][W - 1] = x.w;
    w[2][0] = y.x; w[2][W - 1] = y.y; w[3][0] = y.z; w[3][W - 1] = y.w;
  } else {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      w[u][0] = w[u][W - 1] = 0u;
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (q < S) w[u][q < 4 ? 0 : W - 1] |= (uint32_t)p[u * S + q] << (8 * (q & 3));
    }
  }
}

template <int SKP, int SVP, bool PAGED>
__global__ void __launch_bounds__(TreeScan<SKP, SVP>::THREADS, TreeScan<SKP, SVP>::WIDE ? 1 : 2)
    tree_scan_kernel(TreeArgs a) {
  using C = TreeScan<SKP, SVP>;
  extern __shared__ __align__(16) unsigned char sm[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r = lane & 3, h = lane >> 2;
  float* sums = reinterpret_cast<float*>(sm + C::TABLES);                    // [2][8][NW]
  unsigned char* codes = sm + C::TABLES + C::SUMS + warp * 2 * C::CODES;     // this warp's [2][K, V]
  pdl_trigger();
  // the weight counters start at zero and every fold leaves them at zero
  for (int f = tid; f < kCodebook * 8; f += C::THREADS) {
    unsigned char* z = sm + C::VOFF + 256 * (f >> 3) + 16 * (f & 7);
    *reinterpret_cast<uint4*>(z) = make_uint4(0, 0, 0, 0);
    if (SVP == 8) *reinterpret_cast<uint4*>(z + 128) = make_uint4(0, 0, 0, 0);
  }
  // per-lane columns of step i of the stage loop (byte i & 1; bytes 2 and 3 zero); v: first and second
  // row of the pair.  A token's code word is first put into the lane's stage order (korder, vorder),
  // so that the selectors of the address permutations are constants.
  uint32_t kcol[(SKP + 1) / 2], vcol[2][(SVP + 1) / 2], korder = 0u, vorder = 0u;
  const uint32_t h4 = (uint32_t)h & 3u, swap = (uint32_t)h >> 2;
#pragma unroll
  for (int i = 0; i < (SKP + 1) / 2; ++i) kcol[i] = 0u;
#pragma unroll
  for (int i = 0; i < (SVP + 1) / 2; ++i) vcol[0][i] = vcol[1][i] = 0u;
#pragma unroll
  for (int i = 0; i < SKP; ++i) {
    const uint32_t s = ((uint32_t)i ^ h4) & (SKP - 1), rep = SKP >= 4 ? 0u : h4 / SKP;
    kcol[i / 2] |= ((s * C::KR + rep) * 32u + r * 8u) << (8 * (i & 1));
    if (i < 4) korder |= (s & 3u) << (4 * i);
  }
#pragma unroll
  for (int i = 0; i < SVP; ++i) {
    const uint32_t s = ((uint32_t)i ^ h4) & (SVP - 1), rep = SVP >= 4 ? 0u : h4 / SVP;
#pragma unroll
    for (uint32_t v = 0; v < 2; ++v)
      vcol[v][i / 2] |= ((s * C::VR + rep) * 32u + r * 8u + (v ^ swap) * 4u) << (8 * (i & 1));
    if (i < 4) vorder |= (s & 3u) << (4 * i);
  }
  // (kept in registers: not worth computing again in every tile)
  asm volatile("" : "+r"(korder), "+r"(vorder));
#pragma unroll
  for (int i = 0; i < (SKP + 1) / 2; ++i) asm volatile("" : "+r"(kcol[i]));
#pragma unroll
  for (int i = 0; i < (SVP + 1) / 2; ++i) asm volatile("" : "+r"(vcol[0][i]), "+r"(vcol[1][i]));
  const uint32_t place = C::place((uint32_t)h, (uint32_t)warp);
  pdl_wait();
  const int64_t per = a.pre[a.B + 1];
  const int64_t items_per_b = (int64_t)a.Hkv * a.NRG;
  const int64_t total = a.pre[a.B] * items_per_b;
  int64_t lo = blockIdx.x * per;
  const int64_t hi = lo + per < total ? lo + per : total;
  if (lo >= hi) return;
  if ((uint32_t)__cvta_generic_to_shared(sm) != kTableBase) {   // (the slots stay unwritten)
    if (tid == 0) set_error(a.err, ZKV_DEVERR_SMEM);
    return;
  }
  // the sequence of the first unit: the last b with pre[b] * items_per_b <= lo (32 at a time: the
  // prefix sums do not fall)
  int b = -1;
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    const unsigned below =
        __ballot_sync(0xffffffffu, b0 + lane < a.B && a.pre[min(b0 + lane, a.B - 1)] * items_per_b <= lo);
    b += __popc(below);
    if (below != 0xffffffffu) break;
  }
  int buf = 0;
  auto load_tables = [&](int64_t item) {      // asynchronous
    const float* t = a.qt.lut + item * (int64_t)(kCodebook * SKP * kTreeRG);
    constexpr int Q = SKP * C::KR * 2;    // 16-byte pieces per codeword
    for (int f = tid; f < kCodebook * Q; f += C::THREADS) {
      const int c = f / Q, q = f % Q, s = (q >> 1) / C::KR;
      cp_async16(sm + 256 * c + 16 * q, t + (c * SKP + s) * kTreeRG + 4 * (q & 1));
    }
  };
  bool first = true;
  while (lo < hi) {
    int64_t base = a.pre[b] * items_per_b, units = a.pre[b + 1] - a.pre[b];
    while (units == 0 || lo >= base + units * items_per_b) {
      ++b;
      base = a.pre[b] * items_per_b;
      units = a.pre[b + 1] - a.pre[b];
    }
    const int64_t in_b = (lo - base) / units;           // item of the sequence
    const int64_t off = lo - base - in_b * units;       // its first unit here
    const int64_t cnt = units - off < hi - lo ? units - off : hi - lo;
    const int64_t item = b * items_per_b + in_b;
    const int kvh = (int)(in_b / a.NRG);
    const int64_t ntok = comp_tokens(a.comp_len, b, a.Tcap, a.max_comp);
    const uint32_t t0 = (uint32_t)(off * kTreeUnit);
    const uint32_t tend = (uint32_t)(ntok < (off + cnt) * kTreeUnit ? ntok : (off + cnt) * kTreeUnit);
    const CodeRows kr = code_rows(a.k_codes, a.table, a.max_pages, a.n_pages, a.pshift, b, kvh,
                                  a.Hkv, a.Tcap, a.Sk, a.err);
    const CodeRows vr = code_rows(a.v_codes, a.table, a.max_pages, a.n_pages, a.pshift, b, kvh,
                                  a.Hkv, a.Tcap, a.Sv, a.err);
    // the item of the block's next segment (this one's item ends here if there is one)
    int64_t next = -1;
    if (lo + cnt < hi) {
      next = item + 1;
      if (in_b + 1 == items_per_b)
        for (int x = b + 1; a.pre[x + 1] == a.pre[x]; ++x) next += items_per_b;
    }
    if (first) load_tables(item);
    first = false;
    cp_async_wait_all();
    __syncthreads();

    // state of this thread's two rows (the same in every thread that has them)
    float ref[2] = {0.f, 0.f};     // (NaN from the first sum on that is not finite: the row is lost)
    float scale[2] = {1.f, 1.f}, used[2] = {0.f, 0.f};     // 1 / unit; the sum since the last fold
    bool chosen = false, dirty = false, folded = false;
    float* slot = a.pw + (item + blockIdx.x) * (int64_t)(a.Sv * kCodebook * kTreeRG);
    const bool exact = a.Sk == SKP && a.Sv == SVP;
    auto first_of = [&](uint32_t tile, int k) { return tile + ((k * C::NW + warp) * 8 + h) * 4; };

    // scores of a token for this lane's rows, less the references
    auto score = [&](const uint32_t (&w)[C::KW], float2 neg_ref) {
      float2 s = neg_ref;
      uint32_t x[C::KW];
#pragma unroll
      for (int i = 0; i < C::KW; ++i) x[i] = byte_perm(w[i], 0u, korder);
#pragma unroll
      for (int i = 0; i < SKP; ++i)
        s = fadd2(s, lds_pair(byte_perm(x[i < 4 ? 0 : C::KW - 1], kcol[i / 2],
                                        (4u + (i & 1)) | ((i & 3u) << 4) | 0x7600u)));
      return s;
    };
    // the value of row x = lane % 8 from the threads that have it
    auto of_row = [&](const float (&v)[2]) {
      const float v0 = __shfl_sync(0xffffffffu, v[0], (lane & 7) >> 1);
      const float v1 = __shfl_sync(0xffffffffu, v[1], (lane & 7) >> 1);
      return lane & 1 ? v1 : v0;
    };
    // counters -> slot, times f (a reference that was raised); lane = word of the codeword's 128-byte
    // row: stage (or copy) lane / 8, row lane % 8
    auto fold = [&](const float (&factor)[2]) {
      // unit = 1 / scale, a power of two
      const float f = of_row(factor), un = __uint_as_float(0x7F000000u - __float_as_uint(of_row(scale)));
      const int col = lane >> 3;
#pragma unroll 4
      for (int c = warp; c < kCodebook; c += C::NW) {
#pragma unroll
        for (int q = 0; q < (SVP == 8 ? 2 : 1); ++q) {
          const int s = (SVP >= 4 ? col : col / C::VR) + 4 * q;
          uint32_t* p = reinterpret_cast<uint32_t*>(sm + C::VOFF + 256 * c + 128 * q) + lane;
          float v = 0.f;
          if (dirty) {
            v = (float)*p;
            *p = 0u;
            if (SVP <= 2) v += __shfl_xor_sync(0xffffffffu, v, 8);      // copies of one counter
            if (SVP == 1) v += __shfl_xor_sync(0xffffffffu, v, 16);
            v *= un;
          }
          if (s < a.Sv && (C::VR == 1 || col % C::VR == 0)) {
            float* o = slot + ((s * kCodebook + c) * kTreeRG + (lane & 7));
            *o = (folded ? v + *o : v) * f;
          }
        }
      }
      folded = true;
      dirty = false;
    };
    // one value per row and thread -> one per row and warp (op) -> x of the block's rows; a barrier
    auto exchange = [&](float2 v, auto op, float (&x)[2]) {
      float t = (h & 1) ? v.x : v.y, k = (h & 1) ? v.y : v.x;      // lane keeps row 2 r + h % 2
      k = op(k, __shfl_xor_sync(0xffffffffu, t, 4));
      k = op(k, __shfl_xor_sync(0xffffffffu, k, 8));
      k = op(k, __shfl_xor_sync(0xffffffffu, k, 16));
      if (h < 2) sums[(buf * kTreeRG + 2 * r + h) * C::NW + warp] = k;
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float* p = sums + (buf * kTreeRG + 2 * r + j) * C::NW;
#pragma unroll
        for (int w = 0; w < C::NW; w += 4) {
          const float4 s4 = *reinterpret_cast<const float4*>(p + w);
          const float y = op(op(s4.x, s4.y), op(s4.z, s4.w));
          x[j] = w ? op(x[j], y) : y;
        }
      }
      buf ^= 1;      // the next exchange's barrier lies between two uses of a buffer
    };
    auto add = [](float x, float y) { return x + y; };
    auto larger = [](float x, float y) { return fmaxf(x, y); };

    // This warp's codes of a tile, copied ahead in 16-byte pieces: 32 tokens in a row for each k, a
    // multiple of 16 bytes whatever S is (capacities and pages are multiples of 16 tokens, so a piece
    // neither crosses a page nor leaves the array).  Pieces behind the last token are not copied.
    auto fetch_kind = [&](auto sc, const CodeRows& rows, int Srt, uint32_t tile, unsigned char* dst) {
      const int S = decltype(sc)::value ? decltype(sc)::value : Srt;
      for (int x = lane; x < 2 * S * (kTreeTK / 4); x += 32) {
        const int k = x / (2 * S), piece = x - k * 2 * S;
        const uint32_t first = tile + (k * C::NW + warp) * 32;
        const uint64_t byte = (uint64_t)first * S + 16 * piece;
        if (byte >= (uint64_t)tend * S) continue;
        const uint8_t* src = rows.base + byte;
        if constexpr (PAGED) {
          const uint32_t t = first + 16 * piece / S, t0p = t >> rows.pshift << rows.pshift;
          src = rows.row(t0p, S);
          if (!src) {
            *reinterpret_cast<uint4*>(dst + 16 * x) = make_uint4(0, 0, 0, 0);
            continue;
          }
          src += byte - (uint64_t)t0p * S;
        }
        cp_async16(dst + 16 * x, src);
      }
    };
    auto fetch = [&](uint32_t tile, int q) {
      unsigned char *dk = codes + q * C::CODES, *dv = dk + 32 * (kTreeTK / 4) * SKP;
      if (tile < tend) {
        if (exact) {
          fetch_kind(std::integral_constant<int, SKP>{}, kr, 0, tile, dk);
          fetch_kind(std::integral_constant<int, SVP>{}, vr, 0, tile, dv);
        } else {
          fetch_kind(std::integral_constant<int, 0>{}, kr, a.Sk, tile, dk);
          fetch_kind(std::integral_constant<int, 0>{}, vr, a.Sv, tile, dv);
        }
      }
      cp_async_commit();
    };
    auto key_codes = [&](auto ex, int q, int k, uint32_t (&w)[4][C::KW]) {
      const int S = decltype(ex)::value ? SKP : a.Sk;
      read_four<SKP, C::KW, decltype(ex)::value>(codes + q * C::CODES + (32 * k + 4 * h) * S, S, w);
    };
    auto value_codes = [&](auto ex, int q, int k, uint32_t (&w)[4][C::VW]) {
      const int S = decltype(ex)::value ? SVP : a.Sv;
      read_four<SVP, C::VW, decltype(ex)::value>(
          codes + q * C::CODES + 32 * (kTreeTK / 4) * SKP + (32 * k + 4 * h) * S, S, w);
    };
    // the rows' largest scores of the tile's first tokens (groups of 32 per warp)
    auto tile_max = [&](uint32_t tile, int q, int groups, float (&x)[2]) {
      float2 mx = make_float2(-INFINITY, -INFINITY);
#pragma unroll 1
      for (int k = 0; k < groups && tile + (k * C::NW + warp) * 32 < tend; ++k) {
        uint32_t w[4][C::KW];
        key_codes(std::false_type{}, q, k, w);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float2 s = score(w[u], make_float2(0.f, 0.f));
          if (first_of(tile, k) + u < tend) mx = make_float2(fmaxf(mx.x, s.x), fmaxf(mx.y, s.y));
        }
      }
      exchange(mx, larger, x);
    };
    // p of this thread's tokens of a tile and their sums
    auto tile_scores = [&](auto full, uint32_t tile, int q, float2 (&p)[kTreeTK]) {
      constexpr bool FULL = decltype(full)::value;
      float2 sum = make_float2(0.f, 0.f);
      const float2 neg = make_float2(-ref[0], -ref[1]);
#pragma unroll
      for (int k = 0; k < kTreeTK / 4; ++k) {
        if (!FULL && tile + (k * C::NW + warp) * 32 >= tend) {     // none of the warp's tokens left
#pragma unroll
          for (int u = 0; u < 4; ++u) p[4 * k + u] = make_float2(0.f, 0.f);
          continue;
        }
        uint32_t w[4][C::KW];
        key_codes(full, q, k, w);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          float2 x = score(w[u], neg);
          if constexpr (!FULL)
            if (first_of(tile, k) + u >= tend) x = make_float2(-INFINITY, -INFINITY);
          p[4 * k + u] = make_float2(ex2_ftz(x.x), ex2_ftz(x.y));
          sum = fadd2(sum, p[4 * k + u]);
        }
      }
      return sum;
    };
    auto tile_add = [&](auto ex, uint32_t tile, int q, const float2 (&p)[kTreeTK], const float (&mul)[2]) {
      const float off = (float)((place + (tile - t0) / C::TILE * C::TURN) >> 8) * 0x1p-24f;     // below 1
#pragma unroll
      for (int k = 0; k < kTreeTK / 4; ++k) {
        if (tile + (k * C::NW + warp) * 32 >= tend) break;
        uint32_t w[4][C::VW];
        value_codes(ex, q, k, w);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const uint32_t u0 = __float2uint_rd(fmaf(p[4 * k + u].x, mul[0], off));
          const uint32_t u1 = __float2uint_rd(fmaf(p[4 * k + u].y, mul[1], off));
          const uint32_t ua = swap ? u1 : u0, ub = swap ? u0 : u1;
          uint32_t x[C::VW];
#pragma unroll
          for (int i = 0; i < C::VW; ++i) x[i] = byte_perm(w[u][i], 0u, vorder);
#pragma unroll
          for (int i = 0; i < SVP; ++i) {
            const uint32_t y = x[i < 4 ? 0 : C::VW - 1], sel = (4u + (i & 1)) | ((i & 3u) << 4) | 0x7600u;
            red_counter<C::VOFF>(byte_perm(y, vcol[0][i / 2], sel), ua);
            red_counter<C::VOFF>(byte_perm(y, vcol[1][i / 2], sel), ub);
          }
        }
      }
    };

    fetch(t0, 0);
    cp_async_wait_all();
    __syncwarp();
    tile_max(t0, 0, 1, ref);
#pragma unroll
    for (int j = 0; j < 2; ++j)
      if (!(fabsf(ref[j]) < 1e30f)) ref[j] = 0.f;
    int q = 0;
    for (uint32_t tile = t0; tile < tend; tile += C::TILE, q ^= 1) {
      fetch(tile + C::TILE, q ^ 1);      // (this warp has read that buffer's tile)
      asm volatile("cp.async.wait_group 1;" ::: "memory");
      __syncwarp();
      float2 p[kTreeTK];
      float sum[2];
      for (int again = 0; again < 2; ++again) {
        const float2 s2 = exact && tend - tile >= C::TILE ? tile_scores(std::true_type{}, tile, q, p)
                                                          : tile_scores(std::false_type{}, tile, q, p);
        exchange(s2, add, sum);
        // every warp holds all eight rows and the same sums: the votes agree in the whole block
        const bool up = (sum[0] > 0x1p64f || sum[1] > 0x1p64f) && !again;
        if (!__any_sync(0xffffffffu, up)) break;
        float mx[2], f[2];
        tile_max(tile, q, kTreeTK / 4, mx);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const bool raise = sum[j] > 0x1p64f && mx[j] < 1e30f;
          f[j] = raise ? ex2_ftz(ref[j] - mx[j]) : 1.f;
          if (raise) ref[j] = mx[j];
        }
        fold(f);                   // (all additions of the previous tile came before the barrier)
        chosen = false;
        __syncthreads();           // the counters are zero before anyone adds
      }
      bool bad[2], full = false;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        bad[j] = !(sum[j] < 3e38f);
        if (bad[j]) ref[j] = NAN;
        full = full || (!bad[j] && used[j] + sum[j] * scale[j] + (float)C::TILE > 4.0e9f);
      }
      if (__any_sync(0xffffffffu, full || !chosen)) {
        if (dirty) {
          const float one[2] = {1.f, 1.f};
          fold(one);
          __syncthreads();
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          // sum = m 2^e, m in [1/2, 1): the unit is 2^(e - 28)
          int e = (int)((__float_as_uint(sum[j]) >> 23) & 255u) - 126;
          e = e < -90 ? -90 : e > 100 ? 100 : e;
          scale[j] = __uint_as_float((uint32_t)(28 - e + 127) << 23);
          used[j] = 0.f;
        }
        chosen = true;
      }
      // the segment's last scores have been taken: the next one's tables take their place meanwhile
      if (next >= 0 && tend - tile <= C::TILE) load_tables(next);
      float mul[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        mul[j] = bad[j] ? 0.f : scale[j];        // (inf and NaN times 0 convert to 0)
        used[j] += sum[j] * mul[j] + (float)C::TILE;
      }
      dirty = true;
      if (exact) tile_add(std::true_type{}, tile, q, p, mul);
      else tile_add(std::false_type{}, tile, q, p, mul);
      __syncwarp();        // every lane has read the codes
    }
    __syncthreads();
    const float one[2] = {1.f, 1.f};
    fold(one);
    if (warp == 0 && h == 0)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        a.pm[(item + blockIdx.x) * kTreeRG + 2 * r + j] = ref[j];
    lo += cnt;
  }
}

// ---------------------------------------------------------------------------------------------
// 3. Contraction with the value codebooks
// ---------------------------------------------------------------------------------------------
// 24 us at 512 rows per kv head, 8 heads, 4 stages, d = 128 (float32 FMA form: about 60 us): reading the
// slots, 31 MB, and the join bound it; the tensor pipe is 23 % busy.
// Block = 8 items of one kv head (64 rows) x 128 codewords of one stage: a product
// [64 rows] x [128 codewords] x [D] with float32 accuracy (mma_split.cuh).  The codewords are read
// and split before the wait for the scan.  Warp = item while the slots are joined by their
// references; a weight takes over the power of two of its codeword, then each row is split.  In the
// product 4 x 2 warps take 16 rows x D / 2 dimensions.
template <int D>
struct TreeContractSmem {
  __half cv[2][kTreeCw * D];        // codewords [c][D], high and low plane
  __half w[2][kTreeCw * 64];        // weights [c][64 rows]
  float cs[kTreeCw];                // 2^e of the codewords
  float ws[64];                     // 2^e of the rows
  int64_t row[8];                   // first row of each item, -1: nothing to write
};

template <int D>
__global__ void __launch_bounds__(256, D <= 128 ? 2 : 1) tree_contract_kernel(TreeArgs a) {
  constexpr int E = D / 32;
  extern __shared__ __align__(16) unsigned char smraw[];
  TreeContractSmem<D>& sm = *reinterpret_cast<TreeContractSmem<D>*>(smraw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int parts = a.Sv * kTreeHalves, part = blockIdx.x % parts;
  const int s = part / kTreeHalves, half = part % kTreeHalves;
  const int kvh = blockIdx.y;
  const int64_t group = blockIdx.x / parts;
  const int64_t j = group * 8 + warp;          // (b, rg) of kvh
  pdl_trigger();
  if (a.vbooks.hi) {
    const int64_t row = ((int64_t)kvh * a.Sv + s) * kCodebook + half * kTreeCw;
    pdl_wait();          // (the planes are this call's)
    copy_split<D>(a.vbooks, row, kTreeCw, sm.cv[0], sm.cv[1], 256);
    cp_async_commit();
    if (tid < kTreeCw) sm.cs[tid] = a.vbooks.scale[row + tid];
  } else {
    // warp w splits codewords w, w + 8, ...; lane = E dimensions in a row
    const float* C = a.Cv + (((int64_t)kvh * a.Sv + s) * kCodebook + half * kTreeCw) * D + lane * E;
#pragma unroll 1
    for (int k0 = 0; k0 < kTreeCw / 8; k0 += 8) {
      float v[8][E];
#pragma unroll
      for (int k = 0; k < 8; ++k)
#pragma unroll
        for (int e = 0; e < E; ++e) v[k][e] = __ldg(C + (int64_t)(8 * (k0 + k) + warp) * D + e);
      float part[8], down_of;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        part[k] = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) part[k] = fmaf(v[k][e], v[k][e], part[k]);
      }
      {
        int own = 0;      // the norms of the eight codewords at once
        const int ex = split_exponent(sqrtf(TransposeSum<8, 8, 16>::run(part, lane, own)));
        down_of = exp2_int(-ex);
        sm.cs[8 * (k0 + own) + warp] = exp2_int(ex);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int c = 8 * (k0 + k) + warp;
        const float down = __shfl_sync(0xffffffffu, down_of, sum_owner<8>(k));
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          alignas(4) __half hi[2], lo[2];
          split(v[k][e] * down, hi[0], lo[0]);
          split(v[k][e + 1] * down, hi[1], lo[1]);
          const int at = tile_at<D>(c, lane * E + e);
          *reinterpret_cast<uint32_t*>(sm.cv[0] + at) = *reinterpret_cast<const uint32_t*>(hi);
          *reinterpret_cast<uint32_t*>(sm.cv[1] + at) = *reinterpret_cast<const uint32_t*>(lo);
        }
      }
    }
  }
  __syncthreads();
  pdl_wait();
  const bool live = j < (int64_t)a.B * a.NRG;
  {
    int64_t n = 0, row = -1, slot0 = 0;
    if (live) {
      const int b = (int)(j / a.NRG), rg = (int)(j % a.NRG);
      const int64_t items_per_b = (int64_t)a.Hkv * a.NRG, in_b = (int64_t)kvh * a.NRG + rg;
      const int64_t units = a.pre[b + 1] - a.pre[b], per = a.pre[a.B + 1];
      const int64_t p0 = a.pre[b] * items_per_b + in_b * units;
      const int64_t first = p0 / per;
      n = units ? (p0 + units - 1) / per - first + 1 : 0;
      slot0 = b * items_per_b + in_b + first;
      row = ((int64_t)b * a.Hkv + kvh) * a.RP + rg * kTreeRG;
    }
    // lane holds rows r4 .. r4 + 3 of codewords lane / 2 + 16 k
    const int r4 = 4 * (lane & 1);
    float m[4];
    bool nan[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) m[q] = -INFINITY, nan[q] = false;
#pragma unroll 4
    for (int64_t k = 0; k < n; ++k) {
      const float4 x = *reinterpret_cast<const float4*>(a.pm + (slot0 + k) * kTreeRG + r4);
      m[0] = fmaxf(m[0], x.x); m[1] = fmaxf(m[1], x.y);
      m[2] = fmaxf(m[2], x.z); m[3] = fmaxf(m[3], x.w);
      nan[0] |= x.x != x.x; nan[1] |= x.y != x.y; nan[2] |= x.z != x.z; nan[3] |= x.w != x.w;
    }
    float acc[kTreeCw / 16][4];
#pragma unroll
    for (int k = 0; k < kTreeCw / 16; ++k)
#pragma unroll
      for (int q = 0; q < 4; ++q) acc[k][q] = 0.f;
#pragma unroll 2
    for (int64_t k = 0; k < n; ++k) {
      const float4 x = *reinterpret_cast<const float4*>(a.pm + (slot0 + k) * kTreeRG + r4);
      const float f[4] = {ex2_approx(x.x - m[0]), ex2_approx(x.y - m[1]), ex2_approx(x.z - m[2]),
                          ex2_approx(x.w - m[3])};
      const float4* src = reinterpret_cast<const float4*>(
                              a.pw + (((slot0 + k) * a.Sv + s) * kCodebook + half * kTreeCw) * (int64_t)kTreeRG) + lane;
#pragma unroll
      for (int c = 0; c < kTreeCw / 16; ++c) {
        const float4 v = src[32 * c];
        acc[c][0] = fmaf(f[0], v.x, acc[c][0]);
        acc[c][1] = fmaf(f[1], v.y, acc[c][1]);
        acc[c][2] = fmaf(f[2], v.z, acc[c][2]);
        acc[c][3] = fmaf(f[3], v.w, acc[c][3]);
      }
    }
    float l[4] = {0.f, 0.f, 0.f, 0.f}, big[4] = {0.f, 0.f, 0.f, 0.f}, down[4];
#pragma unroll
    for (int c = 0; c < kTreeCw / 16; ++c) {
      const float cs = sm.cs[16 * c + (lane >> 1)];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        l[q] += acc[c][q];
        acc[c][q] *= cs;
        big[q] = fmaxf(big[q], fabsf(acc[c][q]));
      }
    }
    // sums and maxima over the lanes with the same rows
#pragma unroll
    for (int o = 2; o < 32; o <<= 1)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        l[q] += __shfl_xor_sync(0xffffffffu, l[q], o);
        big[q] = fmaxf(big[q], __shfl_xor_sync(0xffffffffu, big[q], o));
      }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int ex = split_exponent(big[q]);
      down[q] = exp2_int(-ex);
      if (lane < 2) sm.ws[8 * warp + r4 + q] = exp2_int(ex);
    }
    if (live && s == 0 && lane < 2) {
      // every token is counted once per stage: the sum of stage 0's weights is the row's sum
      const int64_t rows = (int64_t)a.B * a.Hkv * a.RP;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        a.rl[half * rows + row + r4 + q] = l[q];
        if (half == 0) a.rm[row + r4 + q] = nan[q] ? NAN : m[q];
      }
    }
#pragma unroll
    for (int c = 0; c < kTreeCw / 16; ++c) {
      alignas(8) __half hi[4], lo[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) split(acc[c][q] * down[q], hi[q], lo[q]);
      const int at = tile_at<64>(16 * c + (lane >> 1), 8 * warp + r4);
      *reinterpret_cast<uint2*>(sm.w[0] + at) = *reinterpret_cast<const uint2*>(hi);
      *reinterpret_cast<uint2*>(sm.w[1] + at) = *reinterpret_cast<const uint2*>(lo);
    }
    if (lane == 0) sm.row[warp] = n ? row : -1;
  }
  cp_async_wait_all();
  __syncthreads();
  const int64_t rows = (int64_t)a.B * a.Hkv * a.RP;
  const int g = lane >> 2, t4 = lane & 3;
  // rows 16 wr .. x 8 NT dimensions from d0 per warp; with at most two items all warps share theirs
  auto product = [&](auto tiles, int wr, int d0) {
    constexpr int NT = decltype(tiles)::value;
    if (sm.row[2 * wr] < 0 && sm.row[2 * wr + 1] < 0) return;
    float acc[NT][4], cross[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[n][i] = cross[n][i] = 0.f;
#pragma unroll 1
    for (int ks = 0; ks < kTreeCw / 16; ++ks) {
      uint32_t ah[4], al[4];
      frag_at<64>(ah, sm.w[0], 16 * wr, ks, lane);
      frag_at<64>(al, sm.w[1], 16 * wr, ks, lane);
      if constexpr (NT == 1) {
        uint32_t bh[4], bl[4];
        frag_bt<D>(bh, sm.cv[0], d0 & ~15, ks, lane);      // (both halves of 16 dimensions: one is used)
        frag_bt<D>(bl, sm.cv[1], d0 & ~15, ks, lane);
        const bool up = d0 & 8;
        mma16816_add(acc[0], ah, up ? bh[2] : bh[0], up ? bh[3] : bh[1]);
        mma16816(cross[0], ah, up ? bl[2] : bl[0], up ? bl[3] : bl[1]);
        mma16816(cross[0], al, up ? bh[2] : bh[0], up ? bh[3] : bh[1]);
      } else {
#pragma unroll
        for (int n = 0; n < NT; n += 2) {
          uint32_t bh[4], bl[4];
          frag_bt<D>(bh, sm.cv[0], d0 + 8 * n, ks, lane);
          frag_bt<D>(bl, sm.cv[1], d0 + 8 * n, ks, lane);
          mma16816_add(acc[n], ah, bh[0], bh[1]);
          mma16816_add(acc[n + 1], ah, bh[2], bh[3]);
          mma16816(cross[n], ah, bl[0], bl[1]);
          mma16816(cross[n + 1], ah, bl[2], bl[3]);
          mma16816(cross[n], al, bh[0], bh[1]);
          mma16816(cross[n + 1], al, bh[2], bh[3]);
        }
      }
    }
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int64_t row = sm.row[2 * wr + q];
      if (row < 0) continue;
      const float ws = sm.ws[16 * wr + 8 * q + g];
      float* o = a.parts + (part * rows + row + g) * D + d0 + 2 * t4;
#pragma unroll
      for (int n = 0; n < NT; ++n)
        *reinterpret_cast<float2*>(o + 8 * n) = make_float2((acc[n][2 * q] + cross[n][2 * q]) * ws,
                                                            (acc[n][2 * q + 1] + cross[n][2 * q + 1]) * ws);
    }
  };
  if ((int64_t)a.B * a.NRG - group * 8 <= 2) product(std::integral_constant<int, D / 64>{}, 0, warp * (D / 8));
  else product(std::integral_constant<int, D / 16>{}, warp & 3, (warp >> 2) * (D / 2));
}

// ---------------------------------------------------------------------------------------------
// 4. Sum of the parts in their order, rotation back, join with the dense part: one warp per row
// ---------------------------------------------------------------------------------------------
template <int D>
__global__ void __launch_bounds__(128) tree_finish_kernel(TreeArgs a) {
  constexpr int E = D / 32, W = 4;             // dimensions per lane; warps
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t x = (int64_t)blockIdx.x * W + warp;      // (pair, rho)
  const int64_t pair = x / a.R;
  const int rho = (int)(x % a.R);
  pdl_wait();
  if (pair >= (int64_t)a.B * a.Hkv) return;
  const int b = (int)(pair / a.Hkv), kvh = (int)(pair % a.Hkv), i = rho / a.G;
  if (i >= present_queries(a.n_draft, b, a.N)) return;   // rows behind the drafts stay as they are
  const int64_t rows = (int64_t)a.B * a.Hkv * a.RP, row = pair * a.RP + rho;
  const float m = a.rm[row], dm = a.dm[row], dl = a.dl[row];
  float l = a.rl[row];
#pragma unroll
  for (int k = 1; k < kTreeHalves; ++k) l += a.rl[k * rows + row];
  float o[E], y[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    o[e] = 0.f;
    y[e] = a.dout[row * D + e * 32 + lane];
  }
  if (m != -INFINITY) {
    static_assert(kTreeHalves == 2, "two parts per stage");
#pragma unroll 4
    for (int p = 0; p < a.Sv; ++p)
#pragma unroll
      for (int e = 0; e < E; ++e)
        o[e] += a.parts[(2 * p * rows + row) * D + e * 32 + lane] +
                a.parts[((2 * p + 1) * rows + row) * D + e * 32 + lane];
    fwht_warp_f32<D>(o, lane);
  }
  const float M = m != m ? m : fmaxf(m, dm), top = M == -INFINITY ? 0.f : M;
  const float fc = ex2_approx(m - top), fd = ex2_approx(dm - top);
  const float total = l * fc + dl * fd;
  const bool none = total == 0.f;
  const float inv = none ? 0.f : 1.f / total;
  const float gc = fc * inv * (float)a.qt.rot, gd = fd * inv;
  const int64_t at = ((int64_t)b * a.N + i) * a.Hq + (int64_t)kvh * a.G + rho % a.G;
#pragma unroll
  for (int e = 0; e < E; ++e)
    a.out[at * D + e * 32 + lane] = none ? 0.f : fmaf(o[e], gc, y[e] * gd);
  if (a.lse && lane == 0) a.lse[at] = none ? -INFINITY : (top + log2f(total)) * kLn2;
}

// ---------------------------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------------------------

static int tree_pad_stages(int S) { return S <= 2 ? S : S <= 4 ? 4 : 8; }

struct TreePlan {
  int R, RP, NRG, SKP, SVP, grid;
  int64_t items, slots, rows;
  bool split;              // the codewords are split by a kernel of their own
  size_t lut, pre, pw, pm, dm, dl, dout, parts, rm, rl, kplanes, kscale, vplanes, vscale, total;
};

static TreePlan tree_plan(const zkv_tree_params* p) {
  TreePlan t{};
  t.R = p->N * (p->Hq / p->Hkv);
  t.NRG = (t.R + kTreeRG - 1) / kTreeRG;
  t.RP = t.NRG * kTreeRG;
  t.SKP = tree_pad_stages(p->Sk);
  t.SVP = tree_pad_stages(p->Sv);
  const int64_t pairs = (int64_t)p->B * p->Hkv;
  t.items = pairs * t.NRG;
  t.rows = pairs * t.RP;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    sms = 148;
  const int64_t units = t.items * ((p->max_comp_len + kTreeUnit - 1) / kTreeUnit);
  const int64_t ctas = (int64_t)sms * (t.SKP == 8 || t.SVP == 8 ? 1 : 2);
  t.grid = (int)std::max<int64_t>(1, std::min(ctas, (units + kTreeMinUnits - 1) / kTreeMinUnits));
  t.slots = t.items + t.grid;
  size_t o = 0;
  auto take = [&](size_t n) { const size_t at = o; o += align256(n); return at; };
  t.lut = take(query_tables_bytes(pairs, t.RP, t.SKP));
  t.pre = take(((size_t)p->B + 2) * 8);
  t.pw = take((size_t)t.slots * p->Sv * kCodebook * kTreeRG * 4);
  t.pm = take((size_t)t.slots * kTreeRG * 4);
  t.dm = take((size_t)t.rows * 4);
  t.dl = take((size_t)t.rows * 4);
  t.dout = take((size_t)t.rows * p->d * 4);
  t.parts = take((size_t)t.rows * p->d * 4 * p->Sv * kTreeHalves);
  t.rm = take((size_t)t.rows * 4);
  t.rl = take((size_t)t.rows * 4 * kTreeHalves);
  // with four blocks of rows or more per kv head every codeword would be split four times or more
  t.split = (int64_t)p->B * t.RP > 3 * kQtRows;
  if (t.split) {
    const int64_t kr = (int64_t)p->Hkv * p->Sk * kCodebook, vr = (int64_t)p->Hkv * p->Sv * kCodebook;
    t.kplanes = take(split_books_bytes(kr, p->d));
    t.kscale = take((size_t)kr * 4);
    t.vplanes = take(split_books_bytes(vr, p->d));
    t.vscale = take((size_t)vr * 4);
  }
  t.total = o;
  return t;
}

static int validate_tree_shapes(const zkv_tree_params* p) {
  if (!p) return ZKV_ERR_INVALID_ARG;
  if (p->B < 1 || p->N < 1 || p->Hq < 1 || p->Hkv < 1 || p->Hq % p->Hkv) return ZKV_ERR_INVALID_ARG;
  if (!supported_d(p->d)) return ZKV_ERR_UNSUPPORTED;
  if (p->Sk < 1 || p->Sk > kMaxStages || p->Sv < 1 || p->Sv > kMaxStages) return ZKV_ERR_UNSUPPORTED;
  if (p->Hq / p->Hkv > 8 || p->N > 256) return ZKV_ERR_UNSUPPORTED;
  if (p->B > 65535 || p->Hkv > 65535) return ZKV_ERR_UNSUPPORTED;
  if ((int64_t)p->B * p->Hkv * p->N > (1 << 24)) return ZKV_ERR_UNSUPPORTED;
  if (p->Tcap < 0 || p->Wcap < 0 || p->max_comp_len < 0 || p->max_comp_len > p->Tcap)
    return ZKV_ERR_INVALID_ARG;
  if (p->Tcap % 16) return ZKV_ERR_INVALID_ARG;
  if (p->Tcap > (int64_t(1) << 28) || p->Wcap > (int64_t(1) << 28)) return ZKV_ERR_UNSUPPORTED;
  return validate_paged(p->block_table, p->page_tokens, p->max_pages, p->n_pages, p->Tcap);
}

static int validate_tree(const zkv_tree_params* p) {
  const int v = validate_tree_shapes(p);
  if (v != ZKV_OK) return v;
  if (!p->q || !p->draft_k || !p->draft_v || !p->comp_len || !p->win_len || !p->out)
    return ZKV_ERR_INVALID_ARG;
  if (!p->k_codes || !p->v_codes || !p->k_codebooks || !p->v_codebooks) return ZKV_ERR_INVALID_ARG;
  if (p->Wcap > 0 && (!p->win_k || !p->win_v)) return ZKV_ERR_INVALID_ARG;
  const uintptr_t al = (uintptr_t)p->q | (uintptr_t)p->draft_k | (uintptr_t)p->draft_v |
                       (uintptr_t)p->k_codes | (uintptr_t)p->v_codes | (uintptr_t)p->k_codebooks |
                       (uintptr_t)p->v_codebooks | (uintptr_t)p->win_k | (uintptr_t)p->win_v;
  if (al & 15) return ZKV_ERR_INVALID_ARG;
  const int64_t st[9] = {p->q_sb, p->q_sn, p->q_sh, p->k_sb, p->k_sn, p->k_sh,
                         p->v_sb, p->v_sn, p->v_sh};
  for (int64_t s : st)
    if (s < 0 || s % 8) return ZKV_ERR_INVALID_ARG;
  if (p->mask && (p->m_sb < 0 || p->m_sn < 0)) return ZKV_ERR_INVALID_ARG;
  return ZKV_OK;
}

template <int SKP, int SVP>
static cudaError_t launch_tree_scan(const TreeArgs& a, cudaStream_t st) {
  using C = TreeScan<SKP, SVP>;
  void (*kernel)(TreeArgs) = a.table ? tree_scan_kernel<SKP, SVP, true> : tree_scan_kernel<SKP, SVP, false>;
  const cudaError_t e = ensure_smem_limit(kernel, C::SMEM);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(a.grid), dim3(C::THREADS), C::SMEM, st, a);
}

template <int SKP>
static cudaError_t launch_tree_scan_v(const TreeArgs& a, int SVP, cudaStream_t st) {
  switch (SVP) {
    case 1: return launch_tree_scan<SKP, 1>(a, st);
    case 2: return launch_tree_scan<SKP, 2>(a, st);
    case 4: return launch_tree_scan<SKP, 4>(a, st);
    default: return launch_tree_scan<SKP, 8>(a, st);
  }
}

template <int D>
static int launch_tree(const TreeArgs& a, const TreePlan& t, cudaStream_t st) {
  const size_t s0 = sizeof(TreeDenseSmem<D>), s1 = sizeof(QtSmem<D>), s2 = tt_smem_bytes<D>(),
               s3 = sizeof(TreeContractSmem<D>);
  static_assert(tt_smem_bytes<D>() <= kTreeSmemMax && sizeof(TreeContractSmem<D>) <= kTreeSmemMax &&
                    sizeof(TreeDenseSmem<D>) <= kTreeSmemMax && sizeof(QtSmem<D>) <= kTreeSmemMax, "fits");
  if (ensure_smem_limit(tree_dense_kernel<D>, s0) != cudaSuccess ||
      ensure_smem_limit(tree_tables_kernel<D>, s1) != cudaSuccess ||
      ensure_smem_limit(tree_tables_tc_kernel<D>, s2) != cudaSuccess ||
      ensure_smem_limit(tree_contract_kernel<D>, s3) != cudaSuccess)
    return ZKV_ERR_CUDA;
  const dim3 dense((unsigned)(1 + (int64_t)a.B * a.Hkv * ((a.R + kTreeDenseRows - 1) / kTreeDenseRows)));
  if (t.split) {
    tree_split_kernel<D><<<(unsigned)(a.Hkv * (a.Sk + a.Sv) * (kCodebook / 64)), kQtThreads, 0, st>>>(a);
    ZKV_CHECK_LAUNCH();
    // blocks that share a tile's stages: the least time over waves of one block per SM, a block's set-up
    // taken as two thirds of a stage
    const int64_t tiles = ((int64_t)a.B * a.RP + kTtRows - 1) / kTtRows * a.Hkv;
    int shares = 1;
    int64_t best = INT64_MAX;
    for (int x = 1; x <= a.Sk; ++x) {
      const int64_t cost = (tiles * x + 147) / 148 * (2 + 3 * ((a.Sk + x - 1) / x));
      if (cost < best) best = cost, shares = x;
    }
    if (launch_pdl(tree_tables_tc_kernel<D>, dim3((unsigned)(tiles * shares)), dim3(kTtThreads), s2, st, a, shares) !=
            cudaSuccess ||
        launch_pdl(tree_dense_kernel<D>, dense, dim3(kTreeDenseThreads), s0, st, a) != cudaSuccess)
      return ZKV_ERR_CUDA;
  } else {
    tree_dense_kernel<D><<<dense, kTreeDenseThreads, s0, st>>>(a);
    ZKV_CHECK_LAUNCH();
    if (launch_pdl(tree_tables_kernel<D>, dim3((unsigned)a.qt.blocks()), dim3(kQtThreads), s1, st, a) != cudaSuccess)
      return ZKV_ERR_CUDA;
  }
  cudaError_t e;
  switch (t.SKP) {
    case 1: e = launch_tree_scan_v<1>(a, t.SVP, st); break;
    case 2: e = launch_tree_scan_v<2>(a, t.SVP, st); break;
    case 4: e = launch_tree_scan_v<4>(a, t.SVP, st); break;
    default: e = launch_tree_scan_v<8>(a, t.SVP, st); break;
  }
  if (e != cudaSuccess) return ZKV_ERR_CUDA;
  const int64_t tiles = ((int64_t)a.B * a.NRG + 7) / 8;
  if (launch_pdl(tree_contract_kernel<D>, dim3((unsigned)(tiles * a.Sv * kTreeHalves), a.Hkv), dim3(256),
                 s3, st, a) != cudaSuccess)
    return ZKV_ERR_CUDA;
  const int64_t rows = (int64_t)a.B * a.Hkv * a.R;
  if (launch_pdl(tree_finish_kernel<D>, dim3((unsigned)((rows + 3) / 4)), dim3(128), 0, st, a) != cudaSuccess)
    return ZKV_ERR_CUDA;
  return ZKV_OK;
}

}  // namespace zkv

using namespace zkv;

extern "C" size_t zkv_tree_workspace_size(const zkv_tree_params* p) {
  if (validate_tree_shapes(p) != ZKV_OK) return 0;
  return tree_plan(p).total;
}

extern "C" int zkv_rvq_tree_attn(const zkv_tree_params* p, void* workspace, size_t workspace_bytes,
                                 void* stream) {
  const int v = validate_tree(p);
  if (v != ZKV_OK) return v;
  const TreePlan t = tree_plan(p);
  if (!workspace || workspace_bytes < t.total || ((uintptr_t)workspace & 255))
    return ZKV_ERR_WORKSPACE;
  unsigned char* ws = reinterpret_cast<unsigned char*>(workspace);
  const float scale = p->softmax_scale > 0.f ? p->softmax_scale : (float)(1.0 / std::sqrt((double)p->d));
  TreeArgs a{};
  a.B = p->B; a.N = p->N; a.G = p->Hq / p->Hkv; a.Hq = p->Hq; a.Hkv = p->Hkv;
  a.Sk = p->Sk; a.Sv = p->Sv; a.R = t.R; a.RP = t.RP; a.NRG = t.NRG; a.grid = t.grid;
  a.Tcap = p->Tcap; a.Wcap = p->Wcap; a.max_comp = p->max_comp_len;
  a.n_draft = p->n_draft;
  a.dk = reinterpret_cast<const __half*>(p->draft_k);
  a.dv = reinterpret_cast<const __half*>(p->draft_v);
  a.k_sb = p->k_sb; a.k_sn = p->k_sn; a.k_sh = p->k_sh;
  a.v_sb = p->v_sb; a.v_sn = p->v_sn; a.v_sh = p->v_sh;
  a.mask = p->mask; a.m_sb = p->m_sb; a.m_sn = p->m_sn;
  a.k_codes = p->k_codes; a.v_codes = p->v_codes; a.comp_len = p->comp_len; a.Cv = p->v_codebooks;
  a.win_k = reinterpret_cast<const __half*>(p->win_k);
  a.win_v = reinterpret_cast<const __half*>(p->win_v);
  a.win_len = p->win_len;
  a.out = p->out; a.lse = p->lse; a.err = p->error_flag;
  a.table = p->block_table; a.max_pages = p->max_pages; a.n_pages = p->n_pages;
  a.pshift = p->block_table ? log2_pow2(p->page_tokens) : 0;
  QueryTables& q = a.qt;
  q.B = p->B; q.N = p->N; q.G = a.G; q.Hkv = p->Hkv; q.Sk = p->Sk; q.SKP = t.SKP; q.RG = kTreeRG;
  q.R = t.R; q.RP = t.RP;
  q.q = reinterpret_cast<const __half*>(p->q);
  q.q_sb = p->q_sb; q.q_sn = p->q_sn; q.q_sh = p->q_sh;
  q.n_query = p->n_draft; q.Ck = p->k_codebooks; q.k_smooth = p->k_smooth;
  q.scale_log2 = (float)((double)scale * 1.4426950408889634);
  q.rot = 1.0 / std::sqrt((double)p->d);
  q.set_divisors();
  q.lut = reinterpret_cast<float*>(ws + t.lut);
  if (t.split) {
    const int64_t kr = (int64_t)p->Hkv * p->Sk * kCodebook, vr = (int64_t)p->Hkv * p->Sv * kCodebook;
    q.books.hi = reinterpret_cast<__half*>(ws + t.kplanes);
    q.books.lo = q.books.hi + kr * p->d;
    q.books.scale = reinterpret_cast<float*>(ws + t.kscale);
    a.vbooks.hi = reinterpret_cast<__half*>(ws + t.vplanes);
    a.vbooks.lo = a.vbooks.hi + vr * p->d;
    a.vbooks.scale = reinterpret_cast<float*>(ws + t.vscale);
  }
  a.pre = reinterpret_cast<int64_t*>(ws + t.pre);
  a.pw = reinterpret_cast<float*>(ws + t.pw);
  a.pm = reinterpret_cast<float*>(ws + t.pm);
  a.dm = reinterpret_cast<float*>(ws + t.dm);
  a.dl = reinterpret_cast<float*>(ws + t.dl);
  a.dout = reinterpret_cast<float*>(ws + t.dout);
  a.parts = reinterpret_cast<float*>(ws + t.parts);
  a.rm = reinterpret_cast<float*>(ws + t.rm);
  a.rl = reinterpret_cast<float*>(ws + t.rl);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  switch (p->d) {
    case 64: return launch_tree<64>(a, t, st);
    case 128: return launch_tree<128>(a, t, st);
    default: return launch_tree<256>(a, t, st);
  }
}
