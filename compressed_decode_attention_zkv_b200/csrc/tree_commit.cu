// Path commit: the drafts that a sequence accepted enter its cache (sm_100a).
//
// Passages: VQKV (gist.science summary of arXiv 2603.16435), section 2.3 "Local Sliding Window"
// (recent tokens uncompressed, older ones compressed to codes); VeloxQuant-MLX 0.5.1 "Quick start"
// (cache.append).  Committing several tokens at once has no counterpart on the pages.
//
// The result is that of n_accept[b] appends of one token each.  With W window slots, wl of them in
// use, and n accepted tokens: tokens i < W - wl fill the free slots wl + i; every later one evicts.
// Eviction k = i - (W - wl) takes slot (head + k) % W and sends what the slot held to position
// comp_len + k of the prefix.  The slot held the token of eviction k - W if k >= W, else the fill
// token of that slot if there was one, else the window's own token.
//
// Kernel 1: the evictions of all sequences are numbered through (a prefix sum that every block
// computes for itself), so a block encodes R evictions of one kv head and of K or V, from whichever
// sequences.  R is 16 (one warp each); where that could make more blocks than SMs it is 32, since a
// block's time is mostly that of the codewords it reads and rounds.  Only the first eviction of a slot
// (k < W) reads the window, and its warp then writes the slot's last token; fill slots that no eviction
// takes are written apart.  So no slot is read by one block and written by another.
// Kernel 2 advances the lengths after all of kernel 1 has read them.
//
// Encode.  Per stage approximate distances ||c||^2 - 2 r . c of the R residuals to all 256 codewords
// come from the tensor cores, residuals and codewords rounded to fp16 (each row scaled by a power of
// two to a norm of 2^14 .. 2^15, so subnormals do not matter), in chunks of CH codewords whose loads
// are in flight during the chunk before.  A product of two roundings is off by 2^-10 of itself, so a
// distance by less than 2^-9 ||r|| ||c||, and the codewords within twice that (and the margin of the
// float32 row encoder for the rest, candidate_margin) of the smallest distance hold the nearest one.
// One such codeword is the choice (for Gaussian codewords 15 times of 16); several are told apart by
// float64 distances, ties to the lowest index, as zkv_rvq_encode decides.
// Chunks take turns in two buffers, so one is rounded while another's products run: one barrier a chunk.
// A call (both kernels) in a graph: 8 sequences, up to 6 tokens each, 8 kv heads, d = 128, 4 + 4 stages
// 26.9 us; 64 sequences, up to 5 each 40.6 us; one head, 2 + 2 stages 12.3 us; pages or smoothing up to
// 1.2 us more.  (The second buffer gained 3 us in the batches; a cluster of 8 CTAs per 8 evictions with
// float32 distances took 50 and 176 us.)
// Bound by a block's chain: per chunk its rounding and products, per stage the decision.  In the batch of
// 64 six to ten blocks of a head convert the same codewords.
#include <cfloat>
#include <cmath>

#include "encode_rows.cuh"
#include "mma_split.cuh"

namespace zkv {

constexpr int kCommitThreads = 512;

struct CommitState {
  int64_t n, wl, head, comp, evict, fill;   // fill: tokens that take free slots
};

// What sequence b commits; false (with the error bits in err) if it is left unchanged.
__device__ __forceinline__ bool commit_state(const zkv_tree_commit_params& p, int64_t b,
                                             CommitState& s, int& err) {
  const int32_t* path = p.path + b * p.M;
  int32_t x[8];                      // (eight loads in flight, the first ones beside the state's)
#pragma unroll
  for (int q = 0; q < 8; ++q) x[q] = path[min(q, p.M - 1)];
  s.n = p.n_accept[b];
  s.wl = p.win_len[b];
  s.head = p.win_head[b];
  s.comp = p.comp_len[b];
  s.evict = s.fill = 0;
  err = 0;
  if (s.n < 0 || s.n > p.M) {
    err = ZKV_DEVERR_DRAFT;
    return false;
  }
  for (int i = 0; i < (int)s.n; i += 8) {
    if (i > 0)
#pragma unroll
      for (int q = 0; q < 8; ++q) x[q] = path[min(i + q, p.M - 1)];
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (i + q < (int)s.n && (x[q] < 0 || x[q] >= p.N)) err = ZKV_DEVERR_DRAFT;
  }
  if (err) return false;
  if (s.wl < 0 || s.wl > p.Wcap) {
    err = ZKV_DEVERR_WIN_LEN;
    return false;
  }
  s.fill = s.n < p.Wcap - s.wl ? s.n : p.Wcap - s.wl;
  const int64_t e = s.n - s.fill;
  if (e > 0) {
    if (s.head < 0 || s.head >= p.Wcap) err = ZKV_DEVERR_WIN_LEN;
    else if (s.comp < 0 || s.comp + e > p.Tcap) err = ZKV_DEVERR_COMP_LEN;
    else if (p.block_table) {
      const int64_t P = p.page_tokens;
      for (int64_t g = s.comp / P; g <= (s.comp + e - 1) / P; ++g) {
        const int64_t pg = p.block_table[b * p.max_pages + g];
        if (pg < 0 || pg >= p.n_pages) err = ZKV_DEVERR_PAGE;
      }
    }
    if (err) {
      s.fill = 0;
      return false;
    }
  }
  s.evict = e;
  return s.n > 0;
}

template <int D, int R>
struct CommitSmem {
  static constexpr int CH = D == 256 ? 64 : 128;      // codewords per chunk (their loads fit in registers)
  __half c[2][CH * D];                                // codewords: chunks take turns
  __half x[R * D];                                    // residuals
  float r[R][D + 4];                        // residuals, float32
  float dist[R][kCodebook + 4];
  float cn[2][kCodebook];                             // squared norms of the codewords, by stage parity
  float cs[2][CH];                                    // scales of the chunk's codewords
  float xs[R];                              // scales of the residuals
  float rn[R];                              // bound of their norms
  uint8_t code[R][kMaxStages];
  int row_b[R];                             // the evictions: sequence (-1: none), k, state
  int64_t row_k[R];
  CommitState row_s[R];
  int64_t warp_sum[kCommitThreads / 32];
};

template <int D, int R>
__global__ void __launch_bounds__(kCommitThreads) tree_commit_kernel(zkv_tree_commit_params p, double rot) {
  constexpr int E = D / 32, CH = CommitSmem<D, R>::CH, NC = kCodebook / CH, CW = CH / 16;   // CW: codewords per warp
  extern __shared__ __align__(16) unsigned char smem_raw[];
  CommitSmem<D, R>& sm = *reinterpret_cast<CommitSmem<D, R>*>(smem_raw);
  pdl_trigger();   // the length update may launch now; it waits for this kernel's completion
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int kind = blockIdx.z;   // 0 = keys, 1 = values
  const int h = blockIdx.y;
  const int64_t row0 = (int64_t)blockIdx.x * R;
  const int S = kind ? p.Sv : p.Sk;
  const float* CB = (kind ? p.v_codebooks : p.k_codebooks) + (size_t)h * S * kCodebook * D;
  __half* win = reinterpret_cast<__half*>(kind ? p.win_v : p.win_k);
  const __half* draft = reinterpret_cast<const __half*>(kind ? p.draft_v : p.draft_k);
  const int64_t sb = kind ? p.v_sb : p.k_sb, sn = kind ? p.v_sn : p.k_sn, sh = kind ? p.v_sh : p.k_sh;
  uint8_t* codes = kind ? p.v_codes : p.k_codes;

  auto token = [&](int64_t b, int64_t i) -> const __half* {     // accepted token i of sequence b
    return draft + b * sb + (int64_t)p.path[b * p.M + i] * sn + (int64_t)h * sh;
  };
  // codewords of a chunk: warp w holds CW w .. CW w + CW - 1, lane = E dimensions in a row
  float cw[CW][E];
  auto load = [&](int q) {       // chunk q of all stages' chunks
    const float* C = CB + ((size_t)q * CH + CW * warp) * D + lane * E;
#pragma unroll
    for (int k = 0; k < CW; ++k) {
      if constexpr (E == 2) {
        const float2 v = __ldg(reinterpret_cast<const float2*>(C + k * D));
        cw[k][0] = v.x; cw[k][1] = v.y;
      } else {
#pragma unroll
        for (int e = 0; e < E; e += 4) {
          const float4 v = __ldg(reinterpret_cast<const float4*>(C + k * D + e));
          cw[k][e] = v.x; cw[k][e + 1] = v.y; cw[k][e + 2] = v.z; cw[k][e + 3] = v.w;
        }
      }
    }
  };
  if (blockIdx.x == 0) load(0);  // in flight while the evictions are numbered (later blocks may have none)
  // a row's D halves per warp, E per lane
  struct alignas(2 * E) Piece {
    __half x[E];
  };
  // whether this warp's first sequence (below) has free slots
  const int64_t fill_b = (int64_t)blockIdx.x * 16 + warp;
  const bool fills = fill_b < p.B && p.win_len[fill_b] != p.Wcap;
  if (tid < R) sm.row_b[tid] = -1;
  int64_t base = 0;
  for (int64_t b0 = 0; b0 < p.B && base < row0 + R; b0 += kCommitThreads) {
    const int64_t b = b0 + tid;
    CommitState s;
    s.evict = 0;
    int err;
    if (b < p.B) commit_state(p, b, s, err);
    int64_t x = s.evict;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) sm.warp_sum[warp] = x;
    __syncthreads();
    int64_t before = base + x - s.evict, all = 0;
    for (int w = 0; w < kCommitThreads / 32; ++w) {
      if (w < warp) before += sm.warp_sum[w];
      all += sm.warp_sum[w];
    }
    for (int r = 0; r < R; ++r) {
      const int64_t k = row0 + r - before;
      if (k >= 0 && k < s.evict) {
        sm.row_b[r] = (int)b;
        sm.row_k[r] = k;
        sm.row_s[r] = s;
      }
    }
    base += all;
  }
  __syncthreads();
  if (sm.row_b[0] >= 0) {          // rows fill from the front
    if (blockIdx.x > 0) load(0);
    // residual row r of this warp: v (elements 32 e + lane) to shared memory, float32 and fp16
    auto put_row = [&](int r, const float (&v)[E]) {
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) ss = fmaf(v[e], v[e], ss);
      ss = warp_sum_f32(ss);
      const int ex = split_exponent(sqrtf(ss));
      const float down = exp2_int(-ex);
      if (lane == 0) {
        sm.xs[r] = exp2_int(ex);
        sm.rn[r] = sqrtf(ss) * 1.0001f;       // (D + 5 roundings of 2^-24 on ss)
      }
#pragma unroll
      for (int e = 0; e < E; ++e) {
        sm.r[r][e * 32 + lane] = v[e];
        sm.x[tile_at<D>(r, e * 32 + lane)] = __float2half_rn(v[e] * down);
      }
    };
#pragma unroll
    for (int r = warp; r < R; r += 16) {
      const int64_t b = sm.row_b[r];
      float y[E];
#pragma unroll
      for (int e = 0; e < E; ++e) y[e] = 0.f;
      if (b >= 0) {
        // (fewer than 2^29 in all: 32-bit quotients)
        const uint32_t W = (uint32_t)p.Wcap;
        const int64_t k = sm.row_k[r], slot = ((uint32_t)sm.row_s[r].head + (uint32_t)k) % W, wl = sm.row_s[r].wl;
        const __half* x = k >= p.Wcap ? token(b, k - wl)               // the token of eviction k - W
                        : slot >= wl  ? token(b, slot - wl)            // a fill token
                                      : win + ((b * p.Hkv + h) * p.Wcap + slot) * D;
        // the slot's last token takes its place once the row has been read (by this warp alone)
        Piece piece;
        __half* dst = nullptr;
        if (k < p.Wcap) {
          const int64_t last = k + (uint32_t)(sm.row_s[r].evict - 1 - k) / W * W;     // the slot's last eviction
          piece = reinterpret_cast<const Piece*>(token(b, p.Wcap - wl + last))[lane];
          dst = win + ((b * p.Hkv + h) * p.Wcap + slot) * D;
        }
        double v[E];
        load_row_f64<E>(x, ZKV_DTYPE_F16, 0, lane, v);
        if (kind == 0 && p.k_smooth) {   // keys: x / lambda per channel before the rotation
#pragma unroll
          for (int e = 0; e < E; ++e) v[e] *= 1.0 / (double)p.k_smooth[(int64_t)h * D + e * 32 + lane];
        }
        fwht_warp_f64<D>(v, lane);
#pragma unroll
        for (int e = 0; e < E; ++e) y[e] = (float)(v[e] * rot);
        __syncwarp();
        if (dst) reinterpret_cast<Piece*>(dst)[lane] = piece;
      }
      put_row(r, y);
    }
    const int g = lane >> 2, t4 = lane & 3;
    // chunk q from registers to shared memory: norms, scales, fp16
    auto convert = [&](int q) {
      // their norms: lane l gets codeword l % CW's (CW sums over the lanes at once)
      float part[CW], down_of;
#pragma unroll
      for (int k = 0; k < CW; ++k) {
        part[k] = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) part[k] = fmaf(cw[k][e], cw[k][e], part[k]);
      }
      {
        int own = 0;
        const float ss = TransposeSum<CW, CW, 16>::run(part, lane, own);
        // no element is larger than the norm: scale by its power of two
        const int ex = split_exponent(sqrtf(ss));
        down_of = exp2_int(-ex);
        sm.cn[q / NC & 1][q % NC * CH + CW * warp + own] = ss;
        sm.cs[q & 1][CW * warp + own] = exp2_int(ex);
      }
#pragma unroll
      for (int k = 0; k < CW; ++k) {
        const int c = CW * warp + k;
        const float down = __shfl_sync(0xffffffffu, down_of, sum_owner<CW>(k));
        alignas(16) __half2 y[E / 2];
#pragma unroll
        for (int e = 0; e < E; e += 2) y[e / 2] = __floats2half2_rn(cw[k][e] * down, cw[k][e + 1] * down);
        __half* at = sm.c[q & 1] + tile_at<D>(c, lane * E);
        if constexpr (E == 2) *reinterpret_cast<uint32_t*>(at) = *reinterpret_cast<const uint32_t*>(y);
        else if constexpr (E == 4) *reinterpret_cast<uint2*>(at) = *reinterpret_cast<const uint2*>(y);
        else *reinterpret_cast<uint4*>(at) = *reinterpret_cast<const uint4*>(y);
      }
    };
    convert(0);
    if (S * NC > 1) load(1);
    for (int s = 0; s < S; ++s) {
      for (int chunk = 0; chunk < NC; ++chunk) {
        const int q = s * NC + chunk;
        // chunk q (and, at the first, the residuals) are there, and chunk q - 1 has been read
        __syncthreads();
        if (8 * warp < CH) {         // 8 codewords per warp
          float acc[R / 16][2][4] = {};         // (two sums: neither waits for the other)
#pragma unroll 4
          for (int ks = 0; ks < D / 16; ks += 2) {
            uint32_t b[4];
            frag_b2<D>(b, sm.c[q & 1], 8 * warp, ks, lane);
#pragma unroll
            for (int m = 0; m < R / 16; ++m)
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                uint32_t x[4];
                frag_a<D>(x, sm.x, 16 * m, ks + i, lane);
                mma16816(acc[m][i], x, b[2 * i], b[2 * i + 1]);
              }
          }
#pragma unroll
          for (int m = 0; m < R / 16; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int c = 8 * warp + 2 * t4 + (i & 1), r = 16 * m + g + 8 * (i >> 1);
              const float dot = (acc[m][0][i] + acc[m][1][i]) * sm.cs[q & 1][c] * sm.xs[r];
              sm.dist[r][chunk * CH + c] = sm.cn[s & 1][chunk * CH + c] - 2.f * dot;
            }
        }
        // the next chunk meanwhile: a warp in its products leaves the issue slots to one that rounds
        if (q + 1 < S * NC) {
          convert(q + 1);
          if (q + 2 < S * NC) load(q + 2);
        }
      }
      __syncthreads();
      // warp w decides rows w, w + 16: lane = codewords lane + 32 j
      float cmax = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) cmax = fmaxf(cmax, sm.cn[s & 1][32 * j + lane]);
      cmax = warp_max_f32(cmax);
#pragma unroll 1
      for (int r = warp; r < R; r += 16) {
        if (sm.row_b[r] < 0) break;
        float d[8], dmin = INFINITY;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          d[j] = sm.dist[r][32 * j + lane];
          dmin = fminf(dmin, d[j]);
        }
        dmin = warp_min_f32(dmin);
        // candidate_margin's bound and 2^-8 ||r|| ||c|| (and a little for the sums of the products) for
        // the fp16 roundings, in float32 arithmetic: 0.1 % and the additions' roundings more
        constexpr float K = 2.5f * (D + 3) / 16777216.f;
        const float bn = sqrtf(cmax) * 1.0001f, both = sm.rn[r] + bn;
        const float thr = dmin + (K * both * both + 0.0040f * sm.rn[r] * bn) * 1.001f + 2.4e-7f * fabsf(dmin) + 1e-30f;
        unsigned cand[8];
        int count = 0, z = kCodebook;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          cand[j] = __ballot_sync(0xffffffffu, d[j] <= thr);
          count += __popc(cand[j]);
          if (cand[j] && z == kCodebook) z = 32 * j + __ffs(cand[j]) - 1;
        }
        const float* C = CB + (size_t)s * kCodebook * D;
        if (count > 1) {           // several within the margin: float64 distances, four at a time
          double best = DBL_MAX;
          z = kCodebook;
          int c[4], have = 0;
          auto weigh = [&]() {
            double a[4];
            float y[4][E];
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
              for (int e = 0; e < E; ++e) y[u][e] = __ldg(C + (size_t)c[u < have ? u : 0] * D + e * 32 + lane);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              a[u] = 0.0;
#pragma unroll
              for (int e = 0; e < E; ++e) {
                const double df = (double)sm.r[r][e * 32 + lane] - (double)y[u][e];
                a[u] = fma(df, df, a[u]);
              }
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
#pragma unroll
              for (int u = 0; u < 4; ++u) a[u] += __shfl_xor_sync(0xffffffffu, a[u], o);
#pragma unroll
            for (int u = 0; u < 4; ++u)
              if (u < have && a[u] < best) {      // (ascending indices: ties keep the lowest)
                best = a[u];
                z = c[u];
              }
            have = 0;
          };
#pragma unroll 1
          for (int j = 0; j < 8; ++j) {
            unsigned x = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (i == j) x = cand[i];
            for (; x; x &= x - 1u) {
              const int cx = 32 * j + __ffs(x) - 1;
              if (have == 0) c[0] = cx;
              else if (have == 1) c[1] = cx;
              else if (have == 2) c[2] = cx;
              else c[3] = cx;
              if (++have == 4) weigh();
            }
          }
          if (have) weigh();
        }
        // a row that is not finite matches no candidate: code 0
        if (z >= kCodebook) z = 0;
        if (lane == 0) sm.code[r][s] = (uint8_t)z;
        if (s + 1 < S) {
          float v[E];
#pragma unroll
          for (int e = 0; e < E; ++e) v[e] = sm.r[r][e * 32 + lane] - __ldg(C + (size_t)z * D + e * 32 + lane);
          put_row(r, v);
        }
      }
    }
    __syncthreads();
    if (tid < R && sm.row_b[tid] >= 0) {
      const int64_t b = sm.row_b[tid], t = sm.row_s[tid].comp + sm.row_k[tid];
      uint8_t* c = codes + ((b * p.Hkv + h) * p.Tcap + t) * S;
      if (p.block_table) {
        const int64_t P = p.page_tokens;
        c = codes + ((p.block_table[b * p.max_pages + t / P] * (int64_t)p.Hkv + h) * P + t % P) * S;
      }
      for (int s = 0; s < S; ++s) c[s] = sm.code[tid][s];
    }
  }
  // fill tokens whose slot no eviction takes: the sequences are shared out over blocks and warps
  for (int64_t b = fill_b; b < p.B; b += (int64_t)gridDim.x * 16) {
    if (b == fill_b ? !fills : p.win_len[b] == p.Wcap) continue;
    CommitState s;
    int err;
    if (!commit_state(p, b, s, err)) continue;
    for (int64_t i = 0; i < s.fill; ++i) {
      const int64_t slot = s.wl + i;
      if (s.evict > 0 && (uint32_t)(slot - s.head + p.Wcap) % (uint32_t)p.Wcap < s.evict) continue;
      const __half* src = token(b, i);
      __half* dst = win + ((b * p.Hkv + h) * p.Wcap + slot) * D;
      reinterpret_cast<Piece*>(dst)[lane] = reinterpret_cast<const Piece*>(src)[lane];
    }
  }
}

__global__ void tree_commit_lengths_kernel(zkv_tree_commit_params p) {
  const int64_t b = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  CommitState s;
  int err = 0;
  const bool ok = b < p.B && commit_state(p, b, s, err);     // (kernel 1 changes nothing of it)
  if (err) set_error(p.error_flag, err);
  const int32_t head = ok ? (int32_t)((uint32_t)(s.head + s.evict) % (uint32_t)p.Wcap) : 0;
  pdl_wait();   // every block of kernel 1 has read the lengths
  if (!ok) return;
  p.win_len[b] = (int32_t)(s.wl + s.fill);
  if (s.evict > 0) {
    p.comp_len[b] = (int32_t)(s.comp + s.evict);
    p.win_head[b] = head;
  }
}

template <int D, int R>
static int launch_tree_commit_rows(const zkv_tree_commit_params& p, cudaStream_t st) {
  const double rot = 1.0 / std::sqrt((double)p.d);
  static_assert(sizeof(CommitSmem<D, R>) <= 227 * 1024, "fits");
  if (ensure_smem_limit(tree_commit_kernel<D, R>, sizeof(CommitSmem<D, R>)) != cudaSuccess) return ZKV_ERR_CUDA;
  const int64_t groups = ((int64_t)p.B * p.M + R - 1) / R;
  tree_commit_kernel<D, R><<<dim3((unsigned)groups, (unsigned)p.Hkv, 2), kCommitThreads, sizeof(CommitSmem<D, R>), st>>>(p, rot);
  ZKV_CHECK_LAUNCH();
  if (launch_pdl(tree_commit_lengths_kernel, dim3((p.B + 127) / 128), dim3(128), 0, st, p) != cudaSuccess)
    return ZKV_ERR_CUDA;
  return ZKV_OK;
}

template <int D>
static int launch_tree_commit(const zkv_tree_commit_params& p, cudaStream_t st) {
  const bool many = ((int64_t)p.B * p.M + 15) / 16 * p.Hkv * 2 > 148;
  return many ? launch_tree_commit_rows<D, 32>(p, st) : launch_tree_commit_rows<D, 16>(p, st);
}

}  // namespace zkv

using namespace zkv;

extern "C" int zkv_rvq_tree_commit(const zkv_tree_commit_params* p, void* stream) {
  if (!p) return ZKV_ERR_INVALID_ARG;
  if (p->B < 1 || p->N < 1 || p->M < 1 || p->Hkv < 1 || p->Tcap < 0 || p->Wcap < 1)
    return ZKV_ERR_INVALID_ARG;
  if (!supported_d(p->d)) return ZKV_ERR_UNSUPPORTED;
  if (p->Sk < 1 || p->Sk > kMaxStages || p->Sv < 1 || p->Sv > kMaxStages) return ZKV_ERR_UNSUPPORTED;
  if (p->Hkv > 65535 || p->B > 65535 || p->M > 256) return ZKV_ERR_UNSUPPORTED;
  if (p->Wcap > (int64_t(1) << 28)) return ZKV_ERR_UNSUPPORTED;
  if (!p->draft_k || !p->draft_v || !p->path || !p->n_accept || !p->win_k || !p->win_v ||
      !p->win_len || !p->win_head || !p->comp_len || !p->k_codes || !p->v_codes ||
      !p->k_codebooks || !p->v_codebooks)
    return ZKV_ERR_INVALID_ARG;
  const uintptr_t al = (uintptr_t)p->win_k | (uintptr_t)p->win_v | (uintptr_t)p->draft_k |
                       (uintptr_t)p->draft_v | (uintptr_t)p->k_codebooks | (uintptr_t)p->v_codebooks;
  if (al & 15) return ZKV_ERR_INVALID_ARG;
  const int64_t str[6] = {p->k_sb, p->k_sn, p->k_sh, p->v_sb, p->v_sn, p->v_sh};
  for (int64_t s : str)
    if (s < 0 || s % 8) return ZKV_ERR_INVALID_ARG;
  const int v = validate_paged(p->block_table, p->page_tokens, p->max_pages, p->n_pages, p->Tcap);
  if (v != ZKV_OK) return v;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  switch (p->d) {
    case 64: return launch_tree_commit<64>(*p, st);
    case 128: return launch_tree_commit<128>(*p, st);
    default: return launch_tree_commit<256>(*p, st);
  }
}
