// Key lookup tables of a block of query rows (sm_100a), shared by the tree attention and the
// attention-weight totals.
//
// A kv head's query rows are numbered rho = i * G + g (query i < N, head g < G of the group) and
// taken in groups of RG rows.  For each (sequence, kv head, row group) the table holds
//   T[c][s][r] = softmax_scale * log2(e) * < H (lambda q_rho) / sqrt(d), Ck[kvh][s][c] >
// (float32, rho = group * RG + r), so that a token's base-2 score is sum_s T[zk_s][s][r].
// Stages s >= Sk up to the padded count SKP, rows rho >= N G and rows of absent queries are 0.
//
// The work is a float32 product [256 codewords] x [d] x [rows]; block = 64 codewords of one stage
// x 64 rows of one kv head (rows of several sequences side by side: they share the codewords).
#pragma once

#include "zkv_internal.cuh"

namespace zkv {

constexpr int kQtRows = 64, kQtCodes = 64, kQtThreads = 256;

struct QueryTables {
  int B, N, G, Hkv, Sk, SKP, RG;
  int R;          // N * G rows of a (sequence, kv head)
  int RP;         // padded to a multiple of RG
  const __half* q;
  int64_t q_sb, q_sn, q_sh;
  const int32_t* n_query;   // [B] present queries, or null (N)
  const float* Ck;
  const float* k_smooth;
  float scale_log2;
  double rot;
  float* lut;     // [B * Hkv][RP / RG][256][SKP][RG]

  __host__ __device__ int row_blocks() const { return (int)(((int64_t)B * RP + kQtRows - 1) / kQtRows); }
  __host__ __device__ int64_t blocks() const {
    return (int64_t)(kCodebook / kQtCodes) * SKP * row_blocks() * Hkv;
  }
};

inline size_t query_tables_bytes(int64_t pairs, int RP, int SKP) {
  return (size_t)pairs * RP * kCodebook * SKP * sizeof(float);
}

__device__ __forceinline__ int present_queries(const int32_t* n, int b, int N) {
  if (!n) return N;
  const int v = n[b];
  return v < 0 ? 0 : v > N ? N : v;
}

template <int D>
struct QtSmem {
  float c[kQtCodes * D];          // codewords, 16-byte pieces swizzled by codeword
  float qT[D][kQtRows + 4];       // rotated queries, transposed
};

template <int D>
__device__ __forceinline__ void query_tables_block(const QueryTables& a, int64_t blk, QtSmem<D>& sm) {
  constexpr int E = D / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int64_t rest = blk;
  const int c0 = (int)(rest % (kCodebook / kQtCodes)) * kQtCodes;
  rest /= kCodebook / kQtCodes;
  const int s = (int)(rest % a.SKP);
  rest /= a.SKP;
  const int row0 = (int)(rest % a.row_blocks()) * kQtRows;
  const int kvh = (int)(rest / a.row_blocks());
  const bool real = s < a.Sk;
  if (real) {
    const float* C = a.Ck + (((size_t)kvh * a.Sk + s) * kCodebook + c0) * D;
    for (int f = tid; f < kQtCodes * D / 4; f += kQtThreads) {
      const int c = f / (D / 4), p = f % (D / 4);
      cp_async16(sm.c + c * D + 4 * (p ^ (c & 7)), C + (size_t)c * D + 4 * p);
    }
    cp_async_commit();
    // the block's rows, rotated (float32 transform): warp w takes rows w, w + 8, ...
    for (int k = 0; k < kQtRows / 8; ++k) {
      const int j = row0 + warp + 8 * k;
      const int b = j / a.RP, rho = j % a.RP;
      float v[E];
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] = 0.f;
      if (b < a.B && rho < a.R && rho / a.G < present_queries(a.n_query, b, a.N)) {
        const __half* qr = a.q + b * a.q_sb + (rho / a.G) * a.q_sn +
                           ((int64_t)kvh * a.G + rho % a.G) * a.q_sh + lane;
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = __half2float(qr[e * 32]);
        if (a.k_smooth) {   // the query absorbs the keys' smoothing: lambda * q
          const float* l = a.k_smooth + (int64_t)kvh * D + lane;
#pragma unroll
          for (int e = 0; e < E; ++e) v[e] *= l[e * 32];
        }
        fwht_warp_f32<D>(v, lane);
        const float rs = (float)a.rot;
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] *= rs;
      }
#pragma unroll
      for (int e = 0; e < E; ++e) sm.qT[e * 32 + lane][warp + 8 * k] = v[e];
    }
    cp_async_wait_all();
    __syncthreads();
  }
  // thread = 4 codewords (cc + 16 u) x 4 rows (4 rq ..)
  const int cc = tid & 15, rq = tid >> 4;
  float acc[4][4];
#pragma unroll
  for (int u = 0; u < 4; ++u)
#pragma unroll
    for (int v = 0; v < 4; ++v) acc[u][v] = 0.f;
  if (real) {
#pragma unroll 2
    for (int p = 0; p < D / 4; ++p) {
      float4 cv[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        cv[u] = *reinterpret_cast<const float4*>(sm.c + (cc + 16 * u) * D + 4 * (p ^ (cc & 7)));
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float4 q4 = *reinterpret_cast<const float4*>(&sm.qT[4 * p + e][4 * rq]);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float x = e == 0 ? cv[u].x : e == 1 ? cv[u].y : e == 2 ? cv[u].z : cv[u].w;
          acc[u][0] = fmaf(q4.x, x, acc[u][0]);
          acc[u][1] = fmaf(q4.y, x, acc[u][1]);
          acc[u][2] = fmaf(q4.z, x, acc[u][2]);
          acc[u][3] = fmaf(q4.w, x, acc[u][3]);
        }
      }
    }
  }
  const int j = row0 + 4 * rq;             // RG is a multiple of 4: the four rows share a group
  const int b = j / a.RP, rho = j % a.RP;
  if (b < a.B) {
    float* t = a.lut + (((int64_t)b * a.Hkv + kvh) * (a.RP / a.RG) + rho / a.RG) *
                           ((int64_t)kCodebook * a.SKP * a.RG) + rho % a.RG;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      float4 o;
      o.x = acc[u][0] * a.scale_log2;
      o.y = acc[u][1] * a.scale_log2;
      o.z = acc[u][2] * a.scale_log2;
      o.w = acc[u][3] * a.scale_log2;
      *reinterpret_cast<float4*>(t + ((int64_t)(c0 + cc + 16 * u) * a.SKP + s) * a.RG) = o;
    }
  }
}

// The code rows of one (sequence, kv head): contiguous or paged.
struct CodeRows {
  const uint8_t* base;      // the pair's row 0, or the page pool
  const int32_t* table;     // the sequence's block-table row, or null
  int64_t head, heads;      // kv head and kv heads (paged)
  int64_t n_pages;
  int pshift;
  int32_t* err;

  // row address of token t, or null for a page outside the pool (flagged)
  __device__ __forceinline__ const uint8_t* row(uint32_t t, int S) const {
    if (!table) return base + (int64_t)t * S;
    const int64_t pg = __ldg(table + (t >> pshift));
    if (pg < 0 || pg >= n_pages) {
      set_error(err, ZKV_DEVERR_PAGE);
      return nullptr;
    }
    return base + (((pg * heads + head) << pshift) + (t & ((1u << pshift) - 1u))) * S;
  }
};

__device__ __forceinline__ CodeRows code_rows(const uint8_t* codes, const int32_t* table,
                                              int64_t max_pages, int64_t n_pages, int pshift, int b,
                                              int kvh, int Hkv, int64_t Tcap, int S, int32_t* err) {
  CodeRows r;
  r.base = table ? codes : codes + ((int64_t)b * Hkv + kvh) * Tcap * S;
  r.table = table ? table + b * max_pages : nullptr;
  r.head = kvh;
  r.heads = Hkv;
  r.n_pages = n_pages;
  r.pshift = pshift;
  r.err = err;
  return r;
}

// The S <= SP code bytes of token t, little-endian in SP / 4 (at least one) words; 0 for a page
// outside the pool.  Rows are S bytes each, so a power of two is one naturally aligned load.
// NC: through the read-only path (the kernel writes no code rows).
template <bool NC, class T>
__device__ __forceinline__ T load_row_part(const T* p) {
  if constexpr (NC) return __ldg(p);
  return *p;
}
template <int SP, bool NC = true>
__device__ __forceinline__ void load_codes(const CodeRows& rows, uint32_t t, int S,
                                           uint32_t (&w)[SP <= 4 ? 1 : 2]) {
#pragma unroll
  for (int i = 0; i < (SP <= 4 ? 1 : 2); ++i) w[i] = 0u;
  const uint8_t* p = rows.row(t, S);
  if (!p) return;
  if (S == 4) {
    w[0] = load_row_part<NC>(reinterpret_cast<const unsigned int*>(p));
  } else if (S == 2) {
    w[0] = load_row_part<NC>(reinterpret_cast<const unsigned short*>(p));
  } else if (S == 8) {
    if constexpr (SP == 8) {
      const uint2 v = load_row_part<NC>(reinterpret_cast<const uint2*>(p));
      w[0] = v.x;
      w[1] = v.y;
    }
  } else {
#pragma unroll
    for (int s = 0; s < SP; ++s)
      if (s < S) w[s >> 2] |= (uint32_t)load_row_part<NC>(p + s) << (8 * (s & 3));
  }
}

}  // namespace zkv
