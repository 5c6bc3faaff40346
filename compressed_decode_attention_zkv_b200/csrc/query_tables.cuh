// Key lookup tables of a block of query rows (sm_100a), shared by the tree attention and the
// attention-weight totals.
//
// A kv head's query rows are numbered rho = i * G + g (query i < N, head g < G of the group) and
// taken in groups of RG rows.  For each (sequence, kv head, row group) the table holds
//   T[c][s][r] = softmax_scale * log2(e) * < H (lambda q_rho) / sqrt(d), Ck[kvh][s][c] >
// (float32, rho = group * RG + r), so that a token's base-2 score is sum_s T[zk_s][s][r].
// Stages s >= Sk up to the padded count SKP, rows rho >= N G and rows of absent queries are 0.
//
// The work is a product [rows] x [d] x [256 codewords] per kv head and stage with float32 accuracy
// (mma_split.cuh).  Block = 64 rows of one kv head (rows of several sequences side by side: they
// share the codewords) x one stage; it rotates its rows once and takes the codewords in chunks of
// 64, the next chunk's loads in flight during a chunk's products.  With few blocks the chunks of a
// stage are shared out over 2 or 4 blocks.  Every block splits the codewords that it uses; where many
// would repeat that, the tree attention takes tree_tables_tc.cuh and codewords split before (SplitBooks).
// 6 us for 8 rows or 32, d = 128, 4 stages: loads, rotation and one chunk's products, all latency.
#pragma once

#include "mma_split.cuh"

namespace zkv {

constexpr int kQtRows = 64, kQtCodes = 64, kQtThreads = 256;

// Codewords split into fp16 planes once (mma_split.cuh): [row][D] each, row = (kv head, stage, codeword)
struct SplitBooks {
  __half *hi, *lo;
  float* scale;            // [row] 2^e
};
inline size_t split_books_bytes(int64_t rows, int D) { return (size_t)rows * D * 4; }

// Quotients by a divisor that a launch fixes: n / d = n m >> 40 with m = floor(2^40 / d) + 1, exact
// while n d < 2^40
struct FixedDivisor {
  int d;
  uint64_t m;
  void set(int x) { d = x; m = (uint64_t(1) << 40) / x + 1; }
  __device__ __forceinline__ int quotient(int n) const { return (int)(((uint64_t)n * m) >> 40); }
};

struct QueryTables {
  int B, N, G, Hkv, Sk, SKP, RG;
  int R;          // N * G rows of a (sequence, kv head)
  int RP;         // padded to a multiple of RG
  FixedDivisor by_rp, by_g, by_rg;      // RP, G and RG
  void set_divisors() { by_rp.set(RP); by_g.set(G); by_rg.set(RG); }
  const __half* q;
  int64_t q_sb, q_sn, q_sh;
  const int32_t* n_query;   // [B] present queries, or null (N)
  const float* Ck;
  const float* k_smooth;
  float scale_log2;
  double rot;
  float* lut;     // [B * Hkv][RP / RG][256][SKP][RG]
  SplitBooks books;         // of Ck, or null planes

  __host__ __device__ int row_blocks() const { return (int)(((int64_t)B * RP + kQtRows - 1) / kQtRows); }
  // blocks that share the chunks of a stage: at least one block per SM where the chunks allow it
  __host__ __device__ int shares() const {
    const int64_t n = (int64_t)SKP * row_blocks() * Hkv;
    return n >= 148 ? 1 : n >= 74 ? 2 : 4;
  }
  __host__ __device__ int64_t blocks() const { return (int64_t)shares() * SKP * row_blocks() * Hkv; }
};

inline size_t query_tables_bytes(int64_t pairs, int RP, int SKP) {
  return (size_t)pairs * RP * kCodebook * SKP * sizeof(float);
}

__device__ __forceinline__ int present_queries(const int32_t* n, int b, int N) {
  if (!n) return N;
  const int v = n[b];
  return v < 0 ? 0 : v > N ? N : v;
}

// 64 rows of a split book into a tile of the two planes (asynchronous)
template <int D>
__device__ __forceinline__ void copy_split(const SplitBooks& books, int64_t row0, int rows, __half* hi, __half* lo,
                                           int threads) {
  for (int f = threadIdx.x; f < rows * (D / 8); f += threads) {
    const int r = f / (D / 8), c = (f % (D / 8)) * 8, at = tile_at<D>(r, c);
    cp_async16(hi + at, books.hi + (row0 + r) * D + c);
    cp_async16(lo + at, books.lo + (row0 + r) * D + c);
  }
}

// Splits 64 rows of [row][D] float32 codewords: warp w takes rows 8 w .. 8 w + 7, lane = D / 32
// dimensions in a row
template <int D>
__device__ __forceinline__ void split_books_block(const float* src, const SplitBooks& books, int64_t row0) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t first = row0 + 8 * warp;
  float v[8][E], part[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    part[k] = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      v[k][e] = __ldg(src + (first + k) * D + lane * E + e);
      part[k] = fmaf(v[k][e], v[k][e], part[k]);
    }
  }
  int own = 0;
  const int ex = split_exponent(sqrtf(TransposeSum<8, 8, 16>::run(part, lane, own)));
  const float down_of = exp2_int(-ex);
  books.scale[first + own] = exp2_int(ex);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float down = __shfl_sync(0xffffffffu, down_of, sum_owner<8>(k));
#pragma unroll
    for (int e = 0; e < E; e += 2) {
      __half2 hi, lo;
      split(v[k][e] * down, hi.x, lo.x);
      split(v[k][e + 1] * down, hi.y, lo.y);
      *reinterpret_cast<__half2*>(books.hi + (first + k) * D + lane * E + e) = hi;
      *reinterpret_cast<__half2*>(books.lo + (first + k) * D + lane * E + e) = lo;
    }
  }
}

template <int D>
struct QtSmem {
  __half q[2][kQtRows * D];       // rotated queries: high and low plane
  __half c[2][kQtCodes * D];      // codewords
  float qs[kQtRows];              // their scales (softmax scale included)
  float cs[kQtCodes];
};

template <int D>
__device__ __forceinline__ void query_tables_block(const QueryTables& a, int64_t blk, QtSmem<D>& sm) {
  constexpr int E = D / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int shares = a.shares(), chunks = kCodebook / kQtCodes / shares;
  int64_t rest = blk;
  const int c0 = (int)(rest % shares) * chunks * kQtCodes;
  rest /= shares;
  const int s = (int)(rest % a.SKP);
  rest /= a.SKP;
  const int row0 = (int)(rest % a.row_blocks()) * kQtRows;
  const int kvh = (int)(rest / a.row_blocks());
  const bool real = s < a.Sk;
  // warp w loads codewords 8 w .. 8 w + 7 of a chunk, lane = E dimensions in a row
  float cw[8][E];
  const int64_t book0 = ((int64_t)kvh * a.Sk + s) * kCodebook + c0;      // the block's first codeword
  auto load = [&](int chunk) {
    const float* C = a.Ck + (book0 + chunk * kQtCodes + 8 * warp) * D;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float* x = C + k * D + lane * E;
      if constexpr (E == 2) {
        const float2 v = __ldg(reinterpret_cast<const float2*>(x));
        cw[k][0] = v.x; cw[k][1] = v.y;
      } else {
#pragma unroll
        for (int e = 0; e < E; e += 4) {
          const float4 v = __ldg(reinterpret_cast<const float4*>(x + e));
          cw[k][e] = v.x; cw[k][e + 1] = v.y; cw[k][e + 2] = v.z; cw[k][e + 3] = v.w;
        }
      }
    }
  };
  if (real) {
    load(0);
    // the block's rows, rotated (float32 transform): warp w takes rows w, w + 8, ...
    const int rows = a.B * a.RP - row0;          // rows from here on
    float v[8][E], part[8], down_of;
    // (rows that are not there read the first one: all loads are in flight together)
    bool there[8];
    int i[8], g[8], b[8], present[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int j = row0 + warp + 8 * k;
      b[k] = a.by_rp.quotient(j);
      const int rho = j - b[k] * a.RP;
      i[k] = a.by_g.quotient(rho);
      g[k] = rho - i[k] * a.G;
      there[k] = warp + 8 * k < rows && rho < a.R;
      if (!there[k]) b[k] = i[k] = g[k] = 0;
      present[k] = a.n_query ? a.n_query[b[k]] : a.N;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const __half* qr = a.q + b[k] * a.q_sb + i[k] * a.q_sn + ((int64_t)kvh * a.G + g[k]) * a.q_sh + lane;
#pragma unroll
      for (int e = 0; e < E; ++e) v[k][e] = __half2float(qr[e * 32]);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (!there[k] || i[k] >= present[k])
#pragma unroll
        for (int e = 0; e < E; ++e) v[k][e] = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      part[k] = 0.f;
      if (warp + 8 * k >= rows) continue;
      if (a.k_smooth) {   // the query absorbs the keys' smoothing: lambda * q
        const float* l = a.k_smooth + (int64_t)kvh * D + lane;
#pragma unroll
        for (int e = 0; e < E; ++e) v[k][e] *= l[e * 32];
      }
      fwht_warp_f32<D>(v[k], lane);
#pragma unroll
      for (int e = 0; e < E; ++e) part[k] = fmaf(v[k][e], v[k][e], part[k]);
    }
    {
      int own = 0;        // the norms of the eight rows at once
      const int ex = split_exponent(sqrtf(TransposeSum<8, 8, 16>::run(part, lane, own)));
      down_of = exp2_int(-ex);
      sm.qs[warp + 8 * own] = exp2_int(ex) * (float)(a.rot * (double)a.scale_log2);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float down = __shfl_sync(0xffffffffu, down_of, sum_owner<8>(k));
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int at = tile_at<D>(warp + 8 * k, e * 32 + lane);
        split(v[k][e] * down, sm.q[0][at], sm.q[1][at]);
      }
    }
  }
  // products: rows 16 wr .. of the block x codewords 8 NT wc .. of the chunk per warp; with at most 16
  // rows all warps share their codewords
  const bool few = (int64_t)a.B * a.RP - row0 <= 16;
  const int wr = few ? 0 : warp & 3, cl0 = few ? 8 * warp : 32 * (warp >> 2);
  const int g = lane >> 2, t4 = lane & 3;
  // this thread's two rows in the tables (null: behind the last), at its first codeword
  float* out[2];
  const int step = a.SKP * a.RG;               // from codeword to codeword
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int j = row0 + 16 * wr + g + 8 * q, b = a.by_rp.quotient(j), rho = j - b * a.RP;
    const int rg = a.by_rg.quotient(rho);
    out[q] = b < a.B ? a.lut + (((int64_t)b * a.Hkv + kvh) * (a.RP / a.RG) + rg) * ((int64_t)kCodebook * step) +
                           (c0 + cl0 + 2 * t4) * step + s * a.RG + (rho - rg * a.RG)
                     : nullptr;
  }
  auto put = [&](int chunk, int n, const float (&acc)[4], const float (&cross)[4]) {
    const int cl = cl0 + 8 * n + 2 * t4, off = (chunk * kQtCodes + 8 * n) * step;
    float2 cs = make_float2(0.f, 0.f);
    if (real) cs = *reinterpret_cast<const float2*>(sm.cs + cl);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      if (!out[q]) continue;
      const float qs = real ? sm.qs[16 * wr + g + 8 * q] : 0.f;
      out[q][off] = real ? (acc[2 * q] + cross[2 * q]) * cs.x * qs : 0.f;
      out[q][off + step] = real ? (acc[2 * q + 1] + cross[2 * q + 1]) * cs.y * qs : 0.f;
    }
  };
  for (int chunk = 0; chunk < chunks; ++chunk) {
    if (real) {
      __syncthreads();              // the previous chunk has been read
      float part[8], down_of;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        part[k] = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) part[k] = fmaf(cw[k][e], cw[k][e], part[k]);
      }
      {
        int own = 0;
        const int ex = split_exponent(sqrtf(TransposeSum<8, 8, 16>::run(part, lane, own)));
        down_of = exp2_int(-ex);
        sm.cs[8 * warp + own] = exp2_int(ex);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int c = 8 * warp + k;
        const float down = __shfl_sync(0xffffffffu, down_of, sum_owner<8>(k));
        alignas(16) __half hi[E], lo[E];
#pragma unroll
        for (int e = 0; e < E; ++e) split(cw[k][e] * down, hi[e], lo[e]);
        const int at = tile_at<D>(c, lane * E);
        if constexpr (E == 2) {
          *reinterpret_cast<uint32_t*>(sm.c[0] + at) = *reinterpret_cast<const uint32_t*>(hi);
          *reinterpret_cast<uint32_t*>(sm.c[1] + at) = *reinterpret_cast<const uint32_t*>(lo);
        } else if constexpr (E == 4) {
          *reinterpret_cast<uint2*>(sm.c[0] + at) = make_uint2(reinterpret_cast<const uint32_t*>(hi)[0], reinterpret_cast<const uint32_t*>(hi)[1]);
          *reinterpret_cast<uint2*>(sm.c[1] + at) = make_uint2(reinterpret_cast<const uint32_t*>(lo)[0], reinterpret_cast<const uint32_t*>(lo)[1]);
        } else {
          const uint32_t *h4 = reinterpret_cast<const uint32_t*>(hi), *l4 = reinterpret_cast<const uint32_t*>(lo);
          *reinterpret_cast<uint4*>(sm.c[0] + at) = make_uint4(h4[0], h4[1], h4[2], h4[3]);
          *reinterpret_cast<uint4*>(sm.c[1] + at) = make_uint4(l4[0], l4[1], l4[2], l4[3]);
        }
      }
      __syncthreads();
      if (chunk + 1 < chunks) load(chunk + 1);
    }
    if (few) {
      float acc[4] = {}, cross[2][4] = {};
      if (real) {
#pragma unroll 2
        for (int ks = 0; ks < D / 16; ks += 2) {
          uint32_t bh[4], bl[4];
          frag_b2<D>(bh, sm.c[0], cl0, ks, lane);
          frag_b2<D>(bl, sm.c[1], cl0, ks, lane);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint32_t ah[4], al[4];
            frag_a<D>(ah, sm.q[0], 0, ks + i, lane);
            frag_a<D>(al, sm.q[1], 0, ks + i, lane);
            mma16816_add(acc, ah, bh[2 * i], bh[2 * i + 1]);
            mma16816(cross[0], ah, bl[2 * i], bl[2 * i + 1]);
            mma16816(cross[1], al, bh[2 * i], bh[2 * i + 1]);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) cross[0][i] += cross[1][i];
      }
      put(chunk, 0, acc, cross[0]);
    } else {
      float acc[4][4] = {}, cross[4][4] = {};
      if (real) {
#pragma unroll 2
        for (int ks = 0; ks < D / 16; ++ks) {
          uint32_t ah[4], al[4];
          frag_a<D>(ah, sm.q[0], 16 * wr, ks, lane);
          frag_a<D>(al, sm.q[1], 16 * wr, ks, lane);
#pragma unroll
          for (int n = 0; n < 4; n += 2) {
            uint32_t bh[4], bl[4];
            frag_b<D>(bh, sm.c[0], cl0 + 8 * n, ks, lane);
            frag_b<D>(bl, sm.c[1], cl0 + 8 * n, ks, lane);
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
      for (int n = 0; n < 4; ++n) put(chunk, n, acc[n], cross[n]);
    }
  }
}

// Table gathers and counter additions take the permuted bytes [column | code] of a packed code word as
// a shared-memory address with the start of the tables as an immediate offset: dynamic shared memory begins at kTableBase, behind the
// reserved system area (the kernel checks it and reports ZKV_DEVERR_SMEM otherwise).  No memory
// clobber: tables and counters are written and read on either side of a barrier.
constexpr int kTableBase = 1024;
__device__ __forceinline__ float2 lds_pair(uint32_t x) {
  float2 v;
  asm volatile("ld.shared.v2.f32 {%0, %1}, [%2+%3];" : "=f"(v.x), "=f"(v.y) : "r"(x), "n"(kTableBase));
  return v;
}
__device__ __forceinline__ float4 lds_quad(uint32_t x) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4+%5];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(x), "n"(kTableBase));
  return v;
}
template <int OFF>
__device__ __forceinline__ void red_counter(uint32_t x, uint32_t u) {
  asm volatile("red.shared.add.u32 [%0+%2], %1;" ::"r"(x), "r"(u), "n"(kTableBase + OFF));
}

__device__ __forceinline__ uint32_t byte_perm(uint32_t a, uint32_t b, uint32_t s) {
  uint32_t d;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(s));
  return d;
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
