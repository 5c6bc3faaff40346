// Cluster encoder of a few rows (sm_100a), shared by the append call and the path commit.
//
// A cluster of 8 CTAs encodes 8 rows of one kv head.  CTA k of the
// cluster owns codewords [32k, 32k + 32) of every stage: it copies its slices with cp.async
// into a ring of kAppendNB buffers (up to kAppendNB - 1 stages ahead; all of them when
// S <= kAppendNB) and computes its 32 x 8 float32 distances.  Its candidates
// are the codewords within the rounding margin (the row encoder's bound, taken with this
// slice's largest codeword norm) of its own row minimum: a superset of the slice's codewords
// within the margin of the global minimum, so the exact argmin is always among them.  Each CTA
// publishes, per row, its best (float64 distance, index) and after one cluster barrier every
// CTA reduces the 8 published bests the same way (decided in float64, ties to the lowest
// index).  Within a CTA, warp r decides row r with no block-wide step (lane = local codeword);
// each CTA writes its per-row bests into every CTA of the cluster before the barrier, so the
// reduction after it reads local shared memory.  Every CTA keeps an identical copy of the
// residuals and reads the chosen codeword from its owner's shared memory.
#pragma once

#include <cooperative_groups.h>

#include "encode_rows.cuh"

namespace zkv {

constexpr int kAppendR = 8;        // rows per cluster
constexpr int kAppendCl = 8;       // CTAs per cluster
constexpr int kAppendCw = kCodebook / kAppendCl;   // codewords per CTA
constexpr int kAppendNB = 4;       // codeword slice buffers (stages in flight)

template <int D>
struct AppendSmem {
  static constexpr int LD = D + 4;            // padded row stride (conflict-free 16-byte reads)
  float cb[kAppendNB][kAppendCw * LD];        // this CTA's codeword slices, ring of stages
  float rows[kAppendR * LD];                  // residuals (identical in every CTA)
  double rn[kAppendR];                        // residual norms
  float dist[kAppendCw][kAppendR];            // float32 distances of this CTA's codewords
  float cnorm[kAppendCw];                     // their squared norms
  // every CTA's per-row best (float64 distance, codeword), written by that CTA into every
  // CTA of the cluster; by stage parity
  double pub_d[2][kAppendCl][kAppendR];
  int pub_c[2][kAppendCl][kAppendR];
  uint8_t code[kAppendR][kMaxStages];
};

// Greedy residual codes of up to 8 rows into sm.code, in every CTA of the cluster.  row(r) is row
// r's fp16 vector (d contiguous) or null (an absent row).  CB: the head's [S][256][D] codebooks;
// smooth: the head's smoothing factors or null.  The caller passes a cluster barrier after its last
// use of sm before it leaves (other CTAs read this CTA's codewords).
template <int D, class Row>
__device__ __forceinline__ void encode_cluster(AppendSmem<D>& sm, const Row& row, const float* CB,
                                               int S, const float* smooth, double rot) {
  namespace cg = cooperative_groups;
  constexpr int E = D / 32;
  constexpr int LD = AppendSmem<D>::LD;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto load_slice = [&](int s) {      // stage s, codewords [32 rank, 32 rank + 32)
    const float* src = CB + ((size_t)s * kCodebook + (size_t)rank * kAppendCw) * D;
    float* dst = sm.cb[s % kAppendNB];
    for (int f = tid; f < kAppendCw * D / 4; f += 256) {
      const int cl = f / (D / 4), q = f % (D / 4);
      cp_async16(dst + cl * LD + 4 * q, src + (size_t)cl * D + 4 * q);
    }
    cp_async_commit();
  };

  // the first slices; every later one is issued (one commit group per stage) after the cluster
  // barrier of the stage whose buffer it reuses has been passed
  for (int q = 0; q < kAppendNB - 1 && q < S; ++q) load_slice(q);
  // rotated rows (every CTA of the cluster computes the same values)
  if (warp < kAppendR) {
    const __half* x = row(warp);
    double ss = 0.0;
    if (x) {
      double v[E];
      load_row_f64<E>(x, ZKV_DTYPE_F16, 0, lane, v);
      if (smooth) {   // keys: x / lambda per channel before the rotation
#pragma unroll
        for (int q = 0; q < E; ++q) v[q] *= 1.0 / (double)smooth[q * 32 + lane];
      }
      fwht_warp_f64<D>(v, lane);
#pragma unroll
      for (int q = 0; q < E; ++q) {
        const float y = (float)(v[q] * rot);
        sm.rows[warp * LD + q * 32 + lane] = y;
        ss += (double)y * (double)y;
      }
    } else {
#pragma unroll
      for (int q = 0; q < E; ++q) sm.rows[warp * LD + q * 32 + lane] = 0.f;
    }
    ss = warp_sum_f64(ss);
    if (lane == 0) sm.rn[warp] = sqrt(ss);
  }

  // distance pass: thread = (codeword pair, row half, dimension slice); slice ks holds the
  // 16-byte chunks 4 ks + 32 j of every vector (conflict-free 16-byte reads)
  const int ks = tid & 7, cpair = (tid >> 3) & 15, rhalf = tid >> 7;
  for (int s = 0; s < S; ++s) {
    // groups committed so far: stages 0 .. min(s + NB - 2, S - 1); stage s must be complete
    const int later = (s + kAppendNB - 2 < S - 1 ? s + kAppendNB - 2 : S - 1) - s;
    if (later >= 2) asm volatile("cp.async.wait_group 2;" ::: "memory");
    else if (later == 1) asm volatile("cp.async.wait_group 1;" ::: "memory");
    else asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();   // slice s and the residuals are ready
    const float* slice = sm.cb[s % kAppendNB];
    {
      float acc[2][4], cn[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        cn[u] = 0.f;
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[u][v] = 0.f;
      }
#pragma unroll
      for (int j = 0; j < D / 32; ++j) {
        const int off = 4 * ks + 32 * j;
        float4 c4[2], x4[4];
#pragma unroll
        for (int u = 0; u < 2; ++u) c4[u] = *reinterpret_cast<const float4*>(slice + (2 * cpair + u) * LD + off);
#pragma unroll
        for (int v = 0; v < 4; ++v) x4[v] = *reinterpret_cast<const float4*>(sm.rows + (4 * rhalf + v) * LD + off);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          cn[u] = fmaf(c4[u].x, c4[u].x, cn[u]);
          cn[u] = fmaf(c4[u].y, c4[u].y, cn[u]);
          cn[u] = fmaf(c4[u].z, c4[u].z, cn[u]);
          cn[u] = fmaf(c4[u].w, c4[u].w, cn[u]);
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            acc[u][v] = fmaf(x4[v].x, c4[u].x, acc[u][v]);
            acc[u][v] = fmaf(x4[v].y, c4[u].y, acc[u][v]);
            acc[u][v] = fmaf(x4[v].z, c4[u].z, acc[u][v]);
            acc[u][v] = fmaf(x4[v].w, c4[u].w, acc[u][v]);
          }
        }
      }
      // sum over the 8 slices (lanes differing in bits 0-2); the rounding bound used for the
      // margin holds for any summation order
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          cn[u] += __shfl_xor_sync(0xffffffffu, cn[u], o);
#pragma unroll
          for (int v = 0; v < 4; ++v) acc[u][v] += __shfl_xor_sync(0xffffffffu, acc[u][v], o);
        }
      }
      if (ks == 0) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          if (rhalf == 0) sm.cnorm[2 * cpair + u] = cn[u];
#pragma unroll
          for (int v = 0; v < 4; ++v) sm.dist[2 * cpair + u][4 * rhalf + v] = cn[u] - 2.f * acc[u][v];
        }
      }
    }
    __syncthreads();
    // warp r decides row r among this CTA's codewords (lane = local codeword): the row minimum
    // of the float32 distances, the candidates within the margin (taken with this slice's
    // largest codeword norm), their float64 distances, the best (lowest index on ties); it
    // then writes that best into every CTA of the cluster
    static_assert(kAppendCw == 32, "one lane per local codeword");
    if (warp < kAppendR) {
      const int r = warp;
      const float dr = sm.dist[lane][r];
      const float cmax = warp_max_f32(sm.cnorm[lane]);
      const float dmin = warp_min_f32(dr);
      const double thr = (double)dmin + candidate_margin(sm.rn[r], cmax, D);
      unsigned cand = __ballot_sync(0xffffffffu, (double)dr <= thr);
      double bd = DBL_MAX;
      int bc = kCodebook;
      while (cand) {
        const int c = __ffs(cand) - 1;
        cand &= cand - 1u;
        double a = 0.0;
#pragma unroll
        for (int q = 0; q < E; ++q) {
          const int i = q * 32 + lane;
          const double df = (double)sm.rows[r * LD + i] - (double)slice[c * LD + i];
          a = fma(df, df, a);
        }
        a = warp_sum_f64(a);
        const int gc = rank * kAppendCw + c;
        if (a < bd || (a == bd && gc < bc)) {
          bd = a;
          bc = gc;
        }
      }
      if (lane < kAppendCl) {
        AppendSmem<D>* o = cluster.map_shared_rank(&sm, lane);
        o->pub_d[s & 1][rank][r] = bd;
        o->pub_c[s & 1][rank][r] = bc;
      }
    }
    // every CTA's bests have arrived here; every read of stage s-1's slices is done
    cluster.sync();
    // the buffer of stage s-1 is free (its remote reads are done): refill it NB - 1 stages ahead
    if (s + kAppendNB - 1 < S) load_slice(s + kAppendNB - 1);
    // warp r: the cluster's best for row r (min over the 8 published bests, lowest index on
    // ties), then the residual update with that codeword, read from its owner's slice
    if (warp < kAppendR) {
      const int r = warp;
      double bd = lane < kAppendCl ? sm.pub_d[s & 1][lane][r] : DBL_MAX;
      int bc = lane < kAppendCl ? sm.pub_c[s & 1][lane][r] : kCodebook;
#pragma unroll
      for (int o = 1; o < kAppendCl; o <<= 1) {
        const double od = __shfl_xor_sync(0xffffffffu, bd, o);
        const int oc = __shfl_xor_sync(0xffffffffu, bc, o);
        if (od < bd || (od == bd && oc < bc)) {
          bd = od;
          bc = oc;
        }
      }
      // every lane of the warp holds the same choice (lanes 0-7 reduced the same set; the
      // others take lane 0's); non-finite rows match no candidate: never index past the
      // stage's codebook
      bc = __shfl_sync(0xffffffffu, bc, 0);
      const int z = bc < kCodebook ? bc : 0;
      const float* src = cluster.map_shared_rank(&sm.cb[s % kAppendNB][0], z / kAppendCw) + (z % kAppendCw) * LD;
      double ss = 0.0;
#pragma unroll
      for (int q = 0; q < E; ++q) {
        const int i = q * 32 + lane;
        const float nr = sm.rows[r * LD + i] - src[i];
        sm.rows[r * LD + i] = nr;
        ss += (double)nr * (double)nr;
      }
      ss = warp_sum_f64(ss);
      if (lane == 0) {
        sm.rn[r] = sqrt(ss);
        sm.code[r][s] = (uint8_t)z;
      }
    }
  }
}

}  // namespace zkv
