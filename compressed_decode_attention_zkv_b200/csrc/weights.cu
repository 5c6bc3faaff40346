// Attention weight that each compressed token received, added to running totals (sm_100a).
//
// Passages: zerokv-neo 4.0.0 (heavy_hitter_budget: tokens are kept by the attention that they
// received); VeloxQuant-MLX 0.5.1, "VecInfer" (the rotation is absorbed into the query, so a key
// score is a sum of per-stage table entries).
//
//   acc[b][kvh][t] += sum over the rows rho of (b, kvh) of 2^(score_rho[t] - lse_rho log2 e)
//
// Two kernels: the key lookup tables of every row (query_tables.cuh), then the scan.  A scan block
// takes kWtTok tokens of one (sequence, kv head) at a time, kWtTU per thread, through all row groups
// (one group's tables are loaded once for all its tokens): each token's total stays in a register and
// is added to memory once, by one thread.  As many blocks as are resident at once share the tokens.  Every token is
// read and written by exactly one thread, so the result does not depend on any order.
//
// Shared memory: the tables of one group of RG rows, a row of 128 bytes or more (copies of smaller ones)
// every 256 bytes per codeword, so that a gather's address is one byte permutation of the packed codes.  A thread reads 16 bytes
// (four rows) at a time.  The eight lanes of a 16-byte phase visit eight distinct 16-byte columns,
// modulo 128 bytes, of their codewords' rows (they start at different stages, row halves or copies),
// so a gather has no bank conflict whatever the codes are.
//
// A call among others: 8 sequences x 32640 tokens, 32 / 8 heads, 4 stages 18.4 us (29.3 MB: 25 % of the
// copy bandwidth), tables 8 us and scan 11 us; 130816 tokens, 28 / 4 heads, 2 stages 10.3 us.  The tables'
// latency and one block's chain (tables in, 8 tokens a thread, totals in and out) bound it.
#include "query_tables.cuh"

#include <cmath>

namespace zkv {

constexpr int kWtThreads = 512;
constexpr int kWtTU = 8;                        // tokens per thread
constexpr int kWtTok = kWtThreads * kWtTU;

struct WeightArgs {
  QueryTables qt;
  int B, N, G, Hkv, Sk, NRG;
  int64_t Tcap, max_comp;
  const float* lse;
  const uint8_t* k_codes;
  const int32_t* comp_len;
  float* acc;
  int32_t* err;
  const int32_t* table;
  int64_t max_pages, n_pages;
  int pshift;
};

template <int D>
__global__ void __launch_bounds__(kQtThreads) weights_tables_kernel(WeightArgs a) {
  extern __shared__ __align__(16) unsigned char smraw[];
  pdl_trigger();
  query_tables_block<D>(a.qt, blockIdx.x, *reinterpret_cast<QtSmem<D>*>(smraw));
}

// RG rows per group (4 or 8), SKP padded stages; a codeword's row: [stage][half][copy] 16-byte pieces
template <int SKP, int RG>
struct WtCfg {
  static constexpr int NH = RG / 4;                                   // 16-byte halves
  static constexpr int PC = SKP * NH > 8 ? SKP * NH : 8;              // 16-byte pieces of a row
  static constexpr int CP = PC / (SKP * NH);                          // table copies
  static constexpr int LS = SKP < 8 / NH ? SKP : 8 / NH;              // stages that lanes start at
  static constexpr int SMEM = kCodebook * 256 + RG * 4;
  static constexpr int KW = SKP <= 4 ? 1 : 2;
};

template <int SKP, int RG>
__global__ void __launch_bounds__(kWtThreads, 2) weights_scan_kernel(WeightArgs a) {
  using C = WtCfg<SKP, RG>;
  extern __shared__ __align__(16) unsigned char sm[];
  float* ls = reinterpret_cast<float*>(sm + kCodebook * 256);   // -lse in base 2; -inf: counts for nothing
  const int tid = threadIdx.x, lane = tid & 31;
  const int64_t pair = blockIdx.y;
  const int b = (int)(pair / a.Hkv), kvh = (int)(pair % a.Hkv);
  int64_t n = a.comp_len[b];
  if (n < 0 || n > a.Tcap) {
    if (tid == 0) set_error(a.err, ZKV_DEVERR_COMP_LEN);
    n = n < 0 ? 0 : a.Tcap;
  }
  if (n > a.max_comp) n = a.max_comp;
  const int present = present_queries(a.qt.n_query, b, a.N);
  if (a.qt.n_query && a.qt.n_query[b] != present && tid == 0) set_error(a.err, ZKV_DEVERR_DRAFT);
  const CodeRows kr = code_rows(a.k_codes, a.table, a.max_pages, a.n_pages, a.pshift, b, kvh, a.Hkv,
                                a.Tcap, a.Sk, a.err);
  // this thread's tokens: t0 + u kWtThreads.  Their codes are in flight across the wait for the tables
  // (that kernel does not write them) and beside the last tokens' additions.  A thread behind the last
  // token takes that one's and adds nothing.
  int64_t t0 = (int64_t)blockIdx.x * kWtTok + tid;
  uint32_t w[kWtTU][C::KW];
  const bool word = !a.table && SKP >= 2 && a.Sk == SKP;        // one aligned machine word per token
  auto load = [&]() {
    if (t0 - tid >= n) return;
    if (word) {
#pragma unroll
      for (int u = 0; u < kWtTU; ++u) {
        const int64_t t = t0 + u * kWtThreads;
        const uint8_t* p = kr.base + (t < n ? t : n - 1) * SKP;
        if constexpr (SKP == 2) {
          w[u][0] = __ldg(reinterpret_cast<const unsigned short*>(p));
        } else if constexpr (SKP == 4) {
          w[u][0] = __ldg(reinterpret_cast<const unsigned int*>(p));
        } else if constexpr (SKP == 8) {
          const uint2 x = __ldg(reinterpret_cast<const uint2*>(p));
          w[u][0] = x.x;
          w[u][C::KW - 1] = x.y;
        }
      }
    } else {
#pragma unroll
      for (int u = 0; u < kWtTU; ++u) {
        const int64_t t = t0 + u * kWtThreads;
        load_codes<SKP>(kr, (uint32_t)(t < n ? t : n - 1), a.Sk, w[u]);
      }
    }
  };
  load();
  // this lane's columns: starting half, stage and copy; the order that a code word's bytes are put in
  const int l8 = lane & 7;
  const int lh = l8 & (C::NH - 1), lst = (l8 / C::NH) & (C::LS - 1);
  const int lc = C::CP > 1 ? l8 / (C::NH * C::LS) : 0;
  uint32_t col[C::NH][(SKP + 1) / 2], order = 0u;
#pragma unroll
  for (int x = 0; x < C::NH; ++x)
#pragma unroll
    for (int i = 0; i < (SKP + 1) / 2; ++i) col[x][i] = 0u;
#pragma unroll
  for (int i = 0; i < SKP; ++i) {
    const int st = i ^ lst;
#pragma unroll
    for (int x = 0; x < C::NH; ++x)
      col[x][i / 2] |= (uint32_t)(16 * ((st * C::NH + (x ^ lh)) * C::CP + lc)) << (8 * (i & 1));
    if (i < 4) order |= (uint32_t)(st & 3) << (4 * i);
  }
  const bool cross = (lst & 4) != 0;           // (8 stages: the second word comes first)
  pdl_wait();
  if (t0 - tid >= n) return;
  if ((uint32_t)__cvta_generic_to_shared(sm) != kTableBase) {
    if (tid == 0) set_error(a.err, ZKV_DEVERR_SMEM);
    return;
  }
  bool loaded = false;
  while (t0 - tid < n) {
    float sum[kWtTU];
#pragma unroll
    for (int u = 0; u < kWtTU; ++u) sum[u] = 0.f;
    for (int rg = 0; rg < a.NRG; ++rg) {
      if (a.NRG > 1 || !loaded) {
        loaded = true;
        __syncthreads();
        if (tid < RG) {
          const int rho = rg * RG + tid;
          float x = -INFINITY;
          if (rho < a.qt.R && rho / a.G < present) {
            const float l = a.lse[((int64_t)b * a.N + rho / a.G) * (a.Hkv * a.G) + (int64_t)kvh * a.G + rho % a.G];
            if (fabsf(l) < INFINITY) x = -l * kLog2e;
          }
          ls[tid] = x;
        }
        __syncthreads();
        // tables; those of rows that count for nothing are zero (their queries may hold anything)
        const float* src = a.qt.lut + (pair * a.NRG + rg) * (int64_t)(kCodebook * SKP * RG);
        // thread = one 16-byte piece of a codeword's row: whole rows are written, no bank conflict
        constexpr int PER = kWtThreads / C::PC, TURNS = kCodebook / PER;
        const int piece = tid % C::PC, q = piece / C::CP, r4 = 4 * (q & (C::NH - 1));
        const bool dead[4] = {ls[r4] == -INFINITY, ls[r4 + 1] == -INFINITY, ls[r4 + 2] == -INFINITY, ls[r4 + 3] == -INFINITY};
#pragma unroll
        for (int k0 = 0; k0 < TURNS; k0 += 4) {
          float4 v[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            v[k] = *reinterpret_cast<const float4*>(src + ((tid / C::PC + (k0 + k) * PER) * SKP * C::NH + q) * 4);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            *reinterpret_cast<float4*>(sm + (tid / C::PC + (k0 + k) * PER) * 256 + 16 * piece) =
              make_float4(dead[0] ? 0.f : v[k].x, dead[1] ? 0.f : v[k].y, dead[2] ? 0.f : v[k].z, dead[3] ? 0.f : v[k].w);
        }
        __syncthreads();
      }
      float2 init[C::NH][2];
#pragma unroll
      for (int x = 0; x < C::NH; ++x)
#pragma unroll
        for (int q = 0; q < 2; ++q)
          init[x][q] = *reinterpret_cast<const float2*>(ls + 4 * (x ^ lh) + 2 * q);
#pragma unroll
      for (int u = 0; u < kWtTU; ++u) {
        float2 s[C::NH][2];
#pragma unroll
        for (int x = 0; x < C::NH; ++x) s[x][0] = init[x][0], s[x][1] = init[x][1];
        uint32_t y[C::KW];
#pragma unroll
        for (int i = 0; i < C::KW; ++i)
          y[i] = byte_perm(C::KW > 1 && cross ? w[u][C::KW - 1 - i] : w[u][i], 0u, order);
#pragma unroll
        for (int i = 0; i < SKP; ++i)
#pragma unroll
          for (int x = 0; x < C::NH; ++x) {
            const float4 v = lds_quad(byte_perm(y[i < 4 ? 0 : C::KW - 1], col[x][i / 2],
                                                (4u + (i & 1)) | ((i & 3u) << 4) | 0x7600u));
            s[x][0] = fadd2(s[x][0], make_float2(v.x, v.y));
            s[x][1] = fadd2(s[x][1], make_float2(v.z, v.w));
          }
#pragma unroll
        for (int x = 0; x < C::NH; ++x)
          sum[u] += (ex2_ftz(s[x][0].x) + ex2_ftz(s[x][0].y)) + (ex2_ftz(s[x][1].x) + ex2_ftz(s[x][1].y));
      }
    }
    float* acc = a.acc + pair * a.Tcap + t0;
    const int left = (int)(n - t0 < 0 ? 0 : n - t0 < kWtTok ? n - t0 : kWtTok);
    t0 += (int64_t)gridDim.x * kWtTok;
    load();
#pragma unroll
    for (int u = 0; u < kWtTU; ++u) sum[u] += u * kWtThreads < left ? acc[u * kWtThreads] : 0.f;
#pragma unroll
    for (int u = 0; u < kWtTU; ++u)
      if (u * kWtThreads < left) acc[u * kWtThreads] = sum[u];
  }
}

static int weights_rows(const zkv_weights_params* p) { return p->N * (p->Hq / p->Hkv); }
static int weights_rg(const zkv_weights_params* p) { return weights_rows(p) <= 4 ? 4 : 8; }
static int weights_pad(int S) { return S <= 2 ? S : S <= 4 ? 4 : 8; }

static int validate_weights_shapes(const zkv_weights_params* p) {
  if (!p) return ZKV_ERR_INVALID_ARG;
  if (p->B < 1 || p->N < 1 || p->Hq < 1 || p->Hkv < 1 || p->Hq % p->Hkv) return ZKV_ERR_INVALID_ARG;
  if (!supported_d(p->d)) return ZKV_ERR_UNSUPPORTED;
  if (p->Sk < 1 || p->Sk > kMaxStages) return ZKV_ERR_UNSUPPORTED;
  if (p->Hq / p->Hkv > 8 || p->N > 256) return ZKV_ERR_UNSUPPORTED;
  if ((int64_t)p->B * p->Hkv > 65535 || (int64_t)p->B * p->Hkv * p->N > (1 << 24))
    return ZKV_ERR_UNSUPPORTED;
  if (p->Tcap < 0 || p->max_comp_len < 0 || p->max_comp_len > p->Tcap || p->Tcap % 16)
    return ZKV_ERR_INVALID_ARG;
  if (p->Tcap > (int64_t(1) << 28)) return ZKV_ERR_UNSUPPORTED;
  return validate_paged(p->block_table, p->page_tokens, p->max_pages, p->n_pages, p->Tcap);
}

static size_t weights_workspace(const zkv_weights_params* p) {
  const int rg = weights_rg(p);
  const int rp = (weights_rows(p) + rg - 1) / rg * rg;
  return align256(query_tables_bytes((int64_t)p->B * p->Hkv, rp, weights_pad(p->Sk)));
}

template <int SKP, int RG>
static cudaError_t launch_weights_scan(const WeightArgs& a, dim3 grid, cudaStream_t st) {
  using C = WtCfg<SKP, RG>;
  const cudaError_t e = ensure_smem_limit(weights_scan_kernel<SKP, RG>, C::SMEM);
  if (e != cudaSuccess) return e;
  return launch_pdl(weights_scan_kernel<SKP, RG>, grid, dim3(kWtThreads), C::SMEM, st, a);
}

template <int D>
static cudaError_t launch_weights_tables(const WeightArgs& a, cudaStream_t st) {
  const cudaError_t e = ensure_smem_limit(weights_tables_kernel<D>, sizeof(QtSmem<D>));
  if (e != cudaSuccess) return e;
  weights_tables_kernel<D><<<(unsigned)a.qt.blocks(), kQtThreads, sizeof(QtSmem<D>), st>>>(a);
  return cudaGetLastError();
}

}  // namespace zkv

using namespace zkv;

extern "C" size_t zkv_weights_workspace_size(const zkv_weights_params* p) {
  if (validate_weights_shapes(p) != ZKV_OK) return 0;
  return weights_workspace(p);
}

extern "C" int zkv_rvq_accumulate_weights(const zkv_weights_params* p, void* workspace,
                                          size_t workspace_bytes, void* stream) {
  const int v = validate_weights_shapes(p);
  if (v != ZKV_OK) return v;
  if (!p->q || !p->lse || !p->k_codes || !p->comp_len || !p->k_codebooks || !p->acc)
    return ZKV_ERR_INVALID_ARG;
  if (((uintptr_t)p->q | (uintptr_t)p->k_codes | (uintptr_t)p->k_codebooks) & 15)
    return ZKV_ERR_INVALID_ARG;
  const int64_t qs[3] = {p->q_sb, p->q_sn, p->q_sh};
  for (int64_t s : qs)
    if (s < 0 || s % 8) return ZKV_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < weights_workspace(p) || ((uintptr_t)workspace & 255))
    return ZKV_ERR_WORKSPACE;
  if (p->max_comp_len == 0) return ZKV_OK;       // no token to add to
  const float scale = p->softmax_scale > 0.f ? p->softmax_scale : (float)(1.0 / std::sqrt((double)p->d));
  const int RG = weights_rg(p);
  WeightArgs a{};
  a.B = p->B; a.N = p->N; a.G = p->Hq / p->Hkv; a.Hkv = p->Hkv; a.Sk = p->Sk;
  a.Tcap = p->Tcap; a.max_comp = p->max_comp_len;
  a.lse = p->lse; a.k_codes = p->k_codes; a.comp_len = p->comp_len; a.acc = p->acc;
  a.err = p->error_flag;
  a.table = p->block_table; a.max_pages = p->max_pages; a.n_pages = p->n_pages;
  a.pshift = p->block_table ? log2_pow2(p->page_tokens) : 0;
  QueryTables& q = a.qt;
  q.B = p->B; q.N = p->N; q.G = a.G; q.Hkv = p->Hkv; q.Sk = p->Sk; q.SKP = weights_pad(p->Sk);
  q.RG = RG;
  q.R = weights_rows(p);
  q.RP = (q.R + RG - 1) / RG * RG;
  a.NRG = q.RP / RG;
  q.q = reinterpret_cast<const __half*>(p->q);
  q.q_sb = p->q_sb; q.q_sn = p->q_sn; q.q_sh = p->q_sh;
  q.n_query = p->n_draft; q.Ck = p->k_codebooks; q.k_smooth = p->k_smooth;
  q.scale_log2 = (float)((double)scale * 1.4426950408889634);
  q.rot = 1.0 / std::sqrt((double)p->d);
  q.set_divisors();
  q.lut = reinterpret_cast<float*>(workspace);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = p->d == 64 ? launch_weights_tables<64>(a, st)
                : p->d == 128 ? launch_weights_tables<128>(a, st) : launch_weights_tables<256>(a, st);
  if (e != cudaSuccess) return ZKV_ERR_CUDA;
  // two blocks per SM are resident
  const int64_t pairs = (int64_t)p->B * p->Hkv, chunks = (p->max_comp_len + kWtTok - 1) / kWtTok;
  const int64_t share = 296 / pairs < 1 ? 1 : 296 / pairs;
  const dim3 grid((unsigned)(chunks < share ? chunks : share), (unsigned)pairs);
  if (RG == 4) {
    e = q.SKP == 1 ? launch_weights_scan<1, 4>(a, grid, st) : q.SKP == 2 ? launch_weights_scan<2, 4>(a, grid, st)
      : q.SKP == 4 ? launch_weights_scan<4, 4>(a, grid, st) : launch_weights_scan<8, 4>(a, grid, st);
  } else {
    e = q.SKP == 1 ? launch_weights_scan<1, 8>(a, grid, st) : q.SKP == 2 ? launch_weights_scan<2, 8>(a, grid, st)
      : q.SKP == 4 ? launch_weights_scan<4, 8>(a, grid, st) : launch_weights_scan<8, 8>(a, grid, st);
  }
  return e == cudaSuccess ? ZKV_OK : ZKV_ERR_CUDA;
}
