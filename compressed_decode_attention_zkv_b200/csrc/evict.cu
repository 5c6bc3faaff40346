// Eviction from the compressed prefix by accumulated attention weight (sm_100a).
//
// Passages: zerokv-neo 4.0.0 (heavy_hitter_budget: a budget of tokens, the newest ones and those
// that received the most attention).
//
// One thread-block cluster per (sequence, kv head).  CTA k owns a contiguous range of the tokens and
// keeps their totals as order-preserving 32-bit keys in its shared memory (read once).
//   1. The key of the last kept old token: a radix selection, 11 + 11 + 10 bits from the top.  Per
//      pass each CTA counts the digit of its keys that match the prefix so far; the clusters' counts
//      are summed over distributed shared memory.
//   2. A token is kept if it is among the newest, if its key is larger than that key, or if it is
//      equal and among the first of those (lowest position).  Flags become a bit mask with counts per
//      32 tokens, and CTA offsets.
//   3. Destination positions, in rounds of ascending order: each thread finds the source of one
//      destination from the bit masks, reads its codes and total, and writes them.  A source never
//      lies before its destination, so reading a whole round before any of it is written (a cluster
//      barrier between) makes the move safe in place.
#include <cooperative_groups.h>

#include "query_tables.cuh"

namespace cg = cooperative_groups;

namespace zkv {

constexpr int kEvThreads = 512;
constexpr int kEvBins = 2048;
constexpr int kEvMaxCl = 8;

struct EvictArgs {
  int B, Hkv, Sk, Sv;
  int64_t Tcap, Tout, keep, recent;
  const uint8_t *k_codes, *v_codes;
  const float* acc;
  const int32_t* comp_len;
  uint8_t *k_out, *v_out;
  float* acc_out;
  int32_t* kept;
  int32_t* err;
  const int32_t *table, *table_out;
  int64_t max_pages, n_pages, max_pages_out, n_pages_out;
  int pshift, pshift_out;
  int chunk;          // tokens per CTA (a multiple of 32)
  int in_place;
};

// Order-preserving key of a total: NaN smallest, -0 as +0.
__device__ __forceinline__ uint32_t total_key(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x == 0.f ? 0.f : x);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

struct EvictSmem {
  uint32_t hist[kEvBins];
  uint32_t sum[kEvBins];
  uint32_t warp[kEvThreads / 32];
  uint32_t digit, before;           // chosen digit; keys of the cluster above it
  uint32_t cnt;                     // this CTA's count of the moment (equal keys, then kept tokens)
};

// exclusive prefix sum over the block; `all` = the block's total
__device__ __forceinline__ uint32_t block_scan(uint32_t x, uint32_t* ws, uint32_t& all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t s = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += y;
  }
  __syncthreads();
  if (lane == 31) ws[warp] = s;
  __syncthreads();
  uint32_t before = 0;
  all = 0;
#pragma unroll
  for (int w = 0; w < kEvThreads / 32; ++w) {
    if (w < warp) before += ws[w];
    all += ws[w];
  }
  return before + s - x;
}

__device__ __forceinline__ uint8_t* out_row(uint8_t* codes, const EvictArgs& a, int b, int kvh,
                                            int64_t t, int S) {
  if (!a.table_out) return codes + (((int64_t)b * a.Hkv + kvh) * a.Tout + t) * S;
  const int64_t pg = a.table_out[b * a.max_pages_out + (t >> a.pshift_out)];
  if (pg < 0 || pg >= a.n_pages_out) {
    set_error(a.err, ZKV_DEVERR_PAGE);
    return nullptr;
  }
  return codes + (((pg * a.Hkv + kvh) << a.pshift_out) + (t & ((1 << a.pshift_out) - 1))) * S;
}

__device__ __forceinline__ void store_codes(uint8_t* p, int S, const uint32_t (&w)[2]) {
  if (!p) return;
  if (S == 4) {
    *reinterpret_cast<uint32_t*>(p) = w[0];
  } else if (S == 2) {
    *reinterpret_cast<unsigned short*>(p) = (unsigned short)w[0];
  } else if (S == 8) {
    *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  } else {
    for (int s = 0; s < S; ++s) p[s] = (uint8_t)(w[s >> 2] >> (8 * (s & 3)));
  }
}

__global__ void __launch_bounds__(kEvThreads) evict_kernel(EvictArgs a) {
  extern __shared__ __align__(16) unsigned char smraw[];
  EvictSmem& sm = *reinterpret_cast<EvictSmem*>(smraw);
  uint32_t* bits = reinterpret_cast<uint32_t*>(smraw + sizeof(EvictSmem));   // [chunk / 32]
  uint32_t* pre = bits + a.chunk / 32;                                       // kept before, per word
  uint32_t* keys = pre + a.chunk / 32;                                       // [chunk]
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31;
  const int64_t pair = blockIdx.x / C;
  const int b = (int)(pair / a.Hkv), kvh = (int)(pair % a.Hkv);
  int64_t n = a.comp_len[b];
  if (n < 0 || n > a.Tcap) {
    if (tid == 0 && rank == 0) set_error(a.err, ZKV_DEVERR_COMP_LEN);
    n = n < 0 ? 0 : a.Tcap;
  }
  const bool all_kept = n <= a.keep;
  const int64_t m = all_kept ? n : a.keep;
  const int64_t old = all_kept ? 0 : n - a.recent;      // tokens before the newest
  const int64_t heavy = all_kept ? 0 : a.keep - a.recent;
  const int64_t begin = (int64_t)rank * a.chunk;
  const int mine = (int)(n - begin < 0 ? 0 : n - begin < a.chunk ? n - begin : a.chunk);
  const int mold = (int)(old - begin < 0 ? 0 : old - begin < a.chunk ? old - begin : a.chunk);
  const float* acc = a.acc + pair * a.Tcap;

  uint32_t threshold = 0u;
  int64_t equal = 0;           // tokens with that key that are kept
  if (heavy > 0) {
    for (int t = tid; t < mold; t += kEvThreads) keys[t] = total_key(acc[begin + t]);
    uint32_t prefix = 0u, mask = 0u;
    int64_t want = heavy;      // rank of the sought key among those that match the prefix
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const int nb = pass == 2 ? 1024 : 2048;
      for (int i = tid; i < kEvBins; i += kEvThreads) sm.hist[i] = 0u;
      __syncthreads();
      for (int t = tid; t < mold; t += kEvThreads) {
        const uint32_t k = keys[t];
        if ((k & mask) == prefix) atomicAdd(&sm.hist[(k >> shift) & (nb - 1)], 1u);
      }
      cluster.sync();
      // the cluster's counts; thread i sums the four highest-first digits 4 i .. 4 i + 3
      uint32_t h[4], tot = 0;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        h[q] = 0u;
        const int d = nb - 1 - (4 * tid + q);
        if (d >= 0)
          for (int c = 0; c < C; ++c) h[q] += cluster.map_shared_rank(&sm.hist[0], c)[d];
        tot += h[q];
      }
      uint32_t all;
      uint32_t before = block_scan(tot, sm.warp, all);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (before < want && want <= (int64_t)before + h[q]) {
          sm.digit = (uint32_t)(nb - 1 - (4 * tid + q));
          sm.before = before;
        }
        before += h[q];
      }
      cluster.sync();          // (every CTA has read the counts, and this block its digit)
      prefix |= sm.digit << shift;
      mask |= (uint32_t)(nb - 1) << shift;
      want -= sm.before;
      __syncthreads();
    }
    threshold = prefix;
    equal = want;
  }
  // equal keys in the CTAs before this one
  int64_t eq_before = 0;
  const int per = (mine + kEvThreads - 1) / kEvThreads + 31;
  const int words = (per / 32) * 1;       // 32-token words per thread, contiguous
  const int w0 = tid * words;
  const int nw = a.chunk / 32;
  if (heavy > 0) {
    uint32_t c = 0;
    for (int w = w0; w < w0 + words && w < nw; ++w)
      for (int i = 0; i < 32; ++i) {
        const int t = 32 * w + ((i + lane) & 31);
        if (t < mold && keys[t] == threshold) ++c;
      }
    uint32_t all;
    const uint32_t mineq = block_scan(c, sm.warp, all);
    if (tid == 0) sm.cnt = all;
    cluster.sync();
    for (int r = 0; r < rank; ++r) eq_before += *cluster.map_shared_rank(&sm.cnt, r);
    eq_before += mineq;
    cluster.sync();
  }
  // flags and counts
  uint32_t count = 0;
  for (int w = w0; w < w0 + words && w < nw; ++w) {
    uint32_t gt = 0, eq = 0, fix = 0;
    for (int i = 0; i < 32; ++i) {
      const int j = (i + lane) & 31, t = 32 * w + j;
      if (t >= mine) continue;
      if (t >= mold) {
        fix |= 1u << j;
      } else if (heavy > 0) {
        if (keys[t] > threshold) gt |= 1u << j;
        else if (keys[t] == threshold) eq |= 1u << j;
      }
    }
    while (eq) {               // the lowest positions first, while there is room
      const uint32_t low = eq & (0u - eq);
      eq ^= low;
      if (eq_before < equal) gt |= low;
      ++eq_before;
    }
    bits[w] = gt | fix;
    count += __popc(gt | fix);
  }
  uint32_t kept_here;
  uint32_t at = block_scan(count, sm.warp, kept_here);
  for (int w = w0; w < w0 + words && w < nw; ++w) {
    pre[w] = at;
    at += __popc(bits[w]);
  }
  // words behind the last token (no thread's share)
  for (int w = kEvThreads * words + tid; w < nw; w += kEvThreads) {
    bits[w] = 0u;
    pre[w] = kept_here;
  }
  if (tid == 0) sm.cnt = kept_here;
  cluster.sync();
  uint32_t off[kEvMaxCl + 1];
  off[0] = 0;
#pragma unroll
  for (int r = 0; r < kEvMaxCl; ++r)
    off[r + 1] = off[r] + (r < C ? *cluster.map_shared_rank(&sm.cnt, r) : 0u);

  const CodeRows kr = code_rows(a.k_codes, a.table, a.max_pages, a.n_pages, a.pshift, b, kvh, a.Hkv,
                                a.Tcap, a.Sk, a.err);
  const CodeRows vr = code_rows(a.v_codes, a.table, a.max_pages, a.n_pages, a.pshift, b, kvh, a.Hkv,
                                a.Tcap, a.Sv, a.err);
  float* acc_out = a.acc_out + pair * a.Tout;
  const int64_t round = (int64_t)C * kEvThreads;
  for (int64_t j0 = 0; j0 < m; j0 += round) {
    const int64_t j = j0 + rank * kEvThreads + tid;
    uint32_t wk[2] = {0u, 0u}, wv[2] = {0u, 0u};
    float x = 0.f;
    int64_t src = -1;
    if (j < m) {
      int r = 0;
#pragma unroll
      for (int q = 1; q < kEvMaxCl; ++q)
        if (q < C && j >= off[q]) r = q;
      const uint32_t local = (uint32_t)(j - off[r]);
      const uint32_t* rp = cluster.map_shared_rank(pre, r);
      const uint32_t* rb = cluster.map_shared_rank(bits, r);
      int lo = 0, hi = nw;     // the last word with pre <= local
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (rp[mid] <= local) lo = mid;
        else hi = mid;
      }
      src = (int64_t)r * a.chunk + 32 * lo + __fns(rb[lo], 0, (int)(local - rp[lo]) + 1);
      load_codes<8, false>(kr, (uint32_t)src, a.Sk, wk);
      load_codes<8, false>(vr, (uint32_t)src, a.Sv, wv);
      x = acc[src];
    }
    if (a.in_place) cluster.sync();
    if (j < m) {
      store_codes(out_row(a.k_out, a, b, kvh, j, a.Sk), a.Sk, wk);
      store_codes(out_row(a.v_out, a, b, kvh, j, a.Sv), a.Sv, wv);
      acc_out[j] = x;
      if (a.kept) a.kept[pair * a.keep + j] = (int32_t)src;
    }
    if (a.in_place) cluster.sync();
  }
  // tokens to come start without a total
  const int64_t zero_to = n < a.Tout ? n : a.Tout;
  for (int64_t j = m + rank * kEvThreads + tid; j < zero_to; j += round) acc_out[j] = 0.f;
  if (a.kept)
    for (int64_t j = m + rank * kEvThreads + tid; j < a.keep; j += round) a.kept[pair * a.keep + j] = -1;
  cluster.sync();              // no CTA leaves while another may read its shared memory
}

// after every CTA has read comp_len (len_out may be the same array)
__global__ void evict_lengths_kernel(int B, int64_t Tcap, int64_t keep, const int32_t* comp_len,
                                     int32_t* len_out) {
  const int b = blockIdx.x * blockDim.x + threadIdx.x;
  if (b >= B) return;
  int64_t n = comp_len[b];
  n = n < 0 ? 0 : n > Tcap ? Tcap : n;
  len_out[b] = (int32_t)(n < keep ? n : keep);
}

static size_t evict_smem(int chunk) { return sizeof(EvictSmem) + (size_t)chunk / 32 * 8 + (size_t)chunk * 4; }

}  // namespace zkv

using namespace zkv;

extern "C" int zkv_rvq_evict(const zkv_evict_params* p, void* stream) {
  if (!p) return ZKV_ERR_INVALID_ARG;
  if (p->B < 1 || p->Hkv < 1 || p->Tcap < 1 || p->Tcap_out < 1) return ZKV_ERR_INVALID_ARG;
  if (p->keep < 1 || p->keep > p->Tcap_out || p->recent < 0 || p->recent > p->keep)
    return ZKV_ERR_INVALID_ARG;
  if (p->Sk < 1 || p->Sk > kMaxStages || p->Sv < 1 || p->Sv > kMaxStages) return ZKV_ERR_UNSUPPORTED;
  if (p->Tcap > ZKV_EVICT_MAX_TOKENS || p->Tcap_out > (int64_t(1) << 28)) return ZKV_ERR_UNSUPPORTED;
  if ((int64_t)p->B * p->Hkv > (1 << 24)) return ZKV_ERR_UNSUPPORTED;
  if (!p->k_codes || !p->v_codes || !p->acc || !p->comp_len || !p->k_out || !p->v_out ||
      !p->acc_out || !p->len_out)
    return ZKV_ERR_INVALID_ARG;
  const uintptr_t al = (uintptr_t)p->k_codes | (uintptr_t)p->v_codes | (uintptr_t)p->k_out |
                       (uintptr_t)p->v_out;
  if (al & 15) return ZKV_ERR_INVALID_ARG;
  int v = validate_paged(p->block_table, p->page_tokens, p->max_pages, p->n_pages, p->Tcap);
  if (v != ZKV_OK) return v;
  v = validate_paged(p->block_table_out, p->page_tokens_out, p->max_pages_out, p->n_pages_out, p->Tcap_out);
  if (v != ZKV_OK) return v;
  const bool codes_in_place = p->k_out == p->k_codes || p->v_out == p->v_codes;
  if (codes_in_place && (p->Tcap_out != p->Tcap || p->block_table_out != p->block_table ||
                         p->page_tokens_out != p->page_tokens))
    return ZKV_ERR_INVALID_ARG;
  if (p->acc_out == p->acc && p->Tcap_out != p->Tcap) return ZKV_ERR_INVALID_ARG;
  EvictArgs a{};
  a.B = p->B; a.Hkv = p->Hkv; a.Sk = p->Sk; a.Sv = p->Sv;
  a.Tcap = p->Tcap; a.Tout = p->Tcap_out; a.keep = p->keep; a.recent = p->recent;
  a.k_codes = p->k_codes; a.v_codes = p->v_codes; a.acc = p->acc; a.comp_len = p->comp_len;
  a.k_out = p->k_out; a.v_out = p->v_out; a.acc_out = p->acc_out; a.kept = p->kept;
  a.err = p->error_flag;
  a.table = p->block_table; a.max_pages = p->max_pages; a.n_pages = p->n_pages;
  a.table_out = p->block_table_out; a.max_pages_out = p->max_pages_out; a.n_pages_out = p->n_pages_out;
  a.pshift = p->block_table ? log2_pow2(p->page_tokens) : 0;
  a.pshift_out = p->block_table_out ? log2_pow2(p->page_tokens_out) : 0;
  a.in_place = codes_in_place || p->acc_out == p->acc;
  int C = 1;
  while (C < kEvMaxCl && p->Tcap > (int64_t)C * 4096) C *= 2;
  const int64_t per = (p->Tcap + C - 1) / C;
  a.chunk = (int)((per + 31) / 32 * 32);
  const size_t smem = evict_smem(a.chunk);
  if (ensure_smem_limit(evict_kernel, smem) != cudaSuccess) return ZKV_ERR_CUDA;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((int64_t)p->B * p->Hkv * C));
  cfg.blockDim = dim3(kEvThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, evict_kernel, a) != cudaSuccess) return ZKV_ERR_CUDA;
  evict_lengths_kernel<<<(p->B + 127) / 128, 128, 0, st>>>(p->B, p->Tcap, p->keep, p->comp_len, p->len_out);
  ZKV_CHECK_LAUNCH();
  return ZKV_OK;
}
