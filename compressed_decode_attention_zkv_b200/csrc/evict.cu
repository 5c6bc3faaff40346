// Eviction from the compressed prefix by accumulated attention weight (sm_100a).
//
// Passages: zerokv-neo 4.0.0 (heavy_hitter_budget: a budget of tokens, the newest ones and those
// that received the most attention).
//
// One thread-block cluster per (sequence, kv head); every CTA owns a contiguous range of the tokens,
// every warp 32 KPT tokens in a row (lane = token of a group of 32), whose totals it keeps in
// registers as order-preserving 32-bit keys: they are read once.
//   1. The key of the last kept old token: a radix selection, 11 + 11 + 10 bits from the top.  Per
//      pass each CTA counts the digits of its keys that match the prefix so far; the cluster's
//      counts are summed over distributed shared memory.
//   2. A token is kept if it is among the newest, if its key is larger than that key, or if it is
//      equal and among the first of those (lowest position).  A ballot makes the flags of 32 tokens
//      a word; with g and e the larger and equal keys before a word, the kept tokens before it are
//      g + min(e, equal keys kept), so one prefix sum gives every destination.
//   3. Copy.  Kept neighbours go to neighbouring places.  In place, a CTA first collects its kept
//      rows in shared memory, four bytes of each at a time, and writes after a cluster barrier: by
//      then every source of the (sequence, kv head) has been read.
// A call in a graph, inputs larger than the L2 except the last: 64 (sequence, kv head)s of 32640 tokens, an
// eighth kept, 4 + 4 stages: 19.7 us to other buffers (pages: 22.0), 26.2 us in place (pages: 29.6); 4 of
// 130816, a quarter kept, 2 + 4 stages: 22.4 (28.8) and 32.3 (37.0); one of 960: 8.2 (9.9) and 11.1 (11.6).
// In place a turn per four bytes of a row, each with a cluster barrier, and the kernel that writes the
// lengths come on top.  Chains of latency bound it (cycles of one CTA of 16320 tokens, to other buffers:
// totals in 3600, three passes 3500 to 4500 each, a cluster barrier and remote counts in each; flags and
// offsets 1700, sources 3000, copies 3800), not bytes (14.6 MB: 11 % of the copy bandwidth).
// The cluster has as many CTAs as the range needs and, up to 8, as leave no SM without work.
#include <cooperative_groups.h>

#include "query_tables.cuh"

namespace cg = cooperative_groups;

namespace zkv {

constexpr int kEvThreads = 1024;
constexpr int kEvWarps = kEvThreads / 32;
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
  int32_t* len_out;                 // null: a kernel after this one writes it (it is comp_len)
  int32_t* err;
  const int32_t *table, *table_out;
  int64_t max_pages, n_pages, max_pages_out, n_pages_out;
  int pshift, pshift_out;
  int in_place;
};

// Order-preserving key of a total: NaN smallest, -0 as +0.
__device__ __forceinline__ uint32_t total_key(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x == 0.f ? 0.f : x);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

struct EvictSmem {
  uint32_t hist[2][kEvBins];        // passes take turns
  uint32_t ws[2][kEvWarps];
  uint32_t digit, before, found;    // chosen digit; keys of the cluster above it, and with it
  alignas(8) uint32_t count[2];     // this CTA's larger and equal keys
};

__device__ __forceinline__ uint32_t warp_scan(uint32_t x, int lane) {   // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

// exclusive prefix sums of two counts over the block's warps, given each warp's totals in every lane
__device__ __forceinline__ void warp_offsets(uint32_t x, uint32_t y, EvictSmem& sm, uint32_t& bx, uint32_t& by,
                                             uint32_t& ax, uint32_t& ay) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  static_assert(kEvWarps == 32, "one lane per warp");
  if (lane == 0) {
    sm.ws[0][warp] = x;
    sm.ws[1][warp] = y;
  }
  __syncthreads();
  const uint32_t u = sm.ws[0][lane], v = sm.ws[1][lane];
  const uint32_t su = warp_scan(u, lane), sv = warp_scan(v, lane);
  bx = __shfl_sync(0xffffffffu, su - u, warp);
  by = __shfl_sync(0xffffffffu, sv - v, warp);
  ax = __shfl_sync(0xffffffffu, su, 31);
  ay = __shfl_sync(0xffffffffu, sv, 31);
  __syncthreads();
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

template <int KPT>
__global__ void __launch_bounds__(kEvThreads) evict_kernel(EvictArgs a) {
  constexpr int CHUNK = kEvThreads * KPT;      // tokens per CTA
  extern __shared__ __align__(16) unsigned char smraw[];
  EvictSmem& sm = *reinterpret_cast<EvictSmem*>(smraw);
  uint32_t* bits = reinterpret_cast<uint32_t*>(smraw + sizeof(EvictSmem));   // [CHUNK / 32] kept flags
  uint32_t* pre = bits + CHUNK / 32;                                         // kept tokens of the CTA before
  uint16_t* src = reinterpret_cast<uint16_t*>(pre + CHUNK / 32);             // [CHUNK] kept tokens
  uint32_t* list = reinterpret_cast<uint32_t*>(src + CHUNK);                 // [CHUNK] (in place)
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t pair = blockIdx.x / C;
  const int b = (int)(pair / a.Hkv), kvh = (int)(pair % a.Hkv);
  pdl_trigger();
  auto cluster_sync = [&]() {
    if (C > 1) cluster.sync();
    else __syncthreads();
  };
  int64_t n = a.comp_len[b];
  if (n < 0 || n > a.Tcap) {
    if (tid == 0 && rank == 0) set_error(a.err, ZKV_DEVERR_COMP_LEN);
    n = n < 0 ? 0 : a.Tcap;
  }
  if (a.len_out && kvh == 0 && rank == 0 && tid == 0) a.len_out[b] = (int32_t)(n < a.keep ? n : a.keep);
  const bool all_kept = n <= a.keep;
  const int m = (int)(all_kept ? n : a.keep);
  const int old = (int)(all_kept ? 0 : n - a.recent);       // tokens before the newest
  const int heavy = (int)(all_kept ? 0 : a.keep - a.recent);
  const int first = rank * CHUNK + warp * 32 * KPT + lane;  // this lane's tokens: first + 32 k
  const float* acc = a.acc + pair * a.Tcap;

  uint32_t threshold = 0u;
  int equal = 0;               // tokens with that key that are kept
  bool ties = false;           // more have it
  uint32_t keys[KPT];
  if (heavy > 0) {
    // (no branch per load: all are in flight together; old > 0 here)
    float x[KPT];
    if (first + 32 * (KPT - 1) < old) {
      const float* from = acc + first;
#pragma unroll
      for (int k = 0; k < KPT; ++k) x[k] = __ldcg(from + 32 * k);
    } else {
#pragma unroll
      for (int k = 0; k < KPT; ++k) x[k] = __ldcg(acc + min(first + 32 * k, old - 1));
    }
#pragma unroll
    for (int k = 0; k < KPT; ++k) keys[k] = total_key(x[k]);
    const bool full = __all_sync(0xffffffffu, first + 32 * (KPT - 1) < old);   // all of the warp's tokens are old
    uint32_t prefix = 0u, mask = 0u;
    uint32_t want = heavy;     // rank of the sought key among those that match the prefix
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const int nb = pass == 2 ? 1024 : 2048;
      // (its last readers, two passes ago, came to the barrier of the pass between)
      uint32_t* hist = sm.hist[pass & 1];
      for (int i = tid; i < kEvBins; i += kEvThreads) hist[i] = 0u;
      __syncthreads();
      if (pass == 0 && full) {
#pragma unroll
        for (int k = 0; k < KPT; ++k) atomicAdd(&hist[keys[k] >> 21], 1u);
      } else if (full) {
#pragma unroll
        for (int k = 0; k < KPT; ++k)
          if (((keys[k] ^ prefix) & mask) == 0u) atomicAdd(&hist[(keys[k] >> shift) & (nb - 1)], 1u);
      } else {
#pragma unroll
        for (int k = 0; k < KPT; ++k)
          if ((first + 32 * k < old) & (((keys[k] ^ prefix) & mask) == 0u))
            atomicAdd(&hist[(keys[k] >> shift) & (nb - 1)], 1u);
      }
      cluster_sync();
      // the cluster's counts from the highest digit down: thread i has digits 2 i and 2 i + 1
      static_assert(kEvBins == 2 * kEvThreads, "two digits per thread");
      const int d0 = nb - 2 - 2 * tid;
      uint2 h = make_uint2(0u, 0u);            // (lower digit first)
      if (d0 >= 0) {
        uint2 x[kEvMaxCl];                     // (all reads in flight)
#pragma unroll
        for (int c = 0; c < kEvMaxCl; ++c)
          x[c] = c < C ? *reinterpret_cast<const uint2*>(cluster.map_shared_rank(hist, c) + d0)
                       : make_uint2(0u, 0u);
#pragma unroll
        for (int c = 0; c < kEvMaxCl; ++c) h.x += x[c].x, h.y += x[c].y;
      }
      const uint32_t tot = h.x + h.y, incl = warp_scan(tot, lane);
      uint32_t bx, by, ax, ay;
      warp_offsets(__shfl_sync(0xffffffffu, incl, 31), 0u, sm, bx, by, ax, ay);
      const uint32_t before = bx + incl - tot;
      if (before < want && want <= before + tot) {
        const bool upper = want <= before + h.y;
        sm.digit = (uint32_t)(d0 + (upper ? 1 : 0));
        sm.before = before + (upper ? 0u : h.y);
        sm.found = upper ? h.y : h.x;
      }
      __syncthreads();         // (the digit is there)
      prefix |= sm.digit << shift;
      mask |= (uint32_t)(nb - 1) << shift;
      want -= sm.before;
    }
    threshold = prefix;
    equal = (int)want;
    ties = sm.found > want;
  }
  // flags: group k of the warp is word warp * KPT + k; its kept-for-certain and equal tokens
  static_assert(KPT <= 32, "one lane per word");
  uint32_t gt_of = 0u, eq_of = 0u;                          // word lane of the warp
  if (heavy == 0) {
#pragma unroll
    for (int k = 0; k < KPT; ++k) {
      const int t = first + 32 * k;
      const unsigned gt = __ballot_sync(0xffffffffu, (t >= old) & (t < n));
      if (lane == k) gt_of = gt;
    }
  } else {
    const int oldest = old - first, end = (int)n - first;      // of this lane's tokens: 32 k
    const uint32_t from = ties ? threshold + 1u : threshold;   // (an infinity's key is 2^32 - 2^23)
    if (__all_sync(0xffffffffu, 32 * (KPT - 1) < oldest)) {
#pragma unroll
      for (int k = 0; k < KPT; ++k) {
        const unsigned gt = __ballot_sync(0xffffffffu, keys[k] >= from);
        if (lane == k) gt_of = gt;
      }
    } else {
#pragma unroll
      for (int k = 0; k < KPT; ++k) {
        const bool is_old = 32 * k < oldest;
        const unsigned gt = __ballot_sync(0xffffffffu, ((!is_old) | (keys[k] >= from)) & (32 * k < end));
        if (lane == k) gt_of = gt;
      }
    }
    if (ties)
#pragma unroll
      for (int k = 0; k < KPT; ++k) {
        const unsigned eq = __ballot_sync(0xffffffffu, (32 * k < oldest) & (keys[k] == threshold));
        if (lane == k) eq_of = eq;
      }
  }
  // (gt, eq) before each word: of the warp, the CTA and the cluster
  const uint32_t g = warp_scan(__popc(gt_of), lane), e = warp_scan(__popc(eq_of), lane);
  uint32_t bg, be, ag, ae;
  warp_offsets(__shfl_sync(0xffffffffu, g, 31), __shfl_sync(0xffffffffu, e, 31), sm, bg, be, ag, ae);
  if (tid == 0) {
    sm.count[0] = ag;
    sm.count[1] = ae;
  }
  cluster_sync();
  uint32_t cg0 = 0, ce0 = 0;   // of the CTAs before this one
#pragma unroll
  for (int r = 0; r < kEvMaxCl - 1; ++r)
    if (r < rank) {
      const uint2 c = *reinterpret_cast<const uint2*>(cluster.map_shared_rank(&sm.count[0], r));
      cg0 += c.x;
      ce0 += c.y;
    }
  auto kept_eq = [&](uint32_t e) { return e < (uint32_t)equal ? e : (uint32_t)equal; };
  const uint32_t base = cg0 + kept_eq(ce0);            // first destination of the CTA
  const uint32_t kept_here = cg0 + ag + kept_eq(ce0 + ae) - base;
  if (lane < KPT) {
    const uint32_t gb = cg0 + bg + g - __popc(gt_of), eb = ce0 + be + e - __popc(eq_of);
    // the lowest equal positions, while there is room
    uint32_t take = eb < (uint32_t)equal ? (uint32_t)equal - eb : 0u, word = gt_of;
    if (take >= (uint32_t)__popc(eq_of)) {
      word |= eq_of;
    } else {
      for (uint32_t x = eq_of; take > 0u; --take, x &= x - 1u) word |= x & (0u - x);
    }
    bits[warp * KPT + lane] = word;
    pre[warp * KPT + lane] = gb + kept_eq(eb) - base;
  }
  __syncwarp();                // a warp reads its own words only
#pragma unroll 4
  for (int k = 0; k < KPT; ++k) {
    const uint32_t word = bits[warp * KPT + k];
    if (!word) continue;
    if (word >> lane & 1u)
      src[pre[warp * KPT + k] + __popc(word & ((1u << lane) - 1u))] = (uint16_t)(warp * 32 * KPT + 32 * k + lane);
  }
  __syncthreads();

  const CodeRows kr = code_rows(a.k_codes, a.table, a.max_pages, a.n_pages, a.pshift, b, kvh, a.Hkv,
                                a.Tcap, a.Sk, a.err);
  const CodeRows vr = code_rows(a.v_codes, a.table, a.max_pages, a.n_pages, a.pshift, b, kvh, a.Hkv,
                                a.Tcap, a.Sv, a.err);
  float* acc_out = a.acc_out + pair * a.Tout;
  const uint32_t begin = (uint32_t)rank * CHUNK;
  // four kept tokens of this thread at a time, their reads in flight together: get(token), put(index
  // among the CTA's kept tokens, what get gave)
  auto each = [&](auto get, auto put) {
    for (uint32_t i0 = tid; i0 < kept_here; i0 += 4 * kEvThreads) {
      decltype(get(0u)) x[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (i0 + u * kEvThreads < kept_here) x[u] = get(begin + src[i0 + u * kEvThreads]);
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (i0 + u * kEvThreads < kept_here) put(i0 + u * kEvThreads, x[u]);
    }
  };
  auto total = [&](uint32_t t) { return acc[t]; };
  if (!a.in_place) {
    // contiguous rows of one machine word each: f(a value of that word's type)
    auto with_word = [](int S, auto f) {
      if (S == 4) f(uint32_t());
      else if (S == 2) f(uint16_t());
      else if (S == 1) f(uint8_t());
      else f(uint2());
    };
    const bool words = !a.table && !a.table_out && !(a.Sk & (a.Sk - 1)) && !(a.Sv & (a.Sv - 1));
    if (words) {
      with_word(a.Sk, [&](auto k_word) {
        with_word(a.Sv, [&](auto v_word) {
          using K = decltype(k_word);
          using V = decltype(v_word);
          struct Row {
            K k;
            V v;
            float x;
          };
          const K* k_from = reinterpret_cast<const K*>(kr.base);
          const V* v_from = reinterpret_cast<const V*>(vr.base);
          const int64_t to = pair * a.Tout + base;
          K* k_to = reinterpret_cast<K*>(a.k_out) + to;
          V* v_to = reinterpret_cast<V*>(a.v_out) + to;
          each([&](uint32_t t) { return Row{k_from[t], v_from[t], acc[t]}; },
               [&](uint32_t i, const Row& r) {
                 k_to[i] = r.k;
                 v_to[i] = r.v;
                 acc_out[base + i] = r.x;
               });
        });
      });
    } else {
      auto move = [&](const CodeRows& rows, uint8_t* out, int S) {
        each([&](uint32_t t) {
               uint32_t w[2];
               load_codes<8, false>(rows, t, S, w);
               return make_uint2(w[0], w[1]);
             },
             [&](uint32_t i, uint2 x) {
               const uint32_t w[2] = {x.x, x.y};
               store_codes(out_row(out, a, b, kvh, base + i, S), S, w);
             });
      };
      move(kr, a.k_out, a.Sk);
      move(vr, a.v_out, a.Sv);
      each(total, [&](uint32_t i, float x) { acc_out[base + i] = x; });
    }
  } else {
    // four bytes of every kept row at a time: K, V (two turns each for more than four stages), totals
    const int tk = (a.Sk + 3) / 4, tv = (a.Sv + 3) / 4;
    for (int turn = 0; turn <= tk + tv; ++turn) {
      const bool is_k = turn < tk, is_acc = turn == tk + tv;
      const int part = is_k ? turn : turn - tk, S = is_k ? a.Sk : a.Sv;
      if (is_acc) {
        each(total, [&](uint32_t i, float x) { list[i] = __float_as_uint(x); });
      } else if (!a.table && S == 4) {
        const uint32_t* from = reinterpret_cast<const uint32_t*>((is_k ? kr : vr).base);
        each([&](uint32_t t) { return from[t]; }, [&](uint32_t i, uint32_t x) { list[i] = x; });
      } else {
        each([&](uint32_t t) {
               uint32_t w[2];
               load_codes<8, false>(is_k ? kr : vr, t, S, w);
               return part == 0 ? w[0] : w[1];
             },
             [&](uint32_t i, uint32_t x) { list[i] = x; });
      }
      cluster_sync();          // every source of this turn has been read
      for (uint32_t i = tid; i < kept_here; i += kEvThreads) {
        const int64_t j = base + i;
        const uint32_t w = list[i];
        if (is_acc) {
          acc_out[j] = __uint_as_float(w);
          continue;
        }
        uint8_t* p = out_row(is_k ? a.k_out : a.v_out, a, b, kvh, j, S);
        if (!p) continue;
        p += 4 * part;
        if (S % 4 == 0) {
          *reinterpret_cast<uint32_t*>(p) = w;
        } else {
          for (int s = 0; s < 4 && 4 * part + s < S; ++s) p[s] = (uint8_t)(w >> (8 * s));
        }
      }
      __syncthreads();         // the list has been written out
    }
  }
  if (a.kept)
    for (uint32_t i = tid; i < kept_here; i += kEvThreads) a.kept[pair * a.keep + base + i] = (int32_t)(begin + src[i]);
  // tokens to come start without a total (a source that another CTA has read by now: in place the
  // totals went last, and all of them were read before the barrier)
  const int64_t zero_to = n < a.Tout ? n : a.Tout, all = (int64_t)C * kEvThreads;
  for (int64_t j = m + rank * kEvThreads + tid; j < zero_to; j += all) acc_out[j] = 0.f;
  if (a.kept)
    for (int64_t j = m + rank * kEvThreads + tid; j < a.keep; j += all) a.kept[pair * a.keep + j] = -1;
  cluster_sync();              // no CTA leaves while another may read its shared memory
}

// after every CTA has read comp_len (len_out may be the same array)
__global__ void evict_lengths_kernel(int B, int64_t Tcap, int64_t keep, const int32_t* comp_len,
                                     int32_t* len_out) {
  const int b = blockIdx.x * blockDim.x + threadIdx.x;
  int64_t n = b < B ? comp_len[b] : 0;         // (the kernel before does not write it)
  pdl_wait();
  if (b >= B) return;
  n = n < 0 ? 0 : n > Tcap ? Tcap : n;
  len_out[b] = (int32_t)(n < keep ? n : keep);
}

template <int KPT>
static cudaError_t launch_evict(const EvictArgs& a, int C, cudaStream_t st) {
  constexpr int CHUNK = kEvThreads * KPT;
  constexpr size_t apart = sizeof(EvictSmem) + CHUNK / 32 * 8 + CHUNK * 2, in_place = apart + CHUNK * 4;
  static_assert(in_place <= 227 * 1024, "fits");
  const cudaError_t e = ensure_smem_limit(evict_kernel<KPT>, in_place);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((int64_t)a.B * a.Hkv * C));
  cfg.blockDim = dim3(kEvThreads);
  cfg.dynamicSmemBytes = a.in_place ? in_place : apart;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, evict_kernel<KPT>, a);
}

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
  // (every block reads comp_len: where len_out is that array, a second kernel writes it)
  a.len_out = p->len_out == p->comp_len ? nullptr : p->len_out;
  // CTAs per cluster: what the capacity needs at 32768 tokens each, then more while there are SMs for
  // them and each keeps 4096 tokens
  const int64_t pairs = (int64_t)p->B * p->Hkv;
  int C = 1;
  while (p->Tcap > (int64_t)C * kEvThreads * 32) C *= 2;
  while (C < kEvMaxCl && pairs * C * 2 <= 148 && p->Tcap > (int64_t)C * 4096) C *= 2;
  const int64_t per = (p->Tcap + C - 1) / C;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = per <= kEvThreads        ? launch_evict<1>(a, C, st)
                        : per <= kEvThreads * 4  ? launch_evict<4>(a, C, st)
                        : per <= kEvThreads * 16 ? launch_evict<16>(a, C, st)
                                                 : launch_evict<32>(a, C, st);
  if (e != cudaSuccess) return ZKV_ERR_CUDA;
  if (a.len_out) return ZKV_OK;
  if (launch_pdl(evict_lengths_kernel, dim3((p->B + 127) / 128), dim3(128), 0, st, (int)p->B, p->Tcap, p->keep,
                 p->comp_len, p->len_out) != cudaSuccess)
    return ZKV_ERR_CUDA;
  return ZKV_OK;
}
