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
// computes for itself), so a cluster of 8 CTAs (append_cluster.cuh) encodes eight evictions of one
// kv head and of K or V, from whichever sequences.  Only the first eviction of a slot (k < W) reads
// the window, and its cluster then writes the slot's last token; fill slots that no eviction takes
// are written apart.  So no slot is read by one cluster and written by another.
// Kernel 2 advances the lengths after all of kernel 1 has read them.
#include "append_cluster.cuh"

#include <cmath>

namespace cg = cooperative_groups;

namespace zkv {

struct CommitState {
  int64_t n, wl, head, comp, evict, fill;   // fill: tokens that take free slots
};

// What sequence b commits; false (with the error bits in err) if it is left unchanged.
__device__ __forceinline__ bool commit_state(const zkv_tree_commit_params& p, int64_t b,
                                             CommitState& s, int& err) {
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
  for (int64_t i = 0; i < s.n; ++i) {
    const int32_t x = p.path[b * p.M + i];
    if (x < 0 || x >= p.N) err = ZKV_DEVERR_DRAFT;
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

template <int D>
__global__ void __cluster_dims__(kAppendCl, 1, 1) __launch_bounds__(256)
    tree_commit_kernel(zkv_tree_commit_params p, double rot) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  AppendSmem<D>& sm = *reinterpret_cast<AppendSmem<D>*>(smem_raw);
  __shared__ int64_t warp_sum[8];
  __shared__ int row_b[kAppendR];                 // the cluster's evictions: sequence (-1: none), k
  __shared__ int64_t row_k[kAppendR];
  __shared__ CommitState row_s[kAppendR];
  pdl_trigger();   // the length update may launch now; it waits for this kernel's completion
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int kind = blockIdx.z;   // 0 = keys, 1 = values
  const int h = blockIdx.y;
  const int64_t group = blockIdx.x / kAppendCl, groups = gridDim.x / kAppendCl;
  const int64_t row0 = group * kAppendR;
  const int S = kind ? p.Sv : p.Sk;
  const float* CB = (kind ? p.v_codebooks : p.k_codebooks) + (size_t)h * S * kCodebook * D;
  __half* win = reinterpret_cast<__half*>(kind ? p.win_v : p.win_k);
  const __half* draft = reinterpret_cast<const __half*>(kind ? p.draft_v : p.draft_k);
  const int64_t sb = kind ? p.v_sb : p.k_sb, sn = kind ? p.v_sn : p.k_sn, sh = kind ? p.v_sh : p.k_sh;
  uint8_t* codes = kind ? p.v_codes : p.k_codes;

  auto token = [&](int64_t b, int64_t i) -> const __half* {     // accepted token i of sequence b
    return draft + b * sb + (int64_t)p.path[b * p.M + i] * sn + (int64_t)h * sh;
  };
  if (tid < kAppendR) row_b[tid] = -1;
  int64_t base = 0;
  for (int64_t b0 = 0; b0 < p.B && base < row0 + kAppendR; b0 += 256) {
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
    if (lane == 31) warp_sum[warp] = x;
    __syncthreads();
    int64_t before = base + x - s.evict, all = 0;
    for (int w = 0; w < 8; ++w) {
      if (w < warp) before += warp_sum[w];
      all += warp_sum[w];
    }
    for (int r = 0; r < kAppendR; ++r) {
      const int64_t k = row0 + r - before;
      if (k >= 0 && k < s.evict) {
        row_b[r] = (int)b;
        row_k[r] = k;
        row_s[r] = s;
      }
    }
    base += all;
  }
  cluster.sync();      // (the rows are known, and every CTA of the cluster runs)
  if (row_b[0] >= 0) {          // the same in every CTA of the cluster: rows fill from the front
    encode_cluster<D>(
        sm,
        [&](int r) -> const __half* {
          const int64_t b = row_b[r];
          if (b < 0) return nullptr;
          const int64_t k = row_k[r];
          if (k >= p.Wcap) return token(b, p.Wcap - row_s[r].wl + k - p.Wcap);
          const int64_t slot = (row_s[r].head + k) % p.Wcap;
          if (slot >= row_s[r].wl) return token(b, slot - row_s[r].wl);
          return win + ((b * p.Hkv + h) * p.Wcap + slot) * D;
        },
        CB, S, kind == 0 && p.k_smooth ? p.k_smooth + (int64_t)h * D : nullptr, rot);
    cluster.sync();   // no CTA leaves while another may still read its shared memory
    if (rank == 0 && tid < kAppendR && row_b[tid] >= 0) {
      const int64_t b = row_b[tid], t = row_s[tid].comp + row_k[tid];
      uint8_t* c = codes + ((b * p.Hkv + h) * p.Tcap + t) * S;
      if (p.block_table) {
        const int64_t P = p.page_tokens;
        c = codes + ((p.block_table[b * p.max_pages + t / P] * (int64_t)p.Hkv + h) * P + t % P) * S;
      }
      for (int s = 0; s < S; ++s) c[s] = sm.code[tid][s];
    }
    // every CTA read the evicted slots before its first cluster barrier
    if (rank == 0 && row_b[warp] >= 0 && row_k[warp] < p.Wcap) {
      const int64_t b = row_b[warp], k = row_k[warp], e = row_s[warp].evict;
      const int64_t last = k + (e - 1 - k) / p.Wcap * p.Wcap;     // the slot's last eviction
      const __half* src = token(b, p.Wcap - row_s[warp].wl + last);
      __half* dst = win + ((b * p.Hkv + h) * p.Wcap + (row_s[warp].head + k) % p.Wcap) * D;
      for (int i = lane; i < D; i += 32) dst[i] = src[i];
    }
  }
  // fill tokens whose slot no eviction takes: the sequences are shared out over CTAs and warps
  for (int64_t b = (group * kAppendCl + rank) * 8 + warp; b < p.B; b += groups * kAppendCl * 8) {
    CommitState s;
    int err;
    if (!commit_state(p, b, s, err)) continue;
    for (int64_t i = 0; i < s.fill; ++i) {
      const int64_t slot = s.wl + i;
      if (s.evict > 0 && (slot - s.head + p.Wcap) % p.Wcap < s.evict) continue;
      const __half* src = token(b, i);
      __half* dst = win + ((b * p.Hkv + h) * p.Wcap + slot) * D;
      for (int x = lane; x < D; x += 32) dst[x] = src[x];
    }
  }
}

__global__ void tree_commit_lengths_kernel(zkv_tree_commit_params p) {
  pdl_wait();   // kernel 1 read the lengths before
  const int64_t b = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (b >= p.B) return;
  CommitState s;
  int err;
  const bool ok = commit_state(p, b, s, err);
  if (err) set_error(p.error_flag, err);
  if (!ok) return;
  p.win_len[b] = (int32_t)(s.wl + s.fill);
  if (s.evict > 0) {
    p.comp_len[b] = (int32_t)(s.comp + s.evict);
    p.win_head[b] = (int32_t)((s.head + s.evict) % p.Wcap);
  }
}

template <int D>
static int launch_tree_commit(const zkv_tree_commit_params& p, cudaStream_t st) {
  const double rot = 1.0 / std::sqrt((double)p.d);
  if (ensure_smem_limit(tree_commit_kernel<D>, sizeof(AppendSmem<D>)) != cudaSuccess)
    return ZKV_ERR_CUDA;
  const int64_t groups = ((int64_t)p.B * p.M + kAppendR - 1) / kAppendR;
  const dim3 grid((unsigned)(groups * kAppendCl), (unsigned)p.Hkv, 2);
  tree_commit_kernel<D><<<grid, 256, sizeof(AppendSmem<D>), st>>>(p, rot);
  ZKV_CHECK_LAUNCH();
  if (launch_pdl(tree_commit_lengths_kernel, dim3((p.B + 127) / 128), dim3(128), 0, st, p) != cudaSuccess)
    return ZKV_ERR_CUDA;
  return ZKV_OK;
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
