// Serving-step cache maintenance: window insert, eviction of the oldest window token, RVQ
// encode of the evicted token onto the compressed prefix (sm_100a).
//
// Passages: VQKV (gist.science summary of arXiv 2603.16435), section 2.3 "Local Sliding
// Window" (recent tokens uncompressed, older "middle" tokens compressed to codes); VeloxQuant-
// MLX 0.5.1 "Quick start" (cache.append(k, v) per token, then cache.attend(q)).
//
// Kernel 1 encodes the evicted rows and writes each new token into its window slot; kernel 2
// advances the lengths.  Both read the same pre-step lengths, so their decisions agree.
//
// Kernel 1 is a cluster of 8 CTAs per (group of 8 sequences, kv head, K or V); the cluster encoder
// is append_cluster.cuh.
#include <cooperative_groups.h>

#include "append_cluster.cuh"
#include "lengths.cuh"

namespace cg = cooperative_groups;

namespace zkv {

template <int D>
__global__ void __cluster_dims__(kAppendCl, 1, 1) __launch_bounds__(256)
    append_cluster_kernel(zkv_append_params p, double rot) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  AppendSmem<D>& sm = *reinterpret_cast<AppendSmem<D>*>(smem_raw);
  pdl_trigger();   // the length update may launch now; it waits for this kernel's completion
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int kind = blockIdx.z;   // 0 = keys, 1 = values
  const int h = blockIdx.y;
  const int64_t row0 = (int64_t)(blockIdx.x / kAppendCl) * kAppendR;
  const int S = kind ? p.Sv : p.Sk;
  const float* CB = (kind ? p.v_codebooks : p.k_codebooks) + (size_t)h * S * kCodebook * D;
  const __half* win = reinterpret_cast<const __half*>(kind ? p.win_v : p.win_k);
  uint8_t* codes = kind ? p.v_codes : p.k_codes;

  auto row_valid = [&](int64_t j) {   // sequence j evicts a token into a prefix with room
    if (j >= p.B) return false;
    const int64_t wl = p.win_len[j], hd = p.win_head[j], c = p.comp_len[j];
    return wl == p.Wcap && hd >= 0 && hd < p.Wcap && c >= 0 && c < p.Tcap;
  };
  encode_cluster<D>(
      sm,
      [&](int r) -> const __half* {
        const int64_t j = row0 + r;
        return row_valid(j) ? win + ((j * p.Hkv + h) * p.Wcap + p.win_head[j]) * D : nullptr;
      },
      CB, S, kind == 0 && p.k_smooth ? p.k_smooth + (int64_t)h * D : nullptr, rot);
  cluster.sync();   // no CTA leaves while another may still read its shared memory
  // Launched as a dependent of the table kernel (the serving step), this kernel completes only
  // after that kernel has: whatever waits for this one then also sees the tables.  Returns at
  // once after a normal launch.
  pdl_wait();
  if (rank != 0) return;
  if (tid < kAppendR) {
    const int64_t j = row0 + tid;
    if (row_valid(j)) {
      const int64_t t = p.comp_len[j];
      uint8_t* c = nullptr;
      if (!p.block_table) {
        c = codes + ((j * p.Hkv + h) * p.Tcap + t) * S;
      } else {   // paged: row (h, t % P) of page block_table[j][t / P]
        const int64_t P = p.page_tokens;
        const int64_t pg = p.block_table[j * p.max_pages + t / P];
        if (pg >= 0 && pg < p.n_pages) c = codes + ((pg * p.Hkv + h) * P + t % P) * S;
        else set_error(p.error_flag, ZKV_DEVERR_PAGE);
      }
      if (c)
        for (int s = 0; s < S; ++s) c[s] = sm.code[tid][s];
    }
  }
  // every CTA read the evicted slots before its first cluster barrier
  if (warp < kAppendR) {
    const int64_t j = row0 + warp;
    if (j >= p.B) return;
    const int64_t wl = p.win_len[j], hd = p.win_head[j], c = p.comp_len[j];
    int64_t slot = -1;
    if (wl >= 0 && wl < p.Wcap) {
      slot = wl;
    } else if (wl == p.Wcap && hd >= 0 && hd < p.Wcap) {
      if (c >= 0 && c < p.Tcap) slot = hd;
      else if (lane == 0 && kind == 0 && h == 0) set_error(p.error_flag, ZKV_DEVERR_COMP_LEN);
    } else if (lane == 0 && kind == 0 && h == 0) {
      set_error(p.error_flag, ZKV_DEVERR_WIN_LEN);
    }
    if (slot < 0) return;
    const __half* src = reinterpret_cast<const __half*>(kind ? p.new_v : p.new_k) + (j * p.Hkv + h) * D;
    __half* dst = reinterpret_cast<__half*>(kind ? p.win_v : p.win_k) + ((j * p.Hkv + h) * p.Wcap + slot) * D;
    for (int i = lane; i < D; i += 32) dst[i] = src[i];
  }
}

__global__ void append_lengths_kernel(int B, int64_t Tcap, int64_t Wcap, int32_t* win_len,
                                      int32_t* win_head, int32_t* comp_len) {
  pdl_wait();   // the encode kernel read the pre-step lengths
  const int b = blockIdx.x * blockDim.x + threadIdx.x;
  if (b >= B) return;
  advance_lengths(b, Tcap, Wcap, win_len, win_head, comp_len);
}

int validate_append(const zkv_append_params* p) {
  if (!p) return ZKV_ERR_INVALID_ARG;
  if (p->B < 1 || p->Hkv < 1 || p->Tcap < 0 || p->Wcap < 1) return ZKV_ERR_INVALID_ARG;
  if (!supported_d(p->d)) return ZKV_ERR_UNSUPPORTED;
  if (p->Sk < 1 || p->Sk > kMaxStages || p->Sv < 1 || p->Sv > kMaxStages) return ZKV_ERR_UNSUPPORTED;
  if (p->Hkv > 65535) return ZKV_ERR_UNSUPPORTED;
  if (!p->new_k || !p->new_v || !p->win_k || !p->win_v || !p->win_len || !p->win_head ||
      !p->comp_len || !p->k_codes || !p->v_codes || !p->k_codebooks || !p->v_codebooks)
    return ZKV_ERR_INVALID_ARG;
  const uintptr_t al = (uintptr_t)p->win_k | (uintptr_t)p->win_v | (uintptr_t)p->k_codebooks |
                       (uintptr_t)p->v_codebooks;
  if (al & 15) return ZKV_ERR_INVALID_ARG;
  return validate_paged(p->block_table, p->page_tokens, p->max_pages, p->n_pages, p->Tcap);
}

// The encode + window-write kernel; with pdl, as a programmatic dependent of the previous
// kernel on the stream (it never reads that kernel's results).
int launch_append_cluster(const zkv_append_params& p, cudaStream_t st, bool pdl) {
  const double rot = 1.0 / std::sqrt((double)p.d);
  const unsigned groups = (unsigned)((p.B + kAppendR - 1) / kAppendR);
  const dim3 grid(groups * kAppendCl, (unsigned)p.Hkv, 2);
  const bool ok =
      ensure_smem_limit(append_cluster_kernel<64>, sizeof(AppendSmem<64>)) == cudaSuccess &&
      ensure_smem_limit(append_cluster_kernel<128>, sizeof(AppendSmem<128>)) == cudaSuccess &&
      ensure_smem_limit(append_cluster_kernel<256>, sizeof(AppendSmem<256>)) == cudaSuccess;
  if (!ok) return ZKV_ERR_CUDA;
  cudaError_t e = cudaSuccess;
  switch (p.d) {
    case 64:
      if (pdl) e = launch_pdl(append_cluster_kernel<64>, grid, dim3(256), sizeof(AppendSmem<64>), st, p, rot);
      else append_cluster_kernel<64><<<grid, 256, sizeof(AppendSmem<64>), st>>>(p, rot);
      break;
    case 128:
      if (pdl) e = launch_pdl(append_cluster_kernel<128>, grid, dim3(256), sizeof(AppendSmem<128>), st, p, rot);
      else append_cluster_kernel<128><<<grid, 256, sizeof(AppendSmem<128>), st>>>(p, rot);
      break;
    default:
      if (pdl) e = launch_pdl(append_cluster_kernel<256>, grid, dim3(256), sizeof(AppendSmem<256>), st, p, rot);
      else append_cluster_kernel<256><<<grid, 256, sizeof(AppendSmem<256>), st>>>(p, rot);
      break;
  }
  if (e != cudaSuccess) return ZKV_ERR_CUDA;
  ZKV_CHECK_LAUNCH();
  return ZKV_OK;
}

}  // namespace zkv

using namespace zkv;

extern "C" int zkv_rvq_append(const zkv_append_params* p, void* stream) {
  const int v = validate_append(p);
  if (v != ZKV_OK) return v;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int rc = launch_append_cluster(*p, st, false);
  if (rc != ZKV_OK) return rc;
  if (launch_pdl(append_lengths_kernel, dim3((p->B + 127) / 128), dim3(128), 0, st, p->B, p->Tcap,
                 p->Wcap, p->win_len, p->win_head, p->comp_len) != cudaSuccess)
    return ZKV_ERR_CUDA;
  return ZKV_OK;
}
