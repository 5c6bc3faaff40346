// Matrix products of fp16 tiles in shared memory with float32 accuracy (sm_100a).
//
// A float32 operand row is scaled by a power of two (its norm or largest magnitude to 2^14 .. 2^15) and split
// into two fp16 planes, x = hi + lo with |x - hi - lo| <= 2^-23 |x| (fp16's subnormals end 2^-39
// below the row's largest); a product is hi hi + hi lo + lo hi, three matrix instructions, and leaves
// out lo lo <= 2^-22 of a term.  The tensor cores align the terms of a sum before they add, so a long
// chain of accumulations would lose bits that float32 additions keep: the hi hi products of every 16
// terms start from zero and are added up by float32 additions; the cross terms, 2^-11 of them, chain.
//
// Tiles are [row][K] fp16, 16-byte pieces of a row permuted by the row's low three bits, so that
// ldmatrix reads eight rows without a bank conflict.
#pragma once

#include "zkv_internal.cuh"

namespace zkv {

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], const __half* p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"((unsigned)__cvta_generic_to_shared(p))
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], const __half* p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"((unsigned)__cvta_generic_to_shared(p))
               : "memory");
}
// d += a b (16 x 8 x 16, fp16 inputs, float32 sums)
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
               "{%8, %9}, {%0, %1, %2, %3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16816_zero(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
               "{%8, %9}, {%10, %10, %10, %10};"
               : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
// d = a b; d += a b with the 16 terms summed from zero and added in float32
__device__ __forceinline__ void mma16816_add(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  float t[4];
  mma16816_zero(t, a, b0, b1);
  const float2 x = fadd2(make_float2(d[0], d[1]), make_float2(t[0], t[1]));
  const float2 y = fadd2(make_float2(d[2], d[3]), make_float2(t[2], t[3]));
  d[0] = x.x; d[1] = x.y; d[2] = y.x; d[3] = y.y;
}

// element (r, c) of a tile with K columns
template <int K>
__device__ __forceinline__ int tile_at(int r, int c) {
  return r * K + ((((c >> 3) ^ (r & 7)) << 3) | (c & 7));
}
// The operand fragments of step ks (16 columns): A of rows r0 .. r0 + 15 of a [row][K] tile, B of 16
// columns n0 .. n0 + 15 given as rows of a [n][K] tile (b[0], b[1]: n0 .. n0 + 7; b[2], b[3]: the rest)
template <int K>
__device__ __forceinline__ void frag_a(uint32_t (&a)[4], const __half* t, int r0, int ks, int lane) {
  ldsm4(a, t + tile_at<K>(r0 + (lane & 15), ks * 16 + 8 * (lane >> 4)));
}
template <int K>
__device__ __forceinline__ void frag_b(uint32_t (&b)[4], const __half* t, int n0, int ks, int lane) {
  ldsm4(b, t + tile_at<K>(n0 + (lane & 7) + ((lane >> 4) << 3), ks * 16 + 8 * ((lane >> 3) & 1)));
}
// B of 8 columns for two steps, ks and ks + 1 (b[0], b[1]: ks; b[2], b[3]: ks + 1)
template <int K>
__device__ __forceinline__ void frag_b2(uint32_t (&b)[4], const __half* t, int n0, int ks, int lane) {
  ldsm4(b, t + tile_at<K>(n0 + (lane & 7), ks * 16 + 8 * (lane >> 3)));
}
// The same from tiles that hold the sum's index as rows: A^T [k][M], B [k][N]
template <int M>
__device__ __forceinline__ void frag_at(uint32_t (&a)[4], const __half* t, int r0, int ks, int lane) {
  ldsm4t(a, t + tile_at<M>(ks * 16 + (lane & 7) + ((lane >> 4) << 3), r0 + 8 * ((lane >> 3) & 1)));
}
template <int N>
__device__ __forceinline__ void frag_bt(uint32_t (&b)[4], const __half* t, int n0, int ks, int lane) {
  ldsm4t(b, t + tile_at<N>(ks * 16 + (lane & 7) + 8 * ((lane >> 3) & 1), n0 + 8 * (lane >> 4)));
}

// a lane that TransposeSum<N, N, 16> leaves the sum of value k with
template <int N>
__device__ __forceinline__ constexpr int sum_owner(int k) {
  int lane = 0;
  for (int n = N / 2, o = 16; n >= 1; n /= 2, o /= 2)
    if (k & n) lane |= o;
  return lane;
}
// The exponent e with x 2^-e in [2^14, 2^15) for a row's largest magnitude (or its norm: no element
// is larger), and 2^e.  Rows below 2^-46 are scaled by 2^60: a norm whose squares underflow to zero
// must not scale its elements beyond fp16.
__device__ __forceinline__ int split_exponent(float largest) {
  int e = (int)((__float_as_uint(largest) >> 23) & 255u) - 127 - 14;
  return e < -60 ? -60 : e;
}
__device__ __forceinline__ float exp2_int(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }
__device__ __forceinline__ void split(float x, __half& hi, __half& lo) {
  hi = __float2half_rn(x);
  lo = __float2half_rn(x - __half2float(hi));
}

}  // namespace zkv
