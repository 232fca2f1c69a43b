// Warp-level matrix instructions and asynchronous copies: for attention of few
// queries, whose 16 rows (mma.sync m16n8k16) would fill an eighth of a 128-row
// tcgen05 tile, and for the scores of the block choice.
#pragma once

#include "common.cuh"

namespace svg {

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ void ldsm_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// c += a (16 x 16, row) * b (16 x 8, column): bf16 operands, fp32 sums.
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 16 bytes global -> shared; `bytes` = 0 writes zeros and reads nothing.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t *>(&b);
}

// Byte offset of 16-byte chunk `ch` of row `r` of a [rows, D] bf16 tile: chunks
// are exchanged by the row's low bits, so that eight rows of one chunk column
// (an ldmatrix phase) lie in different banks.
template <int D>
__device__ __forceinline__ uint32_t tile_at(int r, int ch) {
  return static_cast<uint32_t>(r * (D * 2) + ((ch ^ (r & 7)) << 4));
}

// This lane's address for an ldmatrix.x4 of a 16 x 16 piece of a tile (at its
// row 0, channel 0): matrices (rows 0-7, ch 0-7), (rows 8-15, ch 0-7), (rows 0-7,
// ch 8-15), (rows 8-15, ch 8-15) = the four registers of an A operand; with
// .trans the two B operands of 16 rows x (2 x 8) channels.
template <int D>
__device__ __forceinline__ uint32_t lane_a(uint32_t tile) {
  const int l = lane_id();
  return tile + tile_at<D>(l & 15, l >> 4);
}

// The same with the middle matrices exchanged: without .trans registers 0, 1
// are the B operand of rows 0-7 and 2, 3 that of rows 8-15 (contraction over
// the 16 channels).
template <int D>
__device__ __forceinline__ uint32_t lane_b(uint32_t tile) {
  const int l = lane_id();
  return tile + tile_at<D>((l & 7) + ((l >> 4) << 3), (l >> 3) & 1);
}

// From such an address to the piece at row r0 (a multiple of 8), channel 16 ks:
// the exchange of chunks is an exclusive or, so the channel is one as well, and
// the row stays an immediate offset.  Tiles must start at multiples of a row:
// they lie first in dynamic shared memory, in kernels without static arrays
// (which would move its start).
template <int D>
__device__ __forceinline__ uint32_t piece(uint32_t lane, int r0, int ks) {
  return (lane ^ (static_cast<uint32_t>(ks) << 5)) + static_cast<uint32_t>(r0 * D * 2);
}

// Row (0-7) of this lane's accumulator elements c[0], c[1] (c[2], c[3]: + 8),
// and the column of c[0], c[2] inside the 8-wide tile.
__device__ __forceinline__ int frag_row() { return lane_id() >> 2; }
__device__ __forceinline__ int frag_col() { return (lane_id() & 3) * 2; }

__device__ __forceinline__ float quad_max(float v) {
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
  return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
}
__device__ __forceinline__ float quad_sum(float v) {
  v += __shfl_xor_sync(0xffffffffu, v, 1);
  return v + __shfl_xor_sync(0xffffffffu, v, 2);
}

}  // namespace svg
