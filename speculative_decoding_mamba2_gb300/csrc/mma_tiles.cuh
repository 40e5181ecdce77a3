// Fragments of m16n8k16 products read from shared memory: bf16 tiles whose rows are whole 16-byte
// chunks, the chunks of row r at position chunk ^ (r & 7), so that the eight rows of an 8x8 matrix
// read (ldmatrix) or written together fall on different banks.
#pragma once

#include "common.cuh"

namespace ssmtree {

// byte offset of 16-byte chunk `chunk` of row `row` in a tile of `row_bytes`-byte rows (a multiple of 128)
__device__ __forceinline__ uint32_t tile_off(int row, int chunk, int row_bytes) {
  return (uint32_t)(row * row_bytes + ((chunk ^ (row & 7)) << 4));
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// A fragment (16 x 16) of a tile stored [m][k]: rows m0.., columns k0.. (k0 a multiple of 16)
__device__ __forceinline__ void frag_a(uint32_t (&r)[4], uint32_t tile, int row_bytes, int m0, int k0, int lane) {
  const int row = m0 + (lane & 15), chunk = (k0 >> 3) + (lane >> 4);
  ldsm4(r, tile + tile_off(row, chunk, row_bytes));
}
// A fragment of a tile stored [k][m]
__device__ __forceinline__ void frag_a_t(uint32_t (&r)[4], uint32_t tile, int row_bytes, int m0, int k0, int lane) {
  const int row = k0 + (lane & 7) + ((lane >> 4) << 3), chunk = (m0 >> 3) + ((lane >> 3) & 1);
  ldsm4_t(r, tile + tile_off(row, chunk, row_bytes));
}
// B fragments of two n-tiles (n0.., n0+8..) of a tile stored [n][k]: r[0..1] the first, r[2..3] the second
__device__ __forceinline__ void frag_b2(uint32_t (&r)[4], uint32_t tile, int row_bytes, int n0, int k0, int lane) {
  const int row = n0 + (lane & 7) + ((lane >> 4) << 3), chunk = (k0 >> 3) + ((lane >> 3) & 1);
  ldsm4(r, tile + tile_off(row, chunk, row_bytes));
}
// B fragments of two n-tiles of a tile stored [k][n]
__device__ __forceinline__ void frag_b2_t(uint32_t (&r)[4], uint32_t tile, int row_bytes, int n0, int k0, int lane) {
  const int row = k0 + (lane & 15), chunk = (n0 >> 3) + (lane >> 4);
  ldsm4_t(r, tile + tile_off(row, chunk, row_bytes));
}

// D += A·B with the B fragment in two registers
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  const uint32_t b[2] = {b0, b1};
  mma_bf16(d, a, b);
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// a pair of bf16 values, 0 in the place of one that is not finite
__device__ __forceinline__ uint32_t finite_or_zero(uint32_t v) {
  return ((v & 0x7f80u) == 0x7f80u ? 0u : v & 0xffffu) | ((v & 0x7f800000u) == 0x7f800000u ? 0u : v & 0xffff0000u);
}

// 2^x on the special-function unit (relative error about 2^-22; 2^-inf = 0)
__device__ __forceinline__ float exp2_sfu(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// cp.async of 16 bytes, or of 16 zero bytes when !there (the source is then not read)
__device__ __forceinline__ void cp_async16_or_zero(uint32_t smem, const void* gmem, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(smem), "l"(gmem), "r"(there ? 16 : 0)
               : "memory");
}

}  // namespace ssmtree
