// What the tcgen05 kernels of prompts and attention share: descriptors of 128-byte swizzled tiles, MMAs, tensor-memory
// loads and stores, bounded waits of a warp, bulk tensor stores and tensor maps.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include "mma_tiles.cuh"
#include "tc.cuh"

namespace ssmtree {

// Descriptors: 128-byte swizzled tiles of 64-column blocks (rows of 128 bytes, groups of 8 rows 1024 bytes apart).
// K-major: the rows are M or N.  MN-major: the rows are K, `block` bytes between 64-element blocks along M or N.
// The upper word is the same for all: group stride, version 1, 128-byte swizzle.
constexpr uint32_t kDescHi = (1024u >> 4) | 1u << 14 | 2u << 29;
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t block) {
  return ((addr >> 4) & 0x3FFFu) | (block >> 4) << 16;
}
__host__ __device__ constexpr uint32_t idesc_major(int M, int N, bool a_mn, bool b_mn) {
  return idesc_bf16(M, N) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u);
}
// one lane of a converged warp, the same at every call
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n selp.u32 %0, 1, 0, q;\n}\n" : "=r"(p));
  return p != 0;
}
// D (TMEM) = A (TMEM) . B (+ D);  D (TMEM) = A . B (+ D)
template <uint32_t IDESC>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b_lo, bool acc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 b;\n setp.ne.b32 p, %4, 0;\n mov.b64 b, {%2, %5};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b_lo), "n"(IDESC), "r"((uint32_t)acc), "n"(kDescHi)
      : "memory");
}
template <uint32_t IDESC>
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, bool acc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 a, b;\n setp.ne.b32 p, %4, 0;\n mov.b64 a, {%1, %5};\n mov.b64 b, {%2, %5};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n}\n" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "n"(IDESC), "r"((uint32_t)acc), "n"(kDescHi)
      : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t addr, const uint32_t (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"r"(addr), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }
// 16 rows x 8 columns of 32 bits, from fragments: v[0], v[2], .. rows lane / 4, v[1], v[3], .. 8 rows on, columns
// lane % 4 and, from v[2] on, 4 further
__device__ __forceinline__ void tmem_st_frag(uint32_t addr, const uint32_t (&v)[4]) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x2.b32 [%0], {%1, %2, %3, %4};\n" ::"r"(addr), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3])
               : "memory");
}
// 16 rows x 16 fp32 columns as accumulator fragments: v[4 j ..]: row lane / 4, columns 8 j + 2 (lane % 4), + 1, then
// row + 8 (to be waited for before their use)
__device__ __forceinline__ void tmem_ld_frag_async(uint32_t addr, float (&v)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
               : "r"(addr));
}
__device__ __forceinline__ void tmem_wait_ld8(float (&v)[8], float (&w)[8]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;\n"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]), "+f"(w[0]),
                 "+f"(w[1]), "+f"(w[2]), "+f"(w[3]), "+f"(w[4]), "+f"(w[5]), "+f"(w[6]), "+f"(w[7])
               :
               : "memory");
}
// a 64 x 64 block of a tile stored by a bulk tensor copy
__device__ __forceinline__ void tma_store_2d(const void* tmap, uint32_t src, int c0, int c1) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];\n" ::"l"(tmap), "r"(c0), "r"(c1),
               "r"(src)
               : "memory");
}
// four 8 x 8 fragments stored transposed, row addresses as frag_a_t's
__device__ __forceinline__ void stsm4_t(uint32_t addr, const uint32_t (&r)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};\n" ::"r"(addr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3])
               : "memory");
}
// 16 columns without the wait (tmem_wait_ld16 before their use)
__device__ __forceinline__ void tmem_ld16_async(uint32_t addr, float (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15}, [%16];\n"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_wait_ld16(float (&v)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;\n"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                 "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15])
               :
               : "memory");
}

// The warp waits together, and all its lanes get the same answer: false once a second has passed or another warp has given
// up.  (A waiter has to see every phase of a barrier: the parity of one that it skipped would let it through early.)
__device__ __forceinline__ bool wait_bar(unsigned long long* bar, uint32_t parity, volatile int* stop) {
  const uint32_t b = smem_u32(bar);
  if (__all_sync(0xffffffffu, mbar_try_wait(b, parity))) return true;
  const unsigned long long t0 = global_time_ns();
#pragma unroll 1
  for (unsigned it = 1; it < kWaitLimit; ++it) {
    if (__all_sync(0xffffffffu, mbar_try_wait(b, parity))) return true;
    if ((it & 63) == 0 && __any_sync(0xffffffffu, *stop || global_time_ns() - t0 > kWaitLimitNs)) break;
  }
  *stop = 1;
  return false;
}
// ---- host ----
// a grid whose blocks may be placed while the stream's kernel before it ends; they call grid_dependency_wait before they
// touch what others write
template <typename... Args, typename... Given>
cudaError_t launch_early(void (*kernel)(Args...), dim3 grid, int threads, int smem, cudaStream_t s, const Given&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<Args>(args)...);
  return e != cudaSuccess ? e : cudaGetLastError();
}
inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  if (!fn) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }
  return fn;
}
// a rows x cols bf16 matrix (row stride ld elements) in boxes of 64 columns x box_rows rows, 128-byte swizzled
inline bool encode_tiles(CUtensorMap* m, const void* base, long long rows, long long cols, long long ld, int box_rows) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint64_t gdim[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t gstride[1] = {(cuuint64_t)ld * 2};
  const cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
  const cuuint32_t estride[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), gdim, gstride, box, estride,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace ssmtree
