// Launch arguments of the calls of an 8-bit cache, of rotary positions (ssm_attention.h) and of token scores (ssm_logits.h),
// and conversions of e4m3 values.
#pragma once

#include <cuda_fp16.h>

#include "prompt.cuh"
#include "ssm_logits.h"

namespace ssmtree {

struct AttendFp8Args {
  AttendArgs a;  // (kp and vp are not read)
  const uint8_t *kp, *vp;
  const float *ks, *vs;
  int block_shift;
};
size_t tree_attention_fp8_workspace_bytes(int S, int n, int Hq, int Hkv, int D, int max_len);
cudaError_t launch_tree_attention_fp8(const AttendFp8Args& a, void* workspace, cudaStream_t s);
constexpr int kFewRows = 16;  // up to so many query rows of a key/value head:
cudaError_t launch_few_attention_fp8(const AttendFp8Args& a, int max_runs, cudaStream_t s);

struct KvCommitFp8Args {
  KvCommitArgs a;  // (kp and vp are not read)
  uint8_t *kp, *vp;
  float *ks, *vs;
  int block_shift;
};
cudaError_t launch_kv_commit_fp8(const KvCommitFp8Args& a, cudaStream_t s);

struct RopeArgs {
  int n_tok, n;  // n: nodes of a tree, 0 where positions are given
  int heads[2], D, rot;
  bool interleaved;
  const unsigned long long* turns;
  float amp;
  const int32_t* pos;
  const ssm_node* layout;
  const int32_t* cache_len;
  const uint16_t* in[2];  // q, k
  uint16_t* out[2];
  long long ldi[2], ldo[2];
  int32_t* status;
};
cudaError_t launch_rope(const RopeArgs& a, cudaStream_t s);

struct ScoreArgs {
  int T, V, m, k;
  const void* x;
  bool f32;
  long long ld;
  float scale;
  const int32_t* tok;
  float *logprob, *entropy;
  int32_t* top;
  float* top_logprob;
  int32_t* status;
};
cudaError_t launch_token_scores(const ScoreArgs& a, cudaStream_t s);

constexpr float kShift = 7.f;  // weights are 2^7 times as large, so that fp16 holds them to 2^-31 of the largest

// two e4m3 values (the lower half of v) as two of fp16 (exact)
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t v) {
  uint32_t r;
  asm("{\n .reg .b16 h, g;\n mov.b32 {h, g}, %1;\n cvt.rn.f16x2.e4m3x2 %0, h;\n}\n" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 f16x2_f32(uint32_t v) { return __half22float2(*reinterpret_cast<const __half2*>(&v)); }
// two values as e4m3, to nearest; NaN stays NaN, and what is beyond 448 becomes 448
__device__ __forceinline__ uint32_t f32_e4m3x2(float lo, float hi) {
  uint32_t r;
  asm("{\n .reg .b16 h;\n cvt.rn.satfinite.e4m3x2.f32 h, %2, %1;\n cvt.u32.u16 %0, h;\n}\n" : "=r"(r) : "f"(lo), "f"(hi));
  return r;
}
// the same of two fp16 values; x * y and x - y of two bf16, two fp16 values
__device__ __forceinline__ uint32_t f16x2_e4m3x2(uint32_t v) {
  uint32_t r;
  asm("{\n .reg .b16 h;\n cvt.rn.satfinite.e4m3x2.f16x2 h, %1;\n cvt.u32.u16 %0, h;\n}\n" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ uint32_t bf16x2_mul(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}
__device__ __forceinline__ uint32_t f16x2_sub(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}
__device__ __forceinline__ float nan_unless_finite(float x) {
  return (__float_as_uint(x) & 0x7f800000u) == 0x7f800000u ? __uint_as_float(0x7fffffffu) : x;
}
__device__ __forceinline__ bool good_scale(float s) { return s >= 0x1p-100f && s <= 0x1p120f; }

}  // namespace ssmtree
