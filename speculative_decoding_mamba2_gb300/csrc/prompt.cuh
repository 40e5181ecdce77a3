// Launch arguments of the prompt kernels (ssm_prompt.h) and of the attention kernels (ssm_attention.h).
#pragma once

#include "common.cuh"
#include "ssm_attention.h"
#include "ssm_prompt.h"

namespace ssmtree {

constexpr int kSMs = 152;  // streaming multiprocessors of a GB300: what the launch plans divide work over

// a kernel's dynamic shared memory, asked for once per device (done: a table of the caller's, one for each kernel)
template <typename Kernel>
cudaError_t allow_smem(Kernel* kernel, int bytes, bool (&done)[64]) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (dev < 64 && done[dev])) return e;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev < 64) done[dev] = true;
  return e;
}

// the token rows and the cache slot of sequence s; false (and the status bit) where they are out of range
struct SeqArgs {
  int n_seq, n_slots, n_tok, max_len;
  const int32_t *cu, *slots;
  int32_t* status;
};
__device__ __forceinline__ bool seq_range(const SeqArgs& q, int s, int& first, int& len, int& slot) {
  first = q.cu[s];
  const long long l = (long long)q.cu[s + 1] - first;
  slot = q.slots ? q.slots[s] : s;
  const bool ok = first >= 0 && l >= 0 && l <= q.max_len && first + l <= q.n_tok && slot >= 0 && slot < q.n_slots;
  len = ok ? (int)l : 0;
  return ok;
}

struct ConvArgs {
  SeqArgs q;
  int L, layer, R, conv_dim;
  const float *conv_w, *conv_b;  // of this layer
  const uint16_t* x;
  long long ldx;
  uint16_t* ring;
  int32_t* ring_head;
  uint16_t* out;
  long long ldo;
};
cudaError_t launch_prompt_conv(const ConvArgs& a, cudaStream_t s);

struct ScanArgs {
  SeqArgs q;
  int H, G, L, layer;
  const float *dt_bias, *A_log, *D;  // of this layer
  const uint16_t *x, *B, *C, *dt;
  long long ldx, ldb, ldc, lddt;
  const float* h_in;
  float* h_out;
  uint16_t* y;
  long long ldy;
  int nseg;         // segments of a sequence (set by launch_prompt_scan)
  float* seg_state;  // workspace: what segments 0 .. nseg-2 add to the state, and their decay
};
size_t prompt_scan_workspace_bytes(int H, int G, int n_seq, int n_tok, int max_len);
cudaError_t launch_prompt_scan(const ScanArgs& a, void* workspace, cudaStream_t s);
// the same on tcgen05 (prompt_scan_tc.cu)
bool prompt_scan_tc_fits(int H, int G, int n_seq, int max_len);
size_t prompt_scan_tc_workspace_bytes(int H, int G, int n_seq, int n_tok, int max_len);
cudaError_t launch_prompt_scan_tc(const ScanArgs& a, void* workspace, cudaStream_t s);
cudaError_t launch_scan_step(const ScanArgs& a, cudaStream_t s);

struct AttendArgs {
  int S, n, Hq, Hkv, D, g;
  const ssm_node* layout;
  const uint16_t *q, *k, *v;
  long long ldq, ldk, ldv;
  const uint16_t *kp, *vp;
  int n_pages, page_shift;
  const int32_t* table;
  int max_pages;
  const int32_t* cache_len;
  int max_len;
  float scale_log2;  // scale · log2(e)
  uint16_t* o;
  long long ldo;
  int32_t* status;
  int max_runs;     // runs of key tiles that the sequences are cut into at most, 0: not cut (set by launch_tree_attention)
  float* part;      // workspace: partial o, (maximum, sum) pairs, each sequence's first run and their number
  float2* part_ml;
  int2* runs;
};
size_t tree_attention_workspace_bytes(int S, int n, int Hq, int Hkv, int D, int max_len);
cudaError_t launch_tree_attention(const AttendArgs& a, void* workspace, cudaStream_t s);

struct KvCommitArgs {
  int L, S, n, Hkv, D, max_path;
  const int32_t *path, *path_len;
  const uint16_t *k, *v;
  uint16_t *kp, *vp;
  int n_pages, page_shift;
  const int32_t* table;
  int max_pages;
  const int32_t* cache_len;
  int32_t *len_out, *status;
};
cudaError_t launch_kv_commit(const KvCommitArgs& a, cudaStream_t s);

}  // namespace ssmtree
