// C ABI of the prompt and attention calls (ssm_prompt.h, ssm_attention.h): host-side validation, then launches.
#include <math.h>
#include <stdio.h>

#include <string>

#include "prompt.cuh"

namespace ssmtree {
void set_error(const std::string& msg);
}

using namespace ssmtree;

namespace {

int pfail(int code, const char* fn, const char* what) {
  char buf[320];
  snprintf(buf, sizeof buf, "%s: %s", fn, what);
  set_error(buf);
  return code;
}

int pfinish(const char* fn, cudaError_t e) {
  if (e != cudaSuccess) {
    char buf[320];
    snprintf(buf, sizeof buf, "%s: CUDA error %d (%s)", fn, (int)e, cudaGetErrorString(e));
    set_error(buf);
    return SSM_ERR_CUDA;
  }
  set_error("");
  return SSM_OK;
}

bool off16(const void* p) { return ((uintptr_t)p & 15) != 0; }

int check_layer(const char* fn, const ssm_dims* d, const ssm_params* p, int32_t layer) {
  if (!d) return pfail(SSM_ERR_INVALID_ARG, fn, "dims is NULL");
  if (d->n_heads < 1 || (long long)d->n_heads * kP > (1 << 24))
    return pfail(SSM_ERR_INVALID_ARG, fn, "n_heads out of range");
  if (d->head_dim != kP) return pfail(SSM_ERR_INVALID_ARG, fn, "head_dim must be 64 in this library");
  if (d->d_state != kN) return pfail(SSM_ERR_INVALID_ARG, fn, "d_state must be 128 in this library");
  if (d->n_layers < 1) return pfail(SSM_ERR_INVALID_ARG, fn, "n_layers must be >= 1");
  if (!p) return pfail(SSM_ERR_INVALID_ARG, fn, "params is NULL");
  if (layer < 0 || layer >= d->n_layers) return pfail(SSM_ERR_RANGE, fn, "layer outside [0, n_layers)");
  return SSM_OK;
}

int check_counts(const char* fn, int32_t n_seq, int32_t n_slots, int32_t n_tok, int32_t max_len) {
  if (n_seq < 0 || n_seq > 65535) return pfail(SSM_ERR_INVALID_ARG, fn, "n_seq must be in [0, 65535]");
  if (n_slots < 0 || n_tok < 0 || max_len < 0)
    return pfail(SSM_ERR_INVALID_ARG, fn, "n_slots, n_tok and max_len must be >= 0");
  return SSM_OK;
}

int check_scan(const char* fn, const ssm_dims* d, const ssm_params* p, int32_t n_groups, long long rows,
               const uint16_t* x, int64_t ldx, const uint16_t* B, int64_t ldb, const uint16_t* C, int64_t ldc,
               const uint16_t* dt, int64_t lddt, const float* h_in, const float* h_out, const uint16_t* y, int64_t ldy) {
  if (n_groups < 1 || d->n_heads % n_groups) return pfail(SSM_ERR_INVALID_ARG, fn, "n_groups must divide n_heads");
  if (!p->dt_bias || !p->A_log || !p->D) return pfail(SSM_ERR_INVALID_ARG, fn, "a parameter pointer is NULL");
  if (!h_out) return pfail(SSM_ERR_INVALID_ARG, fn, "h_out is NULL");
  if (off16(h_in) || off16(h_out)) return pfail(SSM_ERR_INVALID_ARG, fn, "h_in and h_out must be 16-byte aligned");
  const int64_t inner = (int64_t)d->n_heads * kP, gn = (int64_t)n_groups * kN;
  if (ldx < inner || ldy < inner || ldb < gn || ldc < gn || lddt < d->n_heads)
    return pfail(SSM_ERR_INVALID_ARG, fn, "a row stride is below the row's width");
  if ((ldx | ldy | ldb | ldc) & 7) return pfail(SSM_ERR_INVALID_ARG, fn, "ldx, ldb, ldc and ldy must be multiples of 8");
  if (rows > 0 && (!x || !B || !C || !dt || !y)) return pfail(SSM_ERR_INVALID_ARG, fn, "a tensor pointer is NULL");
  if (off16(x) || off16(B) || off16(C) || off16(y))
    return pfail(SSM_ERR_INVALID_ARG, fn, "x, B, C and y must be 16-byte aligned");
  return SSM_OK;
}

ScanArgs scan_args(const ssm_dims* d, const ssm_params* p, int32_t layer, int32_t G, const uint16_t* x, int64_t ldx,
                   const uint16_t* B, int64_t ldb, const uint16_t* C, int64_t ldc, const uint16_t* dt, int64_t lddt,
                   const float* h_in, float* h_out, uint16_t* y, int64_t ldy) {
  ScanArgs a{};
  a.H = d->n_heads, a.G = G, a.L = d->n_layers, a.layer = layer;
  const size_t at = (size_t)layer * d->n_heads;
  a.dt_bias = p->dt_bias + at, a.A_log = p->A_log + at, a.D = p->D + at;
  a.x = x, a.B = B, a.C = C, a.dt = dt;
  a.ldx = ldx, a.ldb = ldb, a.ldc = ldc, a.lddt = lddt;
  a.h_in = h_in, a.h_out = h_out, a.y = y, a.ldy = ldy;
  return a;
}

int check_attend_shape(const char* fn, int32_t S, int32_t n, int32_t Hq, int32_t Hkv, int32_t D, int32_t max_len) {
  if (S < 0 || S > 65535) return pfail(SSM_ERR_INVALID_ARG, fn, "n_seq must be in [0, 65535]");
  if (n < 1) return pfail(SSM_ERR_INVALID_ARG, fn, "n_nodes must be >= 1");
  if (n > SSM_MAX_NODES) return pfail(SSM_ERR_CAPACITY, fn, "n_nodes above SSM_MAX_NODES");
  if (Hkv < 1 || Hq < 1 || Hq % Hkv) return pfail(SSM_ERR_INVALID_ARG, fn, "Hkv must divide Hq");
  if (Hkv > 1024 || Hq / Hkv > 32) return pfail(SSM_ERR_CAPACITY, fn, "more than 1024 kv heads or 32 query heads for each");
  if (D != 64 && D != 128) return pfail(SSM_ERR_INVALID_ARG, fn, "D must be 64 or 128");
  if (max_len < 0 || max_len > (1 << 30)) return pfail(SSM_ERR_INVALID_ARG, fn, "max_cache_len must be in [0, 2^30]");
  return SSM_OK;
}

int page_shift(int32_t page) {  // -1: not a power of two in [8, 1024]
  for (int k = 3; k <= 10; ++k)
    if (page == 1 << k) return k;
  return -1;
}

}  // namespace

extern "C" int ssm_prompt_conv(const ssm_dims* dims, const ssm_params* prm, int32_t layer, int32_t n_seq,
                               int32_t n_slots, int32_t n_tok, int32_t max_len, const int32_t* cu_seqlens,
                               const int32_t* slots, const uint16_t* xBC, int64_t ldx, uint16_t* ring,
                               int32_t* ring_head, uint16_t* out, int64_t ldo, int32_t* dev_status, void* stream) {
  const char* fn = "ssm_prompt_conv";
  if (int rc = check_layer(fn, dims, prm, layer)) return rc;
  if (dims->conv_width != kW) return pfail(SSM_ERR_INVALID_ARG, fn, "conv_width must be 4");
  if (dims->ring_cap < 3) return pfail(SSM_ERR_INVALID_ARG, fn, "ring_cap must be >= 3");
  if (!prm->conv_w || !prm->conv_b) return pfail(SSM_ERR_INVALID_ARG, fn, "a parameter pointer is NULL");
  if (int rc = check_counts(fn, n_seq, n_slots, n_tok, max_len)) return rc;
  const int64_t cd = (int64_t)dims->n_heads * kP + 2 * kN;
  if (n_seq > 0 && (!cu_seqlens || !ring || !ring_head)) return pfail(SSM_ERR_INVALID_ARG, fn, "cu_seqlens, ring or ring_head is NULL");
  if (n_tok > 0 && (!xBC || !out)) return pfail(SSM_ERR_INVALID_ARG, fn, "a tensor pointer is NULL");
  if (ldx < cd || ldo < cd || ((ldx | ldo) & 7))
    return pfail(SSM_ERR_INVALID_ARG, fn, "ldx and ldo must be >= conv_dim and multiples of 8");
  if (off16(xBC) || off16(out) || off16(ring) || off16(prm->conv_w) || off16(prm->conv_b))
    return pfail(SSM_ERR_INVALID_ARG, fn, "xBC, out, ring, conv_w and conv_b must be 16-byte aligned");
  if (n_tok > 0 && xBC == out) return pfail(SSM_ERR_INVALID_ARG, fn, "out must not be xBC");
  ConvArgs a{};
  a.q = SeqArgs{n_seq, n_slots, n_tok, max_len, cu_seqlens, slots, dev_status};
  a.L = dims->n_layers, a.layer = layer, a.R = dims->ring_cap, a.conv_dim = (int)cd;
  a.conv_w = prm->conv_w + (size_t)layer * cd * kW, a.conv_b = prm->conv_b + (size_t)layer * cd;
  a.x = xBC, a.ldx = ldx, a.ring = ring, a.ring_head = ring_head, a.out = out, a.ldo = ldo;
  return pfinish(fn, launch_prompt_conv(a, (cudaStream_t)stream));
}

extern "C" size_t ssm_prompt_scan_workspace_size(const ssm_dims* dims, int32_t n_seq, int32_t n_tok, int32_t max_len,
                                                 int32_t n_groups) {
  const char* fn = "ssm_prompt_scan_workspace_size";
  static const ssm_params none{};
  if (check_layer(fn, dims, &none, 0) || check_counts(fn, n_seq, 0, n_tok, max_len)) return 0;
  if (n_groups < 1 || dims->n_heads % n_groups) {
    pfail(SSM_ERR_INVALID_ARG, fn, "n_groups must divide n_heads");
    return 0;
  }
  set_error("");
  return prompt_scan_workspace_bytes(dims->n_heads, n_groups, n_seq, n_tok, max_len < n_tok ? max_len : n_tok);
}

extern "C" int ssm_prompt_scan(const ssm_dims* dims, const ssm_params* prm, int32_t layer, int32_t n_groups,
                               int32_t n_seq, int32_t n_slots, int32_t n_tok, int32_t max_len,
                               const int32_t* cu_seqlens, const int32_t* slots, const uint16_t* x, int64_t ldx,
                               const uint16_t* B, int64_t ldb, const uint16_t* C, int64_t ldc, const uint16_t* dt,
                               int64_t lddt, const float* h_in, float* h_out, uint16_t* y, int64_t ldy,
                               void* workspace, size_t workspace_bytes, int32_t* dev_status, void* stream) {
  const char* fn = "ssm_prompt_scan";
  if (int rc = check_layer(fn, dims, prm, layer)) return rc;
  if (int rc = check_counts(fn, n_seq, n_slots, n_tok, max_len)) return rc;
  if (int rc = check_scan(fn, dims, prm, n_groups, n_tok, x, ldx, B, ldb, C, ldc, dt, lddt, h_in, h_out, y, ldy)) return rc;
  if (n_seq > 0 && !cu_seqlens) return pfail(SSM_ERR_INVALID_ARG, fn, "cu_seqlens is NULL");
  if (max_len > n_tok) max_len = n_tok;  // no sequence is longer than that
  if (!workspace || ((uintptr_t)workspace & 255)) return pfail(SSM_ERR_INVALID_ARG, fn, "workspace must be 256-byte aligned");
  if (workspace_bytes < prompt_scan_workspace_bytes(dims->n_heads, n_groups, n_seq, n_tok, max_len))
    return pfail(SSM_ERR_CAPACITY, fn, "workspace too small (ssm_prompt_scan_workspace_size)");
  ScanArgs a = scan_args(dims, prm, layer, n_groups, x, ldx, B, ldb, C, ldc, dt, lddt, h_in, h_out, y, ldy);
  a.q = SeqArgs{n_seq, n_slots, n_tok, max_len, cu_seqlens, slots, dev_status};
  return pfinish(fn, launch_prompt_scan(a, workspace, (cudaStream_t)stream));
}

extern "C" int ssm_scan_step(const ssm_dims* dims, const ssm_params* prm, int32_t layer, int32_t n_groups,
                             int32_t n_seq, int32_t n_slots, const int32_t* slots, const uint16_t* x, int64_t ldx,
                             const uint16_t* B, int64_t ldb, const uint16_t* C, int64_t ldc, const uint16_t* dt,
                             int64_t lddt, const float* h_in, float* h_out, uint16_t* y, int64_t ldy,
                             int32_t* dev_status, void* stream) {
  const char* fn = "ssm_scan_step";
  if (int rc = check_layer(fn, dims, prm, layer)) return rc;
  if (int rc = check_counts(fn, n_seq, n_slots, n_seq, 1)) return rc;
  if (int rc = check_scan(fn, dims, prm, n_groups, n_seq, x, ldx, B, ldb, C, ldc, dt, lddt, h_in, h_out, y, ldy)) return rc;
  ScanArgs a = scan_args(dims, prm, layer, n_groups, x, ldx, B, ldb, C, ldc, dt, lddt, h_in, h_out, y, ldy);
  a.q = SeqArgs{n_seq, n_slots, n_seq, 1, nullptr, slots, dev_status};
  return pfinish(fn, launch_scan_step(a, (cudaStream_t)stream));
}

extern "C" size_t ssm_tree_attention_workspace_size(int32_t n_seq, int32_t n_nodes, int32_t Hq, int32_t Hkv, int32_t D,
                                                    int32_t max_cache_len) {
  if (check_attend_shape("ssm_tree_attention_workspace_size", n_seq, n_nodes, Hq, Hkv, D, max_cache_len)) return 0;
  set_error("");
  return tree_attention_workspace_bytes(n_seq, n_nodes, Hq, Hkv, D, max_cache_len);
}

extern "C" int ssm_tree_attention(int32_t n_seq, int32_t n_nodes, int32_t Hq, int32_t Hkv, int32_t D,
                                  const ssm_node* layout, const uint16_t* q, int64_t ldq, const uint16_t* k,
                                  int64_t ldk, const uint16_t* v, int64_t ldv, const uint16_t* k_pages,
                                  const uint16_t* v_pages, int32_t n_pages, int32_t page_size,
                                  const int32_t* page_table, int32_t max_pages, const int32_t* cache_len,
                                  int32_t max_cache_len, float scale, uint16_t* o, int64_t ldo, void* workspace,
                                  size_t workspace_bytes, int32_t* dev_status, void* stream) {
  const char* fn = "ssm_tree_attention";
  if (int rc = check_attend_shape(fn, n_seq, n_nodes, Hq, Hkv, D, max_cache_len)) return rc;
  const int shift = page_shift(page_size);
  if (shift < 0) return pfail(SSM_ERR_INVALID_ARG, fn, "page_size must be a power of two in [8, 1024]");
  if (n_pages < 0 || max_pages < 0) return pfail(SSM_ERR_INVALID_ARG, fn, "n_pages and max_pages must be >= 0");
  if ((long long)n_pages * Hkv * page_size > INT32_MAX || (long long)n_seq * n_nodes > INT32_MAX)
    return pfail(SSM_ERR_CAPACITY, fn, "more than 2^31 - 1 rows of pages");
  if (!(scale > 0.f) || isinf(scale)) return pfail(SSM_ERR_RANGE, fn, "scale must be positive and finite");
  if (n_seq > 0 && (!layout || !q || !k || !v || !o || !cache_len)) return pfail(SSM_ERR_INVALID_ARG, fn, "a pointer is NULL");
  if (max_cache_len > 0 && (!k_pages || !v_pages || !page_table))
    return pfail(SSM_ERR_INVALID_ARG, fn, "k_pages, v_pages or page_table is NULL");
  if (off16(q) || off16(k) || off16(v) || off16(k_pages) || off16(v_pages) || off16(o))
    return pfail(SSM_ERR_INVALID_ARG, fn, "q, k, v, the pages and o must be 16-byte aligned");
  if (ldq < (int64_t)Hq * D || ldo < (int64_t)Hq * D || ldk < (int64_t)Hkv * D || ldv < (int64_t)Hkv * D ||
      ((ldq | ldo | ldk | ldv) & 7))
    return pfail(SSM_ERR_INVALID_ARG, fn, "row strides must be at least the row's width and multiples of 8");
  if (!workspace || ((uintptr_t)workspace & 255)) return pfail(SSM_ERR_INVALID_ARG, fn, "workspace must be 256-byte aligned");
  if (workspace_bytes < tree_attention_workspace_bytes(n_seq, n_nodes, Hq, Hkv, D, max_cache_len))
    return pfail(SSM_ERR_CAPACITY, fn, "workspace too small (ssm_tree_attention_workspace_size)");
  AttendArgs a{};
  a.S = n_seq, a.n = n_nodes, a.Hq = Hq, a.Hkv = Hkv, a.D = D, a.g = Hq / Hkv;
  a.layout = layout, a.q = q, a.k = k, a.v = v, a.ldq = ldq, a.ldk = ldk, a.ldv = ldv;
  a.kp = k_pages, a.vp = v_pages, a.n_pages = n_pages, a.page_shift = shift;
  a.table = page_table, a.max_pages = max_pages, a.cache_len = cache_len, a.max_len = max_cache_len;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.o = o, a.ldo = ldo, a.status = dev_status;
  return pfinish(fn, launch_tree_attention(a, workspace, (cudaStream_t)stream));
}

extern "C" int ssm_kv_commit(int32_t n_layers, int32_t n_seq, int32_t n_nodes, int32_t Hkv, int32_t D, int32_t max_path,
                             const int32_t* path, const int32_t* path_len, const uint16_t* k, const uint16_t* v,
                             uint16_t* k_pages, uint16_t* v_pages, int32_t n_pages, int32_t page_size,
                             const int32_t* page_table, int32_t max_pages, const int32_t* cache_len, int32_t* len_out,
                             int32_t* dev_status, void* stream) {
  const char* fn = "ssm_kv_commit";
  if (n_seq < 0 || n_seq > 65535) return pfail(SSM_ERR_INVALID_ARG, fn, "n_seq must be in [0, 65535]");
  if (n_layers < 1 || n_nodes < 1 || Hkv < 1) return pfail(SSM_ERR_INVALID_ARG, fn, "n_layers, n_nodes and Hkv must be >= 1");
  if (max_path < 1 || max_path > SSM_MAX_PATH) return pfail(SSM_ERR_INVALID_ARG, fn, "max_path must be in [1, SSM_MAX_PATH]");
  if (D != 64 && D != 128) return pfail(SSM_ERR_INVALID_ARG, fn, "D must be 64 or 128");
  if ((long long)n_layers * max_path * Hkv * (D / 8) > (1ll << 30))
    return pfail(SSM_ERR_CAPACITY, fn, "n_layers * max_path * Hkv * D too large");
  const int shift = page_shift(page_size);
  if (shift < 0) return pfail(SSM_ERR_INVALID_ARG, fn, "page_size must be a power of two in [8, 1024]");
  if (n_pages < 0 || max_pages < 0) return pfail(SSM_ERR_INVALID_ARG, fn, "n_pages and max_pages must be >= 0");
  if (n_seq > 0 && (!path || !path_len || !k || !v || !k_pages || !v_pages || !page_table || !cache_len || !len_out))
    return pfail(SSM_ERR_INVALID_ARG, fn, "a pointer is NULL");
  if (off16(k) || off16(v) || off16(k_pages) || off16(v_pages))
    return pfail(SSM_ERR_INVALID_ARG, fn, "k, v and the pages must be 16-byte aligned");
  KvCommitArgs a{};
  a.L = n_layers, a.S = n_seq, a.n = n_nodes, a.Hkv = Hkv, a.D = D, a.max_path = max_path;
  a.path = path, a.path_len = path_len, a.k = k, a.v = v, a.kp = k_pages, a.vp = v_pages;
  a.n_pages = n_pages, a.page_shift = shift, a.table = page_table, a.max_pages = max_pages;
  a.cache_len = cache_len, a.len_out = len_out, a.status = dev_status;
  return pfinish(fn, launch_kv_commit(a, (cudaStream_t)stream));
}
