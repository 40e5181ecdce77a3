// Attention of a draft tree's nodes over an 8-bit paged cache and their ancestors, and the commit of the accepted path into it
// (ssm_attention.h).
#include "decode.cuh"
#include "mma_tiles.cuh"

namespace ssmtree {
namespace {

// One warp to a query row, D / 32 columns a lane; a row of keys at a time.
template <int D>
__global__ void __launch_bounds__(128) attend8_kernel(AttendFp8Args f) {
  constexpr int V = D / 32;
  const AttendArgs& a = f.a;
  const long long row = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (row >= (long long)a.S * a.n * a.Hq) return;
  const long long tok = row / a.Hq;
  const int head = (int)(row % a.Hq), s = (int)(tok / a.n), node = (int)(tok % a.n), kvh = head / a.g;
  int len = a.cache_len[s];
  if (len < 0 || len > a.max_len || (long long)len > ((long long)a.max_pages << a.page_shift)) {
    if (lane == 0) flag(a.status, SSM_STATUS_SEQ_RANGE);
    len = 0;
  }
  float q[V], o[V], m = -INFINITY, l = 0.f;
  for (int v = 0; v < V; ++v) q[v] = bf16f(a.q[tok * a.ldq + head * D + lane * V + v]), o[v] = 0.f;
  auto add = [&](const float (&k)[V], const float (&val)[V]) {
    float d = 0.f;
    for (int v = 0; v < V; ++v) d = fmaf(q[v], k[v], d);
    const float x = warp_sum(d) * a.scale_log2, to = fmaxf(m, x), ref = to == -INFINITY ? 0.f : to;
    const float g = exp2_sfu(m - ref), p = exp2_sfu(x - ref);
    l = l * g + p, m = to;
    for (int v = 0; v < V; ++v) o[v] = fmaf(p, val[v], o[v] * g);
  };
  for (int i = 0; i < len; ++i) {
    const int pg = a.table[(long long)s * a.max_pages + (i >> a.page_shift)], r = i & ((1 << a.page_shift) - 1);
    if (pg < 0 || pg >= a.n_pages) {
      if (lane == 0) flag(a.status, SSM_STATUS_SEQ_RANGE);
      continue;
    }
    const long long at = (((long long)pg * a.Hkv + kvh) << a.page_shift) + r, sc = at >> f.block_shift;
    const float ks = f.ks[sc], vs = f.vs[sc];
    if (!good_scale(ks) || !good_scale(vs)) {
      if (lane == 0) flag(a.status, SSM_STATUS_SCALE);
      continue;
    }
    float k[V], v[V];
    for (int j = 0; j < V; j += 2) {
      const float2 x = f16x2_f32(e4m3x2_f16x2(*reinterpret_cast<const uint16_t*>(f.kp + at * D + lane * V + j)));
      const float2 y = f16x2_f32(e4m3x2_f16x2(*reinterpret_cast<const uint16_t*>(f.vp + at * D + lane * V + j)));
      k[j] = x.x * ks, k[j + 1] = x.y * ks, v[j] = y.x * vs, v[j + 1] = y.y * vs;
    }
    add(k, v);
  }
  for (int u = node, hops = 0; u >= 0 && hops < a.n; ++hops) {
    float k[V], v[V];
    const long long at = (long long)s * a.n + u;
    for (int j = 0; j < V; ++j) k[j] = bf16f(a.k[at * a.ldk + kvh * D + lane * V + j]), v[j] = bf16f(a.v[at * a.ldv + kvh * D + lane * V + j]);
    add(k, v);
    const int p = u > 0 ? a.layout[(long long)s * a.n + u].parent : -1;
    if (u > 0 && (p < 0 || p >= u)) {
      if (lane == 0) flag(a.status, SSM_STATUS_BAD_LAYOUT);
      break;
    }
    u = p;
  }
  const float inv = 1.f / l;
  for (int j = 0; j < V; j += 2)
    *reinterpret_cast<uint32_t*>(a.o + tok * a.ldo + head * D + lane * V + j) = pack_bf16x2(o[j] * inv, o[j + 1] * inv);
}

// Commit.  A cluster of 8 CTAs for each sequence, a warp for each block of tokens of a layer, head and K or V: the largest of its new
// rows gives the scale that they need, the block takes that or its own, rows that it holds are rounded again if it grew.  The
// sequence's length is written by one of the CTAs once all eight have read it, so len_out may be cache_len.
constexpr int CCTAS = 8, CTHREADS = 512;

__device__ __forceinline__ float least_scale(uint32_t most) {  // of a largest magnitude's bits: 448 is 1.75 * 2^8
  const int e = (int)(most >> 23) - 127 - 8 + ((most & 0x7fffffu) > 0x600000u);
  return __uint_as_float((uint32_t)(max(e, -100) + 127) << 23);
}
__device__ __forceinline__ uint32_t finite_bits(float x) {  // |x|, 0 where it is not finite
  const uint32_t b = __float_as_uint(x) & 0x7fffffffu;
  return b < 0x7f800000u ? b : 0u;
}
__device__ __forceinline__ float nan_unless_finite(float x) {
  return (__float_as_uint(x) & 0x7f800000u) == 0x7f800000u ? __uint_as_float(0x7fffffffu) : x;
}

template <int D>
__global__ void __cluster_dims__(CCTAS, 1, 1) __launch_bounds__(CTHREADS) kv_commit8_kernel(KvCommitFp8Args f) {
  constexpr int W = D / 64;  // 32-bit words of bf16 of a row in a lane
  const KvCommitArgs& a = f.a;
  const int s = blockIdx.y, part = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __shared__ int path_s[SSM_MAX_PATH], rows_s;
  const int len = a.cache_len[s];
  if (threadIdx.x < 32) {  // the path's length: up to its first bad entry, and what the pages hold
    int want = a.path_len[s], bits = 0;
    if (want < 0 || want > a.max_path) bits |= SSM_STATUS_PATH_RANGE, want = want < 0 ? 0 : a.max_path;
    const long long room = min((long long)a.max_pages << a.page_shift, (long long)INT32_MAX) - len;  // (a length is an int32)
    if (len < 0 || room < 0) bits |= SSM_STATUS_SEQ_RANGE, want = 0;
    int n = want;
    for (int i0 = 0; i0 < want; i0 += 32) {
      const int i = i0 + lane;
      int why = 0;
      if (i < want) {
        const int v = a.path[(long long)s * a.max_path + i];
        path_s[i] = v;
        if (v < 0 || v >= a.n) {
          why = SSM_STATUS_PATH_RANGE;
        } else if (i >= room) {
          why = SSM_STATUS_SEQ_RANGE;
        } else {
          const int pg = a.table[(long long)s * a.max_pages + ((len + i) >> a.page_shift)];
          if (pg < 0 || pg >= a.n_pages) why = SSM_STATUS_SEQ_RANGE;
        }
      }
      const unsigned stop = __ballot_sync(0xffffffffu, why != 0);
      if (stop) {
        n = i0 + __ffs(stop) - 1;
        bits |= __shfl_sync(0xffffffffu, why, __ffs(stop) - 1);
        break;
      }
    }
    if (lane == 0) {
      rows_s = n;
      if (bits && part == 0) flag(a.status, bits);
    }
  }
  __syncthreads();
  asm volatile("barrier.cluster.arrive.release.aligned;\n" ::: "memory");
  const int n = rows_s;
  if (n > 0) {
    const int first = len >> f.block_shift, blocks = ((len + n - 1) >> f.block_shift) - first + 1;
    const int units = a.L * a.Hkv * 2 * blocks;
    for (int u = part * (CTHREADS / 32) + warp; u < units; u += CCTAS * (CTHREADS / 32)) {
      const int b = u % blocks, kv = u / blocks & 1, lh = u / blocks / 2, head = lh % a.Hkv, layer = lh / a.Hkv;
      const int start = (first + b) << f.block_shift;  // the block's first row of the sequence
      // rows that it holds, the first new one on the path, and their number (a row's own index may be the last int32)
      const int held = max(len - start, 0), from = max(start - len, 0), rows = min((1 << f.block_shift) - held, n - from);
      const int pg = a.table[(long long)s * a.max_pages + (start >> a.page_shift)];
      const long long row0 = ((((long long)layer * a.n_pages + pg) * a.Hkv + head) << a.page_shift) + (start & ((1 << a.page_shift) - 1));
      uint8_t* page = (kv ? f.vp : f.kp) + row0 * D + lane * 2 * W;
      float* scale_at = (kv ? f.vs : f.ks) + (row0 >> f.block_shift);
      const uint16_t* src = (kv ? a.v : a.k) + ((long long)layer * a.S + s) * a.n * a.Hkv * D + head * D + lane * 2 * W;
      const float old = held > 0 ? *scale_at : 0.f;
      auto get = [&](int r, uint32_t (&x)[W]) {
        const uint32_t* p = reinterpret_cast<const uint32_t*>(src + (long long)path_s[from + r] * a.Hkv * D);
        if constexpr (W == 2) {
          const uint2 v = *reinterpret_cast<const uint2*>(p);
          x[0] = v.x, x[1] = v.y;
        } else {
          x[0] = *p;
        }
      };
      uint32_t x[4][W], most = 0;
      for (int r0 = 0; r0 < rows; r0 += 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (r0 + i < rows) get(r0 + i, x[i]);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (r0 + i < rows)
#pragma unroll
            for (int w = 0; w < W; ++w) most = max(most, max(finite_bits(bf16_lo(x[i][w])), finite_bits(bf16_hi(x[i][w]))));
      }
      float scale = least_scale(__reduce_max_sync(0xffffffffu, most));
      if (held > 0) {
        if (!good_scale(old)) {
          if (lane == 0) flag(a.status, SSM_STATUS_SCALE);
        } else if (old >= scale) {
          scale = old;
        } else {  // the block grows: what it holds, in units of the new scale
          const float by = old / scale;
          for (int r = 0; r < held; ++r) {
            uint8_t* p = page + r * D;
            if constexpr (W == 2) {
              const uint32_t v = *reinterpret_cast<const uint32_t*>(p);
              const float2 y = f16x2_f32(e4m3x2_f16x2(v & 0xffffu)), z = f16x2_f32(e4m3x2_f16x2(v >> 16));
              *reinterpret_cast<uint32_t*>(p) = f32_e4m3x2(y.x * by, y.y * by) | f32_e4m3x2(z.x * by, z.y * by) << 16;
            } else {
              const float2 y = f16x2_f32(e4m3x2_f16x2(*reinterpret_cast<const uint16_t*>(p)));
              *reinterpret_cast<uint16_t*>(p) = (uint16_t)f32_e4m3x2(y.x * by, y.y * by);
            }
          }
        }
      }
      if (lane == 0 && scale != old) *scale_at = scale;
      page += held * D;
      for (int r0 = (rows - 1) / 4 * 4, here = 1; r0 >= 0; r0 -= 4, here = 0) {  // (from the last four: they are here)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (r0 + i < rows) {
            if (!here) get(r0 + i, x[i]);
            uint32_t v[W];
#pragma unroll
            for (int w = 0; w < W; ++w)
              v[w] = f32_e4m3x2(nan_unless_finite(bf16_lo(x[i][w])) / scale, nan_unless_finite(bf16_hi(x[i][w])) / scale);
            uint8_t* p = page + (r0 + i) * D;
            if constexpr (W == 2)
              *reinterpret_cast<uint32_t*>(p) = v[0] | v[1] << 16;
            else
              *reinterpret_cast<uint16_t*>(p) = (uint16_t)v[0];
          }
      }
    }
  }
  asm volatile("barrier.cluster.wait.acquire.aligned;\n" ::: "memory");
  if (part == 0 && threadIdx.x == 0) a.len_out[s] = len + n;
}

}  // namespace

size_t tree_attention_fp8_workspace_bytes(int S, int n, int Hq, int Hkv, int D, int max_len) { return 256; }

cudaError_t launch_tree_attention_fp8(const AttendFp8Args& f, void* workspace, cudaStream_t s) {
  if (f.a.S == 0) return cudaSuccess;
  const long long rows = (long long)f.a.S * f.a.n * f.a.Hq;
  const unsigned grid = (unsigned)((rows + 3) / 4);
  if (f.a.D == 64)
    attend8_kernel<64><<<grid, 128, 0, s>>>(f);
  else
    attend8_kernel<128><<<grid, 128, 0, s>>>(f);
  return cudaGetLastError();
}

cudaError_t launch_kv_commit_fp8(const KvCommitFp8Args& f, cudaStream_t s) {
  if (f.a.S == 0) return cudaSuccess;
  const dim3 grid(CCTAS, (unsigned)f.a.S);
  if (f.a.D == 64)
    kv_commit8_kernel<64><<<grid, CTHREADS, 0, s>>>(f);
  else
    kv_commit8_kernel<128><<<grid, CTHREADS, 0, s>>>(f);
  return cudaGetLastError();
}

}  // namespace ssmtree
