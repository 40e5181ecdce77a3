// Log probabilities of given tokens, entropy and the largest logits of each row (ssm_logits.h).
//
// One pass over a row: every thread keeps the maximum m of its logits and, relative to it and in powers of two,
//     l = sum 2^t,   a = sum 2^t t,   t = (x - m) scale log2(e),
// so that lse = m scale + ln l and the entropy is ln l - ln 2 a / l once the threads' triples are joined.  The largest k come
// from the maxima that are there anyway: the k-th largest of the threads' maxima is at most the row's k-th largest value, so
// only threads whose maximum reaches it hold any of them, about k of the block's 512, and those threads' logits alone are read again.
// A row is shared by a cluster of up to eight blocks, whose triples and sorted k are joined in the first one's shared memory.
#include <cooperative_groups.h>

#include "decode.cuh"
#include "mma_tiles.cuh"

namespace ssmtree {
namespace {

namespace cg = cooperative_groups;

constexpr int STHREADS = 512, SWARPS = STHREADS / 32;
constexpr int CAP = STHREADS;  // candidates at a time
constexpr int FEW = 64;    // threads whose logits are read again by a warp each; more of them: all logits, in order
typedef unsigned long long u64;

struct ScoreSmem {
  u64 key[CAP], sorted[SSM_MAX_TOP];
  u64 all[8 * SSM_MAX_TOP];   // (first block) the blocks' sorted candidates
  float mla[SWARPS][3];
  float part[8][3];           // (first block) the blocks' triples
  unsigned int most[STHREADS];
  int few[FEW];
  int n_few, count;
  unsigned int bound32;
  u64 bound;
};

// order of logits as unsigned integers; a NaN comes before minus infinity, zeros of both signs are one
__device__ __forceinline__ unsigned int order_of(float x) {
  const unsigned int b = __float_as_uint(x + 0.f);
  return x != x ? 0u : b ^ ((unsigned int)((int)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(unsigned int o) {
  return o == 0u ? __uint_as_float(0x7fffffffu) : __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}

// a row as vectors of 16 aligned bytes, of which the first and the last may lie in the row in part
template <typename T>
struct Row {
  static constexpr int E = 16 / sizeof(T);
  const T* x;
  int V, off, vecs;
  __device__ __forceinline__ Row(const T* p, int n) : x(p), V(n) {
    off = (int)(((uintptr_t)p & 15) / sizeof(T));
    vecs = (int)(((long long)n + off + E - 1) / E);
  }
  __device__ __forceinline__ void get(int j, float (&v)[E]) const {
    const long long at = (long long)j * E - off;
    if (at >= 0 && at + E <= V) {
      const uint4 u = __ldg(reinterpret_cast<const uint4*>(x + at));
      if constexpr (E == 4) {
        v[0] = __uint_as_float(u.x), v[1] = __uint_as_float(u.y), v[2] = __uint_as_float(u.z), v[3] = __uint_as_float(u.w);
      } else {
        v[0] = bf16_lo(u.x), v[1] = bf16_hi(u.x), v[2] = bf16_lo(u.y), v[3] = bf16_hi(u.y);
        v[4] = bf16_lo(u.z), v[5] = bf16_hi(u.z), v[6] = bf16_lo(u.w), v[7] = bf16_hi(u.w);
      }
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] = at + e >= 0 && at + e < V ? one(at + e) : -INFINITY;
    }
  }
  __device__ __forceinline__ float one(long long i) const {
    if constexpr (E == 4)
      return x[i];
    else
      return bf16f(reinterpret_cast<const uint16_t*>(x)[i]);
  }
};

// a triple made relative to the maximum `to`; (minus infinity less itself is no number: nothing is there to be counted)
__device__ __forceinline__ void rebase(float m, float to, float c, float& l, float& a) {
  const float d = fmaxf((m - to) * c, -1e4f), f = exp2_sfu(d);
  a = f * fmaf(l, d, a), l *= f;
}
__device__ __forceinline__ void join(float& m, float& l, float& a, float m2, float l2, float a2, float c) {
  const float to = fmaxf(m, m2);
  rebase(m, to, c, l, a), rebase(m2, to, c, l2, a2);
  m = to, l += l2, a += a2;
}

// the k largest of the candidates, sorted, in key and sorted; what counts from now on is above the k-th.  Many are first cut
// down to the k by bisecting their k-th (a block's count a bit; no two are alike).
__device__ __forceinline__ void prune(ScoreSmem& sm, int k) {
  __syncthreads();
  int n = min(sm.count, CAP);
  u64 mine = threadIdx.x < (unsigned)n ? sm.key[threadIdx.x] : 0ull;
  if (n > 128) {
    u64 b = 0;
#pragma unroll 1
    for (int bit = 63; bit >= 0; --bit) {
      const int above = __syncthreads_count(mine >= (b | 1ull << bit));
      if (above >= k) b |= 1ull << bit;
      if (above == k) break;
    }
    if (threadIdx.x == 0) sm.count = 0;
    __syncthreads();
    if (mine >= b) sm.key[atomicAdd(&sm.count, 1)] = mine;
    __syncthreads();
    n = k, mine = threadIdx.x < (unsigned)n ? sm.key[threadIdx.x] : 0ull;
  }
  if (threadIdx.x < (unsigned)n) {
    int rank = 0;
    for (int j = 0; j < n; ++j) rank += sm.key[j] > mine;
    if (rank < k) sm.sorted[rank] = mine;
  }
  __syncthreads();
  n = min(n, k);
  if (threadIdx.x < (unsigned)n) sm.key[threadIdx.x] = sm.sorted[threadIdx.x];
  if (threadIdx.x == 0) {
    sm.count = n;
    if (n == k) sm.bound = sm.sorted[k - 1];
  }
  __syncthreads();
}

// a vector's logits that are above the bound, by every thread of the block together
template <typename T>
__device__ __forceinline__ void collect(ScoreSmem& sm, const Row<T>& row, int j, bool there, int k) {
  constexpr int E = Row<T>::E;
  float v[E];
  unsigned int todo = 0;
  if (there) {
    row.get(j, v);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const long long at = (long long)j * E - row.off + e;
      if (at >= 0 && at < row.V && order_of(v[e]) >= sm.bound32) todo |= 1u << e;
    }
  }
  for (;;) {
    bool left = false;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      if (!(todo >> e & 1)) continue;
      const u64 key = (u64)order_of(v[e]) << 32 | (0xffffffffu - (unsigned int)((long long)j * E - row.off + e));
      if (key <= *(volatile u64*)&sm.bound) {
        todo &= ~(1u << e);
      } else {
        const int at = atomicAdd(&sm.count, 1);
        if (at < CAP)
          sm.key[at] = key, todo &= ~(1u << e);
        else
          left = true;
      }
    }
    if (!__syncthreads_or(left)) return;
    prune(sm, k);
  }
}

template <typename T, bool TOP>
__global__ void __launch_bounds__(STHREADS, 2) scores_kernel(ScoreArgs a) {
  constexpr int E = Row<T>::E, U = 4;
  __shared__ ScoreSmem sm;
  cg::cluster_group cluster = cg::this_cluster();
  const int parts = (int)cluster.num_blocks(), part = (int)cluster.block_rank();
  const int t = (int)(blockIdx.x / parts), tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Row<T> row(reinterpret_cast<const T*>(a.x) + (long long)t * a.ld, a.V);
  const int per = (row.vecs + parts - 1) / parts, j0 = part * per, j1 = min(j0 + per, row.vecs);
  const float c = a.scale * 1.4426950408889634f;
  if (parts > 1) cluster.barrier_arrive();  // (awaited before another block's shared memory is written)

  // given tokens: asked for early
  int tok = -1;
  float given = 0.f;
  if (part == 0 && tid < a.m) {
    tok = a.tok[(long long)t * a.m + tid];
    if (tok >= 0 && tok < a.V) given = row.one(tok);
  }

  float m = -INFINITY, l = 0.f, s = 0.f;
#pragma unroll 1
  for (int j = j0 + tid; j < j1; j += U * STHREADS) {
    float v[U][E];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (j + u * STHREADS < j1) {
        row.get(j + u * STHREADS, v[u]);
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e) v[u][e] = -INFINITY;
      }
    }
    float mx = m;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int e = 0; e < E; ++e) mx = fmaxf(mx, v[u][e]);
    if (mx > m) rebase(m, mx, c, l, s), m = mx;
    const float ref = m == -INFINITY ? 0.f : m;  // (taken off before the product: logits far from 0 cost nothing then)
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float d = (v[u][e] - ref) * c, p = exp2_sfu(d);
        l += p, s = fmaf(p, fmaxf(d, -200.f), s);  // (0 times minus infinity is no number)
      }
  }
  const float mine = m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    join(m, l, s, __shfl_xor_sync(0xffffffffu, m, o), __shfl_xor_sync(0xffffffffu, l, o), __shfl_xor_sync(0xffffffffu, s, o), c);
  if (lane == 0) sm.mla[warp][0] = m, sm.mla[warp][1] = l, sm.mla[warp][2] = s;
  if (TOP) sm.most[tid] = order_of(mine);
  if (tid == 0) sm.n_few = 0, sm.count = 0, sm.bound = 0;
  __syncthreads();
  m = sm.mla[0][0], l = sm.mla[0][1], s = sm.mla[0][2];
#pragma unroll 1
  for (int w = 1; w < SWARPS; ++w) join(m, l, s, sm.mla[w][0], sm.mla[w][1], sm.mla[w][2], c);

  if (TOP) {
    if (warp == 0) {  // the k-th largest of the threads' maxima, or a little less
      unsigned int q[SWARPS], b = 0;
#pragma unroll
      for (int i = 0; i < SWARPS; ++i) q[i] = sm.most[i * 32 + lane];
#pragma unroll 1
      for (int bit = 31; bit >= 0; --bit) {
        const unsigned int to = b | 1u << bit;
        int n = 0;
#pragma unroll
        for (int i = 0; i < SWARPS; ++i) n += q[i] >= to;
        n = __reduce_add_sync(0xffffffffu, n);
        if (n >= a.k) {
          b = to;
          if (n <= a.k + 4) break;
        }
      }
      // nothing above minus infinity in some of them: they may stand for threads without logits
      if (lane == 0) sm.bound32 = b <= order_of(-INFINITY) ? 0u : b;
    }
    __syncthreads();
    const bool in = order_of(mine) >= sm.bound32;
    if (in) {
      const int at = atomicAdd(&sm.n_few, 1);
      if (at < FEW) sm.few[at] = tid;
    }
    __syncthreads();
    const int n = sm.n_few, mines = (j1 - j0 + STHREADS - 1) / STHREADS;  // a thread's vectors at most
    if (n <= FEW) {
#pragma unroll 1
      for (int f = 0; f < n; f += SWARPS)
#pragma unroll 1
        for (int i = 0; i < mines; i += 32) {
          const bool some = f + warp < n;
          const int j = j0 + (some ? sm.few[f + warp] : 0) + (i + lane) * STHREADS;
          collect(sm, row, j, some && j < j1, a.k);
        }
    } else {
#pragma unroll 1
      for (int j = j0; j < j1; j += STHREADS) collect(sm, row, j + tid, j + tid < j1, a.k);
    }
    prune(sm, a.k);
  }
  if (parts > 1) {
    ScoreSmem* first = cluster.map_shared_rank(&sm, 0);
    cluster.barrier_wait();
    if (tid == 0) first->part[part][0] = m, first->part[part][1] = l, first->part[part][2] = s;
    if (TOP && tid < SSM_MAX_TOP) first->all[part * SSM_MAX_TOP + tid] = tid < sm.count ? sm.sorted[tid] : 0ull;
    cluster.sync();
    if (part > 0) return;
    m = sm.part[0][0], l = sm.part[0][1], s = sm.part[0][2];
    for (int i = 1; i < parts; ++i) join(m, l, s, sm.part[i][0], sm.part[i][1], sm.part[i][2], c);
    if (TOP) {
      const u64 key = tid < parts * SSM_MAX_TOP ? sm.all[tid] : 0ull;
      int rank = 0;
      if (key)
        for (int i = 0; i < parts * SSM_MAX_TOP; ++i) rank += sm.all[i] > key;
      if (key && rank < a.k) sm.sorted[rank] = key;
      __syncthreads();
    }
  }
  const float log_l = logf(l);
  if (tid == 0 && a.entropy) a.entropy[t] = log_l - 0.6931471805599453f * (s / l);
  for (int i = tid; i < a.m; i += STHREADS) {
    if (i >= STHREADS) {
      tok = a.tok[(long long)t * a.m + i];
      if (tok >= 0 && tok < a.V) given = row.one(tok);
    }
    float r = fmaf(given - m, a.scale, -log_l);
    if (tok == -1) {
      r = 0.f;
    } else if (tok < 0 || tok >= a.V) {
      r = __uint_as_float(0x7fffffffu);
      flag(a.status, SSM_STATUS_TOKEN_RANGE);
    }
    a.logprob[(long long)t * a.m + i] = r;
  }
  if (TOP && tid < a.k) {
    const u64 key = sm.sorted[tid];
    a.top[(long long)t * a.k + tid] = (int)(0xffffffffu - (unsigned int)key);
    if (a.top_logprob) a.top_logprob[(long long)t * a.k + tid] = fmaf(value_of((unsigned int)(key >> 32)) - m, a.scale, -log_l);
  }
}

template <typename T>
cudaError_t run_scores(const ScoreArgs& a, int parts, cudaStream_t s) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)a.T * parts);
  cfg.blockDim = dim3(STHREADS);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)parts, attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr, cfg.numAttrs = 1;
  const cudaError_t e = a.k > 0 ? cudaLaunchKernelEx(&cfg, scores_kernel<T, true>, a) : cudaLaunchKernelEx(&cfg, scores_kernel<T, false>, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_token_scores(const ScoreArgs& a, cudaStream_t s) {
  if (a.T == 0) return cudaSuccess;
  const long long bytes = (long long)a.V * (a.f32 ? 4 : 2);
  int parts = 1;
  while (parts < 8 && (long long)a.T * parts < 4 * kSMs && bytes / parts > 2 * 16 * STHREADS) parts *= 2;
  return a.f32 ? run_scores<float>(a, parts, s) : run_scores<uint16_t>(a, parts, s);
}

}  // namespace ssmtree
