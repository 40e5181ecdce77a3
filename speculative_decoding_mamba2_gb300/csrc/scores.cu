// Log probabilities of given tokens, entropy and the largest logits of each row (ssm_logits.h).
//
// One pass over a row: every thread keeps the maximum m of its logits and, relative to it and in powers of two,
//     l = sum 2^t,   s = sum 2^t t,   t = (x - m) scale log2(e),
// so that lse = m scale + ln l and the entropy is ln l - ln 2 s / l once the threads' triples are joined: five instructions a
// logit of either type, two at a time.  The largest k come from the maxima that are there anyway: the k-th largest of the 32
// eights of threads' maxima is at most the row's k-th largest value, so only the runs of a few vectors whose own maximum (each
// thread keeps up to 32 of them in shared memory) reaches it hold any of them, a dozen or two for k = 8, and those alone are read
// again.  (With one maximum a thread, each 256th of a row read again cost more than half of the pass: 116 us for 640 rows of
// 151936 logits.)  Rows with many equal values there (masked vocabularies, constants) are read again in whole, the candidates
// cut down to the k best whenever their space is full.
// A row is shared by a cluster of up to eight blocks, whose triples and sorted k are joined in the first one's shared memory.
#include <cooperative_groups.h>
#include <limits.h>

#include "decode.cuh"
#include "mma_tiles.cuh"

namespace ssmtree {
namespace {

namespace cg = cooperative_groups;

constexpr int STHREADS = 256, SWARPS = STHREADS / 32;
constexpr int sblocks(bool f32) { return f32 ? 5 : 4; }  // blocks on an SM (of fp32 fewer registers, and 640 rows then are one round)
constexpr int CAP = STHREADS;  // candidates at a time
constexpr int RUNS = 32;       // runs of a thread's vectors
constexpr int FEW = 256;       // runs that are read again; more of them: all logits, in order
typedef unsigned long long u64;

struct ScoreSmem {
  u64 key[CAP], sorted[SSM_MAX_TOP];
  u64 all[8 * SSM_MAX_TOP];  // (first block) the blocks' sorted candidates
  float mls[SWARPS][3], total[3];
  float part[8][3];          // (first block) the blocks' triples
  unsigned int most[32];     // of each eight threads
  unsigned short few[FEW];   // run * STHREADS + thread
  unsigned int run[RUNS][STHREADS];
  int n_few, count;
  u64 bound;                 // (all logits) what a key has to be above
};

// order of logits as unsigned integers; a NaN comes before minus infinity, zeros of both signs are one
__device__ __forceinline__ unsigned int order_of(float x) {
  const unsigned int b = __float_as_uint(x + 0.f);
  return x != x ? 0u : b ^ ((unsigned int)((int)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(unsigned int o) {
  return o == 0u ? __uint_as_float(0x7fffffffu) : __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}
__device__ __forceinline__ u64 key_of(float x, unsigned int i) { return (u64)order_of(x) << 32 | (0xffffffffu - i); }
__device__ __forceinline__ u64 fadd2(u64 a, u64 b) {
  u64 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// A row: `vecs` vectors of 32 aligned bytes (a sector) from x + head on; the few logits before and behind them are its edge.
struct Vec {
  uint32_t w[8];
};
template <typename T>
struct Row {
  static constexpr int E = 32 / sizeof(T);
  const T* x;
  int V, head, vecs, edge;
  __device__ __forceinline__ Row(const T* p, int n) : x(p), V(n) {
    head = min(n, (int)((32 - ((uintptr_t)p & 31)) % 32 / sizeof(T)));
    vecs = (n - head) / E;
    edge = n - vecs * E;
  }
  __device__ __forceinline__ Vec raw(int j) const {
    Vec v;
    asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(v.w[0]), "=r"(v.w[1]), "=r"(v.w[2]), "=r"(v.w[3]), "=r"(v.w[4]), "=r"(v.w[5]), "=r"(v.w[6]), "=r"(v.w[7])
                 : "l"(x + head + (long long)j * E));
    return v;
  }
  __device__ __forceinline__ int edge_at(int e) const { return e < head ? e : e + vecs * E; }
  __device__ __forceinline__ float one(int i) const {
    if constexpr (E == 8)
      return x[i];
    else
      return bf16f(reinterpret_cast<const uint16_t*>(x)[i]);
  }
};
template <int E>
__device__ __forceinline__ void values(const Vec& u, float (&v)[E]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if constexpr (E == 8)
      v[j] = __uint_as_float(u.w[j]);
    else
      v[2 * j] = bf16_lo(u.w[j]), v[2 * j + 1] = bf16_hi(u.w[j]);
  }
}
__device__ __forceinline__ float max_or_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t max_or_nan_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// the largest of a vector (a NaN does not count)
template <int E>
__device__ __forceinline__ float largest(const Vec& u) {
  if constexpr (E == 8) {
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < 8; j += 2) m = fmaxf(fmaxf(m, __uint_as_float(u.w[j])), __uint_as_float(u.w[j + 1]));
    return m;
  } else {
    uint32_t m = 0xff80ff80u;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max_bf16x2(m, u.w[j]);
    return fmaxf(bf16_lo(m), bf16_hi(m));
  }
}

// a triple made relative to the maximum `to`; (minus infinity less itself is no number: nothing is there to be counted)
__device__ __forceinline__ void rebase(float m, float to, float c, float& l, float& s) {
  const float d = fmaxf((m - to) * c, -1e4f), f = exp2_sfu(d);
  s = f * fmaf(l, d, s), l *= f;
}
__device__ __forceinline__ void join(float& m, float& l, float& s, float m2, float l2, float s2, float c) {
  const float to = fmaxf(m, m2);
  rebase(m, to, c, l, s), rebase(m2, to, c, l2, s2);
  m = to, l += l2, s += s2;
}
// the triples of a warp's lanes as one, in all of them
__device__ __forceinline__ void join_warp(float& m, float& l, float& s, float c) {
  const float to = value_of(__reduce_max_sync(0xffffffffu, max(order_of(m), order_of(-INFINITY))));
  rebase(m, to, c, l, s);
  m = to, l = warp_sum(l), s = warp_sum(s);
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
#pragma unroll 4
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

// values that are candidates where there is room for them: false where there was not
template <int E>
__device__ __forceinline__ bool offer(ScoreSmem& sm, const float (&v)[E], unsigned int at, unsigned int least) {
  bool fits = true;
#pragma unroll
  for (int e = 0; e < E; ++e)
    if (order_of(v[e]) >= least) {
      const int to = atomicAdd(&sm.count, 1);
      if (to < CAP)
        sm.key[to] = key_of(v[e], at + e);
      else
        fits = false;
    }
  return fits;
}
// the same, by all threads together and whatever the room: those that are above the bound, which rises
template <int E>
__device__ __forceinline__ void collect(ScoreSmem& sm, const float (&v)[E], unsigned int at, bool there, int k) {
  unsigned int todo = there ? (1u << E) - 1 : 0;
  for (;;) {
    bool left = false;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      if (!(todo >> e & 1)) continue;
      const u64 key = key_of(v[e], at + e);
      if (key <= *(volatile u64*)&sm.bound) {
        todo &= ~(1u << e);
      } else {
        const int to = atomicAdd(&sm.count, 1);
        if (to < CAP)
          sm.key[to] = key, todo &= ~(1u << e);
        else
          left = true;
      }
    }
    if (!__syncthreads_or(left)) return;
    prune(sm, k);
  }
}

template <typename T, bool TOP>
__global__ void __launch_bounds__(STHREADS, sblocks(sizeof(T) == 4)) scores_kernel(ScoreArgs a) {
  constexpr int E = Row<T>::E, U = 2;
  __shared__ ScoreSmem sm;
  cg::cluster_group cluster = cg::this_cluster();
  const int parts = (int)cluster.num_blocks(), part = (int)cluster.block_rank();
  const int t = (int)(blockIdx.x / parts), tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Row<T> row(reinterpret_cast<const T*>(a.x) + (long long)t * a.ld, a.V);
  const int per = (row.vecs + parts - 1) / parts, j0 = min(part * per, row.vecs), j1 = min(j0 + per, row.vecs);
  const float c = a.scale * 1.4426950408889634f;
  // Beside a maximum m of half its size or less, nothing below this has a weight (it is 5e37 min(c, 1) powers of two below m, and c is at
  // least 2^-100), so what is below counts as this: (x - m) c then stays finite, which 0 times minus infinity would not be.  (With m
  // farther from 0, on either side, logits are taken one by one.)
  const float low = __uint_as_float(__float_as_uint(-1e38f / fmaxf(c, 1.f)) & 0xffff0000u);
  const uint32_t low2 = __float_as_uint(low) >> 16 | __float_as_uint(low);
  if (parts > 1) cluster.barrier_arrive();  // (awaited before another block's shared memory is written)

  // given tokens, and the row's edge (a logit to each of the first block's first threads): asked for early
  int tok = -1;
  float given = 0.f, edge = -INFINITY;
  const bool has_edge = part == 0 && tid < row.edge;
  if (has_edge) edge = row.one(row.edge_at(tid));
  if (part == 0 && tid < a.m) {
    tok = a.tok[(long long)t * a.m + tid];
    if (tok >= 0 && tok < a.V) given = row.one(tok);
  }
  if (tid == 0) sm.n_few = 0, sm.count = 0, sm.bound = 0;

  float m = -INFINITY, l = 0.f, s = 0.f;
  auto add_one = [&](float x, float ref) {
    const float d = (x - ref) * c, p = exp2_sfu(d);
    l += p, s = fmaf(p, fmaxf(d, -200.f), s);
  };
  auto add = [&](const Vec& u, float ref) {  // a vector's logits
    if (__builtin_expect(fabsf(ref) > -0.5f * low, 0)) {
      float v[E];
      values(u, v);
#pragma unroll 1
      for (int e = 0; e < E; ++e) {
        add_one(v[0], ref);
#pragma unroll
        for (int i = 1; i < E; ++i) v[i - 1] = v[i];
      }
      return;
    }
    const u64 ref2 = pack2(-ref, -ref), c2 = pack2(c, c), one2 = pack2(1.f, 1.f);
    u64 l2 = pack2(l, 0.f), s2 = pack2(s, 0.f);
#pragma unroll
    for (int j = 0; j < E / 2; ++j) {
      u64 v;
      if constexpr (E == 8) {
        v = pack2(max_or_nan(__uint_as_float(u.w[2 * j]), low), max_or_nan(__uint_as_float(u.w[2 * j + 1]), low));
      } else {
        const uint32_t b = max_or_nan_bf16x2(u.w[j], low2);
        v = pack2(bf16_lo(b), bf16_hi(b));
      }
      const u64 d = fmul2(fadd2(v, ref2), c2);  // (the maximum off before the product: logits far from 0 cost nothing then)
      const float2 e = unpack2(d);
      const u64 p = pack2(exp2_sfu(e.x), exp2_sfu(e.y));
      l2 = ffma2(one2, p, l2), s2 = ffma2(p, d, s2);
    }
    l = pair_sum(l2), s = pair_sum(s2);
  };
  auto reach = [&](float to) {  // a new maximum
    if (to > m) rebase(m, to, c, l, s), m = to;
    return m == -INFINITY ? 0.f : m;
  };
  // a thread's vectors j0 + tid, + STHREADS, ...: in runs of `turns` times U of them
  const int mines = (j1 - j0 + STHREADS - 1) / STHREADS, turns = max((mines + U * RUNS - 1) / (U * RUNS), 1);
  const int runs = (mines + turns * U - 1) / (turns * U);
#pragma unroll 1
  for (int r = 0, j = j0 + tid; r < runs; ++r) {
    float most = -INFINITY;
#pragma unroll 1
    for (int i = 0; i < turns; ++i, j += U * STHREADS) {
      if (j + (U - 1) * STHREADS < j1) {
        Vec u[U];
#pragma unroll
        for (int k = 0; k < U; ++k) u[k] = row.raw(j + k * STHREADS);
#pragma unroll
        for (int k = 0; k < U; ++k) most = fmaxf(most, largest<E>(u[k]));
        const float ref = reach(most);
#pragma unroll
        for (int k = 0; k < U; ++k) add(u[k], ref);
      } else {
#pragma unroll 1
        for (int k = 0; j + k * STHREADS < j1; ++k) {
          const Vec u = row.raw(j + k * STHREADS);
          most = fmaxf(most, largest<E>(u));
          add(u, reach(most));
        }
      }
    }
    if (TOP) sm.run[r][tid] = order_of(most);
  }
  if (has_edge) add_one(edge, reach(edge));
  const unsigned int mine = order_of(m);
  if (TOP) {
    unsigned int g = mine;
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) g = max(g, __shfl_xor_sync(0xffffffffu, g, o));
    if ((lane & 7) == 0) sm.most[tid >> 3] = g;
  }
  join_warp(m, l, s, c);
  if (lane == 0) sm.mls[warp][0] = m, sm.mls[warp][1] = l, sm.mls[warp][2] = s;
  __syncthreads();
  if (warp == 0) {
    m = lane < SWARPS ? sm.mls[lane][0] : -INFINITY, l = lane < SWARPS ? sm.mls[lane][1] : 0.f, s = lane < SWARPS ? sm.mls[lane][2] : 0.f;
    join_warp(m, l, s, c);
    if (lane == 0) sm.total[0] = m, sm.total[1] = l, sm.total[2] = s;
  }

  if (TOP) {
    // the k-th largest of the 32 maxima: a lane's rank among them
    const unsigned int g = sm.most[lane];
    int rank = 0;
#pragma unroll
    for (int o = 0; o < 32; ++o) {
      const unsigned int h = __shfl_sync(0xffffffffu, g, o);
      rank += h > g || (h == g && o < lane);
    }
    unsigned int least = __shfl_sync(0xffffffffu, g, __ffs(__ballot_sync(0xffffffffu, rank == a.k - 1)) - 1);
    // nothing above minus infinity in some of them: they may stand for threads without logits
    if (least <= order_of(-INFINITY)) least = 0;
    if (mine >= least)
#pragma unroll 1
      for (int r = 0; r < runs; ++r)
        if (sm.run[r][tid] >= least) {
          const int at = atomicAdd(&sm.n_few, 1);
          if (at < FEW) sm.few[at] = (unsigned short)(r * STHREADS + tid);
        }
    __syncthreads();
    const int n = sm.n_few, len = turns * U;
    bool fits = n <= FEW;
    if (fits) {
#pragma unroll 1
      for (int f = tid; f < n * len; f += STHREADS) {
        const int which = sm.few[f / len], i = j0 + which % STHREADS + (which / STHREADS * len + f % len) * STHREADS;
        if (i < j1) {
          float v[E];
          values(row.raw(i), v);
          fits = offer(sm, v, row.head + i * E, least) && fits;
        }
      }
      const float one[1] = {edge};
      if (has_edge) fits = offer(sm, one, row.edge_at(tid), least) && fits;
    }
    if (!__syncthreads_and(fits)) {
      if (tid == 0) sm.count = 0, sm.bound = least ? ((u64)least << 32) - 1 : 0;
      __syncthreads();
      // from the lowest index on, so that of equal values the first found stay
      const float one[1] = {edge};
      collect(sm, one, has_edge ? row.edge_at(tid) : 0, has_edge && row.edge_at(tid) < row.head, a.k);
      for (int i = j0; i < j1; i += STHREADS) {
        float v[E] = {};
        if (i + tid < j1) values(row.raw(i + tid), v);
        collect(sm, v, row.head + (i + tid) * E, i + tid < j1, a.k);
      }
      collect(sm, one, has_edge ? row.edge_at(tid) : 0, has_edge && row.edge_at(tid) >= row.head, a.k);
    }
    prune(sm, a.k);
  } else {
    __syncthreads();
  }
  m = sm.total[0], l = sm.total[1], s = sm.total[2];
  if (parts > 1) {
    ScoreSmem* first = cluster.map_shared_rank(&sm, 0);
    cluster.barrier_wait();
    if (tid == 0) first->part[part][0] = m, first->part[part][1] = l, first->part[part][2] = s;
    if (TOP && tid < SSM_MAX_TOP) first->all[part * SSM_MAX_TOP + tid] = tid < sm.count ? sm.sorted[tid] : 0ull;
    cluster.sync();
    if (part > 0) return;
    m = sm.part[0][0], l = sm.part[0][1], s = sm.part[0][2];
#pragma unroll 1
    for (int i = 1; i < parts; ++i) join(m, l, s, sm.part[i][0], sm.part[i][1], sm.part[i][2], c);
    if (TOP) {
      const int n = parts * SSM_MAX_TOP;
      const u64 key = tid < n ? sm.all[tid] : 0ull;
      if (key) {  // its rank: those of its own block that are larger, and of each other block's, sorted, as many as are larger
        int rank = tid % SSM_MAX_TOP;
#pragma unroll 1
        for (int i = 0; i < parts; ++i) {
          if (i == tid / SSM_MAX_TOP) continue;
          const u64* other = sm.all + i * SSM_MAX_TOP;
          int at = 0;
#pragma unroll
          for (int step = SSM_MAX_TOP / 2; step > 0; step >>= 1)
            if (other[at + step - 1] > key) at += step;
          rank += at + (other[at] > key);
        }
        if (rank < a.k) sm.sorted[rank] = key;
      }
      __syncthreads();
    }
  }
  const float log_l = logf(l), twice = 2.f * a.scale;
  if (tid == 0 && a.entropy) a.entropy[t] = log_l - 0.6931471805599453f * (s / l);
  for (int i = tid; i < a.m; i += STHREADS) {
    if (i >= STHREADS) {
      tok = a.tok[(long long)t * a.m + i];
      if (tok >= 0 && tok < a.V) given = row.one(tok);
    }
    float r = fmaf(0.5f * given - 0.5f * m, twice, -log_l);  // (halves: the difference itself may be beyond fp32)
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
    if (a.top_logprob) a.top_logprob[(long long)t * a.k + tid] = fmaf(0.5f * value_of((unsigned int)(key >> 32)) - 0.5f * m, twice, -log_l);
  }
}
static_assert(RUNS * STHREADS <= 65536 && 2 * 31 < STHREADS, "a run's number in 16 bits, a thread to each logit of the edge");
static_assert(8 * SSM_MAX_TOP <= STHREADS, "a thread to each of the blocks' candidates");

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
  // Blocks to a row: what takes least, rounds of blocks times a block's bytes and what it takes beside them, about as long as 32 KB
  // (256 rows of 128259 in bf16: 27 us with four, 21 with two, 24 with one; 640 of 151936 in fp32: 67 with one, 74 with four).
  const long long bytes = (long long)a.V * (a.f32 ? 4 : 2);
  const long long slots = (long long)sblocks(a.f32) * kSMs;
  long long best = LLONG_MAX;
  int parts = 1;
  for (int p = 1; p <= 8; p *= 2) {
    const long long rounds = ((long long)a.T * p + slots - 1) / slots, est = rounds * (bytes / p + 32768);
    if (est < best) best = est, parts = p;
  }
  return a.f32 ? run_scores<float>(a, parts, s) : run_scores<uint16_t>(a, parts, s);
}

}  // namespace ssmtree
