// What the tree attention kernels over caches of either width share: how the caches are cut into runs of tiles, a tree's
// ancestor words, the join of the runs' partial sums.
#pragma once

#include "prompt.cuh"
#include "umma.cuh"

namespace ssmtree {

constexpr int KT = 64;  // keys per tile

__device__ __forceinline__ float max3f(float a, float b, float c) { return fmaxf(fmaxf(a, b), c); }

// a sequence's cached rows; -1: not a length there is room for
__device__ __forceinline__ int cached_rows(const AttendArgs& a, int s) {
  const int len = a.cache_len[s];
  return len < 0 || len > a.max_len || (long long)len > ((long long)a.max_pages << a.page_shift) ? -1 : len;
}

// Splits.  Every sequence's tiles are cut into runs of the same length, and every CTA works out that length from the lengths
// in device memory: of 189 from the longest sequence's tiles down to a 64th of them, each tried by a thread, the one whose
// CTAs take least, where a CTA costs about four tiles beside its own and joining about two.  (Cut by the longest sequence
// alone, eight ragged caches of up to 8117 rows took 50 us and four of up to 40009 rows, 101 us.)
constexpr int CANDIDATES = 189;
struct SplitScratch {        // of each warp: tiles of the longest sequence, the least estimate
  int most[12];
  unsigned int least[12];
};
template <int THREADS>
__device__ __forceinline__ int choose_split(const AttendArgs& a, int per, int* tiles, SplitScratch* ms) {
  static_assert(THREADS <= 384, "a place for each warp");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int most = 0;
  for (int s = tid; s < a.S; s += THREADS) most = max(most, tiles[s] = (max(cached_rows(a, s), 0) + KT - 1) / KT + 1);
  most = __reduce_max_sync(0xffffffffu, most);
  if (lane == 0) ms->most[warp] = most;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) most = max(most, ms->most[w]);
  unsigned int key = 0xffffffffu;
  for (int c = tid; c < CANDIDATES; c += THREADS) {
    const unsigned int tps = (3u * most + c + 2) / (c + 3);
    unsigned int runs = 0;
    float total = 0.f;
    for (int s = 0; s < a.S; ++s) runs += (tiles[s] + tps - 1) / tps, total += (float)tiles[s];
    if (runs <= (unsigned)a.max_runs) {  // (one run to a sequence always is)
      constexpr float slots = 2 * kSMs;
      const float ctas = (float)(runs * per), len = tps + 4.f;
      const float waves = ceilf(ctas / slots) * len, list = (total * per + 4.f * ctas) / slots + len;
      const float est = fminf(waves, list) + (runs > (unsigned)a.S ? 2.f : 0.f);
      key = min(key, (unsigned int)fminf(est / most * 65536.f, 16777215.f) << 8 | (unsigned int)c);
    }
  }
  key = __reduce_min_sync(0xffffffffu, key);
  if (lane == 0) ms->least[warp] = key;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) key = min(key, ms->least[w]);
  const unsigned int c = key & 255u;
  return (int)((3u * most + c + 2) / (c + 3));
}
// the sequence of the run-th run, its first run and their number
__device__ __forceinline__ bool find_run(int S, const int* tiles, int tps, int run, int& s, int& first, int& runs) {
  const int lane = threadIdx.x & 31;
  for (int b = 0, before = 0; b < S; b += 32) {
    const int k = b + lane < S ? (tiles[b + lane] + tps - 1) / tps : 0;
    int upto = k;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += u;
    }
    const unsigned int past = __ballot_sync(0xffffffffu, before + upto > run);
    if (past) {
      const int l = __ffs(past) - 1;
      s = b + l, runs = __shfl_sync(0xffffffffu, k, l), first = before + __shfl_sync(0xffffffffu, upto, l) - runs;
      return true;
    }
    before += __shfl_sync(0xffffffffu, upto, 31);
  }
  return false;
}

// a warp: each node's ancestors and itself as bits: a node's own bit, then its parent's word, its grandparent's, ... by doubling
__device__ __forceinline__ void ancestor_words(const AttendArgs& a, int s, unsigned long long* anc, bool report) {
  const int lane = threadIdx.x & 31;
  unsigned long long w[2];
  int p[2];
  bool bad = false;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int v = lane + 32 * k;
    p[k] = -1;
    if (v > 0 && v < a.n) {
      p[k] = a.layout[(long long)s * a.n + v].parent;
      if (p[k] < 0 || p[k] >= v) p[k] = -1, bad = true;
    }
    w[k] = 1ull << v;
  }
  if (bad && report) flag(a.status, SSM_STATUS_BAD_LAYOUT);
#pragma unroll 1
  for (int far = 1; far < a.n; far *= 2) {
    unsigned long long up[2];
    int pp[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {  // the word and the link of node p[k], which lane p[k] % 32 holds
      const int from = p[k] & 31;
      const unsigned long long u0 = __shfl_sync(0xffffffffu, w[0], from), u1 = __shfl_sync(0xffffffffu, w[1], from);
      const int q0 = __shfl_sync(0xffffffffu, p[0], from), q1 = __shfl_sync(0xffffffffu, p[1], from);
      up[k] = p[k] < 32 ? u0 : u1, pp[k] = p[k] < 32 ? q0 : q1;
    }
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (p[k] >= 0) w[k] |= up[k], p[k] = pp[k];
  }
  anc[lane] = w[0], anc[lane + 32] = w[1];
}

// ---- host ----
// Row tiles, and the most runs that the sequences are cut into (0: they are not cut, where the CTAs
// fill the SMs twice over or the longest sequence is too short for what joining costs).  Uncut, one long cache among many
// short ones is walked by a CTA for each of its heads: 128 single tokens of 8 heads over 1000 rows each take 98 us, with
// 64000 rows for one of them 698; 72 of them, which are cut, 112.
struct AttendPlan {
  int row_tiles, max_runs;
};
inline AttendPlan plan_attend(int S, int n, int Hq, int Hkv, int max_len) {
  AttendPlan p;
  const int rows = n * (Hq / Hkv);
  p.row_tiles = (rows + 127) / 128;
  const long long per = (long long)Hkv * p.row_tiles, slots = 2 * kSMs;
  p.max_runs = max_len > 5 * KT && S * per < 2 * slots ? S + (int)((slots + per - 1) / per) : 0;
  return p;
}
inline size_t attend_workspace_bytes(const AttendPlan& p, int S, int n, int Hq, int Hkv, int D) {
  return 256 + (p.max_runs ? (size_t)p.max_runs * Hkv * n * (Hq / Hkv) * (D + 2) * sizeof(float) + S * sizeof(int2) : 0);
}
inline void lay_workspace(AttendArgs& a, const AttendPlan& p, void* workspace) {
  const size_t parts = (size_t)p.max_runs * a.Hkv * a.n * a.g;
  a.max_runs = p.max_runs;
  a.part = static_cast<float*>(workspace);
  a.part_ml = reinterpret_cast<float2*>(a.part + parts * a.D);
  a.runs = reinterpret_cast<int2*>(a.part_ml + parts);
}
// o = sum over a row's runs of 2^(m_i - m) o_i / sum of 2^(m_i - m) l_i, of rows that are cut into more than one
cudaError_t launch_attend_join(const AttendArgs& a, cudaStream_t s);

}  // namespace ssmtree
