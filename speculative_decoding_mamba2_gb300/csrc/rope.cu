// Rotary positions of q and k rows (ssm_attention.h).
//
// A pair (a, b) of a row at position p becomes (a cos - b sin, b cos + a sin) at the angle p f.  The angle is taken in turns, as
// a 64-bit fraction: p times the table's f / (2 pi) 2^64 modulo 2^64 is exact (the table's own rounding, 2^-55 of a turn, is all that
// grows with the position), and its upper 32 bits are the angle of a sine and cosine in half turns.
// One thread has eight columns (and their eight partners, half a rotated part on) of a row, makes their sines once and turns
// a run of eight heads with them; where there are few rows a run is one head, so that all heads are under way at once.  Bound by
// HBM where there are many rows: 8191 rows of 40 heads of 128 in 31 us (168 MB: 5.3 TB/s; runs of 4 or 20 heads 33 and 32).
#include <type_traits>

#include "decode.cuh"
#include "mma_tiles.cuh"

namespace ssmtree {
namespace {

constexpr int RTHREADS = 256;

struct Turn {
  float c, s;
};
__device__ __forceinline__ Turn turn_of(const RopeArgs& a, int pos, int pair) {
  const unsigned long long t = (unsigned long long)(long long)pos * a.turns[pair];
  Turn r;
  sincospif((float)(int)(t >> 32) * 0x1p-31f, &r.s, &r.c);
  r.c *= a.amp, r.s *= a.amp;
  return r;
}
__device__ __forceinline__ int position(const RopeArgs& a, int row) {
  if (a.n == 0) return a.pos[row];
  int len = a.cache_len[row / a.n], d = a.layout[row].depth, bits = 0;
  if (len < 0) len = 0, bits |= SSM_STATUS_SEQ_RANGE;
  if (d < 0 || d >= a.n) d = 0, bits |= SSM_STATUS_BAD_LAYOUT;
  if (bits) flag(a.status, bits);
  return (int)min((long long)len + d, (long long)INT32_MAX);
}

// V: columns of a vector (8, or 1 where the rotated part does not divide into vectors)
template <int V, bool INTER>
__global__ void __launch_bounds__(RTHREADS) rope_kernel(RopeArgs a, int run, int runs, int rows_per_block) {
  using Vec = typename std::conditional<V == 8, uint4, uint16_t>::type;
  constexpr int NP = V == 1 ? 1 : INTER ? V / 2 : V;  // pairs of a thread
  const int half = a.rot / 2, turning = INTER && V > 1 ? a.rot / V : half / (V == 1 ? 1 : V);
  const int slots = turning + (a.D - a.rot) / V, per = slots * runs, heads = a.heads[0] + a.heads[1];
  const int row0 = blockIdx.x * rows_per_block, rows = min(rows_per_block, a.n_tok - row0);
#pragma unroll 1
  for (int i = threadIdx.x; i < rows * per; i += RTHREADS) {
    const int row = row0 + i / per, slot = i % per % slots, h0 = i % per / slots * run, h1 = min(h0 + run, heads);
    const bool turns = slot < turning;
    Turn t[NP];
    if (turns) {
      const int pos = position(a, row);
#pragma unroll
      for (int j = 0; j < NP; ++j) t[j] = turn_of(a, pos, slot * NP + j);
    }
    const int first = !turns ? a.rot + (slot - turning) * V : V == 1 && INTER ? 2 * slot : slot * V;
    const int second = V == 1 && INTER ? 1 : half;  // columns from a pair's first to its second
#pragma unroll 2
    for (int h = h0; h < h1; ++h) {
      const int which = h >= a.heads[0];
      const int col = (which ? h - a.heads[0] : h) * a.D + first;
      const uint16_t* in = a.in[which] + row * a.ldi[which] + col;
      uint16_t* out = a.out[which] + row * a.ldo[which] + col;
      Vec x = *reinterpret_cast<const Vec*>(in);
      if (!turns) {
        if (in != out) *reinterpret_cast<Vec*>(out) = x;
        continue;
      }
      if constexpr (V == 1) {
        const float p = bf16f(x), q = bf16f(in[second]);
        const uint32_t r = pack_bf16x2(p * t[0].c - q * t[0].s, q * t[0].c + p * t[0].s);
        out[0] = (uint16_t)r, out[second] = (uint16_t)(r >> 16);
      } else {
        uint32_t u[4] = {x.x, x.y, x.z, x.w};
        if constexpr (INTER) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float p = bf16_lo(u[j]), q = bf16_hi(u[j]);
            u[j] = pack_bf16x2(p * t[j].c - q * t[j].s, q * t[j].c + p * t[j].s);
          }
        } else {
          const uint4 y = *reinterpret_cast<const uint4*>(in + second);
          uint32_t w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float p0 = bf16_lo(u[j]), p1 = bf16_hi(u[j]), q0 = bf16_lo(w[j]), q1 = bf16_hi(w[j]);
            const Turn &t0 = t[2 * j], &t1 = t[2 * j + 1];
            u[j] = pack_bf16x2(p0 * t0.c - q0 * t0.s, p1 * t1.c - q1 * t1.s);
            w[j] = pack_bf16x2(q0 * t0.c + p0 * t0.s, q1 * t1.c + p1 * t1.s);
          }
          *reinterpret_cast<uint4*>(out + second) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        *reinterpret_cast<uint4*>(out) = make_uint4(u[0], u[1], u[2], u[3]);
      }
    }
  }
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, cudaStream_t s) {
  const int heads = a.heads[0] + a.heads[1];
  if (a.n_tok == 0 || heads == 0) return cudaSuccess;
  const bool vec = a.rot % (a.interleaved ? 8 : 16) == 0;
  const int v = vec ? 8 : 1, slots = (a.interleaved && vec ? a.rot / 8 : a.rot / 2 / v) + (a.D - a.rot) / v;
  const long long all = (long long)a.n_tok * slots * heads;
  // (the sines of many rows cost more than their heads one after the other: 640 rows, half of each head, 7.7 us with runs of one,
  // 4.8 with runs of eight; 300 whole ones 4.2 and 5.3)
  const int run = all > 8ll * kSMs * RTHREADS ? (heads < 8 ? heads : 8) : 1;
  const int runs = (heads + run - 1) / run, per = slots * runs;
  const int rows = per >= RTHREADS ? 1 : RTHREADS / per;
  const unsigned grid = ((unsigned)a.n_tok + rows - 1) / rows;
  if (vec && a.interleaved)
    rope_kernel<8, true><<<grid, RTHREADS, 0, s>>>(a, run, runs, rows);
  else if (vec)
    rope_kernel<8, false><<<grid, RTHREADS, 0, s>>>(a, run, runs, rows);
  else if (a.interleaved)
    rope_kernel<1, true><<<grid, RTHREADS, 0, s>>>(a, run, runs, rows);
  else
    rope_kernel<1, false><<<grid, RTHREADS, 0, s>>>(a, run, runs, rows);
  return cudaGetLastError();
}

}  // namespace ssmtree
