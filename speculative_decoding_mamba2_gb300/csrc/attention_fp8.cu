// Attention of a draft tree's nodes over an 8-bit paged cache and their ancestors, and the commit of the accepted path into it
// (ssm_attention.h).
#include <type_traits>

#include "attend.cuh"
#include "decode.cuh"

namespace ssmtree {
namespace {

// The plan is that of the 16-bit kernel (attention.cu): up to 128 query rows of a key/value head walk tiles of 64 keys,
//     S = Q . K^T,   P = 2^(S - m),   O += P . V
// on tcgen05, softmax statistics in a row's thread, two CTAs to an SM, the caches cut into runs.  What 8 bits change:
//  * K is multiplied as it is (kind::f8f6f4).  Q goes as two e4m3 terms of a row scale that is a power of two: bf16's 8 bits are
//    4 + 4, so nothing is lost but what is below 2^-18 of a row's largest.  Twice the products at twice bf16's rate, and half the
//    bytes.  Eight warps make the terms, a row's columns side by side (a thread to a row, in registers, spilled: 10 % of all).
//  * V is made fp16 (exact) by four warps on the way, since P in e4m3 would not do: P goes as fp16, whose 11 bits are more than
//    bf16's.  Converting V costs a cvt for two values; splitting P into two terms would cost four for two of as many.  (The
//    softmax's own warps converting it: 8 trees 50 us and not 40, wide trees 149 and not 113.)
//  * A block's scale of K multiplies its scores in the softmax's own multiply-add.  Its scale of V is part of the weight: m is the
//    maximum of S + log2 vs, so the weight w = 2^(S + log2 vs - m) fits fp16 whatever the scales, and the row's sum adds w / vs.  Scales
//    of V count relative to one of them, v0, so that neither sum leaves fp32.
// Weights are 2^7 times as large (at most 2^15 with a maximum that lags by 2^8), so that fp16 holds them to 2^-31 of the largest.
// The tree's own rows are bf16 and the first tile of a sequence's first run: their products are bf16's, with Q as it came in the columns
// that O will take, and their K and V in the places of the first two fp16 tiles of V.  O is in units of v0, which is there the least of
// the first scales of V: the tree's weights 2^(S - m) go into the sum as they are and into the product divided by v0, in bf16, whose
// range is fp32's.  (With 1 for v0, wide trees over a flat cache of 320 rows that has half of the weights were off by 4 % of o at values of
// 2^-16, by half at 2^-20.)
//
// In a CUDA graph, 32 query and 8 (wide trees: 4) key/value heads of 128: 8 trees of 16 nodes over up to 8117 rows 41 us (84 MB of
// cache at 2.0 TB/s), 4 of 40 over up to 40009 rows 113 us (760 TFLOP/s with Q's terms counted once); with heads of 64 37 and 99.
// (Up to 16 query rows of a key/value head are attention_fp8_few.cu's.)  Wide trees are bound by the round trips of the two tiles under
// way (P to P . V to S to the softmax) on top of the products: without copies, conversion or Q's lower terms they take as long; with
// an idle softmax 15 % less, with that and no products a third less.
constexpr int A8THREADS = 384;  // 4 softmax warps; copies, MMAs of S, MMAs of P . V, what keys a tile has; 4 warps that make V fp16
// registers of the three groups of four warps: the block has 384 x 80
constexpr int R_SOFTMAX = 136, R_MMA = 48, R_CONVERT = 56;
static_assert(R_SOFTMAX + R_MMA + R_CONVERT == 3 * 80, "what the block is launched with");
constexpr int BLK = KT * 128;   // 64 rows x 64 columns of 16 bits
// tensor memory columns: S of even and of odd tiles, each then overwritten by its P; O
constexpr int A_S = 0, A_O = 128, A_COLS = 256;

template <int D>
struct Attend8Smem {
  static constexpr int KU = D == 128 ? 3 : 6, VU = D == 128 ? 2 : 6;  // tiles of K and of V in e4m3, in rings
  static constexpr int TILE8 = KT * D, TILE16 = KT * D * 2;
  static constexpr int OFF_V16 = 2 * 128 * D;        // after Q's two terms
  static constexpr int OFF_K = OFF_V16 + 2 * TILE16, OFF_V = OFF_K + KU * TILE8;
  static constexpr int OFF_MISC = OFF_V + VU * TILE8;
  static constexpr int BYTES = OFF_MISC + 2688;
  static_assert(BYTES <= 228 * 1024 / 2 - 1024, "two to an SM");
  static constexpr uint32_t DESC_HI = D == 128 ? kDescHi : (512u >> 4) | 1u << 14 | 4u << 29;  // 128- or 64-byte rows, swizzled
  // byte offset of 16-byte chunk `chunk` of row `row` of a tile of D-byte rows
  static __device__ __forceinline__ uint32_t off8(int row, int chunk) {
    return D == 128 ? tile_off(row, chunk, 128) : (uint32_t)(row * 64 + ((chunk ^ (row >> 1 & 3)) << 4));
  }
};
constexpr int INFOS = 8;  // a tile of V is copied once five tiles before are done with
struct TileInfo {  // of each 8 keys: scale of k, log2 of the scale of v and its inverse, relative to the run's; which keys there are
  float ks[8], lv[8], rv[8];
  unsigned long long mask;
  unsigned long long pad;
};
struct Attend8Misc {
  TileInfo info[INFOS];        // of tile i, at i % INFOS
  unsigned long long anc[64];  // ancestors and self of each node
  unsigned long long k_full[6], k_free[6], v_full[6], v_free[6], v16_full[2], v16_free[2], info_full[INFOS], q_full, s_full[2], p_full[2], o_done[2], all_done, tree_full, v0_full, drain[2];
  SplitScratch split;
  unsigned int odd[2];         // tree rows with a value of v that is not finite
  float qs[128];               // a row's scale of Q
  uint32_t tmem;
  int stop;
  float v0;                    // what the run's scales of v are relative to
};
static_assert(sizeof(Attend8Misc) <= 2688, "space");
static_assert(Attend8Smem<64>::VU + 2 <= INFOS && Attend8Smem<128>::VU + 2 <= INFOS, "a place is free when its next tile is there");

__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool b_mn) {  // fp16 x fp16 -> fp32
  return (1u << 4) | (b_mn ? 1u << 16 : 0u) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ float least_scale(uint32_t most) {  // of a largest magnitude's bits: 448 is 1.75 * 2^8
  const int e = (int)(most >> 23) - 127 - 8 + ((most & 0x7fffffu) > 0x600000u);
  return __uint_as_float((uint32_t)(max(e, -100) + 127) << 23);
}
__device__ __forceinline__ uint32_t finite_bits(float x) {  // |x|, 0 where it is not finite
  const uint32_t b = __float_as_uint(x) & 0x7fffffffu;
  return b < 0x7f800000u ? b : 0u;
}

template <int D>
__global__ void __launch_bounds__(A8THREADS, 2)
    attend8_kernel(const __grid_constant__ CUtensorMap tkp, const __grid_constant__ CUtensorMap tkt,
                   const __grid_constant__ CUtensorMap tvt, AttendFp8Args f) {
  using Sh = Attend8Smem<D>;
  constexpr int DB = D / 64, KU = Sh::KU, VU = Sh::VU;
  const AttendArgs& a = f.a;
  extern __shared__ __align__(1024) unsigned char smem[];  // (there is no room to move it: where it is not aligned, nothing runs)
  const uint32_t sb = smem_u32(smem);
  Attend8Misc* ms = reinterpret_cast<Attend8Misc*>(smem + Sh::OFF_MISC);
  volatile int* stop = &ms->stop;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int rows = a.n * a.g, rt = (rows + 127) / 128;
  const int r0 = (blockIdx.x % rt) * 128, run = blockIdx.x / rt, kvh = blockIdx.y;
  if (smem_u32(smem) & 1023u) {
    grid_dependency_wait();  // no grid ends before the one that it depends on
    if (tid == 0) flag(a.status, SSM_STATUS_TIMEOUT);
    if (tid == 0 && run < a.S && a.max_runs > 0) a.runs[run] = make_int2(0, 1);  // nothing to join
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < 6; ++i) {
      mbar_init(smem_u32(&ms->k_full[i]), 1);
      mbar_init(smem_u32(&ms->k_free[i]), 1);
      mbar_init(smem_u32(&ms->v_full[i]), 1);
      mbar_init(smem_u32(&ms->v_free[i]), 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&ms->v16_full[i]), 4);
      mbar_init(smem_u32(&ms->v16_free[i]), 1);
      mbar_init(smem_u32(&ms->s_full[i]), 2);
      mbar_init(smem_u32(&ms->p_full[i]), 4);
      mbar_init(smem_u32(&ms->o_done[i]), 1);
      mbar_init(smem_u32(&ms->drain[i]), 1);
    }
    for (int i = 0; i < INFOS; ++i) mbar_init(smem_u32(&ms->info_full[i]), 1);
    mbar_init(smem_u32(&ms->q_full), 8);
    mbar_init(smem_u32(&ms->all_done), 1);
    mbar_init(smem_u32(&ms->tree_full), 1);
    mbar_init(smem_u32(&ms->v0_full), 1);
    ms->stop = 0;
    ms->odd[0] = ms->odd[1] = 0;
    fence_barrier_init();
  }
  grid_dependency_wait();  // what the stream's kernels before this one write
  // (not before that: a kernel that lets this one's blocks in before it has its own tensor memory would wait for them for ever)
  if (warp == 5) tmem_alloc_warp(smem_u32(&ms->tmem), A_COLS);
  int s = run, sp = 0, tps = 1 << 30, splits = 1;
  bool any = true;
  if (a.max_runs > 0) {
    int* tiles = reinterpret_cast<int*>(smem);  // space not in use yet
    int first;
    tps = choose_split<A8THREADS>(a, a.Hkv * rt, tiles, &ms->split);
    any = find_run(a.S, tiles, tps, run, s, first, splits);
    sp = any ? run - first : 0;
    fence_async_smem();  // (before the barrier behind which the copies may write there)
    if (any && sp == 0 && kvh == 0 && r0 == 0 && tid == 0) a.runs[s] = make_int2(first, splits);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  launch_dependents();  // (not before the tensor memory is there: the next grid's blocks may take some before they wait for this one)
  const uint32_t tmem = __shfl_sync(0xffffffffu, ms->tmem, 0);
  if (!any) {
    if (warp == 5) tmem_free_warp(tmem, A_COLS);
    return;
  }
  int len = __shfl_sync(0xffffffffu, cached_rows(a, s), 0);
  if (len < 0) {
    if (sp == 0 && kvh == 0 && r0 == 0 && tid == 0) flag(a.status, SSM_STATUS_SEQ_RANGE);
    len = 0;
  }
  const int ct = (len + KT - 1) / KT;  // tiles of the cache; the tree's is before them
  const int i0 = sp * tps, n = min(ct + 1 - i0, tps), has_tree = sp == 0;
  // tile i of the run is cache tile i0 + i - 1, the (i - has_tree)-th of the rings; its S, P and fp16 V are at i % 2, and every
  // barrier of those is one of two: who waits could otherwise find it two phases on, and take that for none

  // Q's two terms: eight columns a thread, a row's columns side by side, two rows at a time, by eight warps.  (Beyond the last row
  // stands anything: it stays in its own row of S and O, whose maximum is not looked at.)
  auto split_q = [&](int t) {
    constexpr int PIECES = D / 8, RI = 256 / PIECES, BATCH = 2;
    const int piece = t % PIECES, last = min(rows - r0, 128);
    int r = t / PIECES;
    const uint16_t* q = a.q + (long long)s * a.n * a.ldq + kvh * a.g * D + piece * 8;
#pragma unroll 1
    for (int r1 = 0; r1 < last; r1 += BATCH * RI) {
      uint32_t w[BATCH][4], most[BATCH];
#pragma unroll
      for (int b = 0; b < BATCH; ++b) {
        const int at = r + b * RI;
        const unsigned int u = (unsigned)(r0 + at) / (unsigned)a.g;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (at < last) v = *reinterpret_cast<const uint4*>(q + u * a.ldq + (r0 + at - u * a.g) * D);
        w[b][0] = v.x, w[b][1] = v.y, w[b][2] = v.z, w[b][3] = v.w;
      }
      bool odd = false;
#pragma unroll
      for (int b = 0; b < BATCH; ++b) {  // the largest magnitude's bits
        const uint32_t two = __vmaxu2(__vmaxu2(w[b][0] & 0x7fff7fffu, w[b][1] & 0x7fff7fffu), __vmaxu2(w[b][2] & 0x7fff7fffu, w[b][3] & 0x7fff7fffu));
        most[b] = max(two & 0xffffu, two >> 16);
        odd = odd || most[b] >= 0x7f80u;
      }
      if (__builtin_expect(__any_sync(0xffffffffu, odd), 0)) {  // what is not finite becomes NaN, and does not count
#pragma unroll
        for (int b = 0; b < BATCH; ++b) {
          most[b] = 0;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t lo = w[b][j] & 0x7fffu, hi = w[b][j] >> 16 & 0x7fffu;
            most[b] = max(most[b], max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u));
            w[b][j] |= (lo < 0x7f80u ? 0u : 0x7fffu) | (hi < 0x7f80u ? 0u : 0x7fff0000u);
          }
        }
      }
#pragma unroll
      for (int o = PIECES / 2; o > 0; o >>= 1)
#pragma unroll
        for (int b = 0; b < BATCH; ++b) most[b] = max(most[b], __shfl_xor_sync(0xffffffffu, most[b], o));
#pragma unroll
      for (int b = 0; b < BATCH; ++b) {
        const float qs = least_scale(most[b] << 16);
        const uint32_t inv = (0x7f000000u - __float_as_uint(qs)) >> 16, inv2 = inv | inv << 16;  // 1 / 2^e
        uint32_t hi[2], lo[2];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t x = bf16x2_mul(w[b][j], inv2), p = pack_f16x2(bf16_lo(x), bf16_hi(x));  // (exact: 8 of 11 bits)
          const uint32_t top = f16x2_e4m3x2(p), rest = f16x2_e4m3x2(f16x2_sub(p, e4m3x2_f16x2(top)));
          hi[j / 2] = j & 1 ? hi[j / 2] | top << 16 : top, lo[j / 2] = j & 1 ? lo[j / 2] | rest << 16 : rest;
        }
        const uint32_t to = Sh::off8(r + b * RI, piece / 2) + piece % 2 * 8;
        *reinterpret_cast<uint2*>(smem + to) = make_uint2(hi[0], hi[1]);
        *reinterpret_cast<uint2*>(smem + 128 * D + to) = make_uint2(lo[0], lo[1]);
        if (piece == 0) ms->qs[r + b * RI] = qs;
      }
      r += BATCH * RI;
    }
  };

  if (warp < 4) {
    take_registers<R_SOFTMAX>();
    const int row = r0 + tid;  // this thread's
    const int node = row < rows ? row / a.g : 0, qh = row < rows ? row % a.g : 0;
    const uint32_t lanes = (uint32_t)(warp * 32) << 16;
    {  // q as it is, where O will be: for the tree's tile
      uint4 x[D / 8];
      if (has_tree) {
        const uint4* q = reinterpret_cast<const uint4*>(a.q + ((long long)s * a.n + node) * a.ldq + (kvh * a.g + qh) * D);
#pragma unroll
        for (int c = 0; c < D / 8; ++c) x[c] = row < rows ? q[c] : make_uint4(0, 0, 0, 0);
      }
      split_q(tid);
      if (has_tree) {
#pragma unroll
        for (int c = 0; c < D / 8; c += 2) {
          const uint32_t u[8] = {x[c].x, x[c].y, x[c].z, x[c].w, x[c + 1].x, x[c + 1].y, x[c + 1].z, x[c + 1].w};
          tmem_st8(tmem + A_O + lanes + 4 * c, u);
        }
        tmem_wait_st();
      }
      tc_fence_before();
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&ms->q_full));
    }
    if (has_tree && warp == 0) ancestor_words(a, s, ms->anc, kvh == 0 && r0 == 0);

    float m = -INFINITY, l = 0.f;
    bool ok = wait_bar(&ms->q_full, 0, stop);
    // this row's scale of Q, times scale log2 e (with ks at least 2^-66: their product is a normal number)
    const float qc = fmaxf(ms->qs[tid] * a.scale_log2, 0x1p-60f);
#pragma unroll 1
    for (int i = 0; i < n && ok; ++i) {
      const bool tree = has_tree && i == 0;
      const uint32_t st = tmem + A_S + (i & 1) * KT + lanes;
      ok = wait_bar(&ms->s_full[i & 1], (i >> 1) & 1, stop);  // (and what the tile's keys are)
      if (!ok) break;
      tc_fence_after();
      const TileInfo* in = &ms->info[i % INFOS];
      float sv[KT];
#pragma unroll
      for (int c = 0; c < KT; c += 16) tmem_ld16_async(st + c, reinterpret_cast<float(&)[16]>(sv[c]));
      unsigned long long there = in->mask;
      const float4 ks0 = *reinterpret_cast<const float4*>(in->ks), ks1 = *reinterpret_cast<const float4*>(in->ks + 4);
      const float4 lv0 = *reinterpret_cast<const float4*>(in->lv), lv1 = *reinterpret_cast<const float4*>(in->lv + 4);
#pragma unroll
      for (int c = 0; c < KT; c += 16) tmem_wait_ld16(reinterpret_cast<float(&)[16]>(sv[c]));
      if (__builtin_expect(tree, 0)) {  // rows of V that are not to be multiplied, and values that are not finite, become zeros
        ok = wait_bar(&ms->tree_full, 0, stop) && wait_bar(&ms->v0_full, 0, stop);
        unsigned char* vt = smem + Sh::OFF_V16;
        // (a warp that gives up here still meets the others below)
#pragma unroll 1
        for (int k = ok ? tid : KT * D / 8; k < KT * D / 8; k += 128) {
          const int vr = k / (D / 8), c = k % (D / 8);
          uint4* v = reinterpret_cast<uint4*>(vt + (c >> 3) * BLK + tile_off(vr, c & 7, 128));
          if (!(there >> vr & 1)) {
            *v = make_uint4(0, 0, 0, 0);
          } else {
            const uint4 x = *v;
            const uint4 y = make_uint4(finite_or_zero(x.x), finite_or_zero(x.y), finite_or_zero(x.z), finite_or_zero(x.w));
            if (x.x != y.x || x.y != y.y || x.z != y.z || x.w != y.w) *v = y, atomicOr(&ms->odd[vr >> 5], 1u << (vr & 31));
          }
        }
        fence_async_smem();
        named_sync(1, 128);  // (and: the ancestor words are there)
        if (!ok) break;
        there &= ms->anc[node];
      }
      // What few tiles need (scores that do not count, the tree's weights as bf16) is rolled up and goes over tensor memory: with it
      // unrolled in registers, the instructions of a tile no longer staying near, wide trees took 136 us and not 125.
      if (__builtin_expect(tree || there != ~0ull, 0)) {
#pragma unroll 1
        for (int c = 0; c < KT; c += 16) {
          float x[16];
          uint32_t y[8];
          tmem_ld16_async(st + c, x);
          tmem_wait_ld16(x);
          const uint32_t bits = (uint32_t)(there >> c);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = bits >> (8 * h + j) & 1 ? __float_as_uint(x[8 * h + j]) : 0xff800000u;
            tmem_st8(st + c + 8 * h, y);
          }
        }
        tmem_wait_st();
#pragma unroll
        for (int c = 0; c < KT; c += 16) tmem_ld16_async(st + c, reinterpret_cast<float(&)[16]>(sv[c]));
#pragma unroll
        for (int c = 0; c < KT; c += 16) tmem_wait_ld16(reinterpret_cast<float(&)[16]>(sv[c]));
      }
      const float by = tree ? a.scale_log2 : qc;
      const float sc[8] = {ks0.x * by, ks0.y * by, ks0.z * by, ks0.w * by, ks1.x * by, ks1.y * by, ks1.z * by, ks1.w * by};
      const float off[8] = {lv0.x, lv0.y, lv0.z, lv0.w, lv1.x, lv1.y, lv1.z, lv1.w};
      float mx = -INFINITY;
#pragma unroll
      for (int g = 0; g < 8; ++g) {
        const float* v = sv + 8 * g;
        const float top = fmaxf(max3f(max3f(v[0], v[1], v[2]), v[3], v[4]), max3f(v[5], v[6], v[7]));
        mx = fmaxf(mx, fmaf(top, sc[g], off[g]));
      }
      if (row >= rows) mx = -INFINITY;
      if (i == 0) m = mx;
      const bool grows = i > 0 && __any_sync(0xffffffffu, mx > m + 8.f);
      if (__builtin_expect(grows, 0)) {  // O is made relative to the new maximum, once the products so far are in it
        // (those of the tile before the last are, since S of this one has taken its P's place)
        ok = wait_bar(&ms->o_done[(i - 1) & 1], ((i - 1) >> 1) & 1, stop);
        if (!ok) break;
        tc_fence_after();
        const float to = mx > m + 8.f ? mx : m, g = to == m ? 1.f : exp2_sfu(m - to);  // (a row's weights do not depend on the other rows)
#pragma unroll 1
        for (int c = 0; c < D; c += 16) {
          float o[16];
          uint32_t u[8];
          tmem_ld16_async(tmem + A_O + lanes + c, o);
          tmem_wait_ld16(o);
#pragma unroll
          for (int half = 0; half < 2; ++half) {
#pragma unroll
            for (int j = 0; j < 8; ++j) u[j] = __float_as_uint(o[8 * half + j] * g);
            tmem_st8(tmem + A_O + lanes + c + 8 * half, u);
          }
        }
        l *= g, m = to;
      }
      const float4 rv0 = *reinterpret_cast<const float4*>(in->rv), rv1 = *reinterpret_cast<const float4*>(in->rv + 4);
      const float rv[8] = {rv0.x, rv0.y, rv0.z, rv0.w, rv1.x, rv1.y, rv1.z, rv1.w};
      const float ref = (m == -INFINITY ? 0.f : m) - kShift;  // minus infinity: a row none of whose keys so far counts
      unsigned long long l2[2] = {pack2(l, 0.f), 0ull};
      uint32_t u[KT / 2];
#pragma unroll
      for (int g = 0; g < 8; ++g) {  // P, and what it adds to the row's sum
        const float b = off[g] - ref, r = rv[g];
        const unsigned long long sc2 = pack2(sc[g], sc[g]), off2 = pack2(b, b), r2 = pack2(r, r);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 e = unpack2(ffma2(pack2(sv[8 * g + 2 * j], sv[8 * g + 2 * j + 1]), sc2, off2));
          const float p0 = exp2_sfu(e.x), p1 = exp2_sfu(e.y);
          l2[j & 1] = ffma2(pack2(p0, p1), r2, l2[j & 1]);
          u[4 * g + j] = pack_f16x2(p0, p1);
        }
      }
      l = pair_sum(l2[0]) + pair_sum(l2[1]);
      if (__builtin_expect(tree, 0)) {  // over S, in columns that have been read
        const float up = 1.f / ms->v0;
#pragma unroll 1
        for (int c = 0; c < KT; c += 16) {
          float x[16];
          uint32_t y[8];
          tmem_ld16_async(st + c, x);
          tmem_wait_ld16(x);
#pragma unroll
          for (int j = 0; j < 8; ++j)
            y[j] = pack_bf16x2(exp2_sfu(fmaf(x[2 * j], by, -ref)) * up, exp2_sfu(fmaf(x[2 * j + 1], by, -ref)) * up);
          tmem_st8(st + c / 2, y);
        }
      } else {
#pragma unroll
        for (int c = 0; c < KT / 2; c += 8) tmem_st8(st + c, reinterpret_cast<const uint32_t(&)[8]>(u[c]));
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&ms->p_full[i & 1]));
    }
    ok = ok && wait_bar(&ms->all_done, 0, stop);
    // a warp that gives up still takes part in the barrier that others may be waiting at
    if (!ok) asm volatile("bar.arrive 1, 128;\n" ::: "memory");
    tc_fence_after();
    if (ok) {
      const unsigned long long odd = has_tree ? (ms->odd[0] | (unsigned long long)ms->odd[1] << 32) & ms->anc[node] : 0ull;
      const long long tok = (long long)s * a.n + node;
      const int head = kvh * a.g + qh;
      const float v0 = ms->v0, inv = v0 / l;
#pragma unroll 1
      for (int c = 0; c < D; c += 16) {
        float o[16];
        __syncwarp();
        tmem_ld16_async(tmem + A_O + lanes + c, o);
        tmem_wait_ld16(o);
#pragma unroll 1
        for (unsigned long long todo = odd; todo; todo &= todo - 1) {  // not finite whatever its weight
          const uint32_t* v = reinterpret_cast<const uint32_t*>(
              a.v + ((long long)s * a.n + __ffsll((long long)todo) - 1) * a.ldv + kvh * D + c);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const uint32_t x = v[j], out = x ^ finite_or_zero(x);
            if (out & 0xffffu) o[2 * j] += bf16_lo(x);
            if (out & 0xffff0000u) o[2 * j + 1] += bf16_hi(x);
          }
        }
        if (row >= rows) {
        } else if (splits == 1) {
          uint32_t u[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) u[j] = pack_bf16x2(o[2 * j] * inv, o[2 * j + 1] * inv);
          uint4* p = reinterpret_cast<uint4*>(a.o + tok * a.ldo + head * D + c);
          p[0] = make_uint4(u[0], u[1], u[2], u[3]), p[1] = make_uint4(u[4], u[5], u[6], u[7]);
        } else {
          float4* p = reinterpret_cast<float4*>(a.part + (((long long)run * a.Hkv + kvh) * rows + row) * D + c);
#pragma unroll
          for (int j = 0; j < 4; ++j) p[j] = make_float4(o[4 * j] * v0, o[4 * j + 1] * v0, o[4 * j + 2] * v0, o[4 * j + 3] * v0);
        }
      }
      if (row < rows && splits > 1) a.part_ml[((long long)run * a.Hkv + kvh) * rows + row] = make_float2(m, l);
    }
  } else if (warp >= 8) {
    split_q(tid - 128);
    fence_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&ms->q_full));
    give_registers<R_CONVERT>();
    // ---- V to fp16: 16 rows of a tile to each of four warps ----
    constexpr int PER = D / 8, STEP = 32 / PER, BATCH = 16 / STEP;  // pieces of 8 values in a row, rows at a time, rows of a lane
    const int piece = lane % PER, first = (warp - 8) * 16 + lane / PER;
    // where a row's piece goes: rows 8 on have the same place in their group of 8
    constexpr int SAME = 8 / STEP;
    uint32_t to[SAME];
#pragma unroll
    for (int b = 0; b < SAME; ++b) to[b] = Sh::OFF_V16 + (piece >> 3) * BLK + tile_off(first + b * STEP, piece & 7, 128);
#pragma unroll 1
    for (int i = has_tree; i < n; ++i) {
      const int use = i - has_tree, unit = use % VU, at = i & 1, k = i >> 1;
      const bool fresh = k == 0 && !(at && has_tree);  // nobody has had this place (of the tree's, S has read K, P . V V)
      bool ok = wait_bar(&ms->info_full[i % INFOS], (i / INFOS) & 1, stop) && wait_bar(&ms->v_full[unit], (use / VU) & 1, stop);
      ok = ok && (fresh || wait_bar(&ms->v16_free[at], (at && has_tree ? k : k - 1) & 1, stop));
      if (!ok) break;
      const unsigned long long mask = ms->info[i % INFOS].mask;
      const unsigned char* src = smem + Sh::OFF_V + unit * Sh::TILE8 + first * D + piece * 8;
      unsigned char* dst = smem + at * Sh::TILE16;
      uint2 x[BATCH];
#pragma unroll
      for (int b = 0; b < BATCH; ++b) x[b] = *reinterpret_cast<const uint2*>(src + b * STEP * D);
      if (__builtin_expect(mask != ~0ull, 0)) {  // (whatever stands where no key is)
#pragma unroll
        for (int b = 0; b < BATCH; ++b)
          if (!(mask >> (first + b * STEP) & 1)) x[b] = make_uint2(0, 0);
      }
#pragma unroll
      for (int b = 0; b < BATCH; ++b)
        *reinterpret_cast<uint4*>(dst + to[b % SAME] + b / SAME * 1024) = make_uint4(
            e4m3x2_f16x2(x[b].x), e4m3x2_f16x2(x[b].x >> 16), e4m3x2_f16x2(x[b].y), e4m3x2_f16x2(x[b].y >> 16));
      fence_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(smem_u32(&ms->v_free[unit]));
        mbar_arrive(smem_u32(&ms->v16_full[at]));
      }
    }
  } else {
    give_registers<R_MMA>();
    if (warp == 4) {
      // ---- copies: lane b the b-th page piece of a tile ----
      const int32_t* table = a.table + (long long)s * a.max_pages;
      const int shift = min(a.page_shift, 6), box = 1 << shift, pieces = KT >> shift, pmask = (1 << a.page_shift) - 1;
      auto lookup = [&](int ti) {  // the piece's page; -1: no such row; -2: out of range
        const int at = ti * KT + lane * box;
        if (lane >= pieces || ti >= ct || at >= len) return -1;
        const int pg = table[at >> a.page_shift];
        return pg < 0 || pg >= a.n_pages ? -2 : pg;
      };
      int k_issued = 0, v_issued = 0, pg = lookup(i0 + has_tree - 1);
      if (has_tree) {  // the tree's V and K, in the places of the first two fp16 tiles
        const uint32_t full = smem_u32(&ms->tree_full);
        if (lane == 0) mbar_arrive_expect_tx(full, 2 * Sh::TILE16);
        __syncwarp();
        if (lane < 2 * DB)
          tma_load_2d(sb + Sh::OFF_V16 + lane * BLK, lane < DB ? &tvt : &tkt, kvh * D + lane % DB * 64, s * a.n, full);
      }
#pragma unroll 1
      for (int i = has_tree; i < n; ++i) {
        const int ti = i0 + i - 1, use = i - has_tree, mine = pg;
        pg = lookup(ti + 1);
        if (__any_sync(0xffffffffu, mine == -2) && lane == 0) flag(a.status, SSM_STATUS_SEQ_RANGE);
        const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, mine >= 0)) * box * D;
        const int crd = ((mine * a.Hkv + kvh) << a.page_shift) + ((ti * KT + lane * box) & pmask);
        if (use >= KU && !wait_bar(&ms->k_free[use % KU], (use / KU - 1) & 1, stop)) break;
        uint32_t full = smem_u32(&ms->k_full[use % KU]);
        if (lane == 0) mbar_arrive_expect_tx(full, bytes);
        __syncwarp();
        if (mine >= 0) tma_load_2d(sb + Sh::OFF_K + use % KU * Sh::TILE8 + lane * box * D, &tkp, 0, crd, full);
        k_issued = use + 1;
        if (use >= VU && !wait_bar(&ms->v_free[use % VU], (use / VU - 1) & 1, stop)) break;
        full = smem_u32(&ms->v_full[use % VU]);
        if (lane == 0) mbar_arrive_expect_tx(full, bytes);
        __syncwarp();
        if (mine >= 0)
          bulk_load(sb + Sh::OFF_V + use % VU * Sh::TILE8 + lane * box * D, f.vp + (long long)crd * D, box * D, full);
        v_issued = use + 1;
      }
      // copies land before the shared memory is given up, whoever gives up, and when (else they have, by the time of the last tile)
      if (lane == 0) {
        if (has_tree) mbar_wait(smem_u32(&ms->tree_full), 0);
        for (int k = max(0, k_issued - KU); k < k_issued; ++k) mbar_wait(smem_u32(&ms->k_full[k % KU]), (k / KU) & 1);
        for (int k = max(0, v_issued - VU); k < v_issued; ++k) mbar_wait(smem_u32(&ms->v_full[k % VU]), (k / VU) & 1);
      }
    } else if (warp == 7) {
      // ---- what a tile's keys are.  Lane 8 j + g has the scales of the g-th 8 keys of tile j of four: they are asked for four tiles
      // ahead, their pages eight (a load that misses the caches takes longer than a tile) ----
      const int32_t* table = a.table + (long long)s * a.max_pages;
      const int grp = lane & 7, t0 = i0 + has_tree - 1, count = n - has_tree, pmask = (1 << a.page_shift) - 1;
      auto page_of = [&](int c) {  // of the lane's keys in the c-th four tiles; -1: no such rows, or their page is out of range
        const int ti = t0 + 4 * c + (lane >> 3), at = ti * KT + grp * 8;
        if (4 * c + (lane >> 3) >= count || at >= len) return -1;
        const int pg = table[at >> a.page_shift];
        return pg < 0 || pg >= a.n_pages ? -1 : pg;
      };
      auto scales_of = [&](int c, int pg) {
        if (pg < 0) return make_float2(1.f, 1.f);
        const int ti = t0 + 4 * c + (lane >> 3);
        const long long at = ((((long long)pg * a.Hkv + kvh) << a.page_shift) + ((ti * KT + grp * 8) & pmask)) >> f.block_shift;
        return make_float2(f.ks[at], f.vs[at]);
      };
      int pg = page_of(0);
      int pg1 = page_of(1);
      float2 sc = scales_of(0, pg);
      if (has_tree) {
        TileInfo* in = &ms->info[0];
        if (lane < 8) in->ks[lane] = 1.f, in->lv[lane] = 0.f, in->rv[lane] = 1.f;
        if (lane == 0) in->mask = a.n < 64 ? (1ull << a.n) - 1 : ~0ull;
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ms->info_full[0]));
      }
      // What scales of v are relative to, a power of two: the largest of the first tile; beside the tree the least of the first four,
      // within 2^60 of 1 (so that what the tree's rows of v add stays in fp32 beside a cache of zeros, whose scale is 2^-100)
      float v0;
      {
        const bool there = pg >= 0 && good_scale(sc.x) && good_scale(sc.y);
        const unsigned int e = __float_as_uint(sc.y) & 0x7f800000u, of = __ballot_sync(0xffffffffu, there) & (has_tree ? ~0u : 0xffu);
        const bool counts = of >> lane & 1;
        const unsigned int least = __reduce_min_sync(0xffffffffu, counts ? e : 0x7f800000u);
        const unsigned int top = __reduce_max_sync(0xffffffffu, counts ? e : 0u);
        v0 = of == 0 ? 1.f : has_tree ? fminf(fmaxf(__uint_as_float(least), 0x1p-60f), 0x1p60f) : __uint_as_float(top);
        if (lane == 0) ms->v0 = v0;
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ms->v0_full));  // (others see it with the first tile's info)
      }
      bool ok = true;
#pragma unroll 1
      for (int c = 0; 4 * c < count && ok; ++c) {
        const float2 next = scales_of(c + 1, pg1);
        const int pg2 = page_of(c + 2);
        const bool good = good_scale(sc.x) && good_scale(sc.y);
        if (__any_sync(0xffffffffu, pg >= 0 && !good) && lane == 0) flag(a.status, SSM_STATUS_SCALE);
        const bool there = pg >= 0 && good;
        if (!there) sc = make_float2(1.f, 1.f);
        const int left = min(max(len - (t0 + 4 * c + (lane >> 3)) * KT - 8 * grp, 0), 8);
        const unsigned long long keys = there ? (unsigned long long)((1u << left) - 1) << 8 * grp : 0ull;
        const float rel = fminf(fmaxf(sc.y / v0, 0x1p-120f), 0x1p120f), lv = log2f(rel), rv = 1.f / rel;
#pragma unroll 1
        for (int j = 0; j < 4 && 4 * c + j < count; ++j) {
          const int use = 4 * c + j, i = use + has_tree;
          const bool mine = lane >> 3 == j;
          const unsigned long long mask = (unsigned long long)__reduce_or_sync(0xffffffffu, mine ? (uint32_t)(keys >> 32) : 0u) << 32 |
                                          __reduce_or_sync(0xffffffffu, mine ? (uint32_t)keys : 0u);
          // (a place among the infos is free by the time that the tile's V is there)
          ok = wait_bar(&ms->v_full[use % VU], (use / VU) & 1, stop);
          if (!ok) break;
          TileInfo* in = &ms->info[i % INFOS];
          if (mine) in->ks[grp] = fmaxf(sc.x, 0x1p-66f), in->lv[grp] = lv, in->rv[grp] = rv;
          if (lane == 0) in->mask = mask;
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&ms->info_full[i % INFOS]));
        }
        pg = pg1, pg1 = pg2, sc = next;
      }
    } else {
      // ---- MMAs: one warp those of S, the other P . V, each behind its own waits ----
      const bool leader = elect_one();
      bool ok = true;
      if (warp == 5) {
        constexpr uint32_t id8 = (1u << 4) | (uint32_t)(KT >> 3) << 17 | (128u >> 4) << 24;  // e4m3 x e4m3 -> fp32
        constexpr uint32_t id_t = idesc_major(128, KT, false, false);
        ok = wait_bar(&ms->q_full, 0, stop);
#pragma unroll 1
        for (int i = 0; i < n && ok; ++i) {
          const bool tree = has_tree && i == 0;
          const int use = i - has_tree, unit = use % KU;
          const uint32_t st = tmem + A_S + (i & 1) * KT;
          ok = tree ? wait_bar(&ms->tree_full, 0, stop) : wait_bar(&ms->k_full[unit], (use / KU) & 1, stop);
          ok = ok && wait_bar(&ms->info_full[i % INFOS], (i / INFOS) & 1, stop);
          ok = ok && (i < 2 || wait_bar(&ms->o_done[i & 1], ((i >> 1) - 1) & 1, stop));  // P . V has read the P that stands there
          if (!ok) break;
          tc_fence_after();
          if (leader) {
            mbar_arrive(smem_u32(&ms->s_full[i & 1]));  // (who sees S then sees the tile's info too)
            if (tree) {
              const uint32_t kd = desc_lo(sb + Sh::OFF_V16 + Sh::TILE16, 16);
#pragma unroll
              for (int k = 0; k < D / 16; ++k)
                mma_ts<id_t>(st, tmem + A_O + k * 8, kd + (((k >> 2) * BLK + (k & 3) * 32) >> 4), k > 0);
              mma_commit(smem_u32(&ms->s_full[i & 1]));
              mma_commit(smem_u32(&ms->v16_free[1]));
            } else {
              const uint32_t qd = desc_lo(sb, 16), kd = desc_lo(sb + Sh::OFF_K + unit * Sh::TILE8, 16);
#pragma unroll
              for (int t = 0; t < 2; ++t)  // Q's upper terms, its lower terms
#pragma unroll
                for (int k = 0; k < D / 32; ++k) mma8_ss<id8, Sh::DESC_HI>(st, qd + t * (128 * D >> 4) + k * 2, kd + k * 2, t + k > 0);
              mma_commit(smem_u32(&ms->s_full[i & 1]));
              mma_commit(smem_u32(&ms->k_free[unit]));
            }
          }
          __syncwarp();
        }
      } else {
        constexpr uint32_t id_o = idesc_f16(128, D, true), id_t = idesc_major(128, D, false, true);
#pragma unroll 1
        for (int i = 0; i < n && ok; ++i) {
          const bool tree = has_tree && i == 0;
          const int at = i & 1;
          const uint32_t st = tmem + A_S + at * KT;
          ok = tree ? wait_bar(&ms->tree_full, 0, stop)
                    : wait_bar(&ms->v16_full[at], ((i >> 1) - (at == 0 ? has_tree : 0)) & 1, stop);
          ok = ok && wait_bar(&ms->p_full[at], (i >> 1) & 1, stop);
          if (!ok) break;
          tc_fence_after();
          if (leader) {
            const uint32_t vd = desc_lo(sb + Sh::OFF_V16 + at * Sh::TILE16, BLK);
#pragma unroll
            for (int k = 0; k < KT / 16; ++k) {  // 16 keys: two groups of 8 rows
              if (tree)
                mma_ts<id_t>(tmem + A_O, st + k * 8, vd + k * (2048 >> 4), k > 0);
              else
                mma_ts<id_o>(tmem + A_O, st + k * 8, vd + k * (2048 >> 4), i + k > 0);
            }
            mma_commit(smem_u32(&ms->o_done[at]));
            mma_commit(smem_u32(&ms->v16_free[at]));
            if (i + 1 == n) mma_commit(smem_u32(&ms->all_done));
          }
          __syncwarp();
        }
      }
      if (leader) {
        mma_commit(smem_u32(&ms->drain[warp - 5]));
        mbar_poll_ns(smem_u32(&ms->drain[warp - 5]), 0, kWaitLimitNs);
      }
      __syncwarp();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && *stop) flag(a.status, SSM_STATUS_TIMEOUT);
  if (warp == 5) {
    __syncwarp();
    tc_fence_after();
    tmem_free_warp(tmem, A_COLS);
  }
}

template <int D>
cudaError_t run_attend8(const AttendFp8Args& f, const AttendPlan& p, cudaStream_t s) {
  using Sh = Attend8Smem<D>;
  const AttendArgs& a = f.a;
  CUtensorMap m[3];
  const long long page_rows = ((long long)a.n_pages * a.Hkv) << a.page_shift, cols = (long long)a.Hkv * D;
  const int box = a.page_shift < 6 ? 1 << a.page_shift : KT;
  // a call without cached rows reads no page: any matrix will do
  const bool none = a.max_len == 0 || page_rows == 0;
  if (!encode_byte_tiles(&m[0], none ? static_cast<const void*>(a.k) : f.kp, none ? 1 : page_rows, D, box) ||
      !encode_tiles(&m[1], a.k, (long long)a.S * a.n, cols, a.ldk, KT) ||
      !encode_tiles(&m[2], a.v, (long long)a.S * a.n, cols, a.ldv, KT))
    return cudaErrorInvalidValue;
  static bool done[64];
  cudaError_t e = allow_smem(attend8_kernel<D>, Sh::BYTES, done);
  if (e != cudaSuccess) return e;
  e = launch_early(attend8_kernel<D>, dim3((unsigned)((p.max_runs ? p.max_runs : a.S) * p.row_tiles), (unsigned)a.Hkv), A8THREADS,
                   Sh::BYTES, s, m[0], m[1], m[2], f);
  return e != cudaSuccess || p.max_runs == 0 ? e : launch_attend_join(a, s);
}
static_assert(2 * 2 * kSMs * 4 <= 2 * Attend8Smem<64>::TILE16, "the lengths stand in the space of V");

// Commit.  A cluster of 8 CTAs for each sequence, a warp for each block of tokens of a layer, head and K or V: the largest of its new
// rows gives the scale that they need, the block takes that or its own, rows that it holds are rounded again if it grew.  The
// sequence's length is written by one of the CTAs once all eight have read it, so len_out may be cache_len.  Bound by latency:
// 4.3 us for one sequence's path of 5 in 4 layers of 8 heads of 128 (in a CUDA graph; its bytes 0.02), 9.2 for 32 sequences' in 8 layers
// (7.6 where L2 holds the pages).
constexpr int CCTAS = 8, CTHREADS = 512;

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
          using Held = typename std::conditional<W == 2, uint32_t, uint16_t>::type;
#pragma unroll 1
          for (int r0 = 0; r0 < held; r0 += 8) {  // (eight rows under way: a block may hold a thousand)
            Held y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (r0 + i < held) y[i] = *reinterpret_cast<const Held*>(page + (r0 + i) * D);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              if (r0 + i >= held) break;
              const float2 lo = f16x2_f32(e4m3x2_f16x2(y[i]));
              uint32_t to = f32_e4m3x2(lo.x * by, lo.y * by);
              if constexpr (W == 2) {
                const float2 hi = f16x2_f32(e4m3x2_f16x2(y[i] >> 16));
                to |= f32_e4m3x2(hi.x * by, hi.y * by) << 16;
              }
              *reinterpret_cast<Held*>(page + (r0 + i) * D) = (Held)to;
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

// The plan of the 16-bit kernel; but few rows, whose blocks are half as large, are not cut either where their blocks fill half of the
// SMs' places and no cache is so long that one block's walk of it takes more than cutting: 64 tokens of 8 heads over up to 1000 rows
// 21 us, cut 32, over up to 400 rows 11 and 21.
AttendPlan plan_attend_fp8(int S, int n, int Hq, int Hkv, int max_len) {
  AttendPlan p = plan_attend(S, n, Hq, Hkv, max_len);
  if (n * (Hq / Hkv) <= kFewRows && S * Hkv >= 2 * kSMs && max_len <= 2048) p.max_runs = 0;
  return p;
}

}  // namespace

size_t tree_attention_fp8_workspace_bytes(int S, int n, int Hq, int Hkv, int D, int max_len) {
  return attend_workspace_bytes(plan_attend_fp8(S, n, Hq, Hkv, max_len), S, n, Hq, Hkv, D);
}

cudaError_t launch_tree_attention_fp8(const AttendFp8Args& args, void* workspace, cudaStream_t s) {
  if (args.a.S == 0) return cudaSuccess;
  AttendFp8Args f = args;
  const AttendPlan p = plan_attend_fp8(f.a.S, f.a.n, f.a.Hq, f.a.Hkv, f.a.max_len);
  lay_workspace(f.a, p, workspace);
  if (f.a.n * f.a.g <= kFewRows) return launch_few_attention_fp8(f, p.max_runs, s);
  return f.a.D == 64 ? run_attend8<64>(f, p, s) : run_attend8<128>(f, p, s);
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
