// Attention of a draft tree's nodes over a paged cache and their ancestors, and the commit of the accepted
// path into the cache (ssm_attention.h).
//
// attend_kernel.  The query rows of one key/value head -- n nodes x g query heads -- share its keys, so a CTA takes up to
// 128 of them (the rows of tensor memory) and walks tiles of 64 keys once, on tcgen05:
//     S [128 x 64] = Q . K^T,   P = 2^(S - m),   O [128 x D] += P . V        (P, O in tensor memory, V read MN-major)
// with the running maximum m and sum of each row's softmax in the row's thread.  O is rescaled only when a maximum has
// grown by more than 2^8 (P then stays below 2^8, and its rounding to bf16 is relative).  One warp copies, one issues the MMAs
// of S, one those of P . V, four do the softmax: S of the next tile is made while the softmax of this one runs, and two CTAs
// to an SM overlap the rest (one CTA with two such streams took 15 to 25 % longer on 320 rows: nothing covered its start and
// its end).  K and V tiles come by TMA from their pages, through a ring.  With S's operands both in shared memory that is
// what binds wide trees (a tile: 384 cycles of reads for S, 128 for P . V, 256 of writes, against 512 of products), so half
// of Q stands in tensor memory, as much as there is room for.
// One tile more than the cache has holds the tree's own rows; there a row keeps its node's ancestors only, read from a
// 64-bit word per node.  Few rows share a tile (n g operations for each byte of the cache), so the keys are split over the
// SMs where the (sequence, head, row tile) triples do not fill them; the partial sums are then joined by combine_kernel.
// Rounding: P to bf16 for the tensor cores, once; the row's sum is that of the unrounded P, in fp32.
// Rows of V that no key of the tile owns, and values of V in tree rows that are not finite, are zeroed in shared memory
// (a weight of 0 would spread them); the latter are added to the rows that see them at the end.
// Measured, both kernels, back to back in a graph (32 query heads, D = 128): one token of one sequence over 16411 rows, 8 heads
// of K and V, 22.6 us (67 MB: 3.0 TB/s; 18 where L2 holds the cache; latency: seven tiles to a CTA); 8 trees of 16 nodes over up
// to 8117 rows 41 us (163 MB: 4.0 TB/s of HBM); 4 trees of 40 nodes over up to 40009 rows, 4 heads, 86 us (85 GFLOP: 0.99 PFLOP/s, 1.19 with the rows
// that fill up the third row tile; tensor pipe 52 % of the time, shared memory the rest).  D = 64, the same rows: 16, 28 and 73 us.
#include "attend.cuh"

namespace ssmtree {
namespace {

constexpr int ATHREADS = 224;   // 4 softmax warps, one for copies, two for MMAs
constexpr int UNITS = 6;        // tiles of K and V, by turns, in the ring: what lets two CTAs share an SM's memory
constexpr int BLK = KT * 128;   // 64 rows x 64 columns of bf16

constexpr int A_S = 0, A_P = 64, A_Q = 96, A_O = 128, A_COLS = 256;  // tensor memory columns: S, P, Q's first 64 columns, O

template <int D>
struct AttendSmem {
  static constexpr int OFF_KV = (D / 64 - 1) * 2 * BLK;      // after Q's other columns: 128 rows of 64
  static constexpr int TILE = (D / 64) * BLK;                // K or V of a tile
  static constexpr int OFF_MISC = OFF_KV + UNITS * TILE;
  static constexpr int BYTES = OFF_MISC + 832;
  static_assert(BYTES <= 228 * 1024 / 2 - 1024, "two to an SM");
};
struct AttendMisc {
  unsigned long long anc[64];  // ancestors and self of each node
  unsigned long long full[UNITS], free_[UNITS], q_full, s_full, s_free, p_full, o_done, drain[2];
  unsigned int odd[2];         // tree rows with a value of v that is not finite
  uint32_t tmem;
  int stop;
  int no_page[8];              // whether a page of tile i (at i % 8) is out of range
  SplitScratch split;
};
static_assert(sizeof(AttendMisc) <= 832, "space");

template <int D>
__global__ void __launch_bounds__(ATHREADS, 2)
    attend_kernel(const __grid_constant__ CUtensorMap tkp, const __grid_constant__ CUtensorMap tvp,
                  const __grid_constant__ CUtensorMap tkt, const __grid_constant__ CUtensorMap tvt, AttendArgs a) {
  using Sh = AttendSmem<D>;
  constexpr int DB = D / 64;  // 64-column blocks
  extern __shared__ __align__(1024) unsigned char smem[];  // (there is no room to move it: where it is not aligned, nothing runs)
  const uint32_t sb = smem_u32(smem);
  AttendMisc* ms = reinterpret_cast<AttendMisc*>(smem + Sh::OFF_MISC);
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
    for (int i = 0; i < UNITS; ++i) {
      mbar_init(smem_u32(&ms->full[i]), 1);
      mbar_init(smem_u32(&ms->free_[i]), 1);
    }
    mbar_init(smem_u32(&ms->q_full), 4);
    mbar_init(smem_u32(&ms->s_full), 1);
    mbar_init(smem_u32(&ms->s_free), 4);
    mbar_init(smem_u32(&ms->p_full), 4);
    mbar_init(smem_u32(&ms->o_done), 1);
    mbar_init(smem_u32(&ms->drain[0]), 1);
    mbar_init(smem_u32(&ms->drain[1]), 1);
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
    int* tiles = reinterpret_cast<int*>(smem);  // space not in use yet: with D = 64 a place of the ring
    int first;
    tps = choose_split<ATHREADS>(a, a.Hkv * rt, tiles, &ms->split);
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
  const int ct = (len + KT - 1) / KT;  // tiles of the cache; one more is the tree's
  const int i0 = sp * tps, n = min(ct + 1 - i0, tps);
  const bool has_tree = i0 + n == ct + 1;

  if (warp < 4) {
    const int row = r0 + tid;  // this thread's
    const int node = row < rows ? row / a.g : 0, qh = row < rows ? row % a.g : 0;
    const uint32_t lanes = (uint32_t)(warp * 32) << 16;
    {  // q (zero beyond the last row): 64 columns in tensor memory, others in shared memory
      const uint4* q = reinterpret_cast<const uint4*>(a.q + ((long long)s * a.n + node) * a.ldq + (kvh * a.g + qh) * D);
      const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int c = 0; c < 8; c += 2) {
        const uint4 x = row < rows ? q[c] : zero, y = row < rows ? q[c + 1] : zero;
        const uint32_t u[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
        tmem_st8(tmem + A_Q + lanes + 4 * c, u);
      }
#pragma unroll
      for (int c = 8; c < D / 8; ++c)
        *reinterpret_cast<uint4*>(smem + ((c >> 3) - 1) * 2 * BLK + tile_off(tid, c & 7, 128)) = row < rows ? q[c] : zero;
      tmem_wait_st();
      tc_fence_before();
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&ms->q_full));
    }
    if (has_tree && warp == 0) ancestor_words(a, s, ms->anc, kvh == 0 && r0 == 0);

    float m = -INFINITY, l = 0.f;
    bool ok = true;
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      const int ti = i0 + i;
      const bool tree = ti == ct;
      const int left = tree ? a.n : len - ti * KT;
      ok = wait_bar(&ms->s_full, i & 1, stop);
      if (!ok) break;
      tc_fence_after();
      float sv[KT];
#pragma unroll
      for (int c = 0; c < KT; c += 16) tmem_ld16_async(tmem + A_S + lanes + c, reinterpret_cast<float(&)[16]>(sv[c]));
#pragma unroll
      for (int c = 0; c < KT; c += 16) tmem_wait_ld16(reinterpret_cast<float(&)[16]>(sv[c]));
      const bool no_page = *(volatile int*)&ms->no_page[i & 7];  // (read before s_free: the copies are three tiles on at most)
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&ms->s_free));
      if (tree || left < KT || no_page) {  // masks, and rows of V that are not to be multiplied
        const int32_t* table = a.table + (long long)s * a.max_pages;
        unsigned long long rowsv = left < KT ? (1ull << left) - 1 : ~0ull;  // the tile's rows that there are
        if (!tree && no_page) {
#pragma unroll 1
          for (int k = 0; k < min(left, KT); ++k) {
            const int pg = table[(ti * KT + k) >> a.page_shift];
            if (pg < 0 || pg >= a.n_pages) rowsv &= ~(1ull << k);
          }
        }
        const int use = 2 * i + 1;
        // (a warp that gives up here still meets the others below: they may be through this wait, and through the next tile's
        // before the products that they then wait for fail to come)
        ok = wait_bar(&ms->full[use % UNITS], (use / UNITS) & 1, stop);
        unsigned char* vt = smem + Sh::OFF_KV + use % UNITS * Sh::TILE;
#pragma unroll 1
        for (int k = ok ? tid : KT * D / 8; k < KT * D / 8; k += 128) {
          const int vr = k / (D / 8), c = k % (D / 8);
          uint4* v = reinterpret_cast<uint4*>(vt + (c >> 3) * BLK + tile_off(vr, c & 7, 128));
          if (!(rowsv >> vr & 1)) {
            *v = make_uint4(0, 0, 0, 0);
          } else if (tree) {
            const uint4 x = *v;
            const uint4 y = make_uint4(finite_or_zero(x.x), finite_or_zero(x.y), finite_or_zero(x.z), finite_or_zero(x.w));
            if (x.x != y.x || x.y != y.y || x.z != y.z || x.w != y.w) *v = y, atomicOr(&ms->odd[vr >> 5], 1u << (vr & 31));
          }
        }
        fence_async_smem();
        named_sync(1, 128);  // (and: the ancestor words are there)
        if (!ok) break;
        if (tree) rowsv &= ms->anc[node];
#pragma unroll
        for (int j = 0; j < KT; ++j)
          if (!((j < 32 ? (uint32_t)rowsv : (uint32_t)(rowsv >> 32)) >> (j & 31) & 1)) sv[j] = -INFINITY;
      }
      float mx = fmaxf(sv[0], sv[1]), my = fmaxf(sv[2], sv[3]);
#pragma unroll
      for (int j = 4; j < KT; j += 4) mx = max3f(mx, sv[j], sv[j + 1]), my = max3f(my, sv[j + 2], sv[j + 3]);
      mx = fmaxf(mx, my) * a.scale_log2;
      if (i == 0) {
        m = mx;
      } else {  // P . V of the last tile has read its P
        ok = wait_bar(&ms->o_done, (i - 1) & 1, stop);
        if (!ok) break;
        tc_fence_after();
      }
      if (i > 0 && __any_sync(0xffffffffu, mx > m + 8.f)) {
        const float to = mx > m + 8.f ? mx : m, f = to == m ? 1.f : exp2_sfu(m - to);  // (a row's weights do not depend on the other rows)
#pragma unroll 1
        for (int c = 0; c < D; c += 16) {
          float o[16];
          uint32_t u[8];
          tmem_ld16_async(tmem + A_O + lanes + c, o);
          tmem_wait_ld16(o);
#pragma unroll
          for (int half = 0; half < 2; ++half) {
#pragma unroll
            for (int j = 0; j < 8; ++j) u[j] = __float_as_uint(o[8 * half + j] * f);
            tmem_st8(tmem + A_O + lanes + c + 8 * half, u);
          }
        }
        l *= f, m = to;
      }
      const float ref = m == -INFINITY ? 0.f : m;  // a row none of whose keys so far counts
      const unsigned long long sc2 = pack2(a.scale_log2, a.scale_log2), ref2 = pack2(-ref, -ref);
      unsigned long long sum2[2] = {0ull, 0ull};
      const unsigned long long one2 = pack2(1.f, 1.f);
      const uint32_t pt = tmem + A_P + lanes;
#pragma unroll
      for (int c = 0; c < KT; c += 16) {
        uint32_t u[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float2 e = unpack2(ffma2(pack2(sv[c + 2 * j], sv[c + 2 * j + 1]), sc2, ref2));
          const float p0 = exp2_sfu(e.x), p1 = exp2_sfu(e.y);
          sum2[j & 1] = ffma2(one2, pack2(p0, p1), sum2[j & 1]);
          u[j] = pack_bf16x2(p0, p1);
        }
        tmem_st8(pt + c / 2, u);
      }
      l += pair_sum(sum2[0]) + pair_sum(sum2[1]);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&ms->p_full));
    }
    ok = ok && wait_bar(&ms->o_done, (n - 1) & 1, stop);
    // a warp that gives up still takes part in the barrier that others may be waiting at
    if (!ok) asm volatile("bar.arrive 1, 128;\n" ::: "memory");
    tc_fence_after();
    if (ok) {
      const unsigned long long odd = has_tree ? (ms->odd[0] | (unsigned long long)ms->odd[1] << 32) & ms->anc[node] : 0ull;
      const long long tok = (long long)s * a.n + node;
      const int head = kvh * a.g + qh;
      const float inv = 1.f / l;
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
          for (int j = 0; j < 4; ++j) p[j] = make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
        }
      }
      if (row < rows && splits > 1) a.part_ml[((long long)run * a.Hkv + kvh) * rows + row] = make_float2(m, l);
    }
  } else if (warp == 4) {
    // ---- copies: lane b the b-th page piece of a tile ----
    const int32_t* table = a.table + (long long)s * a.max_pages;
    const int shift = min(a.page_shift, 6), box = 1 << shift, pieces = KT >> shift, pmask = (1 << a.page_shift) - 1;
    auto lookup = [&](int ti) {  // the piece's page; -1: no such row; -2: out of range
      const int at = ti * KT + lane * box;
      if (lane >= pieces || ti >= ct || at >= len) return -1;
      const int pg = table[at >> a.page_shift];
      return pg < 0 || pg >= a.n_pages ? -2 : pg;
    };
    int issued = 0, pg = lookup(i0);
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      const int ti = i0 + i, mine = pg;
      pg = lookup(ti + 1);
      const bool bad = __any_sync(0xffffffffu, mine == -2);
      if (bad && lane == 0) flag(a.status, SSM_STATUS_SEQ_RANGE);
      const bool tree = ti == ct;
      const uint32_t bytes = (tree ? KT : __popc(__ballot_sync(0xffffffffu, mine >= 0)) * box) * D * 2;
      const int crd = ((mine * a.Hkv + kvh) << a.page_shift) + ((ti * KT + lane * box) & pmask);
      bool ok = true;
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const int use = 2 * i + kv, unit = use % UNITS;
        const uint32_t full = smem_u32(&ms->full[unit]), dst = sb + Sh::OFF_KV + unit * Sh::TILE;
        if (use >= UNITS) ok = ok && wait_bar(&ms->free_[unit], (use / UNITS - 1) & 1, stop);
        if (!ok) break;
        if (kv == 0 && lane == 0) *(volatile int*)&ms->no_page[i & 7] = bad;
        if (lane == 0) mbar_arrive_expect_tx(full, bytes);
        __syncwarp();
        if (tree) {
          if (lane < DB) tma_load_2d(dst + lane * BLK, kv ? &tvt : &tkt, kvh * D + lane * 64, s * a.n, full);
        } else if (mine >= 0) {
#pragma unroll
          for (int c = 0; c < DB; ++c) tma_load_2d(dst + c * BLK + lane * box * 128, kv ? &tvp : &tkp, c * 64, crd, full);
        }
        issued = use + 1;
      }
      if (!ok) break;
    }
    // copies land before the shared memory is given up, whoever gives up, and when (else they have, by the time of the last tile)
    for (int k = max(0, issued - UNITS); k < issued && lane == 0; ++k) mbar_wait(smem_u32(&ms->full[k % UNITS]), (k / UNITS) & 1);
  } else {
    // ---- MMAs: one warp those of S, the other P . V, each behind its own waits ----
    const bool leader = elect_one();
    bool ok = true;
    if (warp == 5) {
      constexpr uint32_t id_s = idesc_major(128, KT, false, false);
      ok = wait_bar(&ms->q_full, 0, stop);
#pragma unroll 1
      for (int i = 0; i < n && ok; ++i) {
        const int use = 2 * i, unit = use % UNITS;
        ok = wait_bar(&ms->full[unit], (use / UNITS) & 1, stop) && (i == 0 || wait_bar(&ms->s_free, (i - 1) & 1, stop));
        if (!ok) break;
        tc_fence_after();
        if (leader) {
          const uint32_t qd = desc_lo(sb, 16), kd = desc_lo(sb + Sh::OFF_KV + unit * Sh::TILE, 16);
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t kk = kd + (((k >> 2) * BLK + (k & 3) * 32) >> 4);
            if (k < 4)
              mma_ts<id_s>(tmem + A_S, tmem + A_Q + k * 8, kk, k > 0);
            else
              mma_ss<id_s>(tmem + A_S, qd + ((((k >> 2) - 1) * 2 * BLK + (k & 3) * 32) >> 4), kk, true);
          }
          mma_commit(smem_u32(&ms->s_full));
          mma_commit(smem_u32(&ms->free_[unit]));
        }
        __syncwarp();
      }
    } else {
      constexpr uint32_t id_o = idesc_major(128, D, false, true);
#pragma unroll 1
      for (int i = 0; i < n && ok; ++i) {
        const int use = 2 * i + 1, unit = use % UNITS;
        ok = wait_bar(&ms->full[unit], (use / UNITS) & 1, stop) && wait_bar(&ms->p_full, i & 1, stop);
        if (!ok) break;
        tc_fence_after();
        if (leader) {
          const uint32_t vd = desc_lo(sb + Sh::OFF_KV + unit * Sh::TILE, BLK);
#pragma unroll
          for (int k = 0; k < KT / 16; ++k)  // 16 keys: two groups of 8 rows
            mma_ts<id_o>(tmem + A_O, tmem + A_P + k * 8, vd + k * (2048 >> 4), i + k > 0);
          mma_commit(smem_u32(&ms->o_done));
          mma_commit(smem_u32(&ms->free_[unit]));
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
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && *stop) flag(a.status, SSM_STATUS_TIMEOUT);
  if (warp == 5) {
    __syncwarp();
    tc_fence_after();
    tmem_free_warp(tmem, A_COLS);
  }
}

// o = sum over the splits of 2^(m_i - m) o_i / sum of 2^(m_i - m) l_i; W warps to a query row, each a part of its splits, D / 32
// columns a lane
template <int D, int W>
__global__ void __launch_bounds__(128) combine_kernel(AttendArgs a) {
  constexpr int V = D / 32;
  __shared__ float part_s[W > 1 ? 4 : 1][W > 1 ? D + 1 : 1];
  launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, w = warp % W;
  const long long row = (long long)blockIdx.x * (4 / W) + warp / W;  // (s, node, head)
  grid_dependency_wait();
  if (row >= (long long)a.S * a.n * a.Hq) return;  // W = 4: the whole block
  const long long tok = row / a.Hq;
  const int head = (int)(row % a.Hq), s = (int)(tok / a.n), g = a.g, rows = a.n * g, kvh = head / g;
  const int2 run = a.runs[s];  // its first, and how many
  const int ns = run.y;
  if (ns == 1) return;  // written already
  const long long step = (long long)a.Hkv * rows;  // between a row's partial sums
  const long long at = run.x * step + (long long)kvh * rows + (int)(tok % a.n) * g + head % g;
  const float2* ml = a.part_ml + at;
  // two splits a lane: there are 64 at most
  const float2 none = make_float2(-INFINITY, 0.f);
  const float2 e0 = lane < ns ? ml[lane * step] : none, e1 = lane + 32 < ns ? ml[(lane + 32) * step] : none;
  float mx = fmaxf(e0.x, e1.x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  const float ref = mx == -INFINITY ? 0.f : mx;
  const float f0 = exp2_sfu(e0.x - ref), f1 = exp2_sfu(e1.x - ref);
  const float sum = warp_sum(fmaf(f0, e0.y, f1 * e1.y));
  float acc[V] = {};
  const float* p = a.part + at * D + lane * V;
#pragma unroll 8
  for (int i = w; i < ns; i += W) {
    const float f = __shfl_sync(0xffffffffu, i < 32 ? f0 : f1, i & 31);
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] = fmaf(f, p[i * step * D + v], acc[v]);
  }
  if (W > 1) {
#pragma unroll
    for (int v = 0; v < V; ++v) part_s[warp][lane * V + v] = acc[v];
    __syncthreads();
    if (w > 0) return;
#pragma unroll
    for (int k = 1; k < W; ++k)
#pragma unroll
      for (int v = 0; v < V; ++v) acc[v] += part_s[warp + k][lane * V + v];
  }
  const float inv = 1.f / sum;
  uint16_t* o = a.o + tok * a.ldo + head * D + lane * V;
#pragma unroll
  for (int v = 0; v < V; v += 2) *reinterpret_cast<uint32_t*>(o + v) = pack_bf16x2(acc[v] * inv, acc[v + 1] * inv);
}

static_assert(2 * 2 * kSMs * 4 <= 6 * 64 * 64 * 2, "the lengths stand in the ring's space");

template <int D>
cudaError_t join_runs(const AttendArgs& a, cudaStream_t s) {
  const long long out_rows = (long long)a.S * a.n * a.Hq;
  // four warps to a row where there are many runs: 38 runs 22.3 us a call with one warp, 18.4 with four; 7 runs 87 and 90
  const bool wide = a.max_runs >= 8 * a.S;
  const dim3 grid((unsigned)(wide ? out_rows : (out_rows + 3) / 4));
  return wide ? launch_early(combine_kernel<D, 4>, grid, 128, 0, s, a) : launch_early(combine_kernel<D, 1>, grid, 128, 0, s, a);
}

template <int D>
cudaError_t run_attend(const AttendArgs& a, const AttendPlan& p, const CUtensorMap (&m)[4], cudaStream_t s) {
  using Sh = AttendSmem<D>;
  static bool done[64];
  cudaError_t e = allow_smem(attend_kernel<D>, Sh::BYTES, done);
  if (e != cudaSuccess) return e;
  return launch_early(attend_kernel<D>, dim3((unsigned)((p.max_runs ? p.max_runs : a.S) * p.row_tiles), (unsigned)a.Hkv),
                      ATHREADS, Sh::BYTES, s, m[0], m[1], m[2], m[3], a);
}
template <int D>
cudaError_t run_attend_d(const AttendArgs& a, const AttendPlan& p, cudaStream_t s) {
  CUtensorMap m[4];
  const long long page_rows = ((long long)a.n_pages * a.Hkv) << a.page_shift, cols = (long long)a.Hkv * D;
  const int box = a.page_shift < 6 ? 1 << a.page_shift : KT;
  // a call without cached rows reads no page: any matrix will do
  const bool none = a.max_len == 0 || page_rows == 0;
  if (!encode_tiles(&m[0], none ? a.k : a.kp, none ? 1 : page_rows, D, none ? a.ldk : D, box) ||
      !encode_tiles(&m[1], none ? a.v : a.vp, none ? 1 : page_rows, D, none ? a.ldv : D, box) ||
      !encode_tiles(&m[2], a.k, (long long)a.S * a.n, cols, a.ldk, KT) ||
      !encode_tiles(&m[3], a.v, (long long)a.S * a.n, cols, a.ldv, KT))
    return cudaErrorInvalidValue;
  cudaError_t e = run_attend<D>(a, p, m, s);
  if (e != cudaSuccess || p.max_runs == 0) return e;
  return join_runs<D>(a, s);
}

// A cluster of 8 CTAs for each sequence: together they copy its path's rows; its length is written by one of them
// once all eight have read it, so len_out may be cache_len.  A few megabytes at most: the chain of loads from the path to the
// page to the row is what takes its 8 us (9 for 32 paths of 8 layers, 7.3 MB), so all rows are asked for at once.
constexpr int CCTAS = 8, CTHREADS = 256;
__global__ void __cluster_dims__(CCTAS, 1, 1) __launch_bounds__(CTHREADS) kv_commit_kernel(KvCommitArgs a) {
  const int s = blockIdx.y, part = blockIdx.x;
  __shared__ int rows_s;
  const int len = a.cache_len[s];
  if (threadIdx.x < 32) {  // the path's length: up to its first bad entry, and what the pages hold
    const int lane = threadIdx.x;
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
  const int n = rows_s, vecs = a.Hkv * a.D / 8, per = a.D / 8;  // 16-byte vectors of a row, of a head
  const int total = a.L * n * vecs;
  for (int u = part * CTHREADS + threadIdx.x; u < total; u += CCTAS * CTHREADS) {
    const int vec = u % vecs, li = u / vecs, i = li % n, layer = li / n;
    const int head = vec / per, at = len + i;
    const int node = a.path[(long long)s * a.max_path + i];
    const int pg = a.table[(long long)s * a.max_pages + (at >> a.page_shift)];
    const long long src = (((long long)layer * a.S + s) * a.n + node) * vecs + vec;
    const long long dst = (((((long long)layer * a.n_pages + pg) * a.Hkv + head) << a.page_shift) +
                           (at & ((1 << a.page_shift) - 1))) * per + vec % per;
    reinterpret_cast<uint4*>(a.kp)[dst] = reinterpret_cast<const uint4*>(a.k)[src];
    reinterpret_cast<uint4*>(a.vp)[dst] = reinterpret_cast<const uint4*>(a.v)[src];
  }
  asm volatile("barrier.cluster.wait.acquire.aligned;\n" ::: "memory");
  if (part == 0 && threadIdx.x == 0) a.len_out[s] = len + n;
}

}  // namespace

size_t tree_attention_workspace_bytes(int S, int n, int Hq, int Hkv, int D, int max_len) {
  return attend_workspace_bytes(plan_attend(S, n, Hq, Hkv, max_len), S, n, Hq, Hkv, D);
}

cudaError_t launch_attend_join(const AttendArgs& a, cudaStream_t s) {
  return a.D == 64 ? join_runs<64>(a, s) : join_runs<128>(a, s);
}

cudaError_t launch_tree_attention(const AttendArgs& args, void* workspace, cudaStream_t s) {
  if (args.S == 0) return cudaSuccess;
  AttendArgs a = args;
  const AttendPlan p = plan_attend(a.S, a.n, a.Hq, a.Hkv, a.max_len);
  lay_workspace(a, p, workspace);
  return a.D == 64 ? run_attend_d<64>(a, p, s) : run_attend_d<128>(a, p, s);
}

cudaError_t launch_kv_commit(const KvCommitArgs& a, cudaStream_t s) {
  if (a.S == 0) return cudaSuccess;
  kv_commit_kernel<<<dim3(CCTAS, (unsigned)a.S), CTHREADS, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace ssmtree
