// Tree attention over an 8-bit paged cache for up to 16 query rows of a key/value head (ssm_attention.h): single tokens, small trees.
//
// The plan of attention_fp8.cu has 128 rows and tiles of 64 keys that pass from warp to warp; a few rows want the cache read as
// fast as memory gives it instead.  Here each warp takes 16 keys at a time by itself, with no barrier between its first row and
// the join (a few rows use little of any tensor core, so its products are warp-level ones):
//     S^T = K . Q^T,   P^T = 2^(S^T + log2 vs - m),   O^T += V^T . P^T
// with K and V made fp16 (exact) in registers, Q fp16 under a row scale that is a power of two (exact down to 2^-38 of a row's
// largest).  The columns of K's rows may stand in any order along a product's inner axis, and those of V's rows in any order along
// its outer one: a lane reads 16 bytes of a row of either and has fragments; two keys' bytes of V are put side by side by byte
// permutes before they are converted.  P^T goes from accumulators to operands by transposing 8 x 8 of fp16.  A lane of each warp asks
// for its rows, three to eight steps ahead (STAGES), by tensor copies into a ring of the warp's own.  Scales, weights and sums are those
// of attention_fp8.cu; the warps' sums are joined in shared memory, runs of a cache as there.
//
// Bound by HBM where caches are long: 76 tokens over up to 16000 rows 253 us (1.32 GB: 5.2 TB/s).  Else by what a block does before
// its first and after its last row (lengths, pages, rows one after the other, the join): in a CUDA graph, 32 query and 8 key/value
// heads of 128, one token over 16411 rows takes 18.1 us (16.4 where L2 holds the cache; the 128-row kernel 21.7 there), 16 over up to
// 4099 rows 25 (41), 64 over up to 1000 rows 21 (65), 128 of them 32.5 (86); 16 query rows, one sequence of 16411 rows 24 (in L2 23;
// 25.3), 8 of up to 8117 rows and 4 heads 26 (26.2); one token with heads of 64 13.9 (in L2 12.4; 19.4).  In L2, rows straight into
// registers, one step ahead: one token 16.9, 128 39.6; by asynchronous copies of 16 bytes: 19.1, 52.
#include "attend.cuh"
#include "decode.cuh"

namespace ssmtree {
namespace {

template <int D, int NT, bool CUT, int BLOCKS>  // NT: eights of rows; BLOCKS: blocks on an SM, which share 16 or 12 warps
struct Few {
  static constexpr int WARPS = (NT == 1 ? 16 : 12) / BLOCKS, THREADS = WARPS * 32, ROWS = 8 * NT, LD = D + 4;
  // a step in a warp's ring: 16 rows of K, 16 of V, as many steps under way as two blocks of an SM have room for
  static constexpr int KB = 16 * D, STEP = 2 * KB, STAGES = (NT == 1 ? 3 : 4) * (128 / D);
  static constexpr int OFF_MISC = WARPS * STAGES * STEP;
  static_assert(WARPS * ROWS * LD * 4 <= OFF_MISC, "the warps' sums stand there at the end");
};
template <int D, int NT, bool CUT, int BLOCKS>
struct FewMisc {
  using Sh = Few<D, NT, CUT, BLOCKS>;
  unsigned long long anc[64];
  unsigned long long full[Sh::WARPS][Sh::STAGES];
  SplitScratch split;
  float m[Sh::WARPS][Sh::ROWS], l[Sh::WARPS][Sh::ROWS];
  unsigned int odd;  // tree rows with a value of v that is not finite
  int stop;
};
template <int D, int NT, bool CUT, int BLOCKS>
constexpr int few_bytes() {
  constexpr int bytes = Few<D, NT, CUT, BLOCKS>::OFF_MISC + (int)sizeof(FewMisc<D, NT, CUT, BLOCKS>);
  static_assert(bytes <= 228 * 1024 / BLOCKS - 1024, "so many to an SM");
  return bytes;
}

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(r) : "r"(x));
  return r;
}
template <int WORDS>
__device__ __forceinline__ void load_words(uint32_t (&x)[WORDS], const unsigned char* p) {
  if constexpr (WORDS == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
  } else {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    x[0] = v.x, x[1] = v.y;
  }
}

// a warp's rows so far: of each eight, this lane's are 2 (lane % 4) and the one behind
template <int D, int NT>
struct FewState {
  float o[D / 16][NT][4];  // columns (lane / 4) D/8 + 2 j, of the two rows, and the column behind
  float m[NT][2], l[NT][2];

  // scores in powers of two (of keys lane/4 of two eights; minus infinity: does not count) to weights; r: what they count in the sum
  __device__ __forceinline__ void weigh(float (&x)[NT][4], float ra, float rb) {
    bool grows = false;
#pragma unroll
    for (int t = 0; t < NT; ++t) grows = grows || fmaxf(x[t][0], x[t][2]) > m[t][0] + 8.f || fmaxf(x[t][1], x[t][3]) > m[t][1] + 8.f;
    if (__any_sync(0xffffffffu, grows)) {  // what there is so far of such rows is made relative to the new maximum
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        float by[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float mx = fmaxf(x[t][e], x[t][2 + e]);
#pragma unroll
          for (int s = 4; s < 32; s *= 2) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, s));
          if (!(mx > m[t][e] + 8.f)) mx = m[t][e];  // (a row's weights do not depend on the other rows)
          by[e] = mx == m[t][e] ? 1.f : exp2_sfu(m[t][e] - mx);
          m[t][e] = mx, l[t][e] *= by[e];
        }
#pragma unroll
        for (int j = 0; j < D / 16; ++j) o[j][t][0] *= by[0], o[j][t][1] *= by[1], o[j][t][2] *= by[0], o[j][t][3] *= by[1];
      }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float ref = (m[t][e] == -INFINITY ? 0.f : m[t][e]) - kShift;
        x[t][e] = exp2_sfu(x[t][e] - ref), x[t][2 + e] = exp2_sfu(x[t][2 + e] - ref);
        l[t][e] = fmaf(x[t][e], ra, fmaf(x[t][2 + e], rb, l[t][e]));
      }
  }
};

template <int D, int NT, bool CUT, int BLOCKS>
__global__ void __launch_bounds__(Few<D, NT, CUT, BLOCKS>::THREADS, BLOCKS)
    attend8_few_kernel(const __grid_constant__ CUtensorMap tkp, const __grid_constant__ CUtensorMap tvp, AttendFp8Args f) {
  using Sh = Few<D, NT, CUT, BLOCKS>;
  constexpr int W = Sh::WARPS, KI = D / 64, VW = D / 32;  // 64-column parts of a row; words of V's row in a lane
  const AttendArgs& a = f.a;
  extern __shared__ __align__(1024) unsigned char smem[];  // (there is no room to move it: where it is not aligned, nothing runs)
  float* o_s = reinterpret_cast<float*>(smem);
  FewMisc<D, NT, CUT, BLOCKS>& ms = *reinterpret_cast<FewMisc<D, NT, CUT, BLOCKS>*>(smem + Sh::OFF_MISC);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31, g = lane >> 2, c = lane & 3;
  const int rows = a.n * a.g, run = blockIdx.x, kvh = blockIdx.y;
  if (smem_u32(smem) & 1023u) {
    grid_dependency_wait();  // no grid ends before the one that it depends on
    if (tid == 0) flag(a.status, SSM_STATUS_TIMEOUT);
    if (CUT && tid == 0 && run < a.S) a.runs[run] = make_int2(0, 1);  // nothing to join
    return;
  }
  if (tid < W * Sh::STAGES) mbar_init(smem_u32(&ms.full[0][0] + tid), 1);
  if (tid == 0) ms.stop = 0;
  fence_barrier_init();
  __syncthreads();
  grid_dependency_wait();  // what the stream's kernels before this one write
  launch_dependents();
  int s = run, sp = 0, tps = 1 << 25, splits = 1;
  if constexpr (CUT) if (a.max_runs > 0) {  // (it is: said once more, nothing spills)
    int* tiles = reinterpret_cast<int*>(o_s);  // space not in use yet
    int first;
    tps = choose_split<Sh::THREADS>(a, a.Hkv, tiles, &ms.split);
    if (!find_run(a.S, tiles, tps, run, s, first, splits)) return;
    fence_async_smem();
    __syncthreads();  // (behind it the copies may write there)
    sp = run - first;
    if (sp == 0 && kvh == 0 && tid == 0) a.runs[s] = make_int2(first, splits);
  }
  // Q: of row g of each eight the columns that a lane has of K's rows, as fp16 of a power of two
  uint32_t qx[NT][KI][4][2];
  float qc[NT][2];
  auto q_row = [&](int t) {
    const int row = min(8 * t + g, rows - 1);
    return reinterpret_cast<const uint4*>(a.q + ((long long)s * a.n + row / a.g) * a.ldq + (kvh * a.g + row % a.g) * D + KI * c * 16);
  };
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int i = 0; i < KI; ++i) {
      const uint4 x = q_row(t)[i * 2], y = q_row(t)[i * 2 + 1];
      qx[t][i][0][0] = x.x, qx[t][i][0][1] = x.y, qx[t][i][1][0] = x.z, qx[t][i][1][1] = x.w;
      qx[t][i][2][0] = y.x, qx[t][i][2][1] = y.y, qx[t][i][3][0] = y.z, qx[t][i][3][1] = y.w;
    }
  // The run's keys of the cache, k0 .. end - 1, in steps of 16: those of this warp are warp + i W, i < mine.  Of 16 steps of the warp a
  // lane knows the eight keys lane & 1 of the lane / 2-th: their first row among the pages' (-1: no such rows, or their page is out
  // of range), the scales, how many there are.  Pages are asked for 16 steps ahead, and before the length is known.
  const bool has_tree = sp == 0;
  const int t0 = sp * tps + has_tree - 1, k0 = t0 * KT;
  const int32_t* table = a.table + (long long)s * a.max_pages;
  auto key_of = [&](int b) { return (unsigned int)k0 + (unsigned int)(warp + (16 * b + (lane >> 1)) * W) * 16 + (lane & 1) * 8; };
  auto page_of = [&](int b) {
    const unsigned int at = key_of(b) >> a.page_shift;
    return at < (a.max_len > 0 ? (unsigned int)a.max_pages : 0u) ? table[at] : -1;  // (without cached rows there may be no table)
  };
  int next_page = page_of(0);
  int len = __shfl_sync(0xffffffffu, cached_rows(a, s), 0);
  if (len < 0) {
    if (sp == 0 && kvh == 0 && tid == 0) flag(a.status, SSM_STATUS_SEQ_RANGE);
    len = 0;
  }
  const int t1 = min(sp * tps + tps - 1, (len + KT - 1) / KT), end = min(t1 * KT, len);
  const int steps = max(end - k0 + 15, 0) / 16, mine = (steps - warp + W - 1) / W;
  auto row_of = [&](int b, int pg) {
    const unsigned int at = key_of(b);
    if (16 * b + (lane >> 1) >= mine || at >= (unsigned int)max(end, 0)) return -1;
    if (pg < 0 || pg >= a.n_pages) {
      flag(a.status, SSM_STATUS_SEQ_RANGE);
      return -1;
    }
    return ((pg * a.Hkv + kvh) << a.page_shift) + (int)(at & ((1u << a.page_shift) - 1));
  };
  int at_row = row_of(0, next_page), next_row = -1, there = 0;
  next_page = page_of(1);
  float ks = 1.f, lv = 0.f, rv = 1.f, v0 = 1.f;

  // One lane asks for a step's rows, box of them at a time, all in one page.  As they land swizzled, a warp's reads have no bank
  // conflicts (two ways where a lane has eight columns of V, in heads of 64).
  unsigned char* ring = smem + warp * Sh::STAGES * Sh::STEP;
  const int box = min(1 << a.page_shift, 16);
  auto ask = [&](int i, int stage, int rows_at) {  // step i of the sixteen whose rows these are
    const int ra = __shfl_sync(0xffffffffu, rows_at, 2 * i & 31), rb = __shfl_sync(0xffffffffu, rows_at, (2 * i & 31) + 1);
    if (lane == 0) {
      const uint32_t bar = smem_u32(&ms.full[warp][stage]), to = smem_u32(ring) + stage * Sh::STEP;
      const bool second = box == 8 && rb >= 0;
      mbar_arrive_expect_tx(bar, ((ra >= 0 ? box : 0) + (second ? 8 : 0)) * 2 * D);
      if (ra >= 0) tma_load_2d(to, &tkp, 0, ra, bar), tma_load_2d(to + Sh::KB, &tvp, 0, ra, bar);
      if (second) tma_load_2d(to + 8 * D, &tkp, 0, rb, bar), tma_load_2d(to + Sh::KB + 8 * D, &tvp, 0, rb, bar);
    }
    __syncwarp();
  };
#pragma unroll 1
  for (int i = 0; i < Sh::STAGES && i < mine; ++i) ask(i, i, at_row);
  const bool tree = has_tree && warp == W - 1;  // this warp has the tree's rows as well (and the fewest steps)
  float2 sc = make_float2(1.f, 1.f);
  auto load_scales = [&](int r) {
    sc = make_float2(1.f, 1.f);
    if (r >= 0) sc = make_float2(f.ks[r >> f.block_shift], f.vs[r >> f.block_shift]);
  };
  load_scales(at_row);

  FewState<D, NT> st;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    st.m[t][0] = st.m[t][1] = -INFINITY, st.l[t][0] = st.l[t][1] = 0.f;
#pragma unroll
    for (int j = 0; j < D / 16; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) st.o[j][t][e] = 0.f;
  }

#pragma unroll
  for (int t = 0; t < NT; ++t) {
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < KI; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t w = qx[t][i][j / 2][j & 1], lo = w << 16 & 0x7fffffffu, hi = w & 0x7fff0000u;
        most = max(most, max(lo < 0x7f800000u ? lo : 0u, hi < 0x7f800000u ? hi : 0u));
      }
    most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
    most = max(most, __shfl_xor_sync(0xffffffffu, most, 2));
    const int e = min(14 - ((int)(most >> 23) - 127), 100);  // the largest to 2^14 .. 2^15
    const float by = __uint_as_float((uint32_t)(127 + e) << 23), back = a.scale_log2 * __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
    for (int i = 0; i < KI; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint32_t& w = qx[t][i][j / 2][j & 1];
        w = pack_f16x2(nan_unless_finite(bf16_lo(w)) * by, nan_unless_finite(bf16_hi(w)) * by);
      }
    qc[t][0] = __shfl_sync(0xffffffffu, back, 8 * c), qc[t][1] = __shfl_sync(0xffffffffu, back, 8 * c + 4);
  }

  if (tree) {  // the tree's own rows, up to 16, in bf16
    const long long row0 = (long long)s * a.n;
    uint4 kt[KI][2][2], vt[KI][4];  // all asked for at once
#pragma unroll
    for (int i = 0; i < KI; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint4* p = reinterpret_cast<const uint4*>(a.k + (row0 + g + 8 * h) * a.ldk + kvh * D + (KI * c + i) * 16);
        kt[i][h][0] = kt[i][h][1] = make_uint4(0, 0, 0, 0);
        if (g + 8 * h < a.n) kt[i][h][0] = p[0], kt[i][h][1] = p[1];
      }
#pragma unroll
    for (int h = 0; h < KI; ++h)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int key = 2 * c + (k & 1) + (k >> 1) * 8;
        vt[h][k] = make_uint4(0, 0, 0, 0);
        if (key < a.n) vt[h][k] = *reinterpret_cast<const uint4*>(a.v + (row0 + key) * a.ldv + kvh * D + g * (D / 8) + h * 8);
      }
    if (lane == 0) ms.odd = 0;
    ancestor_words(a, s, ms.anc, kvh == 0);
    __syncwarp();
    float x[NT][4] = {};
#pragma unroll
    for (int i = 0; i < KI; ++i) {
      uint32_t w[2][8];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint4 y0 = kt[i][h][0], y1 = kt[i][h][1];
        w[h][0] = y0.x, w[h][1] = y0.y, w[h][2] = y0.z, w[h][3] = y0.w;
        w[h][4] = y1.x, w[h][5] = y1.y, w[h][6] = y1.z, w[h][7] = y1.w;
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const uint4 y0 = q_row(t)[i * 2], y1 = q_row(t)[i * 2 + 1];
        const uint32_t q[8] = {y0.x, y0.y, y0.z, y0.w, y1.x, y1.y, y1.z, y1.w};
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          const uint32_t ka[4] = {w[0][j], w[1][j], w[0][j + 1], w[1][j + 1]}, qb[2] = {q[j], q[j + 1]};
          mma_bf16(x[t], ka, qb);
        }
      }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int node = min(8 * t + 2 * c + (e & 1), rows - 1) / a.g;
        x[t][e] = ms.anc[node] >> (g + (e >> 1) * 8) & 1 ? x[t][e] * a.scale_log2 : -INFINITY;
      }
    st.weigh(x, 1.f, 1.f);
    {  // what this warp's scales of v are relative to: the least of its first ones, as a power of two within 2^60 of 1
      const bool counts = at_row >= 0 && good_scale(sc.x) && good_scale(sc.y);
      const unsigned int least = __reduce_min_sync(0xffffffffu, counts ? __float_as_uint(sc.y) & 0x7f800000u : 0x7f800000u);
      v0 = least == 0x7f800000u ? 1.f : fminf(fmaxf(__uint_as_float(least), 0x1p-60f), 0x1p60f);
    }
    const float up = 1.f / v0;
    uint32_t p[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t)
      p[t][0] = transposed(pack_bf16x2(x[t][0] * up, x[t][1] * up)), p[t][1] = transposed(pack_bf16x2(x[t][2] * up, x[t][3] * up));
#pragma unroll
    for (int h = 0; h < KI; ++h) {  // eight of a lane's columns
      uint32_t w[4][4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int key = 2 * c + (k & 1) + (k >> 1) * 8;
        const uint4 y = vt[h][k];
        w[k][0] = finite_or_zero(y.x), w[k][1] = finite_or_zero(y.y), w[k][2] = finite_or_zero(y.z), w[k][3] = finite_or_zero(y.w);
        if (w[k][0] != y.x || w[k][1] != y.y || w[k][2] != y.z || w[k][3] != y.w) atomicOr(&ms.odd, 1u << key);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t va[4] = {__byte_perm(w[0][j], w[1][j], 0x5410), __byte_perm(w[0][j], w[1][j], 0x7632),
                                __byte_perm(w[2][j], w[3][j], 0x5410), __byte_perm(w[2][j], w[3][j], 0x7632)};
#pragma unroll
        for (int t = 0; t < NT; ++t) mma_bf16(st.o[4 * h + j][t], va, p[t]);
      }
    }
  }

  // where a lane's bytes of a step are: 16 bytes of 64 columns of K's rows g and 8 + g, its columns of V's rows 2 c + e and 8 + 2 c + e
  auto k_at = [&](int h, int e) { return (g + 8 * e) * D + ((KI == 2 ? (2 * c + h) ^ g : c ^ (g >> 1)) << 4); };
  auto v_at = [&](int e, int b) {
    return Sh::KB + (2 * c + e + 8 * b) * D + (KI == 2 ? (g ^ (2 * c + e)) << 4 : (((g >> 1) ^ c) << 4) + (g & 1) * 8);
  };
  bool ok = true;
  int i = 0, stage = 0, phase = 0;
#pragma unroll 1
  for (; i < mine; ++i) {
    if ((i & 15) == 0) {  // what the next 16 steps' keys are
      if (i > 0) at_row = next_row;
      next_row = row_of(i / 16 + 1, next_page), next_page = page_of(i / 16 + 2);
      const bool good = good_scale(sc.x) && good_scale(sc.y);
      if (!good) {
        flag(a.status, SSM_STATUS_SCALE);
        sc = make_float2(1.f, 1.f);
      }
      there = at_row >= 0 && good ? min(end - (int)key_of(i / 16), 8) : 0;
      if (i == 0 && !tree) {  // what this warp's scales of v are relative to: one of them, as a power of two
        const unsigned int top = __reduce_max_sync(0xffffffffu, there > 0 ? __float_as_uint(sc.y) & 0x7f800000u : 0u);
        v0 = top ? __uint_as_float(top) : 1.f;
      }
      const float rel = fminf(fmaxf(sc.y / v0, 0x1p-120f), 0x1p120f);
      ks = sc.x, lv = log2f(rel), rv = 1.f / rel;
    }
    if ((i & 15) == 8) load_scales(next_row);
    const int from = 2 * i & 31;
    const int ta = __shfl_sync(0xffffffffu, there, from), tb = __shfl_sync(0xffffffffu, there, from + 1);
    const float ka = __shfl_sync(0xffffffffu, ks, from), kb = __shfl_sync(0xffffffffu, ks, from + 1);
    const float la = __shfl_sync(0xffffffffu, lv, from), lb = __shfl_sync(0xffffffffu, lv, from + 1);
    const float ia = __shfl_sync(0xffffffffu, rv, from), ib = __shfl_sync(0xffffffffu, rv, from + 1);
    ok = wait_bar(&ms.full[warp][stage], phase, &ms.stop);
    if (!ok) break;
    const unsigned char* step = ring + stage * Sh::STEP;
    float x[NT][4] = {};
#pragma unroll
    for (int h = 0; h < KI; ++h) {
      uint32_t kx[2][4];
#pragma unroll
      for (int e = 0; e < 2; ++e) load_words(kx[e], step + k_at(h, e));
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t ak[4] = {e4m3x2_f16x2(kx[0][j]), e4m3x2_f16x2(kx[1][j]), e4m3x2_f16x2(kx[0][j] >> 16),
                                e4m3x2_f16x2(kx[1][j] >> 16)};
#pragma unroll
        for (int t = 0; t < NT; ++t) mma_f16(x[t], ak, qx[t][h][j][0], qx[t][h][j][1]);
      }
    }
    uint32_t vx[2][2][VW];  // (read before the weights are made)
#pragma unroll
    for (int e = 0; e < 2; ++e) load_words(vx[0][e], step + v_at(e, 0)), load_words(vx[1][e], step + v_at(e, 1));
    __syncwarp();
    const int then = i + Sh::STAGES;
    if (then < mine) ask(then, stage, (then ^ i) & ~15 ? next_row : at_row);
    if (++stage == Sh::STAGES) stage = 0, phase ^= 1;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float y = fmaf(x[t][e], qc[t][e & 1] * (e < 2 ? ka : kb), e < 2 ? la : lb);
        x[t][e] = g < (e < 2 ? ta : tb) ? y : -INFINITY;
      }
    st.weigh(x, ia, ib);
    uint32_t p[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) p[t][0] = transposed(pack_f16x2(x[t][0], x[t][1])), p[t][1] = transposed(pack_f16x2(x[t][2], x[t][3]));
    if (ta + tb < 16) {  // (whatever stands where no key is)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int w = 0; w < VW; ++w) vx[0][e][w] = 2 * c + e < ta ? vx[0][e][w] : 0u, vx[1][e][w] = 2 * c + e < tb ? vx[1][e][w] : 0u;
    }
#pragma unroll
    for (int w = 0; w < VW; ++w) {
      const uint32_t a01 = __byte_perm(vx[0][0][w], vx[0][1][w], 0x5140), a23 = __byte_perm(vx[0][0][w], vx[0][1][w], 0x7362);
      const uint32_t b01 = __byte_perm(vx[1][0][w], vx[1][1][w], 0x5140), b23 = __byte_perm(vx[1][0][w], vx[1][1][w], 0x7362);
      const uint32_t v01[4] = {e4m3x2_f16x2(a01), e4m3x2_f16x2(a01 >> 16), e4m3x2_f16x2(b01), e4m3x2_f16x2(b01 >> 16)};
      const uint32_t v23[4] = {e4m3x2_f16x2(a23), e4m3x2_f16x2(a23 >> 16), e4m3x2_f16x2(b23), e4m3x2_f16x2(b23 >> 16)};
#pragma unroll
      for (int t = 0; t < NT; ++t) mma_f16(st.o[2 * w][t], v01, p[t][0], p[t][1]), mma_f16(st.o[2 * w + 1][t], v23, p[t][0], p[t][1]);
    }
  }
  if (!ok) {  // copies land before the shared memory is given up
    if (lane == 0) {
      flag(a.status, SSM_STATUS_TIMEOUT);
      for (int k = i; k < min(i + Sh::STAGES, mine); ++k) {
        mbar_wait(smem_u32(&ms.full[warp][stage]), phase);
        if (++stage == Sh::STAGES) stage = 0, phase ^= 1;
      }
    }
    __syncwarp();
  }

  // the warps' sums as one
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float l = st.l[t][e];
#pragma unroll
      for (int k = 4; k < 32; k *= 2) l += __shfl_xor_sync(0xffffffffu, l, k);
      if (g == 0) ms.m[warp][8 * t + 2 * c + e] = st.m[t][e], ms.l[warp][8 * t + 2 * c + e] = l;
    }
  __syncthreads();  // (the tile counts are not read any more either)
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int row = 8 * t + 2 * c + e;
      float top = ms.m[0][row];
#pragma unroll
      for (int w = 1; w < W; ++w) top = fmaxf(top, ms.m[w][row]);
      const float by = st.m[t][e] == -INFINITY ? 0.f : exp2_sfu(st.m[t][e] - top) * v0;
      float* to = o_s + (warp * Sh::ROWS + row) * Sh::LD + g * (D / 8);
#pragma unroll
      for (int j = 0; j < D / 16; ++j) *reinterpret_cast<float2*>(to + 2 * j) = make_float2(st.o[j][t][e] * by, st.o[j][t][2 + e] * by);
    }
  __syncthreads();
  for (int u = tid; u < rows * (D / 4); u += Sh::THREADS) {
    const int row = u / (D / 4), col = u % (D / 4) * 4, node = row / a.g, head = kvh * a.g + row % a.g;
    float top = ms.m[0][row], l = 0.f;
#pragma unroll
    for (int w = 1; w < W; ++w) top = fmaxf(top, ms.m[w][row]);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float4 x = *reinterpret_cast<const float4*>(o_s + (w * Sh::ROWS + row) * Sh::LD + col);
      o.x += x.x, o.y += x.y, o.z += x.z, o.w += x.w;
      l = fmaf(ms.l[w][row], ms.m[w][row] == -INFINITY ? 0.f : exp2_sfu(ms.m[w][row] - top), l);
    }
    const long long tok = (long long)s * a.n + node;
    if (has_tree) {
#pragma unroll 1
      for (unsigned int odd = ms.odd & (unsigned int)ms.anc[node]; odd; odd &= odd - 1) {  // not finite whatever its weight
        const uint2 x = *reinterpret_cast<const uint2*>(a.v + ((long long)s * a.n + __ffs((int)odd) - 1) * a.ldv + kvh * D + col);
        const uint2 out = make_uint2(x.x ^ finite_or_zero(x.x), x.y ^ finite_or_zero(x.y));
        if (out.x & 0xffffu) o.x += bf16_lo(x.x);
        if (out.x & 0xffff0000u) o.y += bf16_hi(x.x);
        if (out.y & 0xffffu) o.z += bf16_lo(x.y);
        if (out.y & 0xffff0000u) o.w += bf16_hi(x.y);
      }
    }
    if (splits == 1) {
      const float inv = 1.f / l;
      *reinterpret_cast<uint2*>(a.o + tok * a.ldo + head * D + col) = make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
    } else {
      const long long at = ((long long)run * a.Hkv + kvh) * rows + row;
      *reinterpret_cast<float4*>(a.part + at * D + col) = o;
      if (col == 0) a.part_ml[at] = make_float2(top, l);
    }
  }
}

template <int D, int NT, bool CUT, int BLOCKS>
cudaError_t run_few(const AttendFp8Args& f, int max_runs, cudaStream_t s) {
  using Sh = Few<D, NT, CUT, BLOCKS>;
  constexpr int bytes = few_bytes<D, NT, CUT, BLOCKS>();
  static_assert(!CUT || 2 * 2 * kSMs * 4 <= Sh::OFF_MISC, "the tile counts stand in the space of the ring");
  const AttendArgs& a = f.a;
  CUtensorMap m[2];
  const long long page_rows = ((long long)a.n_pages * a.Hkv) << a.page_shift;
  const int box = a.page_shift < 4 ? 8 : 16;
  // a call without cached rows reads no page: any matrix will do
  const bool none = a.max_len == 0 || page_rows == 0;
  if (!encode_byte_tiles(&m[0], none ? static_cast<const void*>(a.k) : f.kp, none ? 1 : page_rows, D, box) ||
      !encode_byte_tiles(&m[1], none ? static_cast<const void*>(a.v) : f.vp, none ? 1 : page_rows, D, box))
    return cudaErrorInvalidValue;
  static bool done[64];
  cudaError_t e = allow_smem(attend8_few_kernel<D, NT, CUT, BLOCKS>, bytes, done);
  if (e != cudaSuccess) return e;
  e = launch_early(attend8_few_kernel<D, NT, CUT, BLOCKS>, dim3((unsigned)(CUT ? max_runs : a.S), (unsigned)a.Hkv), Sh::THREADS, bytes, s, m[0], m[1], f);
  return e != cudaSuccess || !CUT ? e : launch_attend_join(a, s);
}

// Where sequences and heads give each SM two blocks or more, blocks are half as large and four to an SM, so that one's beginning and
// end pass under the others' rows (128 tokens over up to 1000 rows 32 us, with two to an SM 36.5; 64 of them, cut into runs, 32.3 and
// 37.5; 76 over up to 16000 rows 252 and 240); below that a larger block takes a run in less time (one token 18.1 us).
template <int D>
cudaError_t run_few(const AttendFp8Args& f, int max_runs, cudaStream_t s) {
  const bool many = f.a.S * f.a.Hkv >= 2 * kSMs;
  if (f.a.n * f.a.g <= 8) {
    if (max_runs == 0) return run_few<D, 1, false, 4>(f, max_runs, s);
    return many ? run_few<D, 1, true, 4>(f, max_runs, s) : run_few<D, 1, true, 2>(f, max_runs, s);
  }
  if (max_runs == 0) return run_few<D, 2, false, 4>(f, max_runs, s);
  return many ? run_few<D, 2, true, 4>(f, max_runs, s) : run_few<D, 2, true, 2>(f, max_runs, s);
}

}  // namespace

cudaError_t launch_few_attention_fp8(const AttendFp8Args& f, int max_runs, cudaStream_t s) {
  return f.a.D == 64 ? run_few<64>(f, max_runs, s) : run_few<128>(f, max_runs, s);
}

}  // namespace ssmtree
