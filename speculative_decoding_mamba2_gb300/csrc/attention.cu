// Attention of a draft tree's nodes over a paged cache and their ancestors, and the commit of the accepted
// path into the cache (ssm_attention.h).
//
// attend_kernel.  The query rows of one key/value head -- n nodes x g query heads -- share its keys, so a CTA
// takes up to RT of them and walks tiles of 64 keys once, with the running maximum and sum of each row's
// softmax: s = q.k, m' = max(m, s), p = 2^(s - m'), l' = l 2^(m - m') + sum p, o' = o 2^(m - m') + p v.
// One tile more than the cache has holds the tree's own rows; there a row keeps its node's ancestors only,
// read from a 64-bit word per node.  Few rows share a tile (n g operations for each byte of the cache), so the
// keys are split over the SMs where the (sequence, head, row tile) triples leave SMs idle; the partial sums
// are then joined by combine_kernel.
#include "mma_tiles.cuh"
#include "prompt.cuh"

namespace ssmtree {
namespace {

constexpr int KT = 64;  // keys per tile
constexpr int ATHREADS = 128;

// WM warps along the rows, MT m16 tiles each; 4 / WM warps along the keys of a tile
template <int D, int WM, int MT>
struct AttendShape {
  static constexpr int RT = WM * MT * 16, WN = 4 / WM;
  static constexpr int STAGES = 2;
  static constexpr int OFF_KV = RT * D * 2;                      // after q
  static constexpr int KV = KT * D * 2;
  static constexpr int OFF_ANC = OFF_KV + STAGES * 2 * KV;       // 64 ancestor words, 64 links
  static constexpr int SMEM = OFF_ANC + 64 * 8 + 64 * 4 + 16;
};

template <int D, int WM, int MT>
__global__ void __launch_bounds__(ATHREADS, 2) attend_kernel(AttendArgs a) {
  using Sh = AttendShape<D, WM, MT>;
  constexpr int RT = Sh::RT, WN = Sh::WN, ROWB = D * 2, CH = D / 8;
  constexpr int KW = KT / WN, NT = KW / 8, DT = D / 8;  // keys, score and output n-tiles of a warp
  extern __shared__ __align__(128) unsigned char smem[];
  unsigned long long* anc = reinterpret_cast<unsigned long long*>(smem + Sh::OFF_ANC);
  volatile int* link = reinterpret_cast<volatile int*>(smem + Sh::OFF_ANC + 64 * 8);
  volatile int* no_page = link + 64;  // whether a row's page is out of range
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g8 = lane >> 2, q4 = lane & 3;
  const int wm = warp % WM, wn = warp / WM;
  const int rows = a.n * a.g, rt = (rows + RT - 1) / RT;
  const int sp = blockIdx.x, kvh = blockIdx.y, s = blockIdx.z / rt, r0 = (blockIdx.z % rt) * RT;
  int len = a.cache_len[s];
  if (len < 0 || len > a.max_len || (long long)len > ((long long)a.max_pages << a.page_shift)) {
    if (sp == 0 && kvh == 0 && r0 == 0 && tid == 0) flag(a.status, SSM_STATUS_SEQ_RANGE);
    len = 0;
  }
  const int ct = (len + KT - 1) / KT, nt = ct + 1;  // tiles: the cache's, then the tree's
  const int i0 = sp * a.tps, i1 = min(nt, i0 + a.tps);
  if (i0 >= i1) return;
  const uint32_t sb = smem_u32(smem);
  const int32_t* table = a.table + (long long)s * a.max_pages;
  const int pmask = (1 << a.page_shift) - 1;

  if (tid == 0) *no_page = 0;
  __syncthreads();
  // q rows (zero beyond the last)
  for (int i = tid; i < RT * CH; i += ATHREADS) {
    const int r = i / CH, ch = i % CH, row = r0 + r;
    const bool there = row < rows;
    const int node = there ? row / a.g : 0, j = there ? row % a.g : 0;
    cp_async16_or_zero(sb + tile_off(r, ch, ROWB),
                       a.q + ((long long)s * a.n + node) * a.ldq + (kvh * a.g + j) * D + ch * 8, there);
  }
  auto load = [&](int i) {
    const uint32_t st = sb + Sh::OFF_KV + (i & 1) * 2 * Sh::KV;
#pragma unroll 4
    for (int u = tid; u < KT * CH; u += ATHREADS) {
      const int r = u / CH, ch = u % CH;
      const uint16_t *kr = a.kp, *vr = a.vp;
      bool there;
      if (i < ct) {
        const int at = i * KT + r;
        there = at < len;
        const int pg = there ? table[at >> a.page_shift] : 0;
        if (pg < 0 || pg >= a.n_pages) {
          flag(a.status, SSM_STATUS_SEQ_RANGE);
          *no_page = 1;
          there = false;
        }
        if (there) {
          const long long off = ((((long long)pg * a.Hkv + kvh) << a.page_shift) + (at & pmask)) * D + ch * 8;
          kr += off, vr += off;
        }
      } else {
        there = r < a.n;
        const long long row = (long long)s * a.n + (there ? r : 0);
        kr = a.k + row * a.ldk + kvh * D + ch * 8;
        vr = a.v + row * a.ldv + kvh * D + ch * 8;
      }
      cp_async16_or_zero(st + tile_off(r, ch, ROWB), kr, there);
      cp_async16_or_zero(st + Sh::KV + tile_off(r, ch, ROWB), vr, there);
    }
    cp_async_commit();
  };
  load(i0);

  // ancestor words: a node's own bit, then its parent's word, its grandparent's, ... by doubling
  if (i1 == nt && warp == 0) {
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
      anc[v] = w[k], link[v] = p[k];
    }
    if (bad && kvh == 0 && r0 == 0) flag(a.status, SSM_STATUS_BAD_LAYOUT);
    for (int step = 0; step < 6; ++step) {
      __syncwarp();
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (p[k] >= 0) w[k] |= reinterpret_cast<volatile unsigned long long*>(anc)[p[k]], p[k] = link[p[k]];
      __syncwarp();
#pragma unroll
      for (int k = 0; k < 2; ++k) anc[lane + 32 * k] = w[k], link[lane + 32 * k] = p[k];
    }
  }

  float o[MT][DT][4], m[MT][2], l[MT][2];
#pragma unroll
  for (int t = 0; t < MT; ++t) {
#pragma unroll
    for (int d = 0; d < DT; ++d) o[t][d][0] = o[t][d][1] = o[t][d][2] = o[t][d][3] = 0.f;
    m[t][0] = m[t][1] = -INFINITY, l[t][0] = l[t][1] = 0.f;
  }

#pragma unroll 1
  for (int i = i0; i < i1; ++i) {
    cp_async_wait<0>();
    __syncthreads();  // the tile is there; the other stage's readers are done
    if (i + 1 < i1) load(i + 1);
    const uint32_t kt = sb + Sh::OFF_KV + (i & 1) * 2 * Sh::KV, vt = kt + Sh::KV;
    const bool tree = i == ct;
    unsigned long long odd = 0;  // tree rows with values of v that are not finite: zero in the tile, added by themselves
    if (tree) {
      if (tid < a.n) {
        bool f = false;
#pragma unroll 1
        for (int ch = 0; ch < CH; ++ch) {
          uint4* v = reinterpret_cast<uint4*>(smem + (vt - sb) + tile_off(tid, ch, ROWB));
          const uint4 x = *v;
          const uint4 y = make_uint4(finite_or_zero(x.x), finite_or_zero(x.y), finite_or_zero(x.z), finite_or_zero(x.w));
          if (x.x != y.x || x.y != y.y || x.z != y.z || x.w != y.w) f = true, *v = y;
        }
        link[tid] = f ? -2 : -1;
      } else if (tid < 64) {
        link[tid] = -1;
      }
      __syncthreads();
      odd = (unsigned long long)__ballot_sync(0xffffffffu, link[lane] == -2) |
            (unsigned long long)__ballot_sync(0xffffffffu, link[lane + 32] == -2) << 32;
    }
    // scores of this warp's keys
    float sc[MT][NT][4];
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int j = 0; j < NT; ++j) sc[t][j][0] = sc[t][j][1] = sc[t][j][2] = sc[t][j][3] = 0.f;
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      uint32_t qf[MT][4];
#pragma unroll
      for (int t = 0; t < MT; ++t) frag_a(qf[t], sb, ROWB, (wm * MT + t) * 16, 16 * k, lane);
#pragma unroll
      for (int j = 0; j < NT / 2; ++j) {
        uint32_t b[4];
        frag_b2(b, kt, ROWB, wn * KW + 16 * j, 16 * k, lane);
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          mma16816(sc[t][2 * j], qf[t], b[0], b[1]);
          mma16816(sc[t][2 * j + 1], qf[t], b[2], b[3]);
        }
      }
    }
    const int left = tree ? a.n : len - i * KT;
    uint32_t pf[MT][NT][2];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      const int ra = r0 + (wm * MT + t) * 16 + g8;
      if (tree || left < KT || *no_page) {
        unsigned long long wa = ~0ull, wb = ~0ull;
        if (tree) {
          wa = ra < rows ? anc[ra / a.g] : 0ull;
          wb = ra + 8 < rows ? anc[(ra + 8) / a.g] : 0ull;
        } else if (*no_page) {  // rows on such pages are absent
#pragma unroll 1
          for (int key = 0; key < min(left, KT); ++key) {
            const int pg = table[(i * KT + key) >> a.page_shift];
            if (pg < 0 || pg >= a.n_pages) wa &= ~(1ull << key);
          }
          wb = wa;
        }
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int key = wn * KW + 8 * j + 2 * q4 + e;
            if (key >= left || !(wa >> key & 1)) sc[t][j][e] = -INFINITY;
            if (key >= left || !(wb >> key & 1)) sc[t][j][2 + e] = -INFINITY;
          }
      }
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        float mx = m[t][half];
#pragma unroll
        for (int j = 0; j < NT; ++j) mx = fmaxf(mx, fmaxf(sc[t][j][2 * half], sc[t][j][2 * half + 1]) * a.scale_log2);
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const float ref = mx == -INFINITY ? 0.f : mx;  // a row none of whose keys so far counts
        const float f = exp2_sfu(m[t][half] - ref);
        m[t][half] = mx;
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const float p0 = exp2_sfu(fmaf(sc[t][j][2 * half], a.scale_log2, -ref));
          const float p1 = exp2_sfu(fmaf(sc[t][j][2 * half + 1], a.scale_log2, -ref));
          sum += p0 + p1;
          pf[t][j][half] = pack_bf16x2(p0, p1);
        }
        l[t][half] = fmaf(l[t][half], f, sum);
#pragma unroll
        for (int d = 0; d < DT; ++d) o[t][d][2 * half] *= f, o[t][d][2 * half + 1] *= f;
      }
    }
#pragma unroll
    for (int j = 0; j < NT / 2; ++j)
#pragma unroll
      for (int d = 0; d < DT / 2; ++d) {
        uint32_t b[4];
        frag_b2_t(b, vt, ROWB, 16 * d, wn * KW + 16 * j, lane);
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          const uint32_t pa[4] = {pf[t][2 * j][0], pf[t][2 * j][1], pf[t][2 * j + 1][0], pf[t][2 * j + 1][1]};
          mma16816(o[t][2 * d], pa, b[0], b[1]);
          mma16816(o[t][2 * d + 1], pa, b[2], b[3]);
        }
      }
    // what the values left out add, in the rows that see them, is not finite whatever its weight
    const unsigned long long mine = WN == 1 ? odd : odd >> (wn * KW) << (wn * KW) & (wn + 1 < WN ? (1ull << (wn + 1) * KW) - 1 : ~0ull);
    if (mine) {  // each by the warp whose key it is
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        const int ra = r0 + (wm * MT + t) * 16 + g8;
        const unsigned long long wa = ra < rows ? anc[ra / a.g] : 0ull, wb = ra + 8 < rows ? anc[(ra + 8) / a.g] : 0ull;
#pragma unroll 1
        for (unsigned long long left = mine & (wa | wb); left; left &= left - 1) {
          const int key = __ffsll((long long)left) - 1;
          const bool sa = wa >> key & 1, sb2 = wb >> key & 1;
          const uint16_t* v = a.v + ((long long)s * a.n + key) * a.ldv + kvh * D + 2 * q4;
#pragma unroll
          for (int d = 0; d < DT; ++d) {
            const uint32_t x = *reinterpret_cast<const uint32_t*>(v + 8 * d), out = x ^ finite_or_zero(x);
            const float x0 = out & 0xffffu ? bf16_lo(x) : 0.f, x1 = out & 0xffff0000u ? bf16_hi(x) : 0.f;
            o[t][d][0] += sa ? x0 : 0.f, o[t][d][1] += sa ? x1 : 0.f;
            o[t][d][2] += sb2 ? x0 : 0.f, o[t][d][3] += sb2 ? x1 : 0.f;
          }
        }
      }
    }
  }
  // row sums over the four lanes of a row
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      l[t][half] += __shfl_xor_sync(0xffffffffu, l[t][half], 1);
      l[t][half] += __shfl_xor_sync(0xffffffffu, l[t][half], 2);
    }
  if (WN > 1) {  // the key groups' sums joined through shared memory (q and the tiles are no longer needed)
    float* ml = reinterpret_cast<float*>(smem);  // [WN][RT][2], then o [RT][D]
    float* os = ml + WN * RT * 2;
    __syncthreads();
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int r = wm * 16 + g8 + 8 * half;
      if (q4 == 0) ml[(wn * RT + r) * 2] = m[0][half], ml[(wn * RT + r) * 2 + 1] = l[0][half];
    }
    __syncthreads();
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int r = wm * 16 + g8 + 8 * half;
      float mx = -INFINITY, sum = 0.f;
      for (int w = 0; w < WN; ++w) mx = fmaxf(mx, ml[(w * RT + r) * 2]);
      const float ref = mx == -INFINITY ? 0.f : mx;
      for (int w = 0; w < WN; ++w) sum = fmaf(ml[(w * RT + r) * 2 + 1], exp2_sfu(ml[(w * RT + r) * 2] - ref), sum);
      const float f = exp2_sfu(m[0][half] - ref);
#pragma unroll
      for (int d = 0; d < DT; ++d) o[0][d][2 * half] *= f, o[0][d][2 * half + 1] *= f;
      m[0][half] = mx, l[0][half] = sum;
    }
    for (int w = 0; w < WN; ++w) {
      if (wn == w)
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            float2* p = reinterpret_cast<float2*>(os + (wm * 16 + g8 + 8 * half) * D + 8 * d + 2 * q4);
            float2 x = make_float2(o[0][d][2 * half], o[0][d][2 * half + 1]);
            if (w > 0) x.x += p->x, x.y += p->y;
            if (w + 1 < WN)
              *p = x;
            else
              o[0][d][2 * half] = x.x, o[0][d][2 * half + 1] = x.y;
          }
      __syncthreads();
    }
    if (wn != WN - 1) return;
  }
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int row = r0 + (wm * MT + t) * 16 + g8 + 8 * half;
      if (row >= rows) continue;
      const int node = row / a.g, j = row % a.g;
      const long long qrow = ((long long)s * a.n + node) * a.Hq + kvh * a.g + j;
      if (a.splits == 1) {
        const float inv = 1.f / l[t][half];
        uint16_t* p = a.o + ((long long)s * a.n + node) * a.ldo + (kvh * a.g + j) * D + 2 * q4;
#pragma unroll
        for (int d = 0; d < DT; ++d)
          *reinterpret_cast<uint32_t*>(p + 8 * d) = pack_bf16x2(o[t][d][2 * half] * inv, o[t][d][2 * half + 1] * inv);
      } else {
        float* p = a.part + (qrow * a.splits + sp) * D + 2 * q4;
#pragma unroll
        for (int d = 0; d < DT; ++d)
          *reinterpret_cast<float2*>(p + 8 * d) = make_float2(o[t][d][2 * half], o[t][d][2 * half + 1]);
        if (q4 == 0)
          *reinterpret_cast<float2*>(a.part_ml + (qrow * a.splits + sp) * 2) = make_float2(m[t][half], l[t][half]);
      }
    }
}

// o = sum over the splits of 2^(m_i - m) o_i / sum of 2^(m_i - m) l_i; a warp per query row, D / 32 columns a lane
template <int D>
__global__ void __launch_bounds__(128) combine_kernel(AttendArgs a) {
  const long long row = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);  // (s, node, head)
  const int lane = threadIdx.x & 31;
  if (row >= (long long)a.S * a.n * a.Hq) return;
  const long long tok = row / a.Hq;
  const int head = (int)(row % a.Hq), s = (int)(tok / a.n);
  int len = a.cache_len[s];
  if (len < 0 || len > a.max_len || (long long)len > ((long long)a.max_pages << a.page_shift)) len = 0;
  const int ns = ((len + KT - 1) / KT + 1 + a.tps - 1) / a.tps;  // splits that had a tile
  const float2* ml = reinterpret_cast<const float2*>(a.part_ml) + row * a.splits;
  float mx = -INFINITY;
  for (int i = lane; i < ns; i += 32) mx = fmaxf(mx, ml[i].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  const float ref = mx == -INFINITY ? 0.f : mx;
  constexpr int V = D / 32;
  float acc[V] = {};
  float sum = 0.f;
  const float* p = a.part + row * a.splits * D + lane * V;
#pragma unroll 4
  for (int i = 0; i < ns; ++i) {
    const float2 e = ml[i];
    const float f = exp2_sfu(e.x - ref);
    sum = fmaf(f, e.y, sum);
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] = fmaf(f, p[(long long)i * D + v], acc[v]);
  }
  const float inv = 1.f / sum;
  uint16_t* o = a.o + tok * a.ldo + head * D + lane * V;
#pragma unroll
  for (int v = 0; v < V; v += 2) *reinterpret_cast<uint32_t*>(o + v) = pack_bf16x2(acc[v] * inv, acc[v + 1] * inv);
}

// Rows per CTA and splits of the keys.
struct AttendPlan {
  int rt, row_tiles, tps, splits;
};
AttendPlan plan_attend(int S, int n, int Hq, int Hkv, int max_len) {
  AttendPlan p;
  const int rows = n * (Hq / Hkv);
  p.rt = rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128;
  p.row_tiles = (rows + p.rt - 1) / p.rt;
  const int nt = (max_len + KT - 1) / KT + 1;
  const long long items = (long long)S * Hkv * p.row_tiles, slots = 2 * kSMs;
  // tiles per split so that the waves of CTAs take least, a split costing about three tiles beside its own
  double best = 1e300;
  p.tps = nt, p.splits = 1;
  for (int sp = 1; sp <= 64 && sp <= nt; ++sp) {
    const int tps = (nt + sp - 1) / sp, used = (nt + tps - 1) / tps;
    const long long waves = (items * used + slots - 1) / slots;
    const double est = (double)waves * (tps + 3.0) + (used > 1 ? 2.0 + 0.1 * used : 0.0);
    if (est < best * 0.999) best = est, p.tps = tps, p.splits = used;
  }
  return p;
}

template <int D, int WM, int MT>
cudaError_t run_attend(const AttendArgs& a, const AttendPlan& p, cudaStream_t s) {
  using Sh = AttendShape<D, WM, MT>;
  cudaError_t e =
      cudaFuncSetAttribute(attend_kernel<D, WM, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::SMEM);
  if (e != cudaSuccess) return e;
  attend_kernel<D, WM, MT>
      <<<dim3((unsigned)p.splits, (unsigned)a.Hkv, (unsigned)(a.S * p.row_tiles)), ATHREADS, Sh::SMEM, s>>>(a);
  return cudaGetLastError();
}
template <int D>
cudaError_t run_attend_d(const AttendArgs& a, const AttendPlan& p, cudaStream_t s) {
  cudaError_t e = p.rt == 16   ? run_attend<D, 1, 1>(a, p, s)
                  : p.rt == 32 ? run_attend<D, 2, 1>(a, p, s)
                  : p.rt == 64 ? run_attend<D, 4, 1>(a, p, s)
                               : run_attend<D, 4, 2>(a, p, s);
  if (e != cudaSuccess || p.splits == 1) return e;
  const long long rows = (long long)a.S * a.n * a.Hq;
  combine_kernel<D><<<(unsigned)((rows + 3) / 4), 128, 0, s>>>(a);
  return cudaGetLastError();
}

// A cluster of 8 CTAs for each sequence: together they copy its path's rows; its length is written by one of them
// once all eight have read it, so len_out may be cache_len.
constexpr int CCTAS = 8, CTHREADS = 256;
__global__ void __cluster_dims__(CCTAS, 1, 1) __launch_bounds__(CTHREADS) kv_commit_kernel(KvCommitArgs a) {
  const int s = blockIdx.y, part = blockIdx.x;
  __shared__ int rows_s;
  const int len = a.cache_len[s];
  if (threadIdx.x < 32) {  // the path's length: up to its first bad entry, and what the pages hold
    const int lane = threadIdx.x;
    int want = a.path_len[s], bits = 0;
    if (want < 0 || want > a.max_path) bits |= SSM_STATUS_PATH_RANGE, want = want < 0 ? 0 : a.max_path;
    const long long room = ((long long)a.max_pages << a.page_shift) - len;
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
  const AttendPlan p = plan_attend(S, n, Hq, Hkv, max_len);
  return 256 + (p.splits > 1 ? (size_t)S * n * Hq * p.splits * (D + 2) * sizeof(float) : 0);
}

cudaError_t launch_tree_attention(const AttendArgs& args, void* workspace, cudaStream_t s) {
  if (args.S == 0) return cudaSuccess;
  AttendArgs a = args;
  const AttendPlan p = plan_attend(a.S, a.n, a.Hq, a.Hkv, a.max_len);
  a.tps = p.tps, a.splits = p.splits;
  a.part = static_cast<float*>(workspace);
  a.part_ml = a.part + (size_t)a.S * a.n * a.Hq * p.splits * a.D;
  return a.D == 64 ? run_attend_d<64>(a, p, s) : run_attend_d<128>(a, p, s);
}

cudaError_t launch_kv_commit(const KvCommitArgs& a, cudaStream_t s) {
  if (a.S == 0) return cudaSuccess;
  kv_commit_kernel<<<dim3(CCTAS, (unsigned)a.S), CTHREADS, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace ssmtree
