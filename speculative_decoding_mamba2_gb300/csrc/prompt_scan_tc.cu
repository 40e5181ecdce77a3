// The chunked scan of prompts on the 5th-generation tensor cores (long prompts; the formulas are in prompt_scan.cu).
//
// A CTA walks the 64-token chunks of a pair of heads that share B and C, everything transposed so that a row of
// tensor memory is one (head, p) of the pair's 128 and one thread owns it:
//     S [128 x 128]  = Xw [128 x 64 tokens] . B [64 x n]       what the chunk adds to the state; Xw = (w_t x_t)^T is
//                      written by its threads into tensor memory in three bf16 parts (24 bits), B is read MN-major
//     Y2 [128 x 64]  = h [128 x n] . C^T                       h rounded to bf16, in tensor memory
//     Y1 [128 x 64]  = x^T [128 x 64] . P^T                    for each head of the pair, P = scores with their decays
//     y = Y1 + e^{S_t} Y2 + D x,   h' = decay h + S            (h in fp32 registers for the whole walk)
// Scores and decays of the chunks are the same for every walk of them, so prep_kernel makes them first, into the
// workspace.  16 warps then walk through a chunk's steps together -- h' from S, Xw of the next chunk, y, h for the tensor
// cores, P of the next chunk -- while one warp issues the MMAs that the steps hand over and one the copies (TMA, three
// stages): the 128 rows of tensor memory are four warps, and the four groups of four share out tokens or columns.  (Warps
// specialised by step, tried first, each ran their own code: 4000 cycles a chunk, most of them waiting for instructions.)
// MMAs run in the order they are issued: S, Y2, Y1.  Every wait is bounded: on a time-out all warps leave, the copies and
// MMAs in flight are waited for (bounded again) and the tensor memory is freed.
// Rounding: h, P and y to bf16 once each (h and P as operands, relative to themselves); the state's own chain -- decays, Xw, S,
// h -- keeps 24 bits.
// Measured: 24571 tokens of 16 prompts, 80 heads, 237 us back to back (604 MB: 2.5 TB/s; 19 us of it prep_kernel); one prompt of
// 8191 tokens 111 us.  The walk is bound by its 16 warps' instructions: issue slots 64 % taken, the tensor pipe busy 38 % of
// the time (46 % with the walks over states).  A warp for each kind of MMA, scalar instead of paired fp32 and two waits in one
// changed nothing.
#include "prompt.cuh"
#include "umma.cuh"

namespace ssmtree {
namespace {

constexpr int Q = 64, WARPS = 16, NT = 32 * WARPS + 64, STAGES = 3;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLeast2 = -120.f * kLog2e;  // as kLeast of prompt_scan.cu, in powers of two

// shared memory: stages of C | B | x (two 64-column blocks each), P, y, decays, barriers
constexpr int BLK = Q * 128;  // a 64 x 64 bf16 block with 128-byte rows
constexpr int ST_BYTES = 6 * BLK, OFF_TB = 2 * BLK, OFF_TX = 4 * BLK;
constexpr int OFF_P = STAGES * ST_BYTES;   // [2][head][BLK]
constexpr int OFF_Y = OFF_P + 4 * BLK;     // [2][64][256]
constexpr int OFF_D = OFF_Y + 4 * BLK;     // [STAGES][head] decay records
constexpr int REC = 1408;                  // bytes of one
constexpr int OFF_ODD = OFF_D + STAGES * 2 * REC;
// Which x are not finite, of chunk i at [i & 3]: written with Xw, read with y.  Two places would not do: a group may write chunk
// i + 1's while another is still at y of chunk i - 1 (it needs S of chunk i, which needs nothing of that y), but not i + 2's.
struct Odd {
  // of a group's 16 tokens and a row, only where its warp has such an x: 2 bits a token, finite, +infinity, -infinity, NaN (y may
  // stand in the place of x when it is needed)
  uint32_t tokens[4][4][128];
  int warp[4][WARPS];          // the last chunk in which a warp has
  int chunk[4];                // in which any has
};
constexpr int OFF_BAR = OFF_ODD + sizeof(Odd);
constexpr int TC_SMEM = OFF_BAR + 256 + 1024 /* alignment */;

// tensor memory columns
constexpr int T_S = 0, T_Y2 = 128, T_Y1 = 192, T_XW = 320, T_H = 416;

struct Decays {  // of one head and chunk (exponents in powers of two)
  float S[64];   // sum from the start of the token's block of 16 up to it
  float D[64];   // step size
  float b[64];   // 2^(sum after the token in its block) D
  float w[64];   // 2^(sum after the token) D
  float e[64];   // 2^(sum up to the token)
  float total, pad[31];  // 2^(sum of the chunk)
};
static_assert(sizeof(Decays) == REC, "record size");

struct Bars {
  unsigned long long full[STAGES], free_[STAGES], s_full, y_full, drain;
  uint32_t tmem;
  int stop;
};
// named barriers: 1 .. 4 a group's y, then all workers, and what they hand to the MMA warp
constexpr int B_ALL = 5, B_XW = 6, B_H = 7, B_P = 8, HANDED = 32 * WARPS + 32;
__device__ __forceinline__ void hand_over(int id) { asm volatile("bar.arrive %0, %1;\n" ::"r"(id), "n"(HANDED) : "memory"); }
static_assert(sizeof(Bars) <= 256, "barrier space");

// x w = hi + mid + lo in bf16 (an infinity: hi alone), for a pair of bf16 values x
__device__ __forceinline__ void scale_split3(uint32_t x, unsigned long long w, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
  const unsigned long long minus1 = 0xbf800000bf800000ull;
  const unsigned long long u = fmul2(pack2(bf16_lo(x), bf16_hi(x)), w);
  const float2 a = unpack2(u);
  hi = pack_bf16x2(a.x, a.y);
  const unsigned long long r = ffma2(pack2(bf16_lo(hi), bf16_hi(hi)), minus1, u);
  const float2 b = unpack2(r);
  mid = pack_bf16x2(b.x, b.y);
  const float2 c = unpack2(ffma2(pack2(bf16_lo(mid), bf16_hi(mid)), minus1, r));
  lo = pack_bf16x2(c.x, c.y);
}

// Xw = x w of 32 rows (a head's columns) and 16 tokens, three bf16 parts of 32 columns of tensor memory each.  False where an
// x is not finite: an infinity is then its own first part, which the careful form sees to.
template <bool CAREFUL>
__device__ __forceinline__ bool write_xw(uint32_t x, const uint32_t (&f_off)[2], const float* w, int q4, uint32_t to) {
  const unsigned long long w0 = *reinterpret_cast<const unsigned long long*>(w + 2 * q4);
  const unsigned long long w1 = *reinterpret_cast<const unsigned long long*>(w + 8 + 2 * q4);
  uint32_t chk = 0;  // sum of 0 x, in pairs: NaN once an x is not finite
#pragma unroll CAREFUL ? 1 : 2
  for (int rh = 0; rh < 2; ++rh) {  // 16 rows, 16 tokens
    uint32_t xf[4], hi[4], mid[4], lo[4];
    ldsm4_t(xf, x + (rh ? f_off[1] : f_off[0]));
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      scale_split3(xf[j], j < 2 ? w0 : w1, hi[j], mid[j], lo[j]);
      if (CAREFUL) {
        if ((hi[j] & 0x7f80u) == 0x7f80u) mid[j] &= 0xffff0000u, lo[j] &= 0xffff0000u;
        if ((hi[j] & 0x7f800000u) == 0x7f800000u) mid[j] &= 0xffffu, lo[j] &= 0xffffu;
      } else {
        asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(chk) : "r"(xf[j]), "r"(0u));
      }
    }
    const uint32_t at = to + ((uint32_t)(16 * rh) << 16);
    tmem_st_frag(at, lo);
    tmem_st_frag(at + 32, mid);
    tmem_st_frag(at + 64, hi);
  }
  return !__any_sync(0xffffffffu, chk & 0x7fff7fffu);
}

// Once for all walks: grid z < G: scores C_t . B_s of a chunk and group, [record][s / 4][t][s % 4] fp32; then the decays
// of a chunk, HEADS heads to a warp.
// A record for each chunk of sequences that share no row, in whatever order they stand: whole chunks by the one row before a
// multiple of Q in them, a sequence's shorter last one by the sequence.
__device__ __forceinline__ long long chunk_record(const SeqArgs& q, int s, int first, int len, int chunk) {
  return (chunk + 1) * Q <= len ? first / Q + chunk : (long long)(q.n_tok / Q) + s;
}
// of a warp: their chains of shuffles and exponentials fill each other's gaps (1: 239, 2: 236, 4: 235.6 us of a scan)
constexpr int HEADS = 4;
__global__ void __launch_bounds__(128) prep_kernel(ScanArgs a, float* scores, Decays* decays, int* order) {
  __shared__ __align__(128) unsigned char sm[2 * Q * kN * 2];
  launch_dependents();
  const int c = blockIdx.x, s = blockIdx.y, grp = blockIdx.z, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (c == 0 && grp == 0) {  // the sequence's place in the order of the walks, longest first
    __shared__ int longer[4];
    const unsigned mine = (unsigned)a.q.cu[s + 1] - (unsigned)a.q.cu[s];
    int before = 0;
    for (int k = tid; k < a.q.n_seq; k += 128) {
      const unsigned l = (unsigned)a.q.cu[k + 1] - (unsigned)a.q.cu[k];
      before += l > mine || (l == mine && k < s);
    }
    before = __reduce_add_sync(0xffffffffu, before);
    if (lane == 0) longer[warp] = before;
    __syncthreads();
    if (tid == 0) order[longer[0] + longer[1] + longer[2] + longer[3]] = s;
  }
  int first, len, slot;
  if (!seq_range(a.q, s, first, len, slot) || c * Q >= len) return;
  if (grp >= a.G) {
    const int h0 = ((grp - a.G) * 4 + warp) * HEADS;
    const int t = c * Q + 2 * lane;  // tokens 2 lane, 2 lane + 1
    const uint16_t* q = a.dt + (long long)(first + t) * a.lddt + h0;
    float dt0[HEADS], dt1[HEADS];
#pragma unroll
    for (int j = 0; j < HEADS; ++j) {
      dt0[j] = h0 + j < a.H && t < len ? bf16f(q[j]) : 0.f;
      dt1[j] = h0 + j < a.H && t + 1 < len ? bf16f(q[a.lddt + j]) : 0.f;
    }
    Decays* rec = decays + chunk_record(a.q, s, first, len, c) * a.H + h0;
#pragma unroll
    for (int j = 0; j < HEADS; ++j) {
      if (h0 + j >= a.H) return;
      const float A2 = neg_exp(a.A_log[h0 + j]) * kLog2e, bias = a.dt_bias[h0 + j];
      const float d0 = t < len ? softplus_f(dt0[j] + bias) : 0.f;
      const float d1 = t + 1 < len ? softplus_f(dt1[j] + bias) : 0.f;
      const float e0 = fmaxf(d0 * A2, kLeast2), e1 = fmaxf(d1 * A2, kLeast2);
      float pre = e0 + e1, suf = pre;  // sums within the lane's block
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) {
        const float u = __shfl_up_sync(0xffffffffu, pre, o, 8), v = __shfl_down_sync(0xffffffffu, suf, o, 8);
        if ((lane & 7) >= o) pre += u;
        if ((lane & 7) + o < 8) suf += v;
      }
      float before = __shfl_up_sync(0xffffffffu, pre, 1, 8), after = __shfl_down_sync(0xffffffffu, suf, 1, 8);
      if ((lane & 7) == 0) before = 0.f;
      if ((lane & 7) == 7) after = 0.f;
      float base = 0.f, rest = 0.f, all = 0.f;  // of the blocks before the lane's, and after
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float v = __shfl_sync(0xffffffffu, pre, 8 * k + 7);
        all += v;
        if (k < lane >> 3) base += v;
        if (k > lane >> 3) rest += v;
      }
      Decays& d = rec[j];
      const float S0 = before + e0;
      *reinterpret_cast<float2*>(&d.S[2 * lane]) = make_float2(S0, pre);
      *reinterpret_cast<float2*>(&d.D[2 * lane]) = make_float2(d0, d1);
      const float a0 = after + e1;  // after token 2 lane, in its block
      *reinterpret_cast<float2*>(&d.b[2 * lane]) = make_float2(exp2_sfu(a0) * d0, exp2_sfu(after) * d1);
      *reinterpret_cast<float2*>(&d.w[2 * lane]) = make_float2(exp2_sfu(a0 + rest) * d0, exp2_sfu(after + rest) * d1);
      *reinterpret_cast<float2*>(&d.e[2 * lane]) = make_float2(exp2_sfu(base + S0), exp2_sfu(base + pre));
      if (lane == 0) d.total = exp2_sfu(all);
    }
    return;
  }
  const uint32_t sb = smem_u32(sm);
  for (int i = tid; i < Q * 16; i += 128) {
    const int row = i >> 4, ch = i & 15;
    const bool there = c * Q + row < len;
    const long long t = there ? first + c * Q + row : first;
    cp_async16_or_zero(sb + tile_off(row, ch, kN * 2), a.C + t * a.ldc + grp * kN + ch * 8, there);
    cp_async16_or_zero(sb + Q * kN * 2 + tile_off(row, ch, kN * 2), a.B + t * a.ldb + grp * kN + ch * 8, there);
  }
  cp_async_commit();
  cp_async_wait<0>();
  __syncthreads();
  float acc[8][4];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
  const int np1 = warp < 2 ? 2 : 4;  // tokens of the first half have no scores in the second
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    uint32_t cf[4];
    frag_a(cf, sb, kN * 2, 16 * warp, 16 * k, lane);
#pragma unroll
    for (int np = 0; np < 4; ++np)
      if (np < np1) {
        uint32_t b[4];
        frag_b2(b, sb + Q * kN * 2, kN * 2, 16 * np, 16 * k, lane);
        mma16816(acc[2 * np], cf, b[0], b[1]);
        mma16816(acc[2 * np + 1], cf, b[2], b[3]);
      }
  }
  float* out = scores + (chunk_record(a.q, s, first, len, c) * a.G + grp) * (Q * Q);
  const int t = 16 * warp + (lane >> 2);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < 2 * np1) {
      const int u = 8 * i + 2 * (lane & 3);
      float* p = out + (u >> 2) * (Q * 4) + (u & 3);
      *reinterpret_cast<float2*>(p + t * 4) = make_float2(acc[i][0], acc[i][1]);
      *reinterpret_cast<float2*>(p + (t + 8) * 4) = make_float2(acc[i][2], acc[i][3]);
    }
}

// Segment j of a sequence's nch chunks: chunks c0 .. c1 - 1.  With k = nseg - 1, the first is two fifths as long as the others:
// its walk, in the first grid, then takes as long as the others' walks over states beside it (1.55 and 0.62 us a chunk).
__device__ __forceinline__ void segment(int nch, int nseg, int j, int& c0, int& c1) {
  const int k = nseg - 1, b = (5 * nch + 5 * k + 1) / (5 * k + 2), f = nseg == 1 ? nch : max(0, nch - k * b);
  c0 = j == 0 ? 0 : f + (j - 1) * b;
  c1 = min(nch, j == 0 ? f : c0 + b);
}

__device__ __forceinline__ void walk(const CUtensorMap& tx, const CUtensorMap& tb, const CUtensorMap& tcm, const CUtensorMap& ty,
                                     const ScanArgs& a, const float* scores, const Decays* decays, const int* order, int rank, int seg) {
  extern __shared__ unsigned char smem_raw[];
  // (shuffles tell the compiler what is the same for a warp: it then keeps it in uniform registers)
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int pair = blockIdx.x;
  unsigned char* smem = smem_raw + (-smem_u32(smem_raw) & 1023u);  // stays a shared-memory pointer to the compiler
  const uint32_t sb = smem_u32(smem);
  Bars* bar = reinterpret_cast<Bars*>(smem + OFF_BAR);
  volatile int* stop = &bar->stop;

  if (tid == 0) {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(smem_u32(&bar->full[i]), 1);
      mbar_init(smem_u32(&bar->free_[i]), 2);
    }
    mbar_init(smem_u32(&bar->s_full), 1);
    mbar_init(smem_u32(&bar->y_full), 1);
    mbar_init(smem_u32(&bar->drain), 1);
    bar->stop = 0;
    fence_barrier_init();
  }
  Odd* marks = reinterpret_cast<Odd*>(smem + OFF_ODD);
  if (tid < 4 * (WARPS + 1)) (&marks->warp[0][0])[tid] = -1;
  // P's entries after their token stay zero
  for (int i = tid; i < 4 * BLK / 16; i += NT) reinterpret_cast<uint4*>(smem + OFF_P)[i] = make_uint4(0, 0, 0, 0);
  fence_async_smem();  // (each thread its own: the tensor cores read them)
  if (warp == WARPS) tmem_alloc_warp(smem_u32(&bar->tmem), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, bar->tmem, 0);
  grid_dependency_wait();  // scores, decays, the order, the states of the segments before
  const int s = __shfl_sync(0xffffffffu, order[rank], 0);
  int first, len, slot;
  const bool there = seq_range(a.q, s, first, len, slot);
  first = __shfl_sync(0xffffffffu, first, 0), len = __shfl_sync(0xffffffffu, len, 0), slot = __shfl_sync(0xffffffffu, slot, 0);
  const int nch = (len + Q - 1) / Q;
  int c0, c1;
  segment(nch, a.nseg, seg, c0, c1);
  const int n = max(0, c1 - c0);
  if (!there || (n == 0 && seg > 0)) {
    if (!there && pair == 0 && seg == 0 && tid == 0) flag(a.q.status, SSM_STATUS_SEQ_RANGE);
    if (warp == WARPS) tmem_free_warp(tmem, 512);
    return;
  }

  if (warp < WARPS) {
    const int w4 = warp & 3, grp4 = warp >> 2;        // rows 32 w4 .. of tensor memory; this group's share
    const uint32_t lanes = (uint32_t)(w4 * 32) << 16;
    const int row = w4 * 32 + lane, hd = row >> 6, p = row & 63, head = 2 * pair + hd;  // (head of the pair, p) of a thread
    const int q4 = lane & 3, p0 = (w4 & 1) * 32;      // the warp's first column of its head's x
    const int tg = 16 * grp4;                         // the group's first token of a chunk
    const int n0 = 32 * grp4;                         // its first column of the state
    auto x_at = [&](unsigned char* stage, int t) {    // x of token t in column p: chunk (p >> 3) ^ (t & 7) of the tile's row
      return reinterpret_cast<uint16_t*>(stage + OFF_TX + hd * BLK + t * 128 + (((p >> 3) ^ (t & 7)) << 4) + (p & 7) * 2);
    };
    // this lane's row of the 8 x 8 matrices of 16 tokens x 16 columns, in a stage's x and in a buffer of y
    const int fr = tg + (lane & 7) + ((lane >> 4) << 3), fc = (p0 >> 3) + ((lane >> 3) & 1);
    const uint32_t f_off[2] = {(uint32_t)(hd * BLK) + tile_off(fr, fc, 128), (uint32_t)(hd * BLK) + tile_off(fr, fc + 2, 128)};

    // the state: columns n0 .. n0 + 31 of the thread's row
    const long long at = (((long long)slot * a.L + a.layer) * a.H + head) * (kP * kN) + p * kN + n0;
    const long long wrec = kP * kN + 32;
    float* ws = a.seg_state + ((long long)s * a.H + head) * (a.nseg - 1) * wrec;
    float h[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) h[j] = 0.f;
    // from the caller's state, or from that after the first segment and what those between add (the caller's, which may be
    // written in place, is read by the first segment alone, in an earlier grid than its last write)
    const float* from = seg == 0 ? (a.h_in ? a.h_in + at : nullptr) : ws + p * kN + n0;
    if (from) {
#pragma unroll
      for (int j = 0; j < 32; j += 4) {
        const float4 v = *reinterpret_cast<const float4*>(from + j);
        h[j] = v.x, h[j + 1] = v.y, h[j + 2] = v.z, h[j + 3] = v.w;
      }
    }
#pragma unroll 1
    for (int k = 1; k < seg; ++k) {
      const float* r = ws + k * wrec;
      const float dk = r[kP * kN];
      r += p * kN + n0;
#pragma unroll
      for (int j = 0; j < 32; j += 4) {
        const float4 v = *reinterpret_cast<const float4*>(r + j);
        h[j] = fmaf(dk, h[j], v.x), h[j + 1] = fmaf(dk, h[j + 1], v.y);
        h[j + 2] = fmaf(dk, h[j + 2], v.z), h[j + 3] = fmaf(dk, h[j + 3], v.w);
      }
    }
    float* out = c1 == nch ? a.h_out + at : seg == 0 ? ws + p * kN + n0 : nullptr;  // for the state at the end
    const float Dh = a.D[head];
    const unsigned long long D2 = pack2(Dh, Dh);

    // P, in blocks of 16 x 16 tokens: a warp makes half of one on the diagonal (4 entries a thread), and twelve of them one
    // below it (8 entries a thread); above it there are zeros
    const int lr = lane & 15, lh = lane >> 4;
    const int dh = warp >> 3, db = (warp >> 1) & 3, dt = 16 * db + lr, du = 16 * db + 8 * (warp & 1) + 4 * lh;
    const bool below = warp < 12;
    const int oh = warp / 6, oj = warp % 6, tb = oj < 3 ? oj + 1 : oj == 3 ? 2 : 3, ub = oj < 3 ? 0 : oj < 5 ? 1 : 2;
    const int ot = 16 * tb + lr, ou = 16 * ub + 8 * lh;
    float4 gd, go[2];
    const float4* gp = reinterpret_cast<const float4*>(scores) + ((first / Q + c0) * (long long)a.G + 2 * pair / (a.H / a.G)) * (Q * Q / 4);
    auto fetch = [&](bool whole) {
      if (!whole) gp += (a.q.n_tok / Q + s - first / Q - nch + 1) * (long long)a.G * (Q * Q / 4);  // the sequence's last chunk
      gd = gp[(du >> 2) * Q + dt];
      if (below) go[0] = gp[(ou >> 2) * Q + ot], go[1] = gp[((ou >> 2) + 1) * Q + ot];
      gp += (long long)a.G * (Q * Q / 4);
    };
    const uint32_t d_off = (uint32_t)(OFF_P + dh * BLK + dt * 128 + (((du >> 3) ^ (dt & 7)) << 4) + (du & 7) * 2);
    const uint32_t o_off = (uint32_t)(OFF_P + oh * BLK + ot * 128 + (((ou >> 3) ^ (ot & 7)) << 4));

    bool ok = true;
    uint32_t cur = 0, nxt = 0, nd = OFF_D, cd = OFF_D, full_par = 0;  // stages (and decays) of chunks i and i + 1
    unsigned long long* full = bar->full;
    int left = len - c0 * Q;                                         // tokens from chunk i + 1 on
#pragma unroll 1
    for (int i = -1; i < n; ++i) {
      // ---- h' = decay h + S of chunk i ----
      if (i >= 0) {
        ok = wait_bar(&bar->s_full, i & 1, stop);
        if (!ok) break;
        tc_fence_after();
        float v0[16], v1[16];
        tmem_ld16_async(tmem + T_S + lanes + n0, v0);
        tmem_ld16_async(tmem + T_S + lanes + n0 + 16, v1);
        const float f = reinterpret_cast<const Decays*>(smem + cd)[hd].total;
        const unsigned long long f2 = pack2(f, f);
        tmem_wait_ld16(v0);
        tmem_wait_ld16(v1);
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
          const float2 u = unpack2(ffma2(f2, pack2(h[j], h[j + 1]), pack2(v0[j], v0[j + 1])));
          const float2 z = unpack2(ffma2(f2, pack2(h[16 + j], h[17 + j]), pack2(v1[j], v1[j + 1])));
          h[j] = u.x, h[j + 1] = u.y, h[16 + j] = z.x, h[17 + j] = z.y;
        }
      }
      // ---- Xw of chunk i + 1 (the MMAs that read the last one are done) ----
      if (i + 1 < n) {
        ok = wait_bar(full, full_par, stop);
        if (!ok) break;
        if (left < Q) {  // rows of B and x after the sequence's last belong to another one
          for (int k = tid; k < (Q - left) * 32; k += 32 * WARPS) {
            const int r = left + (k >> 5), blk = (k >> 3) & 3, ch = k & 7;
            *reinterpret_cast<uint4*>(smem + nxt + OFF_TB + blk * BLK + r * 128 + ch * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_async_smem();
          named_sync(B_ALL, 32 * WARPS);
        }
        const float* w = reinterpret_cast<const Decays*>(smem + nd)[hd].w + tg;
        const uint32_t xw = tmem + T_XW + lanes + (tg >> 1);
        if (!write_xw<false>(sb + nxt + OFF_TX, f_off, w, q4, xw)) {  // seldom
          write_xw<true>(sb + nxt + OFF_TX, f_off, w, q4, xw);
          // such values leave the tile (each thread its row's): the product with a zero of P would spread them
          uint32_t odd = 0;
#pragma unroll 1
          for (int u = 0; u < 16; ++u) {
            uint16_t* v = x_at(smem + nxt, tg + u);
            const uint32_t b = *v;
            if ((b & 0x7f80u) == 0x7f80u) odd |= (b & 0x7fu ? 3u : b & 0x8000u ? 2u : 1u) << (2 * u), *v = 0;
          }
          fence_async_smem();
          marks->tokens[(i + 1) & 3][grp4][row] = odd;
          marks->warp[(i + 1) & 3][warp] = i + 1;
          marks->chunk[(i + 1) & 3] = i + 1;
        }
        // the store of the chunk before this one's y has read its buffer
        if (w4 == 0) asm volatile("cp.async.bulk.wait_group.read 0;\n" ::: "memory");
        tmem_wait_st();
        tc_fence_before();
        hand_over(B_XW);
        fetch(left >= Q);  // for P below: the loads' time passes during y
      }
      // ---- y of chunk i ----
      if (i >= 0) {
        const Decays& d = reinterpret_cast<const Decays*>(smem + cd)[hd];
        const uint32_t yb = OFF_Y + (uint32_t)(i & 1) * 2 * BLK;
        const unsigned long long e0 = *reinterpret_cast<const unsigned long long*>(&d.e[tg + 2 * q4]);
        const unsigned long long e1 = *reinterpret_cast<const unsigned long long*>(&d.e[tg + 8 + 2 * q4]);
        uint32_t xf[2][4];
        ldsm4_t(xf[0], sb + cur + OFF_TX + f_off[0]);
        ldsm4_t(xf[1], sb + cur + OFF_TX + f_off[1]);
        ok = wait_bar(&bar->y_full, i & 1, stop);
        if (!ok) break;
        tc_fence_after();
        float y1[2][8], y2[2][8];
#pragma unroll
        for (int rh = 0; rh < 2; ++rh) {  // 16 rows, 16 tokens
          const uint32_t from = tmem + lanes + ((uint32_t)(16 * rh) << 16) + tg;
          tmem_ld_frag_async(from + T_Y1 + hd * 64, y1[rh]);
          tmem_ld_frag_async(from + T_Y2, y2[rh]);
        }
#pragma unroll
        for (int rh = 0; rh < 2; ++rh) {
          uint32_t o[4];
          tmem_wait_ld8(y1[rh], y2[rh]);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 y = unpack2(ffma2(D2, pack2(bf16_lo(xf[rh][j]), bf16_hi(xf[rh][j])),
                                           ffma2(j < 2 ? e0 : e1, pack2(y2[rh][2 * j], y2[rh][2 * j + 1]),
                                                 pack2(y1[rh][2 * j], y1[rh][2 * j + 1]))));
            o[j] = pack_bf16x2(y.x, y.y);
          }
          stsm4_t(sb + yb + f_off[rh], o);
        }
        if (marks->chunk[i & 3] == i) {  // what those values add is not finite, so it can be added to the rounded y
          __syncwarp();
          const unsigned char* pt = smem + OFF_P + ((i & 1) * 2 + hd) * BLK;
#pragma unroll 1
          for (int u = 0; u < tg + 16; ++u) {
            if (marks->warp[i & 3][(u >> 4) * 4 + w4] != i) continue;
            const uint32_t what = marks->tokens[i & 3][u >> 4][row] >> (2 * (u & 15)) & 3u;
            if (what == 0) continue;
            // (the bits of what: with an infinity's exponent there, its upper one is the sign)
            const float xv = __uint_as_float(0x7f800000u | what << 30 | (what == 3 ? 1u << 22 : 0u));
#pragma unroll 1
            for (int r = max(u, tg); r < tg + 16; ++r) {
              uint16_t* y = reinterpret_cast<uint16_t*>(smem + yb + hd * BLK + tile_off(r, p >> 3, 128) + (p & 7) * 2);
              const uint16_t w = *reinterpret_cast<const uint16_t*>(pt + r * 128 + (((u >> 3) ^ (r & 7)) << 4) + (u & 7) * 2);
              float v = fmaf(bf16f(w), xv, bf16f(*y));
              if (r == u) v = fmaf(Dh, xv, v);
              *y = (uint16_t)(pack_bf16x2(v, 0.f) & 0xffffu);
            }
          }
        }
        tc_fence_before();
        fence_async_smem();
        named_sync(1 + grp4, 128);  // the group's 16 rows of y are in shared memory
        const int valid = left + Q - tg;  // of the group's tokens
        if (valid >= 16) {
          if (w4 == 0 && lane == 0) {
            tma_store_2d(&ty, sb + yb + tg * 128, 2 * pair * kP, first + (c0 + i) * Q + tg);
            tma_store_2d(&ty, sb + yb + BLK + tg * 128, 2 * pair * kP + 64, first + (c0 + i) * Q + tg);
            asm volatile("cp.async.bulk.commit_group;\n" ::: "memory");
          }
        } else {  // the rows after the last are another sequence's
          uint16_t* yo = a.y + (long long)(first + (c0 + i) * Q) * a.ldy + pair * 2 * kP;
#pragma unroll 1
          for (int k = tid & 127; k < valid * 16; k += 128) {
            const int r = tg + (k >> 4), ch = k & 15;
            *reinterpret_cast<uint4*>(yo + (long long)r * a.ldy + ch * 8) =
                *reinterpret_cast<const uint4*>(smem + yb + (ch >> 3) * BLK + tile_off(r, ch & 7, 128));
          }
        }
      }
      if (i + 1 >= n) break;
      // ---- the state for the next chunk's y, rounded to bf16 (y2 of this chunk, which read the last, is done) ----
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        uint32_t v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = pack_bf16x2(h[16 * k + 2 * j], h[16 * k + 2 * j + 1]);
        tmem_st8(tmem + T_H + lanes + (n0 >> 1) + 8 * k, v);
      }
      tmem_wait_st();
      tc_fence_before();
      hand_over(B_H);
      // ---- P of chunk i + 1 ----
      const uint32_t buf = ((i + 1) & 1) * 2 * BLK;
      {  // 2^(S_t - S_u) D_u
        const Decays& d = reinterpret_cast<const Decays*>(smem + nd)[dh];
        const float St = d.S[dt];
        const float4 S = *reinterpret_cast<const float4*>(&d.S[du]), D = *reinterpret_cast<const float4*>(&d.D[du]);
        const float w0 = du <= dt ? gd.x * (exp2_sfu(St - S.x) * D.x) : 0.f;
        const float w1 = du + 1 <= dt ? gd.y * (exp2_sfu(St - S.y) * D.y) : 0.f;
        const float w2 = du + 2 <= dt ? gd.z * (exp2_sfu(St - S.z) * D.z) : 0.f;
        const float w3 = du + 3 <= dt ? gd.w * (exp2_sfu(St - S.w) * D.w) : 0.f;
        *reinterpret_cast<uint2*>(smem + d_off + buf) = make_uint2(pack_bf16x2(w0, w1), pack_bf16x2(w2, w3));
      }
      if (below) {  // to the end of u's block, and from there
        const Decays& d = reinterpret_cast<const Decays*>(smem + nd)[oh];
        float x = d.S[ot];
        if (tb - ub > 1) x += d.S[16 * tb - 1];
        if (tb - ub > 2) x += d.S[16 * tb - 17];
        const float E = exp2_sfu(x);
        const float4 f0 = *reinterpret_cast<const float4*>(&d.b[ou]), f1 = *reinterpret_cast<const float4*>(&d.b[ou + 4]);
        *reinterpret_cast<uint4*>(smem + o_off + buf) = make_uint4(
            pack_bf16x2(go[0].x * (f0.x * E), go[0].y * (f0.y * E)), pack_bf16x2(go[0].z * (f0.z * E), go[0].w * (f0.w * E)),
            pack_bf16x2(go[1].x * (f1.x * E), go[1].y * (f1.y * E)), pack_bf16x2(go[1].z * (f1.z * E), go[1].w * (f1.w * E)));
      }
      fence_async_smem();
      hand_over(B_P);
      cur = nxt, cd = nd, left -= Q;
      nxt += ST_BYTES, nd += 2 * REC, ++full;
      if (nxt == STAGES * ST_BYTES) nxt = 0, nd = OFF_D, full = bar->full, full_par ^= 1;
    }
    if (w4 == 0) asm volatile("cp.async.bulk.wait_group 0;\n" ::: "memory");
    if (!ok) {  // a warp that gives up still takes part in the barriers that others may be waiting at
      asm volatile("bar.arrive %0, %1;\n" ::"r"(1 + grp4), "n"(128) : "memory");
      asm volatile("bar.arrive %0, %1;\n" ::"n"(B_ALL), "n"(32 * WARPS) : "memory");
      hand_over(B_XW);
      hand_over(B_H);
      hand_over(B_P);
    }
    if (ok && out) {
#pragma unroll
      for (int j = 0; j < 32; j += 4) *reinterpret_cast<float4*>(out + j) = make_float4(h[j], h[j + 1], h[j + 2], h[j + 3]);
    }
  } else if (warp == WARPS + 1) {
    // ---- copies ----
    int issued = 0;
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      const int st = i % STAGES;
      if (i >= STAGES && !wait_bar(&bar->free_[st], (i / STAGES - 1) & 1, stop)) break;
      if (lane == 0) {
        const uint32_t f = smem_u32(&bar->full[st]), d = sb + st * ST_BYTES;
        const int t = first + (c0 + i) * Q, bn = 2 * pair / (a.H / a.G) * kN;
        mbar_arrive_expect_tx(f, ST_BYTES + 2 * REC);
        tma_load_2d(d + OFF_TX, &tx, 2 * pair * kP, t, f);
        tma_load_2d(d + OFF_TX + BLK, &tx, 2 * pair * kP + 64, t, f);
        bulk_load(sb + OFF_D + st * 2 * REC, decays + chunk_record(a.q, s, first, len, c0 + i) * a.H + 2 * pair, 2 * REC, f);
        tma_load_2d(d + OFF_TB, &tb, bn, t, f);
        tma_load_2d(d + OFF_TB + BLK, &tb, bn + 64, t, f);
        tma_load_2d(d, &tcm, bn, t, f);
        tma_load_2d(d + BLK, &tcm, bn + 64, t, f);
      }
      issued = i + 1;
    }
    // copies land before the shared memory is given up, whoever gives up, and when
    for (int i = max(0, issued - STAGES); i < issued && lane == 0; ++i) mbar_wait(smem_u32(&bar->full[i % STAGES]), (i / STAGES) & 1);
  } else {
    // ---- MMAs ----
    constexpr uint32_t id_s = idesc_major(128, 128, false, true), id_y2 = idesc_major(128, 64, false, false),
                       id_y1 = idesc_major(128, 64, true, false);
    const bool leader = elect_one();
    uint32_t tile = sb, pd = desc_lo(sb + OFF_P, 16);
    unsigned long long *fr = bar->free_, *last = nullptr;  // stages of this chunk and the one before
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      named_sync(B_XW, HANDED);  // Xw of this chunk; S of the last has been read
      if (*stop) break;
      tc_fence_after();
      if (leader) {
        const uint32_t bd = desc_lo(tile + OFF_TB, BLK);
#pragma unroll
        for (int k = 0; k < 4; ++k)  // 16 tokens: two groups of 8 rows
#pragma unroll
          for (int part = 0; part < 3; ++part)
            mma_ts<id_s>(tmem + T_S, tmem + T_XW + part * 32 + k * 8, bd + k * (2048 >> 4), k + part > 0);
        mma_commit(smem_u32(&bar->s_full));
      }
      __syncwarp();
      named_sync(B_H, HANDED);  // h; y of the last chunk has been read
      if (*stop) break;
      tc_fence_after();
      if (leader) {
        if (i > 0) mbar_arrive(smem_u32(last));
        const uint32_t cd = desc_lo(tile, 16);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          mma_ts<id_y2>(tmem + T_Y2, tmem + T_H + k * 8, cd + ((k >> 2) * (BLK >> 4) + (k & 3) * 2), k != 0);
      }
      __syncwarp();
      named_sync(B_P, HANDED);
      if (*stop) break;
      tc_fence_after();
      if (leader) {
        const uint32_t xd = desc_lo(tile + OFF_TX, BLK);
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_ss<id_y1>(tmem + T_Y1 + e * 64, xd + k * (2048 >> 4), pd + e * (BLK >> 4) + k * 2, k != 0);
        mma_commit(smem_u32(&bar->y_full));
      }
      __syncwarp();
      if (leader) mma_commit(smem_u32(fr));
      __syncwarp();
      last = fr;
      pd ^= desc_lo(sb + OFF_P, 16) ^ desc_lo(sb + OFF_P + 2 * BLK, 16);
      tile += ST_BYTES, ++fr;
      if (fr == bar->free_ + STAGES) fr = bar->free_, tile = sb;
    }
    if (leader) {
      mma_commit(smem_u32(&bar->drain));
      mbar_poll_ns(smem_u32(&bar->drain), 0, kWaitLimitNs);
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && *stop) flag(a.q.status, SSM_STATUS_TIMEOUT);
  if (warp == WARPS) {
    __syncwarp();
    tc_fence_after();
    tmem_free_warp(tmem, 512);
  }
}

// What a segment adds to the state, and its decay: the walk above without y.  Two chunks are under way, each with
// its own S and Xw in tensor memory: the S of one is made while the one before it is added up and the next one's Xw written
// (with one, 43 chunks took 55 us instead of 34, each step waiting for the one before).  Segments before a
// sequence's last have whole chunks only.
constexpr int S_STAGES = 6, S_BYTES = 4 * BLK;        // stages of B | x
constexpr int S_OFF_D = S_STAGES * S_BYTES, S_OFF_BAR = S_OFF_D + S_STAGES * 2 * REC;
constexpr int S_SMEM = S_OFF_BAR + 256 + 1024 /* alignment */;
constexpr int T_S2 = 0, T_XW2 = 256;                  // two of 128 columns, two of 96
struct StateBars {
  unsigned long long full[S_STAGES], free_[S_STAGES], s_full[2], drain;
  uint32_t tmem;
  int stop;
};
static_assert(sizeof(StateBars) <= 256 && S_SMEM <= TC_SMEM, "space");

__device__ __forceinline__ void state_walk(const CUtensorMap& tx, const CUtensorMap& tb, const ScanArgs& a, const Decays* decays,
                                           const int* order, int rank, int seg) {
  extern __shared__ unsigned char smem_raw[];
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int pair = blockIdx.x;
  unsigned char* smem = smem_raw + (-smem_u32(smem_raw) & 1023u);
  const uint32_t sb = smem_u32(smem);
  StateBars* bar = reinterpret_cast<StateBars*>(smem + S_OFF_BAR);
  volatile int* stop = &bar->stop;
  if (tid == 0) {
    for (int i = 0; i < S_STAGES; ++i) {
      mbar_init(smem_u32(&bar->full[i]), 1);
      mbar_init(smem_u32(&bar->free_[i]), 1);
    }
    mbar_init(smem_u32(&bar->s_full[0]), 1);
    mbar_init(smem_u32(&bar->s_full[1]), 1);
    mbar_init(smem_u32(&bar->drain), 1);
    bar->stop = 0;
    fence_barrier_init();
  }
  if (warp == WARPS) tmem_alloc_warp(smem_u32(&bar->tmem), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, bar->tmem, 0);
  grid_dependency_wait();  // decays, the order
  const int s = __shfl_sync(0xffffffffu, order[rank], 0);
  int first, len, slot;
  const bool there = seq_range(a.q, s, first, len, slot);
  first = __shfl_sync(0xffffffffu, first, 0), len = __shfl_sync(0xffffffffu, len, 0);
  const int nch = (len + Q - 1) / Q;
  int c0, c1;
  segment(nch, a.nseg, seg, c0, c1);
  const int n = c1 - c0;
  if (!there || c1 >= nch) {  // none behind it
    if (warp == WARPS) tmem_free_warp(tmem, 512);
    return;
  }

  if (warp < WARPS) {
    const int w4 = warp & 3, grp4 = warp >> 2;  // as in walk
    const uint32_t lanes = (uint32_t)(w4 * 32) << 16;
    const int row = w4 * 32 + lane, hd = row >> 6, p = row & 63, head = 2 * pair + hd;
    const int q4 = lane & 3, p0 = (w4 & 1) * 32, tg = 16 * grp4, n0 = 32 * grp4;
    const int fr = tg + (lane & 7) + ((lane >> 4) << 3), fc = (p0 >> 3) + ((lane >> 3) & 1);
    const uint32_t f_off[2] = {(uint32_t)(hd * BLK) + tile_off(fr, fc, 128), (uint32_t)(hd * BLK) + tile_off(fr, fc + 2, 128)};
    float h[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) h[j] = 0.f;
    float seg_decay = 1.f, f0 = 0.f, f1 = 0.f;  // decays of chunks i and i + 1
    bool ok = true;
    uint32_t st = 0, full_par = 0;  // stage of chunk i + 2
#pragma unroll 1
    for (int i = -2; i < n; ++i) {
      const uint32_t par = i & 1;
      if (i >= 0) {
        ok = wait_bar(&bar->s_full[par], (i >> 1) & 1, stop);
        if (!ok) break;
        tc_fence_after();
        float v0[16], v1[16];
        tmem_ld16_async(tmem + T_S2 + par * 128 + lanes + n0, v0);
        tmem_ld16_async(tmem + T_S2 + par * 128 + lanes + n0 + 16, v1);
        const unsigned long long f2 = pack2(f0, f0);
        seg_decay *= f0;
        tmem_wait_ld16(v0);
        tmem_wait_ld16(v1);
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
          const float2 u = unpack2(ffma2(f2, pack2(h[j], h[j + 1]), pack2(v0[j], v0[j + 1])));
          const float2 z = unpack2(ffma2(f2, pack2(h[16 + j], h[17 + j]), pack2(v1[j], v1[j + 1])));
          h[j] = u.x, h[j + 1] = u.y, h[16 + j] = z.x, h[17 + j] = z.y;
        }
      }
      f0 = f1;
      if (i + 2 < n) {  // (the MMAs that read this Xw's place are done)
        ok = wait_bar(&bar->full[st], full_par, stop);
        if (!ok) break;
        const Decays& d = reinterpret_cast<const Decays*>(smem + S_OFF_D + st * 2 * REC)[hd];
        const uint32_t x = sb + st * S_BYTES + 2 * BLK, xw = tmem + T_XW2 + par * 96 + lanes + (tg >> 1);
        f1 = d.total;
        if (!write_xw<false>(x, f_off, d.w + tg, q4, xw)) write_xw<true>(x, f_off, d.w + tg, q4, xw);
        tmem_wait_st();
        tc_fence_before();
        hand_over(B_XW + par);
        if (++st == S_STAGES) st = 0, full_par ^= 1;
      }
    }
    if (!ok) {  // (as in walk)
      hand_over(B_XW);
      hand_over(B_XW + 1);
    } else {
      float* out = a.seg_state + (((long long)s * a.H + head) * (a.nseg - 1) + seg) * (kP * kN + 32) + p * kN + n0;
#pragma unroll
      for (int j = 0; j < 32; j += 4) *reinterpret_cast<float4*>(out + j) = make_float4(h[j], h[j + 1], h[j + 2], h[j + 3]);
      if (p == 0 && n0 == 0) out[kP * kN] = seg_decay;
    }
  } else if (warp == WARPS + 1) {
    // ---- copies ----
    int issued = 0;
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      const int st = i % S_STAGES;
      if (i >= S_STAGES && !wait_bar(&bar->free_[st], (i / S_STAGES - 1) & 1, stop)) break;
      if (lane == 0) {
        const uint32_t f = smem_u32(&bar->full[st]), d = sb + st * S_BYTES;
        const int t = first + (c0 + i) * Q, bn = 2 * pair / (a.H / a.G) * kN;
        mbar_arrive_expect_tx(f, S_BYTES + 2 * REC);
        tma_load_2d(d + 2 * BLK, &tx, 2 * pair * kP, t, f);
        tma_load_2d(d + 3 * BLK, &tx, 2 * pair * kP + 64, t, f);
        bulk_load(sb + S_OFF_D + st * 2 * REC, decays + chunk_record(a.q, s, first, len, c0 + i) * a.H + 2 * pair, 2 * REC, f);
        tma_load_2d(d, &tb, bn, t, f);
        tma_load_2d(d + BLK, &tb, bn + 64, t, f);
      }
      issued = i + 1;
    }
    // copies land before the shared memory is given up, whoever gives up, and when
    for (int i = max(0, issued - S_STAGES); i < issued && lane == 0; ++i) mbar_wait(smem_u32(&bar->full[i % S_STAGES]), (i / S_STAGES) & 1);
  } else {
    // ---- MMAs ----
    constexpr uint32_t id_s = idesc_major(128, 128, false, true);
    const bool leader = elect_one();
    uint32_t st = 0;
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      const uint32_t par = i & 1;
      named_sync(B_XW + par, HANDED);  // Xw of this chunk; S of the last but one has been read
      if (*stop) break;
      tc_fence_after();
      if (leader) {
        const uint32_t bd = desc_lo(sb + st * S_BYTES, BLK);
#pragma unroll
        for (int k = 0; k < 4; ++k)  // 16 tokens: two groups of 8 rows
#pragma unroll
          for (int part = 0; part < 3; ++part)
            mma_ts<id_s>(tmem + T_S2 + par * 128, tmem + T_XW2 + par * 96 + part * 32 + k * 8, bd + k * (2048 >> 4), k + part > 0);
        mma_commit(smem_u32(&bar->s_full[par]));
        mma_commit(smem_u32(&bar->free_[st]));
      }
      __syncwarp();
      if (++st == S_STAGES) st = 0;
    }
    if (leader) {
      mma_commit(smem_u32(&bar->drain));
      mbar_poll_ns(smem_u32(&bar->drain), 0, kWaitLimitNs);
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && *stop) flag(a.q.status, SSM_STATUS_TIMEOUT);
  if (warp == WARPS) {
    __syncwarp();
    tc_fence_after();
    tmem_free_warp(tmem, 512);
  }
}

// A sequence in one segment, or its segments from the second on.
__global__ void __launch_bounds__(NT, 1)
    scan_tc_kernel(const __grid_constant__ CUtensorMap tx, const __grid_constant__ CUtensorMap tb,
                   const __grid_constant__ CUtensorMap tcm, const __grid_constant__ CUtensorMap ty, ScanArgs a,
                   const float* scores, const Decays* decays, const int* order) {
  const int per = max(1, a.nseg - 1);
  walk(tx, tb, tcm, ty, a, scores, decays, order, blockIdx.y / per, a.nseg == 1 ? 0 : blockIdx.y % per + 1);
}
// Before it, where there are several: the first segment, and beside it the states of those between the first and the last.  (One
// kernel for both grids made every walk 10 % longer.)
__global__ void __launch_bounds__(NT, 1)
    scan_first_kernel(const __grid_constant__ CUtensorMap tx, const __grid_constant__ CUtensorMap tb,
                      const __grid_constant__ CUtensorMap tcm, const __grid_constant__ CUtensorMap ty, ScanArgs a,
                      const float* scores, const Decays* decays, const int* order) {
  const int rank = blockIdx.y / (a.nseg - 1), j = blockIdx.y % (a.nseg - 1);
  if (j == 0)
    walk(tx, tb, tcm, ty, a, scores, decays, order, rank, 0);
  else
    state_walk(tx, tb, a, decays, order, rank, j);
}

// Segments of a sequence's chunks, for one CTA of a head pair to an SM: where sequences and pairs leave SMs idle, the pass over
// the segments' states pays for itself.  (us back to back, in one segment | in several: 10 chunks of 16 pairs 28 | 33 in two;
// 16 chunks of 40 pairs 37 | 39 in four; up to 20 chunks of 24 pairs 43 | 38 in five, 37 in four; up to 81 chunks of 48 pairs
// 137 | 86 in four; 128 chunks of 40 pairs 190 | 111 in four.)
int plan_segments_tc(int H, int n_seq, int max_len) {
  const long long items = (long long)(H / 2) * n_seq;
  const int nch = (max_len + Q - 1) / Q;
  if (nch < 12) return 1;
  int nseg = (int)(kSMs / (items > 0 ? items : 1));
  if (nseg > nch / 5) nseg = nch / 5;
  if (nseg > 16) nseg = 16;
  return nseg < 2 ? 1 : nseg + 1;
}

// workspace: scores, decays, then what segments add to the state; records (chunk_record) up to n_tok / Q + n_seq
size_t chunk_count(int n_seq, int n_tok) { return (size_t)(n_tok / Q) + n_seq + 1; }
size_t score_bytes(int n_seq, int n_tok, int G) { return chunk_count(n_seq, n_tok) * G * Q * Q * sizeof(float); }
size_t decay_bytes(int n_seq, int n_tok, int H) { return chunk_count(n_seq, n_tok) * H * REC; }
size_t order_bytes(int n_seq) { return ((size_t)n_seq * sizeof(int) + 255) & ~(size_t)255; }

}  // namespace

// Pairs of heads have to share B and C.  One chunk to a sequence leaves nothing to walk, and two do not cover the walk's start
// where each SM has three walks at most: the kernel of prompt_scan.cu takes these in one launch.  80 heads, event times in us,
// there | here, sequences x tokens:
//   1 x 64: 13 | 20    8 x 64: 33 | 43     64 x 64: 171 | 203
//   1 x 128: 17 | 21   8 x 128: 48 | 48    64 x 65: 246 | 232    64 x 128: 257 | 238
//   1 x 192: 21 | 23   8 x 192: 60 | 54    64 x 192: 347 | 274   1 x 256: 25 | 25   1 x 512: 48 | 31   64 x 512: 798 | 417
bool prompt_scan_tc_fits(int H, int G, int n_seq, int max_len) {
  return (H / G) % 2 == 0 && max_len > ((long long)n_seq * (H / 2) > 3 * kSMs ? 64 : 128);
}

size_t prompt_scan_tc_workspace_bytes(int H, int G, int n_seq, int n_tok, int max_len) {
  const int nseg = plan_segments_tc(H, n_seq, max_len);
  return 256 + score_bytes(n_seq, n_tok, G) + decay_bytes(n_seq, n_tok, H) + order_bytes(n_seq) +
         (size_t)n_seq * H * (nseg - 1) * (kP * kN + 32) * sizeof(float);
}

cudaError_t launch_prompt_scan_tc(const ScanArgs& args, void* workspace, cudaStream_t s) {
  ScanArgs a = args;
  a.nseg = plan_segments_tc(a.H, a.q.n_seq, a.q.max_len);
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  float* scores = reinterpret_cast<float*>(ws);
  ws += score_bytes(a.q.n_seq, a.q.n_tok, a.G);
  Decays* decays = reinterpret_cast<Decays*>(ws);
  ws += decay_bytes(a.q.n_seq, a.q.n_tok, a.H);
  int* order = reinterpret_cast<int*>(ws);
  ws += order_bytes(a.q.n_seq);
  a.seg_state = reinterpret_cast<float*>(ws);
  static bool done[2][64];
  cudaError_t e = allow_smem(scan_tc_kernel, TC_SMEM, done[0]);
  if (e == cudaSuccess) e = allow_smem(scan_first_kernel, TC_SMEM, done[1]);
  if (e != cudaSuccess) return e;
  CUtensorMap tx, tb, tcm, ty;
  if (!encode_tiles(&tx, a.x, a.q.n_tok, (long long)a.H * kP, a.ldx, Q) || !encode_tiles(&tb, a.B, a.q.n_tok, (long long)a.G * kN, a.ldb, Q) ||
      !encode_tiles(&tcm, a.C, a.q.n_tok, (long long)a.G * kN, a.ldc, Q) || !encode_tiles(&ty, a.y, a.q.n_tok, (long long)a.H * kP, a.ldy, 16))
    return cudaErrorInvalidValue;
  prep_kernel<<<dim3((unsigned)((a.q.max_len + Q - 1) / Q), (unsigned)a.q.n_seq, (unsigned)(a.G + (a.H + 4 * HEADS - 1) / (4 * HEADS))), 128, 0, s>>>(
      a, scores, decays, order);
  const dim3 grid((unsigned)(a.H / 2), (unsigned)(a.q.n_seq * max(1, a.nseg - 1)));
  if (a.nseg > 1) {
    e = launch_early(scan_first_kernel, grid, NT, TC_SMEM, s, tx, tb, tcm, ty, a, (const float*)scores, (const Decays*)decays,
                     (const int*)order);
    if (e != cudaSuccess) return e;
  }
  return launch_early(scan_tc_kernel, grid, NT, TC_SMEM, s, tx, tb, tcm, ty, a, (const float*)scores, (const Decays*)decays,
                      (const int*)order);
}

}  // namespace ssmtree
