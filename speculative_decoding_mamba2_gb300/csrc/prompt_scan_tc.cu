// The chunked scan of prompts on the 5th-generation tensor cores (long prompts; the formulas are in prompt_scan.cu).
//
// A CTA walks the 64-token chunks of a pair of heads that share B and C, everything transposed so that a row of
// tensor memory is one (head, p) of the pair's 128 and one thread owns it:
//     S [128 x 128]  = Xw [128 x 64 tokens] . B [64 x n]       what the chunk adds to the state; Xw = (w_t x_t)^T is
//                      written by its threads into tensor memory in three bf16 parts (24 bits), B is read MN-major
//     Y2 [128 x 64]  = h [128 x n] . C^T                       h rounded to bf16, in tensor memory
//     Y1 [128 x 64]  = x^T [128 x 64] . P^T                    for each head of the pair, P = scores with their decays
//     y = Y1 + e^{S_t} Y2 + D x,   h' = decay h + S            (h in fp32 registers for the whole walk)
// The scores C.B^T are the same for every head: scores_kernel computes them once, chunk by chunk, into the workspace.
//
// Warps by role, each waiting only for what it needs, so that the chunks overlap: 4 make Xw, 4 make P, 4 finish y, 8
// carry the state, one issues copies (TMA, three stages), one the MMAs, two the decays of their head.  MMAs run in the
// order they are issued: S, Y2, Y1.  Every wait is bounded: on a time-out all roles leave, the copies and MMAs in
// flight are waited for (bounded again) and the tensor memory is freed.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "mma_tiles.cuh"
#include "prompt.cuh"
#include "tc.cuh"

namespace ssmtree {
namespace {

constexpr int Q = 64, NT = 768, STAGES = 3;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLeast2 = -120.f * kLog2e;  // as kLeast of prompt_scan.cu, in powers of two

// shared memory: stages of C | B | x (two 64-column blocks each), P, y, decays, barriers
constexpr int BLK = Q * 128;  // a 64 x 64 bf16 block with 128-byte rows
constexpr int ST_BYTES = 6 * BLK, OFF_TB = 2 * BLK, OFF_TX = 4 * BLK;
constexpr int OFF_P = STAGES * ST_BYTES;   // [2][head][BLK]
constexpr int OFF_Y = OFF_P + 4 * BLK;     // [2][64][256]
constexpr int OFF_D = OFF_Y + 4 * BLK;     // [STAGES][head] decay records
constexpr int OFF_ODD = OFF_D + STAGES * 2 * 320 * 4;  // [2][128] tokens whose x is not finite
constexpr int OFF_BAR = OFF_ODD + 2 * 128 * 8;
constexpr int TC_SMEM = OFF_BAR + 256 + 1024 /* alignment */;

// tensor memory columns
constexpr int T_S = 0, T_Y2 = 128, T_Y1 = 192, T_XW = 320, T_H = 416;

struct Decays {  // of one head and chunk (exponents in powers of two)
  float S[64];   // sum from the start of the token's half of the chunk
  float D[64];   // step size
  float E1[32];  // 2^(sum after the token in the first half) D
  float w[64];   // 2^(sum after the token) D
  float e[64];   // 2^(sum up to the token)
  float total, pad[31];  // 2^(sum of the chunk)
};
static_assert(sizeof(Decays) == 320 * 4, "record size");

struct Bars {
  unsigned long long full[STAGES], free_[STAGES], dt_full[STAGES], dt_free[STAGES];
  unsigned long long xw_full[2], xw_free, s_full, s_free, h_ready, y2_done, p_full[2], p_free[2], y_full, y_free, drain;
  uint32_t tmem;
  int stop;
};
static_assert(sizeof(Bars) <= 256, "barrier space");

// Descriptors: 128-byte swizzled tiles of 64-column blocks (rows of 128 bytes, groups of 8 rows 1024 bytes apart).
// K-major: the rows are M or N.  MN-major: the rows are K, `block` bytes between 64-element blocks along M or N.
// The upper word is the same for all: group stride, version 1, 128-byte swizzle.
constexpr uint32_t kDescHi = (1024u >> 4) | 1u << 14 | 2u << 29;
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t block) {
  return ((addr >> 4) & 0x3FFFu) | (block >> 4) << 16;
}
__host__ __device__ constexpr uint32_t idesc_major(int M, int N, bool a_mn, bool b_mn) {
  return idesc_bf16(M, N) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u);
}
// one lane of a converged warp, the same at every call
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n selp.u32 %0, 1, 0, q;\n}\n" : "=r"(p));
  return p != 0;
}
// D (TMEM) = A (TMEM) . B (+ D);  D (TMEM) = A . B (+ D)
template <uint32_t IDESC>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b_lo, bool acc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 b;\n setp.ne.b32 p, %4, 0;\n mov.b64 b, {%2, %5};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b_lo), "n"(IDESC), "r"((uint32_t)acc), "n"(kDescHi)
      : "memory");
}
template <uint32_t IDESC>
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, bool acc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 a, b;\n setp.ne.b32 p, %4, 0;\n mov.b64 a, {%1, %5};\n mov.b64 b, {%2, %5};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n}\n" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "n"(IDESC), "r"((uint32_t)acc), "n"(kDescHi)
      : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t addr, const uint32_t (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"r"(addr), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }
// 16 rows x 8 columns of 32 bits, from fragments: v[0], v[2], .. rows lane / 4, v[1], v[3], .. 8 rows on, columns
// lane % 4 and, from v[2] on, 4 further
__device__ __forceinline__ void tmem_st_frag(uint32_t addr, const uint32_t (&v)[4]) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x2.b32 [%0], {%1, %2, %3, %4};\n" ::"r"(addr), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3])
               : "memory");
}
// 16 rows x 16 fp32 columns as accumulator fragments: v[4 j ..]: row lane / 4, columns 8 j + 2 (lane % 4), + 1, then
// row + 8 (to be waited for before their use)
__device__ __forceinline__ void tmem_ld_frag_async(uint32_t addr, float (&v)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
               : "r"(addr));
}
__device__ __forceinline__ void tmem_wait_ld8(float (&v)[8], float (&w)[8]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;\n"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]), "+f"(w[0]),
                 "+f"(w[1]), "+f"(w[2]), "+f"(w[3]), "+f"(w[4]), "+f"(w[5]), "+f"(w[6]), "+f"(w[7])
               :
               : "memory");
}
// four 8 x 8 fragments stored transposed, row addresses as frag_a_t's
__device__ __forceinline__ void stsm4_t(uint32_t addr, const uint32_t (&r)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};\n" ::"r"(addr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3])
               : "memory");
}
// 16 columns without the wait (tmem_wait_ld16 before their use)
__device__ __forceinline__ void tmem_ld16_async(uint32_t addr, float (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15}, [%16];\n"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_wait_ld16(float (&v)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;\n"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                 "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15])
               :
               : "memory");
}

// The warp waits together, suspended for up to 20 us at a time (spinning took 40 % of the SM's issue slots from the warps
// at work).  False once kTries of those have passed or another role has given up.
constexpr int kTries = 50000;
__device__ __forceinline__ bool try_wait_20us(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 20000;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return __all_sync(0xffffffffu, done);
}
__device__ __forceinline__ bool wait_bar(unsigned long long* bar, uint32_t parity, volatile int* stop) {
  const uint32_t b = smem_u32(bar);
  if (try_wait_20us(b, parity)) return true;
#pragma unroll 1
  for (int it = 0; it < kTries && !*stop; ++it)
    if (try_wait_20us(b, parity)) return true;
  *stop = 1;
  return false;
}
__device__ __forceinline__ void arrive_warp(unsigned long long* bar, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(smem_u32(bar));
}

// x = hi + mid + lo in bf16 (an infinity: hi alone), pairs of values
__device__ __forceinline__ void split3_pair(float x0, float x1, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
  hi = pack_bf16x2(x0, x1);
  const float r0 = x0 - bf16_lo(hi), r1 = x1 - bf16_hi(hi);
  mid = pack_bf16x2(r0, r1);
  lo = pack_bf16x2(r0 - bf16_lo(mid), r1 - bf16_hi(mid));
}

// Scores C_t . B_s of every chunk and group, once for all heads: [record][s / 4][t][s % 4] fp32.
__device__ __forceinline__ long long score_record(int first, int s, int chunk, int G, int grp) {
  return ((long long)(first / Q) + s + chunk) * G + grp;
}
__global__ void __launch_bounds__(128) scores_kernel(ScanArgs a, float* scores) {
  __shared__ __align__(128) unsigned char sm[2 * Q * kN * 2];
  launch_dependents();
  const int c = blockIdx.x, s = blockIdx.y, grp = blockIdx.z, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int first, len, slot;
  if (!seq_range(a.q, s, first, len, slot) || c * Q >= len) return;
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
  float* out = scores + score_record(first, s, c, a.G, grp) * (Q * Q);
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

// Registers per thread by role: launched with 80, 6 x 80 = 72 + 96 + 80 + 88 + 88 + 56.
template <int N>
__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(N)); }

template <bool STATE_ONLY>
__global__ void __launch_bounds__(NT, 1)
    scan_tc_kernel(const __grid_constant__ CUtensorMap tx, const __grid_constant__ CUtensorMap tb,
                   const __grid_constant__ CUtensorMap tcm, ScanArgs a, const float* scores) {
  extern __shared__ unsigned char smem_raw[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, wg = warp >> 2;
  const int pair = blockIdx.x, nseg = STATE_ONLY ? a.nseg - 1 : a.nseg;
  const int s = blockIdx.y / nseg, seg = blockIdx.y % nseg;
  int first, len, slot;
  if (!seq_range(a.q, s, first, len, slot)) {
    if (pair == 0 && seg == 0 && tid == 0) flag(a.q.status, SSM_STATUS_SEQ_RANGE);
    grid_dependency_wait();
    return;
  }
  const int nch = (len + Q - 1) / Q, per = (nch + a.nseg - 1) / a.nseg;
  const int c0 = seg * per, c1 = min(nch, c0 + per), n = max(0, c1 - c0);
  if (STATE_ONLY ? c1 >= nch : (n == 0 && seg > 0)) {
    grid_dependency_wait();  // the grid does not end before the one it depends on
    return;
  }
  unsigned char* smem = smem_raw + (-smem_u32(smem_raw) & 1023u);  // stays a shared-memory pointer to the compiler
  const uint32_t sb = smem_u32(smem);
  Decays* dec = reinterpret_cast<Decays*>(smem + OFF_D);
  Bars* bar = reinterpret_cast<Bars*>(smem + OFF_BAR);
  volatile int* stop = &bar->stop;

  if (tid == 0) {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(smem_u32(&bar->full[i]), 1);
      mbar_init(smem_u32(&bar->free_[i]), 1 + 4);
      mbar_init(smem_u32(&bar->dt_full[i]), 2);
      mbar_init(smem_u32(&bar->dt_free[i]), STATE_ONLY ? 12 : 20);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&bar->xw_full[i]), 4);
      mbar_init(smem_u32(&bar->p_full[i]), 4);
      mbar_init(smem_u32(&bar->p_free[i]), 4);
    }
    mbar_init(smem_u32(&bar->xw_free), 1);
    mbar_init(smem_u32(&bar->s_full), 1);
    mbar_init(smem_u32(&bar->s_free), 8);
    mbar_init(smem_u32(&bar->h_ready), 8);
    mbar_init(smem_u32(&bar->y2_done), 1);
    mbar_init(smem_u32(&bar->y_full), 1);
    mbar_init(smem_u32(&bar->y_free), 4);
    mbar_init(smem_u32(&bar->drain), 1);
    bar->stop = 0;
    fence_barrier_init();
  }
  if (!STATE_ONLY)  // P's entries after their token stay zero for the whole walk
    for (int i = tid; i < 4 * BLK / 16; i += NT) reinterpret_cast<uint4*>(smem + OFF_P)[i] = make_uint4(0, 0, 0, 0);
  if (warp == 21) tmem_alloc_warp(smem_u32(&bar->tmem), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bar->tmem;
  const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;  // this warp's rows of tensor memory
  const int row = (warp & 3) * 32 + lane;                    // (head of the pair, p) of a thread
  const int hd = row >> 6, p = row & 63, head = 2 * pair + hd;

  const uint32_t xcol = (uint32_t)(OFF_TX + hd * BLK + (p & 7) * 2);  // column p of head hd in a tile of x
  // x of token t in it: the 16-byte chunk of row t is (p >> 3) ^ (t & 7)
  auto x_at = [&](unsigned char* stage, int t) {
    return reinterpret_cast<uint16_t*>(stage + xcol + t * 128 + (((p >> 3) ^ (t & 7)) << 4));
  };
  unsigned long long* odd_tokens = reinterpret_cast<unsigned long long*>(smem + OFF_ODD);
  const int q4 = lane & 3, p0 = (warp & 1) * 32;  // p0: this warp's first column of its head's x
  if (wg == 0) {
    // ---- Xw ----
    if (!STATE_ONLY) regs_dec<72>();
    bool ok = true;
#pragma unroll 1
    for (int i = 0; i < n && ok; ++i) {
      const int st = i % STAGES, valid = min(Q, len - (c0 + i) * Q);
      unsigned char* sp = smem + st * ST_BYTES;
      ok = wait_bar(&bar->full[st], (i / STAGES) & 1, stop) && wait_bar(&bar->dt_full[st], (i / STAGES) & 1, stop);
      if (!ok) break;
      if (valid < Q) {  // rows after the sequence's last belong to another one
        for (int k = tid; k < (Q - valid) * 32; k += 128) {
          const int r = valid + (k >> 5), blk = (k >> 3) & 3, ch = k & 7;  // blocks of B, then of x
          *reinterpret_cast<uint4*>(sp + OFF_TB + blk * BLK + r * 128 + ch * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_async_smem();
        named_sync(1, 128);
      }
      const Decays& d = dec[st * 2 + hd];
      const uint32_t tile = sb + st * ST_BYTES + OFF_TX + hd * BLK;
      uint32_t chk = 0;  // sum of 0 x, in pairs: NaN once an x is not finite
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {
        if (i > 0) {
          ok = wait_bar(half ? &bar->s_full : &bar->xw_free, (i - 1) & 1, stop);
          if (!ok) break;
          tc_fence_after();
        }
        bool odd_half = false;
#pragma unroll 1
        for (int b = 0; b < 4; ++b) {  // 16 tokens, 16 rows.  (Rolled up: the roles' loops share the instruction caches)
          const int t0 = 32 * half + 16 * (b >> 1), rh = b & 1;
          uint32_t xf[4], hi[4], mid[4], lo[4];
          frag_a_t(xf, tile, 128, p0 + 16 * rh, t0, lane);
          const float2 w0 = *reinterpret_cast<const float2*>(&d.w[t0 + 2 * q4]);
          const float2 w1 = *reinterpret_cast<const float2*>(&d.w[t0 + 8 + 2 * q4]);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 w = j < 2 ? w0 : w1;
            split3_pair(bf16_lo(xf[j]) * w.x, bf16_hi(xf[j]) * w.y, hi[j], mid[j], lo[j]);
            asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(chk) : "r"(xf[j]), "r"(0u));
          }
          if (odd_half) {  // an infinity is its own first part
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              if ((hi[j] & 0x7f80u) == 0x7f80u) mid[j] &= 0xffff0000u, lo[j] &= 0xffff0000u;
              if ((hi[j] & 0x7f800000u) == 0x7f800000u) mid[j] &= 0xffffu, lo[j] &= 0xffffu;
            }
          }
          const uint32_t at = tmem + T_XW + lanes + ((uint32_t)(16 * rh) << 16) + (t0 >> 1);
          tmem_st_frag(at, lo);
          tmem_st_frag(at + 32, mid);
          tmem_st_frag(at + 64, hi);
          if (b == 3 && !odd_half && __any_sync(0xffffffffu, chk & 0x7fff7fffu)) odd_half = true, b = -1;  // once more
        }
        if (half == 1 && !STATE_ONLY) {
          unsigned long long odd = 0;
          if (__any_sync(0xffffffffu, chk & 0x7fff7fffu)) {
            // such values leave the tile (each thread its row's): the product with a zero of P would spread them
#pragma unroll 1
            for (int t = 0; t < Q; ++t) {
              uint16_t* v = x_at(sp, t);
              if ((*v & 0x7f80u) == 0x7f80u) odd |= 1ull << t, *v = 0;
            }
            fence_async_smem();
          }
          odd_tokens[(i & 1) * 128 + row] = odd;
        }
        tmem_wait_st();
        tc_fence_before();
        arrive_warp(&bar->xw_full[half], lane);
      }
      if (!ok) break;
      if (STATE_ONLY) arrive_warp(&bar->free_[st], lane);
      arrive_warp(&bar->dt_free[st], lane);
    }
    // a warp that gives up still takes part in the barrier that the other three may be waiting at
    if (!ok) asm volatile("bar.arrive 1, 128;\n" ::: "memory");
  } else if (wg == 1) {
    // ---- P ----
    if (!STATE_ONLY) {
      regs_inc<96>();
      const int ph = (warp >> 1) & 1, t = (warp & 1) * 32 + lane;  // head and token of this thread's row of P
      const bool late = (warp & 1) != 0;                           // the second half of the chunk
      const int grp = 2 * pair / (a.H / a.G);
      grid_dependency_wait();  // the scores
      float4 gq[16];
      auto fetch = [&](int i) {
        const float4* g = reinterpret_cast<const float4*>(scores + score_record(first, s, c0 + i, a.G, grp) * (Q * Q)) + t;
#pragma unroll
        for (int j = 0; j < 16; ++j)
          if (j < 8 || late) gq[j] = g[j * Q];
      };
      if (n > 0) fetch(0);
#pragma unroll 1
      for (int i = 0; i < n; ++i) {
        const int st = i % STAGES;
        if (!wait_bar(&bar->dt_full[st], (i / STAGES) & 1, stop)) break;
        if (i >= 2 && !wait_bar(&bar->p_free[i & 1], (i / 2 - 1) & 1, stop)) break;
        const Decays& d = dec[st * 2 + ph];
        unsigned char* pr = smem + OFF_P + ((i & 1) * 2 + ph) * BLK + t * 128;
        const float St = d.S[t];
        auto put = [&](int j8, const uint32_t (&v)[4]) {
          *reinterpret_cast<uint4*>(pr + ((j8 ^ (t & 7)) << 4)) = make_uint4(v[0], v[1], v[2], v[3]);
        };
        if (late) {  // the first half's tokens: their factor times this token's
          const float E2 = exp2_sfu(St);
#pragma unroll
          for (int j8 = 0; j8 < 4; ++j8) {
            uint32_t v[4];
#pragma unroll
            for (int m = 0; m < 2; ++m) {
              const float4 g = gq[2 * j8 + m], f = *reinterpret_cast<const float4*>(&d.E1[8 * j8 + 4 * m]);
              v[2 * m] = pack_bf16x2(g.x * (f.x * E2), g.y * (f.y * E2));
              v[2 * m + 1] = pack_bf16x2(g.z * (f.z * E2), g.w * (f.w * E2));
            }
            put(j8, v);
          }
        }
        const int s0 = late ? 32 : 0;
#pragma unroll
        for (int j8 = 0; j8 < 4; ++j8) {  // the token's own half
          uint32_t v[4];
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            const int u = 8 * j8 + 4 * m;
            const float4 g = late ? gq[8 + 2 * j8 + m] : gq[2 * j8 + m];
            const float4 S = *reinterpret_cast<const float4*>(&d.S[s0 + u]), D = *reinterpret_cast<const float4*>(&d.D[s0 + u]);
            const float w0 = u <= lane ? g.x * (exp2_sfu(St - S.x) * D.x) : 0.f;
            const float w1 = u + 1 <= lane ? g.y * (exp2_sfu(St - S.y) * D.y) : 0.f;
            const float w2 = u + 2 <= lane ? g.z * (exp2_sfu(St - S.z) * D.z) : 0.f;
            const float w3 = u + 3 <= lane ? g.w * (exp2_sfu(St - S.w) * D.w) : 0.f;
            v[2 * m] = pack_bf16x2(w0, w1), v[2 * m + 1] = pack_bf16x2(w2, w3);
          }
          put((s0 >> 3) + j8, v);
        }
        fence_async_smem();
        arrive_warp(&bar->p_full[i & 1], lane);
        arrive_warp(&bar->dt_free[st], lane);
        if (i + 1 < n) fetch(i + 1);
      }
    }
  } else if (wg == 2) {
    // ---- y ----
    if (!STATE_ONLY) {
      const int wt = tid - 256;
      const float Dh = a.D[head];
      bool ok = true;
#pragma unroll 1
      for (int i = 0; i < n && ok; ++i) {
        const int st = i % STAGES, c = c0 + i, valid = min(Q, len - c * Q);
        unsigned char* ys = smem + OFF_Y + (i & 1) * 2 * BLK;
        const Decays& d = dec[st * 2 + hd];
        const uint32_t tile = sb + st * ST_BYTES + OFF_TX + hd * BLK, yb = sb + OFF_Y + (i & 1) * 2 * BLK;
        ok = wait_bar(&bar->y_full, i & 1, stop);
        if (!ok) break;
        tc_fence_after();
#pragma unroll 1
        for (int b = 0; b < 8; ++b) {  // 16 tokens, 16 rows
          const int t0 = 16 * (b >> 1), rh = b & 1;
          const uint32_t at = tmem + lanes + ((uint32_t)(16 * rh) << 16) + t0;
          float y1[8], y2[8];
          uint32_t xf[4], o[4];
          tmem_ld_frag_async(at + T_Y1 + hd * 64, y1);
          tmem_ld_frag_async(at + T_Y2, y2);
          frag_a_t(xf, tile, 128, p0 + 16 * rh, t0, lane);
          const float2 e0 = *reinterpret_cast<const float2*>(&d.e[t0 + 2 * q4]);
          const float2 e1 = *reinterpret_cast<const float2*>(&d.e[t0 + 8 + 2 * q4]);
          tmem_wait_ld8(y1, y2);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 e = j < 2 ? e0 : e1;
            o[j] = pack_bf16x2(fmaf(Dh, bf16_lo(xf[j]), fmaf(e.x, y2[2 * j], y1[2 * j])),
                               fmaf(Dh, bf16_hi(xf[j]), fmaf(e.y, y2[2 * j + 1], y1[2 * j + 1])));
          }
          const int r = t0 + (lane & 7) + ((lane >> 4) << 3);
          stsm4_t(yb + tile_off(r, hd * 8 + ((p0 + 16 * rh) >> 3) + ((lane >> 3) & 1), 256), o);
        }
        const unsigned long long odd = odd_tokens[(i & 1) * 128 + row];
        if (__any_sync(0xffffffffu, odd != 0)) {  // what those values add is not finite, so it can be added to the rounded y
          __syncwarp();
          const unsigned char* pt = smem + OFF_P + ((i & 1) * 2 + hd) * BLK;
#pragma unroll 1
          for (int u = 0; u < Q; ++u) {
            if (!(odd >> u & 1)) continue;
            const float xv = bf16f(a.x[(long long)(first + c * Q + u) * a.ldx + head * kP + p]);
#pragma unroll 1
            for (int r = u; r < Q; ++r) {
              uint16_t* y = reinterpret_cast<uint16_t*>(ys + tile_off(r, row >> 3, 256) + (row & 7) * 2);
              const uint16_t w = *reinterpret_cast<const uint16_t*>(pt + r * 128 + (((u >> 3) ^ (r & 7)) << 4) + (u & 7) * 2);
              float v = fmaf(bf16f(w), xv, bf16f(*y));
              if (r == u) v = fmaf(Dh, xv, v);
              *y = (uint16_t)(pack_bf16x2(v, 0.f) & 0xffffu);
            }
          }
        }
        tc_fence_before();
        arrive_warp(&bar->y_free, lane);
        arrive_warp(&bar->free_[st], lane);
        arrive_warp(&bar->dt_free[st], lane);
        arrive_warp(&bar->p_free[i & 1], lane);
        named_sync(2, 128);  // y of the chunk is in shared memory
        uint16_t* yo = a.y + (long long)(first + c * Q) * a.ldy + pair * 2 * kP;
#pragma unroll 2
        for (int k = 0; k < 8; ++k) {
          const int r = k * 8 + (wt >> 4), ch = wt & 15;
          if (r < valid)
            *reinterpret_cast<uint4*>(yo + (long long)r * a.ldy + ch * 8) =
                *reinterpret_cast<const uint4*>(ys + tile_off(r, ch, 256));
        }
      }
      if (!ok) asm volatile("bar.arrive 2, 128;\n" ::: "memory");
    }
  } else if (wg < 5) {
    // ---- the state: 64 of a row's 128 columns ----
    if (!STATE_ONLY) regs_inc<88>();
    const int n0 = (wg - 3) * 64;
    const long long at = (((long long)slot * a.L + a.layer) * a.H + head) * (kP * kN) + p * kN + n0;
    const long long wrec = kP * kN + 32;
    float* ws = a.seg_state + ((long long)s * a.H + head) * (a.nseg - 1) * wrec;
    float h[64];
    if (!STATE_ONLY && a.h_in) {
#pragma unroll
      for (int j = 0; j < 64; j += 4) {
        const float4 v = *reinterpret_cast<const float4*>(a.h_in + at + j);
        h[j] = v.x, h[j + 1] = v.y, h[j + 2] = v.z, h[j + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 64; ++j) h[j] = 0.f;
    }
    if (!STATE_ONLY)
#pragma unroll 1
      for (int k = 0; k < seg; ++k) {
        const float* r = ws + k * wrec;
        const float dk = r[kP * kN];
        r += p * kN + n0;
#pragma unroll
        for (int j = 0; j < 64; j += 4) {
          const float4 v = *reinterpret_cast<const float4*>(r + j);
          h[j] = fmaf(dk, h[j], v.x), h[j + 1] = fmaf(dk, h[j + 1], v.y);
          h[j + 2] = fmaf(dk, h[j + 2], v.z), h[j + 3] = fmaf(dk, h[j + 3], v.w);
        }
      }
    auto put_h = [&]() {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = pack_bf16x2(h[16 * k + 2 * j], h[16 * k + 2 * j + 1]);
        tmem_st8(tmem + T_H + lanes + (n0 >> 1) + 8 * k, v);
      }
      tmem_wait_st();
      tc_fence_before();
      arrive_warp(&bar->h_ready, lane);
    };
    if (!STATE_ONLY) put_h();
    float seg_decay = 1.f;
    bool ok = true;
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      const int st = i % STAGES;
      ok = wait_bar(&bar->dt_full[st], (i / STAGES) & 1, stop) && wait_bar(&bar->s_full, i & 1, stop);
      if (!ok) break;
      const float f = dec[st * 2 + hd].total;
      tc_fence_after();
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float v[16];
        tmem_ld16_async(tmem + T_S + lanes + n0 + 16 * k, v);
        tmem_wait_ld16(v);
#pragma unroll
        for (int j = 0; j < 16; ++j) h[16 * k + j] = fmaf(f, h[16 * k + j], v[j]);
      }
      seg_decay *= f;
      tc_fence_before();
      arrive_warp(&bar->s_free, lane);
      arrive_warp(&bar->dt_free[st], lane);
      if (!STATE_ONLY && i + 1 < n) {
        ok = wait_bar(&bar->y2_done, i & 1, stop);
        if (!ok) break;
        tc_fence_after();
        put_h();
      }
    }
    if (ok && (STATE_ONLY || c1 == nch)) {
      float* out = STATE_ONLY ? ws + seg * wrec + p * kN + n0 : a.h_out + at;
#pragma unroll
      for (int j = 0; j < 64; j += 4) *reinterpret_cast<float4*>(out + j) = make_float4(h[j], h[j + 1], h[j + 2], h[j + 3]);
      if (STATE_ONLY && p == 0 && n0 == 0) ws[seg * wrec + kP * kN] = seg_decay;
    }
  } else {
    if (!STATE_ONLY) regs_dec<56>();
  if (warp == 20) {
    // ---- copies ----
    int issued = 0;
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      const int st = i % STAGES;
      if (i >= STAGES && !wait_bar(&bar->free_[st], (i / STAGES - 1) & 1, stop)) break;
      if (lane == 0) {
        const uint32_t f = smem_u32(&bar->full[st]), d = sb + st * ST_BYTES;
        const int t = first + (c0 + i) * Q, bn = 2 * pair / (a.H / a.G) * kN;
        mbar_arrive_expect_tx(f, STATE_ONLY ? 4 * BLK : 6 * BLK);
        tma_load_2d(d + OFF_TX, &tx, 2 * pair * kP, t, f);
        tma_load_2d(d + OFF_TX + BLK, &tx, 2 * pair * kP + 64, t, f);
        tma_load_2d(d + OFF_TB, &tb, bn, t, f);
        tma_load_2d(d + OFF_TB + BLK, &tb, bn + 64, t, f);
        if (!STATE_ONLY) {
          tma_load_2d(d, &tcm, bn, t, f);
          tma_load_2d(d + BLK, &tcm, bn + 64, t, f);
        }
      }
      issued = i + 1;
    }
    if (lane == 0 && *stop) {  // copies in flight land before the shared memory is given up
      for (int i = max(0, issued - STAGES); i < issued; ++i)
        mbar_poll_ns(smem_u32(&bar->full[i % STAGES]), (i / STAGES) & 1, kWaitLimitNs);
    }
  } else if (warp == 21) {
    // ---- MMAs ----
    constexpr uint32_t id_s = idesc_major(128, 128, false, true), id_y2 = idesc_major(128, 64, false, false),
                       id_y1 = idesc_major(128, 64, true, false);
    const bool leader = elect_one();
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    bool ok = true;
#pragma unroll 1
    for (int i = 0; i < n && ok; ++i) {
      const int st = i % STAGES;
      const uint32_t tile = sb + st * ST_BYTES;
      ok = wait_bar(&bar->full[st], (i / STAGES) & 1, stop) && (i == 0 || wait_bar(&bar->s_free, (i - 1) & 1, stop));
#pragma unroll 1
      for (int half = 0; half < 2 && ok; ++half) {
        ok = wait_bar(&bar->xw_full[half], i & 1, stop);
        if (!ok) break;
        tc_fence_after();
        if (leader) {
          const uint32_t bd = desc_lo(tile + OFF_TB + half * 4096, BLK), xw = tm + T_XW + half * 16;
#pragma unroll
          for (int k = 0; k < 2; ++k)  // 16 tokens: two groups of 8 rows
#pragma unroll
            for (int part = 0; part < 3; ++part)
              mma_ts<id_s>(tm + T_S, xw + part * 32 + k * 8, bd + k * (2048 >> 4), k + part > 0 || half > 0);
          mma_commit(smem_u32(half ? &bar->s_full : &bar->xw_free));
        }
        __syncwarp();
      }
      if (!STATE_ONLY) {
        ok = ok && wait_bar(&bar->h_ready, i & 1, stop) && (i == 0 || wait_bar(&bar->y_free, (i - 1) & 1, stop));
        if (!ok) break;
        tc_fence_after();
        if (leader) {
          const uint32_t cd = desc_lo(tile, 16);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            mma_ts<id_y2>(tm + T_Y2, tm + T_H + k * 8, cd + ((k >> 2) * (BLK >> 4) + (k & 3) * 2), k != 0);
          mma_commit(smem_u32(&bar->y2_done));
        }
        __syncwarp();
        ok = wait_bar(&bar->p_full[i & 1], (i / 2) & 1, stop);
        if (!ok) break;
        tc_fence_after();
        if (leader) {
          const uint32_t xd = desc_lo(tile + OFF_TX, BLK), pd = desc_lo(sb + OFF_P + (i & 1) * 2 * BLK, 16);
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_ss<id_y1>(tm + T_Y1 + e * 64, xd + k * (2048 >> 4), pd + e * (BLK >> 4) + k * 2, k != 0);
          mma_commit(smem_u32(&bar->y_full));
        }
        __syncwarp();
      }
      if (ok && leader) mma_commit(smem_u32(&bar->free_[st]));
      __syncwarp();
    }
    if (leader) {
      mma_commit(smem_u32(&bar->drain));
      mbar_poll_ns(smem_u32(&bar->drain), 0, kWaitLimitNs);
    }
    __syncwarp();
  } else {
    // ---- the decays of one head: tokens 2 lane, 2 lane + 1 ----
    const int dh = warp - 22, hh = 2 * pair + dh;
    const float A2 = neg_exp(a.A_log[hh]) * kLog2e, bias = a.dt_bias[hh];
    auto fetch = [&](int i, uint32_t& v0, uint32_t& v1) {
      const int t = (c0 + i) * Q + 2 * lane;
      const uint16_t* q = a.dt + (long long)(first + t) * a.lddt + hh;
      v0 = t < len ? q[0] : 0u, v1 = t + 1 < len ? q[a.lddt] : 0u;
    };
    uint32_t r0 = 0, r1 = 0;
    if (n > 0) fetch(0, r0, r1);
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      const int st = i % STAGES, t = (c0 + i) * Q + 2 * lane;
      if (i >= STAGES && !wait_bar(&bar->dt_free[st], (i / STAGES - 1) & 1, stop)) break;
      const float d0 = t < len ? softplus_f(bf16f((uint16_t)r0) + bias) : 0.f;
      const float d1 = t + 1 < len ? softplus_f(bf16f((uint16_t)r1) + bias) : 0.f;
      if (i + 1 < n) fetch(i + 1, r0, r1);
      const float e0 = fmaxf(d0 * A2, kLeast2), e1 = fmaxf(d1 * A2, kLeast2);
      float pre = e0 + e1, suf = pre;  // sums within the lane's half of the chunk
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) {
        const float u = __shfl_up_sync(0xffffffffu, pre, o, 16), v = __shfl_down_sync(0xffffffffu, suf, o, 16);
        if ((lane & 15) >= o) pre += u;
        if ((lane & 15) + o < 16) suf += v;
      }
      const float sum0 = __shfl_sync(0xffffffffu, pre, 15), sum1 = __shfl_sync(0xffffffffu, pre, 31);
      float before = __shfl_up_sync(0xffffffffu, pre, 1, 16), after = __shfl_down_sync(0xffffffffu, suf, 1, 16);
      if ((lane & 15) == 0) before = 0.f;
      if ((lane & 15) == 15) after = 0.f;
      const bool low = lane < 16;
      Decays& d = dec[st * 2 + dh];
      const float base = low ? 0.f : sum0, rest = low ? sum1 : 0.f, S0 = before + e0;
      *reinterpret_cast<float2*>(&d.S[2 * lane]) = make_float2(S0, pre);
      *reinterpret_cast<float2*>(&d.D[2 * lane]) = make_float2(d0, d1);
      const float a0 = after + e1;  // after token 2 lane, in its half
      if (low) *reinterpret_cast<float2*>(&d.E1[2 * lane]) = make_float2(exp2_sfu(a0) * d0, exp2_sfu(after) * d1);
      *reinterpret_cast<float2*>(&d.w[2 * lane]) = make_float2(exp2_sfu(a0 + rest) * d0, exp2_sfu(after + rest) * d1);
      *reinterpret_cast<float2*>(&d.e[2 * lane]) = make_float2(exp2_sfu(base + S0), exp2_sfu(base + pre));
      if (lane == 0) d.total = exp2_sfu(sum0 + sum1);
      arrive_warp(&bar->dt_full[st], lane);
    }
  }
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && *stop) flag(a.q.status, SSM_STATUS_TIMEOUT);
  if (warp == 21) {
    __syncwarp();
    tc_fence_after();
    tmem_free_warp(tmem, 512);
  }
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  if (!fn) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }
  return fn;
}
bool encode(CUtensorMap* m, const void* base, long long rows, long long cols, long long ld) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t gdim[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t gstride[1] = {(cuuint64_t)ld * 2};
  const cuuint32_t box[2] = {64, Q};
  const cuuint32_t estride[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), gdim, gstride, box, estride,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// as plan_segments of prompt_scan.cu, for one CTA of a head pair to an SM
int plan_segments_tc(int H, int n_seq, int max_len) {
  const long long items = (long long)(H / 2) * n_seq;
  const int nch = (max_len + Q - 1) / Q;
  int nseg = (int)(kSMs / (items > 0 ? items : 1));
  if (nseg > nch / 4) nseg = nch / 4;
  if (nseg > 16) nseg = 16;
  return nseg < 2 ? 1 : nseg;
}

size_t score_bytes(int n_seq, int n_tok, int G) { return ((size_t)(n_tok / Q) + n_seq + 1) * G * Q * Q * sizeof(float); }

}  // namespace

bool prompt_scan_tc_fits(int H, int G, int n_seq, int max_len) { return (H / G) % 2 == 0 && max_len > 64; }

size_t prompt_scan_tc_workspace_bytes(int H, int G, int n_seq, int n_tok, int max_len) {
  const int nseg = plan_segments_tc(H, n_seq, max_len);
  return 256 + score_bytes(n_seq, n_tok, G) + (size_t)n_seq * H * (nseg - 1) * (kP * kN + 32) * sizeof(float);
}

cudaError_t launch_prompt_scan_tc(const ScanArgs& args, void* workspace, cudaStream_t s) {
  ScanArgs a = args;
  a.nseg = plan_segments_tc(a.H, a.q.n_seq, a.q.max_len);
  float* scores = static_cast<float*>(workspace);
  a.seg_state = scores + score_bytes(a.q.n_seq, a.q.n_tok, a.G) / sizeof(float);
  cudaError_t e = cudaFuncSetAttribute(scan_tc_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, TC_SMEM);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(scan_tc_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, TC_SMEM);
  if (e != cudaSuccess) return e;
  CUtensorMap tx, tb, tcm;
  if (!encode(&tx, a.x, a.q.n_tok, (long long)a.H * kP, a.ldx) || !encode(&tb, a.B, a.q.n_tok, (long long)a.G * kN, a.ldb) ||
      !encode(&tcm, a.C, a.q.n_tok, (long long)a.G * kN, a.ldc))
    return cudaErrorInvalidValue;
  if (a.nseg > 1)
    scan_tc_kernel<true><<<dim3((unsigned)(a.H / 2), (unsigned)(a.q.n_seq * (a.nseg - 1))), NT, TC_SMEM, s>>>(tx, tb, tcm, a, scores);
  scores_kernel<<<dim3((unsigned)((a.q.max_len + Q - 1) / Q), (unsigned)a.q.n_seq, (unsigned)a.G), 128, 0, s>>>(a, scores);
  // the walk starts while the scores are made; its P warps wait for them
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(a.H / 2), (unsigned)(a.q.n_seq * a.nseg));
  cfg.blockDim = dim3(NT);
  cfg.dynamicSmemBytes = TC_SMEM;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, scan_tc_kernel<false>, tx, tb, tcm, a, (const float*)scores);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace ssmtree
