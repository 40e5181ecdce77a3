// Linear attention with a decay for each head over ragged prompts (ssm_prompt.h), in chunks of Q tokens.
//
// With S_t the sum of D_s A over the chunk's tokens up to and with t, and h the state before the chunk,
//     y_t = e^{S_t} C_t h + sum_{s <= t} (C_t . B_s) e^{S_t - S_s} D_s x_s + D x_t
//     h' = e^{S_Q} h + sum_s (e^{S_Q - S_s} D_s x_s) (x) B_s
// which turns the token-by-token recurrence into products of the tensor cores.
#include "mma_tiles.cuh"
#include "prompt.cuh"

namespace ssmtree {
namespace {

constexpr int Q = 64;          // tokens per chunk
constexpr int THREADS = 128;   // warp w: tokens 16w.. of y, rows 16w.. (head_dim) of the state
constexpr float kLog2e = 1.4426950408889634f;
// Decays below e^-120 are 0 in fp32 however they are formed: a token's exponent is raised to -120, so that sums of
// them stay finite and small sums after it keep their bits.
constexpr float kLeast = -120.f;

constexpr int STAGE = Q * (kN + kN + kP) * 2;  // C, B, x of one chunk
constexpr int OFF_B = Q * kN * 2, OFF_X = 2 * Q * kN * 2;
constexpr int OFF_H = 2 * STAGE;                       // bf16 state [p][n]
constexpr int OFF_T = OFF_H + kP * kN * 2;             // per warp: S, w and D of the chunk's tokens
constexpr int SMEM = OFF_T + 4 * 3 * Q * 4;

// fp32 -> three bf16 parts of its 24 bits: x = hi + mid + lo (an infinity: hi alone)
__device__ __forceinline__ void split3(float x0, float x1, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
  hi = pack_bf16x2(x0, x1);
  const float r0 = fabsf(x0) < INFINITY ? x0 - bf16_lo(hi) : 0.f, r1 = fabsf(x1) < INFINITY ? x1 - bf16_hi(hi) : 0.f;
  mid = pack_bf16x2(r0, r1);
  lo = pack_bf16x2(r0 - bf16_lo(mid), r1 - bf16_hi(mid));
}

// STATE_ONLY: what the segment adds to a zero state, and its decay, into the workspace
template <bool STATE_ONLY>
__global__ void __launch_bounds__(THREADS, 2) prompt_scan_kernel(ScanArgs a) {
  extern __shared__ __align__(128) unsigned char smem[];
  const int h = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int nseg = STATE_ONLY ? a.nseg - 1 : a.nseg;  // segments this grid walks
  const int s = blockIdx.y / nseg, seg = blockIdx.y % nseg;
  int first, len, slot;
  if (!seq_range(a.q, s, first, len, slot)) {
    if (h == 0 && seg == 0 && tid == 0) flag(a.q.status, SSM_STATUS_SEQ_RANGE);
    return;
  }
  const int nch = (len + Q - 1) / Q, per = (nch + a.nseg - 1) / a.nseg;
  const int c0 = seg * per, c1 = min(nch, c0 + per);
  if (STATE_ONLY ? c1 >= nch : (c0 >= c1 && seg > 0)) return;  // no segment after it; nothing in it
  const long long hbase = (((long long)slot * a.L + a.layer) * a.H + h) * (kP * kN);
  const long long wrec = kP * kN + 32;  // a workspace record: the state, then the decay
  float* ws = a.seg_state + ((long long)s * a.H + h) * a.nseg * wrec;  // the last record: the caller's state
  const uint32_t sb = smem_u32(smem);
  const int grp = h / (a.H / a.G), g = lane >> 2, q4 = lane & 3;
  const float A = neg_exp(a.A_log[h]), bias = a.dt_bias[h], Dh = a.D[h];

  auto load = [&](int c) {
    const uint32_t st = sb + (c & 1) * STAGE;
    const int t0 = c * Q;
#pragma unroll 4
    for (int i = tid; i < Q * 16; i += THREADS) {
      const int row = i >> 4, ch = i & 15;
      const bool there = t0 + row < len;
      const long long t = there ? first + t0 + row : first;
      if (!STATE_ONLY)
        cp_async16_or_zero(st + tile_off(row, ch, kN * 2), a.C + t * a.ldc + grp * kN + ch * 8, there);
      cp_async16_or_zero(st + OFF_B + tile_off(row, ch, kN * 2), a.B + t * a.ldb + grp * kN + ch * 8, there);
    }
#pragma unroll 4
    for (int i = tid; i < Q * 8; i += THREADS) {
      const int row = i >> 3, ch = i & 7;
      const bool there = t0 + row < len;
      const long long t = there ? first + t0 + row : first;
      cp_async16_or_zero(st + OFF_X + tile_off(row, ch, kP * 2), a.x + t * a.ldx + h * kP + ch * 8, there);
    }
    cp_async_commit();
  };
  if (c0 < c1) load(c0);

  // the state: warp w rows 16w + g and + 8, columns 8 nt + 2 q4, + 1 (the accumulator fragments)
  // (the caller's state may be written in place by a sequence's last segment: where there are several, the first grid copies it)
  float hs[16][4];
  const float* from = !a.h_in || (STATE_ONLY && seg > 0)  ? nullptr
                      : STATE_ONLY || (seg == 0 && c1 == nch) ? a.h_in + hbase
                                                              : ws + (a.nseg - 1) * wrec;
#pragma unroll
  for (int nt = 0; nt < 16; ++nt) {
    const int n = nt * 8 + 2 * q4;
    float2 lo = make_float2(0.f, 0.f), hi = lo;
    if (from) {
      lo = *reinterpret_cast<const float2*>(from + (16 * warp + g) * kN + n);
      hi = *reinterpret_cast<const float2*>(from + (16 * warp + g + 8) * kN + n);
      if (STATE_ONLY) {
        float* copy = ws + (a.nseg - 1) * wrec;
        *reinterpret_cast<float2*>(copy + (16 * warp + g) * kN + n) = lo;
        *reinterpret_cast<float2*>(copy + (16 * warp + g + 8) * kN + n) = hi;
        lo = hi = make_float2(0.f, 0.f);
      }
    }
    if (!STATE_ONLY) {
#pragma unroll 1
      for (int i = 0; i < seg; ++i) {
        const float* r = ws + i * wrec;
        const float d = r[kP * kN];
        const float2 u = *reinterpret_cast<const float2*>(r + (16 * warp + g) * kN + n);
        const float2 v = *reinterpret_cast<const float2*>(r + (16 * warp + g + 8) * kN + n);
        lo.x = fmaf(d, lo.x, u.x), lo.y = fmaf(d, lo.y, u.y);
        hi.x = fmaf(d, hi.x, v.x), hi.y = fmaf(d, hi.y, v.y);
      }
    }
    hs[nt][0] = lo.x, hs[nt][1] = lo.y, hs[nt][2] = hi.x, hs[nt][3] = hi.y;
  }
  auto put_state = [&]() {  // the state as the products read it, rounded to bf16
#pragma unroll
    for (int nt = 0; nt < 16; ++nt) {
      const uint32_t r0 = sb + OFF_H + tile_off(16 * warp + g, nt, kN * 2) + 4 * q4;
      const uint32_t r1 = sb + OFF_H + tile_off(16 * warp + g + 8, nt, kN * 2) + 4 * q4;
      asm volatile("st.shared.b32 [%0], %1;" ::"r"(r0), "r"(pack_bf16x2(hs[nt][0], hs[nt][1])) : "memory");
      asm volatile("st.shared.b32 [%0], %1;" ::"r"(r1), "r"(pack_bf16x2(hs[nt][2], hs[nt][3])) : "memory");
    }
  };
  if (!STATE_ONLY) put_state();

  float* sS = reinterpret_cast<float*>(smem + OFF_T) + warp * 3 * Q;
  float *sW = sS + Q, *sD = sW + Q;
  float seg_sum = 0.f;  // of the exponents of the whole segment
#pragma unroll 1
  for (int c = c0; c < c1; ++c) {
    const uint32_t st = sb + (c & 1) * STAGE;
    // each warp by itself: exponents of the chunk's tokens 2 lane, 2 lane + 1, their prefix and suffix sums
    float d0 = 0.f, d1 = 0.f, e0 = 0.f, e1 = 0.f;
    {
      const int t = c * Q + 2 * lane;
      const uint16_t* p = a.dt + (long long)(first + t) * a.lddt + h;
      if (t < len) d0 = softplus_f(bf16f(p[0]) + bias), e0 = fmaxf(d0 * A, kLeast);
      if (t + 1 < len) d1 = softplus_f(bf16f(p[a.lddt]) + bias), e1 = fmaxf(d1 * A, kLeast);
    }
    float pre = e0 + e1, suf = pre;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const float u = __shfl_up_sync(0xffffffffu, pre, o), v = __shfl_down_sync(0xffffffffu, suf, o);
      if (lane >= o) pre += u;
      if (lane + o < 32) suf += v;
    }
    const float total = __shfl_sync(0xffffffffu, pre, 31);
    float after = __shfl_down_sync(0xffffffffu, suf, 1);  // sum of the tokens after 2 lane + 1
    if (lane == 31) after = 0.f;
    float before = __shfl_up_sync(0xffffffffu, pre, 1);  // sum of the tokens before 2 lane
    if (lane == 0) before = 0.f;
    __syncwarp();  // the previous chunk's values have been read
    sS[2 * lane] = before + e0, sS[2 * lane + 1] = pre;
    sW[2 * lane] = exp2_sfu((after + e1) * kLog2e) * d0, sW[2 * lane + 1] = exp2_sfu(after * kLog2e) * d1;
    sD[2 * lane] = d0, sD[2 * lane + 1] = d1;
    seg_sum += total;
    const float decay = exp2_sfu(total * kLog2e);

    cp_async_wait<0>();
    __syncthreads();  // the chunk's tiles and the state are in shared memory; the other stage is free
    if (c + 1 < c1) load(c + 1);

    if (!STATE_ONLY) {
      // whether a value of x is not finite: products with masked (zero) scores would spread it
      bool odd = false;
#pragma unroll
      for (int i = 0; i < Q * 8 / THREADS; ++i) {
        uint4 v;
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                     : "r"(st + OFF_X + (uint32_t)(tid + i * THREADS) * 16));
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 4; ++k)
          odd |= (w[k] & 0x7f80u) == 0x7f80u || (w[k] & 0x7f800000u) == 0x7f800000u;
      }
      uint32_t cf[8][4];
#pragma unroll
      for (int k = 0; k < 8; ++k) frag_a(cf[k], st, kN * 2, 16 * warp, 16 * k, lane);
      float acc[8][4];
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
      // e^{S_t} C_t h
#pragma unroll
      for (int k = 0; k < 8; ++k)
#pragma unroll
        for (int np = 0; np < 4; ++np) {
          uint32_t b[4];
          frag_b2(b, sb + OFF_H, kN * 2, 16 * np, 16 * k, lane);
          mma16816(acc[2 * np], cf[k], b[0], b[1]);
          mma16816(acc[2 * np + 1], cf[k], b[2], b[3]);
        }
      const int ta = 16 * warp + g, tb = ta + 8;
      const float Sa = sS[ta], Sb = sS[tb];
      const float ea = exp2_sfu(Sa * kLog2e), eb = exp2_sfu(Sb * kLog2e);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i][0] *= ea, acc[i][1] *= ea, acc[i][2] *= eb, acc[i][3] *= eb;
      const bool any_odd = __syncthreads_or(odd);  // and: every warp has read the state
      // the chunk's own tokens, 16 at a time
#pragma unroll 1
      for (int jb = 0; jb <= warp; ++jb) {
        float gs[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i) gs[i][0] = gs[i][1] = gs[i][2] = gs[i][3] = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          uint32_t b[4];
          frag_b2(b, st + OFF_B, kN * 2, 16 * jb, 16 * k, lane);
          mma16816(gs[0], cf[k], b[0], b[1]);
          mma16816(gs[1], cf[k], b[2], b[3]);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int u = 16 * jb + 8 * i + 2 * q4 + e;
            const float Su = sS[u], Du = sD[u];
            gs[i][e] = u <= ta ? gs[i][e] * (exp2_sfu((Sa - Su) * kLog2e) * Du) : 0.f;
            gs[i][2 + e] = u <= tb ? gs[i][2 + e] * (exp2_sfu((Sb - Su) * kLog2e) * Du) : 0.f;
          }
        const uint32_t pa[4] = {pack_bf16x2(gs[0][0], gs[0][1]), pack_bf16x2(gs[0][2], gs[0][3]),
                                pack_bf16x2(gs[1][0], gs[1][1]), pack_bf16x2(gs[1][2], gs[1][3])};
#pragma unroll
        for (int np = 0; np < 4; ++np) {
          uint32_t b[4];
          frag_b2_t(b, st + OFF_X, kP * 2, 16 * np, 16 * jb, lane);
          if (any_odd)
#pragma unroll
            for (int i = 0; i < 4; ++i) b[i] = finite_or_zero(b[i]);
          mma16816(acc[2 * np], pa, b[0], b[1]);
          mma16816(acc[2 * np + 1], pa, b[2], b[3]);
        }
        if (any_odd) {  // the values left out, each only in the rows at or after its token
#pragma unroll
          for (int i = 0; i < 4; ++i)  // pa[i]: rows g + 8 (i & 1), tokens 8 (i >> 1) + 2 q4, + 1
#pragma unroll 1
            for (int k = 0; k < 8; ++k) {
              const int u = 16 * jb + 8 * (i >> 1) + k, t = i & 1 ? tb : ta;
              const uint32_t w = __shfl_sync(0xffffffffu, pa[i], (lane & ~3) | (k >> 1));
              const float p = k & 1 ? bf16_hi(w) : bf16_lo(w);
#pragma unroll
              for (int nt = 0; nt < 8; ++nt) {
                const uint32_t v =
                    *reinterpret_cast<const uint32_t*>(smem + (st - sb) + OFF_X + tile_off(u, nt, kP * 2) + 4 * q4);
                const uint32_t kept = finite_or_zero(v);
                if (u <= t && (v ^ kept) & 0xffffu) acc[nt][2 * (i & 1)] = fmaf(p, bf16_lo(v), acc[nt][2 * (i & 1)]);
                if (u <= t && (v ^ kept) & 0xffff0000u)
                  acc[nt][2 * (i & 1) + 1] = fmaf(p, bf16_hi(v), acc[nt][2 * (i & 1) + 1]);
              }
            }
        }
      }
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int tr = half ? tb : ta, t = c * Q + tr;
        if (t < len) {
          uint16_t* yr = a.y + (long long)(first + t) * a.ldy + h * kP + 2 * q4;
#pragma unroll
          for (int nt = 0; nt < 8; ++nt) {
            const uint32_t v =
                *reinterpret_cast<const uint32_t*>(smem + (st - sb) + OFF_X + tile_off(tr, nt, kP * 2) + 4 * q4);
            *reinterpret_cast<uint32_t*>(yr + nt * 8) =
                pack_bf16x2(fmaf(Dh, bf16_lo(v), acc[nt][2 * half]), fmaf(Dh, bf16_hi(v), acc[nt][2 * half + 1]));
          }
        }
      }
    }
    // h' = decay h + sum_s (w_s x_s) (x) B_s, the first factor in three bf16 parts
#pragma unroll
    for (int i = 0; i < 16; ++i) hs[i][0] *= decay, hs[i][1] *= decay, hs[i][2] *= decay, hs[i][3] *= decay;
#pragma unroll
    for (int k = 0; k < Q / 16; ++k) {
      uint32_t xf[4], hi[4], mid[4], lo[4];
      frag_a_t(xf, st + OFF_X, kP * 2, 16 * warp, 16 * k, lane);
      const float2 w0 = *reinterpret_cast<const float2*>(sW + 16 * k + 2 * q4);
      const float2 w1 = *reinterpret_cast<const float2*>(sW + 16 * k + 8 + 2 * q4);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 w = i < 2 ? w0 : w1;
        split3(bf16_lo(xf[i]) * w.x, bf16_hi(xf[i]) * w.y, hi[i], mid[i], lo[i]);
      }
#pragma unroll
      for (int np = 0; np < 8; ++np) {
        uint32_t b[4];
        frag_b2_t(b, st + OFF_B, kN * 2, 16 * np, 16 * k, lane);
        mma16816(hs[2 * np], lo, b[0], b[1]);
        mma16816(hs[2 * np + 1], lo, b[2], b[3]);
        mma16816(hs[2 * np], mid, b[0], b[1]);
        mma16816(hs[2 * np + 1], mid, b[2], b[3]);
        mma16816(hs[2 * np], hi, b[0], b[1]);
        mma16816(hs[2 * np + 1], hi, b[2], b[3]);
      }
    }
    if (!STATE_ONLY && c + 1 < c1) put_state();
  }
  if (STATE_ONLY || c1 == nch) {
    float* out = STATE_ONLY ? ws + seg * wrec : a.h_out + hbase;
#pragma unroll
    for (int nt = 0; nt < 16; ++nt) {
      const int n = nt * 8 + 2 * q4;
      *reinterpret_cast<float2*>(out + (16 * warp + g) * kN + n) = make_float2(hs[nt][0], hs[nt][1]);
      *reinterpret_cast<float2*>(out + (16 * warp + g + 8) * kN + n) = make_float2(hs[nt][2], hs[nt][3]);
    }
    if (STATE_ONLY && tid == 0) out[kP * kN] = exp2_sfu(seg_sum * kLog2e);
  }
}

// Segments per sequence.  A sequence's chunks run one after the other in a CTA, two CTAs to an SM; where the (sequence,
// head) pairs leave SMs idle its chunks are cut into segments: a first grid computes what each segment but the last adds
// to the state, the second runs all of them from their start states.  A segment has four chunks at least.
int plan_segments(int H, int n_seq, int max_len) {
  const long long pairs = (long long)H * n_seq, slots = 2 * kSMs;
  const int nch = (max_len + Q - 1) / Q;
  int nseg = (int)(slots / (pairs > 0 ? pairs : 1));
  if (nseg > nch / 4) nseg = nch / 4;
  if (nseg > 16) nseg = 16;
  return nseg < 2 ? 1 : nseg;
}

}  // namespace

size_t prompt_scan_workspace_bytes(int H, int G, int n_seq, int n_tok, int max_len) {
  if (prompt_scan_tc_fits(H, G, n_seq, max_len)) return prompt_scan_tc_workspace_bytes(H, G, n_seq, n_tok, max_len);
  const int nseg = plan_segments(H, n_seq, max_len);
  return 256 + (size_t)n_seq * H * (nseg > 1 ? nseg : 0) * (kP * kN + 32) * sizeof(float);
}

cudaError_t launch_prompt_scan(const ScanArgs& args, void* workspace, cudaStream_t s) {
  if (args.q.n_seq == 0) return cudaSuccess;
  if (prompt_scan_tc_fits(args.H, args.G, args.q.n_seq, args.q.max_len)) return launch_prompt_scan_tc(args, workspace, s);
  ScanArgs a = args;
  a.nseg = plan_segments(a.H, a.q.n_seq, a.q.max_len);
  a.seg_state = static_cast<float*>(workspace);
  static bool done[2][64];
  cudaError_t e = allow_smem(prompt_scan_kernel<false>, SMEM, done[0]);
  if (e == cudaSuccess) e = allow_smem(prompt_scan_kernel<true>, SMEM, done[1]);
  if (e != cudaSuccess) return e;
  if (a.nseg > 1)
    prompt_scan_kernel<true><<<dim3((unsigned)a.H, (unsigned)(a.q.n_seq * (a.nseg - 1))), THREADS, SMEM, s>>>(a);
  prompt_scan_kernel<false><<<dim3((unsigned)a.H, (unsigned)(a.q.n_seq * a.nseg)), THREADS, SMEM, s>>>(a);
  return cudaGetLastError();
}

}  // namespace ssmtree
