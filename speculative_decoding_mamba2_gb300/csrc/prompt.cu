// The conv of prompts and the recurrence of single tokens (ssm_prompt.h).
//
// prompt_conv_kernel.  post[t][c] = SiLU(b[c] + sum_k w[c][k] row[t-3+k][c]): four products and one SiLU
// per element against 4 bytes of traffic, so HBM binds long prompts.  A CTA takes TB tokens of one
// sequence and all channels, a thread 8 channels (16-byte loads); its rows and the three before them are
// in flight together and the window then slides in registers, so a row is read 1 + 3/TB times, all but
// the first time from L2.  Blocks follow the sequences (grid y), not the token rows: only a sequence's
// first block reads its ring, and the same threads then write the ring's new rows and advance its head,
// so one launch needs no order between CTAs.
//
// scan_step_kernel.  h' = a h + D x (x) B, y = C h' + D x for one token: 4 operations for each 8 bytes of
// state, HBM bound.  A CTA takes one head's 64 x 128 state, a warp 8 of its rows with their 8 row loads in
// flight, lane l columns 4l .. 4l+3; the 8 row sums of C h' are reduced together (each shuffle halves the
// rows a lane carries: 9 shuffles instead of 40).
#include "prompt.cuh"

namespace ssmtree {
namespace {

constexpr int TB = 8;  // tokens per conv CTA

struct Row8 {  // 8 channels of a row, fp32
  float v[8];
};
__device__ __forceinline__ Row8 row8(uint4 u) {
  Row8 r;
  r.v[0] = bf16_lo(u.x), r.v[1] = bf16_hi(u.x), r.v[2] = bf16_lo(u.y), r.v[3] = bf16_hi(u.y);
  r.v[4] = bf16_lo(u.z), r.v[5] = bf16_hi(u.z), r.v[6] = bf16_lo(u.w), r.v[7] = bf16_hi(u.w);
  return r;
}
__device__ __forceinline__ uint32_t pack2bf(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__global__ void __launch_bounds__(256) prompt_conv_kernel(ConvArgs a) {
  const int s = blockIdx.y, t0 = blockIdx.x * TB;
  int first, len, slot;
  if (!seq_range(a.q, s, first, len, slot)) {
    if (t0 == 0 && threadIdx.x == 0) flag(a.q.status, SSM_STATUS_SEQ_RANGE);
    return;
  }
  if (t0 >= len) return;
  const int nt = min(TB, len - t0), cd = a.conv_dim;
  const long long inst = (long long)slot * a.L + a.layer;
  const int head = t0 == 0 ? a.ring_head[inst] : 0;
  uint16_t* ring = a.ring + inst * a.R * cd;
  for (int c = 8 * threadIdx.x; c < cd; c += 8 * blockDim.x) {
    const uint16_t* x = a.x + (long long)(first + t0) * a.ldx + c;
    uint4 in[TB + 3];
    if (t0 == 0) {
#pragma unroll
      for (int j = 0; j < 3; ++j)
        in[j] = *reinterpret_cast<const uint4*>(ring + (long long)ring_pos(head, j - 3, a.R) * cd + c);
    } else {
#pragma unroll
      for (int j = 0; j < 3; ++j) in[j] = *reinterpret_cast<const uint4*>(x + (j - 3) * a.ldx);
    }
#pragma unroll
    for (int j = 0; j < TB; ++j)
      if (j < nt) in[3 + j] = *reinterpret_cast<const uint4*>(x + j * a.ldx);
    float4 w[8];
    float b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      w[i] = *reinterpret_cast<const float4*>(a.conv_w + (size_t)(c + i) * 4);
      b[i] = a.conv_b[c + i];
    }
    uint16_t* o = a.out + (long long)(first + t0) * a.ldo + c;
    Row8 r0 = row8(in[0]), r1 = row8(in[1]), r2 = row8(in[2]);
#pragma unroll
    for (int j = 0; j < TB; ++j) {
      if (j < nt) {
        const Row8 r3 = row8(in[3 + j]);
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = silu_fast(conv4_acc(w[i], b[i], r0.v[i], r1.v[i], r2.v[i], r3.v[i]));
        *reinterpret_cast<uint4*>(o + j * a.ldo) =
            make_uint4(pack2bf(v[0], v[1]), pack2bf(v[2], v[3]), pack2bf(v[4], v[5]), pack2bf(v[6], v[7]));
        r0 = r1, r1 = r2, r2 = r3;
      }
    }
    if (t0 == 0) {  // the sequence's last rows into the ring (this thread has read its channels of the old ones)
      const uint16_t* xl = a.x + (long long)first * a.ldx + c;
      for (int t = max(0, len - 3); t < len; ++t)
        *reinterpret_cast<uint4*>(ring + (long long)ring_pos(head, t, a.R) * cd + c) =
            *reinterpret_cast<const uint4*>(xl + t * a.ldx);
    }
  }
  if (t0 == 0) {
    __syncthreads();  // every thread has read the head
    if (threadIdx.x == 0) a.ring_head[inst] = head + len;
  }
}

__global__ void __launch_bounds__(256) scan_step_kernel(ScanArgs a) {
  const int h = blockIdx.x, s = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int slot = a.q.slots ? a.q.slots[s] : s;
  if (slot < 0 || slot >= a.q.n_slots) {
    if (h == 0 && threadIdx.x == 0) flag(a.q.status, SSM_STATUS_SEQ_RANGE);
    return;
  }
  const long long base = (((long long)slot * a.L + a.layer) * a.H + h) * (kP * kN) + warp * 8 * kN + 4 * lane;
  float4 hv[8];
  if (a.h_in) {
#pragma unroll
    for (int i = 0; i < 8; ++i) hv[i] = *reinterpret_cast<const float4*>(a.h_in + base + i * kN);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) hv[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  const int grp = h / (a.H / a.G);
  const uint2 bb = *reinterpret_cast<const uint2*>(a.B + (long long)s * a.ldb + grp * kN + 4 * lane);
  const uint2 cc = *reinterpret_cast<const uint2*>(a.C + (long long)s * a.ldc + grp * kN + 4 * lane);
  const uint4 xx = *reinterpret_cast<const uint4*>(a.x + (long long)s * a.ldx + h * kP + warp * 8);
  const float delta = softplus_f(bf16f(a.dt[(long long)s * a.lddt + h]) + a.dt_bias[h]);
  const float decay = decay_of(delta, neg_exp(a.A_log[h]));
  const Row8 x = row8(xx);
  const float4 b = make_float4(bf16_lo(bb.x), bf16_hi(bb.x), bf16_lo(bb.y), bf16_hi(bb.y));
  const float4 c = make_float4(bf16_lo(cc.x), bf16_hi(cc.x), bf16_lo(cc.y), bf16_hi(cc.y));
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float u = delta * x.v[i];
    hv[i].x = ssm_update(decay, hv[i].x, u, b.x);
    hv[i].y = ssm_update(decay, hv[i].y, u, b.y);
    hv[i].z = ssm_update(decay, hv[i].z, u, b.z);
    hv[i].w = ssm_update(decay, hv[i].w, u, b.w);
    *reinterpret_cast<float4*>(a.h_out + base + i * kN) = hv[i];
    y[i] = fmaf(hv[i].x, c.x, fmaf(hv[i].y, c.y, fmaf(hv[i].z, c.z, hv[i].w * c.w)));
  }
  // 8 row sums over 32 lanes: after the exchange over lane bit 4, 3, 2 a lane carries 4, 2, 1 rows
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float keep = lane & 16 ? y[i + 4] : y[i], give = lane & 16 ? y[i] : y[i + 4];
    y[i] = keep + __shfl_xor_sync(0xffffffffu, give, 16);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float keep = lane & 8 ? y[i + 2] : y[i], give = lane & 8 ? y[i] : y[i + 2];
    y[i] = keep + __shfl_xor_sync(0xffffffffu, give, 8);
  }
  {
    const float keep = lane & 4 ? y[1] : y[0], give = lane & 4 ? y[0] : y[1];
    y[0] = keep + __shfl_xor_sync(0xffffffffu, give, 4);
  }
  y[0] += __shfl_xor_sync(0xffffffffu, y[0], 2);
  y[0] += __shfl_xor_sync(0xffffffffu, y[0], 1);
  if ((lane & 3) == 0) {
    const int row = lane >> 2;  // lane bits 4, 3, 2 = row bits 2, 1, 0
    const float xr = bf16f(a.x[(long long)s * a.ldx + h * kP + warp * 8 + row]);
    a.y[(long long)s * a.ldy + h * kP + warp * 8 + row] = (uint16_t)(pack2bf(fmaf(a.D[h], xr, y[0]), 0.f) & 0xffffu);
  }
}

}  // namespace

cudaError_t launch_prompt_conv(const ConvArgs& a, cudaStream_t s) {
  if (a.q.n_seq == 0 || a.q.n_tok == 0 || a.q.max_len == 0) return cudaSuccess;
  // channel vectors in equal passes of at most 256 threads, whole warps
  const int nv = a.conv_dim / 8, passes = (nv + 255) / 256;
  const int threads = ((nv + passes - 1) / passes + 31) / 32 * 32;
  const dim3 grid((unsigned)((min(a.q.max_len, a.q.n_tok) + TB - 1) / TB), (unsigned)a.q.n_seq);
  prompt_conv_kernel<<<grid, threads, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_scan_step(const ScanArgs& a, cudaStream_t s) {
  if (a.q.n_seq == 0) return cudaSuccess;
  scan_step_kernel<<<dim3((unsigned)a.H, (unsigned)a.q.n_seq), 256, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace ssmtree
