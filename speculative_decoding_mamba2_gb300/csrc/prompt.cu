// The conv of prompts and the recurrence of single tokens (ssm_prompt.h).
//
// prompt_conv_kernel.  post[t][c] = SiLU(b[c] + sum_k w[c][k] row[t-3+k][c]): four products and one SiLU per element against
// 4 bytes of traffic, so HBM and the special-function unit (two results an element) bind long prompts.  A block takes TB
// tokens of one sequence and up to CB channels: all its rows and the three before them are asked for at once (cp.async,
// 54 KB a block, four blocks to an SM), then a thread slides over them with its pair of channels, eight
// tokens as soon as they are there; a row is read 1 + 3/TB times, the second time from L2.  8209 tokens of 5376 channels take
// 35 us (177 MB: 5.0 TB/s; issue slots 74 % taken).  With the rows in registers the loads of a block could not run beside
// another's arithmetic: 60 us at best.  Tiles follow the sequences (grid y), not the token rows: only a sequence's first tile
// reads its ring, and the same threads then write the ring's new rows; the head is advanced once the channel blocks, a
// cluster, have read it, so one launch needs no other order.
//
// scan_step_kernel.  h' = a h + D x (x) B, y = C h' + D x for one token: 4 operations for each 8 bytes of
// state, HBM bound.  A CTA takes one head's 64 x 128 state, a warp 8 of its rows with their 8 row loads in
// flight, lane l columns 4l .. 4l+3; the 8 row sums of C h' are reduced together (each shuffle halves the
// rows a lane carries: 9 shuffles instead of 40).  Back to back, 128 sequences of 80 heads take 101 us: 674 MB
// at 6.7 TB/s.
#include "mma_tiles.cuh"
#include "prompt.cuh"

namespace ssmtree {
namespace {

constexpr int TB = 32;              // tokens per conv block
constexpr int CB = 768;             // channels at most
constexpr int CONV_THREADS = CB / 2;
constexpr int CONV_SMEM = (TB + 3) * CB * 2;

__device__ __forceinline__ uint32_t pack2bf(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

struct Row8 {  // 8 channels of a row, fp32
  float v[8];
};
__device__ __forceinline__ Row8 row8(uint4 u) {
  Row8 r;
  r.v[0] = bf16_lo(u.x), r.v[1] = bf16_hi(u.x), r.v[2] = bf16_lo(u.y), r.v[3] = bf16_hi(u.y);
  r.v[4] = bf16_lo(u.z), r.v[5] = bf16_hi(u.z), r.v[6] = bf16_lo(u.w), r.v[7] = bf16_hi(u.w);
  return r;
}
// SiLU v / (1 + 2^(-v log2 e)) on the special-function unit (relative error about 1e-6; where 2^t is infinite the quotient is 0)
__device__ __forceinline__ float silu_sfu(float v) {
  float e, q;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(v * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(q) : "f"(1.f + e));
  return v * q;
}

__global__ void __launch_bounds__(CONV_THREADS, 4) prompt_conv_kernel(ConvArgs a) {
  extern __shared__ __align__(16) uint16_t rows_s[];
  const int s = blockIdx.y, t0 = blockIdx.x * TB, tid = threadIdx.x, cb = 2 * blockDim.x;
  int first, len, slot;
  if (!seq_range(a.q, s, first, len, slot)) {
    if (t0 == 0 && blockIdx.z == 0 && tid == 0) flag(a.q.status, SSM_STATUS_SEQ_RANGE);
    return;
  }
  if (t0 >= len) return;
  const int nt = min(TB, len - t0), cd = a.conv_dim;
  const long long inst = (long long)slot * a.L + a.layer;
  const int head = t0 == 0 ? a.ring_head[inst] : 0;
  if (t0 == 0) asm volatile("barrier.cluster.arrive.release.aligned;\n" ::: "memory");  // the head has been read
  uint16_t* ring = a.ring + inst * a.R * cd;
#pragma unroll 1
  for (int c0 = blockIdx.z * cb; c0 < cd; c0 += cb * gridDim.z) {  // (more than once above 8 blocks of channels)
    if (c0 >= cb * gridDim.z) __syncthreads();  // the last rows have been read
    {  // rows t0 - 3 .. t0 + nt - 1, four at a time, in groups of eight
      const int chunks = cb / 8, ch = tid % chunks, r0 = tid / chunks;
      uint16_t* dst = rows_s + r0 * cb + ch * 8;
      const int last = c0 + ch * 8 < cd ? nt + 3 : 0;
      const long long step = 4 * a.ldx;
      const uint16_t* x = a.x + (long long)(first + t0 - 3 + r0) * a.ldx + c0 + ch * 8;
#pragma unroll
      for (int k = 0; k < (TB + 3 + 3) / 4; ++k) {
        if (r0 + 4 * k < last)
          cp_async16(dst, k == 0 && t0 == 0 && r0 < 3 ? ring + (long long)ring_pos(head, r0 - 3, a.R) * cd + c0 + ch * 8 : x);
        x += step, dst += 4 * cb;
        if (k & 1) cp_async_commit();
      }
      cp_async_commit();
    }
    const int c = c0 + 2 * tid;
    const bool mine = c < cd;
    float4 u = {}, v = {};
    float2 bb = {};
    if (mine) {
      u = *reinterpret_cast<const float4*>(a.conv_w + (size_t)c * 4);
      v = *reinterpret_cast<const float4*>(a.conv_w + (size_t)c * 4 + 4);
      bb = *reinterpret_cast<const float2*>(a.conv_b + c);
    }
    const uint32_t* col = reinterpret_cast<const uint32_t*>(rows_s) + tid;
    const int pitch = cb / 2;  // words of a row
    uint32_t* o = reinterpret_cast<uint32_t*>(a.out + (long long)(first + t0) * a.ldo + c);
    const long long ld = a.ldo / 2;
    const int stores = mine ? nt : 0;
    float l0 = 0.f, l1 = 0.f, l2 = 0.f, h0 = 0.f, h1 = 0.f, h2 = 0.f;  // the three rows before, of either channel
#pragma unroll
    for (int g = 0; g < TB / 8; ++g) {  // eight tokens: their rows are in the first g + 2 groups
      if (8 * g >= nt && g > 0) continue;  // (the same for the whole block)
      if (g == 0)
        cp_async_wait<TB / 8 - 1>();
      else if (g == 1)
        cp_async_wait<TB / 8 - 2>();
      else if (g == 2)
        cp_async_wait<TB / 8 - 3>();
      else
        cp_async_wait<0>();
      __syncthreads();
      if (g == 0) {
        const uint32_t r0 = col[0], r1 = col[pitch], r2 = col[2 * pitch];
        l0 = bf16_lo(r0), l1 = bf16_lo(r1), l2 = bf16_lo(r2), h0 = bf16_hi(r0), h1 = bf16_hi(r1), h2 = bf16_hi(r2);
        col += 3 * pitch;
      }
#pragma unroll
      for (int j = 8 * g; j < 8 * g + 8; ++j) {
        const uint32_t r = *col;  // (behind the last row: whatever stands there, for no output)
        col += pitch;
        const float l3 = bf16_lo(r), h3 = bf16_hi(r);
        const uint32_t y = pack2bf(silu_sfu(conv4_acc(u, bb.x, l0, l1, l2, l3)), silu_sfu(conv4_acc(v, bb.y, h0, h1, h2, h3)));
        if (j < stores) *o = y;
        o += ld;  // (a pointer that moves: products j * ldo took three quarters of the instructions)
        l0 = l1, l1 = l2, l2 = l3, h0 = h1, h1 = h2, h2 = h3;
      }
    }
    if (t0 == 0 && mine) {  // the sequence's last rows into the ring (its old ones are in shared memory)
      const uint16_t* xl = a.x + (long long)first * a.ldx + c;
#pragma unroll 1
      for (int t = max(0, len - 3); t < len; ++t)
        *reinterpret_cast<uint32_t*>(ring + (long long)ring_pos(head, t, a.R) * cd + c) =
            *reinterpret_cast<const uint32_t*>(xl + t * a.ldx);
    }
  }
  if (t0 == 0) {
    asm volatile("barrier.cluster.wait.acquire.aligned;\n" ::: "memory");
    if (blockIdx.z == 0 && tid == 0) a.ring_head[inst] = head + len;
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
  if (a.q.n_seq == 0) return cudaSuccess;
  // the channels over blocks of equal size, whole warps; a cluster has 8 of them at most
  const int need = (a.conv_dim + CB - 1) / CB, blocks = min(8, need);
  static bool done[64];
  cudaError_t e = allow_smem(prompt_conv_kernel, CONV_SMEM, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  const int tiles = max(1, (min(a.q.max_len, a.q.n_tok) + TB - 1) / TB);  // (the first one checks the sequence)
  cfg.gridDim = dim3((unsigned)tiles, (unsigned)a.q.n_seq, (unsigned)blocks);
  cfg.blockDim = dim3((unsigned)(((a.conv_dim + need - 1) / need + 63) / 64 * 32));
  cfg.dynamicSmemBytes = (size_t)(TB + 3) * cfg.blockDim.x * 4;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 1, attr[0].val.clusterDim.y = 1, attr[0].val.clusterDim.z = (unsigned)blocks;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, prompt_conv_kernel, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_scan_step(const ScanArgs& a, cudaStream_t s) {
  if (a.q.n_seq == 0) return cudaSuccess;
  scan_step_kernel<<<dim3((unsigned)a.H, (unsigned)a.q.n_seq), 256, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace ssmtree
