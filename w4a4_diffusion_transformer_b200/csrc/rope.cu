// Rotary positions with several axes, with the per-head RMS norm of queries
// and keys in front of them.
//
// A head of D values rotates its first R = sum of the axes' sizes; pair p of
// axis a with position s turns by the angle s theta^(-2i/d), i the pair's index
// in its axis and d the axis' size (or i = p, d = R with the span-wide
// frequencies):
//
//   n = x / sqrt(mean(x^2) + eps) w              (optional, over the whole head)
//   u' = u cos - v sin,  v' = v cos + u sin      (u, v) = n's pair p
//
// Pairs are neighbours (2p, 2p + 1) or half the span apart (p, p + R/2).  The
// angle is formed in turns, in float64, and reduced to one turn before it
// becomes FP32: positions of many thousands keep their angle to FP32 accuracy.
// Everything else is FP32 with one rounding to BF16.
//
// Memory bound: every value of q and k is read and written once.  A warp takes
// one token (S warps share one when there are few): its lanes own 8 consecutive
// values of a head, so the cosines and sines of a lane are computed once per
// token and stay in registers for all heads, and its frequencies once per
// kernel.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kernels.h"
#include "sm100.cuh"

namespace svdq {

namespace {

constexpr int kWarps = 8;
constexpr int kUnroll = 4;                              // heads in flight per lane

__device__ __forceinline__ float2 unpack2(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// kLanes lanes hold a head (the power of two that holds D / 8).
template <int kLanes, bool kHalf>
__device__ __forceinline__ void rotate_heads(const RopeParams& p, const RopeTensor& t, int b, int tok, int split,
                                             const float (&cs)[kHalf ? 8 : 4], const float (&sn)[kHalf ? 8 : 4],
                                             int partner, int turned) {
  constexpr int kPerWarp = 32 / kLanes;                 // heads a warp handles at once
  const int lane = threadIdx.x & 31;
  const int c = lane % kLanes, sub = lane / kLanes;
  const bool act = 8 * c < p.D;
  const __nv_bfloat16* in = t.in + b * t.in_batch + tok * t.in_token + 8 * c;
  __nv_bfloat16* out = t.out + b * t.out_batch + tok * t.out_token + 8 * c;
  // the weight of this lane's values, and (halves) of its partner's
  uint4 wq = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u), wp = wq;
  if (t.weight && act) {
    wq = *reinterpret_cast<const uint4*>(t.weight + 8 * c);
    if (kHalf) wp = *reinterpret_cast<const uint4*>(t.weight + 8 * (partner % kLanes));
  }
  const uint32_t wa[4] = {wq.x, wq.y, wq.z, wq.w}, wb[4] = {wp.x, wp.y, wp.z, wp.w};
  const float invD = 1.0f / (float)p.D;
  const int step = kPerWarp * p.splits;
  for (int h0 = split * kPerWarp; h0 < t.heads; h0 += step * kUnroll) {
    uint4 raw[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int h = h0 + u * step + sub;
      raw[u] = make_uint4(0u, 0u, 0u, 0u);
      if (act && h < t.heads) raw[u] = *reinterpret_cast<const uint4*>(in + h * t.in_head);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int h = h0 + u * step + sub;
      const uint32_t w[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
      float2 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = unpack2(w[i]);
      float r = 1.0f;
      if (p.norm) {
        float2 a = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < 4; ++i) a = __ffma2_rn(v[i], v[i], a);
        float s = a.x + a.y;
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        r = rsqrtf(s * invD + p.eps);
      }
      const float2 r2 = make_float2(r, r);
      float2 q[4];                                      // halves: the partner's values
      if (kHalf) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          q[i] = unpack2(__shfl_sync(0xffffffffu, w[i], partner));
          if (p.norm) q[i] = __fmul2_rn(__fmul2_rn(q[i], r2), unpack2(wb[i]));
        }
      }
      if (p.norm) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __fmul2_rn(__fmul2_rn(v[i], r2), unpack2(wa[i]));
      }
      uint32_t o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (kHalf)                                      // sn carries the sign of this lane's half
          o[i] = pack2(v[i].x * cs[(2 * i) & 7] + q[i].x * sn[(2 * i) & 7],
                       v[i].y * cs[(2 * i + 1) & 7] + q[i].y * sn[(2 * i + 1) & 7]);
        else
          o[i] = pack2(v[i].x * cs[i & 3] - v[i].y * sn[i & 3], v[i].y * cs[i & 3] + v[i].x * sn[i & 3]);
        // values past the span are not multiplied at all: an infinity or NaN
        // beside one stays where it is
        if (i >= turned) o[i] = pack2(v[i].x, v[i].y);
      }
      if (act && h < t.heads) *reinterpret_cast<uint4*>(out + h * t.out_head) = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

template <int kLanes, bool kHalf>
__global__ void __launch_bounds__(kWarps * 32) rope_kernel(const RopeParams p) {
  constexpr int kAng = kHalf ? 8 : 4;                   // angles of a lane's 8 values
  dev::griddep_launch_dependents();
  const int lane = threadIdx.x & 31, c = lane % kLanes;
  const int R2 = p.R / 2;
  // this lane's frequencies in turns per position, and their axes
  double freq[kAng];
  int axis[kAng];
  // this lane's pairs of neighbouring values that turn: its first `turned`
  const int turned = max(0, min(4, (p.R - 8 * c) / 2));
#pragma unroll
  for (int i = 0; i < kAng; ++i) {
    int pr = kHalf ? 8 * c + i : 4 * c + i;
    bool in = kHalf ? 8 * c + i < p.R : pr < R2;
    if (kHalf && pr >= R2) pr -= R2;
    freq[i] = 0.0;
    axis[i] = 0;
    if (in) {
      int first = 0, a = 0;
      while (a + 1 < p.axes && pr >= first + p.dim[a] / 2) first += p.dim[a++] / 2;
      const double e = p.span ? 2.0 * pr / p.R : 2.0 * (pr - first) / p.dim[a];
      freq[i] = exp2(-e * p.log2_theta) * 0.15915494309189533577;   // 1 / (2 pi)
      axis[i] = a;
    }
  }
  int partner = lane;
  float sign = 1.0f;
  if (kHalf && 8 * c < p.R) {
    const bool first = 8 * c < R2;
    partner = first ? lane + R2 / 8 : lane - R2 / 8;
    sign = first ? -1.0f : 1.0f;
  }
  dev::griddep_wait();                                  // q, k and the positions may be the preceding kernel's

  const long long units = (long long)p.B * p.T * p.splits;
  for (long long u = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5); u < units;
       u += (long long)gridDim.x * kWarps) {
    const int split = (int)(u % p.splits);
    const int row = (int)(u / p.splits), b = row / p.T, tok = row % p.T;
    const float* pos = p.positions + b * p.pos_batch + (long long)tok * p.axes;
    float cs[kAng], sn[kAng];
#pragma unroll
    for (int i = 0; i < kAng; ++i) {
      const double turns = (double)pos[axis[i]] * freq[i];
      sincospif(2.0f * (float)(turns - rint(turns)), &sn[i], &cs[i]);
      if (kHalf) sn[i] *= sign;
    }
    rotate_heads<kLanes, kHalf>(p, p.q, b, tok, split, cs, sn, partner, turned);
    if (p.k.heads > 0) rotate_heads<kLanes, kHalf>(p, p.k, b, tok, split, cs, sn, partner, turned);
  }
}

template <int kLanes>
cudaError_t launch(const RopeParams& p, int grid, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return p.half ? cudaLaunchKernelEx(&cfg, rope_kernel<kLanes, true>, p)
                : cudaLaunchKernelEx(&cfg, rope_kernel<kLanes, false>, p);
}

}  // namespace

cudaError_t launch_rope(RopeParams p, int num_sms, cudaStream_t stream) {
  int lanes = 1;
  while (lanes * 8 < p.D) lanes *= 2;
  // Enough warps to fill the GPU (32 per SM) by splitting a token's heads when
  // there are few tokens; a split below one unrolled step brings nothing.
  const long long rows = (long long)p.B * p.T;
  const int heads = p.q.heads > p.k.heads ? p.q.heads : p.k.heads;
  const int most = (heads * lanes + 31) / 32;
  const long long want = (32LL * num_sms + rows - 1) / rows;
  p.splits = (int)(want < 1 ? 1 : want > most ? most : want);
  const long long units = rows * p.splits, blocks = (units + kWarps - 1) / kWarps;
  const int grid = (int)(blocks < 8LL * num_sms ? blocks : 8LL * num_sms);
  switch (lanes) {
    case 1: return launch<1>(p, grid, stream);
    case 2: return launch<2>(p, grid, stream);
    case 4: return launch<4>(p, grid, stream);
    case 8: return launch<8>(p, grid, stream);
    case 16: return launch<16>(p, grid, stream);
    default: return launch<32>(p, grid, stream);
  }
}

}  // namespace svdq
