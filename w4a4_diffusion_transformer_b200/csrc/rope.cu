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
// Memory bound: every value of q and k is read and written once.  A CTA takes
// 4 / S tokens of a sequence, S warps to a token.  Its threads first form the
// tokens' angles together (as every warp's own work, with the frequencies, they
// cost more than the rotation itself) while each warp's first heads are already
// on their way.  A lane then owns 8 consecutive values of a head: the products of
// its weights with its cosines and sines stay in registers for all heads, so that
// a head costs its norm and two multiply-adds a value.
//
// 4608 tokens, 24 + 24 heads of 128: 21.6 us, 5.25 TB/s of a copy's 6.56 (a warp
// per token with its own angles: 40.3); 2 x 14040 tokens, 12 + 12 heads: 70.0 us,
// 4.93 TB/s.  What counts is warps in flight: 32 per SM at 64 registers (24 at
// 80: 27.0 us), and few instructions in front of a token's heads (8 head steps
// a warp instead of 24: 27.0 us).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kernels.h"
#include "sm100.cuh"

namespace svdq {

namespace {

constexpr int kWarps = 4;
constexpr int kSteps = 32;                              // head steps of a warp when there are tokens enough
constexpr int kUnroll = 4;                              // heads in flight per lane

__device__ __forceinline__ float2 unpack2(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// The heads of one tensor that a warp takes of its token: h0, h0 + step, ...
struct Walk {
  const __nv_bfloat16* in;                              // this lane's values of the next head to load
  __nv_bfloat16* out;                                   // ... to store
  long long in_step, out_step;
  int loads, stores;                                    // heads left

  __device__ __forceinline__ void load(uint4 (&raw)[kUnroll]) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      raw[u] = make_uint4(0u, 0u, 0u, 0u);
      if (loads > 0) raw[u] = *reinterpret_cast<const uint4*>(in);
      in += in_step;
      --loads;
    }
  }
  __device__ __forceinline__ void store(const uint4& v) {
    if (stores > 0) *reinterpret_cast<uint4*>(out) = v;
    out += out_step;
    --stores;
  }
};

template <int kLanes>
__device__ __forceinline__ Walk walk(const RopeParams& p, const RopeTensor& t, int b, int tok, int split) {
  const int lane = threadIdx.x & 31, c = lane % kLanes;
  const int h0 = split * (32 / kLanes) + lane / kLanes, step = (32 / kLanes) << p.log2_splits;
  Walk w;
  w.in = t.in + b * t.in_batch + tok * t.in_token + h0 * t.in_head + 8 * c;
  w.out = t.out + b * t.out_batch + tok * t.out_token + h0 * t.out_head + 8 * c;
  w.in_step = step * t.in_head;
  w.out_step = step * t.out_head;
  w.loads = 8 * c < p.D && tok < p.T ? (t.heads - h0 + step - 1) / step : 0;
  w.stores = w.loads;
  return w;
}

// One tensor's heads.  kLanes lanes hold a head (the power of two that holds
// D / 8); raw: the first heads, already loaded; angle: cosine and sine of this
// lane's first pair.
template <int kLanes, bool kHalf>
__device__ __forceinline__ void rotate_heads(const RopeParams& p, const RopeTensor& t, Walk& w,
                                             uint4 (&raw)[kUnroll], const float2* angle, int partner, int turned,
                                             float sign) {
  const int c = (threadIdx.x & 31) % kLanes;
  // out = x a + (the pair's other value) b, both with the weight that x and the
  // other carry; the head's 1 / sqrt follows
  float2 a[4], b[4];
  {
    uint4 q = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u), o = q;   // ones
    if (p.norm && t.weight && 8 * c < p.D) {
      q = *reinterpret_cast<const uint4*>(t.weight + 8 * c);
      o = *reinterpret_cast<const uint4*>(t.weight + 8 * (partner % kLanes));
    }
    const uint32_t qs[4] = {q.x, q.y, q.z, q.w}, os[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 x = unpack2(qs[i]);
      if (kHalf) {
        float2 u = make_float2(1.f, 0.f), v = u;
        if (turned > 0) {
          u = angle[2 * i];
          v = angle[2 * i + 1];
        }
        const float2 y = unpack2(os[i]);
        a[i] = make_float2(x.x * u.x, x.y * v.x);
        b[i] = make_float2(sign * y.x * u.y, sign * y.y * v.y);
      } else {
        const float2 u = i < turned ? angle[i] : make_float2(1.f, 0.f);
        a[i] = make_float2(x.x * u.x, x.y * u.x);
        b[i] = make_float2(-x.y * u.y, x.x * u.y);
      }
    }
  }
  const float invD = 1.0f / (float)p.D;
  const bool whole = p.R == p.D;                        // every value of a head turns
  const int step = (32 / kLanes) << p.log2_splits;
  for (int h = 0; h < t.heads; h += kUnroll * step) {   // uniform over the warp: the shuffles need every lane
    if (h > 0) w.load(raw);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (u > 0 && h + u * step >= t.heads) break;      // uniform too
      const uint32_t x[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
      float2 v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = unpack2(x[k]);
      float2 r2 = make_float2(1.f, 1.f);
      if (p.norm) {
        float2 q = __fmul2_rn(v[0], v[0]);
#pragma unroll
        for (int k = 1; k < 4; ++k) q = __ffma2_rn(v[k], v[k], q);
        float s = q.x + q.y;
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        r2.x = r2.y = rsqrtf(s * invD + p.eps);
      }
      uint32_t o[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 other = kHalf ? unpack2(__shfl_sync(0xffffffffu, x[k], partner)) : make_float2(v[k].y, v[k].x);
        const float2 y = __fmul2_rn(__ffma2_rn(v[k], a[k], __fmul2_rn(other, b[k])), r2);
        o[k] = pack2(y.x, y.y);
      }
      if (!whole) {
        // values past the span are not multiplied by a sine at all: an infinity
        // or NaN beside one stays where it is
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 y = __fmul2_rn(__fmul2_rn(v[k], a[k]), r2);
          if (k >= turned) o[k] = pack2(y.x, y.y);
        }
      }
      w.store(make_uint4(o[0], o[1], o[2], o[3]));
    }
  }
}

template <int kLanes, bool kHalf>
__global__ void __launch_bounds__(kWarps * 32, 8) rope_kernel(const __grid_constant__ RopeParams p) {
  __shared__ float2 angles[kWarps * 128];               // cosine, sine of [token][pair]
  dev::griddep_launch_dependents();
  dev::griddep_wait();                                  // q, k and the positions may be the preceding kernel's
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = lane % kLanes;
  const int R2 = p.R / 2, b = blockIdx.y, tok0 = blockIdx.x * (kWarps >> p.log2_splits);
  const int tok = tok0 + (warp >> p.log2_splits), split = warp & ((1 << p.log2_splits) - 1);
  Walk w = walk<kLanes>(p, p.q, b, tok, split);
  uint4 raw[kUnroll];
  w.load(raw);

  // angles [token][2^log2_pairs]: no division to find a thread's token and pair
  const float* pos = p.positions + b * p.pos_batch;
  for (int i = threadIdx.x; i < (kWarps >> p.log2_splits) << p.log2_pairs; i += kWarps * 32) {
    const int t = tok0 + (i >> p.log2_pairs), pr = i & ((1 << p.log2_pairs) - 1);
    if (t < p.T && pr < R2) {
      int axis = 0;
      for (int last = p.dim[0] / 2; pr >= last; last += p.dim[axis] / 2) ++axis;
      const double turns = (double)pos[(long long)t * p.axes + axis] * p.turns[pr];
      float2 v;
      sincospif(2.0f * (float)(turns - rint(turns)), &v.y, &v.x);
      angles[i] = v;
    }
  }
  __syncthreads();
  if (tok >= p.T) return;

  // this lane's first `turned` pairs of neighbouring values turn (half-span
  // pairs: all 8 values or none)
  const int turned = kHalf ? (8 * c < p.R ? 4 : 0) : max(0, min(4, (p.R - 8 * c) / 2));
  const bool second = kHalf && 8 * c >= R2;
  int partner = lane;
  if (kHalf && turned > 0) partner = second ? lane - R2 / 8 : lane + R2 / 8;
  const float2* angle = angles + ((warp >> p.log2_splits) << p.log2_pairs) + (kHalf ? 8 * c - (second ? R2 : 0) : 4 * c);
  const float sign = second ? 1.0f : -1.0f;
  rotate_heads<kLanes, kHalf>(p, p.q, w, raw, angle, partner, turned, sign);
  if (p.k.heads > 0) {
    w = walk<kLanes>(p, p.k, b, tok, split);
    w.load(raw);
    rotate_heads<kLanes, kHalf>(p, p.k, w, raw, angle, partner, turned, sign);
  }
}

template <int kLanes>
cudaError_t launch(const RopeParams& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  const int tokens = kWarps >> p.log2_splits;
  cfg.gridDim = dim3((unsigned)((p.T + tokens - 1) / tokens), (unsigned)p.B);
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

cudaError_t launch_rope(RopeParams& p, int num_sms, cudaStream_t stream) {
  int lanes = 1;
  while (lanes * 8 < p.D) lanes *= 2;
  // Warps to a token: enough to leave each at most kSteps steps of heads, and with few
  // tokens enough to fill the GPU (16 warps per SM).
  const long long rows = (long long)p.B * p.T;
  const int per = 32 / lanes, steps = (p.q.heads + per - 1) / per + (p.k.heads + per - 1) / per;
  p.log2_splits = 0;
  while ((1 << p.log2_splits) < kWarps &&
         (steps > kSteps << p.log2_splits || (steps > 1 << p.log2_splits && rows << p.log2_splits < 16LL * num_sms)))
    ++p.log2_splits;
  p.log2_pairs = 0;
  while (1 << p.log2_pairs < p.R / 2) ++p.log2_pairs;
  switch (lanes) {
    case 1: return launch<1>(p, stream);
    case 2: return launch<2>(p, stream);
    case 4: return launch<4>(p, stream);
    case 8: return launch<8>(p, stream);
    case 16: return launch<16>(p, stream);
    default: return launch<32>(p, stream);
  }
}

}  // namespace svdq
