// Normalisation fused with the first kernel's work: residual addition, RMS or
// layer norm, modulation, and everything svdq_quantize_act writes for the
// normalised rows (codes, scales, XL), in one pass over X.
//
//   h  = bf16(x + r)                                 (stored; h = x without r)
//   n  = (h - mu) / sqrt(mean((h - mu)^2) + eps)     (mu = mean(h), or 0: RMS)
//   y  = bf16(n w (1 + scale) + shift)               (one rounding from FP32)
//   codes, scales = the layer's quantizer on y       (k1_quant.cu's arithmetic)
//   XL = bf16(y L1d)                                 (and bf16(y A), an adapter)
//
// h is rounded before the statistics because the stored stream is what every
// later layer reads, and y because it is the layer's BF16 input: the codes are
// then bit for bit those of the unfused sequence on the same y.  Sums, means
// and products are FP32.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kernels.h"
#include "nvfp4_quant.cuh"
#include "sm100.cuh"

namespace svdq {

namespace {

// A thread owns 16 columns of every row of its CTA's tile of R rows: the
// parameters of its columns are read once per tile, a thread's 16 columns are
// one NVFP4 group, a quarter of an INT4 group and one 16-byte chunk of INT8
// codes, and a row's sums need two barriers whatever R.
constexpr int kCols = 16;

__device__ __forceinline__ float2 unpack2(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ uint32_t pack2(float2 v) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(v.x, v.y);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// 32 bytes (16 BF16 values) of global memory.
__device__ __forceinline__ void load16(const __nv_bfloat16* p, uint32_t (&w)[8]) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  const uint4 b = *(reinterpret_cast<const uint4*>(p) + 1);
  w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
  w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
}

// The tile's R row totals of v, in every thread: warps reduce by shuffles, the
// warps' partials meet in shared memory and are added in warp order.
template <int R, bool kMax>
__device__ __forceinline__ void reduce_rows(float (&v)[R], float* part, int nwarps) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float u = __shfl_xor_sync(0xffffffffu, v[r], o);
      v[r] = kMax ? fmaxf(v[r], u) : v[r] + u;
    }
  if (lane == 0)
#pragma unroll
    for (int r = 0; r < R; ++r) part[warp * R + r] = v[r];
  __syncthreads();
#pragma unroll
  for (int r = 0; r < R; ++r) v[r] = part[r];
  for (int w = 1; w < nwarps; ++w)
#pragma unroll
    for (int r = 0; r < R; ++r) v[r] = kMax ? fmaxf(v[r], part[w * R + r]) : v[r] + part[w * R + r];
}

__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Shared memory in front of the y tile: three reduction buffers and the constants.
__host__ __device__ constexpr int head_bytes(int R, int nwarps) { return (3 * R * nwarps * 4 + 64 + 15) / 16 * 16; }

template <int R, int kFmt>
__global__ void __launch_bounds__(R > 2 ? 512 : 1024) norm_quant_kernel(const NormParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  const int K = p.K, M = p.M;
  const int nwarps = blockDim.x >> 5;
  const int ystride = 2 * K + 64;                       // bytes between rows of the y tile (bank shift by rows)
  float* part0 = reinterpret_cast<float*>(smem);        // three reductions, a buffer each
  float* part1 = part0 + R * nwarps;
  float* part2 = part1 + R * nwarps;
  float* rcp = part2 + R * nwarps;                      // the NVFP4 quantizer's constants
  uint8_t* ytile = smem + head_bytes(R, nwarps);
  const int tid = threadIdx.x;
  const int c0 = tid * kCols;
  const bool act = c0 < K;
  const int row0 = blockIdx.x * R;

  dev::griddep_launch_dependents();
  if (kFmt == kFmtNvfp4 && tid < 16) rcp[tid] = p.rcp[tid];
  // X may be the preceding kernel's output, and that kernel may still read the
  // buffers this one writes
  dev::griddep_wait();

  uint32_t h[R][8];
  float s[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
#pragma unroll
    for (int i = 0; i < 8; ++i) h[r][i] = 0u;
    if (act && row0 + r < M) load16(p.x + (size_t)(row0 + r) * K + c0, h[r]);
  }
  if (p.residual) {
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (act && row0 + r < M) {
        uint32_t q[8];
        load16(p.residual + (size_t)(row0 + r) * K + c0, q);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 a = unpack2(h[r][i]), b = unpack2(q[i]);
          h[r][i] = pack2(make_float2(a.x + b.x, a.y + b.y));
        }
      }
  }
  if (p.sum) {
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (act && row0 + r < M) {
        uint4* o = reinterpret_cast<uint4*>(p.sum + (size_t)(row0 + r) * K + c0);
        o[0] = make_uint4(h[r][0], h[r][1], h[r][2], h[r][3]);
        o[1] = make_uint4(h[r][4], h[r][5], h[r][6], h[r][7]);
      }
  }

  // ---- statistics: the mean first (layer norm), then the mean square about it
  const float invK = 1.0f / (float)K;
  float mu[R];
#pragma unroll
  for (int r = 0; r < R; ++r) mu[r] = 0.f;
  if (p.center) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float2 a = make_float2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < 8; ++i) a = __fadd2_rn(a, unpack2(h[r][i]));
      mu[r] = a.x + a.y;
    }
    reduce_rows<R, false>(mu, part0, nwarps);
#pragma unroll
    for (int r = 0; r < R; ++r) mu[r] *= invK;
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    float2 a = make_float2(0.f, 0.f);
    const float2 m2 = make_float2(-mu[r], -mu[r]);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 d = __fadd2_rn(unpack2(h[r][i]), m2);
      a = __ffma2_rn(d, d, a);
    }
    s[r] = act ? a.x + a.y : 0.f;                       // a thread past K holds zeros, not values
  }
  reduce_rows<R, false>(s, part1, nwarps);
#pragma unroll
  for (int r = 0; r < R; ++r) s[r] = rsqrtf(s[r] * invK + p.eps);   // 1 / sqrt

  // ---- y = bf16(n w (1 + scale) + shift), in h's place
  float amax[R];
#pragma unroll
  for (int r = 0; r < R; ++r) amax[r] = 0.f;
  if (act) {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int col = c0 + 8 * half;
      float2 g[4], sh[4], il[4];
      int cur = -1;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float4 v = *reinterpret_cast<const float4*>(p.inv_lam + col + 4 * j);
        il[2 * j] = make_float2(v.x, v.y);
        il[2 * j + 1] = make_float2(v.z, v.w);
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int row = min(row0 + r, M - 1);
        const int mr = p.rows_per_mod > 0 ? row / p.rows_per_mod : 0;
        if (mr != cur) {                                // uniform over the CTA
          cur = mr;
          uint4 w = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);   // ones
          if (p.weight) w = *reinterpret_cast<const uint4*>(p.weight + col);
          const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            g[i] = unpack2(ws[i]);
            sh[i] = make_float2(0.f, 0.f);
          }
          if (p.scale) {
            const uint4 q = *reinterpret_cast<const uint4*>(p.scale + (size_t)mr * p.mod_stride + col);
            const uint32_t qs[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) g[i] = __fmul2_rn(g[i], __fadd2_rn(make_float2(1.f, 1.f), unpack2(qs[i])));
          }
          if (p.shift) {
            const uint4 q = *reinterpret_cast<const uint4*>(p.shift + (size_t)mr * p.mod_stride + col);
            const uint32_t qs[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) sh[i] = unpack2(qs[i]);
          }
        }
        const float2 m2 = make_float2(-mu[r], -mu[r]), s2 = make_float2(s[r], s[r]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 n = __fmul2_rn(__fadd2_rn(unpack2(h[r][4 * half + i]), m2), s2);
          const uint32_t y = pack2(__ffma2_rn(n, g[i], sh[i]));
          h[r][4 * half + i] = y;
          if (kFmt == kFmtInt8) {
            const float2 v = __fmul2_rn(unpack2(y), il[i]);
            amax[r] = dev::fmax3(amax[r], fabsf(v.x), fabsf(v.y));
          }
        }
        if (p.nmt > 0)
          *reinterpret_cast<uint4*>(ytile + r * ystride + col * 2) =
              make_uint4(h[r][4 * half], h[r][4 * half + 1], h[r][4 * half + 2], h[r][4 * half + 3]);
        if (p.y && row0 + r < M)
          *reinterpret_cast<uint4*>(p.y + (size_t)(row0 + r) * K + col) =
              make_uint4(h[r][4 * half], h[r][4 * half + 1], h[r][4 * half + 2], h[r][4 * half + 3]);
      }
    }
  }

  // ---- the layer's quantizer (the arithmetic of k1_quant.cu)
  if (kFmt == kFmtInt8) reduce_rows<R, true>(amax, part2, nwarps);
  float2 il[8];
  if (act) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float4 v = *reinterpret_cast<const float4*>(p.inv_lam + c0 + 4 * j);
      il[2 * j] = make_float2(v.x, v.y);
      il[2 * j + 1] = make_float2(v.z, v.w);
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int row = row0 + r;
    const bool live = row < M;                          // rows M .. mpad - 1: zero codes and scales
    float2 v[8];
    if (act) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = __fmul2_rn(unpack2(h[r][i]), il[i]);
    }
    if (kFmt == kFmtInt8) {
      const float sc = live ? __fmul_rn(amax[r], 1.0f / 127.0f) : 0.f;
      const float inv = sc == 0.f ? 0.f : __frcp_rn(sc);
      if (tid == 0) {
        float* sx = reinterpret_cast<float*>(p.scales);
        sx[row] = sc;
        sx[p.mpad + row] = inv;
      }
      if (act) {
        const float2 i2 = make_float2(inv, inv);
        uint32_t w8[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 q0 = __fmul2_rn(v[2 * j], i2), q1 = __fmul2_rn(v[2 * j + 1], i2);
          const int c[4] = {max(-127, min(127, __float2int_rn(q0.x))), max(-127, min(127, __float2int_rn(q0.y))),
                            max(-127, min(127, __float2int_rn(q1.x))), max(-127, min(127, __float2int_rn(q1.y)))};
          w8[j] = (uint32_t)(c[0] & 0xFF) | ((uint32_t)(c[1] & 0xFF) << 8) | ((uint32_t)(c[2] & 0xFF) << 16) |
                  ((uint32_t)(c[3] & 0xFF) << 24);
        }
        *reinterpret_cast<uint4*>(p.codes + act_tile_offset(row, c0 >> 7, (c0 & 127) >> 4, p.nst)) =
            make_uint4(w8[0], w8[1], w8[2], w8[3]);
      }
    } else if (kFmt == kFmtNvfp4) {
      uint32_t packed[2] = {0u, 0u}, sb = 0u;
      if (act && live) sb = dev::nvfp4_quant16(v, p.c_x, p.g_x_exp, rcp, packed);
      // four neighbouring groups' scale bytes are one 32-bit word of the layout
      uint32_t word = sb << (8 * (tid & 3));
      word |= __shfl_xor_sync(0xffffffffu, word, 1);
      word |= __shfl_xor_sync(0xffffffffu, word, 2);
      if (act) {
        if ((tid & 3) == 0) *reinterpret_cast<uint32_t*>(p.scales + sf_offset(row, tid, K)) = word;
        *reinterpret_cast<uint2*>(p.codes + act_tile_offset(row, c0 >> 8, (c0 & 255) >> 5, p.nst) + (tid & 1) * 8) =
            make_uint2(packed[0], packed[1]);
      }
    } else {
      // INT4: a group of 64 is four neighbouring threads
      float a = 0.f;
      if (act) {
#pragma unroll
        for (int i = 0; i < 8; ++i) a = dev::fmax3(a, fabsf(v[i].x), fabsf(v[i].y));
      }
      a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
      a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 2));
      const __nv_bfloat16 sb = __float2bfloat16_rn(live ? __fmul_rn(a, 1.0f / 7.0f) : 0.f);
      const float sc = __bfloat162float(sb);
      if (act) {
        uint32_t packed[2] = {0u, 0u};
        if (sc != 0.f) {
          const float inv = __frcp_rn(sc);
          const float2 i2 = make_float2(inv, inv);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            uint32_t t = 0u;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              // the sum with 1.5 * 2^23 holds the rounded integer in its low
              // bits; the product is rounded before (no fused multiply-add)
              const float2 q = __fmul2_rn(v[4 * j + e], i2);
              t |= (__float_as_uint(__fadd_rn(q.x, 12582912.0f)) & 0xFu) << (8 * e);
              t |= (__float_as_uint(__fadd_rn(q.y, 12582912.0f)) & 0xFu) << (8 * e + 4);
            }
            packed[j] = t;
          }
        }
        if ((tid & 3) == 0)
          reinterpret_cast<uint16_t*>(p.scales)[(size_t)(tid >> 2) * p.mpad + row] = __bfloat16_as_ushort(sb);
        if (live)
          *reinterpret_cast<uint2*>(p.codes + (size_t)row * (K / 2) + tid * 8) = make_uint2(packed[0], packed[1]);
      }
    }
  }
  if (p.nmt == 0) return;

  // ---- XL: 16 rank rows x 8 tokens per MMA, K split over the warps.  The order
  // of k inside a block of 32 is free as long as both operands agree: lane
  // (g, c) = (lane / 4, lane % 4) takes columns 8c .. 8c + 7 of the block, so
  // each operand row is one 16-byte load and feeds two MMAs.
  __syncthreads();                                      // the y tile is complete
  const int warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  float acc[4][4];
#pragma unroll
  for (int mt = 0; mt < 4; ++mt)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[mt][i] = 0.f;
  const uint8_t* yrow = ytile + g * ystride + c * 16;
#pragma unroll 2
  for (int kb = warp; kb < K / 32; kb += nwarps) {
    uint4 b = make_uint4(0u, 0u, 0u, 0u);
    if (g < R) b = *reinterpret_cast<const uint4*>(yrow + kb * 64);
#pragma unroll
    for (int mt = 0; mt < 4; ++mt)
      if (mt < p.nmt) {
        const __nv_bfloat16* a = p.amat[mt] + (size_t)g * K + kb * 32 + c * 8;
        const uint4 lo = *reinterpret_cast<const uint4*>(a);
        const uint4 hi = *reinterpret_cast<const uint4*>(a + 8 * (size_t)K);
        mma_16816(acc[mt], lo.x, hi.x, lo.y, hi.y, b.x, b.y);
        mma_16816(acc[mt], lo.z, hi.z, lo.w, hi.w, b.z, b.w);
      }
  }
  __syncthreads();                                      // the y tile has been read: the partials take its place
  float* red = reinterpret_cast<float*>(ytile);         // [warp][nmt * 16][8]
#pragma unroll
  for (int mt = 0; mt < 4; ++mt)
    if (mt < p.nmt) {
      float* o = red + ((size_t)(warp * p.nmt + mt) * 16 + g) * 8 + 2 * c;
      *reinterpret_cast<float2*>(o) = make_float2(acc[mt][0], acc[mt][1]);
      *reinterpret_cast<float2*>(o + 64) = make_float2(acc[mt][2], acc[mt][3]);
    }
  __syncthreads();
  for (int i = tid; i < p.nmt * 16 * R; i += blockDim.x) {
    const int j = i % (p.nmt * 16), r = i / (p.nmt * 16);   // rank row, token
    if (row0 + r < M) {
      float t = 0.f;
      for (int w = 0; w < nwarps; ++w) t += red[((size_t)w * p.nmt * 16 + j) * 8 + r];
      p.xl[(size_t)(row0 + r) * p.xl_stride + p.xl_col[j >> 4] + (j & 15)] = __float2bfloat16_rn(t);
    }
  }
  if (p.xl_zero > 0)
    for (int i = tid; i < 16 * R; i += blockDim.x)
      if (row0 + (i >> 4) < M) p.xl[(size_t)(row0 + (i >> 4)) * p.xl_stride + p.xl_zero + (i & 15)] = __float2bfloat16_rn(0.f);
}

size_t smem_bytes(int R, const NormParams& p, int threads) {
  const size_t nwarps = threads / 32, head = head_bytes(R, (int)nwarps);
  const size_t tile = (size_t)R * (2 * (size_t)p.K + 64), red = nwarps * p.nmt * 16 * 8 * 4;
  return head + (p.nmt > 0 ? (tile > red ? tile : red) : 0);
}

template <int R, int kFmt>
cudaError_t launch(const NormParams& p, int threads, cudaStream_t stream) {
  const size_t smem = smem_bytes(R, p, threads);
  auto kern = norm_quant_kernel<R, kFmt>;
  static thread_local int configured_device = -1;
  int dev = 0;
  cudaGetDevice(&dev);
  if (configured_device != dev) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kNormMaxSmem);
    if (e != cudaSuccess) return e;
    configured_device = dev;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.mpad / R));
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

template <int R>
cudaError_t launch_fmt(const NormParams& p, int fmt, int threads, cudaStream_t stream) {
  if (fmt == kFmtNvfp4) return launch<R, kFmtNvfp4>(p, threads, stream);
  if (fmt == kFmtInt4) return launch<R, kFmtInt4>(p, threads, stream);
  return launch<R, kFmtInt8>(p, threads, stream);
}

}  // namespace

bool norm_supported(int K) { return K <= kNormMaxK; }

cudaError_t launch_norm_quant(const NormParams& p, int fmt, int num_sms, cudaStream_t stream) {
  const int threads = (p.K / kCols + 31) / 32 * 32;
  const bool wide = threads <= 512 && smem_bytes(4, p, threads) <= kNormMaxSmem;
  if (wide && p.M >= 4 * num_sms) return launch_fmt<4>(p, fmt, threads, stream);
  return launch_fmt<2>(p, fmt, threads, stream);
}

}  // namespace svdq
