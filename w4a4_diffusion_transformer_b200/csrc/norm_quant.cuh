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
//
// One B200, 4608 x 3072 with a residual: codes and scales alone W8A8 22.2 us (4.5
// TB/s of what it reads and writes; 18432 rows 70.6 us, 5.6 TB/s; a copy 6.56), NVFP4
// 21.2, INT4 24.5; with XL W8A8 29.1, NVFP4 31.4, INT4 36.8; one row 3.2 us, with XL
// 5.2 to 5.9.  Without XL it is bound by memory latency at the ends of a CTA's few
// tiles, then by memory; with XL by the dependent chains of a tile's phases (40 % of
// the issue slots), two tiles per SM at this size.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kernels.h"
#include "nvfp4_quant.cuh"
#include "sm100.cuh"

namespace svdq {

namespace {

// A CTA of 8 or 16 warps (launch_plain and launch_project below choose) handles
// tiles of 8 / W or 16 / W rows, W warps to a row; a lane of the row's warp w owns
// the C chunks of 8 values 32 (C w + c) + lane and keeps them in registers, as FP32, from the load to the
// codes: unpacking BF16 pairs again for every pass took twice the instructions,
// and those are what bounds the kernel before memory does.  Twelve chunks of the
// NVFP4 quantizer do not fit that way; kept as BF16 and unpacked per pass they
// spill less (4608 x 3072 codes and XL: 24.3 against 26.1 us, with a residual
// 32.2 against 35.0 when it was chosen; INT4 38.2 against 38.0, so it keeps FP32).  Consecutive
// chunks lie a constant apart in every operand and layout, so that their addresses
// are immediates.  The columns' parameters w (1 + scale), shift and 1/lam sit in
// shared memory as FP32, filled once per CTA and modulation row; chunk q's eight
// values are two 16-byte words at q and q + K/8, so that a warp's reads are free
// of bank conflicts.  (Two rows to a warp, which read the parameters once and
// share a group's scale arithmetic, need the registers of both: 31.7 us.  Bringing
// the next tile's rows into L2 meanwhile: 27.6 us.)
// A lane's chunks: at most 6 (12 with a projection, which wants many rows in a tile).
constexpr int kChunks = 6, kChunksMost = 12;
constexpr size_t kSmSmem = 228 * 1024;                  // shared memory of an SM

__device__ __forceinline__ float2 unpack2(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ uint32_t pack2(float2 v) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(v.x, v.y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t add_bf16x2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 h =
      __hadd2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Eight FP32 parameters of chunk q.
__device__ __forceinline__ void param8(const float4* t, int q, int nch, float2 (&v)[4]) {
  const float4 a = t[q], b = t[q + nch];
  v[0] = make_float2(a.x, a.y);
  v[1] = make_float2(a.z, a.w);
  v[2] = make_float2(b.x, b.y);
  v[3] = make_float2(b.z, b.w);
}

// A row's total (or maximum) in every lane of its W warps: shuffles, then the
// warps' partials through `slot` (W floats of this row), added in warp order.
template <bool kMax>
__device__ __forceinline__ float reduce_row(float v, float* slot, int W, int w, int bar) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float u = __shfl_xor_sync(0xffffffffu, v, o);
    v = kMax ? fmaxf(v, u) : v + u;
  }
  if (W > 1) {
    if ((threadIdx.x & 31) == 0) slot[w] = v;
    dev::named_barrier(bar, 32 * W);
    v = slot[0];
    for (int i = 1; i < W; ++i) v = kMax ? fmaxf(v, slot[i]) : v + slot[i];
  }
  return v;
}

__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// kMt: blocks of 16 branch columns to project (0: no projection).  kFull: every
// lane has C chunks (K = 256 C W), so that no access needs a predicate.
template <int kFmt, int C, int kWarps, int kMt, bool kFull>
__global__ void __launch_bounds__(kWarps * 32, 16 / kWarps) norm_quant_kernel(const __grid_constant__ NormParams p) {
  constexpr int kThreads = kWarps * 32;
  constexpr bool kPacked = kFmt == kFmtNvfp4 && C > 6;
  extern __shared__ __align__(16) uint8_t smem[];
  const int K = p.K, M = p.M, nch = K >> 3;             // chunks of 8 values in a row
  const int W = 1 << p.log2_warps, rows = kWarps >> p.log2_warps;
  float* slots = reinterpret_cast<float*>(smem);        // [2][3][kWarps]: tile parity, reduction, warp
  float* rcp = slots + 2 * 3 * kWarps;                  // the NVFP4 quantizer's constants
  float4* gain = reinterpret_cast<float4*>(rcp + 16);   // w (1 + scale)
  float4* shift = gain + 2 * nch;
  float4* ilam = shift + 2 * nch;
  uint8_t* ytile = reinterpret_cast<uint8_t*>(ilam + 2 * nch);
  const int ystride = 2 * K + 64;                       // 64 bytes: rows shifted by half the banks
  float* red = reinterpret_cast<float*>(ytile + rows * ystride);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rg = warp >> p.log2_warps, w = warp & (W - 1);   // this warp's row of the tile, its place in the row
  const int q0 = w * (32 * C) + lane;                   // first chunk; the next are 32 apart
  const int nc = kFull ? C : min(C, max(0, (nch - q0 + 31) >> 5));   // this lane's chunks

  dev::griddep_launch_dependents();
  if (kFmt == kFmtNvfp4 && threadIdx.x < 16) rcp[threadIdx.x] = p.rcp[threadIdx.x];
  for (int i = threadIdx.x; i < 2 * nch; i += kThreads)
    ilam[(i >> 1) + (i & 1) * nch] = reinterpret_cast<const float4*>(p.inv_lam)[i];
  // X may be the preceding kernel's output, and that kernel may still read the
  // buffers this one writes
  dev::griddep_wait();

  const float invK = 1.0f / (float)K;
  // this CTA's tiles: p.tiles_each, and one more for the first p.tiles_extra CTAs
  const int b = (int)blockIdx.x;
  const int t0 = b * p.tiles_each + min(b, p.tiles_extra), t1 = t0 + p.tiles_each + (b < p.tiles_extra ? 1 : 0);
  int loaded = -1;                                      // modulation row in shared memory
  for (int tile = t0; tile < t1; ++tile) {
    const int row = tile * rows + rg;
    const bool live = row < M;                          // rows M .. mpad - 1: zero codes and scales
    const uint32_t keep = live ? 0xFFFFFFFFu : 0u;
    // a dead row computes on the last one's values and stores zeros
    const size_t at = (size_t)min(row, M - 1) * K + 8 * q0;
    float* slot = slots + ((tile & 1) * 3) * kWarps + rg * W;
    // Only one of the two is used: hp, the BF16 h, or f, its FP32 values -- in turn
    // h, h - mu and y / lam.
    uint4 hp[C];
    float2 f[C][4], nmu = make_float2(0.f, 0.f);        // nmu: -mu
    const auto centred = [&](int c, float2 (&t)[4]) {   // chunk c of h - mu; zeros past K
      if (kPacked) {
        const bool in = kFull || c < nc;
        t[0] = in ? __fadd2_rn(unpack2(hp[c].x), nmu) : make_float2(0.f, 0.f);
        t[1] = in ? __fadd2_rn(unpack2(hp[c].y), nmu) : make_float2(0.f, 0.f);
        t[2] = in ? __fadd2_rn(unpack2(hp[c].z), nmu) : make_float2(0.f, 0.f);
        t[3] = in ? __fadd2_rn(unpack2(hp[c].w), nmu) : make_float2(0.f, 0.f);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) t[i] = f[c][i];
      }
    };
    // ---- h = bf16(x + r)
    {
      uint4 v[C];
#pragma unroll
      for (int c = 0; c < C; ++c) {
        v[c] = make_uint4(0u, 0u, 0u, 0u);
        if (c < nc) v[c] = *reinterpret_cast<const uint4*>(p.x + at + 256 * c);
      }
      if (p.residual) {
        const __nv_bfloat16* r = p.residual + at;
#pragma unroll
        for (int c = 0; c < C; ++c)
          if (c < nc) {
            const uint4 u = *reinterpret_cast<const uint4*>(r + 256 * c);
            v[c] = make_uint4(add_bf16x2(v[c].x, u.x), add_bf16x2(v[c].y, u.y), add_bf16x2(v[c].z, u.z),
                              add_bf16x2(v[c].w, u.w));
          }
      }
      if (p.sum && live) {
        __nv_bfloat16* o = p.sum + at;
#pragma unroll
        for (int c = 0; c < C; ++c)
          if (c < nc) *reinterpret_cast<uint4*>(o + 256 * c) = v[c];
      }
#pragma unroll
      for (int c = 0; c < C; ++c) {
        if (kPacked) {
          hp[c] = v[c];
        } else {
          f[c][0] = unpack2(v[c].x);
          f[c][1] = unpack2(v[c].y);
          f[c][2] = unpack2(v[c].z);
          f[c][3] = unpack2(v[c].w);
        }
      }
    }
    // ---- the tile's modulation rows: one, but where two sequences meet
    int m0 = 0, m1 = 0, mine = 0;
    if (p.rows_per_mod > 0) {
      m0 = min(tile * rows, M - 1) / p.rows_per_mod;
      m1 = min(tile * rows + rows - 1, M - 1) / p.rows_per_mod;
      mine = m0 == m1 ? m0 : min(row, M - 1) / p.rows_per_mod;
    }
    // ---- statistics: the mean first (layer norm), then the mean square about it
    if (p.center) {
      float2 a = make_float2(0.f, 0.f);
#pragma unroll
      for (int c = 0; c < C; ++c) {
        float2 t[4];
        centred(c, t);
#pragma unroll
        for (int i = 0; i < 4; ++i) a = __fadd2_rn(a, t[i]);
      }
      // a division, not a product with 1/K: the mean of K equal values is the
      // value itself then, and their variance 0 (with 1/K, 14336 values of 1000
      // normalised to 0.17)
      const float mu = __fdiv_rn(reduce_row<false>(a.x + a.y, slot, W, w, 1 + rg), (float)K);
      nmu = make_float2(-mu, -mu);
      if (!kPacked)
#pragma unroll
        for (int c = 0; c < C; ++c)
          if (c < nc) {                                 // a chunk past K keeps its zeros
#pragma unroll
            for (int i = 0; i < 4; ++i) f[c][i] = __fadd2_rn(f[c][i], nmu);
          }
    }
    float2 a2 = make_float2(0.f, 0.f);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float2 t[4];
      centred(c, t);
#pragma unroll
      for (int i = 0; i < 4; ++i) a2 = __ffma2_rn(t[i], t[i], a2);
    }
    const float rstd = rsqrtf(reduce_row<false>(a2.x + a2.y, slot + kWarps, W, w, 1 + rg) * invK + p.eps);
    const float2 rstd2 = make_float2(rstd, rstd);

    float amax = 0.f;
    for (int m = m0; m <= m1; ++m) {
      if (m != loaded) {                                // uniform over the CTA
        __syncthreads();
        for (int q = threadIdx.x; q < nch; q += kThreads) {
          uint4 u = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);   // ones
          if (p.weight) u = *reinterpret_cast<const uint4*>(p.weight + 8 * q);
          float2 g[4] = {unpack2(u.x), unpack2(u.y), unpack2(u.z), unpack2(u.w)}, s[4] = {};
          if (p.scale) {
            u = *reinterpret_cast<const uint4*>(p.scale + m * p.mod_stride + 8 * q);
            const float2 e[4] = {unpack2(u.x), unpack2(u.y), unpack2(u.z), unpack2(u.w)};
#pragma unroll
            for (int i = 0; i < 4; ++i) g[i] = __fmul2_rn(g[i], __fadd2_rn(make_float2(1.f, 1.f), e[i]));
          }
          if (p.shift) {
            u = *reinterpret_cast<const uint4*>(p.shift + m * p.mod_stride + 8 * q);
            s[0] = unpack2(u.x); s[1] = unpack2(u.y); s[2] = unpack2(u.z); s[3] = unpack2(u.w);
          }
          gain[q] = make_float4(g[0].x, g[0].y, g[1].x, g[1].y);
          gain[q + nch] = make_float4(g[2].x, g[2].y, g[3].x, g[3].y);
          shift[q] = make_float4(s[0].x, s[0].y, s[1].x, s[1].y);
          shift[q + nch] = make_float4(s[2].x, s[2].y, s[3].x, s[3].y);
        }
        loaded = m;
        __syncthreads();
      }
      if (m != mine) continue;
      // ---- y = bf16(n w (1 + scale) + shift), and the 4-bit quantizers
      uint8_t* codes_at = nullptr;
      uint8_t* scales_at = nullptr;
      if (kFmt == kFmtNvfp4) {
        codes_at = p.codes + act_tile_offset(row, q0 >> 5, lane >> 2, p.nst) + (lane & 3) * 4;
        scales_at = p.scales + sf_offset(row, q0 >> 1, K);
      }
      __nv_bfloat16* yout = p.y && live ? p.y + at : nullptr;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int q = q0 + 32 * c;
        const bool act = c < nc;
        float2 own[4];
        if (kPacked) centred(c, own);
        float2 (&t)[4] = kPacked ? own : f[c];
        if (act) {
          float2 g[4], sh[4], il[4];
          param8(gain, q, nch, g);
          param8(shift, q, nch, sh);
          param8(ilam, q, nch, il);
          uint32_t y[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            y[i] = pack2(__ffma2_rn(__fmul2_rn(t[i], rstd2), g[i], sh[i]));
            t[i] = __fmul2_rn(unpack2(y[i]), il[i]);
          }
          if (kMt > 0) *reinterpret_cast<uint4*>(ytile + rg * ystride + q * 16) = make_uint4(y[0], y[1], y[2], y[3]);
          if (yout) *reinterpret_cast<uint4*>(yout + 256 * c) = make_uint4(y[0], y[1], y[2], y[3]);
        }
        float a = fmaxf(fabsf(t[0].x), fabsf(t[0].y));
#pragma unroll
        for (int i = 1; i < 4; ++i) a = dev::fmax3(a, fabsf(t[i].x), fabsf(t[i].y));
        if (kFmt == kFmtInt8) {
          amax = fmaxf(amax, a);
        } else if (kFmt == kFmtNvfp4) {
          // a group of 16 is two lanes' chunks
          a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
          uint32_t codes = 0u;
          const uint32_t sb = dev::nvfp4_quant8(t, a, p.c_x, p.g_x_exp, rcp, codes) & keep;
          // four groups' scale bytes are one word of the layout
          uint32_t word = sb << (8 * ((lane >> 1) & 3));
          word |= __shfl_xor_sync(0xffffffffu, word, 2);
          word |= __shfl_xor_sync(0xffffffffu, word, 4);
          if (act) {
            if ((lane & 7) == 0) *reinterpret_cast<uint32_t*>(scales_at + 2048 * c) = word;
            *reinterpret_cast<uint32_t*>(codes_at + 16384 * c) = codes & keep;
          }
        } else {
          // a group of 64 is eight lanes' chunks
          a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
          a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 2));
          a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 4));
          const __nv_bfloat16 sb = __float2bfloat16_rn(live ? __fmul_rn(a, 1.0f / 7.0f) : 0.f);
          const float sc = __bfloat162float(sb);
          uint32_t codes = 0u;
          const float inv = sc == 0.f ? 0.f : __frcp_rn(sc);
          const float2 i2 = make_float2(inv, inv);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            // the sum with 1.5 * 2^23 holds the rounded integer in its low
            // bits; the product is rounded before (no fused multiply-add)
            const float2 k = __fmul2_rn(t[i], i2);
            codes |= (__float_as_uint(__fadd_rn(k.x, 12582912.0f)) & 0xFu) << (8 * i);
            codes |= (__float_as_uint(__fadd_rn(k.y, 12582912.0f)) & 0xFu) << (8 * i + 4);
          }
          if (act) {
            if ((lane & 7) == 0)
              reinterpret_cast<uint16_t*>(p.scales)[(size_t)(q >> 3) * p.mpad + row] = __bfloat16_as_ushort(sb);
            if (live) *reinterpret_cast<uint32_t*>(p.codes + (size_t)row * (K / 2) + q0 * 4 + 128 * c) = codes;
          }
        }
      }
    }
    if (kFmt == kFmtInt8) {
      // one scale per token, from the whole row
      amax = reduce_row<true>(amax, slot + 2 * kWarps, W, w, 1 + rg);
      const float sc = live ? __fmul_rn(amax, 1.0f / 127.0f) : 0.f;
      const float inv = sc == 0.f ? 0.f : __frcp_rn(sc);
      if (w == 0 && lane == 0) {
        float* sx = reinterpret_cast<float*>(p.scales);
        sx[row] = sc;
        sx[p.mpad + row] = inv;
      }
      float2 i2 = make_float2(inv, inv);
      if (inv > 3.40282347e38f) {
        // a scale below 2^-128 has no finite reciprocal: everything but zero clamps
        // to +-127, as in the first kernel
        i2 = make_float2(1.f, 1.f);
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            f[c][i] = make_float2(f[c][i].x == 0.f ? 0.f : copysignf(127.f, f[c][i].x),
                                  f[c][i].y == 0.f ? 0.f : copysignf(127.f, f[c][i].y));
      }
      // stages of 128 codes: chunk q is half of a 16-byte piece of stage q / 16
      uint8_t* o = p.codes + act_tile_offset(row, q0 >> 4, (q0 & 15) >> 1, p.nst) + (lane & 1) * 8;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        if (c < nc) {
          uint32_t t[8];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            // the sum with 1.5 * 2^23 holds the rounded integer, two's
            // complement, in its low byte (|q| <= 127 (1 + 2^-20): no clamp)
            const float2 k = __fmul2_rn(f[c][i], i2);
            t[2 * i] = __float_as_uint(__fadd_rn(k.x, 12582912.0f));
            t[2 * i + 1] = __float_as_uint(__fadd_rn(k.y, 12582912.0f));
          }
          uint2 v;
          v.x = __byte_perm(__byte_perm(t[0], t[1], 0x0040), __byte_perm(t[2], t[3], 0x0040), 0x5410);
          v.y = __byte_perm(__byte_perm(t[4], t[5], 0x0040), __byte_perm(t[6], t[7], 0x0040), 0x5410);
          if (sc == 0.f) v.x = v.y = 0u;
          *reinterpret_cast<uint2*>(o + 2 * 16384 * c) = v;
        }
      }
    }
    if (kMt == 0 || tile * rows >= M) continue;         // uniform over the CTA

    // ---- XL: 16 rank rows x 8 tokens per MMA, K split over the warps.  The
    // order of k inside a block of 32 is free as long as both operands agree:
    // lane (g, c) = (lane / 4, lane % 4) takes columns 8c .. 8c + 7 of the
    // block, so each operand row is one 16-byte load and feeds two MMAs.  The
    // factor comes from L2 for every tile (rank 32: 64 K bytes), which is why a
    // tile is 16 rows and no fewer.
    __syncthreads();                                    // the y tile is complete
    constexpr int kAcc = kMt > 0 ? kMt : 1, kTok = kWarps;   // a tile has at most a row per warp
    const int g = lane >> 2, c = lane & 3;
    float acc[kAcc][2][4];
#pragma unroll
    for (int mt = 0; mt < kAcc; ++mt)
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[mt][i >> 2][i & 3] = 0.f;
    const uint8_t* yrow = ytile + g * ystride + c * 16;
    const bool first = g < rows, second = kTok > 8 && g + 8 < rows;
#pragma unroll(kMt == 4 ? 2 : 3)
    for (int kb = warp; kb < K / 32; kb += kWarps) {
      uint4 lo[kAcc], hi[kAcc], b0 = make_uint4(0u, 0u, 0u, 0u), b1 = b0;
#pragma unroll
      for (int mt = 0; mt < kMt; ++mt) {
        const uint4* a = reinterpret_cast<const uint4*>(p.amat[mt]) + kb * 128 + lane;
        lo[mt] = a[0];
        hi[mt] = a[32];
      }
      if (first) b0 = *reinterpret_cast<const uint4*>(yrow + kb * 64);
      if (second) b1 = *reinterpret_cast<const uint4*>(yrow + 8 * ystride + kb * 64);
#pragma unroll
      for (int mt = 0; mt < kMt; ++mt) {
        mma_16816(acc[mt][0], lo[mt].x, hi[mt].x, lo[mt].y, hi[mt].y, b0.x, b0.y);
        mma_16816(acc[mt][0], lo[mt].z, hi[mt].z, lo[mt].w, hi[mt].w, b0.z, b0.w);
        if (kTok > 8) {
          mma_16816(acc[mt][1], lo[mt].x, hi[mt].x, lo[mt].y, hi[mt].y, b1.x, b1.y);
          mma_16816(acc[mt][1], lo[mt].z, hi[mt].z, lo[mt].w, hi[mt].w, b1.z, b1.w);
        }
      }
    }
    constexpr int kRank = kMt * 16;
#pragma unroll
    for (int mt = 0; mt < kMt; ++mt)                    // partials [warp][rank][token]
#pragma unroll
      for (int h = 0; h < kTok / 8; ++h) {
        float* o = red + ((size_t)warp * kRank + mt * 16 + g) * kTok + 8 * h + 2 * c;
        *reinterpret_cast<float2*>(o) = make_float2(acc[mt][h][0], acc[mt][h][1]);
        *reinterpret_cast<float2*>(o + 8 * kTok) = make_float2(acc[mt][h][2], acc[mt][h][3]);
      }
    __syncthreads();                                    // ... and the y tile has been read
    for (int i = threadIdx.x; i < kRank * rows; i += kThreads) {
      const int t = i & (rows - 1), j = i / rows, r = tile * rows + t;   // token, rank row
      if (r < M) {
        float v = 0.f;
#pragma unroll
        for (int u = 0; u < kWarps; ++u) v += red[((size_t)u * kRank + j) * kTok + t];
        p.xl[(size_t)r * p.xl_stride + p.xl_col[j >> 4] + (j & 15)] = __float2bfloat16_rn(v);
      }
    }
    if (p.xl_zero > 0 && threadIdx.x < 16 * rows) {
      const int r = tile * rows + (threadIdx.x >> 4);
      if (r < M) p.xl[(size_t)r * p.xl_stride + p.xl_zero + (threadIdx.x & 15)] = __float2bfloat16_rn(0.f);
    }
  }
}

size_t smem_bytes(int K, int nmt, int warps, int log2_warps) {
  const size_t head = (2 * 3 * warps + 16) * 4, params = (size_t)K * 12;
  const size_t tile = (size_t)(warps >> log2_warps) * (2 * (size_t)K + 64), red = (size_t)warps * nmt * 16 * warps * 4;
  return head + params + (nmt > 0 ? tile + red : 0);
}

template <int kFmt, int C, int kWarps, int kMt, bool kFull>
cudaError_t launch_t(NormParams& p, int num_sms, cudaStream_t stream) {
  const size_t smem = smem_bytes(p.K, kMt, kWarps, p.log2_warps);
  if (smem > kNormMaxSmem) return cudaErrorInvalidValue;
  auto kern = norm_quant_kernel<kFmt, C, kWarps, kMt, kFull>;
  static thread_local int configured_device = -1;
  int dev = 0;
  cudaGetDevice(&dev);
  if (configured_device != dev) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kNormMaxSmem);
    if (e != cudaSuccess) return e;
    configured_device = dev;
  }
  // persistent: as many CTAs as an SM holds (1 KB of shared memory per CTA its
  // own), each a contiguous range of tiles
  const int rows = kWarps >> p.log2_warps, tiles = p.mpad / rows;
  const int fit = (int)(kSmSmem / (smem + 1024)), per_sm = fit < 16 / kWarps ? fit : 16 / kWarps;
  const int grid = tiles < per_sm * num_sms ? tiles : per_sm * num_sms;
  p.tiles_each = tiles / grid;
  p.tiles_extra = tiles % grid;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kWarps * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

template <int kFmt, int C, int kWarps, int kMt>
cudaError_t launch(NormParams& p, int num_sms, cudaStream_t stream) {
  // Without predicates where every lane is full: 4608 rows of 3072 W8A8 22.0 instead
  // of 22.7 us, NVFP4 21.1 / 22.5, INT4 24.4 / 25.8; with XL NVFP4 31.2 / 34.5, INT4
  // 36.7 / 37.3; of 4096 NVFP4 29.5 / 31.4; 2048 of 12288 NVFP4 with XL 109.7 / 125.
  // Twelve chunks kept as FP32 spill more that way beside W8A8's projection (224
  // against 28 bytes; 31.6 against 29.0 us, 6144 columns 66.8 / 63.8) and beside 64
  // XL columns (INT4 45.6 / 44.8).  Rows of up to three chunks gain 0.1 to 0.3 us, not
  // worth their code; four chunks of 16 warps without a projection are never full.
  constexpr bool kSpills = C == 12 && kWarps == 16 && (kFmt == kFmtInt8 || (kFmt == kFmtInt4 && kMt == 4));
  constexpr bool kFull = C >= 4 && !kSpills && !(kMt == 0 && kWarps == 16 && C == 4);
  return kFull && p.K == (256 * C) << p.log2_warps ? launch_t<kFmt, C, kWarps, kMt, kFull>(p, num_sms, stream)
                                                   : launch_t<kFmt, C, kWarps, kMt, false>(p, num_sms, stream);
}

// Chunks of a lane with 2^l warps to a row.
int lane_chunks(int K, int l) { return (K / 8 + (32 << l) - 1) / (32 << l); }

// Without a projection: 8 warps, two CTAs per SM.  More registers a thread and
// all of a row's loads in flight beat more warps (4608 x 3072 W8A8: 23.1 us at 16
// warps of 128 registers, 25.0 at 24 of 80).  Rows of more than 8192 columns, which
// 8 warps could take only one at a time (and whose parameters soon leave no room
// for a second CTA), get one CTA of 16 warps: 4608 x 9216 W8A8 78.3 instead of 88.4
// us, x 12288 86.6 instead of 122; x 8192 67.8 instead of 66.6.
template <int kFmt>
cudaError_t launch_plain(NormParams& p, int num_sms, cudaStream_t stream) {
  int l = 0;
  if (lane_chunks(p.K, 3) > 4) {
    while (l < 4 && lane_chunks(p.K, l) > kChunks) ++l;
    while (l < 4 && (p.M + (16 >> l) - 1) / (16 >> l) < num_sms) ++l;
    p.log2_warps = l;
    return lane_chunks(p.K, l) <= 4 ? launch<kFmt, 4, 16, 0>(p, num_sms, stream)
                                    : launch<kFmt, 6, 16, 0>(p, num_sms, stream);
  }
  while (l < 3 && lane_chunks(p.K, l) > kChunks) ++l;
  // with few rows, more warps to a row
  while (l < 3 && (p.M + (8 >> l) - 1) / (8 >> l) < num_sms) ++l;
  p.log2_warps = l;
  const int chunks = lane_chunks(p.K, l);
  if (chunks <= 1) return launch<kFmt, 1, 8, 0>(p, num_sms, stream);
  if (chunks <= 2) return launch<kFmt, 2, 8, 0>(p, num_sms, stream);
  if (chunks <= 3) return launch<kFmt, 3, 8, 0>(p, num_sms, stream);
  if (chunks <= 4) return launch<kFmt, 4, 8, 0>(p, num_sms, stream);
  return launch<kFmt, 6, 8, 0>(p, num_sms, stream);
}

// With a projection: 16 warps, one CTA per SM, tiles of up to 16 rows; 8 warps
// where 16 rows of so many columns do not fit in shared memory.
template <int kFmt, int kMt>
cudaError_t launch_project(NormParams& p, int num_sms, cudaStream_t stream) {
  int l = 0;
  while (l < 3 && lane_chunks(p.K, l) > kChunksMost) ++l;
  if (smem_bytes(p.K, kMt, 16, l) > kNormMaxSmem) {
    p.log2_warps = l;
    return launch<kFmt, 12, 8, kMt>(p, num_sms, stream);
  }
  while (l < 3 && (p.M + (16 >> l) - 1) / (16 >> l) < num_sms) ++l;
  p.log2_warps = l;
  const int chunks = lane_chunks(p.K, l);
  if (chunks <= 2) return launch<kFmt, 2, 16, kMt>(p, num_sms, stream);
  if (chunks <= 4) return launch<kFmt, 4, 16, kMt>(p, num_sms, stream);
  if (chunks <= 6) return launch<kFmt, 6, 16, kMt>(p, num_sms, stream);
  return launch<kFmt, 12, 16, kMt>(p, num_sms, stream);
}

}  // namespace
}  // namespace svdq
