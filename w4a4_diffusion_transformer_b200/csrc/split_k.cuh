// K split over the CTAs of a cluster, for GEMMs with too few tiles to fill the
// GPU: the S CTAs of a cluster compute one output tile, each over its share of K.
// When their products are summed, each writes its accumulator to its own shared
// memory (the operand ring, idle by then), the cluster synchronises, and each
// finishes its share of the tile's eight 32-column chunks, [8 r / S, 8 (r + 1) / S)
// for rank r: it adds the S partial sums in rank order over distributed shared
// memory, so the result does not depend on timing and no workspace is needed.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "residual.cuh"
#include "sm100.cuh"

namespace svdq {
namespace dev {

// Shared memory of the dump: [256 columns][128 rows] FP32, so that a warp's 32
// rows of a column are 128 consecutive bytes.
constexpr int kDumpBytes = 256 * 128 * 4;

__device__ __forceinline__ void dump_chunk(float* dump, int c, int row, const uint32_t (&v)[32]) {
#pragma unroll
  for (int i = 0; i < 32; ++i) dump[(c * 32 + i) * 128 + row] = __uint_as_float(v[i]);
}

// Row `row` of columns 32 c .. 32 c + 31, summed over the cluster's CTAs.
__device__ __forceinline__ void sum_chunk(const float* dump, int S, int c, int row, float (&v)[32]) {
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = 0.f;
  for (int s = 0; s < S; ++s) {
    const uint32_t at = map_to_rank(dump + c * 32 * 128 + row, (uint32_t)s);
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      float x;
      asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(at + (uint32_t)i * 512u) : "memory");
      v[i] += x;
    }
  }
}

// residual_chunk without a residual: bf16(act(y)) into buf.
template <class Y>
__device__ __forceinline__ void plain_chunk(uint8_t* buf, bool gelu, Y&& y) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float v[8];
    y(8 * j, v);
    if (gelu) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = gelu_tanh(v[i]);
    }
    uint32_t o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
      o[e] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(buf + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

// This warp's chunks of a split tile, c0, c0 + step .. below c1: the residual of
// its first two (start, before the accumulator is due) ...
__device__ __forceinline__ void start_chunks(const ResidualLoads& loads, int c0, int c1, int step, int n0, int row0) {
  for (int i = 0; i < 2; ++i) {
    if (c0 + i * step < c1) loads.issue(i, n0 + (c0 + i * step) * 32, row0);
    else loads.skip();
  }
}

// ... and, once the cluster has synchronised, Y = bf16([residual + gate *] act(alpha
// sum + bias)), stored through the warp's chunk buffers.
template <bool kRes, bool kResGelu>
__device__ __forceinline__ void finish_chunks(const CUtensorMap* tm_y, const float* dump, int S, int c0, int c1,
                                              int step, const ResidualLoads& loads, const Gate<256>& gate, int n0,
                                              int row0, float alpha, const float* bias_all, bool gelu) {
  const int lane = threadIdx.x & 31, row = (threadIdx.x & 127);   // the warp's quarter of the tile's rows
  const int N = loads.N;
  int b = 0;
#pragma unroll 1
  for (int c = c0; c < c1; c += step, b ^= 1) {
    float sum[32], bias[32];
    sum_chunk(dump, S, c, row, sum);
#pragma unroll
    for (int f = 0; f < 8; ++f) {
      const int col = n0 + c * 32 + 4 * f;
      const float4 b4 = col < N ? __ldg(reinterpret_cast<const float4*>(bias_all + col))
                                : make_float4(0.f, 0.f, 0.f, 0.f);
      bias[4 * f] = b4.x;
      bias[4 * f + 1] = b4.y;
      bias[4 * f + 2] = b4.z;
      bias[4 * f + 3] = b4.w;
    }
    const auto y = [&](int i, float (&v)[8]) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = alpha * sum[i + e] + bias[i + e];
    };
    uint8_t* buf = loads.buf + b * 2048;
    if (kRes) {
      loads.wait();
      residual_chunk<kResGelu>(buf, gate, c, n0, N, y);
    } else {
      if (lane == 0) bulk_wait_group_read<1>();
      __syncwarp();
      plain_chunk(buf, gelu, y);
    }
    fence_async_shared();
    __syncwarp();
    if (lane == 0) {
      tma_store_2d(tm_y, buf, n0 + c * 32, row0);
      bulk_commit_group();
    }
    if (kRes) {
      if (c + 2 * step < c1) {
        if (lane == 0) bulk_wait_group_read<0>();
        __syncwarp();
        loads.issue(b, n0 + (c + 2 * step) * 32, row0);
      } else {
        loads.skip();
      }
    }
  }
  if (kRes) cp_async_wait_all();
  if (lane == 0) bulk_wait_group_all();
}

}  // namespace dev

// CTAs per tile: the largest number up to 8 whose clusters all run at once (no
// tile waits for another) and that leaves each CTA at least `least` of the
// `blocks` K blocks; 1: no split.  active[S]: clusters of S that fit the GPU.
inline int split_of(int tiles, int blocks, int least, const int (&active)[9]) {
  for (int s = 8; s > 1; --s)
    if (tiles <= active[s] && blocks >= least * s) return s;
  return 1;
}

// Fills `active` for a kernel of `threads` threads and `smem` bytes per CTA.
template <class Kernel>
cudaError_t active_clusters(Kernel kern, int threads, size_t smem, int (&active)[9]) {
  for (int s = 2; s <= 8; ++s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)s);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)s;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaOccupancyMaxActiveClusters(&active[s], kern, &cfg);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace svdq
