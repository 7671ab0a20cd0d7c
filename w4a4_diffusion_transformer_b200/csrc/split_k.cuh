// K split over the CTAs of a cluster, for GEMMs with too few tiles to fill the
// GPU: the S CTAs of a cluster compute one output tile, each over its share of K.
// When their products are summed, each writes its accumulator to its own shared
// memory (the operand ring, idle by then), the cluster synchronises, and each
// finishes the tile's columns [256 r / S, 256 (r + 1) / S), r its rank: it adds
// the S partial sums in rank order over distributed shared memory, so the result
// does not depend on timing and needs no workspace.
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

}  // namespace dev

// CTAs per tile: the largest of 8, 4, 2 whose clusters all run at once (no tile
// waits for another) and that leaves each CTA at least `least` of the `blocks`
// K blocks; 1: no split.  `active`: clusters of 2, 4, 8 that fit the GPU.
inline int split_of(int tiles, int blocks, int least, const int (&active)[3]) {
  for (int i = 2; i >= 0; --i)
    if (tiles <= active[i] && blocks >= least * (2 << i)) return 2 << i;
  return 1;
}

// Fills `active` for a kernel of `threads` threads and `smem` bytes per CTA.
template <class Kernel>
cudaError_t active_clusters(Kernel kern, int threads, size_t smem, int (&active)[3]) {
  for (int i = 0; i < 3; ++i) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(8);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2u << i;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaOccupancyMaxActiveClusters(&active[i], kern, &cfg);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace svdq
