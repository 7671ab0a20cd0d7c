// The residual and gate of a GEMM's epilogue: Y = bf16(residual + gate * y).
//
// A warp's output chunk of 32 rows x 32 columns is staged in one of its two
// 2 KB shared-memory buffers for its TMA store anyway, so the residual's chunk
// is copied into the same buffer, in the same 64-byte swizzle: each lane reads
// its row's residual where it then writes Y.  A tile's first two chunks arrive
// while its products are still being summed, the others (brought into L2
// meanwhile) as soon as a buffer's store has been read.  The copies are
// cp.async: as TMA boxes of 64-byte rows they shared that engine with the
// operand stream (4608 x 3072 -> 3072: NVFP4 30.0 against 29.2 us, W8A8 45.3
// against 44.5, INT4 122.4 against 123.1; without a residual 25.9, 40.4, 119.1).
#pragma once

#include <cstdint>

#include "kernels.h"
#include "sm100.cuh"

namespace svdq {
namespace dev {

// One warp's residual chunks, every lane taking part: copies are groups of
// cp.async, one group per chunk (an empty one where there is no chunk), so that
// chunk j has arrived when at most one younger group is in flight.
struct ResidualLoads {
  const __nv_bfloat16* residual;
  uint8_t* buf;                 // two chunk buffers
  int M, N;

  // Copy the 32 x 32 chunk at (x, y) into buffer b, whose last store has been read.
  __device__ __forceinline__ void issue(int b, int x, int y) const {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 8 * i + (lane >> 2), j = lane & 3;  // row, 16-byte piece
      const bool in = y + r < M && x + 8 * j < N;
      cp_async16(buf + b * 2048 + r * 64 + ((j ^ ((r >> 1) & 3)) << 4),
                 residual + (in ? (size_t)(y + r) * N + x + 8 * j : 0), in ? 16u : 0u);
    }
    cp_async_commit();
  }
  __device__ __forceinline__ void skip() const { cp_async_commit(); }
  // The older of the two chunks in flight is in its buffer.
  __device__ __forceinline__ void wait() const {
    cp_async_wait_group<1>();
    __syncwarp();
  }
  // Bring kCols columns from x of this lane's row into L2.
  template <int kCols>
  __device__ __forceinline__ void prefetch(int x, int y) const {
    const int row = y + (threadIdx.x & 31);
    if (row >= M) return;
#pragma unroll
    for (int c = 0; c < kCols; c += 64)
      if (x + c < N) prefetch_l2(residual + (size_t)row * N + x + c);
  }
};

// A warp's gate over kCols columns of a tile.  Where its 32 rows share a gate row
// -- all but where two sequences meet -- the row's values are staged in shared
// memory before the accumulator is due (ones without a gate); otherwise each
// lane reads its own row from global memory, a chunk at a time.
template <int kCols>
struct Gate {
  const __nv_bfloat16* row;     // this lane's gate row at the tile's first column
  uint4* staged;                // kCols / 8 words of this warp
  bool shared;

  __device__ __forceinline__ void tile(const ResidualParams& r, int row0, int M, int col0, int N) {
    const int lane = threadIdx.x & 31;
    int g = 0;
    if (r.gate && r.rows_per_gate > 0) g = min(row0 + lane, M - 1) / r.rows_per_gate;
    row = r.gate + (r.gate ? g * r.gate_stride + col0 : 0);
    shared = __all_sync(0xffffffffu, g == __shfl_sync(0xffffffffu, g, 0));
    if (shared && lane < kCols / 8) {
      uint4 v = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);   // ones
      if (r.gate && col0 + 8 * lane < N) v = *reinterpret_cast<const uint4*>(row + 8 * lane);
      staged[lane] = v;
    }
  }
  // The values of columns c .. c + 31 (c a multiple of 32); past N: anything finite.
  __device__ __forceinline__ void values(int c, int col0, int N, uint4 (&g)[4]) const {
    if (shared) {
#pragma unroll
      for (int j = 0; j < 4; ++j) g[j] = staged[(c >> 3) + j];
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        g[j] = make_uint4(0u, 0u, 0u, 0u);
        if (col0 + c + 8 * j < N) g[j] = *reinterpret_cast<const uint4*>(row + c + 8 * j);
      }
    }
  }
};

// bf16(residual + gate * y) of a pair of neighbouring columns.
__device__ __forceinline__ uint32_t add_gated(uint32_t res, uint32_t gate, float y0, float y1) {
  const float r0 = __uint_as_float(res << 16), r1 = __uint_as_float(res & 0xFFFF0000u);
  const float g0 = __uint_as_float(gate << 16), g1 = __uint_as_float(gate & 0xFFFF0000u);
  const __nv_bfloat162 h = __floats2bfloat162_rn(fmaf(g0, y0, r0), fmaf(g1, y1, r1));
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Columns 32 c .. 32 c + 31 of this lane's row: the residual in buf becomes
// bf16(residual + gate * act(y)).  y(i, v): the eight values before the
// activation from column i of the chunk.  A warp runs this alone on its
// scheduler's issue slots for long stretches, so what counts is the length of
// its dependent chains: the gate is read and the branch over its two sources
// taken before the loop, the activation is a compile-time choice, and the next
// eight columns' residual is read before the present ones are written (the
// compiler must take the two for the same addresses).  With the branches inside
// the loop a chunk took 1150 cycles, without them 480.
template <bool kGelu, int kCols, class Y>
__device__ __forceinline__ void residual_chunk(uint8_t* buf, const Gate<kCols>& gate, int c, int col0, int N, Y&& y) {
  const int lane = threadIdx.x & 31;
  uint8_t* line = buf + lane * 64;
  const int swz = (lane >> 1) & 3;                      // 64-byte swizzle
  uint4 g[4];
  gate.values(32 * c, col0, N, g);
  uint4 r = *reinterpret_cast<const uint4*>(line + (swz << 4));
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float v[8];
    y(8 * j, v);
    uint4 next = r;
    if (j < 3) next = *reinterpret_cast<const uint4*>(line + (((j + 1) ^ swz) << 4));
    if (kGelu) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = gelu_tanh(v[i]);
    }
    uint4 o;
    o.x = add_gated(r.x, g[j].x, v[0], v[1]);
    o.y = add_gated(r.y, g[j].y, v[2], v[3]);
    o.z = add_gated(r.z, g[j].z, v[4], v[5]);
    o.w = add_gated(r.w, g[j].w, v[6], v[7]);
    *reinterpret_cast<uint4*>(line + ((j ^ swz) << 4)) = o;
    r = next;
  }
}

}  // namespace dev
}  // namespace svdq
