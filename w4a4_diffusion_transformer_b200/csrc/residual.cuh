// The residual and gate of a GEMM's epilogue: Y = bf16(residual + gate * y).
//
// A warp's output chunk of 32 rows x 32 columns is staged in one of its two
// 2 KB shared-memory buffers for its TMA store anyway, so the residual's chunk
// is loaded by TMA into the same buffer, in the same 64-byte swizzle, two
// chunks ahead: the first two of a tile arrive while its products are still
// being summed.  Each lane reads its row's residual where it then writes Y.
#pragma once

#include <cstdint>

#include "kernels.h"
#include "sm100.cuh"

namespace svdq {
namespace dev {

constexpr int kResChunkBytes = 32 * 64;

// One warp's chunk loads: chunk j goes to buffer j & 1 and completes bar[j & 1].
struct ResidualLoads {
  const CUtensorMap* map;
  uint64_t* bar;                // [2], one arrival each
  uint8_t* buf;                 // two chunk buffers
  int issued;

  // Lane 0: load the next chunk from (x, y); its buffer's last store has been read.
  __device__ __forceinline__ void issue(int x, int y) {
    uint64_t* b = bar + (issued & 1);
    mbar_arrive_expect_tx(b, kResChunkBytes);
    tma_load_2d(buf + (issued & 1) * kResChunkBytes, map, b, x, y);
    ++issued;
  }
  // All lanes: wait for chunk j.
  __device__ __forceinline__ bool wait(int j, const volatile int* abort_flag, uint64_t budget_ns) const {
    return mbar_wait(bar + (j & 1), (uint32_t)(j >> 1) & 1u, abort_flag, budget_ns);
  }
  // Lane 0, before it leaves: no load may be in flight (at most the last two are).
  __device__ __forceinline__ void drain(const volatile int* abort_flag, uint64_t budget_ns) const {
    for (int j = max(0, issued - 2); j < issued; ++j) wait(j, abort_flag, budget_ns);
  }
};

// Pointer to the gate row of an output row, or null (a gate of 1).
__device__ __forceinline__ const __nv_bfloat16* gate_row(const ResidualParams& r, int row, int M) {
  if (!r.gate) return nullptr;
  const int m = min(row, M - 1);
  return r.gate + (r.rows_per_gate > 0 ? m / r.rows_per_gate : 0) * r.gate_stride;
}

// Eight gate values from column col (a multiple of 8; past N: zeros).
__device__ __forceinline__ uint4 gate8(const __nv_bfloat16* row, int col, int N) {
  if (!row) return make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);   // ones
  return col < N ? *reinterpret_cast<const uint4*>(row + col) : make_uint4(0u, 0u, 0u, 0u);
}

// bf16(residual + gate * y) of a pair of neighbouring columns.
__device__ __forceinline__ uint32_t add_gated(uint32_t res, uint32_t gate, float y0, float y1) {
  const float r0 = __uint_as_float(res << 16), r1 = __uint_as_float(res & 0xFFFF0000u);
  const float g0 = __uint_as_float(gate << 16), g1 = __uint_as_float(gate & 0xFFFF0000u);
  const __nv_bfloat162 h = __floats2bfloat162_rn(fmaf(g0, y0, r0), fmaf(g1, y1, r1));
  return *reinterpret_cast<const uint32_t*>(&h);
}

}  // namespace dev
}  // namespace svdq
