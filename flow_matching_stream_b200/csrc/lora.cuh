// Low-rank adapters on the tensor cores: how the low-rank product t = scale A downᵀ is cut into units
// and laid out between the kernel that writes it (lora_tc.cu) and the GEMM that reads it
// (gemm_tcgen05.cu).
//
// A unit is a pair (row tile of 128 rows, request with an adapter and with rows in that tile). Requests
// are consecutive runs of rows, so both parts of the pair never fall from one unit to the next and one of
// them always grows: (row tile + request) names the unit. A unit's slab of t is 128 rows x 2 rankp bf16:
// [high halves | low halves] of the fp32 values (t = high + low to 16 bits of mantissa), zero in the rows
// of other requests and in the columns past the rank.
// Requests of one tile that share an adapter are units of their own all the same, each with a cluster that reads the
// tile of A and with K steps that load the adapter's up: in a tile of one-row requests each adds about 0.6 us at rank 16
// and 0.9 us at rank 64, whether they share an adapter or not (6144 x 6144: one request of 128 rows 26 us, 8 requests
// 27 to 30, 64 requests 60 to 83, 128 requests 98 to 139).
#pragma once
#include <stdint.h>

#include "krea2_internal.h"
#include "ragged.cuh"

namespace krea2 {

// Columns of each half: the K step of an MMA is 16, a stage holds 64 columns (both halves up to rank 32).
__host__ __device__ inline int lora_rankp(int rank) { return rank <= 32 ? (rank + 15) / 16 * 16 : (rank + 63) / 64 * 64; }
__host__ __device__ inline int lora_chunks(int rankp) { return (2 * rankp + 63) / 64; }
__host__ __device__ inline int lora_units(int M, int R) { return (M + 127) / 128 + R; }

#ifdef __CUDACC__
// Rows that belong to requests: [0, row_start[R]), kept inside [0, M].
__device__ __forceinline__ int used_rows(const Krea2Lora& l, int M) { return min(max(__ldg(l.row_start + l.R), 0), M); }

struct LoraUnit {
  int r = -1, adapter = -1;
  __device__ __forceinline__ bool exists() const { return r >= 0; }
};

// The tile's first request from `r` on that has an adapter and rows in the tile.
__device__ __forceinline__ LoraUnit unit_from(const Krea2Lora& l, int M, int mt, int r) {
  const int t0 = mt * 128, t1 = min(t0 + 128, M);
  LoraUnit u;
  for (; r < l.R; ++r) {
    const int a = __ldg(l.row_start + r), b = __ldg(l.row_start + r + 1);
    if (a >= t1) break;
    if (max(a, t0) >= min(b, t1)) continue;
    const int id = __ldg(l.adapter + r);
    if (id < 0 || id >= l.n_adapters) continue;
    u.r = r;
    u.adapter = id;
    break;
  }
  return u;
}
__device__ __forceinline__ LoraUnit first_unit(const Krea2Lora& l, int M, int mt) {
  return unit_from(l, M, mt, request_of_row(l.row_start, l.R, mt * 128));
}
__device__ __forceinline__ LoraUnit next_unit(const Krea2Lora& l, int M, int mt, const LoraUnit& u) {
  return unit_from(l, M, mt, u.r + 1);
}

// Waits until the grid that this one was launched behind as a programmatic dependent has ended and
// its writes are visible.
__device__ __forceinline__ void lora_wait_prior_grid() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("fence.proxy.async.global;" ::: "memory");  // and for the TMA loads that follow
}
#endif

}  // namespace krea2
