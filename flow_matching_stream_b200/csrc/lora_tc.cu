// The low-rank product of the adapters on the tensor cores: t = scale[a] (A down[a]ᵀ), bf16 in, fp32
// accumulation, written as [high | low] bf16 halves per unit (lora.cuh) for the GEMM that adds t upᵀ.
//
// Bound by reading A (and down) once: 2 M K r operations on 2 M K bytes are 16 operations a byte at
// rank 16. One cluster per unit; its CTAs split K, each accumulates its part in TMEM (tcgen05, M = 128,
// N = rank), puts the fp32 part into its own shared memory, and sums a slice of the rows over all parts
// through distributed shared memory in a fixed order, so that results repeat bit for bit. t is kept to 16 bits
// of mantissa as two halves: rounded to bf16 once, it would be the largest error of an fp32 residual, and the
// second half costs the GEMM one more K step of 16 to 64 per 6144 or more. Measured: 16 us for 1589 x 6144,
// rank 64; 38 us for 4818 x 16384, rank 32 (4.1 TB/s).
#include <cuda.h>

#include "krea2_device.cuh"
#include "krea2_internal.h"
#include "lora.cuh"
#include "ragged.cuh"

namespace krea2 {

int make_tmap_bf16_chunks(CUtensorMap* m, const void* ptr, uint64_t cols, uint64_t rows, uint64_t batches,
                          uint32_t box_rows, uint32_t box_chunks);

KREA2_DEFINE_ERROR_READER(take_device_error_lora_tc)

namespace {

constexpr int MAX_STAGES = 6;
// Alignment, and the rows behind a short batch's that an MMA of 128 rows reads past the last stage's.
constexpr int SMEM_SLACK = 1024 + (8 << 10);
constexpr int DOWN_THREADS = 192;  // producer, MMA, 4 warps that empty TMEM; all of them reduce

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float ld_peer(uint32_t saddr, uint32_t rank) {
  uint32_t a;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(saddr), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}

// The (row tile, request) of unit u, if u is one. request + start / 128 never falls and is at most u for
// the request sought and all before it.
__device__ __forceinline__ LoraUnit unit_of(const Krea2Lora& l, int M, int u, int* mt) {
  int lo = 0, hi = l.R;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (mid + (__ldg(l.row_start + mid) >> 7) <= u) lo = mid;
    else hi = mid;
  }
  *mt = u - lo;
  LoraUnit x;
  if (*mt < 0) return x;
  x = unit_from(l, M, *mt, lo);
  if (x.r != lo) x.r = -1;
  return x;
}

// splits: CTAs per cluster; N: rank rounded up to 16; kch: K steps of 64 columns per stage (one thread's
// turn of a wait and two loads takes about 0.3 us whatever it loads), A's a_pitch bytes apart.
__global__ void __launch_bounds__(DOWN_THREADS) lora_down_tc_kernel(const __grid_constant__ CUtensorMap tmA,
                                                                    const __grid_constant__ CUtensorMap tmD,
                                                                    Krea2Lora l, int M, int K, int N, int stages,
                                                                    int splits, int tmem_cols, int rankp, int a_pitch, int kch,
                                                                    __nv_bfloat16* __restrict__ t) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full_bar[MAX_STAGES];
  __shared__ __align__(8) uint64_t empty_bar[MAX_STAGES];
  __shared__ __align__(8) uint64_t done_bar;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t base_u32 = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* base = smem_raw + (base_u32 - smem_u32(smem_raw));
  const int split = (int)cluster_rank();
  const int unit = blockIdx.x / splits;
  if (blockIdx.x == 0) {  // the batch arrays: row starts ascend from 0 to at most M, adapter numbers exist
    for (int r = threadIdx.x; r < l.R; r += DOWN_THREADS) {
      const int a = l.row_start[r], b = l.row_start[r + 1], id = l.adapter[r];
      if (a < 0 || b < a || b > M || (r == 0 && a != 0) || id < -1 || id >= l.n_adapters)
        atomicOr(&g_device_error, ERR_BAD_BATCH);
    }
  }
  const int used = used_rows(l, M);
  int mt;
  const LoraUnit x = unit_of(l, used, unit, &mt);
  if (!x.exists()) return;  // the whole cluster

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    mbar_init(&done_bar, 1);
    abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) tmem_alloc(&tmem_slot, tmem_cols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  volatile int* abort = &abort_flag;
  // the GEMM behind this grid may start (it waits for t itself): this CTA has its TMEM
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int nk = (K / 64 + kch - 1) / kch;  // stages over the whole of K (chunks past it read as zeros)
  const int k0 = (int)((long)split * nk / splits), k1 = (int)((long)(split + 1) * nk / splits);
  const int d_off = kch * a_pitch, stage_bytes = d_off + kch * N * 128;

  if (warp == 0) {
    if (lane == 0) {
      uint32_t stage = 0, phase = 0;
      IssuedFills fills;
      for (int kb = k0; kb < k1; ++kb) {
        if (!mbar_wait(&empty_bar[stage], phase ^ 1, abort)) break;
        uint8_t* sa = base + stage * stage_bytes;
        mbar_arrive_expect_tx(&full_bar[stage], stage_bytes);
        tma_load_4d(sa, &tmA, &full_bar[stage], 0, mt * 128, kb * kch, 0);
        tma_load_4d(sa + d_off, &tmD, &full_bar[stage], 0, 0, kb * kch, x.adapter);
        fills.note(stage, phase);
        if (++stage == (uint32_t)stages) {
          stage = 0;
          phase ^= 1;
        }
      }
      if (*abort) fills.drain(full_bar, stages);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      uint32_t stage = 0, phase = 0;
      const uint32_t idesc = idesc_bf16_f32(128, N);
      const uint64_t da0 = smem_desc_sw128(smem_u32(base), 16, 1024);
      for (int kb = k0; kb < k1; ++kb) {
        if (!mbar_wait(&full_bar[stage], phase, abort)) break;
        tc_fence_after();
        uint64_t ad = da0 + (uint64_t)(stage * (stage_bytes >> 4));
        uint64_t bd = ad + (uint64_t)(d_off >> 4);
        for (int c = 0; c < kch; ++c, ad += a_pitch >> 4, bd += N * 128 >> 4)
#pragma unroll
          for (int k = 0; k < 4; ++k) tc_mma_bf16(tmem, ad + 2 * k, bd + 2 * k, idesc, kb > k0 || c > 0 || k > 0);
        tc_commit(&empty_bar[stage]);
        if (++stage == (uint32_t)stages) {
          stage = 0;
          phase ^= 1;
        }
      }
      // also on the abort path: the MMAs issued so far must end before TMEM is released
      tc_commit(&done_bar);
      mbar_wait_drain(&done_bar, 0);
    }
    __syncwarp();
  }
  // every MMA has ended (and with it every use of the ring) once warp 1 is here
  __syncthreads();
  tc_fence_after();
  float* part = reinterpret_cast<float*>(base);  // [128][N + 1] over the ring
  const int ld = N + 1;
  if (warp >= 2) {
    const int row = (warp & 3) * 32 + lane;
    for (int c = 0; c < N; c += 16) {
      uint32_t r[16];
      asm volatile(
          "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
          "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
          "tcgen05.wait::ld.sync.aligned;"
          : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
            "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
          : "r"(tmem + ((uint32_t)((warp & 3) * 32) << 16) + c)
          : "memory");
#pragma unroll
      for (int e = 0; e < 16; ++e) part[row * ld + c + e] = __uint_as_float(r[e]);
    }
  }
  tc_fence_before();
  cluster_sync();  // all parts are in shared memory

  // this CTA's rows of the unit: sum over the cluster's parts, scale, split into halves
  const int row_a = split * 128 / splits, row_b = (split + 1) * 128 / splits;
  const int a = max(__ldg(l.row_start + x.r), mt * 128) - mt * 128;
  const int b = min(min(__ldg(l.row_start + x.r + 1), used), mt * 128 + 128) - mt * 128;
  const float scale = l.scale[x.adapter];
  const uint32_t part_u32 = smem_u32(part);
  __nv_bfloat16* dst = t + (size_t)unit * 128 * (2 * rankp);
  for (int i = threadIdx.x; i < (row_b - row_a) * rankp; i += DOWN_THREADS) {
    const int row = row_a + i / rankp, c = i % rankp;
    float v = 0.f;
    if (c < N && row >= a && row < b) {
      for (int s = 0; s < splits; ++s) v += ld_peer(part_u32 + (uint32_t)(row * ld + c) * 4u, s);
      v *= scale;
    }
    const __nv_bfloat16 high = __float2bfloat16_rn(v);
    dst[(size_t)row * (2 * rankp) + c] = high;
    // an infinite value has no low half (infinity minus itself would be NaN)
    const float low = isinf(__bfloat162float(high)) ? 0.f : v - __bfloat162float(high);
    dst[(size_t)row * (2 * rankp) + rankp + c] = __float2bfloat16_rn(low);
  }
  cluster_sync();  // no CTA ends while a peer still reads its part
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, tmem_cols);
  }
}

}  // namespace

size_t lora_t_bytes(int M, int R, int rank) { return (size_t)lora_units(M, R) * 128 * 2 * lora_rankp(rank) * 2; }

int launch_lora_down_tc(const void* A, int M, int K, const Krea2Lora& l, void* t, cudaStream_t stream) {
  const int N = (l.rank + 15) / 16 * 16, rankp = lora_rankp(l.rank);
  const int units = lora_units(M, l.R) - 1;  // the largest unit number is (row tiles - 1) + (R - 1)
  const int a_rows = M < 128 ? (M + 7) / 8 * 8 : 128;  // the rows behind them are not used
  const int a_pitch = a_rows * 128, step = a_pitch + N * 128;
  const int kch = 4 * step <= (36 << 10) ? 4 : 2 * step <= (48 << 10) ? 2 : 1;
  const int stage_bytes = kch * step;
  const int nk = (K / 64 + kch - 1) / kch;
  // two CTAs fit an SM up to N = 128: as many parts of K as fill the SMs once
  const int slots = N > 128 ? num_sms() : 2 * num_sms();
  int splits = slots / units;
  splits = splits < 1 ? 1 : splits > 8 ? 8 : splits;
  if (splits > nk) splits = nk;
  int stages = N > 128 ? 4 : (96 << 10) / stage_bytes;
  if (stages > MAX_STAGES) stages = MAX_STAGES;
  if (stages > (nk + splits - 1) / splits) stages = (nk + splits - 1) / splits;
  int smem = stages * stage_bytes;
  const int part = 128 * (N + 1) * 4;
  if (smem < part) smem = part;
  smem += SMEM_SLACK;
  constexpr int MOST = 4 * (128 + 256) * 128 + SMEM_SLACK;  // N = 256
  static std::atomic<uint64_t> attr_done{0};
  const uint64_t dev_bit = device_bit();
  if (!(attr_done.load(std::memory_order_acquire) & dev_bit) || !dev_bit) {
    if (cudaFuncSetAttribute(lora_down_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, MOST) != cudaSuccess)
      return set_error(KREA2_ERR_CUDA, "cudaFuncSetAttribute(lora_down) failed");
    attr_done.fetch_or(dev_bit, std::memory_order_release);
  }
  CUtensorMap ta, td;
  int rc;
  if ((rc = make_tmap_bf16_chunks(&ta, A, K, M, 1, a_rows, kch)) ||
      (rc = make_tmap_bf16_chunks(&td, l.down, K, l.rank, l.n_adapters, N, kch)))
    return rc;
  int tmem_cols = 32;
  while (tmem_cols < N) tmem_cols *= 2;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(units * splits));
  cfg.blockDim = dim3(DOWN_THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = splits;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, lora_down_tc_kernel, ta, td, l, M, K, N, stages, splits, tmem_cols, rankp, a_pitch, kch,
                                           reinterpret_cast<__nv_bfloat16*>(t));
  count_launch();
  if (e != cudaSuccess) return set_error(KREA2_ERR_CUDA, "lora_down launch failed: %s", cudaGetErrorString(e));
  return KREA2_OK;
}

}  // namespace krea2
