// Projections with low-rank adapters of many requests:
//   y = A Wᵀ + scale[a] (A down[a]ᵀ) up[a]ᵀ,  a = adapter of the row's request,
// then the epilogue of krea2_linear on y. This file has the dispatch and the fp32 path (SIMT, reference
// precision); bf16 runs on the tensor cores (lora_tc.cu, gemm_tcgen05.cu). The low-rank product
// t = scale A downᵀ is (rows, rank), so it goes through the workspace; its product with up is added in the
// projection's accumulators. The fp32 path at full width, rank 16: 512 rows by 15360 x 6144 4.3 ms, by 32768 x 6144
// (SwiGLU) 8.4 ms, by 6144 x 16384 (residual) 4.8 ms, 21 to 25 TFLOP/s; one row by 6144 x 6144 172 us.
#include <math.h>

#include "krea2_device.cuh"
#include "krea2_internal.h"
#include "lora.cuh"
#include "ragged.cuh"

namespace krea2 {

KREA2_DEFINE_ERROR_READER(take_device_error_lora)

namespace {

// Block 0 checks the batch arrays: row starts ascend from 0 to at most M, adapter numbers exist.
__device__ __forceinline__ void check_lora(const Krea2Lora& l, int M) {
  if (blockIdx.x || blockIdx.y) return;
  for (int r = threadIdx.x; r < l.R; r += blockDim.x) {
    const int a = l.row_start[r], b = l.row_start[r + 1], id = l.adapter[r];
    if (a < 0 || b < a || b > M || (r == 0 && a != 0) || id < -1 || id >= l.n_adapters)
      atomicOr(&g_device_error, ERR_BAD_BATCH);
  }
}

__device__ __forceinline__ int adapter_of_row(const Krea2Lora& l, int row) {
  const int id = l.adapter[request_of_row(l.row_start, l.R, row)];
  return id >= 0 && id < l.n_adapters ? id : -1;
}

// t (M, rank) fp32: one warp per (row, rank column).
__global__ void __launch_bounds__(256) lora_down_simt_kernel(Krea2Lora l, int M, int K, const float* __restrict__ A,
                                                             float* __restrict__ t) {
  check_lora(l, M);
  // the projection behind this grid may start (it waits for t itself)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const long gw = (long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int row = (int)(gw / l.rank), j = (int)(gw % l.rank);
  if (row >= used_rows(l, M)) return;
  const int id = adapter_of_row(l, row);
  float s = 0.f;
  if (id >= 0) {
    const float* x = A + (long)row * K;
    const float* d = reinterpret_cast<const float*>(l.down) + ((long)id * l.rank + j) * K;
    for (int k = lane; k < K; k += 32) s += x[k] * d[k];
    s = warp_sum(s) * l.scale[id];
  }
  if (lane == 0) t[(long)row * l.rank + j] = s;
}

// TM x TN tiles of the output. A tile's columns are TN / 2 neighbours of the first and the same of the second half
// of a 128-column group, so that a SwiGLU output's gate and up columns meet in one thread; a thread holds RM rows
// and HC columns of each half.
template <int TM, int TN, int RM, int HC, int BK, int EPI>
__global__ void __launch_bounds__((TM / RM) * (TN / (2 * HC)))
    lora_linear_simt_kernel(Krea2Lora l, int M, int N, int K, const float* __restrict__ A, const float* __restrict__ W,
                            const float* __restrict__ t, void* out, const float* __restrict__ gate, int rows_per_batch,
                            long long gate_stride) {
  constexpr int TX = TN / (2 * HC), NT = (TM / RM) * TX, HALF = TN / 2, PER_GROUP = 128 / TN;
  constexpr int LA = TM * BK / NT, LW = TN * BK / NT;
  __shared__ float As[BK][TM + 1];
  __shared__ float Ws[BK][TN + 1];
  const int tx = threadIdx.x % TX, ty = threadIdx.x / TX;
  const int m0 = blockIdx.y * TM, c0 = (blockIdx.x / PER_GROUP) * 128 + (blockIdx.x % PER_GROUP) * HALF;
  auto col = [&](int c) { return c0 + (c % HALF) + (c / HALF) * 64; };  // of the tile's column c
  const int used = used_rows(l, M);
  if (m0 >= used) {
    lora_wait_prior_grid();
    return;
  }
  float acc[RM][2 * HC];
#pragma unroll
  for (int i = 0; i < RM; ++i)
#pragma unroll
    for (int j = 0; j < 2 * HC; ++j) acc[i][j] = 0.f;
  float ra[LA], rw[LW];  // the next K step's elements, on their way while this one is multiplied
  auto load = [&](int k0) {
#pragma unroll
    for (int i = 0; i < LA; ++i) {
      const int e = threadIdx.x + i * NT, r = m0 + e / BK, k = k0 + e % BK;
      ra[i] = (r < used && k < K) ? A[(long long)r * K + k] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < LW; ++i) {
      const int e = threadIdx.x + i * NT, n = col(e / BK), k = k0 + e % BK;
      rw[i] = (n < N && k < K) ? W[(long long)n * K + k] : 0.f;
    }
  };
  load(0);
  for (int k0 = 0; k0 < K; k0 += BK) {
#pragma unroll
    for (int i = 0; i < LA; ++i) As[(threadIdx.x + i * NT) % BK][(threadIdx.x + i * NT) / BK] = ra[i];
#pragma unroll
    for (int i = 0; i < LW; ++i) Ws[(threadIdx.x + i * NT) % BK][(threadIdx.x + i * NT) / BK] = rw[i];
    __syncthreads();
    if (k0 + BK < K) load(k0 + BK);
#pragma unroll 16
    for (int k = 0; k < BK; ++k) {
      float a[RM], w[2 * HC];
#pragma unroll
      for (int i = 0; i < RM; ++i) a[i] = As[k][ty * RM + i];
#pragma unroll
      for (int j = 0; j < HC; ++j) {
        w[j] = Ws[k][tx * HC + j];
        w[HC + j] = Ws[k][HALF + tx * HC + j];
      }
#pragma unroll
      for (int i = 0; i < RM; ++i)
#pragma unroll
        for (int j = 0; j < 2 * HC; ++j) acc[i][j] += a[i] * w[j];
    }
    __syncthreads();
  }
  lora_wait_prior_grid();  // t is written by the grid before this one
#pragma unroll
  for (int i = 0; i < RM; ++i) {
    const int r = m0 + ty * RM + i;
    if (r >= used) continue;
    const int id = adapter_of_row(l, r);
    if (id >= 0) {  // rank is a multiple of 8: whole 16-byte loads
      const float4* tr = reinterpret_cast<const float4*>(t + (long long)r * l.rank);
      const float* up = reinterpret_cast<const float*>(l.up) + (long long)id * N * l.rank;
#pragma unroll
      for (int j = 0; j < 2 * HC; ++j) {
        const int c = col(j < HC ? tx * HC + j : HALF + tx * HC + j - HC);
        if (c >= N) continue;
        const float4* u = reinterpret_cast<const float4*>(up + (long long)c * l.rank);
        for (int k = 0; k < l.rank / 4; ++k) {
          const float4 x = tr[k], y = u[k];
          acc[i][j] += x.x * y.x;
          acc[i][j] += x.y * y.y;
          acc[i][j] += x.z * y.z;
          acc[i][j] += x.w * y.w;
        }
      }
    }
    if constexpr (EPI == EPI_SWIGLU) {
      float* o = reinterpret_cast<float*>(out) + (long long)r * (N / 2) + c0 / 128 * 64 + c0 % 128;
#pragma unroll
      for (int j = 0; j < HC; ++j) o[tx * HC + j] = acc[i][j] / (1.f + expf(-acc[i][j])) * acc[i][HC + j];
    } else {
#pragma unroll
      for (int j = 0; j < 2 * HC; ++j) {
        const int c = col(j < HC ? tx * HC + j : HALF + tx * HC + j - HC);
        if (c >= N) continue;
        if constexpr (EPI == EPI_RESID) {
          const int b = rows_per_batch > 0 ? r / rows_per_batch : request_of_row(l.row_start, l.R, r);
          reinterpret_cast<float*>(out)[(long long)r * N + c] += gate[(long long)b * gate_stride + c] * acc[i][j];
        } else {
          reinterpret_cast<float*>(out)[(long long)r * N + c] = acc[i][j];
        }
      }
    }
  }
}

int check_launch(const char* what) {
  count_launch();
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return set_error(KREA2_ERR_CUDA, "%s launch failed: %s", what, cudaGetErrorString(e));
  return KREA2_OK;
}

int lora_simt(int epi, const LoraLinearArgs& a, const Krea2Lora& l, float* t, cudaStream_t stream) {
  const float* A = reinterpret_cast<const float*>(a.A);
  const float* W = reinterpret_cast<const float*>(a.W);
  // 64 x 128 tiles, or 16 x 32 where those would leave most SMs without one (73 x 640, K 256: 10 large tiles take
  // 55 us, 100 small ones 8 us; from two large tiles per SM on the large ones' reuse wins)
  const int groups = (a.N + 127) / 128;
  const bool small = (long long)groups * ((a.M + 63) / 64) < 2L * num_sms();
  const dim3 grid(small ? groups * 4 : groups, small ? (a.M + 15) / 16 : (a.M + 63) / 64);
  if (grid.y > 65535) return set_error(KREA2_ERR_UNSUPPORTED, "more than %d rows", 65535 * 64);
  const long warps = (long)a.M * l.rank;
  lora_down_simt_kernel<<<(unsigned)((warps + 7) / 8), 256, 0, stream>>>(l, a.M, a.K, A, t);
  int rc = check_launch("lora_down");
  if (rc) return rc;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(small ? 128 : 256);
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  cudaError_t e;
#define KREA2_LORA(E)                                                                                              \
  e = cudaLaunchKernelEx(&cfg, small ? lora_linear_simt_kernel<16, 32, 1, 2, 64, E>                                \
                                     : lora_linear_simt_kernel<64, 128, 4, 4, 16, E>,                              \
                         l, a.M, a.N, a.K, A, W, (const float*)t, a.out, a.gate, a.rows_per_batch, a.gate_stride)
  if (epi == EPI_STORE) {
    KREA2_LORA(EPI_STORE);
  } else if (epi == EPI_SWIGLU) {
    KREA2_LORA(EPI_SWIGLU);
  } else {
    KREA2_LORA(EPI_RESID);
  }
#undef KREA2_LORA
  count_launch();
  if (e != cudaSuccess) return set_error(KREA2_ERR_CUDA, "lora_linear launch failed: %s", cudaGetErrorString(e));
  return KREA2_OK;
}

}  // namespace

size_t lora_workspace_bytes(int dtype, int epi, int M, int N, int K, int R, int rank) {
  (void)epi, (void)N, (void)K;
  return dtype == KREA2_BF16 ? lora_t_bytes(M, R, rank) : (size_t)M * rank * 4;
}

int launch_lora_linear(int dtype, int epi, const LoraLinearArgs& a, const Krea2Lora& l, void* ws, cudaStream_t stream) {
  if (dtype != KREA2_BF16) return lora_simt(epi, a, l, reinterpret_cast<float*>(ws), stream);
  int rc = launch_lora_down_tc(a.A, a.M, a.K, l, ws, stream);
  if (rc) return rc;
  GemmParams p{};
  p.M = a.M; p.N = a.N; p.K = a.K; p.out = a.out;
  p.gate = a.gate; p.rows_per_batch = a.rows_per_batch; p.gate_stride = a.gate_stride;
  return gemm_bf16_lora(epi, p, a.A, a.W, l, ws, stream);
}

}  // namespace krea2
