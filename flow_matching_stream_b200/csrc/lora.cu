// Projections with low-rank adapters of many requests:
//   y = A Wᵀ + scale[a] (A down[a]ᵀ) up[a]ᵀ,  a = adapter of the row's request,
// then the epilogue of krea2_linear on y. This file has the dispatch and the fp32 path (SIMT, reference
// precision); bf16 runs on the tensor cores (lora_tc.cu, gemm_tcgen05.cu). The low-rank product
// t = scale A downᵀ is (rows, rank), so it goes through the workspace; its product with up is added in the
// projection's accumulators.
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
  const long gw = (long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int row = (int)(gw / l.rank), j = (int)(gw % l.rank);
  if (row >= used_rows(l, M)) return;
  const int id = adapter_of_row(l, row);
  float s = 0.f;
  if (id >= 0) {
    const float* x = A + (long)row * K;
    const float* d = reinterpret_cast<const float*>(l.down) + ((long)id * l.rank + j) * K;
    for (int k = lane; k < K; k += 32) s += (x[k]) * (d[k]);
    s = warp_sum(s) * l.scale[id];
  }
  if (lane == 0) t[(long)row * l.rank + j] = s;
}

constexpr int LBM = 64, LBN = 128, LBK = 16;

// 64 x 128 tiles; thread (tx, ty) holds rows ty*4.. and columns tx*4.. of both 64-column halves, so that
// a SwiGLU tile's gate and up columns of one output meet in one thread.
template <int EPI>
__global__ void __launch_bounds__(256) lora_linear_simt_kernel(Krea2Lora l, int M, int N, int K,
                                                               const float* __restrict__ A, const float* __restrict__ W,
                                                               const float* __restrict__ t, void* out,
                                                               const float* __restrict__ gate, int rows_per_batch,
                                                               long long gate_stride) {
  __shared__ float As[LBK][LBM + 4];
  __shared__ float Ws[LBK][LBN + 4];
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int m0 = blockIdx.y * LBM, n0 = blockIdx.x * LBN;
  const int used = used_rows(l, M);
  if (m0 >= used) return;
  float acc[4][8];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[i][j] = 0.f;
  for (int k0 = 0; k0 < K; k0 += LBK) {
    for (int i = threadIdx.x; i < LBM * LBK; i += 256) {
      const int r = i / LBK, k = i % LBK;
      As[k][r] = (m0 + r < used && k0 + k < K) ? (A[(long)(m0 + r) * K + k0 + k]) : 0.f;
    }
    for (int i = threadIdx.x; i < LBN * LBK; i += 256) {
      const int r = i / LBK, k = i % LBK;
      Ws[k][r] = (n0 + r < N && k0 + k < K) ? (W[(long)(n0 + r) * K + k0 + k]) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < LBK; ++k) {
      float a[4], w[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) a[i] = As[k][ty * 4 + i];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        w[j] = Ws[k][tx * 4 + j];
        w[4 + j] = Ws[k][64 + tx * 4 + j];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[i][j] += a[i] * w[j];
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = m0 + ty * 4 + i;
    if (r >= used) continue;
    const int id = adapter_of_row(l, r);
    if (id >= 0) {
      const float* tr = t + (long)r * l.rank;
      const float* up = reinterpret_cast<const float*>(l.up) + (long)id * N * l.rank;
#pragma unroll
      for (int jj = 0; jj < 8; ++jj) {
        const int c = n0 + (jj < 4 ? tx * 4 + jj : 60 + tx * 4 + jj);
        if (c >= N) continue;
        const float* u = up + (long)c * l.rank;
        for (int k = 0; k < l.rank; ++k) acc[i][jj] += tr[k] * (u[k]);
      }
    }
    if constexpr (EPI == EPI_SWIGLU) {
      float* o = reinterpret_cast<float*>(out) + (long)r * (N / 2) + blockIdx.x * 64;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        o[tx * 4 + j] = acc[i][j] / (1.f + expf(-acc[i][j])) * acc[i][4 + j];
      }
    } else {
#pragma unroll
      for (int jj = 0; jj < 8; ++jj) {
        const int c = n0 + (jj < 4 ? tx * 4 + jj : 60 + tx * 4 + jj);
        if (c >= N) continue;
        if constexpr (EPI == EPI_RESID) {
          const int b = rows_per_batch > 0 ? r / rows_per_batch : request_of_row(l.row_start, l.R, r);
          reinterpret_cast<float*>(out)[(long)r * N + c] += gate[(long)b * gate_stride + c] * acc[i][jj];
        } else {
          reinterpret_cast<float*>(out)[(long)r * N + c] = acc[i][jj];
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
  const long warps = (long)a.M * l.rank;
  lora_down_simt_kernel<<<(unsigned)((warps + 7) / 8), 256, 0, stream>>>(l, a.M, a.K, A, t);
  int rc = check_launch("lora_down");
  if (rc) return rc;
  dim3 grid((a.N + LBN - 1) / LBN, (a.M + LBM - 1) / LBM);
  if (grid.y > 65535) return set_error(KREA2_ERR_UNSUPPORTED, "more than %d rows", 65535 * LBM);
#define KREA2_LORA(E)                                                                                            \
  lora_linear_simt_kernel<E><<<grid, 256, 0, stream>>>(l, a.M, a.N, a.K, A, W, t, a.out, a.gate, a.rows_per_batch, \
                                                       a.gate_stride)
  if (epi == EPI_STORE) KREA2_LORA(EPI_STORE);
  else if (epi == EPI_SWIGLU) KREA2_LORA(EPI_SWIGLU);
  else KREA2_LORA(EPI_RESID);
#undef KREA2_LORA
  return check_launch("lora_linear");
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
