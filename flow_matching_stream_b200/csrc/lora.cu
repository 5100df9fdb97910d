// Projections with low-rank adapters of many requests:
//   y = A Wᵀ + scale[a] (A down[a]ᵀ) up[a]ᵀ,  a = adapter of the row's request,
// then the epilogue of krea2_linear on y. The low-rank product t = scale A downᵀ is (rows, rank), so it
// goes through the workspace; its own product with up is added in the projection's accumulators.
#include <math.h>

#include "krea2_device.cuh"
#include "krea2_internal.h"
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

// Rows that belong to requests: [0, row_start[R]), kept inside [0, M].
__device__ __forceinline__ int used_rows(const Krea2Lora& l, int M) { return min(max(__ldg(l.row_start + l.R), 0), M); }

__device__ __forceinline__ int adapter_of_row(const Krea2Lora& l, int row) {
  const int id = l.adapter[request_of_row(l.row_start, l.R, row)];
  return id >= 0 && id < l.n_adapters ? id : -1;
}

template <typename T>
__device__ __forceinline__ float to_f(T x) {
  if constexpr (sizeof(T) == 2) return __bfloat162float(x);
  else return x;
}

// t (M, rank) fp32: one warp per (row, rank column).
template <typename T>
__global__ void __launch_bounds__(256) lora_down_simt_kernel(Krea2Lora l, int M, int K, const T* __restrict__ A,
                                                             float* __restrict__ t) {
  check_lora(l, M);
  const long gw = (long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int row = (int)(gw / l.rank), j = (int)(gw % l.rank);
  if (row >= used_rows(l, M)) return;
  const int id = adapter_of_row(l, row);
  float s = 0.f;
  if (id >= 0) {
    const T* x = A + (long)row * K;
    const T* d = reinterpret_cast<const T*>(l.down) + ((long)id * l.rank + j) * K;
    for (int k = lane; k < K; k += 32) s += to_f(x[k]) * to_f(d[k]);
    s = warp_sum(s) * l.scale[id];
  }
  if (lane == 0) t[(long)row * l.rank + j] = s;
}

constexpr int LBM = 64, LBN = 128, LBK = 16;

// 64 x 128 tiles; thread (tx, ty) holds rows ty*4.. and columns tx*4.. of both 64-column halves, so that
// a SwiGLU tile's gate and up columns of one output meet in one thread.
template <typename T, int EPI>
__global__ void __launch_bounds__(256) lora_linear_simt_kernel(Krea2Lora l, int M, int N, int K,
                                                               const T* __restrict__ A, const T* __restrict__ W,
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
      As[k][r] = (m0 + r < used && k0 + k < K) ? to_f(A[(long)(m0 + r) * K + k0 + k]) : 0.f;
    }
    for (int i = threadIdx.x; i < LBN * LBK; i += 256) {
      const int r = i / LBK, k = i % LBK;
      Ws[k][r] = (n0 + r < N && k0 + k < K) ? to_f(W[(long)(n0 + r) * K + k0 + k]) : 0.f;
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
      const T* up = reinterpret_cast<const T*>(l.up) + (long)id * N * l.rank;
#pragma unroll
      for (int jj = 0; jj < 8; ++jj) {
        const int c = n0 + (jj < 4 ? tx * 4 + jj : 60 + tx * 4 + jj);
        if (c >= N) continue;
        const T* u = up + (long)c * l.rank;
        for (int k = 0; k < l.rank; ++k) acc[i][jj] += tr[k] * to_f(u[k]);
      }
    }
    if constexpr (EPI == EPI_SWIGLU) {
      T* o = reinterpret_cast<T*>(out) + (long)r * (N / 2) + blockIdx.x * 64;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float y = acc[i][j] / (1.f + expf(-acc[i][j])) * acc[i][4 + j];
        if constexpr (sizeof(T) == 2) o[tx * 4 + j] = __float2bfloat16_rn(y);
        else o[tx * 4 + j] = y;
      }
    } else {
#pragma unroll
      for (int jj = 0; jj < 8; ++jj) {
        const int c = n0 + (jj < 4 ? tx * 4 + jj : 60 + tx * 4 + jj);
        if (c >= N) continue;
        if constexpr (EPI == EPI_RESID) {
          const int b = rows_per_batch > 0 ? r / rows_per_batch : request_of_row(l.row_start, l.R, r);
          reinterpret_cast<float*>(out)[(long)r * N + c] += gate[(long)b * gate_stride + c] * acc[i][jj];
        } else if constexpr (sizeof(T) == 2) {
          reinterpret_cast<T*>(out)[(long)r * N + c] = __float2bfloat16_rn(acc[i][jj]);
        } else {
          reinterpret_cast<T*>(out)[(long)r * N + c] = acc[i][jj];
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

template <typename T>
int lora_simt(int epi, const LoraLinearArgs& a, const Krea2Lora& l, float* t, cudaStream_t stream) {
  const T* A = reinterpret_cast<const T*>(a.A);
  const T* W = reinterpret_cast<const T*>(a.W);
  const long warps = (long)a.M * l.rank;
  lora_down_simt_kernel<T><<<(unsigned)((warps + 7) / 8), 256, 0, stream>>>(l, a.M, a.K, A, t);
  int rc = check_launch("lora_down");
  if (rc) return rc;
  dim3 grid((a.N + LBN - 1) / LBN, (a.M + LBM - 1) / LBM);
  if (grid.y > 65535) return set_error(KREA2_ERR_UNSUPPORTED, "more than %d rows", 65535 * LBM);
#define KREA2_LORA(E)                                                                                            \
  lora_linear_simt_kernel<T, E><<<grid, 256, 0, stream>>>(l, a.M, a.N, a.K, A, W, t, a.out, a.gate,              \
                                                          a.rows_per_batch, a.gate_stride)
  if (epi == EPI_STORE) KREA2_LORA(EPI_STORE);
  else if (epi == EPI_SWIGLU) KREA2_LORA(EPI_SWIGLU);
  else KREA2_LORA(EPI_RESID);
#undef KREA2_LORA
  return check_launch("lora_linear");
}

}  // namespace

size_t lora_workspace_bytes(int dtype, int epi, int M, int N, int K, int R, int rank) {
  return (size_t)M * rank * 4;
}

int launch_lora_linear(int dtype, int epi, const LoraLinearArgs& a, const Krea2Lora& l, void* ws, cudaStream_t stream) {
  float* t = reinterpret_cast<float*>(ws);
  return dtype == KREA2_BF16 ? lora_simt<__nv_bfloat16>(epi, a, l, t, stream) : lora_simt<float>(epi, a, l, t, stream);
}

}  // namespace krea2
