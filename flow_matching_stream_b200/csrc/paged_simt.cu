// Paged key/value cache of a ragged batch: the append of new tokens, and a SIMT attention for fp32 and
// for the shapes that the tensor-core attention does not take (attention_paged_tc.cu).
//
//   append     k_hat = RoPE(k / rms(k) (1 + w)), v as projected, into row t % page_size of page
//              page_table[r, t / page_size] for the token at position t of request r
//   attention  out = sigmoid(g) sum_t softmax_t(q_hat k_hat_t / sqrt(D)) v_t over the readable keys
//              (page "Diffusers 中的 Krea2Transformer2DModel … 架构全解", §四.3; block-causal limits from
//              page "QwenImage21Transformer2DModel")
#include <math.h>

#include "krea2_device.cuh"
#include "krea2_internal.h"
#include "ragged.cuh"

namespace krea2 {

KREA2_DEFINE_ERROR_READER(take_device_error_paged)

namespace {

PagedArgs args_of(const Krea2PagedBatch& b) {
  return PagedArgs{b.R, b.M, b.q_start, b.kv_len, b.page_table, b.max_pages, b.page_size, b.num_pages};
}

__device__ __forceinline__ void report_bad_batch() { atomicOr(&g_device_error, ERR_BAD_BATCH); }

// Requests without a row are seen by no row's thread: block 0 looks at every request's lengths.
__device__ __forceinline__ void check_requests(const PagedArgs& p) {
  if (blockIdx.x) return;
  RequestRows q;
  for (int r = threadIdx.x; r < p.R; r += blockDim.x)
    if (!request_rows(r, p.M, (long long)p.max_pages * p.page_size, p.q_start, p.kv_len, &q)) report_bad_batch();
}

template <typename T>
__device__ __forceinline__ float to_f(T x) {
  if constexpr (sizeof(T) == 2) return __bfloat162float(x);
  else return x;
}
template <typename T>
__device__ __forceinline__ T from_f(float x) {
  if constexpr (sizeof(T) == 2) return __float2bfloat16_rn(x);
  else return x;
}

// NE consecutive elements as fp32 (16-byte loads; p is 16-byte aligned for NE * sizeof(T) >= 16).
template <int NE, typename T>
__device__ __forceinline__ void load_f(const T* p, float* v) {
  constexpr int PER = 16 / sizeof(T);
#pragma unroll
  for (int c = 0; c < NE / PER; ++c) {
    const uint4 u = *reinterpret_cast<const uint4*>(p + c * PER);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if constexpr (sizeof(T) == 2) {
        v[c * PER + 2 * e] = bf16_lo(w[e]);
        v[c * PER + 2 * e + 1] = bf16_hi(w[e]);
      } else {
        v[c * PER + e] = __uint_as_float(w[e]);
      }
    }
  }
}

template <typename T, int E>
struct alignas(sizeof(T) * E) Pack {
  T v[E];
};

// One warp per (row, four KV heads), bound by its bytes: k and v of the four heads are on their way (8 or 16 bytes a
// lane) while the row's request and page are looked up. Each lane holds D / 32 columns (whole rotation pairs).
// 8192 tokens of 12 heads: 20.6 us, 5.1 TB/s (78 % of a copy's rate); with one head a warp it took 38.9 us.
constexpr int APPEND_HEADS = 4;
template <typename T, int D>
__global__ void __launch_bounds__(256) paged_append_kernel(PagedArgs p, const T* __restrict__ qkvg, int H, int Hkv,
                                                           float eps, const float* __restrict__ kw,
                                                           const float* __restrict__ cs, const float* __restrict__ sn,
                                                           T* __restrict__ kp, T* __restrict__ vp) {
  check_requests(p);
  constexpr int E = D / 32;
  using V = Pack<T, E>;
  using F = Pack<float, E>;
  using F2 = Pack<float, E / 2>;
  const int parts = (Hkv + APPEND_HEADS - 1) / APPEND_HEADS;
  const long gw = (long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int row = (int)(gw / parts), h0 = (int)(gw % parts) * APPEND_HEADS;
  // rows behind the last request are not read; a bad end is caught by the look-up below
  if (row >= p.M || row >= __ldg(p.q_start + p.R)) return;
  const T* x = qkvg + (long)row * (2L * (H + Hkv) * D);
  V kr[APPEND_HEADS], vr[APPEND_HEADS];
#pragma unroll
  for (int i = 0; i < APPEND_HEADS; ++i) {
    const int hh = min(h0 + i, Hkv - 1);
    kr[i] = *reinterpret_cast<const V*>(x + (long)(H + hh) * D + lane * E);
    vr[i] = *reinterpret_cast<const V*>(x + (long)(H + Hkv + hh) * D + lane * E);
  }
  const F w = *reinterpret_cast<const F*>(kw + lane * E);
  const F2 c = *reinterpret_cast<const F2*>(cs + (long)row * (D / 2) + lane * (E / 2));
  const F2 sv = *reinterpret_cast<const F2*>(sn + (long)row * (D / 2) + lane * (E / 2));
  RequestRows q;
  bool bad;
  const int r = checked_request_of_row(p, row, &q, &bad);
  if (r < 0) return;  // a request that check_requests reports
  const int t = q.L - q.n + (row - q.row0);
  const int page = p.page_table[(long)r * p.max_pages + t / p.page_size];
  if (page < 0 || page >= p.num_pages) {
    report_bad_batch();
    return;
  }
  const long d = ((long)page * p.page_size + t % p.page_size) * (long)(Hkv * D) + lane * E;
#pragma unroll
  for (int i = 0; i < APPEND_HEADS; ++i) {
    float v[E], ss = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      v[e] = to_f(kr[i].v[e]);
      ss += v[e] * v[e];
    }
    const float rs = rsqrtf(warp_sum(ss) / (float)D + eps);
    V o;
#pragma unroll
    for (int e = 0; e < E; e += 2) {
      // the grouping and the fused products of the contiguous cache's append, so that both give the same bits
      const float x0 = v[e] * (rs * (1.f + w.v[e])), x1 = v[e + 1] * (rs * (1.f + w.v[e + 1]));
      o.v[e] = from_f<T>(__fmaf_rn(x0, c.v[e / 2], -__fmul_rn(x1, sv.v[e / 2])));
      o.v[e + 1] = from_f<T>(__fmaf_rn(x0, sv.v[e / 2], __fmul_rn(x1, c.v[e / 2])));
    }
    if (h0 + i < Hkv) {
      *reinterpret_cast<V*>(kp + d + (long)(h0 + i) * D) = o;
      *reinterpret_cast<V*>(vp + d + (long)(h0 + i) * D) = vr[i];
    }
  }
}

// One block per (row, head). Eight lanes share a key (D / 8 dims each), so the 32 eight-lane groups
// of the block take 32 keys at a time; every group keeps its own running maximum, sum and output
// over its keys, and the groups are joined at the end. No block shares K and V with another, so the time goes by
// rows x heads x keys, 4 to 7 TFLOP/s: 512 tokens over 1024 keys take 3.1 ms in fp32 (48 q / 12 kv heads x 128), 1.0 ms
// in bf16 with 32 / 8 heads x 64, 0.68 ms with 18 / 6 heads x 128; eight single tokens over 2048 keys in fp32 121 us.
template <typename T, int D>
__global__ void __launch_bounds__(256) paged_attn_simt_kernel(PagedArgs p, PagedAttnArgs a) {
  check_requests(p);
  constexpr int E = D / 8;
  __shared__ float part[32][D + 2];
  const int h = blockIdx.x % a.H, row = blockIdx.x / a.H;
  const int tid = threadIdx.x, group = tid >> 3, sub = tid & 7;
  RequestRows rq;
  bool bad;
  const int r = checked_request_of_row(p, row, &rq, &bad);
  if (r < 0) return;  // block-uniform
  const int Hkv = a.Hkv, j = h / (a.H / Hkv);
  const T* x = reinterpret_cast<const T*>(a.qkvg) + (long)row * (2L * (a.H + Hkv) * D);
  float q[E], o[E];
  load_f<E>(x + (long)h * D + sub * E, q);
  float ss = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) ss += q[e] * q[e];
#pragma unroll
  for (int m = 4; m > 0; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
  const float rs = rsqrtf(ss / (float)D + a.eps) * a.scale_log2;  // scores in powers of two
#pragma unroll
  for (int e = 0; e < E; e += 2) {
    const int d = sub * E + e;
    const float c = a.cos[(long)row * (D / 2) + d / 2], s = a.sin[(long)row * (D / 2) + d / 2];
    const float x0 = q[e] * rs * (1.f + a.q_norm_w[d]), x1 = q[e + 1] * rs * (1.f + a.q_norm_w[d + 1]);
    q[e] = x0 * c - x1 * s;
    q[e + 1] = x1 * c + x0 * s;
    o[e] = o[e + 1] = 0.f;
  }
  int end = rq.L;
  if (a.key_end) end = min(max(a.key_end[row], rq.L - rq.n + (row - rq.row0) + 1), rq.L);
  const uint8_t* mask = a.text_mask ? a.text_mask + (long)r * a.T : nullptr;
  const T* kp = reinterpret_cast<const T*>(a.k_pages) + (long)j * D + sub * E;
  const T* vp = reinterpret_cast<const T*>(a.v_pages) + (long)j * D + sub * E;
  float m = -INFINITY, l = 0.f;
  for (int t0 = 0; t0 < end; t0 += 32) {
    const int t = t0 + group;
    bool use = t < end && !(mask && t < a.T && !mask[t]);
    long off = 0;
    if (use) {
      const int page = p.page_table[(long)r * p.max_pages + t / p.page_size];
      if (page < 0 || page >= p.num_pages) {
        if (sub == 0) report_bad_batch();
        use = false;
      } else {
        off = ((long)page * p.page_size + t % p.page_size) * (long)(Hkv * D);
      }
    }
    float dot = 0.f;
    if (use) {
      float k[E];
      load_f<E>(kp + off, k);
#pragma unroll
      for (int e = 0; e < E; ++e) dot += q[e] * k[e];
    }
#pragma unroll
    for (int s = 4; s > 0; s >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, s);
    if (use) {
      float v[E];
      load_f<E>(vp + off, v);
      const float mn = fmaxf(m, dot);
      const float alpha = m == -INFINITY ? 0.f : exp2f(m - mn);
      const float w = dot == -INFINITY ? 0.f : exp2f(dot - (mn == -INFINITY ? 0.f : mn));  // a NaN score stays NaN
      l = l * alpha + w;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = o[e] * alpha + w * v[e];
      m = mn;
    }
  }
#pragma unroll
  for (int e = 0; e < E; ++e) part[group][sub * E + e] = o[e];
  if (sub == 0) {
    part[group][D] = m;
    part[group][D + 1] = l;
  }
  __syncthreads();
  if (tid >= D) return;
  float top = -INFINITY;
  for (int g = 0; g < 32; ++g) top = fmaxf(top, part[g][D]);
  float acc = 0.f, sum = 0.f;
  for (int g = 0; g < 32; ++g) {
    const float w = part[g][D] == -INFINITY ? 0.f : exp2f(part[g][D] - top);
    acc += w * part[g][tid];
    sum += w * part[g][D + 1];
  }
  const float gate = to_f(x[(long)(a.H + 2 * Hkv) * D + (long)h * D + tid]);
  const float res = sum > 0.f ? acc / sum : (sum == 0.f ? 0.f : sum);  // no readable key: zeros; NaN stays
  reinterpret_cast<T*>(a.out)[(long)row * (a.H * D) + (long)h * D + tid] = from_f<T>(res / (1.f + expf(-gate)));
}

int check_launch(const char* what) {
  count_launch();
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return set_error(KREA2_ERR_CUDA, "%s launch failed: %s", what, cudaGetErrorString(e));
  return KREA2_OK;
}

}  // namespace

int launch_paged_append(const Krea2PagedBatch& b, const Krea2Dims* d, bool bf16, const void* qkvg, const float* kw,
                        const float* cs, const float* sn, cudaStream_t stream) {
  const PagedArgs p = args_of(b);
  const long warps = (long)b.M * ((d->Hkv + APPEND_HEADS - 1) / APPEND_HEADS);
  if ((warps + 7) / 8 > 0x7fffffffL) return set_error(KREA2_ERR_UNSUPPORTED, "too many rows x KV heads");
  const unsigned grid = (unsigned)((warps + 7) / 8);
#define KREA2_APPEND(T, DD)                                                                                      \
  paged_append_kernel<T, DD><<<grid, 256, 0, stream>>>(p, reinterpret_cast<const T*>(qkvg), d->H, d->Hkv, d->eps, \
                                                       kw, cs, sn, reinterpret_cast<T*>(b.k_pages),              \
                                                       reinterpret_cast<T*>(b.v_pages))
  if (bf16 && d->D == 128) KREA2_APPEND(__nv_bfloat16, 128);
  else if (bf16) KREA2_APPEND(__nv_bfloat16, 64);
  else if (d->D == 128) KREA2_APPEND(float, 128);
  else KREA2_APPEND(float, 64);
#undef KREA2_APPEND
  return check_launch("paged_kv_append");
}

int launch_paged_attn_simt(const Krea2PagedBatch& b, const PagedAttnArgs& a, int D, bool bf16, cudaStream_t stream) {
  const PagedArgs p = args_of(b);
  const long blocks = (long)b.M * a.H;
  if (blocks > 0x7fffffffL) return set_error(KREA2_ERR_UNSUPPORTED, "too many rows x heads (%ld)", blocks);
  if (bf16 && D == 128) paged_attn_simt_kernel<__nv_bfloat16, 128><<<(unsigned)blocks, 256, 0, stream>>>(p, a);
  else if (bf16) paged_attn_simt_kernel<__nv_bfloat16, 64><<<(unsigned)blocks, 256, 0, stream>>>(p, a);
  else if (D == 128) paged_attn_simt_kernel<float, 128><<<(unsigned)blocks, 256, 0, stream>>>(p, a);
  else paged_attn_simt_kernel<float, 64><<<(unsigned)blocks, 256, 0, stream>>>(p, a);
  return check_launch("paged_attention");
}

}  // namespace krea2
