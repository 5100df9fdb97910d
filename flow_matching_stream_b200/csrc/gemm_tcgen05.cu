// Dense bf16 projections of the Krea 2 block on the sm_100a tensor cores (tcgen05 + TMEM),
// fed by TMA: out = A · Wᵀ with A (M, K) and W (N, K) both K-major (row-major, K contiguous).
//
// Used for the block's four linears (page "Diffusers 中的 Krea2Transformer2DModel … 架构全解",
// §四.2 block and §四.3 attention): the fused [to_q | to_k | to_v | to_gate] projection, to_out
// with the gated residual, the SwiGLU gate/up projection with silu(gate)*up, and the down
// projection with the second gated residual.
//
// Design (one CTA per SM, persistent over output tiles):
//   warp 0      TMA producer: A tile 128x64 and W tile BNx64 per stage, 128-byte swizzle,
//               STAGES-deep ring guarded by full/empty mbarriers, into this CTA's own shared memory.
//   warp 1      allocates TMEM (2 accumulators x BN fp32 columns) and issues tcgen05.mma
//               (M=128, N=BN, K=16) from one thread; tcgen05.commit frees smem stages and
//               signals a finished accumulator.
//   warps 2..5  epilogue: each thread owns one accumulator row (TMEM lane), reads 32 columns
//               at a time with tcgen05.ld and applies the fused epilogue, while the MMA warp
//               already accumulates the next tile into the other TMEM buffer. The bf16
//               epilogues (plain, SwiGLU, q/k/v/gate) write each warp's 32 rows into swizzled
//               shared-memory boxes that TMA stores; the fp32 residual and the row-mapped
//               output pass through a padded shared tile so that global accesses run in whole
//               128-byte row segments.
// With low-rank adapters (LORA) a tile's K steps go on past K: for each request with an adapter among
// the tile's rows, steps whose A operand is the request's low-rank product t (rows of other requests
// are zero) and whose W operand is the adapter's up matrix, into the same accumulator. lora_tc.cu
// says how t is laid out. The row count is then read on the device.
// Tiles are visited in raster groups of row tiles, sized so that one wave of tiles reads about
// as many A bytes as W bytes per K step and so that concurrently running CTAs share A and W
// tiles through L2.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <cmath>
#include <cstring>

#include "krea2_device.cuh"
#include "krea2_internal.h"
#include "lora.cuh"
#include "ragged.cuh"

namespace krea2 {

namespace {

constexpr int BM = 128;
constexpr int BK = 64;
// Row tiles per raster group (group_rows below): at least as many as keep the group's A tiles
// (128 x K bf16 each) within about 24 MB of L2, so W streams from HBM once per group pass, and
// at least as many as make one wave of tiles read about as many A bytes as W bytes per K step.
constexpr size_t GROUP_A_BYTES = 24ull << 20;
// Epilogue warps: 8 for the residual (two per TMEM lane quarter, each on half the tile's
// columns), 4 for the others. The residual's read-modify-write of h is bound by the loads in
// flight; with 4 warps it took longer per tile than to_out's mainloop (K = 6144).
template <int EPI>
constexpr int epi_warps() { return EPI == EPI_RESID ? 8 : 4; }
template <int EPI>
constexpr int gemm_threads() { return 64 + 32 * epi_warps<EPI>(); }

template <int BN>
struct GemmCfg {
  static constexpr int A_BYTES = BM * BK * 2;   // 16 KB
  static constexpr int B_BYTES = BN * BK * 2;   // 32 KB (BN=256) or 16 KB (BN=128)
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int STAGES = (BN == 256) ? 4 : (BN == 128) ? 6 : 8;
  // Epilogue staging per warp: two 4 KB swizzled 32x64 bf16 boxes (TMA-store epilogues), or one
  // padded 32x33 fp32 tile (residual and row-mapped epilogues), at 8 KB spacing.
  static constexpr int EPI_WARP_BYTES = 8192;
  static constexpr int EPI_BYTES = 4 * EPI_WARP_BYTES;
  static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + EPI_BYTES + 1024;  // + alignment slack
  static constexpr int TMEM_COLS = 2 * BN;                         // double-buffered fp32
  static constexpr uint32_t IDESC = idesc_bf16_f32(BM, BN);
};

struct TileMap {
  int tiles_m, tiles_n, group_m;
  __device__ __forceinline__ void map(int t, int& mt, int& nt) const {
    int per_group = group_m * tiles_n;
    int g = t / per_group;
    int first_m = g * group_m;
    int gsize = min(tiles_m - first_m, group_m);
    int local = t - g * per_group;
    mt = first_m + local % gsize;
    nt = local / gsize;
  }
};

// The bf16 epilogues hand each warp's 32 rows to the TMA unit through boxes in shared memory:
// 32 rows x 128 bytes (64 bf16 columns), 128-byte swizzle, so 16-byte chunk j of box
// row r sits at position j ^ (r & 7) and a warp's row-wise 16-byte stores spread over all banks.
// Rows and columns outside the output are clipped by the tensor map. Each warp owns two boxes
// and alternates between them; a box is rewritten only once the TMA operation issued from it two
// boxes earlier has finished reading it.
struct EpiBoxes {
  uint8_t* smem;
  int n;
  __device__ __forceinline__ uint8_t* next(int lane) {
    uint8_t* b = smem + (n++ & 1) * 4096;
    if (lane == 0) bulk_wait_group_read<1>();
    __syncwarp();
    return b;
  }
};

__device__ __forceinline__ void box_put16(uint8_t* box, int lane, int j, uint4 v) {
  *reinterpret_cast<uint4*>(box + lane * 128 + ((j ^ (lane & 7)) << 4)) = v;
}

// Thread `lane` holds row `lane` of a 32 x 64 bf16 block as 32 packed pairs; the warp stores the
// block at output column x, row y (issue = false skips a block wholly past the last row).
__device__ __forceinline__ void store_box_bf16(uint8_t* box, const uint32_t* pk, int lane, const CUtensorMap* tm,
                                               int x, int y, bool issue) {
#pragma unroll
  for (int j = 0; j < 8; ++j) box_put16(box, lane, j, make_uint4(pk[4 * j], pk[4 * j + 1], pk[4 * j + 2], pk[4 * j + 3]));
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0 && issue) {
    tma_store_2d(tm, box, x, y);
    bulk_commit_group();
  }
}

// A row of a 32 x 64 bf16 block straight to global memory (the block that the last request's last row
// cuts: a TMA store would write the rows behind it too).
__device__ __forceinline__ void store_row_bf16(__nv_bfloat16* dst, const uint32_t* pk) {
  uint4* o = reinterpret_cast<uint4*>(dst);
#pragma unroll
  for (int j = 0; j < 8; ++j) o[j] = make_uint4(pk[4 * j], pk[4 * j + 1], pk[4 * j + 2], pk[4 * j + 3]);
}

// What the adapters' K steps need; tmT: t (units * 128 rows, 2 rankp), tmU: up (n_adapters, N, rank).
struct LoraTail {
  const CUtensorMap* tmT;
  const CUtensorMap* tmU;
  Krea2Lora l;
  int rankp;
  // A stage holds kch K steps (64 columns each): A's chunks a_pitch bytes apart, then W's.
  int kch, a_pitch, stage_bytes, stages;
};
constexpr int MAX_STAGES = 8;

// LORA: the adapters' K steps follow those of K. WIDE (with LORA, one row tile): stages of several K steps.
template <int BN, int EPI, bool LORA, bool WIDE>
__device__ __forceinline__ void gemm_body(const CUtensorMap& tmA, const CUtensorMap& tmB, const CUtensorMap& tmC,
                                          const GemmParams& p, const LoraTail& lt) {
  using Cfg = GemmCfg<BN>;
  const int STAGES = WIDE ? lt.stages : Cfg::STAGES;
  const int stage_bytes = WIDE ? lt.stage_bytes : Cfg::STAGE_BYTES;
  const int kch = WIDE ? lt.kch : 1;
  const int w_off = WIDE ? lt.kch * lt.a_pitch : Cfg::A_BYTES;  // W's part of a stage

  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full_bar[WIDE ? MAX_STAGES : Cfg::STAGES];
  __shared__ __align__(8) uint64_t empty_bar[WIDE ? MAX_STAGES : Cfg::STAGES];
  __shared__ __align__(8) uint64_t tfull_bar[2];
  __shared__ __align__(8) uint64_t tempty_bar[2];
  __shared__ __align__(8) uint64_t drain_bar;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  // LORA: whether the tile has a K step after this stage's (from the last step of K on), written by the
  // producer before the stage's full barrier, read by the MMA thread after it
  __shared__ int stage_more[WIDE ? MAX_STAGES : LORA ? Cfg::STAGES : 1];

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t base_u32 = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* base = smem_raw + (base_u32 - smem_u32(smem_raw));

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull_bar[a], 1);
      mbar_init(&tempty_bar[a], 32 * epi_warps<EPI>());
    }
    mbar_init(&drain_bar, 1);
    abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
  }
  if (warp == 1) tmem_alloc(&tmem_slot, Cfg::TMEM_COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = tmem_slot;
  volatile int* abort = &abort_flag;

  int M = p.M, tiles_m = p.tiles_m;
  if constexpr (LORA) {
    M = used_rows(lt.l, p.M);
    tiles_m = (M + BM - 1) / BM;
  }
  const TileMap tm{tiles_m, p.tiles_n, p.group_m};
  const int total = tiles_m * p.tiles_n;
  const int nk = (p.K / BK + kch - 1) / kch;  // stages of a tile (chunks past K read as zeros)

  if (warp == 0) {
    if (lane == 0) {
      uint32_t stage = 0, phase = 0;
      IssuedFills fills;
      for (int t = blockIdx.x; t < total; t += gridDim.x) {
        int mt, nt;
        tm.map(t, mt, nt);
        LoraUnit unit;
        for (int kb = 0; kb < nk; ++kb) {
          if (!mbar_wait(&empty_bar[stage], phase ^ 1, abort)) goto producer_done;
          uint8_t* sa = base + stage * stage_bytes;
          if (LORA && kb == nk - 1) {
            unit = first_unit(lt.l, M, mt);
            stage_more[stage] = unit.exists();
          }
          mbar_arrive_expect_tx(&full_bar[stage], stage_bytes);
          if constexpr (WIDE) {
            tma_load_4d(sa, &tmA, &full_bar[stage], 0, mt * BM, kb * kch, 0);
            tma_load_4d(sa + w_off, &tmB, &full_bar[stage], 0, nt * BN, kb * kch, 0);
          } else {
            tma_load_2d(sa, &tmA, &full_bar[stage], kb * BK, mt * BM);
            tma_load_2d(sa + Cfg::A_BYTES, &tmB, &full_bar[stage], kb * BK, nt * BN);
          }
          fills.note(stage, phase);
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1;
          }
        }
        if constexpr (LORA) {
          const int chunks = lora_chunks(lt.rankp), up_chunks = (lt.rankp + 63) / 64;
          if (unit.exists()) lora_wait_prior_grid();  // t is written by the grid before this one
          while (unit.exists()) {
            const LoraUnit next = next_unit(lt.l, M, mt, unit);
            for (int c = 0; c < chunks; ++c) {
              if (!mbar_wait(&empty_bar[stage], phase ^ 1, abort)) goto producer_done;
              uint8_t* sa = base + stage * stage_bytes;
              stage_more[stage] = c < chunks - 1 || next.exists();
              mbar_arrive_expect_tx(&full_bar[stage], (WIDE ? lt.a_pitch : Cfg::A_BYTES) + Cfg::B_BYTES);
              tma_load_2d(sa, lt.tmT, &full_bar[stage], c * 64, (mt + unit.r) * BM);
              tma_load_3d(sa + w_off, lt.tmU, &full_bar[stage], (c % up_chunks) * 64, nt * BN, unit.adapter);
              fills.note(stage, phase);
              if (++stage == STAGES) {
                stage = 0;
                phase ^= 1;
              }
            }
            unit = next;
          }
        }
      }
    producer_done:
      // a wait expired somewhere: let the copies this thread issued land before the CTA exits
      if (*abort) fills.drain(full_bar, STAGES);
      // no CTA ends before the grid that writes t has, so the next launch in the stream follows both
      if constexpr (LORA) lora_wait_prior_grid();
    }
  } else if (warp == 1) {
    // LORA: the whole warp runs along, so that descriptors and counters are warp-uniform (they live in uniform registers,
    // where the MMA takes them from), and one elected lane issues.
    if (LORA || lane == 0) {
      const bool leader = LORA ? elect_one() : true;
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        return LORA ? warp_wait(bar, parity, abort) : mbar_wait(bar, parity, abort);
      };
      uint32_t stage = 0, phase = 0;
      int local = 0;
      bool issued = false;
      // stage s's A tile starts s * STAGE_BYTES into the ring and its W tile A_BYTES later; a
      // K step of 16 is 32 bytes: only the descriptor's start-address field (16-byte units)
      // changes, so each MMA takes a base descriptor plus a constant
      const uint64_t da0 = smem_desc_sw128(smem_u32(base), 16, 1024);
      for (int t = blockIdx.x; t < total; t += gridDim.x, ++local) {
        const int acc = local & 1;
        const uint32_t acc_phase = (local >> 1) & 1;
        if (!wait(&tempty_bar[acc], acc_phase ^ 1)) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + acc * BN;
        bool ok = true;
        int more = 0;
        for (int kb = 0; kb < nk; ++kb) {
          if (!wait(&full_bar[stage], phase)) {
            ok = false;
            break;
          }
          tc_fence_after();
          uint64_t ad = da0 + (uint64_t)(stage * (stage_bytes >> 4));
          uint64_t bd = ad + (uint64_t)(w_off >> 4);
          if (leader)
#pragma unroll
            for (int k = 0; k < BK / 16; ++k) tc_mma_bf16(d_tmem, ad + 2 * k, bd + 2 * k, Cfg::IDESC, (kb | k) != 0);
          if constexpr (WIDE)
            for (int c = 1; c < kch; ++c) {
              ad += lt.a_pitch >> 4;
              bd += Cfg::B_BYTES >> 4;
              if (leader)
#pragma unroll
                for (int k = 0; k < BK / 16; ++k) tc_mma_bf16(d_tmem, ad + 2 * k, bd + 2 * k, Cfg::IDESC, 1u);
            }
          issued = true;
          if constexpr (LORA) {
            if (kb == nk - 1) {
              more = *(volatile int*)&stage_more[stage];
              __syncwarp();  // all lanes have it before the stage is handed back
            }
          }
          if (leader) tc_commit(&empty_bar[stage]);
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1;
          }
        }
        if constexpr (LORA) {
          // columns of t: [high halves | low halves]; each meets the same columns of up
          const int steps = min(2 * lt.rankp / 16, 4), wrap = min(lt.rankp / 16, 4);
          while (ok && more) {
            if (!wait(&full_bar[stage], phase)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint64_t ad = da0 + (uint64_t)(stage * (stage_bytes >> 4));
            const uint64_t bd = ad + (uint64_t)(w_off >> 4);
            if (leader)
              for (int k = 0; k < steps; ++k)
                tc_mma_bf16(d_tmem, ad + 2 * k, bd + 2 * (k >= wrap ? k - wrap : k), Cfg::IDESC, 1u);
            more = *(volatile int*)&stage_more[stage];
            __syncwarp();
            if (leader) tc_commit(&empty_bar[stage]);
            if (++stage == STAGES) {
              stage = 0;
              phase ^= 1;
            }
          }
        }
        if (!ok) break;
        if (leader) tc_commit(&tfull_bar[acc]);
      }
      if (*abort && issued) {
        // let every MMA already issued finish before TMEM is released
        if (leader) tc_commit(&drain_bar);
        mbar_wait(&drain_bar, 0, &abort_flag /* already set: bounded by the timer below */);
        unsigned long long t0 = globaltimer_ns();
        while (!mbar_try_wait(&drain_bar, 0) && globaltimer_ns() - t0 < WAIT_LIMIT_NS) {
        }
      }
    }
  } else {
    // epilogue warps 2.. -> TMEM lane quarters 2, 3, 0, 1 (2, 3, 0, 1 again for the residual's
    // second four warps, which take the other half of the columns)
    const int quarter = warp & 3;
    const int part = (warp - 2) >> 2;
    EpiBoxes boxes{base + Cfg::STAGES * Cfg::STAGE_BYTES + (warp - 2) * Cfg::EPI_WARP_BYTES, 0};
    int local = 0;
    for (int t = blockIdx.x; t < total; t += gridDim.x, ++local) {
      int mt, nt;
      tm.map(t, mt, nt);
      const int acc = local & 1;
      const uint32_t acc_phase = (local >> 1) & 1;
      if (!mbar_wait(&tfull_bar[acc], acc_phase, abort)) break;
      tc_fence_after();
      const int row = mt * BM + quarter * 32 + lane;
      const bool row_ok = row < M;
      const uint32_t tbase = tmem_base + ((uint32_t)(quarter * 32) << 16) + acc * BN;

      const int row0 = mt * BM + quarter * 32;
      const int nrows = min(32, M - row0);
      uint8_t* epi_smem = base + Cfg::STAGES * Cfg::STAGE_BYTES + (warp - 2) * Cfg::EPI_WARP_BYTES;
      uint32_t* xpk = reinterpret_cast<uint32_t*>(epi_smem);
      const bool rows_in = row0 < M;  // warp-uniform: this 32-row block holds output rows
      const bool cut = LORA && row0 + 32 > M;  // warp-uniform: stored row by row
      if constexpr (EPI == EPI_STORE) {
        const int n_store = p.n_store ? p.n_store : p.N;
#pragma unroll 1
        for (int c = 0; c < BN / 64; ++c) {
          if (nt * BN + c * 64 >= n_store) break;  // warp-uniform: padding columns of W are not stored
          float v[64];
          tmem_ld64(tbase + c * 64, v);
          if (p.bias) {
            const float4* bp = reinterpret_cast<const float4*>(p.bias + (size_t)nt * BN + c * 64);
#pragma unroll
            for (int q = 0; q < 16; ++q) {
              const float4 bv = __ldg(bp + q);
              v[q * 4 + 0] += bv.x;
              v[q * 4 + 1] += bv.y;
              v[q * 4 + 2] += bv.z;
              v[q * 4 + 3] += bv.w;
            }
          }
          uint32_t pk[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) pk[e] = pack_bf16x2(v[2 * e], v[2 * e + 1]);
          if (cut) {
            if (row_ok) store_row_bf16(reinterpret_cast<__nv_bfloat16*>(p.out) + (size_t)row * p.N + nt * BN + c * 64, pk);
          } else {
            store_box_bf16(boxes.next(lane), pk, lane, &tmC, nt * BN + c * 64, row0, rows_in);
          }
        }
      } else if constexpr (EPI == EPI_BIAS_ROWMAP) {
        // fp32 out[map(row), col] = acc + bias[col], rows transposed through shared memory like the
        // residual epilogue below; lane i holds the destination row of tile row row0 + i
        float* xp = reinterpret_cast<float*>(xpk);
        const int rr = min(row0 + lane, M - 1);
        const long long my_dst = (long long)(rr / p.map_N) * p.map_S + p.map_T + rr % p.map_N;
#pragma unroll 1
        for (int c = 0; c < BN / 32; ++c) {
          float v[32];
          tmem_ld32(tbase + c * 32, v);
#pragma unroll
          for (int e = 0; e < 32; ++e) xp[lane * 33 + e] = v[e];
          __syncwarp();
          const int col = nt * BN + c * 32 + lane;
          const float bv = p.bias ? __ldg(p.bias + col) : 0.f;
          float* out = reinterpret_cast<float*>(p.out) + col;
#pragma unroll 8
          for (int i = 0; i < 32; ++i) {
            const long long dst = __shfl_sync(0xffffffffu, my_dst, i);
            if (i < nrows) out[dst * p.N] = xp[i * 33 + lane] + bv;
          }
          __syncwarp();
        }
      } else if constexpr (EPI == EPI_SWIGLU) {
        // interleaved 64-row groups: columns [128g, 128g+64) gate, [128g+64, 128g+128) up; each
        // group gives 64 output columns
#pragma unroll 1
        for (int g = 0; g < BN / 128; ++g) {
          uint32_t pk[32];
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            float gv[32], uv[32];
            tmem_ld32(tbase + g * 128 + half * 32, gv);
            tmem_ld32(tbase + g * 128 + 64 + half * 32, uv);
#pragma unroll
            for (int e = 0; e < 16; ++e)
              pk[half * 16 + e] = pack_bf16x2(silu_f(gv[2 * e]) * uv[2 * e], silu_f(gv[2 * e + 1]) * uv[2 * e + 1]);
          }
          if (cut) {
            if (row_ok)
              store_row_bf16(reinterpret_cast<__nv_bfloat16*>(p.out) + (size_t)row * (p.N / 2) + nt * (BN / 2) + g * 64, pk);
          } else {
            store_box_bf16(boxes.next(lane), pk, lane, &tmC, nt * (BN / 2) + g * 64, row0, rows_in);
          }
        }
      } else if constexpr (EPI == EPI_QKV) {
        // [q | k | v | gate] columns; 128-wide q/k heads get RMSNorm (1 + w) and RoPE here,
        // once per element, on the fp32 accumulator (page §四.3 order: norm, then RoPE)
        const int pos = row_ok ? row % p.rows_per_batch : 0;
        const float* cs = p.cos + (size_t)pos * 64;
        const float* sn = p.sin + (size_t)pos * 64;
#pragma unroll 1
        for (int u = 0; u < BN / 128; ++u) {
          const int c0 = nt * BN + u * 128;
          const bool is_q = c0 < p.HD;
          const bool is_k = !is_q && c0 < p.HD + p.KVD;
          const uint32_t ub = tbase + u * 128;
          float r = 1.f;
          if (is_q || is_k) {  // pass 1: sum of squares over the head's 128 columns
            float s4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
            for (int h2 = 0; h2 < 2; ++h2) {
              float v[64];
              tmem_ld64(ub + h2 * 64, v);
#pragma unroll
              for (int e = 0; e < 64; ++e) s4[e & 3] += v[e] * v[e];
            }
            r = rsqrtf(((s4[0] + s4[1]) + (s4[2] + s4[3])) * (1.f / 128.f) + p.eps);
          }
          const float4* w4 = reinterpret_cast<const float4*>(is_q ? p.qw : p.kw);
#pragma unroll 1
          for (int h2 = 0; h2 < 2; ++h2) {  // pass 2: normalise, rotate, store 64 columns at a time
            float v[64];
            tmem_ld64(ub + h2 * 64, v);
            if (is_q || is_k) {
              const float4* c4 = reinterpret_cast<const float4*>(cs + h2 * 32);
              const float4* s4p = reinterpret_cast<const float4*>(sn + h2 * 32);
#pragma unroll
              for (int q = 0; q < 8; ++q) {  // 8 dims (4 rotated pairs) per step
                const float4 wa = __ldg(w4 + h2 * 16 + 2 * q), wb = __ldg(w4 + h2 * 16 + 2 * q + 1);
                const float4 co = __ldg(c4 + q), si = __ldg(s4p + q);
                const float wv[8] = {wa.x, wa.y, wa.z, wa.w, wb.x, wb.y, wb.z, wb.w};
                const float cv[4] = {co.x, co.y, co.z, co.w}, sv[4] = {si.x, si.y, si.z, si.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const int d = q * 8 + 2 * e;
                  const float x0 = v[d] * r * (1.f + wv[2 * e]);
                  const float x1 = v[d + 1] * r * (1.f + wv[2 * e + 1]);
                  v[d] = x0 * cv[e] - x1 * sv[e];
                  v[d + 1] = x1 * cv[e] + x0 * sv[e];
                }
              }
            }
            uint32_t pk[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) pk[e] = pack_bf16x2(v[2 * e], v[2 * e + 1]);
            store_box_bf16(boxes.next(lane), pk, lane, &tmC, nt * BN + u * 128 + h2 * 64, row0, rows_in);
          }
        }
      } else {  // EPI_RESID: h[row, col] += gate[b, col] * acc
        // A plain read-modify-write of h through L1/L2, not a TMA reduce-add: h is also written
        // by plain stores (img_in, the text rows, the caller), and in one launch sequence a TMA
        // reduce-add of this epilogue returned the value h held before the img_in kernel, several
        // launches earlier in the same stream. After tcgen05.ld each thread holds one row of a
        // 32-column chunk; row-by-row global accesses would touch 32 cache lines per warp access,
        // so the warp transposes its 32x32 block through shared memory (XOR-swizzled: element
        // (row i, column e) at i * 32 + (e ^ i), conflict-free both ways) and walks the rows: each
        // access is one 128-byte line, and 16 rows of loads are in flight before any store. Warp
        // part 0 takes the tile's first BN / 2 columns, part 1 the rest.
        // Lane i knows the batch row of tile row row0 + i (clamped to M - 1, so that rows of the
        // ragged last tile read an in-bounds gate; their results are never stored).
        float* xp = reinterpret_cast<float*>(base + Cfg::STAGES * Cfg::STAGE_BYTES) + (warp - 2) * (32 * 32);
        const int my_row = min(row0 + lane, M - 1);
        int my_b;
        if (LORA && p.rows_per_batch == 0) my_b = request_of_row(lt.l.row_start, lt.l.R, my_row);
        else my_b = my_row / p.rows_per_batch;
#pragma unroll 1
        for (int c = part * (BN / 64); c < (part + 1) * (BN / 64); ++c) {
          float v[32];
          tmem_ld32(tbase + c * 32, v);
#pragma unroll
          for (int e = 0; e < 32; ++e) xp[lane * 32 + (e ^ lane)] = v[e];
          __syncwarp();
          const int col = nt * BN + c * 32 + lane;
#pragma unroll 1
          for (int i0 = 0; i0 < 32; i0 += 16) {
            float* hp = reinterpret_cast<float*>(p.out) + (size_t)(row0 + i0) * p.N + col;
            float hv[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) hv[i] = i0 + i < nrows ? hp[(size_t)i * p.N] : 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int bb = __shfl_sync(0xffffffffu, my_b, i0 + i);
              hv[i] += __ldg(p.gate + (size_t)bb * p.gate_stride + col) * xp[(i0 + i) * 32 + (lane ^ (i0 + i))];
            }
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (i0 + i < nrows) hp[(size_t)i * p.N] = hv[i];
          }
          __syncwarp();
        }
      }
      tc_fence_before();
      mbar_arrive(&tempty_bar[acc]);
    }
    // the TMA stores must be complete (their boxes read, the output written) before
    // this CTA's shared memory goes away
    if (lane == 0) bulk_wait_all();
  }

  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, Cfg::TMEM_COLS);
  }
}

template <int BN, int EPI>
__global__ void __launch_bounds__(gemm_threads<EPI>(), 1)
    gemm_bf16_tcgen05_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                             const __grid_constant__ CUtensorMap tmC, GemmParams p) {
  gemm_body<BN, EPI, false, false>(tmA, tmB, tmC, p, LoraTail{});
}

template <int BN, int EPI, bool WIDE>
__global__ void __launch_bounds__(gemm_threads<EPI>(), 1)
    gemm_lora_tcgen05_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                             const __grid_constant__ CUtensorMap tmC, const __grid_constant__ CUtensorMap tmT,
                             const __grid_constant__ CUtensorMap tmU, GemmParams p, LoraTail lt) {
  lt.tmT = &tmT;
  lt.tmU = &tmU;
  gemm_body<BN, EPI, true, WIDE>(tmA, tmB, tmC, p, lt);
}

}  // namespace

PFN_cuTensorMapEncodeTiled_v12000 tmap_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  if (!fn) {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  }
  return fn;
}

// Row-major bf16 matrix (rows, cols) as a 2-D TMA map with a (box_cols x box_rows) box and
// 128-byte swizzle (box_cols * 2 bytes must be 128).
int make_tmap_bf16_2d(CUtensorMap* m, const void* ptr, uint64_t cols, uint64_t rows, uint64_t row_stride_elems,
                      uint32_t box_cols, uint32_t box_rows) {
  auto enc = tmap_encoder();
  if (!enc) return set_error(KREA2_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
  if ((reinterpret_cast<uintptr_t>(ptr) & 15) || ((row_stride_elems * 2) & 15))
    return set_error(KREA2_ERR_ARG, "TMA operand must be 16-byte aligned with a 16-byte multiple row stride");
  cuuint64_t dims[2] = {cols, rows};
  cuuint64_t strides[1] = {row_stride_elems * 2};
  cuuint32_t box[2] = {box_cols, box_rows};
  cuuint32_t es[2] = {1, 1};
  CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(ptr), dims, strides, box, es,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return set_error(KREA2_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
  return KREA2_OK;
}

// Row-major bf16 matrices (batches, rows, cols), cols a multiple of 64, viewed as (batches, chunks of 64 columns,
// rows, 64): a box is box_chunks K-major operand tiles of box_rows x 64, one behind the other in shared memory.
// Chunks and rows past the matrix read as zeros.
int make_tmap_bf16_chunks(CUtensorMap* m, const void* ptr, uint64_t cols, uint64_t rows, uint64_t batches,
                          uint32_t box_rows, uint32_t box_chunks) {
  auto enc = tmap_encoder();
  if (!enc) return set_error(KREA2_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
  if (reinterpret_cast<uintptr_t>(ptr) & 15) return set_error(KREA2_ERR_ARG, "TMA operand must be 16-byte aligned");
  cuuint64_t dims[4] = {64, rows, cols / 64, batches};
  cuuint64_t strides[3] = {cols * 2, 128, rows * cols * 2};
  cuuint32_t box[4] = {64, box_rows, box_chunks, 1};
  cuuint32_t es[4] = {1, 1, 1, 1};
  CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(ptr), dims, strides, box, es,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return set_error(KREA2_ERR_CUDA, "cuTensorMapEncodeTiled (chunks) failed (%d)", (int)r);
  return KREA2_OK;
}

// Row-major bf16 matrix viewed as (batches, rows, cols) with `row_stride_elems` between rows and
// rows*row_stride between batches; box (box_cols x box_rows x 1), 128-byte swizzle. Rows past
// `rows` in a batch read as zero.
// (cols, rows, batches) view with batch b starting batch_rows rows after batch b-1 (batch_rows >=
// rows); rows at or beyond `rows` read as zeros, also when the buffer holds more.
int make_tmap_bf16_3d(CUtensorMap* m, const void* ptr, uint64_t cols, uint64_t rows, uint64_t batches,
                      uint64_t row_stride_elems, uint32_t box_cols, uint32_t box_rows, uint64_t batch_rows) {
  auto enc = tmap_encoder();
  if (!enc) return set_error(KREA2_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
  if ((reinterpret_cast<uintptr_t>(ptr) & 15) || ((row_stride_elems * 2) & 15))
    return set_error(KREA2_ERR_ARG, "TMA operand must be 16-byte aligned with a 16-byte multiple row stride");
  cuuint64_t dims[3] = {cols, rows, batches};
  if (batch_rows < rows) return set_error(KREA2_ERR_ARG, "batch stride of %llu rows is below the %llu rows read",
                                          (unsigned long long)batch_rows, (unsigned long long)rows);
  cuuint64_t strides[2] = {row_stride_elems * 2, row_stride_elems * 2 * batch_rows};
  cuuint32_t box[3] = {box_cols, box_rows, 1};
  cuuint32_t es[3] = {1, 1, 1};
  CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(ptr), dims, strides, box, es,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return set_error(KREA2_ERR_CUDA, "cuTensorMapEncodeTiled (3-D) failed (%d)", (int)r);
  return KREA2_OK;
}

namespace {

// Row tiles per raster group. The persistent CTAs run about `sms` consecutive tiles at once: r
// row tiles by c = sms / r column tiles of one group. Per K step that wave reads r*BM rows of A
// and c*BN rows of W, which is least at r = sqrt(sms * BN / BM) (18 for BN = 256 on 148 SMs);
// with much fewer rows, each wave streams nearly all of W from HBM. The row tiles are then split
// into groups of equal size.
int group_rows(int tiles_m, int K, int BN, int sms) {
  const int by_l2 = (int)(GROUP_A_BYTES / ((size_t)BM * K * 2));
  const int by_wave = (int)std::ceil(std::sqrt((double)sms * BN / BM));
  int g = by_l2 > by_wave ? by_l2 : by_wave;
  if (g >= tiles_m) return tiles_m;
  const int groups = (tiles_m + g - 1) / g;
  return (tiles_m + groups - 1) / groups;
}

template <int BN, int EPI>
int launch_gemm_bn(const GemmParams& p0, const void* A, const void* W, cudaStream_t stream) {
  using Cfg = GemmCfg<BN>;
  static std::atomic<uint64_t> attr_done{0};
  auto kern = gemm_bf16_tcgen05_kernel<BN, EPI>;
  const uint64_t dev_bit = device_bit();
  if (!(attr_done.load(std::memory_order_acquire) & dev_bit) || !dev_bit) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::SMEM_BYTES) != cudaSuccess)
      return set_error(KREA2_ERR_CUDA, "cudaFuncSetAttribute(gemm) failed");
    attr_done.fetch_or(dev_bit, std::memory_order_release);
  }
  CUtensorMap ta, tb, tc;
  int rc = make_tmap_bf16_2d(&ta, A, p0.K, p0.M, p0.K, BK, BM);
  if (rc) return rc;
  rc = make_tmap_bf16_2d(&tb, W, p0.K, p0.w_rows ? p0.w_rows : p0.N, p0.K, BK, BN);
  if (rc) return rc;
  GemmParams p = p0;
  // the bf16 epilogues' TMA target: 32-row boxes of 128 bytes (64 bf16 columns)
  memset(&tc, 0, sizeof(tc));
  if constexpr (EPI == EPI_RESID) {
    // plain loads and stores (see the epilogue); the 16-byte rule keeps the API uniform
    if (reinterpret_cast<uintptr_t>(p.out) & 15)
      return set_error(KREA2_ERR_ARG, "residual output must be 16-byte aligned");
  } else if constexpr (EPI == EPI_STORE) {
    if ((rc = make_tmap_bf16_2d(&tc, p.out, p.n_store ? p.n_store : p.N, p.M, p.out_ld ? p.out_ld : p.N, 64, 32)))
      return rc;
  } else if constexpr (EPI == EPI_SWIGLU) {
    if ((rc = make_tmap_bf16_2d(&tc, p.out, p.N / 2, p.M, p.N / 2, 64, 32))) return rc;
  } else if constexpr (EPI == EPI_QKV) {
    if ((rc = make_tmap_bf16_2d(&tc, p.out, p.N, p.M, p.N, 64, 32))) return rc;
  }
  p.tiles_m = (p.M + BM - 1) / BM;
  p.tiles_n = p.N / BN;
  p.group_m = group_rows(p.tiles_m, p.K, BN, num_sms());
  const int total = p.tiles_m * p.tiles_n;
  const int grid = total < num_sms() ? total : num_sms();
  kern<<<grid, gemm_threads<EPI>(), Cfg::SMEM_BYTES, stream>>>(ta, tb, tc, p);
  count_launch();
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return set_error(KREA2_ERR_CUDA, "gemm launch failed: %s", cudaGetErrorString(e));
  return KREA2_OK;
}

// The GEMM with the adapters' K steps, launched as a programmatic dependent of lora_down: its CTAs
// may start once every lora_down CTA runs, and wait for t only when they first load it. A CTA takes nearly all of an
// SM's shared memory, so it starts where lora_down's CTAs have left; with many rows that is near lora_down's end. Bound by the tensor
// cores, under the power cap: gate/up of 5760 rows, rank 16, 1.82 to 1.87 ms by box with t's own kernel (90 to 93 % of
// the sustained matrix rate). The shared projection alone takes 1.74 to 1.81 ms from run to run.
template <int BN, int EPI, bool WIDE>
int launch_gemm_lora_bn(const GemmParams& p0, const void* A, const void* W, const Krea2Lora& l, const void* t,
                        cudaStream_t stream) {
  using Cfg = GemmCfg<BN>;
  static std::atomic<uint64_t> attr_done{0};
  auto kern = gemm_lora_tcgen05_kernel<BN, EPI, WIDE>;
  const uint64_t dev_bit = device_bit();
  if (!(attr_done.load(std::memory_order_acquire) & dev_bit) || !dev_bit) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::SMEM_BYTES) != cudaSuccess)
      return set_error(KREA2_ERR_CUDA, "cudaFuncSetAttribute(gemm with adapters) failed");
    attr_done.fetch_or(dev_bit, std::memory_order_release);
  }
  GemmParams p = p0;
  p.tiles_m = (p.M + BM - 1) / BM;
  p.tiles_n = p.N / BN;
  p.group_m = group_rows(p.tiles_m, p.K, BN, num_sms());
  LoraTail lt{};
  lt.l = l;
  lt.rankp = lora_rankp(l.rank);
  CUtensorMap ta, tb, tc, tt, tu;
  int rc, a_rows = BM;
  if constexpr (WIDE) {
    // Rows past M would be zero-filled; the accumulator rows that other shared memory gives instead are not
    // stored (the MMA reads 128 rows from each chunk on, which ends inside the ring or the epilogue's boxes).
    if (p.M < BM) a_rows = (p.M + 7) / 8 * 8;
    lt.a_pitch = a_rows * BK * 2;
    // One row tile streams W once, and a stage's turn (a wait, a load of A and one of W by one thread) takes
    // about 0.3 us whatever it loads: as many K steps a stage as leave three stages. One row by 6144 x 6144 with an
    // adapter: 30.9 us with one K step a stage (30.8 us for N = 1024 too), 22.9 with two, 21.2 with four. What is
    // left (20.0 us of device time) is about 7.5 us of start, end and two launches, and 2.0 ns a column of K, a CTA's
    // own 64 columns of W at 64 GB/s. That part goes by K, not by N, until the CTAs together reach the memory's rate:
    // N = 1024 (16 CTAs) 18.3 us, N = 6144 (96 CTAs, 6.1 TB/s while they stream) 20.0, and with K of 1536 and 12288
    // 10.4 and 32.0; N = 15360 in 128 columns 34.8. Without an adapter 0.4 us less. A ring holds two steps of 128
    // rows at least.
    const int step = lt.a_pitch + Cfg::B_BYTES, ring = Cfg::STAGES * Cfg::STAGE_BYTES;
    lt.kch = 12 * step <= ring ? 4 : 2;
    lt.stage_bytes = lt.kch * step;
    lt.stages = ring / lt.stage_bytes;
    if (lt.stages > MAX_STAGES) lt.stages = MAX_STAGES;
    if ((rc = make_tmap_bf16_chunks(&ta, A, p.K, p.M, 1, a_rows, lt.kch))) return rc;
    if ((rc = make_tmap_bf16_chunks(&tb, W, p.K, p.N, 1, BN, lt.kch))) return rc;
  } else {
    if ((rc = make_tmap_bf16_2d(&ta, A, p.K, p.M, p.K, BK, BM))) return rc;
    if ((rc = make_tmap_bf16_2d(&tb, W, p.K, p.N, p.K, BK, BN))) return rc;
  }
  if ((rc = make_tmap_bf16_2d(&tt, t, 2 * lt.rankp, (uint64_t)lora_units(p.M, l.R) * BM, 2 * lt.rankp, 64, a_rows)))
    return rc;
  if ((rc = make_tmap_bf16_3d(&tu, l.up, l.rank, p.N, l.n_adapters, l.rank, 64, BN, p.N))) return rc;
  memset(&tc, 0, sizeof(tc));
  const int out_cols = EPI == EPI_SWIGLU ? p.N / 2 : p.N;
  if constexpr (EPI != EPI_RESID)
    if ((rc = make_tmap_bf16_2d(&tc, p.out, out_cols, p.M, out_cols, 64, 32))) return rc;
  const int total = p.tiles_m * p.tiles_n;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(total < num_sms() ? total : num_sms());
  cfg.blockDim = dim3(gemm_threads<EPI>());
  cfg.dynamicSmemBytes = Cfg::SMEM_BYTES;
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, ta, tb, tc, tt, tu, p, lt);
  count_launch();
  if (e != cudaSuccess) return set_error(KREA2_ERR_CUDA, "gemm with adapters launch failed: %s", cudaGetErrorString(e));
  return KREA2_OK;
}

// Wave efficiency of a tile count on the SMs (1.0 = every wave full).
double wave_eff(long tiles, int sms) {
  long waves = (tiles + sms - 1) / sms;
  return (double)tiles / (double)(waves * sms);
}

}  // namespace

KREA2_DEFINE_ERROR_READER(take_device_error_gemm)

int gemm_bf16(int epi, const GemmParams& p, const void* A, const void* W, cudaStream_t stream) {
  // choose the N tile: 256 unless 128 fills the machine clearly better
  const int sms = num_sms();
  const long tm = (p.M + BM - 1) / BM;
  int bn = 128;
  if (p.N % 256 == 0) {
    const double e256 = wave_eff(tm * (p.N / 256), sms);
    const double e128 = wave_eff(tm * (p.N / 128), sms);
    bn = (e256 >= 0.8 * e128 || tm * (p.N / 256) >= 4L * sms) ? 256 : 128;
  }
  if (bn == 256) {
    switch (epi) {
      case EPI_STORE: return launch_gemm_bn<256, EPI_STORE>(p, A, W, stream);
      case EPI_SWIGLU: return launch_gemm_bn<256, EPI_SWIGLU>(p, A, W, stream);
      case EPI_QKV: return launch_gemm_bn<256, EPI_QKV>(p, A, W, stream);
      case EPI_BIAS_ROWMAP: return launch_gemm_bn<256, EPI_BIAS_ROWMAP>(p, A, W, stream);
      default: return launch_gemm_bn<256, EPI_RESID>(p, A, W, stream);
    }
  }
  switch (epi) {
    case EPI_STORE: return launch_gemm_bn<128, EPI_STORE>(p, A, W, stream);
    case EPI_SWIGLU: return launch_gemm_bn<128, EPI_SWIGLU>(p, A, W, stream);
    case EPI_QKV: return launch_gemm_bn<128, EPI_QKV>(p, A, W, stream);
    case EPI_BIAS_ROWMAP: return launch_gemm_bn<128, EPI_BIAS_ROWMAP>(p, A, W, stream);
    default: return launch_gemm_bn<128, EPI_RESID>(p, A, W, stream);
  }
}

int gemm_bf16_lora(int epi, const GemmParams& p, const void* A, const void* W, const Krea2Lora& l, const void* t,
                   cudaStream_t stream) {
  const int sms = num_sms();
  const long tm = (p.M + BM - 1) / BM;
  const double e128 = wave_eff(tm * (p.N / 128), sms);
  if (tm == 1) {
    // few tiles: narrower ones put more SMs on the stream of W (a SwiGLU tile is 128 columns at least). One row
    // by 6144 x 6144: 21.2 us in 64 columns, 24.8 in 128; x 15360, where both fill the SMs: 38.0 and 36.5.
    const bool narrow = wave_eff(p.N / 64, sms) > 1.25 * e128;
    if (epi == EPI_SWIGLU) return launch_gemm_lora_bn<128, EPI_SWIGLU, true>(p, A, W, l, t, stream);
    if (epi == EPI_STORE)
      return narrow ? launch_gemm_lora_bn<64, EPI_STORE, true>(p, A, W, l, t, stream)
                    : launch_gemm_lora_bn<128, EPI_STORE, true>(p, A, W, l, t, stream);
    return narrow ? launch_gemm_lora_bn<64, EPI_RESID, true>(p, A, W, l, t, stream)
                  : launch_gemm_lora_bn<128, EPI_RESID, true>(p, A, W, l, t, stream);
  }
  const long t256 = tm * (p.N / 256);
  if (p.N % 256 == 0 && (wave_eff(t256, sms) >= 0.8 * e128 || t256 >= 4L * sms)) {
    switch (epi) {
      case EPI_STORE: return launch_gemm_lora_bn<256, EPI_STORE, false>(p, A, W, l, t, stream);
      case EPI_SWIGLU: return launch_gemm_lora_bn<256, EPI_SWIGLU, false>(p, A, W, l, t, stream);
      default: return launch_gemm_lora_bn<256, EPI_RESID, false>(p, A, W, l, t, stream);
    }
  }
  switch (epi) {
    case EPI_STORE: return launch_gemm_lora_bn<128, EPI_STORE, false>(p, A, W, l, t, stream);
    case EPI_SWIGLU: return launch_gemm_lora_bn<128, EPI_SWIGLU, false>(p, A, W, l, t, stream);
    default: return launch_gemm_lora_bn<128, EPI_RESID, false>(p, A, W, l, t, stream);
  }
}

}  // namespace krea2
