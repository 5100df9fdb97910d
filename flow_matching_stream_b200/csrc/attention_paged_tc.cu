// Attention of a ragged batch's new tokens over a paged key/value cache on the sm_100a tensor cores:
//   out = sigmoid(g) softmax(q_hat k_hatᵀ / sqrt(D)) v,  q_hat = RoPE(q / rms(q) (1 + w)),
// one pass over the keys with the running maximum and sum of each row's softmax.
//
// Bound: the tensor cores and the exponentials for many new tokens (4 D H operations a token and key),
// reading K and V once (512 bytes a key and KV head) for few. Measured (48 q / 12 kv heads, pages of 64): two
// requests of 4096 new tokens over 8704 keys 1.69 to 1.80 ms by box, 970 to 1040 TFLOP/s under the power cap (71 to
// 75 % of the sustained matrix rate), with tensor pipe, exponentials and issue slots each about half busy (a smaller
// batch: 48, 52 and 53 %); eight single tokens over 521 to 8704 keys 50 to 53 us, 4.3 to 4.6 TB/s, the join 7 of them.
// (These rates count all keys. Tiles that the text mask removes whole are neither loaded nor computed: in these
// batches 3 to 5 % of the keys, up to 7.5 % by the drawn masks.)
//
// Roundings: q_hat and P go to the tensor cores in bf16, as K and V come; maxima, sums and O are fp32. Against fp64
// the output is off by 0.0025 to 0.0029 of its size, where its own rounding to bf16 makes 0.0017. Carrying what those
// roundings leave in further MMAs gave 0.0017 for single tokens and took 13 % longer; a mixed batch went from 0.0025
// to 0.0022 and took 23 % longer, two requests of 4096 new tokens 35 %.
//
// An item is (request, KV head, 256 / G new tokens): two teams with 128 MMA rows each, row = token * G + head,
// so that few tokens fill whole warps and leave the others idle. The teams share the item's K and V tiles in
// shared memory: 1.76 ms where one team per CTA and two CTAs per SM, each with its own K and V, took 1.85 ms.
// Work is cut into key tiles of 64. Every CTA (all resident) takes
//   * whole items in turn, as many rounds as every CTA gets one item of a request: neighbours work on
//     the same K and V at the same time;
//   * an equal share of the key tiles of what is left, cut without regard to items. A cut item's parts
//     (unnormalised O, row maximum and sum, fp32) go to the workspace, and a second kernel joins them in
//     key order. One new token over a long cache is spread over all SMs this way.
// An item weighs all tiles of its request, also where its tokens' key ends drop many of them, so shares of causal
// prompts are unequal: 4096 tokens read from nothing take 315 us where all of them read all keys in 410, four of 1000
// 162 and 176 (half the operations each).
// Batches of about one new token per request have items of one team with 16 rows, two CTAs per SM.
//
// Roles as in attention_tc.cu, but the CTA runs through segments (an item or a part of one):
//   warp 0        cuts the work into segments and publishes them, looks up pages, loads K and V tiles by
//                 TMA, one box per page and tile (per 16, 32 or 64 keys), into a ring
//   one warp per team   S = Q Kᵀ into one of two TMEM buffers, O += P V with P in TMEM
//   eight warps per team   normalise and rotate the team's queries into shared memory, softmax, output. Where
//                 keys of a tile are masked or lie behind the request's last key, they clear those rows of V
//                 in shared memory, so that whatever the page holds there meets no probability of zero.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <type_traits>

#include "attention_device.cuh"
#include "krea2_device.cuh"
#include "krea2_internal.h"
#include "ragged.cuh"

namespace krea2 {

KREA2_DEFINE_ERROR_READER(take_device_error_paged_tc)

namespace {

constexpr int KT = 64;            // keys per tile
constexpr int SOFTMAX_WARPS = 8;  // of a team
constexpr int KV_CHUNK = KT * 128;  // 64 keys x 64 bf16
constexpr int KV_TILE_BYTES = 2 * KV_CHUNK;

// FEW: batches of about one new token per request. With few rows a tile's time is that of its loads, and the room
// of the other queries goes to K and V. (The MMA still reads 128 rows from each chunk of Q on, K's tiles behind the
// 16; those accumulator rows are not used.)
template <int G, bool FEW>
struct Cfg {
  static constexpr int TEAMS = FEW ? 1 : 2;
  static constexpr int ROWS = FEW ? 16 : 128;   // query rows of a team
  static constexpr int QPOS = TEAMS * ROWS / G;  // tokens of an item
  static constexpr int STAGES = FEW ? 3 : 5;
  static constexpr int CTAS_PER_SM = FEW ? 2 : 1;
  static constexpr int FIRST_SOFTMAX = 1 + TEAMS;  // warp number
  static constexpr int THREADS = 32 * (1 + TEAMS + 8 * TEAMS);
  static constexpr int Q_CHUNK = ROWS * 128;    // ROWS x 64 bf16
  static constexpr int OFF_K = TEAMS * 2 * Q_CHUNK;
  static constexpr int OFF_V = OFF_K + STAGES * KV_TILE_BYTES;
  static constexpr int SMEM_BYTES = OFF_V + STAGES * KV_TILE_BYTES + 1024;
};
constexpr uint32_t TEAM_COLS = 256;  // TMEM of a team: S0 [0,64), S1 [64,128), O [128,256)
constexpr uint32_t O_COL = 128;
constexpr uint32_t IDESC_QK = idesc_bf16_f32(128, KT, 0, 0);
constexpr uint32_t IDESC_PV = idesc_bf16_f32(128, AD, 0, 1);
constexpr int MIN_SHARE = 4;         // key tiles: below that a CTA's start costs more than it shares
// What a segment's start and end cost, in tiles: items weigh that much more. A mixed batch of seven requests took
// 322 us with 0, 287 with 4, 271 with 7, 265 with 10 and 274 with 16.
constexpr int SEGMENT_COST = 10;
constexpr int TILE_RING = 8;         // tile numbers in flight between warp 0 and the softmax warps

struct Args {
  PagedArgs b;
  int H, Hkv, T;
  float eps, scale_log2;
  const __nv_bfloat16* qkvg;
  const float* qw;
  const float* cos;
  const float* sin;
  const uint8_t* text_mask;
  const int32_t* key_end;
  __nv_bfloat16* out;
  float* part_o;   // (2 CTAs, part_rows, 128)
  float* part_ml;  // (2 CTAs, part_rows, 2): maximum in powers of two, sum
  struct Join* joins;  // (CTAs): the item that the start of each CTA's share cuts
  int part_rows;
  int group;       // keys per TMA box: 16, 32 or 64, a divisor of the page size
  int split;       // items may be cut
  int ctas;
};

// A cut item as paged_attn_join_kernel needs it. Entry c: the item that CTA c's share starts inside; its parts are
// those of the CTAs c - 1 to last, row0 the packed row of its first token; rows 0: nothing to join at this place.
struct Join {
  int rows, row0, j, last;
};

struct ItemPlan {
  RequestRows q;
  int tiles, qtiles, rounds, rest;  // rest: items beyond the whole rounds
  int unit;                         // weight of an item: its tiles and SEGMENT_COST (1 where items are not cut)
  long long weight;                 // of the rest
  // First tile of an item's part that starts at weight `at` within the item.
  __device__ __forceinline__ int tile_at(int at) const { return min(max(at - SEGMENT_COST, 0), tiles); }
};

template <int QPOS>
__device__ __forceinline__ ItemPlan plan_of(const Args& a, int r, bool* bad) {
  ItemPlan p;
  *bad = !request_rows(r, a.b.M, (long long)a.b.max_pages * a.b.page_size, a.b.q_start, a.b.kv_len, &p.q);
  if (*bad) p.q.n = 0;
  p.tiles = p.q.n ? (p.q.L + KT - 1) / KT : 1;
  p.qtiles = (p.q.n + QPOS - 1) / QPOS;
  const unsigned items = (unsigned)p.qtiles * (unsigned)a.Hkv;  // below 2^32: launch_paged_attn_tc checks it
  p.rounds = (int)(items / (unsigned)a.ctas);
  p.rest = (int)(items - (unsigned)p.rounds * (unsigned)a.ctas);
  p.unit = a.split ? p.tiles + SEGMENT_COST : 1;
  p.weight = (long long)p.rest * p.unit;
  return p;
}

// The batch's shared work (every request's rest, in order) and the place `part * share` in it. All threads
// of the block call it.
struct Place {
  long long total, share, offset;  // offset: within request r's weight
  int r;                           // a.b.R: the place is behind the end
  int rounds;                      // whether a request has whole rounds
};
template <int QPOS>
__device__ Place find_place(const Args& a, int part, Place* shared, long long* warp_sums) {
  const int tid = threadIdx.x, nt = blockDim.x, warp = tid >> 5, lane = tid & 31;
  const int per = (a.b.R + nt - 1) / nt, r0 = min(tid * per, a.b.R), r1 = min(r0 + per, a.b.R);
  long long sum = 0;
  int rounds = 0;
  for (int r = r0; r < r1; ++r) {
    bool bad;
    const ItemPlan p = plan_of<QPOS>(a, r, &bad);
    if (bad && blockIdx.x == 0) atomicOr(&g_device_error, ERR_BAD_BATCH);
    sum += p.weight;
    rounds |= p.rounds;
  }
  long long incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) warp_sums[warp] = incl;
  if (tid == 0) shared->r = a.b.R;
  rounds = __syncthreads_or(rounds);
  long long before = 0, total = 0;
  for (int w = 0; w < nt / 32; ++w) {
    if (w < warp) before += warp_sums[w];
    total += warp_sums[w];
  }
  // 32-bit where it fits: a 64-bit division is a few hundred cycles of every CTA's start
  const long long up = total + a.ctas - 1;
  long long share = up <= 0xffffffffLL ? (long long)((unsigned)up / (unsigned)a.ctas) : up / a.ctas;
  if (a.split && share < MIN_SHARE) share = MIN_SHARE;
  if (share < 1) share = 1;
  const long long at = part * share, lo = before + incl - sum;
  if (at >= lo && at < lo + sum) {  // one thread at most
    long long left = at - lo;
    for (int r = r0; r < r1; ++r) {
      bool bad;
      const ItemPlan p = plan_of<QPOS>(a, r, &bad);
      if (left < p.weight) {
        shared->r = r;
        shared->offset = left;
        break;
      }
      left -= p.weight;
    }
  }
  __syncthreads();
  Place x = *shared;
  x.total = total;
  x.share = share;
  x.rounds = rounds;
  return x;
}

// What the roles know of a segment.
struct Segment {
  int row0, n;        // packed row of its first token, tokens (n < 0: no more segments)
  int r, L, pos0;     // request, its keys, the first token's position
  int j;              // KV head
  int tiles;          // key tiles that are computed (tiles of masked keys are left out)
  int kmin;           // keys below it need no per-row limit
  int slot;           // part number, or -1: the whole item
};

__device__ __forceinline__ bool key_used(const Args& a, int r, int L, int t) {
  if (t >= L) return false;
  return !(a.text_mask && t < a.T) || a.text_mask[(long long)r * a.T + t] != 0;
}

// Whether each of the 32 tiles from t0 on (below t1, and wholly among the request's first T keys) has a key to
// compute: bit i for tile t0 + i. The whole warp reads a tile's 64 mask bytes at once, four tiles in flight.
__device__ __forceinline__ uint32_t used_tiles(const Args& a, int r, int L, int t0, int t1, int lane) {
  const uint8_t* mask = a.text_mask + (long long)r * a.T;
  uint32_t word = 0;
  for (int i = 0; i < 32 && t0 + i < t1; i += 4) {
    bool used[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int k = (t0 + i + q) * KT + lane, end = t0 + i + q < t1 ? L : 0;
      const uint8_t m0 = k < end ? mask[k] : 0, m1 = k + 32 < end ? mask[k + 32] : 0;
      used[q] = (m0 | m1) != 0;
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) word |= (uint32_t)__any_sync(0xffffffffu, used[q]) << (i + q);
  }
  return word;
}

// One arrival per warp: 32 lanes' arrivals on one barrier are taken one after the other.
__device__ __forceinline__ void warp_arrive(uint64_t* bar, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

template <int G, bool FEW>
__global__ void __launch_bounds__(Cfg<G, FEW>::THREADS, Cfg<G, FEW>::CTAS_PER_SM)
    paged_attn_tc_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, Args a) {
  using C = Cfg<G, FEW>;
  constexpr int TEAMS = C::TEAMS, ROWS = C::ROWS, QPOS = C::QPOS, STAGES = C::STAGES, THREADS = C::THREADS;
  constexpr int Q_CHUNK = C::Q_CHUNK, OFF_K = C::OFF_K, OFF_V = C::OFF_V, FIRST_SOFTMAX = C::FIRST_SOFTMAX;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t seg_full[2], seg_empty[2];
  __shared__ __align__(8) uint64_t q_full[TEAMS];
  __shared__ __align__(8) uint64_t k_full[STAGES], k_empty[STAGES], v_full[STAGES], v_empty[STAGES];
  __shared__ __align__(8) uint64_t s_full[TEAMS][2], p_full[TEAMS][2], pv_done[TEAMS][2];
  __shared__ __align__(8) uint64_t drain_bar[TEAMS];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  __shared__ Segment segs[2];
  __shared__ int tile_of[TILE_RING];
  __shared__ Place place_sh;
  __shared__ long long warp_sums[THREADS / 32];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t base_u32 = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* base = smem_raw + (base_u32 - smem_u32(smem_raw));

  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(&seg_full[s], 1);
      mbar_init(&seg_empty[s], TEAMS * (SOFTMAX_WARPS + 1));
    }
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], TEAMS);
      mbar_init(&v_full[s], 1);
      mbar_init(&v_empty[s], TEAMS);
    }
    for (int t = 0; t < TEAMS; ++t) {
      for (int s = 0; s < 2; ++s) {
        mbar_init(&s_full[t][s], 1);
        mbar_init(&p_full[t][s], SOFTMAX_WARPS);
        mbar_init(&pv_done[t][s], 1);
      }
      mbar_init(&q_full[t], SOFTMAX_WARPS);
      mbar_init(&drain_bar[t], 1);
    }
    abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  if (warp == 1) tmem_alloc(&tmem_slot, TEAMS * TEAM_COLS);
  const Place place = find_place<QPOS>(a, blockIdx.x, &place_sh, warp_sums);
  // the join kernel behind this grid may be made ready (it waits for this grid's end)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = tmem_slot;
  volatile int* abort = &abort_flag;

  if (warp == 0) {
    // ---- segments and K/V loads. The whole warp runs along; lane 0 signs for the bytes, lanes issue boxes.
    int it = 0, seg = 0;  // tiles and segments so far
    int k_st = 0, k_ph = 0, v_st = 0, v_ph = 0;  // next stages of K and of V, and their phases
    auto step = [](int& st, int& ph) {
      if (++st == STAGES) {
        st = 0;
        ph ^= 1;
      }
    };
    IssuedFills k_fills, v_fills;
    const int per_page = a.b.page_size / a.group, boxes = KT / a.group;
    // Of the last request looked at: the tiles with keys to compute from mask_t0 on, and lane i's page and slot of box
    // `cached` + i. The items of a request's heads and tokens follow one another and start with the same tiles.
    int mask_r = -1, mask_t0 = 0, page_r = -1, cached = 0, my_page = 0, my_slot = 0;
    uint32_t mask_word = 0;
    bool ok = true;

    auto publish = [&](const Segment& s) -> bool {
      if (!warp_wait(&seg_empty[seg & 1], ((seg >> 1) & 1) ^ 1, abort)) return false;
      if (lane == 0) {
        segs[seg & 1] = s;
        mbar_arrive(&seg_full[seg & 1]);
      }
      ++seg;
      return true;
    };
    // One item (or the tiles [t0, t1) of it): the segment, then its tiles.
    auto run_item = [&](const ItemPlan& p, int r, int item, int t0, int t1, int slot) -> bool {
      Segment s;
      const int qt = item % p.qtiles;
      s.j = item / p.qtiles;
      s.r = r;
      s.L = p.q.L;
      s.row0 = p.q.row0 + qt * QPOS;
      s.n = min(QPOS, p.q.n - qt * QPOS);
      s.pos0 = p.q.L - p.q.n + qt * QPOS;
      s.slot = slot;
      s.kmin = p.q.L;
      int te = t1;
      if (a.key_end) {
        int hi = 0, lo = p.q.L;
        for (int i = lane; i < s.n; i += 32) {
          const int e = min(max(a.key_end[s.row0 + i], s.pos0 + i + 1), p.q.L);
          hi = max(hi, e);
          lo = min(lo, e);
        }
        s.kmin = __reduce_min_sync(0xffffffffu, lo);
        te = min(te, (__reduce_max_sync(0xffffffffu, hi) + KT - 1) / KT);
      }
      s.tiles = max(te - t0, 0);
      const int text_tiles = a.text_mask ? min(te, a.T / KT) : 0;  // tiles that may hold masked keys only
      const int all_text = a.text_mask ? min(p.tiles, a.T / KT) : 0;
      uint32_t first_used = 0;
      for (int t = t0; t < text_tiles; t += 32) {
        uint32_t w;
        if (t == t0) {
          if (mask_r != r || mask_t0 != t0) {
            mask_word = used_tiles(a, r, p.q.L, t0, all_text, lane);
            mask_r = r;
            mask_t0 = t0;
          }
          w = first_used = mask_word;
        } else {
          w = used_tiles(a, r, p.q.L, t, all_text, lane);
        }
        if (text_tiles - t < 32) w &= (1u << (text_tiles - t)) - 1u;
        s.tiles -= min(32, text_tiles - t) - __popc(w);
      }
      if (!publish(s)) return false;

      const int32_t* pages = a.b.page_table + (long long)r * a.b.max_pages;
      const int groups = (p.q.L + a.group - 1) / a.group;  // boxes that hold keys
      uint32_t used = 0;
      int prev_tile = -1;                          // the tile whose V is still to be loaded
      int prev_page = 0, prev_slot = 0;
      bool prev_has = false;
      int prev_count = 0;
      auto load_v = [&]() -> bool {
        const int st = v_st;
        if (!warp_wait(&v_empty[st], v_ph ^ 1, abort)) return false;
        uint8_t* vd = base + OFF_V + st * KV_TILE_BYTES;
        if (lane == 0) mbar_arrive_expect_tx(&v_full[st], prev_count * a.group * (2 * AD));
        __syncwarp();
        if (a.group == KT) {
          if (lane == 0) tma_load_4d(vd, &tmV, &v_full[st], 0, prev_slot, s.j * 2, prev_page);
        } else if (prev_has) {
          tma_load_4d(vd + (lane & 1) * KV_CHUNK + (lane >> 1) * a.group * 128, &tmV, &v_full[st], 0, prev_slot,
                      s.j * 2 + (lane & 1), prev_page);
        }
        v_fills.note(st, v_ph);
        step(v_st, v_ph);
        return true;
      };
      for (int t = t0; t < te; ++t) {
        if (t < text_tiles) {
          if (t == t0) used = first_used;
          else if ((t - t0) % 32 == 0) used = used_tiles(a, r, p.q.L, t, all_text, lane);
          if (!((used >> ((t - t0) & 31)) & 1u)) continue;
        }
        // pages of the tile's boxes: 32 boxes looked up at once
        const int g0 = t * boxes;
        if (page_r != r || g0 < cached || g0 + boxes > cached + 32) {
          page_r = r;
          cached = g0;
          const int g = g0 + lane;
          my_page = a.b.num_pages;  // outside the pool: reads as zeros
          my_slot = 0;
          if (g < groups) {
            const int pg = pages[g / per_page];
            my_slot = (g % per_page) * a.group;
            if (pg >= 0 && pg < a.b.num_pages) my_page = pg;
            else atomicOr(&g_device_error, ERR_BAD_BATCH);
          }
        }
        const int count = min(boxes, groups - g0);
        // lane 2 b + c: box b, 64-column chunk c (one box per tile: both chunks at once, by lane 0)
        const int src = min(g0 - cached + (a.group == KT ? 0 : lane >> 1), 31);
        const int page = __shfl_sync(0xffffffffu, my_page, src), slot_in = __shfl_sync(0xffffffffu, my_slot, src);
        const bool has = (lane >> 1) < count;
        const int st = k_st;
        if (!warp_wait(&k_empty[st], k_ph ^ 1, abort)) return false;
        uint8_t* kd = base + OFF_K + st * KV_TILE_BYTES;
        if (lane == 0) {
          // bit 0: keys of the tile may be unused, bit 1: rows end inside it
          const int k0 = t * KT;
          tile_of[it % TILE_RING] = k0 | ((a.text_mask && k0 < a.T) || k0 + KT > s.L ? 1 : 0) | (k0 + KT > s.kmin ? 2 : 0);
          mbar_arrive_expect_tx(&k_full[st], count * a.group * (2 * AD));
        }
        __syncwarp();
        if (a.group == KT) {
          if (lane == 0) tma_load_4d(kd, &tmK, &k_full[st], 0, slot_in, s.j * 2, page);
        } else if (has) {
          tma_load_4d(kd + (lane & 1) * KV_CHUNK + (lane >> 1) * a.group * 128, &tmK, &k_full[st], 0, slot_in,
                      s.j * 2 + (lane & 1), page);
        }
        k_fills.note(st, k_ph);
        step(k_st, k_ph);
        // V runs one tile behind K: V stages free up after P V only
        if (prev_tile >= 0 && !load_v()) return false;
        ++it;
        prev_tile = t;
        prev_page = page;
        prev_slot = slot_in;
        prev_has = has;
        prev_count = count;
      }
      return prev_tile < 0 || load_v();
    };

    if (place.rounds)
      for (int r = 0; r < a.b.R && ok; ++r) {
        bool bad;
        const ItemPlan p = plan_of<QPOS>(a, r, &bad);
        for (int k = 0; k < p.rounds && ok; ++k) ok = run_item(p, r, k * a.ctas + blockIdx.x, 0, p.tiles, -1);
      }
    long long left = min(place.share, place.total - blockIdx.x * place.share), off = place.offset;
    for (int r = place.r; r < a.b.R && left > 0 && ok; ++r, off = 0) {
      bool bad;
      const ItemPlan p = plan_of<QPOS>(a, r, &bad);
      while (off < p.weight && left > 0 && ok) {
        const int nth = (int)(off / p.unit), at = (int)(off - (long long)nth * p.unit);
        const int item = p.rounds * a.ctas + nth;
        const int len = (int)min((long long)(p.unit - at), left);
        if (a.split) {
          const int from = p.tile_at(at), to = at + len == p.unit ? p.tiles : p.tile_at(at + len);
          // a part that does not start its item is the CTA's first, one that does not end it its last
          const int slot = from == 0 && to == p.tiles ? -1 : 2 * blockIdx.x + (from == 0 ? 1 : 0);
          if (from < to) ok = run_item(p, r, item, from, to, slot);
        } else {
          ok = run_item(p, r, item, 0, p.tiles, -1);
        }
        off += len;
        left -= len;
      }
    }
    if (ok) {
      Segment end{};
      end.n = -1;
      publish(end);
    }
    if (*abort && lane == 0) {
      k_fills.drain(k_full, STAGES);
      v_fills.drain(v_full, STAGES);
    }
    __syncwarp();
  } else if (warp <= TEAMS) {
    // ---- a team's MMAs. The whole warp runs along, so that descriptors and loop counters are warp-uniform (they
    // live in uniform registers, where the MMA takes them from); one elected lane issues.
    const int team = warp - 1;
    const bool leader = elect_one();
    const uint32_t tmem = tmem_base + team * TEAM_COLS;
    const uint64_t dq0 = smem_desc_sw128(smem_u32(base + team * 2 * Q_CHUNK), 16, 1024);
    const uint64_t dk0 = smem_desc_sw128(smem_u32(base + OFF_K), 16, 1024);
    const uint64_t dv0 = smem_desc_sw128(smem_u32(base + OFF_V), KV_CHUNK, 1024);
    bool issued = false, ok = true;
    int it = 0;       // the team's tiles so far
    int queries = 0;  // its segments with rows and tiles so far
    int k_st = 0, k_ph = 0, v_st = 0, v_ph = 0;
    auto step = [](int& st, int& ph) {
      if (++st == STAGES) {
        st = 0;
        ph ^= 1;
      }
    };
    auto wait = [&](uint64_t* bar, int parity) { return warp_wait(bar, parity, abort); };
    for (int seg = 0; ok; ++seg) {
      if (!wait(&seg_full[seg & 1], (seg >> 1) & 1)) break;
      const int n = segs[seg & 1].n, tiles = segs[seg & 1].tiles;
      __syncwarp();
      if (leader) mbar_arrive(&seg_empty[seg & 1]);
      if (n < 0) break;
      if (n * G <= team * ROWS) {  // no rows of this team: its share of the stages is free as soon as they are full
        for (int i = 0; i < tiles && ok; ++i) {
          ok = wait(&k_full[k_st], k_ph);
          if (ok && leader) mbar_arrive(&k_empty[k_st]);
          ok = ok && wait(&v_full[v_st], v_ph);
          if (ok && leader) mbar_arrive(&v_empty[v_st]);
          step(k_st, k_ph);
          step(v_st, v_ph);
        }
        continue;
      }
      if (tiles == 0) continue;  // no product, and no arrival on q_full
      if (!wait(&q_full[team], queries++ & 1)) break;
      tc_fence_after();
      // Step i issues P V of tile i - 2, then Q K of tile i into the scores that P overlaid. Of the waits only the one
      // for P is not long over, so it comes last; s_full is committed first: from a tile's P to the scores two tiles
      // on and their softmax is the loop that sets the pace.
      const int first = it, end = first + tiles;
      for (; it < end + 2; ++it) {
        const bool qk = it < end, pv = it - 2 >= first;
        // the three tests go out together
        const uint32_t k_ok = qk ? mbar_try_wait(&k_full[k_st], k_ph) : 1, v_ok = pv ? mbar_try_wait(&v_full[v_st], v_ph) : 1;
        const uint32_t p_ok = pv ? mbar_try_wait(&p_full[team][it & 1], ((it - 2) >> 1) & 1) : 1;
        if (!__all_sync(0xffffffffu, k_ok & v_ok & p_ok)) {
          if (qk && !wait(&k_full[k_st], k_ph)) ok = false;
          if (ok && pv && !(wait(&v_full[v_st], v_ph) && wait(&p_full[team][it & 1], ((it - 2) >> 1) & 1))) ok = false;
          if (!ok) break;
        }
        tc_fence_after();
        if (leader) {
          const uint32_t d_s = tmem + (it & 1) * KT;  // the scores of tile it, and P of tile it - 2
          if (pv) {
            const uint64_t dv = dv0 + (uint64_t)(v_st * (KV_TILE_BYTES >> 4));
#pragma unroll
            for (int kk = 0; kk < KT / 16; ++kk)
              tc_mma_bf16_ts(tmem + O_COL, d_s + kk * 8, dv + (uint64_t)(kk * 16 * 128 >> 4), IDESC_PV,
                             (it - 2 > first || kk > 0) ? 1u : 0u);
          }
          if (qk) {
            const uint64_t dk = dk0 + (uint64_t)(k_st * (KV_TILE_BYTES >> 4));
#pragma unroll
            for (int kk = 0; kk < AD / 16; ++kk) {
              const uint32_t qo = (kk >> 2) * Q_CHUNK + (kk & 3) * 32;
              const uint32_t ko = (kk >> 2) * KV_CHUNK + (kk & 3) * 32;
              tc_mma_bf16(d_s, dq0 + (uint64_t)(qo >> 4), dk + (uint64_t)(ko >> 4), IDESC_QK, kk > 0 ? 1u : 0u);
            }
            tc_commit(&s_full[team][it & 1]);
            tc_commit(&k_empty[k_st]);
          }
          if (pv) {
            tc_commit(&pv_done[team][it & 1]);
            tc_commit(&v_empty[v_st]);
          }
        }
        __syncwarp();
        issued = true;
        if (qk) step(k_st, k_ph);
        if (pv) step(v_st, v_ph);
      }
      it = end;
    }
    if (*abort && issued) {
      if (leader) tc_commit(&drain_bar[team]);
      mbar_wait_drain(&drain_bar[team], 0);
    }
    __syncwarp();
  } else {
    // ---- queries, softmax and output: warps w and w + 4 share TMEM lane quarter w & 3, 16 rows each;
    // threads t and t + 16 hold the same row and split its 64 scores and 128 output columns
    const int team = (warp - FIRST_SOFTMAX) >> 3;
    const int quarter = warp & 3, sub = ((warp - FIRST_SOFTMAX) >> 2) & 1, half = lane >> 4;
    const int team_row = quarter * 32 + sub * 16;                   // the warp's first row in its team's tile
    const int warp_row = team * ROWS + team_row;                    // and among the item's rows
    const int row = warp_row + (lane & 15);
    const uint32_t lane_off = (uint32_t)team_row << 16;
    const uint32_t tmem = tmem_base + team * TEAM_COLS;
    uint8_t* q_smem = base + team * 2 * Q_CHUNK;
    const float sl2 = a.scale_log2;
    const long long qc = 2LL * (a.H + a.Hkv) * AD;
    constexpr int HK = KT / 2;
    int it = 0, seg = 0;                 // the team's tiles, segments
    int tile_no = 0, v_st = 0, v_ph = 0;  // the CTA's tiles, with the stage of V
    Segment s;
    // Segment's queries, normalised and rotated, into shared memory (row = token * G + head, 128-byte swizzle)
    auto next_segment = [&]() -> bool {
      if (!warp_wait(&seg_full[seg & 1], (seg >> 1) & 1, abort)) return false;
      s = segs[seg & 1];
      if (s.n < 0) return false;
      // without tiles there is nothing to wait for on the other side, so q_full must not advance either: the
      // phase of a later segment could complete before the MMA thread has seen this one
      if (s.tiles == 0 || s.n * G <= team * ROWS) return true;
      const float4 w4 = *reinterpret_cast<const float4*>(a.qw + lane * 4);
      const int rows = min(16, s.n * G - warp_row);
#pragma unroll 1
      for (int i0 = 0; i0 < rows; i0 += 4) {
        uint2 raw[4];
        float2 c[4], sn[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int rr = warp_row + min(i0 + i, rows - 1), prow = s.row0 + rr / G;
          raw[i] = *reinterpret_cast<const uint2*>(a.qkvg + prow * qc + (s.j * G + rr % G) * AD + lane * 4);
          c[i] = *reinterpret_cast<const float2*>(a.cos + (long long)prow * (AD / 2) + lane * 2);
          sn[i] = *reinterpret_cast<const float2*>(a.sin + (long long)prow * (AD / 2) + lane * 2);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int rr = warp_row + min(i0 + i, rows - 1) - team * ROWS;
          float v[4] = {bf16_lo(raw[i].x), bf16_hi(raw[i].x), bf16_lo(raw[i].y), bf16_hi(raw[i].y)};
          const float ss = warp_sum(v[0] * v[0] + v[1] * v[1] + v[2] * v[2] + v[3] * v[3]);
          const float rs = rsqrtf(ss / (float)AD + a.eps);
          v[0] *= rs * (1.f + w4.x);
          v[1] *= rs * (1.f + w4.y);
          v[2] *= rs * (1.f + w4.z);
          v[3] *= rs * (1.f + w4.w);
          uint2 o;
          o.x = pack_bf16x2(v[0] * c[i].x - v[1] * sn[i].x, v[1] * c[i].x + v[0] * sn[i].x);
          o.y = pack_bf16x2(v[2] * c[i].y - v[3] * sn[i].y, v[3] * c[i].y + v[2] * sn[i].y);
          *reinterpret_cast<uint2*>(q_smem + (lane >> 4) * Q_CHUNK + rr * 128 + ((((lane & 15) >> 1) ^ (rr & 7)) << 4) +
                                    (lane & 1) * 8) = o;
        }
      }
      fence_proxy_async_smem();
      warp_arrive(&q_full[team], lane);
      return true;
    };

    // One tile of scores to P. Tiles with masked keys, with row limits inside them or with V rows to clear take a form of
    // their own: with its tests in the common one, that took 8 % longer.
    bool active = false;  // the warp holds rows of the segment
    auto softmax_tile = [&](auto partial, int tile, int i, int n, int st, int ph, const Segment& cur, int row_kend,
                            float& m, float& l) -> bool {
      constexpr bool PARTIAL = decltype(partial)::value;
      const int sb = n & 1, t0 = tile & ~(KT - 1);
      uint32_t vm0 = 0xffffffffu, vm1 = 0xffffffffu;
      const uint32_t sbase = tmem + lane_off + sb * KT;
      if constexpr (PARTIAL) {
        if (tile & 1) {
          vm0 = __ballot_sync(0xffffffffu, key_used(a, cur.r, cur.L, t0 + lane));
          vm1 = __ballot_sync(0xffffffffu, key_used(a, cur.r, cur.L, t0 + 32 + lane));
          if ((vm0 & vm1) != 0xffffffffu) {  // the same for all warps: clear the V rows of unused keys
            if (!warp_wait(&v_full[st], ph, abort)) return false;
            const int key = ((warp - FIRST_SOFTMAX) & 7) * 8 + (lane >> 2), part = lane & 3;
            const uint32_t vm = key < 32 ? vm0 : vm1;
            if (!((vm >> (key & 31)) & 1u)) {
              uint8_t* v = base + OFF_V + st * KV_TILE_BYTES + (part >> 1) * KV_CHUNK + key * 128 + (part & 1) * 64;
#pragma unroll
              for (int q = 0; q < 4; ++q) reinterpret_cast<uint4*>(v)[q] = make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();
          }
        }
      }
      if (PARTIAL && !active) return true;
      float v[HK];
      tmem_ld32_pair<HK>(sbase, v);
      if constexpr (PARTIAL) {
        const uint32_t vm = half ? vm1 : vm0;
        if ((tile & 1) && (vm0 & vm1) != 0xffffffffu) {
#pragma unroll
          for (int e = 0; e < HK; ++e)
            if (!((vm >> e) & 1u)) v[e] = -INFINITY;
        }
        if (tile & 2) {
          const int lim = row_kend - (t0 + half * HK);
#pragma unroll
          for (int e = 0; e < HK; ++e)
            if (e >= lim) v[e] = -INFINITY;
        }
      }
      // the half row's maximum as a tree of three-input maxima
      float m11[11], m4[4];
#pragma unroll
      for (int k = 0; k < 10; ++k) m11[k] = fmax3(v[3 * k], v[3 * k + 1], v[3 * k + 2]);
      m11[10] = fmaxf(v[30], v[31]);
#pragma unroll
      for (int k = 0; k < 3; ++k) m4[k] = fmax3(m11[3 * k], m11[3 * k + 1], m11[3 * k + 2]);
      m4[3] = fmaxf(m11[9], m11[10]);
      const float hm = fmaxf(fmax3(m4[0], m4[1], m4[2]), m4[3]);
      const float mx = fmaxf(hm, __shfl_xor_sync(0xffffffffu, hm, 16));
      const float mnew = fmaxf(m, mx * sl2);
      const bool grow = mnew > m + 8.0f;  // m = -inf on the first tile
      float alpha = 1.f;
      const bool any_grow = __any_sync(0xffffffffu, grow);
      if (grow) {
        alpha = ex2(m - mnew);  // 0 on the first tile
        m = mnew;
      }
      uint32_t pk[HK / 2];
      const float rs = exp_tile<HK>(v, sl2, m == -INFINITY ? 0.f : m, pk);
      l = l * alpha + rs;
      tmem_st16_pair<HK / 2>(sbase, pk);
      if (i >= 1 && any_grow) {
        if (!warp_wait(&pv_done[team][(n - 1) & 1], ((n - 1) >> 1) & 1, abort)) return false;
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < AD / 64; ++c) {
          float o[32];
          const uint32_t oa = tmem + lane_off + O_COL + c * 32;
          tmem_ld32_pair<AD / 2>(oa, o);
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] *= alpha;
          tmem_st32_pair<AD / 2>(oa, o);
        }
      }
      tmem_wait_st();
      return true;
    };

    bool ok = next_segment();
    while (ok) {
      const Segment cur = s;
      active = warp_row < cur.n * G;
      const int tiles = cur.n * G > team * ROWS ? cur.tiles : 0;  // without rows the team computes none
      const int tok = row / G;
      int row_kend = cur.L;
      if (a.key_end && tok < cur.n) row_kend = min(max(a.key_end[cur.row0 + tok], cur.pos0 + tok + 1), cur.L);
      float m = -INFINITY, l = 0.f;
      for (int i = 0; i < tiles; ++i, ++it) {
        const int sb = it & 1, st = v_st, ph = v_ph;
        if (++v_st == STAGES) {
          v_st = 0;
          v_ph ^= 1;
        }
        if (!warp_wait(&s_full[team][sb], (it >> 1) & 1, abort)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const int tile = tile_of[(tile_no + i) % TILE_RING];
        if ((tile & 3) == 0) {
          if (active) ok = softmax_tile(std::false_type(), tile, i, it, st, ph, cur, row_kend, m, l);
        } else {
          ok = softmax_tile(std::true_type(), tile, i, it, st, ph, cur, row_kend, m, l);
        }
        if (!ok) break;
        tc_fence_before();
        warp_arrive(&p_full[team][sb], lane);
      }
      if (!ok) break;
      tile_no += cur.tiles;
      for (int i = tiles; i < cur.tiles; ++i)
        if (++v_st == STAGES) {
          v_st = 0;
          v_ph ^= 1;
        }
      // the last s_full was the last use of Q: the next segment's queries go in, and its first product
      // starts while this segment's output is written
      ++seg;
      const bool more = next_segment();
      // the gates of a whole item, on their way before the last product is waited for
      const bool row_ok = tok < cur.n;
      const int h = cur.j * G + row % G;
      const long long prow = cur.row0 + tok;
      const uint4* gp =
          reinterpret_cast<const uint4*>(a.qkvg + prow * qc + (a.H + 2 * a.Hkv + h) * AD + half * (AD / 2));
      uint4 gates[4];
      const bool gated = active && row_ok && cur.slot < 0;
      if (gated)
#pragma unroll
        for (int q = 0; q < 4; ++q) gates[q] = __ldg(gp + q);
      if (tiles > 0) {
        const int i = it - 1;
        if (!warp_wait(&pv_done[team][i & 1], (i >> 1) & 1, abort)) break;
        tc_fence_after();
      }
      if (active) {
        const float lt = l + __shfl_xor_sync(0xffffffffu, l, 16);
        const float inv_l = lt > 0.f ? 1.f / lt : (lt == 0.f ? 0.f : lt);  // no readable key: zeros; NaN stays
#pragma unroll 1
        for (int c = 0; c < AD / 64; ++c) {
          const int col = half * (AD / 2) + c * 32;
          float o[32];
          if (tiles > 0) {
            tmem_ld32_pair<AD / 2>(tmem + lane_off + O_COL + c * 32, o);
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = 0.f;
          }
          if (row_ok && cur.slot >= 0) {
            float4* po = reinterpret_cast<float4*>(a.part_o + ((long long)cur.slot * a.part_rows + row) * AD + col);
#pragma unroll
            for (int q = 0; q < 8; ++q) po[q] = make_float4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
          } else if (row_ok) {
            uint4* op = reinterpret_cast<uint4*>(a.out + prow * (a.H * AD) + h * AD + col);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const uint4 gv = gates[q];
              if (c == 0) gates[q] = __ldg(gp + 4 + q);
              const uint32_t gw[4] = {gv.x, gv.y, gv.z, gv.w};
              uint32_t ow[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                ow[e] = pack_bf16x2(o[q * 8 + 2 * e] * inv_l * sigmoid_fast(bf16_lo(gw[e])),
                                    o[q * 8 + 2 * e + 1] * inv_l * sigmoid_fast(bf16_hi(gw[e])));
              op[q] = make_uint4(ow[0], ow[1], ow[2], ow[3]);
            }
          }
          __syncwarp();
        }
        if (cur.slot >= 0 && row_ok && half == 0) {
          float2* ml = reinterpret_cast<float2*>(a.part_ml) + (long long)cur.slot * a.part_rows + row;
          *ml = make_float2(m, lt);
        }
      }
      tc_fence_before();
      warp_arrive(&seg_empty[(seg - 1) & 1], lane);
      ok = more;
    }
  }

  if (a.joins && threadIdx.x == 32) {  // what it joins at the start of this CTA's share
    Join x{};
    if (place.r < a.b.R) {
      bool bad;
      const ItemPlan p = plan_of<QPOS>(a, place.r, &bad);
      const int nth = (int)(place.offset / p.unit), at = (int)(place.offset - (long long)nth * p.unit);
      // the first place that leaves tiles on both sides joins the item
      const long long start = (long long)blockIdx.x * place.share - at;
      if (at > SEGMENT_COST && at - place.share <= SEGMENT_COST) {
        const int item = p.rounds * a.ctas + nth, qt = item % p.qtiles;
        x.j = item / p.qtiles;
        x.rows = min(QPOS, p.q.n - qt * QPOS) * G;
        x.row0 = p.q.row0 + qt * QPOS;
        x.last = (int)((start + p.unit - 1) / place.share);
      }
    }
    a.joins[blockIdx.x] = x;
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, TEAMS * TEAM_COLS);
  }
}

constexpr int JOIN_ROWS = 8;  // one per warp

// Joins the parts of cut items: block (c, y), for eight rows, looks at the place where CTA c's share starts, and
// joins the item that is cut there if no earlier place cuts it. Parts come in key order, so results repeat bit
// for bit. Launched as a programmatic dependent of the kernel above.
template <int G>
__global__ void __launch_bounds__(256) paged_attn_join_kernel(Args a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int c = blockIdx.x + 1, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Join x = a.joins[c];
  const long long qc = 2LL * (a.H + a.Hkv) * AD;
  const int end = min(x.rows, (int)(blockIdx.y + 1) * JOIN_ROWS);
  for (int row = blockIdx.y * JOIN_ROWS + warp; row < end; row += 8) {
    const int h = x.j * G + row % G;
    const long long prow = x.row0 + row / G;
    const uint2 g = *reinterpret_cast<const uint2*>(a.qkvg + prow * qc + (a.H + 2 * a.Hkv + h) * AD + lane * 4);
    const float2* ml = reinterpret_cast<const float2*>(a.part_ml) + row;
    const float4* po = reinterpret_cast<const float4*>(a.part_o + (long long)row * AD) + lane;
    auto slot_of = [&](int k) { return (long long)(k == 0 ? 2 * (c - 1) + 1 : 2 * (c - 1 + k)) * a.part_rows; };
    float o[4] = {0.f, 0.f, 0.f, 0.f}, sum = 0.f, top = -INFINITY;
    // 32 parts at a time: a lane takes a part's maximum and sum, then the warp takes the parts' rows, four in flight
    const int parts = x.last - c + 2;
    for (int k0 = 0; k0 < parts; k0 += 32) {
      float2 v = make_float2(-INFINITY, 0.f);
      if (k0 + lane < parts) v = ml[slot_of(k0 + lane)];
      float m = fmaxf(top, v.x);
#pragma unroll
      for (int s = 16; s > 0; s >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, s));
      const float old = top == -INFINITY ? 0.f : ex2(top - m);
      // a part without a readable key counts nothing
      const float w = v.x == -INFINITY && v.y == 0.f ? 0.f : ex2(v.x - m);
      sum = sum * old + warp_sum(w * v.y);
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] *= old;
      const int n = min(32, parts - k0);
#pragma unroll 4
      for (int k = 0; k < n; ++k) {
        const float4 y = po[slot_of(k0 + k) * (AD / 4)];
        const float wk = __shfl_sync(0xffffffffu, w, k);
        o[0] += wk * y.x;
        o[1] += wk * y.y;
        o[2] += wk * y.z;
        o[3] += wk * y.w;
      }
      top = m;
    }
    const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
    uint2 r;
    r.x = pack_bf16x2(o[0] * inv * sigmoid_fast(bf16_lo(g.x)), o[1] * inv * sigmoid_fast(bf16_hi(g.x)));
    r.y = pack_bf16x2(o[2] * inv * sigmoid_fast(bf16_lo(g.y)), o[3] * inv * sigmoid_fast(bf16_hi(g.y)));
    *reinterpret_cast<uint2*>(a.out + prow * (a.H * AD) + h * AD + lane * 4) = r;
  }
}

int make_tmap_pages(CUtensorMap* m, const void* ptr, int Hkv, const Krea2PagedBatch& b, int group) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = tmap_encoder();
  if (!enc) return set_error(KREA2_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
  const cuuint64_t row = (cuuint64_t)Hkv * AD * 2;
  cuuint64_t dims[4] = {64, (cuuint64_t)b.page_size, (cuuint64_t)Hkv * 2, (cuuint64_t)b.num_pages};
  cuuint64_t strides[3] = {row, 128, row * b.page_size};
  // both 64-column chunks of a head at once where a box is a whole tile
  cuuint32_t box[4] = {64, (cuuint32_t)group, group == KT ? 2u : 1u, 1};
  cuuint32_t es[4] = {1, 1, 1, 1};
  CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(ptr), dims, strides, box, es,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return set_error(KREA2_ERR_CUDA, "cuTensorMapEncodeTiled (pages) failed (%d)", (int)r);
  return KREA2_OK;
}

// Launch sizes from what the host knows: row and request counts and the longest sequence the table holds.
struct Shape {
  int few, ctas, split, part_rows;
  size_t o_bytes, ml_bytes, join_bytes;
};
Shape shape_of(const Krea2PagedBatch& b, int H, int Hkv) {
  const int G = H / Hkv;
  Shape s;
  // About one new token per request, or so few that an item of 16 rows holds them. 16 rows against 256 rows an item:
  // eight single tokens over 521 to 8704 keys 49.9 and 52.7 us, 128 over 2048 keys 255 and 276, 128 of these beside a
  // chunk of 128 over 8704 443 and 478. The host knows rows and requests only, not how the rows are spread: one chunk
  // of 600 over 8704 keys beside 299 empty requests takes 793 us in 16-row items, 153 in the others. A batch that may
  // hold such a chunk should have more than two rows per request (rows behind the last request are no work).
  s.few = b.M <= 2LL * b.R || b.M * (long long)G <= 16;
  const int rows = s.few ? 16 : 256, qpos = rows / G;
  const long long qtiles = b.M < b.M / qpos + b.R ? b.M : b.M / qpos + (long long)b.R;
  const long long tiles = ((long long)b.max_pages * b.page_size + KT - 1) / KT;
  s.split = tiles > MIN_SHARE;
  const long long most = qtiles * Hkv * (s.split ? (tiles + MIN_SHARE - 1) / MIN_SHARE : 1);
  const long long resident = (s.few ? 2LL : 1LL) * num_sms();
  s.ctas = (int)(most < resident ? most : resident);
  if (s.ctas == 1) s.split = 0;
  s.part_rows = (long long)b.M * G < rows ? b.M * G : rows;
  s.o_bytes = s.split ? 2ull * s.ctas * s.part_rows * AD * 4 : 0;
  s.ml_bytes = s.split ? 2ull * s.ctas * s.part_rows * 2 * 4 : 0;
  s.join_bytes = s.split ? sizeof(Join) * s.ctas : 0;
  return s;
}

template <int G, bool FEW>
int launch(const Krea2PagedBatch& b, const PagedAttnArgs& pa, const Shape& sh, void* ws, cudaStream_t stream) {
  constexpr int SMEM_BYTES = Cfg<G, FEW>::SMEM_BYTES;
  static std::atomic<uint64_t> attr_done{0};
  auto kern = paged_attn_tc_kernel<G, FEW>;
  const uint64_t dev_bit = device_bit();
  if (!(attr_done.load(std::memory_order_acquire) & dev_bit) || !dev_bit) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES) != cudaSuccess ||
        cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared) !=
            cudaSuccess)
      return set_error(KREA2_ERR_CUDA, "cudaFuncSetAttribute(paged attention) failed");
    attr_done.fetch_or(dev_bit, std::memory_order_release);
  }
  Args a{};
  a.b = PagedArgs{b.R, b.M, b.q_start, b.kv_len, b.page_table, b.max_pages, b.page_size, b.num_pages};
  a.H = pa.H; a.Hkv = pa.Hkv; a.T = pa.T; a.eps = pa.eps; a.scale_log2 = pa.scale_log2;
  a.qkvg = reinterpret_cast<const __nv_bfloat16*>(pa.qkvg);
  a.qw = pa.q_norm_w; a.cos = pa.cos; a.sin = pa.sin; a.text_mask = pa.text_mask; a.key_end = pa.key_end;
  a.out = reinterpret_cast<__nv_bfloat16*>(pa.out);
  a.split = sh.split; a.ctas = sh.ctas; a.part_rows = sh.part_rows;
  if (sh.split) {
    uint8_t* w = reinterpret_cast<uint8_t*>(ws);
    a.part_o = reinterpret_cast<float*>(w);
    a.part_ml = reinterpret_cast<float*>(w + sh.o_bytes);
    a.joins = reinterpret_cast<Join*>(w + sh.o_bytes + sh.ml_bytes);
  }
  a.group = b.page_size % 64 == 0 ? 64 : b.page_size % 32 == 0 ? 32 : 16;
  CUtensorMap tk, tv;
  int rc;
  if ((rc = make_tmap_pages(&tk, pa.k_pages, pa.Hkv, b, a.group)) || (rc = make_tmap_pages(&tv, pa.v_pages, pa.Hkv, b, a.group)))
    return rc;
  kern<<<sh.ctas, Cfg<G, FEW>::THREADS, SMEM_BYTES, stream>>>(tk, tv, a);
  count_launch();
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess && sh.split) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(sh.ctas - 1, (sh.part_rows + JOIN_ROWS - 1) / JOIN_ROWS);
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, paged_attn_join_kernel<G>, a);
    count_launch();
  }
  if (e != cudaSuccess) return set_error(KREA2_ERR_CUDA, "paged attention launch failed: %s", cudaGetErrorString(e));
  return KREA2_OK;
}

template <int G>
int launch_g(const Krea2PagedBatch& b, const PagedAttnArgs& a, void* ws, cudaStream_t stream) {
  const Shape s = shape_of(b, a.H, a.Hkv);
  return s.few ? launch<G, true>(b, a, s, ws, stream) : launch<G, false>(b, a, s, ws, stream);
}

}  // namespace

size_t paged_attn_tc_workspace(const Krea2PagedBatch& b, int H, int Hkv) {
  const Shape s = shape_of(b, H, Hkv);
  return s.o_bytes + s.ml_bytes + s.join_bytes;
}

int launch_paged_attn_tc(const Krea2PagedBatch& b, const PagedAttnArgs& a, void* ws, cudaStream_t stream) {
  if ((long long)b.M * a.Hkv > 0x7fffffffLL)  // items (at most one per token and KV head) are counted in 32 bits
    return set_error(KREA2_ERR_UNSUPPORTED, "too many rows x KV heads (%lld)", (long long)b.M * a.Hkv);
  switch (a.H / a.Hkv) {
    case 1: return launch_g<1>(b, a, ws, stream);
    case 2: return launch_g<2>(b, a, ws, stream);
    default: return launch_g<4>(b, a, ws, stream);
  }
}

}  // namespace krea2
