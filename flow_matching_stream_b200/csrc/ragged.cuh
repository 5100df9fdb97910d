// Requests of a ragged batch (Krea2PagedBatch, Krea2Lora): rows, keys and pages of a request, and the
// checks that keep every access inside the arrays whatever the device arrays hold.
#pragma once
#include <stdint.h>

namespace krea2 {

// Batch arrays as the kernels take them.
struct PagedArgs {
  int R, M;
  const int32_t* q_start;
  const int32_t* kv_len;
  const int32_t* page_table;
  int max_pages, page_size, num_pages;
};

struct RequestRows {
  int row0, n, L;  // first packed row, new tokens, keys (new tokens included)
};

// Request r's rows and keys; false if its lengths are inconsistent.
__host__ __device__ inline bool request_rows(int r, int M, long long capacity, const int32_t* q_start,
                                             const int32_t* kv_len, RequestRows* out) {
  const int a = q_start[r], b = q_start[r + 1], L = kv_len[r];
  out->row0 = a;
  out->n = b - a;
  out->L = L;
  return a >= 0 && b >= a && b <= M && L >= b - a && L <= capacity && (r > 0 || a == 0);
}

// Largest r in [0, R) with start[r] <= row, 0 if there is none: the row's request where the starts
// ascend, in bounds whatever they hold.
__device__ __forceinline__ int request_of_row(const int32_t* start, int R, int row) {
  int lo = 0, hi = R;  // start[lo] <= row < start[hi] for ascending starts
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(start + mid) <= row) lo = mid;
    else hi = mid;
  }
  return lo;
}

#ifdef __CUDACC__
// A request's row: its request, or -1 for a row that belongs to none (or to an inconsistent one).
__device__ __forceinline__ int checked_request_of_row(const PagedArgs& p, int row, RequestRows* q, bool* bad) {
  const int r = request_of_row(p.q_start, p.R, row);
  *bad = !request_rows(r, p.M, (long long)p.max_pages * p.page_size, p.q_start, p.kv_len, q);
  return !*bad && row >= q->row0 && row - q->row0 < q->n ? r : -1;
}
#endif

}  // namespace krea2
