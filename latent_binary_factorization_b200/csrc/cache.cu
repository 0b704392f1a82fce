// The paged cache: rotary positions, rows into and out of pages, and the page
// bookkeeping (littlebit.h, "The paged cache").
//
// Row movement (rotary, write, read) is one kernel over a short list of row
// tensors, each side of which is either token rows or rows of pages, so a
// serving step's q, k and v go in one launch.  It is bound by HBM at prompt
// sizes and by launch latency at decode sizes.
//
// Bookkeeping (extend, fork, compact) is decided by one block of 1024 threads:
// the decisions are a scan over the lists and over refs[], a few KB to a few
// hundred KB, where a second block would only add a grid-wide wait.  The rows
// that move afterwards are copied by a grid of their own.  Each decision takes
// 3 to 4 us at decode sizes, a chain of about six trips to L2 (slots, lengths,
// claims and back, references, tables).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>

#include "lb_internal.h"

namespace {

constexpr int kMaxList = 4096;      // entries of a slot list
constexpr int kMaxPlanes = 1024;    // planes of a cache
constexpr int kPlaneBatch = 64;     // planes per copy launch (kernel parameter size)
constexpr int kMaxJobs = 8;         // row tensors per launch
constexpr int kBookThreads = 1024;
constexpr unsigned kStatusPages = 1u << LB_ERR_PAGES;
constexpr unsigned kStatusIndex = 1u << LB_ERR_INDEX;

// Error bits of the cache's calls on this device (littlebit_device_status).
__device__ unsigned int g_status;

std::atomic<unsigned int*> g_status_addr[lb::kMaxDevices];

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

int elem_bytes(lb_dtype dt) { return dt == LB_F32 ? 4 : dt == LB_I8 ? 1 : 2; }

lb_status launched(cudaError_t e) { return e == cudaSuccess ? LB_OK : lb::cuda_fail(e); }

// ------------------------------------------------------------------ rows

// One side of a row tensor, in bytes.  Token rows: stride_row = 0 and
// stride_major per token.  Rows of pages: stride_major per page, stride_row
// per row of the page.
struct Side {
  unsigned char* data;
  long long stride_major, stride_row, stride_head;
  int paged;
};
struct RowJob {
  Side src, dst;
  int units;         // units of one row: a unit is 16 bytes, or the two 16-byte halves of eight pairs
  lb::Divisor by_units;
  int rot_units;     // the first rot_units of them are rotated
  unsigned first;    // first item of the job within a token
};
struct RowArgs {
  RowJob job[kMaxJobs];
  int n_jobs, n_tokens, per_block;   // per_block: tokens of one block
  unsigned items;                    // items of one token, over all jobs
  lb::Divisor by_items, by_half;
  int page_shift;
  long long n_rows;                  // rows of the cache (bound of where)
  const long long* where;
  const int* positions;
  const uint64_t* phases;
  int half;                          // pairs per head (0: nothing is rotated)
  int interleaved, inverse;
  float scale;
};

template <class T> __device__ __forceinline__ float to_f(T v);
template <> __device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
template <> __device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <> __device__ __forceinline__ float to_f(float v) { return v; }
template <class T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ __half from_f(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ float from_f(float v) { return v; }

template <class T>
union Chunk {
  uint4 u;
  T e[16 / sizeof(T)];
};

__device__ __forceinline__ unsigned char* side_at(const Side& s, int t, long long w, int shift) {
  return s.data + (s.paged ? (w >> shift) * s.stride_major + (w & ((1ll << shift) - 1)) * s.stride_row
                           : (long long)t * s.stride_major);
}

// What one item of the kernel is.
struct Item {
  unsigned char* dst;      // null: nothing to do
  int unit, rot, second;   // second: bytes from the first chunk to the pair's second (0: one chunk)
  int token;               // within the block
};

// Mathematics: (a, b) -> (a cos - b sin, b cos + a sin).  The angle in turns
// is pos * phase / 2^64 modulo 1: an integer product that wraps exactly, so
// the fp32 argument of sincospi is within half a step of the true angle at
// every position.
//
// A block takes per_block tokens.  Its threads first put cos and sin of the
// tokens' pairs into shared memory (once for all heads of all tensors), with
// the loads of their first items already under way; then each item is one or
// two 16-byte loads, the rotation in fp32, and as many stores.  One item a
// thread at a time: eight blocks an SM hide the latency, and two or four items
// a thread cost more in registers than they bring (a rotary prompt of 2048
// tokens x 72 heads, bf16: 18.5 us with one, 19.8 with two, 33 with four).  4096
// tokens of 64 + 8 + 8 heads written: 31 us, 5.4 TB/s, 82 % of the copy rate (33
// in runs of seconds, under the power cap).
template <class T>
__global__ void __launch_bounds__(256) rows_kernel(const __grid_constant__ RowArgs a) {
  constexpr int E = 16 / sizeof(T);
  extern __shared__ float2 turn[];   // [per_block][half]
  lb::dependent_begin();
  const int t0 = blockIdx.x * a.per_block;
  const int n_tok = min(a.per_block, a.n_tokens - t0);
  const int total = (int)a.items * n_tok, step = gridDim.y * blockDim.x;

  Item o;
  Chunk<T> x, y;
  // item i of the block: where it is, and its loads
  auto begin = [&](int i) {
    o.dst = nullptr;
    if (i >= total) return;
    o.token = a.per_block > 1 ? a.by_items(i) : 0;
    const int r = i - o.token * (int)a.items;
    int j = 0;
    while (j + 1 < a.n_jobs && r >= (int)a.job[j + 1].first) ++j;
    const RowJob& J = a.job[j];
    const int k = r - (int)J.first;
    const int head = J.by_units(k);
    o.unit = k - head * J.units;
    o.rot = o.unit < J.rot_units;
    // half layout: rotated units hold two chunks half a rotary width apart
    const int halves = J.rot_units > 0 && !a.interleaved;
    const int chunk = halves && !o.rot ? o.unit + J.rot_units : o.unit;
    o.second = halves && o.rot ? J.rot_units * 16 : 0;
    const int t = t0 + o.token;
    long long w = 0;
    if (J.src.paged || J.dst.paged) {
      w = a.where[t];
      if (w < 0 || w >= a.n_rows) {
        if (w != -1) atomicOr(&g_status, kStatusIndex);
        return;
      }
    }
    const unsigned char* src = side_at(J.src, t, w, a.page_shift) + (long long)head * J.src.stride_head + 16 * chunk;
    o.dst = side_at(J.dst, t, w, a.page_shift) + (long long)head * J.dst.stride_head + 16 * chunk;
    x.u = *reinterpret_cast<const uint4*>(src);
    if (o.second) y.u = *reinterpret_cast<const uint4*>(src + o.second);
  };
  auto finish = [&]() {
    if (!o.dst) return;
    if (o.rot) {
      const float2* cs = turn + o.token * a.half;
      if (a.interleaved) {
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          const float2 w = cs[(o.unit * E + e) >> 1];
          const float p = to_f(x.e[e]), q = to_f(x.e[e + 1]);
          x.e[e] = from_f<T>(p * w.x - q * w.y);
          x.e[e + 1] = from_f<T>(q * w.x + p * w.y);
        }
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float2 w = cs[o.unit * E + e];
          const float p = to_f(x.e[e]), q = to_f(y.e[e]);
          x.e[e] = from_f<T>(p * w.x - q * w.y);
          y.e[e] = from_f<T>(q * w.x + p * w.y);
        }
      }
    }
    *reinterpret_cast<uint4*>(o.dst) = x.u;
    if (o.second) *reinterpret_cast<uint4*>(o.dst + o.second) = y.u;
  };

  int it = blockIdx.y * blockDim.x + threadIdx.x;
  begin(it);
  if (a.half) {
    for (int i = threadIdx.x; i < n_tok * a.half; i += blockDim.x) {
      const int t = a.by_half(i);
      // signed fraction of a turn in 64 bits; times 2^-63: the argument of sincospi
      const long long f = (long long)((uint64_t)(long long)a.positions[t0 + t] * a.phases[i - t * a.half]);
      float s, c;
      sincospif((float)f * 0x1p-63f, &s, &c);
      turn[i] = make_float2(c * a.scale, (a.inverse ? -s : s) * a.scale);
    }
    __syncthreads();
  }
  for (; it < total; begin(it)) {
    finish();
    it += step;
  }
}

// ------------------------------------------------------------------ block scan

// Exclusive sum over the block (kBookThreads threads) and its total.
__device__ __forceinline__ int block_scan(int v, int& total, int* warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  __syncthreads();   // warp_sums may still be read from the last call
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  int w = warp_sums[lane];   // kBookThreads / 32 == 32 entries
  int s = w;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, s, d);
    if (lane >= d) s += y;
  }
  total = __shfl_sync(0xffffffffu, s, 31);
  return x - v + __shfl_sync(0xffffffffu, s - w, warp);
}

// Walks refs[] for free pages in ascending order and calls take(rank, page)
// for the ranks below `want`; returns how many were found (at most want).
template <class F>
__device__ __forceinline__ int take_free(const int* refs, int n_pages, int want, int* warp_sums, F take) {
  int found = 0;
  for (int base = 0; base < n_pages && found < want; base += 4 * kBookThreads) {
    const int p0 = base + 4 * (int)threadIdx.x;
    unsigned free4 = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (p0 + i < n_pages && refs[p0 + i] == 0) free4 |= 1u << i;
    int total;
    int rank = found + block_scan(__popc(free4), total, warp_sums);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (free4 >> i & 1u) {
        if (rank < want) take(rank, p0 + i);
        ++rank;
      }
    found += total;
    __syncthreads();
  }
  return min(found, want);
}

// Exclusive sums of need[0..n) in place; returns the total.
__device__ __forceinline__ int scan_list(int* need, int n, int* warp_sums) {
  int base = 0;
  for (int i0 = 0; i0 < n; i0 += kBookThreads) {
    const int i = i0 + (int)threadIdx.x;
    int total;
    const int e = block_scan(i < n ? need[i] : 0, total, warp_sums);
    if (i < n) need[i] = base + e;
    base += total;
  }
  __syncthreads();
  return base;
}

// The last i in [0, n) with off[i] <= r (off ascending, off[0] = 0).
__device__ __forceinline__ int owner_of(const int* off, int n, int r) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (off[mid] <= r) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

struct Tables {
  int* table;
  long long table_stride;
  int* length;
  int* refs;
  int n_pages, page_size, page_shift, n_slots, max_pages;
};

__device__ __forceinline__ int pages_of(int tokens, const Tables& c) {
  return (int)(((long long)tokens + c.page_size - 1) >> c.page_shift);
}

// Token t's place among the list's sequences: the sequence and its first token, or -1.
__device__ __forceinline__ int sequence_of(const int* starts, int n, int n_tokens, int t, int& first) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (starts[mid] <= t) lo = mid;
    else hi = mid - 1;
  }
  first = min(max(starts[lo], 0), n_tokens);
  return t >= first && t < starts[lo + 1] ? lo : -1;
}

// A slot named twice: the first entry of the list wins.  Claims are made in
// length[] itself (a claimed slot holds -(n - i), the smallest for the first
// entry) and replaced by the real length before the kernel ends, so no scratch
// has to be kept clean between calls.
__device__ __forceinline__ int claim_value(int n, int i) { return -(n - i); }

// ------------------------------------------------------------------ extend

__global__ void __launch_bounds__(kBookThreads, 1)
    extend_kernel(const Tables c, const int* slots, const int* starts, int n, int n_tokens, int prefix, long long* where,
                  int* positions) {
  extern __shared__ int sm[];
  int* s_start = sm;              // [n + 1]
  int* s_len = s_start + n + 1;   // [n] tokens before the call; -1: not extended
  int* s_off = s_len + n;         // [n] new pages, then those of the sequences before
  int* s_slot = s_off + n;        // [n]
  __shared__ int warp_sums[32];
  const int tid = threadIdx.x;
  lb::dependent_begin();
  for (int i = tid; i <= n; i += kBookThreads) s_start[i] = starts[i];
  __syncthreads();
  auto count = [&](int i) {
    const int a = min(max(s_start[i], 0), n_tokens), b = min(max(s_start[i + 1], a), n_tokens);
    return b - a;
  };
  unsigned bad = 0;
  for (int i = tid; i < n; i += kBookThreads) {
    const int s = slots[i];
    const int a = s_start[i], b = s_start[i + 1];
    if (a < 0 || b < a || b > n_tokens) bad |= kStatusIndex;
    int len = -1;
    if (s >= 0 && s < c.n_slots) {
      len = c.length[s];
      const int rest = len & (c.page_size - 1);
      if (len < 0 || pages_of(len, c) > c.max_pages) {
        len = -1;
        bad |= kStatusIndex;
      } else if (rest && count(i)) {   // the rows to come lie in the last page: it has to be this slot's own
        const int p = c.table[s * c.table_stride + (len >> c.page_shift)];
        if (p < 0 || p >= c.n_pages || c.refs[p] != 1) {
          len = -1;
          bad |= kStatusIndex;
        }
      }
    } else if (s != -1) {
      bad |= kStatusIndex;
    }
    s_slot[i] = s;
    s_len[i] = len;
  }
  __syncthreads();
  for (int i = tid; i < n; i += kBookThreads)
    if (s_len[i] >= 0) atomicMin(&c.length[s_slot[i]], claim_value(n, i));
  __syncthreads();
  for (int i = tid; i < n; i += kBookThreads) {
    int need = 0;
    if (s_len[i] >= 0) {
      if (c.length[s_slot[i]] != claim_value(n, i)) {
        s_len[i] = -1;
        bad |= kStatusIndex;
      } else {
        const long long want = ((long long)s_len[i] + count(i) + c.page_size - 1) >> c.page_shift;
        if (want > c.max_pages) {
          c.length[s_slot[i]] = s_len[i];
          s_len[i] = -1;
          bad |= kStatusPages;
        } else {
          need = (int)want - pages_of(s_len[i], c);
        }
      }
    }
    s_off[i] = need;
  }
  __syncthreads();
  auto take = [&](int want) {
    return take_free(c.refs, c.n_pages, want, warp_sums, [&](int rank, int page) {
      const int i = owner_of(s_off, n, rank);
      c.table[s_slot[i] * c.table_stride + pages_of(s_len[i], c) + rank - s_off[i]] = page;
      c.refs[page] = 1;
    });
  };
  const int want = scan_list(s_off, n, warp_sums), found = take(want);
  if (found < want) {
    // Too few: all are given back, the sequences that do not fit what those before them leave are refused, one after
    // another (rare; 166 us for 4096), and the others take theirs.
    __syncthreads();
    for (int i = tid; i < n; i += kBookThreads) {
      if (s_len[i] < 0) continue;
      const int need = (i + 1 < n ? s_off[i + 1] : want) - s_off[i];
      for (int k = 0; k < need && s_off[i] + k < found; ++k) {
        int* e = &c.table[s_slot[i] * c.table_stride + pages_of(s_len[i], c) + k];
        c.refs[*e] = 0;
        *e = -1;
      }
    }
    __syncthreads();
    for (int i = tid; i < n; i += kBookThreads)
      s_off[i] = s_len[i] < 0 ? 0 : pages_of(s_len[i] + count(i), c) - pages_of(s_len[i], c);
    __syncthreads();
    if (tid == 0) {
      int left = found;
      for (int i = 0; i < n; ++i) {
        if (s_off[i] <= left) {
          left -= s_off[i];
        } else {
          c.length[s_slot[i]] = s_len[i];
          s_len[i] = -1;
          s_off[i] = 0;
          bad |= kStatusPages;
        }
      }
    }
    __syncthreads();
    take(scan_list(s_off, n, warp_sums));
  }
  __syncthreads();
  for (int i = tid; i < n; i += kBookThreads)
    if (s_len[i] >= 0) c.length[s_slot[i]] = s_len[i] + count(i);
  __syncthreads();
  int shift = 0;
  if (prefix >= 0) shift = max(c.length[prefix], 0);
  for (int t = tid; t < n_tokens; t += kBookThreads) {
    int first;
    const int i = sequence_of(s_start, n, n_tokens, t, first);
    long long w = -1;
    int p = -1;
    if (i >= 0 && s_len[i] >= 0) {
      const int at = s_len[i] + t - first;
      const int page = c.table[s_slot[i] * c.table_stride + (at >> c.page_shift)];
      w = (long long)page * c.page_size + (at & (c.page_size - 1));
      p = at + shift;
    }
    where[t] = w;
    positions[t] = p;
  }
  if (bad) atomicOr(&g_status, bad);
}

__global__ void __launch_bounds__(256)
    locate_kernel(const Tables c, const int* slots, const int* starts, const int* begin, int n, int n_tokens, int prefix,
                  long long* where, int* positions) {
  lb::dependent_begin();
  const int t = blockIdx.x * blockDim.x + threadIdx.x;
  for (int i = t; i < n; i += gridDim.x * blockDim.x)
    if (starts[i] < 0 || starts[i + 1] < starts[i] || starts[i + 1] > n_tokens) atomicOr(&g_status, kStatusIndex);
  if (t >= n_tokens) return;
  int first;
  const int i = sequence_of(starts, n, n_tokens, t, first);
  long long w = -1;
  int p = -1;
  if (i >= 0 && slots[i] != -1) {
    const int s = slots[i];
    bool ok = s >= 0 && s < c.n_slots;
    const long long at = (long long)t - first + (begin ? begin[i] : 0);
    if (ok) ok = at >= 0 && at < c.length[s] && (at >> c.page_shift) < c.max_pages;
    if (ok) {
      const int page = c.table[s * c.table_stride + (at >> c.page_shift)];
      ok = page >= 0 && page < c.n_pages;
      if (ok) {
        w = (long long)page * c.page_size + (at & (c.page_size - 1));
        p = (int)at + (prefix >= 0 ? max(c.length[prefix], 0) : 0);
      }
    }
    if (!ok) atomicOr(&g_status, kStatusIndex);
  }
  where[t] = w;
  positions[t] = p;
}

__global__ void __launch_bounds__(128) free_kernel(const Tables c, const int* slots) {
  lb::dependent_begin();
  const int s = slots[blockIdx.x];
  if (s < 0 || s >= c.n_slots) {
    if (s != -1 && threadIdx.x == 0) atomicOr(&g_status, kStatusIndex);
    return;
  }
  __shared__ int held;
  if (threadIdx.x == 0) held = atomicExch(&c.length[s], 0);   // the first of two entries gets it
  __syncthreads();
  const int n = min(pages_of(max(held, 0), c), c.max_pages);
  for (int k = threadIdx.x; k < n; k += blockDim.x) {
    int* e = &c.table[s * c.table_stride + k];
    const int p = *e;
    *e = -1;
    if (p < 0 || p >= c.n_pages || atomicSub(&c.refs[p], 1) <= 0) {
      if (p >= 0 && p < c.n_pages) atomicAdd(&c.refs[p], 1);
      atomicOr(&g_status, kStatusIndex);
    }
  }
}

// ------------------------------------------------------------------ page copies

struct PlaneDev {
  unsigned char* data;
  long long stride_page, stride_head, stride_row;   // bytes
  int heads, row_chunks;                            // 16-byte chunks of a row
};
struct CopyArgs {
  PlaneDev plane[kPlaneBatch];
  int n_planes, page_size;
  int by_warp;   // an item is a warp's, not a block's
};
struct CopyJob {
  int src, dst, rows, aux;
};

// Copies the first job.rows rows of page job.src to page job.dst in every
// plane.  An item is one (job, plane); gridDim.y blocks share it, or, where the
// pages are small and many, it is one warp's, so that a thread has work for its
// four loads under way (64 children x 64 planes of 12 KB pages: 13.9 us as
// blocks' items, 12.8 as warps').  Rows that follow one another in memory are
// copied as one run, so a whole page of a plain tensor is one run of all its
// heads.  Bound by HBM for large pages (about 470 of 2048 pages moved in 16 planes
// of 64 KB pages: 169 us, 5.7 TB/s), by latency for few items.
template <class F>
__device__ __forceinline__ void copy_items(const CopyArgs& a, int count, F job_at) {
  // blocks of 256 threads: eight workers of a warp, or one
  const int items = count * a.n_planes, per = a.by_warp ? 32 : 256, workers = a.by_warp ? 8 : 1;
  const int lane = threadIdx.x & (per - 1), worker = a.by_warp ? threadIdx.x >> 5 : 0;
  for (int item = blockIdx.x * workers + worker; item < items; item += gridDim.x * workers) {
    const CopyJob job = job_at(item / a.n_planes);
    if (job.dst < 0) continue;
    const PlaneDev& P = a.plane[item % a.n_planes];
    const unsigned char* src = P.data + job.src * P.stride_page;
    unsigned char* dst = P.data + job.dst * P.stride_page;
    int run = P.row_chunks, per_head = job.rows;   // chunks of a run, runs of a head
    if (P.stride_row == 16ll * P.row_chunks) {
      run *= job.rows;
      per_head = 1;
      if (job.rows == a.page_size && P.stride_head == 16ll * run) run *= P.heads;
    }
    const int total = P.heads * job.rows * P.row_chunks;
    auto offset = [&](int c) -> long long {
      const int r = c / run;
      const int h = r / per_head;
      return h * P.stride_head + (r - h * per_head) * P.stride_row + 16ll * (c - r * run);
    };
    const int step = gridDim.y * per;
    int c = blockIdx.y * per + lane;
    for (; c + 3 * step < total; c += 4 * step) {
      long long o[4];
      uint4 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        o[i] = offset(c + i * step);
        v[i] = *reinterpret_cast<const uint4*>(src + o[i]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4*>(dst + o[i]) = v[i];
    }
    for (; c < total; c += step) {
      const long long o = offset(c);
      *reinterpret_cast<uint4*>(dst + o) = *reinterpret_cast<const uint4*>(src + o);
    }
  }
}

// ------------------------------------------------------------------ fork

// A child's part of a fork: parent slot and tokens held (child slot -1: left out), and the copy of the last page.
struct ForkJob {
  int parent, child, tokens, pad;
};

__global__ void __launch_bounds__(kBookThreads, 1)
    fork_kernel(const Tables c, const int* parents, const int* children, int n, ForkJob* fork, CopyJob* copy) {
  extern __shared__ int sm[];
  int* s_len = sm;            // [n] tokens of the parent; -1: left out
  int* s_off = s_len + n;     // [n]
  int* s_child = s_off + n;   // [n]
  int* s_last = s_child + n;  // [n] the parent's partly filled last page
  __shared__ int warp_sums[32];
  const int tid = threadIdx.x;
  lb::dependent_begin();
  unsigned bad = 0;
  for (int i = tid; i < n; i += kBookThreads) {
    const int p = parents[i], ch = children[i];
    int len = -1, last = -1;
    if (p == -1 || ch == -1) {
      ;   // padding
    } else if (p < 0 || p >= c.n_slots || ch < 0 || ch >= c.n_slots || p == ch) {
      bad |= kStatusIndex;
    } else {
      len = c.length[p];
      const bool lost = len < 0 || pages_of(len, c) > c.max_pages;
      if (!lost && (len & (c.page_size - 1))) last = c.table[p * c.table_stride + (len >> c.page_shift)];
      const bool outside = last < 0 ? len & (c.page_size - 1) : last >= c.n_pages;
      if (lost || c.length[ch] != 0 || outside) {
        len = -1;
        bad |= kStatusIndex;
      }
    }
    s_len[i] = len;
    s_last[i] = last;
    s_child[i] = ch;
    copy[i] = CopyJob{-1, -1, 0, 0};
  }
  __syncthreads();
  for (int i = tid; i < n; i += kBookThreads)
    if (s_len[i] >= 0) atomicMin(&c.length[s_child[i]], claim_value(n, i));
  __syncthreads();
  for (int i = tid; i < n; i += kBookThreads) {
    if (s_len[i] >= 0 && c.length[s_child[i]] != claim_value(n, i)) {
      s_len[i] = -1;
      bad |= kStatusIndex;
    }
    s_off[i] = s_len[i] >= 0 && (s_len[i] & (c.page_size - 1)) ? 1 : 0;
  }
  __syncthreads();
  const int want = scan_list(s_off, n, warp_sums);
  const int found = take_free(c.refs, c.n_pages, want, warp_sums, [&](int rank, int page) {
    const int i = owner_of(s_off, n, rank);
    const int full = s_len[i] >> c.page_shift;
    c.refs[page] = 1;
    c.table[s_child[i] * c.table_stride + full] = page;
    copy[i] = CopyJob{s_last[i], page, s_len[i] & (c.page_size - 1), 0};
  });
  __syncthreads();
  for (int i = tid; i < n; i += kBookThreads) {
    ForkJob f{-1, -1, 0, 0};
    if (s_len[i] >= 0) {
      const int need = (i + 1 < n ? s_off[i + 1] : want) - s_off[i];
      if (need > 0 && s_off[i] >= found) {
        c.length[s_child[i]] = 0;
        bad |= kStatusPages;
      } else {
        c.length[s_child[i]] = s_len[i];
        f = ForkJob{parents[i], s_child[i], s_len[i], 0};
      }
    }
    fork[i] = f;
  }
  if (bad) atomicOr(&g_status, bad);
}

// Blocks y = 0 first share out the children's table rows, then all copy the last pages.
__global__ void __launch_bounds__(256)
    fork_copy_kernel(const __grid_constant__ CopyArgs a, const Tables c, const ForkJob* fork, const CopyJob* copy, int n,
                     int with_tables) {
  lb::dependent_begin();
  if (with_tables && blockIdx.y == 0)
    for (int i = blockIdx.x; i < n; i += gridDim.x) {
      const ForkJob f = fork[i];
      if (f.child < 0) continue;
      const int full = f.tokens >> c.page_shift;
      for (int k = threadIdx.x; k < full; k += blockDim.x) {
        const int p = c.table[f.parent * c.table_stride + k];
        c.table[f.child * c.table_stride + k] = p;
        if (p >= 0 && p < c.n_pages) atomicAdd(&c.refs[p], 1);
        else atomicOr(&g_status, kStatusIndex);
      }
    }
  copy_items(a, n, [&](int i) { return copy[i]; });
}

// ------------------------------------------------------------------ compact

__global__ void __launch_bounds__(kBookThreads, 1)
    compact_kernel(const Tables c, int* refs_out, int* count_out, CopyJob* jobs, int* moved, int* n_jobs) {
  __shared__ int warp_sums[32];
  const int tid = threadIdx.x;
  lb::dependent_begin();
  int live = 0;
  for (int p = tid; p < c.n_pages; p += kBookThreads) live += c.refs[p] > 0;
  int count;
  block_scan(live, count, warp_sums);
  int movers = 0, holes = 0;
  for (int base = 0; base < c.n_pages; base += 4 * kBookThreads) {
    const int p0 = base + 4 * tid;
    int r[4];
    int packed = 0;   // movers in the high half, holes in the low half (at most 4096 each)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      r[i] = p0 + i < c.n_pages ? c.refs[p0 + i] : 0;
      if (p0 + i < c.n_pages) packed += r[i] > 0 ? (p0 + i >= count) << 16 : (p0 + i < count);
    }
    int total;
    const int e = block_scan(packed, total, warp_sums);
    int m = movers + (e >> 16), h = holes + (e & 0xffff);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int p = p0 + i;
      if (p >= c.n_pages) break;
      if (r[i] > 0 && p >= count) {
        jobs[m].src = p;
        jobs[m].rows = c.page_size;
        jobs[m].aux = r[i];
        ++m;
        refs_out[p] = 0;
      } else if (r[i] > 0) {
        refs_out[p] = r[i];
      } else if (p < count) {
        jobs[h++].dst = p;
      } else {
        refs_out[p] = 0;
        moved[p] = p;
      }
    }
    movers += total >> 16;
    holes += total & 0xffff;
  }
  __syncthreads();
  for (int k = tid; k < movers; k += kBookThreads) {
    refs_out[jobs[k].dst] = jobs[k].aux;
    moved[jobs[k].src] = jobs[k].dst;
  }
  if (tid == 0) {
    *count_out = count;
    *n_jobs = movers;
  }
}

__global__ void __launch_bounds__(256)
    compact_copy_kernel(const __grid_constant__ CopyArgs a, const Tables c, int* table_out, const int* count,
                        const CopyJob* jobs, const int* moved, const int* n_jobs, int with_tables) {
  lb::dependent_begin();
  if (with_tables) {
    const int live = *count;
    const long long n = (long long)c.n_slots * c.max_pages;
    const long long step = (long long)gridDim.x * gridDim.y * blockDim.x;
    for (long long i = ((long long)blockIdx.y * gridDim.x + blockIdx.x) * blockDim.x + threadIdx.x; i < n; i += step) {
      const long long at = i / c.max_pages * c.table_stride + i % c.max_pages;
      const int p = c.table[at];
      table_out[at] = p >= live && p < c.n_pages ? moved[p] : p;
    }
  }
  copy_items(a, *n_jobs, [&](int i) { return jobs[i]; });
}

__global__ void __launch_bounds__(256)
    copy_kernel(const __grid_constant__ CopyArgs a, const int* src, const int* dst, int n, int n_pages) {
  lb::dependent_begin();
  copy_items(a, n, [&](int i) {
    CopyJob j{src[i], dst[i], a.page_size, 0};
    if (j.src == -1 && j.dst == -1) return j;   // padding
    if (j.src < 0 || j.src >= n_pages || j.dst < 0 || j.dst >= n_pages) {
      if ((threadIdx.x & 31) == 0) atomicOr(&g_status, kStatusIndex);   // an item may be any warp's
      j.dst = -1;
    }
    return j;
  });
}

// ------------------------------------------------------------------ host

lb_status check_plane(const lb_cache& c, const lb_plane& P) {
  if (!P.data) return LB_ERR_ARG;
  if (P.dt != LB_F16 && P.dt != LB_BF16 && P.dt != LB_F32 && P.dt != LB_I8) return LB_ERR_ARG;
  if (P.heads < 1 || P.width < 1 || P.heads > 4096 || P.width > 65536) return LB_ERR_SHAPE;
  const int64_t b = elem_bytes(P.dt);
  if (P.stride_page < 0 || P.stride_head < 0 || P.stride_row < 0) return LB_ERR_SHAPE;
  if ((int64_t)P.heads * c.page_size * P.width * b >= (int64_t)1 << 31) return LB_ERR_SHAPE;
  if (!aligned16(P.data) || (P.width * b) % 16 || (P.stride_page * b) % 16 || (P.stride_head * b) % 16 ||
      (P.stride_row * b) % 16)
    return LB_ERR_ALIGN;
  return LB_OK;
}

lb_status check_rows(const lb_rows& r, lb_dtype dt) {
  if (!r.data) return LB_ERR_ARG;
  if (r.heads < 1 || r.width < 1 || r.heads > 4096 || r.width > 65536) return LB_ERR_SHAPE;
  const int64_t b = elem_bytes(dt);
  if (!aligned16(r.data) || (r.width * b) % 16 || (r.stride_token * b) % 16 || (r.stride_head * b) % 16)
    return LB_ERR_ALIGN;
  return LB_OK;
}

int log2_of(int v) {
  int s = 0;
  while ((1 << s) < v) ++s;
  return s;
}

Tables tables_of(const lb_cache& c) {
  return Tables{c.table, c.table_stride, c.length, c.refs, c.n_pages, c.page_size, log2_of(c.page_size), c.n_slots,
                c.max_pages};
}

CopyArgs planes_of(const lb_cache& c, int begin) {
  CopyArgs a;
  a.n_planes = std::min(kPlaneBatch, c.n_planes - begin);
  a.page_size = c.page_size;
  for (int i = 0; i < a.n_planes; ++i) {
    const lb_plane& P = c.planes[begin + i];
    const int64_t b = elem_bytes(P.dt);
    a.plane[i] = PlaneDev{static_cast<unsigned char*>(P.data), P.stride_page * b, P.stride_head * b,
                          P.stride_row * b, P.heads, (int)(P.width * b / 16)};
  }
  return a;
}

// Grid of a page copy: y blocks share an item (32 KB or more each, so that
// small pages are not cut up), and x covers the items up to eight blocks an SM.
// Where there may be more items than that, pages of up to 16 KB are a warp's.
dim3 copy_grid(CopyArgs& a, int64_t jobs, int page_size) {
  int64_t most = 1;
  for (int i = 0; i < a.n_planes; ++i)
    most = std::max(most, (int64_t)a.plane[i].heads * a.plane[i].row_chunks * page_size);
  const int y = (int)std::min<int64_t>(8, std::max<int64_t>(1, most / 2048));
  a.by_warp = most <= 1024 && jobs * a.n_planes > 148 * 8;
  const int64_t x = std::min<int64_t>(a.by_warp ? (jobs * a.n_planes + 7) / 8 : jobs * a.n_planes, 148 * 8 / y);
  return dim3((unsigned)std::max<int64_t>(1, x), (unsigned)y);
}

template <class K>
cudaError_t allow_smem(K kern, lb::PerDevice& slot, int bytes) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  int v = 0;
  return static_cast<cudaError_t>(slot.get(dev, v, [&](int& out) -> int {
    const cudaError_t r = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    out = 1;
    return r;
  }));
}

template <class T>
lb_status launch_rows_of(const RowArgs& a, cudaStream_t st) {
  const int x = lb::ceil_div(a.n_tokens, a.per_block);
  // blocks that share a group's items: four blocks an SM, four a group at least, none without work
  const int64_t need = ((int64_t)a.items * a.per_block + 255) / 256;
  const int y = (int)std::min<int64_t>(std::min<int64_t>(need, 1024), std::max(a.per_block, 148 * 4 / x));
  return launched(lb::launch_dependent_on(st, rows_kernel<T>, dim3(x, y), 256,
                                          (size_t)a.per_block * a.half * sizeof(float2), a));
}

// Fills and launches rows_kernel.
struct RowLaunch {
  RowArgs a;
  lb_dtype dt;

  RowLaunch(int n_tokens, lb_dtype t) : a{}, dt(t) { a.n_tokens = n_tokens; }

  static Side tokens(const lb_rows& r, lb_dtype dt) {
    const int64_t b = elem_bytes(dt);
    return Side{static_cast<unsigned char*>(r.data), r.stride_token * b, 0, r.stride_head * b, 0};
  }
  static Side paged(const lb_plane& P) {
    const int64_t b = elem_bytes(P.dt);
    return Side{static_cast<unsigned char*>(P.data), P.stride_page * b, P.stride_row * b, P.stride_head * b, 1};
  }
  // rotary_dim 0: the rows are moved as they are
  void add(const Side& src, const Side& dst, int heads, int width, int rotary_dim) {
    const int E = 16 / elem_bytes(dt);
    RowJob& J = a.job[a.n_jobs++];
    J.src = src;
    J.dst = dst;
    J.rot_units = rotary_dim / (a.interleaved ? 1 : 2) / E;
    J.units = J.rot_units + (width - rotary_dim) / E;
    J.by_units = lb::divisor(J.units);
    J.first = a.items;
    a.items += (unsigned)heads * (unsigned)J.units;
  }
  void rope(const lb_rotary& r, const int32_t* positions, int inverse) {
    a.phases = r.phases;
    a.half = r.rotary_dim / 2;
    a.interleaved = r.interleaved;
    a.scale = r.scale;
    a.positions = positions;
    a.inverse = inverse;
  }
  void pages(const lb_cache& c, const int64_t* where) {
    a.page_shift = log2_of(c.page_size);
    a.n_rows = (long long)c.n_pages * c.page_size;
    a.where = reinterpret_cast<const long long*>(where);
  }
  lb_status launch(cudaStream_t st) {
    // four tokens share a block's set-up when that leaves blocks enough (4096 tokens written: 30.9 us, 31.6 with one)
    a.per_block = a.n_tokens >= 148 * 4 ? 4 : 1;
    a.by_items = lb::divisor((int)a.items);
    a.by_half = lb::divisor(std::max(a.half, 1));
    switch (dt) {
      case LB_F16: return launch_rows_of<__half>(a, st);
      case LB_BF16: return launch_rows_of<__nv_bfloat16>(a, st);
      default: return launch_rows_of<float>(a, st);
    }
  }
};

bool row_dtype(lb_dtype dt) { return dt == LB_F16 || dt == LB_BF16 || dt == LB_F32; }

lb_status check_rope(const lb_rotary* r, const int32_t* positions) {
  if (!r || !r->phases || !positions || (r->interleaved != 0 && r->interleaved != 1)) return LB_ERR_ARG;
  if (r->rotary_dim < 16 || r->rotary_dim % 16 || r->rotary_dim > 1024) return LB_ERR_SHAPE;
  return LB_OK;
}

}  // namespace

namespace lb {

lb_status check_cache(const lb_cache* c) {
  if (!c || !c->planes || !c->table || !c->length || !c->refs) return LB_ERR_ARG;
  if (c->n_planes < 1 || c->n_planes > kMaxPlanes || c->n_pages < 1 || c->n_slots < 1 || c->max_pages < 1)
    return LB_ERR_SHAPE;
  if (c->page_size < 8 || c->page_size > 1024 || (c->page_size & (c->page_size - 1))) return LB_ERR_SHAPE;
  // token counts of a slot and row numbers within a plane's head fit 31 bits
  if ((int64_t)c->max_pages * c->page_size >= (int64_t)1 << 31 || c->table_stride < c->max_pages) return LB_ERR_SHAPE;
  return LB_OK;
}

lb_status check_list(const lb_cache* c, const void* slots, const void* starts, int n, int n_tokens, int prefix) {
  if (!slots || !starts) return LB_ERR_ARG;
  if (n < 1 || n > kMaxList || n_tokens < 0) return LB_ERR_SHAPE;
  if (prefix < -1 || prefix >= c->n_slots) return LB_ERR_ARG;
  return LB_OK;
}

lb_status check_cache_plane(const lb_cache* c, int i) {
  if (i < 0 || i >= c->n_planes) return LB_ERR_ARG;
  return check_plane(*c, c->planes[i]);
}

lb_status check_token_rows(const lb_rows* r, lb_dtype dt) { return r ? check_rows(*r, dt) : LB_ERR_ARG; }

unsigned int* cache_status_word(int dev) {
  return dev < 0 || dev >= kMaxDevices ? nullptr : g_status_addr[dev].load(std::memory_order_acquire);
}

cudaError_t touch_cache_status(unsigned int** word) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  unsigned int* w = cache_status_word(dev);
  if (!w) {
    void* p = nullptr;
    e = cudaGetSymbolAddress(&p, g_status);
    if (e != cudaSuccess) return e;
    w = static_cast<unsigned int*>(p);
    if (dev < kMaxDevices) g_status_addr[dev].store(w, std::memory_order_release);
  }
  if (word) *word = w;
  return cudaSuccess;
}

}  // namespace lb

using lb::check_cache;
using lb::check_list;

extern "C" {

lb_status littlebit_rotary_phases(int rotary_dim, double base, double factor, double original, double slow,
                                  double fast, int log_ramp, uint64_t* phases) {
  if (!phases || !(base > 0) || !(factor > 0) || !std::isfinite(base) || !std::isfinite(factor)) return LB_ERR_ARG;
  if (original > 0 && (!(fast > slow) || (log_ramp && !(slow > 0)))) return LB_ERR_ARG;
  if (rotary_dim < 2 || rotary_dim % 2) return LB_ERR_SHAPE;
  const long double two_pi = 6.283185307179586476925286766559005768L;
  for (int i = 0; i < rotary_dim / 2; ++i) {
    long double turns = powl((long double)base, -2.0L * i / rotary_dim) / two_pi;   // per token
    long double keep = 0;
    if (original > 0) {
      const long double n = original * turns;
      keep = log_ramp ? (logl(n) - logl(slow)) / (logl(fast) - logl(slow)) : (n - slow) / ((long double)fast - slow);
      keep = std::min(1.0L, std::max(0.0L, keep));
    }
    turns = turns * keep + turns / factor * (1 - keep);
    turns -= floorl(turns);
    phases[i] = (uint64_t)ldexpl(turns, 64);
  }
  return LB_OK;
}

lb_status littlebit_rotary(const lb_rows* src, const lb_rows* dst, int n, int n_tokens, lb_dtype dt,
                           const int32_t* positions, const lb_rotary* rope, int inverse, void* stream) {
  if (!src || !dst || !row_dtype(dt)) return LB_ERR_ARG;
  if (n < 1 || n > kMaxJobs || n_tokens < 0) return LB_ERR_SHAPE;
  lb_status r = check_rope(rope, positions);
  if (r != LB_OK) return r;
  RowLaunch L(n_tokens, dt);
  L.rope(*rope, positions, inverse != 0);
  for (int i = 0; i < n; ++i) {
    if ((r = check_rows(src[i], dt)) != LB_OK || (r = check_rows(dst[i], dt)) != LB_OK) return r;
    if (src[i].heads != dst[i].heads || src[i].width != dst[i].width || rope->rotary_dim > src[i].width)
      return LB_ERR_SHAPE;
    L.add(RowLaunch::tokens(src[i], dt), RowLaunch::tokens(dst[i], dt), src[i].heads, src[i].width,
          rope->rotary_dim);
  }
  return n_tokens ? L.launch(static_cast<cudaStream_t>(stream)) : LB_OK;
}

lb_status littlebit_cache_extend(const lb_cache* c, const int32_t* slots, const int32_t* starts, int n, int n_tokens,
                                 int prefix, int64_t* where, int32_t* positions, void* stream) {
  lb_status r = check_cache(c);
  if (r != LB_OK || (r = check_list(c, slots, starts, n, n_tokens, prefix)) != LB_OK) return r;
  if (n_tokens && (!where || !positions)) return LB_ERR_ARG;
  static lb::PerDevice smem;
  const int most = (4 * kMaxList + 1) * (int)sizeof(int);
  cudaError_t e = lb::touch_cache_status(nullptr);
  if (e == cudaSuccess) e = allow_smem(extend_kernel, smem, most);
  if (e != cudaSuccess) return lb::cuda_fail(e);
  return launched(lb::launch_dependent_on(static_cast<cudaStream_t>(stream), extend_kernel, dim3(1), kBookThreads,
                                          (4 * n + 1) * sizeof(int), tables_of(*c), slots, starts, n, n_tokens, prefix,
                                          reinterpret_cast<long long*>(where), positions));
}

lb_status littlebit_cache_locate(const lb_cache* c, const int32_t* slots, const int32_t* starts, const int32_t* first,
                                 int n, int n_tokens, int prefix, int64_t* where, int32_t* positions, void* stream) {
  lb_status r = check_cache(c);
  if (r != LB_OK || (r = check_list(c, slots, starts, n, n_tokens, prefix)) != LB_OK) return r;
  if (!n_tokens) return LB_OK;
  if (!where || !positions) return LB_ERR_ARG;
  const cudaError_t e = lb::touch_cache_status(nullptr);
  if (e != cudaSuccess) return lb::cuda_fail(e);
  return launched(lb::launch_dependent_on(static_cast<cudaStream_t>(stream), locate_kernel,
                                          dim3(lb::ceil_div(n_tokens, 256)), 256, 0, tables_of(*c), slots, starts,
                                          first, n, n_tokens, prefix, reinterpret_cast<long long*>(where), positions));
}

lb_status littlebit_cache_write(const lb_cache* c, const int* planes, const lb_rows* rows, int n, int n_tokens,
                                const int64_t* where, const lb_rotary* rope, const int32_t* positions,
                                unsigned int rotated, const lb_rows* q, const lb_rows* q_out, void* stream) {
  lb_status r = check_cache(c);
  if (r != LB_OK) return r;
  if (!planes || !rows || !where || (q != nullptr) != (q_out != nullptr)) return LB_ERR_ARG;
  if (n < 1 || n > kMaxJobs - 1 || n_tokens < 0 || rotated >> n) return LB_ERR_SHAPE;
  if ((r = lb::check_cache_plane(c, planes[0])) != LB_OK) return r;
  const lb_dtype dt = c->planes[planes[0]].dt;
  if (!row_dtype(dt)) return LB_ERR_UNSUPPORTED;
  RowLaunch L(n_tokens, dt);
  if (rotated || q) {
    if ((r = check_rope(rope, positions)) != LB_OK) return r;
    L.rope(*rope, positions, 0);
  }
  L.pages(*c, where);
  for (int i = 0; i < n; ++i) {
    if ((r = lb::check_cache_plane(c, planes[i])) != LB_OK || (r = check_rows(rows[i], dt)) != LB_OK) return r;
    const lb_plane& P = c->planes[planes[i]];
    const int turn = rotated >> i & 1u ? rope->rotary_dim : 0;
    if (P.dt != dt) return LB_ERR_ARG;
    if (P.heads != rows[i].heads || P.width != rows[i].width || turn > P.width) return LB_ERR_SHAPE;
    L.add(RowLaunch::tokens(rows[i], dt), RowLaunch::paged(P), P.heads, P.width, turn);
  }
  if (q) {
    if ((r = check_rows(*q, dt)) != LB_OK || (r = check_rows(*q_out, dt)) != LB_OK) return r;
    if (q->heads != q_out->heads || q->width != q_out->width || rope->rotary_dim > q->width) return LB_ERR_SHAPE;
    L.add(RowLaunch::tokens(*q, dt), RowLaunch::tokens(*q_out, dt), q->heads, q->width, rope->rotary_dim);
  }
  const cudaError_t e = lb::touch_cache_status(nullptr);
  if (e != cudaSuccess) return lb::cuda_fail(e);
  return n_tokens ? L.launch(static_cast<cudaStream_t>(stream)) : LB_OK;
}

lb_status littlebit_cache_read(const lb_cache* c, const int* planes, const lb_rows* rows, int n, int n_tokens,
                               const int64_t* where, void* stream) {
  lb_status r = check_cache(c);
  if (r != LB_OK) return r;
  if (!planes || !rows || !where) return LB_ERR_ARG;
  if (n < 1 || n > kMaxJobs || n_tokens < 0) return LB_ERR_SHAPE;
  if ((r = lb::check_cache_plane(c, planes[0])) != LB_OK) return r;
  const lb_dtype dt = c->planes[planes[0]].dt;
  if (!row_dtype(dt)) return LB_ERR_UNSUPPORTED;
  RowLaunch L(n_tokens, dt);
  L.pages(*c, where);
  for (int i = 0; i < n; ++i) {
    if ((r = lb::check_cache_plane(c, planes[i])) != LB_OK || (r = check_rows(rows[i], dt)) != LB_OK) return r;
    const lb_plane& P = c->planes[planes[i]];
    if (P.dt != dt) return LB_ERR_ARG;
    if (P.heads != rows[i].heads || P.width != rows[i].width) return LB_ERR_SHAPE;
    L.add(RowLaunch::paged(P), RowLaunch::tokens(rows[i], dt), P.heads, P.width, 0);
  }
  const cudaError_t e = lb::touch_cache_status(nullptr);
  if (e != cudaSuccess) return lb::cuda_fail(e);
  return n_tokens ? L.launch(static_cast<cudaStream_t>(stream)) : LB_OK;
}

lb_status littlebit_cache_free(const lb_cache* c, const int32_t* slots, int n, void* stream) {
  const lb_status r = check_cache(c);
  if (r != LB_OK) return r;
  if (!slots) return LB_ERR_ARG;
  if (n < 1 || n > kMaxList) return LB_ERR_SHAPE;
  const cudaError_t e = lb::touch_cache_status(nullptr);
  if (e != cudaSuccess) return lb::cuda_fail(e);
  return launched(lb::launch_dependent_on(static_cast<cudaStream_t>(stream), free_kernel, dim3(n), 128, 0,
                                          tables_of(*c), slots));
}

size_t littlebit_cache_fork_work(int n) {
  return n < 1 || n > kMaxList ? 0 : (size_t)n * (sizeof(ForkJob) + sizeof(CopyJob));
}

lb_status littlebit_cache_fork(const lb_cache* c, const int32_t* parents, const int32_t* children, int n, void* work,
                               void* stream) {
  lb_status r = check_cache(c);
  if (r != LB_OK) return r;
  if (!parents || !children || !work) return LB_ERR_ARG;
  if (n < 1 || n > kMaxList) return LB_ERR_SHAPE;
  if (!aligned16(work)) return LB_ERR_ALIGN;
  for (int i = 0; i < c->n_planes; ++i)
    if ((r = check_plane(*c, c->planes[i])) != LB_OK) return r;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  ForkJob* fork = static_cast<ForkJob*>(work);
  CopyJob* copy = reinterpret_cast<CopyJob*>(fork + n);
  static lb::PerDevice smem;
  cudaError_t e = lb::touch_cache_status(nullptr);
  if (e == cudaSuccess) e = allow_smem(fork_kernel, smem, 4 * kMaxList * (int)sizeof(int));
  if (e != cudaSuccess) return lb::cuda_fail(e);
  r = launched(lb::launch_dependent_on(st, fork_kernel, dim3(1), kBookThreads, 4 * n * sizeof(int), tables_of(*c),
                                       parents, children, n, fork, copy));
  if (r != LB_OK) return r;
  for (int b = 0; b < c->n_planes; b += kPlaneBatch) {
    CopyArgs a = planes_of(*c, b);
    const dim3 grid = copy_grid(a, n, c->page_size);
    r = launched(lb::launch_dependent_on(st, fork_copy_kernel, grid, 256, 0, a, tables_of(*c),
                                         fork, copy, n, b == 0));
    if (r != LB_OK) return r;
  }
  return LB_OK;
}

size_t littlebit_cache_compact_work(int n_pages) {
  // [job count, padded][jobs: at most half of the pages move][new numbers]
  return n_pages < 1 ? 0 : 16 + ((size_t)n_pages / 2 + 1) * sizeof(CopyJob) + (size_t)n_pages * sizeof(int);
}

lb_status littlebit_cache_compact(const lb_cache* c, int32_t* table_out, int32_t* refs_out, int32_t* count,
                                  void* work, void* stream) {
  lb_status r = check_cache(c);
  if (r != LB_OK) return r;
  if (!table_out || !refs_out || !count || !work) return LB_ERR_ARG;
  if (!aligned16(work)) return LB_ERR_ALIGN;
  for (int i = 0; i < c->n_planes; ++i)
    if ((r = check_plane(*c, c->planes[i])) != LB_OK) return r;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int* n_jobs = static_cast<int*>(work);
  CopyJob* jobs = reinterpret_cast<CopyJob*>(n_jobs + 4);
  const int most = c->n_pages / 2;
  int* moved = reinterpret_cast<int*>(jobs + most + 1);
  const cudaError_t e = lb::touch_cache_status(nullptr);
  if (e != cudaSuccess) return lb::cuda_fail(e);
  r = launched(lb::launch_dependent_on(st, compact_kernel, dim3(1), kBookThreads, 0, tables_of(*c), refs_out, count,
                                       jobs, moved, n_jobs));
  if (r != LB_OK) return r;
  for (int b = 0; b < c->n_planes; b += kPlaneBatch) {
    CopyArgs a = planes_of(*c, b);
    const dim3 grid = copy_grid(a, std::max(most, 1), c->page_size);
    r = launched(lb::launch_dependent_on(st, compact_copy_kernel, grid, 256, 0,
                                         a, tables_of(*c), table_out, count, jobs, moved, n_jobs, b == 0));
    if (r != LB_OK) return r;
  }
  return LB_OK;
}

lb_status littlebit_cache_copy(const lb_cache* c, const int32_t* src, const int32_t* dst, int n, void* stream) {
  lb_status r = check_cache(c);
  if (r != LB_OK) return r;
  if (!src || !dst) return LB_ERR_ARG;
  if (n < 1 || n > 1 << 20) return LB_ERR_SHAPE;
  for (int i = 0; i < c->n_planes; ++i)
    if ((r = check_plane(*c, c->planes[i])) != LB_OK) return r;
  const cudaError_t e = lb::touch_cache_status(nullptr);
  if (e != cudaSuccess) return lb::cuda_fail(e);
  for (int b = 0; b < c->n_planes; b += kPlaneBatch) {
    CopyArgs a = planes_of(*c, b);
    const dim3 grid = copy_grid(a, n, c->page_size);
    r = launched(lb::launch_dependent_on(static_cast<cudaStream_t>(stream), copy_kernel, grid,
                                         256, 0, a, src, dst, n, c->n_pages));
    if (r != LB_OK) return r;
  }
  return LB_OK;
}

}  // extern "C"
