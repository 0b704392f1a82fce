// Attention of new tokens over the paged cache, for a batch that shares a
// prefix (littlebit.h, littlebit_cache_attend).
//
// Mathematics.  With scores s_j = scale q.k_j, o = sum_j e^{s_j} v_j / sum_j
// e^{s_j}.  Any set of keys gives a partial (m, l, O) = (max s, sum e^{s-m},
// sum e^{s-m} v), and two partials join as l = sum_p e^{m_p - M} l_p, O
// likewise.  So the keys of a row may be cut anywhere: the prefix is one set,
// handled once for the rows of all sequences, a sequence's own tokens another,
// and both are cut further to share the work out evenly.
//
// Work.  A segment is (K and V head, tile of query rows, key set), its query
// rows being (token, query head of the group) pairs, so that a K and V head is
// read once for its whole group.  A segment's extent counts what it costs: its
// key tiles, and a few units for its beginning and end.  The extents of all
// segments lie in a row of U units, and with W = ceil(U / grid) block c takes
// units [c W, (c + 1) W): every block gets the same amount of work whatever the
// lengths.  A block writes one fp32 partial for each segment that it touches,
// its rows from row R + c kRows of the work memory on, R being the rows of the
// segments before and kRows the most that a segment has (along the row of units
// R grows by a segment's rows or c by one from partial to partial, so no two
// meet), and join_kernel adds a row's partials in the order of their blocks: the
// result does not depend on timing.  The lengths are read on the device, so a
// captured graph follows a growing cache.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "lb_internal.h"

namespace {

constexpr unsigned kStatusIndex = 1u << LB_ERR_INDEX;

// How a kernel cuts its segments: query rows of a tile, keys of a tile, units
// that a segment's beginning and end are worth, units of one key tile.  A wide
// row tile, of more than 128 rows, costs two (see many_rows_kernel).  ManyCut's
// kSetup is measured: with 3, 5, 6 and 9 a batch of pieces of prompts (16 sequences
// of up to 130 tokens over a prefix of 12000, each with own keys) takes 671, 596,
// 592 and 594 us, as its short segments end late or early, and one of 48 single
// tokens over a prefix of 8192 61.4, 62.0, 61.6 and 61.9.
// `stored`: rows of a partial of a segment whose query rows end `left` from its
// first: those of a narrow tile of many_rows_kernel come in two ways, 128 apart.
struct FewCut {
  static constexpr int kRows = 16, kKeys = 64, kSetup = 1;
  static __host__ __device__ constexpr int stored(int left) { return left < 16 ? left : 16; }
};
struct ManyCut {
  static constexpr int kRows = 256, kKeys = 128, kSetup = 6;
  static __host__ __device__ constexpr int stored(int left) { return left > 256 ? 256 : left > 128 ? left : 128 + left; }
};
// Of all segments of `rows` query rows.
template <class C>
__host__ __device__ constexpr int stored_rows(int rows) {
  const int full = rows / C::kRows * C::kRows;   // kRows: a power of two
  return rows > full ? full + C::stored(rows - full) : full;
}
constexpr int kMaxUnits = 0x7fffffff;
// More stored rows than any call has (2^29 + 2^24 by its limits): sums end here, so that lists whose starts descend, and
// overlap, cannot wrap them.
constexpr int kMaxStored = 1 << 30;

using lb::Divisor;

// A plane of one cache, strides in bytes.
struct PlaneArg {
  const unsigned char* data;
  long long stride_page, stride_head, stride_row;
};

// What both the partial kernels and the join know of a launch.
struct PlanHead {
  int width;                // units of a block; 0: more units than can be counted, nothing is done
  int t0, t1;               // tokens of the batch
  int p_rows, p_rt, p_kt;   // prefix: query rows, row tiles a head, key tiles
  int p_head;               // units of one head's segments
  int pad;
};
struct SeqPlan {
  int units_before;   // units of the launch before this sequence's (the prefix's included)
  int rows_before;    // stored rows before this sequence's (the prefix's included)
  int first, count;   // tokens
  int len, before;    // see Seq
  int head;           // units of one head's segments
  int pad;
};

struct AttendArgs {
  PlaneArg k, v;
  const unsigned char* q;
  long long q_token, q_head;   // bytes
  const int* table;
  long long table_stride;
  const int* length;
  int n_pages, page_shift, n_slots, max_pages;
  const int* slots;
  const int* starts;
  int n, n_tokens, prefix;
  int heads, group;            // K and V heads; query heads of each
  Divisor by_group;
  float scale_log2;
  int do_prefix, do_own;       // which key sets this launch takes
  int after_many;              // the launch before is many_rows_kernel of the same call
  PlanHead* head;              // written by block 0 for the join
  SeqPlan* seqs;
  float2* ml;                  // [n_rows] maximum (times log2 e) and sum
  float* part;                 // [n_rows][D]
  int n_rows;                  // below kMaxStored
  unsigned* status;
};

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The larger of two, NaN if one is: a NaN score makes its row NaN, as a sum over it would be.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ uint32_t shared_addr(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// ------------------------------------------------------------------ the plan

struct Seq {
  int first, count;   // tokens of the batch
  int len;            // keys
  int before;         // keys before the first of the tokens: token j sees before + j + 1 of them
  int slot;
};

__device__ __forceinline__ Seq load_seq(const AttendArgs& a, int i) {
  Seq s;
  s.slot = a.slots[i];
  s.first = min(max(a.starts[i], 0), a.n_tokens);
  const int end = min(max(a.starts[i + 1], s.first), a.n_tokens);
  const bool ok = s.slot >= 0 && s.slot < a.n_slots;
  s.len = ok ? min(max(a.length[s.slot], 0), a.max_pages << a.page_shift) : 0;
  s.count = end - s.first;
  s.before = s.len - s.count;
  return s;
}

__device__ __forceinline__ int up_div(int a, int b) { return (a + b - 1) / b; }   // b: a constant; a + b fits (cap)

// Key tiles that row tile r of a sequence sees any key of.
template <class C>
__device__ __forceinline__ int own_tiles(const Divisor& by_group, int rows, int len, int before, int r) {
  const int last = by_group(min((r + 1) * C::kRows, rows) - 1);
  return up_div(min(len, max(before + last + 1, 0)), C::kKeys);
}
// A segment's extent.
template <class C>
__device__ __forceinline__ int extent(int tiles, int rows_left) {
  return tiles ? C::kSetup + (rows_left > 128 ? 2 * tiles : tiles) : 0;
}
// Units of one head's segments of a sequence.
template <class C>
__device__ __forceinline__ int own_head(const Divisor& by_group, int rows, int len, int before) {
  unsigned sum = 0;   // an extent is below 2^19: the cap below is reached before the sum wraps
#pragma unroll 1
  for (int r = 0; r * C::kRows < rows && sum < kMaxUnits; ++r)
    sum += extent<C>(own_tiles<C>(by_group, rows, len, before, r), rows - r * C::kRows);
  return (int)min(sum, (unsigned)kMaxUnits);
}

// Where a block begins.
struct Begin {
  int u0, u1;                // its units
  int p_rt, p_kt, p_rows, p_head, p_len, t0;
  int seq;                   // sequence of u0; -1: the prefix
  int seq_u;                 // units before it
  int seq_rows;              // stored rows before it
};

// Run by the whole block (THREADS threads): a sweep over the sequences, THREADS
// at a time, for the total, and another for the place of u0, which a list that
// fits one step need not take.  Block 0 leaves the plan for join_kernel.
template <class C, int THREADS>
__device__ __forceinline__ Begin plan_block(const AttendArgs& a) {
  constexpr int W = THREADS / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  __shared__ long long warp_u[W];
  __shared__ int warp_s[W], found[3];              // sequence, units before, stored rows before
  Begin b;
  long long p_units = 0, u = 0;         // the sums of units are taken in 64 bits, and used if they fit 31
  int stored = 0;
  // this thread's sequence of the step: its units, and those and the stored rows before it
  long long mine = 0, before_u = 0;
  int before_s = 0;
  auto step = [&](int i0, bool leave) {
    const int i = i0 + tid;
    int mine_s = 0, head = 0;
    Seq s{};
    mine = 0;
    if (i < a.n) {
      s = load_seq(a, i);
      const int rows = s.count * a.group;
      mine_s = stored_rows<C>(rows) * a.heads;
      head = own_head<C>(a.by_group, rows, s.len, s.before);
      mine = (long long)head * a.heads;
      if (leave) {
        const int from = a.starts[i], to = a.starts[i + 1];
        if (s.slot < -1 || s.slot >= a.n_slots || from < 0 || to < from || to > a.n_tokens) atomicOr(a.status, kStatusIndex);
      }
    }
    long long xu = mine;
    int xs = mine_s;
#pragma unroll 1
    for (int d = 1; d < 32; d <<= 1) {
      const long long yu = __shfl_up_sync(0xffffffffu, xu, d);
      const int ys = __shfl_up_sync(0xffffffffu, xs, d);
      if (lane >= d) {
        xu += yu;
        xs = min(xs + ys, kMaxStored);
      }
    }
    __syncthreads();
    if (lane == 31) {
      warp_u[warp] = xu;
      warp_s[warp] = xs;
    }
    __syncthreads();
    before_u = u + xu - mine;
    before_s = min(stored + (xs - mine_s), kMaxStored);
#pragma unroll 1
    for (int w = 0; w < W; ++w) {
      if (w < warp) {
        before_u += warp_u[w];
        before_s = min(before_s + warp_s[w], kMaxStored);
      }
      u += warp_u[w];
      stored = min(stored + warp_s[w], kMaxStored);
    }
    if (leave && i < a.n)
      a.seqs[i] = SeqPlan{(int)min(before_u, (long long)kMaxUnits), before_s, s.first, s.count, s.len, s.before, head, 0};
  };

  // everything that depends on nothing is asked for before the first use of any of it
  const int start0 = a.starts[0], start_n = a.starts[a.n], p_len = a.do_prefix ? a.length[a.prefix] : 0;
  const int warm = a.do_own && tid < a.n ? a.slots[tid] + a.starts[tid] + a.starts[tid + 1] : 0;
  asm volatile("" ::"r"(start0), "r"(start_n), "r"(p_len), "r"(warm));
  b.t0 = min(max(start0, 0), a.n_tokens);
  const int t1 = min(max(start_n, b.t0), a.n_tokens);
  b.p_rows = b.p_rt = b.p_kt = b.p_len = 0;
  if (a.do_prefix) {
    b.p_len = min(max(p_len, 0), a.max_pages << a.page_shift);
    b.p_rows = (t1 - b.t0) * a.group;
    b.p_rt = up_div(b.p_rows, C::kRows);
    b.p_kt = up_div(b.p_len, C::kKeys);
    if (b.p_rt)
      p_units = (b.p_rt - 1ll) * extent<C>(b.p_kt, C::kRows) + extent<C>(b.p_kt, b.p_rows - (b.p_rt - 1) * C::kRows);
  }
  b.p_head = (int)min(p_units, (long long)kMaxUnits);
  p_units *= a.heads;
  const int p_stored = stored_rows<C>(b.p_rows) * a.heads, n = a.do_own ? a.n : 0;
  u = p_units;
  stored = p_stored;
#pragma unroll 1
  for (int i0 = 0; i0 < n; i0 += THREADS) step(i0, blockIdx.x == 0);

  // every block but the last ones has the same number of units; a block inside a segment always has some
  const bool fits = u <= kMaxUnits - 1024 * 1024;
  const int width = fits ? max(((int)u + (int)gridDim.x - 1) / (int)gridDim.x, 1) : 0;
  b.u0 = (int)min((long long)width * blockIdx.x, u);
  b.u1 = (int)min((long long)width * (blockIdx.x + 1), u);
  b.seq = -1;
  b.seq_u = b.seq_rows = 0;
  if (blockIdx.x == 0 && tid == 0) {
    *a.head = PlanHead{width, b.t0, t1, b.p_rows, b.p_rt, b.p_kt, b.p_head, 0};
    if (!fits) atomicOr(a.status, kStatusIndex);
  }
  if (b.u0 < p_units || b.u0 >= b.u1) return b;
  u = p_units;
  stored = p_stored;
  if (n > THREADS && tid == 0) {   // lengths that changed since the first sweep may leave u0 without a place
    found[0] = 0;
    found[1] = b.u0;
    found[2] = p_stored;
  }
#pragma unroll 1
  for (int i0 = 0; i0 < n; i0 += THREADS) {
    if (n > THREADS) step(i0, false);
    if (b.u0 >= before_u && b.u0 < before_u + mine) {
      found[0] = i0 + tid;
      found[1] = (int)before_u;
      found[2] = before_s;
    }
  }
  __syncthreads();
  b.seq = found[0];
  b.seq_u = found[1];
  b.seq_rows = found[2];
  return b;
}

// A block's part of one segment, key tiles t0 .. t1 - 1 (there may be none),
// and the walk to the next.  Every warp keeps its own; the values are the same
// in all of them.
template <class C>
struct Piece {
  int seq;                   // -1: the prefix
  int h, r;                  // head, row tile
  unsigned row0;             // stored rows of the segments before
  int rows;                  // query rows of the key set
  int first, len, before;    // first token; keys; keys before the first token
  const int* table;          // page table row
  int t0, t1;
  int left;                  // units of the block still to come

  __device__ __forceinline__ int rows_left() const { return rows - r * C::kRows; }
  // Keys that token `tok` of the key set sees.
  __device__ __forceinline__ int sees(int tok) const { return seq < 0 ? len : min(len, before + tok + 1); }

  __device__ __forceinline__ void enter(const AttendArgs& a) {
    const Seq s = load_seq(a, seq);
    rows = s.count * a.group;
    first = s.first;
    len = s.len;
    before = s.before;
    table = a.table + s.slot * a.table_stride;
  }
  __device__ __forceinline__ int ext(const AttendArgs& a) const {
    return extent<C>(seq < 0 ? up_div(len, C::kKeys) : own_tiles<C>(a.by_group, rows, len, before, r), rows_left());
  }
  // Units x .. e - 1 of the segment, as far as they are this block's.
  __device__ __forceinline__ void cut(int x, int e) {
    const int n = min(e - x, left), wide = rows_left() > 128;
    left -= n;
    t0 = max(x - C::kSetup + wide, 0) >> wide;
    t1 = max(x + n - C::kSetup + wide, 0) >> wide;
  }
  __device__ __forceinline__ void begin(const AttendArgs& a, const Begin& b) {
    left = b.u1 - b.u0;
    seq = b.seq;
    int head = b.p_head;
    if (seq < 0) {
      rows = b.p_rows;
      first = b.t0;
      len = before = b.p_len;
      table = a.table + a.prefix * a.table_stride;
    } else {
      enter(a);
      head = own_head<C>(a.by_group, rows, len, before);
    }
    int x = b.u0 - b.seq_u;
    h = x / max(head, 1);
    x -= h * head;
    const int rt = up_div(rows, C::kRows);
    r = 0;
    if (seq < 0) {
      const int e = extent<C>(b.p_kt, C::kRows);
      r = min(x / max(e, 1), rt - 1);
      x -= r * e;
    }
    int e = ext(a);
#pragma unroll 1
    while (x >= e && r + 1 < rt) {
      x -= e;
      ++r;
      e = ext(a);
    }
    row0 = b.seq_rows + h * stored_rows<C>(rows) + r * C::kRows;
    cut(x, e);
  }
  __device__ __forceinline__ bool next(const AttendArgs& a) {
    if (left <= 0) return false;
    int e;
#pragma unroll 1
    do {
      row0 += C::stored(rows_left());
      ++r;
      if (rows_left() <= 0) {
        r = 0;
        if (++h == a.heads) {
          h = 0;
#pragma unroll 1
          do {
            if (++seq >= a.n) {   // lengths that changed under way
              left = 0;
              return false;
            }
            enter(a);
          } while (rows == 0);
        }
      }
      e = ext(a);
    } while (e == 0);
    cut(0, e);
    return true;
  }
};

// ------------------------------------------------------------------ few rows

// Tiles of 16 query rows, for key sets that at most a few rows read: bound by
// HBM, one byte of K or V is worth at most 16 products.
//
// A block has four warps and a unit 64 keys, 16 of each warp.  A warp copies
// the K and V rows of its keys into its own ring in shared memory (cp.async,
// 16 bytes, rows past the end zero-filled, so nothing a page holds there
// reaches a product), takes scores and output with mma.sync m16n8k16, and
// keeps its own running maximum and sum: the main loop has no block barrier.
// mma.sync is enough here: a tile's two products take about 600 cycles of the
// 1400 in which HBM delivers it to an SM.  The four partials are joined through
// shared memory when a segment ends.  Measured: 8 sequences of up to 4000 tokens
// over a prefix of 32000, 32 heads of 128, fp16, with the join: 135 us, 5.9 TB/s,
// 91 % of the copy rate, in bursts of a few ms at 1965 MHz; 147 us, 5.5 TB/s, in
// runs of seconds, which the power cap holds at 1.8 GHz.  Every byte of K and V is
// read once.
constexpr int kFewRows = FewCut::kRows, kFewKeys = FewCut::kKeys, kFewThreads = 128;

template <int D> constexpr int kFewStages = D == 128 ? 3 : 6;
template <int D> constexpr int kFewStage = 2 * 16 * D * 2;   // bytes of a warp's stage: K and V rows of 16 keys
constexpr int kFewJoinBytes = 4 * 16 * 64 * 4;
template <int D> constexpr int kFewSmem = 4 * kFewStages<D> * kFewStage<D> + kFewJoinBytes;

template <class T> struct Mma;
template <> struct Mma<__half> {
  static __device__ __forceinline__ void run(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
};
template <> struct Mma<__nv_bfloat16> {
  static __device__ __forceinline__ void run(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
};

template <bool TRANS>
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  if (TRANS)
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
  else
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

template <class T, int D>
__global__ void __launch_bounds__(kFewThreads, 2) few_rows_kernel(const __grid_constant__ AttendArgs a) {
  constexpr int S = kFewStages<D>, CH = D / 8;   // stages, 16-byte chunks of a row
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ float2 stat[4][16];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, c = lane & 3;
  // Behind a launch of many_rows_kernel nothing of that one is needed here (it began after all work before it was
  // done), so blocks start as its blocks leave; but the join needs both done, so the last block ends after it.
  auto wait_last = [&]() {
    if (a.after_many && blockIdx.x == gridDim.x - 1) asm volatile("griddepcontrol.wait;" ::: "memory");
  };
  if (a.after_many) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  else lb::dependent_begin();
  const Begin b = plan_block<FewCut, kFewThreads>(a);
  if (b.u0 >= b.u1) {
    wait_last();
    return;
  }
  const uint32_t ring = shared_addr(smem) + warp * S * kFewStage<D>;
  float* joined = reinterpret_cast<float*>(smem + 4 * S * kFewStage<D>);

  // ---- loads: page numbers one tile ahead of the copies, copies S - 1 tiles ahead of the products
  Piece<FewCut> lp;
  lp.begin(a, b);
  Piece<FewCut> w = lp;   // the piece that is computed
  int lt = lp.t0;   // next tile to copy
  bool more = true;
  int page[2] = {0, 0};
  auto fetch_pages = [&]() {
#pragma unroll 1
    while (more && lt >= lp.t1) {
      more = lp.next(a);
      lt = lp.t0;
    }
    if (!more) return;
    const int key = lt * kFewKeys + 16 * warp;
#pragma unroll
    for (int i = 0; i < 2; ++i) page[i] = key + 8 * i < lp.len ? lp.table[(key + 8 * i) >> a.page_shift] : 0;
  };
  fetch_pages();
  unsigned bad = 0;
  auto issue = [&](int stage) {
    if (more) {
      const int key = lt * kFewKeys + 16 * warp;
      if (key < lp.len) {
        const uint32_t dst = ring + stage * kFewStage<D>;
        const long long head_k = lp.h * a.k.stride_head, head_v = lp.h * a.v.stride_head;
#pragma unroll
        for (int i = 0; i < CH / 2; ++i) {
          const int row = (i * 32 + lane) / CH, ch = lane % CH;
          const int p = page[row >> 3];
          const bool in = (unsigned)p < (unsigned)a.n_pages;
          if (!in) bad = kStatusIndex;
          const bool use = in && key + row < lp.len;
          const long long off = use ? (key + row) & ((1 << a.page_shift) - 1) : 0;
          const long long pg = use ? p : 0;
          const uint32_t at = dst + row * (2 * D) + ((ch ^ (row & 7)) << 4);
          copy16(at, a.k.data + pg * a.k.stride_page + off * a.k.stride_row + head_k + 16 * ch, use ? 16 : 0);
          copy16(at + 32 * D, a.v.data + pg * a.v.stride_page + off * a.v.stride_row + head_v + 16 * ch, use ? 16 : 0);
        }
      }
      ++lt;
      fetch_pages();
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  // ---- products
  uint32_t qf[D / 16][4];
  float o[D / 8][4];
  float m[2], l[2];
  int lim[2];   // keys that rows g and g + 8 see
  int stage = 0, ahead = 0, t = 0;      // ahead: copies begun, up to S - 1
  int row0 = 0, rows = 0;               // of the piece's partial
  bool fresh = true, begun = false;     // fresh: a new piece
  for (;;) {
    if (fresh) {
      fresh = false;
#pragma unroll 1
      for (;;) {
        if (begun && !w.next(a)) goto done;
        begun = true;
        row0 = w.row0 + blockIdx.x * kFewRows;
        rows = (unsigned)row0 <= (unsigned)(a.n_rows - kFewRows) ? min(kFewRows, w.rows_left()) : 0;
        if (w.t0 < w.t1) break;
        // units of the segment's beginning only
        if (threadIdx.x < rows) a.ml[row0 + threadIdx.x] = make_float2(-INFINITY, 0.f);
      }
      t = w.t0;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int row = w.r * kFewRows + g + 8 * i;
        const int tok = a.by_group(row);
        const bool in = row < w.rows;
        lim[i] = in ? w.sees(tok) : 0;
        const unsigned char* src =
            a.q + (long long)(w.first + tok) * a.q_token + (long long)(w.h * a.group + row - tok * a.group) * a.q_head;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          qf[k][i] = in ? *reinterpret_cast<const uint32_t*>(src + k * 32 + c * 4) : 0;
          qf[k][i + 2] = in ? *reinterpret_cast<const uint32_t*>(src + k * 32 + 16 + c * 4) : 0;
        }
        m[i] = -INFINITY;
        l[i] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    }
    if (ahead == S - 1) {
      asm volatile("cp.async.wait_group %0;" ::"n"(S - 2) : "memory");
      __syncwarp();
    }
    // the one place that copies; the first S - 1 rounds do nothing else
    issue(ahead < S - 1 ? ahead : stage == 0 ? S - 1 : stage - 1);
    if (ahead < S - 1) {
      ++ahead;
      continue;
    }
    const int key = t * kFewKeys + 16 * warp;
    if (key < w.len) {
      const uint32_t kb = ring + stage * kFewStage<D>, vb = kb + 32 * D;
      float s[2][4] = {};
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        uint32_t f[4];
        const int row = ((lane >> 4) << 3) + (lane & 7), ch = 2 * k + ((lane >> 3) & 1);
        ldmatrix4<false>(f, kb + row * (2 * D) + ((ch ^ (row & 7)) << 4));
        Mma<T>::run(s[0], qf[k], f[0], f[1]);
        Mma<T>::run(s[1], qf[k], f[2], f[3]);
      }
      // scores in units of log 2; keys a row does not see get -inf
      float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int at = key + 8 * n + 2 * c + (e & 1);
          s[n][e] = at < lim[e >> 1] ? s[n][e] * a.scale_log2 : -INFINITY;
          top[e >> 1] = max_nan(top[e >> 1], s[n][e]);
        }
      float alpha[2], base[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        top[i] = max_nan(top[i], __shfl_xor_sync(0xffffffffu, top[i], 1));
        top[i] = max_nan(top[i], __shfl_xor_sync(0xffffffffu, top[i], 2));
        const float now = max_nan(m[i], top[i]);
        base[i] = now == -INFINITY ? 0.f : now;
        alpha[i] = exp2_fast(m[i] - base[i]);
        m[i] = now;
      }
      float sum[2] = {0.f, 0.f};
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[n][e] = exp2_fast(s[n][e] - base[e >> 1]);
          sum[e >> 1] += s[n][e];
        }
      l[0] = l[0] * alpha[0] + sum[0];
      l[1] = l[1] * alpha[1] + sum[1];
      const uint32_t p[4] = {Mma<T>::pack(s[0][0], s[0][1]), Mma<T>::pack(s[0][2], s[0][3]),
                             Mma<T>::pack(s[1][0], s[1][1]), Mma<T>::pack(s[1][2], s[1][3])};
      if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          o[i][0] *= alpha[0];
          o[i][1] *= alpha[0];
          o[i][2] *= alpha[1];
          o[i][3] *= alpha[1];
        }
      }
#pragma unroll
      for (int d = 0; d < D / 16; ++d) {
        uint32_t f[4];
        const int row = lane & 15, ch = 2 * d + (lane >> 4);
        ldmatrix4<true>(f, vb + row * (2 * D) + ((ch ^ (row & 7)) << 4));
        Mma<T>::run(o[2 * d], p, f[0], f[1]);
        Mma<T>::run(o[2 * d + 1], p, f[2], f[3]);
      }
    }
    stage = stage + 1 == S ? 0 : stage + 1;
    if (++t < w.t1) continue;
    // ---- join the four warps' partials and write the segment's
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
      if (c == 0) stat[warp][g + 8 * i] = make_float2(m[i], l[i]);
    }
    __syncthreads();
    float f[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float top = -INFINITY;
#pragma unroll
      for (int x = 0; x < 4; ++x) top = max_nan(top, stat[x][g + 8 * i].x);
      f[i] = top == -INFINITY ? 0.f : exp2_fast(m[i] - top);
    }
    if (threadIdx.x < rows) {
      float top = -INFINITY, sum = 0.f;
#pragma unroll
      for (int x = 0; x < 4; ++x) top = max_nan(top, stat[x][threadIdx.x].x);
      if (top != -INFINITY)
#pragma unroll
        for (int x = 0; x < 4; ++x) sum += exp2_fast(stat[x][threadIdx.x].x - top) * stat[x][threadIdx.x].y;
      a.ml[row0 + threadIdx.x] = make_float2(top, sum);
    }
#pragma unroll
    for (int half = 0; half < D / 64; ++half) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float(&v)[4] = o[half * 8 + i];
        float* at = joined + (warp * 16 + g) * 64 + 8 * i + 2 * c;
        *reinterpret_cast<float2*>(at) = make_float2(v[0] * f[0], v[1] * f[0]);
        *reinterpret_cast<float2*>(at + 8 * 64) = make_float2(v[2] * f[1], v[3] * f[1]);
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int e = (i * kFewThreads + threadIdx.x) * 4, row = e >> 6, col = e & 63;
        if (row < rows) {
          float4 v = *reinterpret_cast<const float4*>(joined + e);
#pragma unroll
          for (int x = 1; x < 4; ++x) {
            const float4 y = *reinterpret_cast<const float4*>(joined + x * 1024 + e);
            v.x += y.x;
            v.y += y.y;
            v.z += y.z;
            v.w += y.w;
          }
          *reinterpret_cast<float4*>(a.part + (long long)(row0 + row) * D + half * 64 + col) = v;
        }
      }
      __syncthreads();
    }
    fresh = true;
  }
done:
  if (bad) atomicOr(a.status, bad);
  wait_last();
}

// ------------------------------------------------------------------ many rows

// Tiles of 128 or 256 query rows on the tcgen05 tensor cores: for the prefix
// of a batch, which all of its rows read, and for sequences with many new
// tokens.
//
// A block has two softmax groups of four warps, each with a tile of 128 query
// rows in shared memory.  One warp loads K and V tiles of 128 keys by TMA, page
// by page, into rings.  The products are
//   S = Q K^T (both from shared memory), O += P V (P from tensor memory, V as
//   it lies, keys down, i.e. N-major).
// Each thread of a group owns one row, so the row's maximum and sum need no
// exchange.
//   wide segments (more than 128 rows): the groups have different rows and
//   share every K and V tile, which halves what has to come out of L2;
//   others: the groups have the same rows and take every other key tile.
// Each group leaves a partial of its own, which in a narrow segment makes two
// `ways` of the same rows.
//
// Tensor memory, of each group: S (fp32, 128 columns), P (16-bit pairs, 64) and
// O (fp32, D).  For D = 128 there is room for two of them only, and P lies in
// the first 64 columns of S.
// A group is one chain, S(i) -> softmax -> PV(i) -> QK(i + 1), and while one is
// in its softmax the other's products run; PV starts when half of P is there.
// The group's first warp issues its products: a warp of their own had to be
// woken for each, and took 700 us for 626.
// A commit tells that all products issued before it are complete, so S(i + 1)
// being there means that PV(i) is, and P and O may be written.  Products with
// different accumulators are promised no order among themselves, though: where
// QK(i + 1) writes over the P that PV(i) reads (D = 128), it is issued when PV(i)
// is complete.  On a batch of pieces of prompts that costs 603 us for 586.
// (Issuing the keys whose scores miss P before it, in products half as wide: 625.
// Tiles of 64 keys with P beside S, whose QK(i + 1) runs beside softmax i, have a
// shorter chain but fetch Q twice as often, 192 bytes of shared memory a cycle
// where there are 128; that form took 700 us where this one took 550.)
// 256 rows x 128 keys take about 4000 cycles here, 2048 of them arithmetic: what
// bounds it is a group's chain, about 1900 cycles of softmax and, behind it, half
// of PV, QK and their latency, of which the other group's products cover a part.
// (All powers of two come from the special-function unit: an eighth or a quarter
// of them by a polynomial on the multiply-add units, exact to 2^-22.5, took 599
// and 602 us for 594.)
// Measured: 16 pieces of up to 130 tokens over a prefix of 12000, 64 query heads
// on 8, bf16, with the join: 558 us, 820 TFLOP/s, in bursts at 1965 MHz, 592 us,
// 773 TFLOP/s, in runs of seconds under the power cap; 4096 tokens of 32 heads
// over 23000 keys, fp16: 766 TFLOP/s in such runs.
// The running maximum is raised, and O rescaled in tensor memory, only when a
// tile's maximum exceeds it by more than 8 (a factor 256, for which the 16-bit
// weights and fp32 sums have room), i.e. hardly ever after the first tiles.  The
// weights are rounded to the type for the product, the sum takes them before: half
// a step each, what a 16-bit product costs, and fp16 weights below 2^-14 of their
// part's reference are off by 2^-25 of it (a part: the keys of one chain).  V rows
// past the end of the keys are zeroed in shared memory (0 x NaN is not 0), scores
// there are masked, so K may hold anything.
constexpr int kTile = 128;          // rows of a group's query tile
constexpr int kKeys = ManyCut::kKeys;
constexpr int kManyThreads = 384;   // two softmax groups, and four warps of which the first loads
// The launch's registers, 168 a thread, are shared out again: 2 x 224 + 56 = 3 x 168.
constexpr int kSoftmaxRegs = 224, kIssueRegs = 56;
template <int D> constexpr int kQueryBytes = kTile * D * 2;
template <int D> constexpr int kKeyBytes = kKeys * D * 2;
// K and V tiles in flight (a K tile is done with half a step earlier).
template <int D> constexpr int kRingK = D == 128 ? 2 : 4;
template <int D> constexpr int kRingV = D == 128 ? 3 : 6;
// First column of P, counted from its group's S: its first, or those that a narrow O leaves.
template <int D> constexpr int kWeights = D == 128 ? 0 : 256 + D;
template <int D> constexpr int kManySmem = 2 * kQueryBytes<D> + (kRingK<D> + kRingV<D>) * kKeyBytes<D> + 1024;
constexpr float kRaise = 8.f;

__device__ __forceinline__ void mbar_init(uint64_t* b, uint32_t n) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(shared_addr(b)), "r"(n) : "memory");
}
__device__ __forceinline__ void mbar_expect(uint64_t* b, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(shared_addr(b)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t* b) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(shared_addr(b)) : "memory");
}
__device__ __forceinline__ bool mbar_try(uint64_t* b, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(shared_addr(b)), "r"(parity), "r"(1000u)
      : "memory");
  return ok != 0;
}
// Bounded: false when the phase has not completed after kSpinLimit polls.
__device__ __forceinline__ bool mbar_wait(uint64_t* b, uint32_t parity) {
  for (int i = 0; i < lb::kSpinLimit; ++i)
    if (mbar_try(b, parity)) return true;
  return false;
}
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(shared_addr(bar))
               : "memory");
}
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}
// Matrix descriptor, 128-byte swizzle: lead = bytes between blocks of 64
// N-values (N-major only), step = bytes between groups of eight 128-byte rows.
__device__ __forceinline__ uint64_t tile_desc(uint32_t addr, uint32_t lead, uint32_t step) {
  return (uint64_t)((addr & 0x3FFFF) >> 4) | (uint64_t)(lead >> 4) << 16 | (uint64_t)(step >> 4) << 32 |
         (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
// fp32 accumulators, A and B fp16 or bf16; b_n_major: B is stored K by N
template <class T>
__device__ __forceinline__ constexpr uint32_t mma_shape(int M, int N, bool b_n_major) {
  const uint32_t f = std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
  return 1u << 4 | f << 7 | f << 10 | (b_n_major ? 1u : 0u) << 16 | (uint32_t)(N >> 3) << 17 | (uint32_t)(M >> 4) << 24;
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t shape, uint32_t add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(shape), "r"(add)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t shape, uint32_t add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(shape), "r"(add)
      : "memory");
}
// 32 columns of this thread's lane of tensor memory
__device__ __forceinline__ void tmem_load32(uint32_t at, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(at));
}
__device__ __forceinline__ void tmem_load8(uint32_t at, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(at));
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_store8(uint32_t at, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(at), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
// The registers of a load are good after this: passing them through keeps every use behind the wait.
__device__ __forceinline__ void tmem_load_wait(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]),
                 "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_store32(uint32_t at, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(at),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
// Two fp32 values in one 64-bit register: sm_100 adds and multiplies them in one instruction.
__device__ __forceinline__ uint64_t pair(uint32_t lo, uint32_t hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}
__device__ __forceinline__ uint64_t pair(float lo, float hi) { return pair(__float_as_uint(lo), __float_as_uint(hi)); }
__device__ __forceinline__ float2 split(uint64_t v) {
  uint32_t lo, hi;
  asm("mov.b64 {%0, %1}, %2;" : "=r"(lo), "=r"(hi) : "l"(v));
  return make_float2(__uint_as_float(lo), __uint_as_float(hi));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// The largest of three, NaN if one is.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ void tmem_store_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// 32 bytes at once, a whole sector: lanes write rows far apart
__device__ __forceinline__ void store32(float* dst, const uint32_t* r) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst), "r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void async_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void tma_page(void* dst, const CUtensorMap* map, int x, int row, int head, int page,
                                         uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];" ::"r"(shared_addr(dst)),
      "l"(map), "r"(x), "r"(row), "r"(head), "r"(page), "r"(shared_addr(bar))
      : "memory");
}

template <class T, int D>
__global__ void __launch_bounds__(kManyThreads, 1)
    many_rows_kernel(const __grid_constant__ AttendArgs a, const __grid_constant__ CUtensorMap map_k,
                     const __grid_constant__ CUtensorMap map_v) {
  constexpr int RK = kRingK<D>, RV = kRingV<D>, QB = kQueryBytes<D>, KB = kKeyBytes<D>;
  constexpr int QHALF = kTile * 128, KHALF = kKeys * 128;   // bytes of 64 columns of a tile
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024 - (shared_addr(smem_raw) & 1023)) & 1023);
  unsigned char* const qs = smem;            // [2] query tiles
  unsigned char* const ks = smem + 2 * QB;   // [RK] K tiles
  unsigned char* const vs = ks + RK * KB;    // [RV] V tiles
  // k_full, v_full: a ring slot holds its tile; k_free: it has been read (both groups say so, or one twice), v_free:
  // likewise; s_full: a group's scores are complete; p_free: its PV is, another QK follows over its P; o_full: a piece's
  // last PV is done; quiet: all products of a group that gave up are.  Every wait on them is bounded.
  // The pieces come from the loading warp, which alone reads the lengths: msg_full, a piece is told; msg_free, all eight
  // softmax warps have heard it.  So the warps of a group always agree on their steps, and may hand over queries and
  // weights by named barriers, which is faster than by mbarriers (550 us for 570 on a batch of pieces of prompts).
  // A parity tells whether a phase has ended only to one who knows that the phase before it has.  Within a group that
  // follows from the order of its steps.  A ring slot's last tile may have been the other group's: `loads` counts the
  // tiles whose loads have begun, and one begins only when the slot's last tile has landed and been read.
  __shared__ __align__(8) uint64_t k_full[RK], k_free[RK], v_full[RV], v_free[RV];
  __shared__ __align__(8) uint64_t s_full[2], p_free[2], o_full[2], msg_full[2], msg_free[2], quiet[2];
  __shared__ Piece<ManyCut> msg[2];
  __shared__ int msg_valid[2];   // 0: no more pieces
  __shared__ uint32_t tmem_slot;
  __shared__ volatile uint32_t loads[2];   // of K, of V
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x < 2)   // the maps are kernel arguments: they can be fetched before the work before this is done
    asm volatile("prefetch.tensormap [%0];" ::"l"(threadIdx.x ? &map_v : &map_k) : "memory");
  lb::dependent_begin();
  const Begin b = plan_block<ManyCut, kManyThreads>(a);
  if (b.u0 >= b.u1) return;   // the whole block
  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(shared_addr(&tmem_slot))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (threadIdx.x == 0) {
    loads[0] = loads[1] = 0;
    for (int i = 0; i < RK; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_free[i], 2);
    }
    for (int i = 0; i < RV; ++i) {
      mbar_init(&v_full[i], 1);
      mbar_init(&v_free[i], 2);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&msg_full[i], 1);
      mbar_init(&msg_free[i], 8);
      mbar_init(&o_full[i], 1);
      mbar_init(&p_free[i], 1);
      mbar_init(&quiet[i], 1);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = tmem_slot;
  bool dead = false;   // a wait ran out: go on without waiting, report, end
  unsigned bad = 0;
  uint32_t n = 0;      // key tiles of the pieces before: the block's x-th is in slots x % RK and x % RV

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
    Piece<ManyCut> pc;
    pc.begin(a, b);
    if (warp == 8) {
      // ---- loads: lane i brings the i-th page of a tile
      const int box = min(1 << a.page_shift, kKeys);   // rows of a copy
      auto load = [&](const CUtensorMap* map, unsigned char* slot, uint64_t* full, int key, int boxes, int page) {
        if (lane == 0) {
          mbar_expect(full, boxes * box * D * 2);
          __threadfence_block();   // before `loads` says so
        }
        __syncwarp();
        if (lane < boxes) {
#pragma unroll
          for (int h = 0; h < D / 64; ++h)
            tma_page(slot + h * KHALF + lane * box * 128, map, 64 * h, key & ((1 << a.page_shift) - 1), pc.h, page, full);
        }
      };
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (!dead) dead = !__all_sync(0xffffffffu, mbar_wait(bar, parity));
      };
      uint32_t told = 0;
      auto tell = [&](bool valid) {
        const uint32_t i = told & 1;
        // dead or not: a piece that not all have heard is not to be told over
        if (told >= 2 && !__all_sync(0xffffffffu, mbar_wait(&msg_free[i], ((told >> 1) - 1) & 1))) dead = true;
        if (lane == 0) {
          msg[i] = pc;
          msg_valid[i] = valid;
          mbar_arrive(&msg_full[i]);
        }
        __syncwarp();
        ++told;
      };
      do {
        tell(true);
        for (int t = pc.t0; t < pc.t1; ++t, ++n) {
          const int key = t * kKeys + lane * box;
          const int held = min(kKeys, pc.len - t * kKeys);
          const int boxes = (held + box - 1) / box;
          int page = 0;
          if (lane < boxes) {
            page = pc.table[key >> a.page_shift];
            if ((unsigned)page >= (unsigned)a.n_pages) {   // outside: the copy's fill, zeros
              page = a.n_pages;
              bad |= kStatusIndex;
            }
          }
          if (n >= RK) wait(&k_free[n % RK], (n / RK - 1) & 1);
          if (dead) break;
          load(&map_k, ks + n % RK * KB, &k_full[n % RK], key, boxes, page);
          if (lane == 0) loads[0] = n + 1;
          if (n >= RV) wait(&v_free[n % RV], (n / RV - 1) & 1);
          if (dead) break;
          load(&map_v, vs + n % RV * KB, &v_full[n % RV], key, boxes, page);
          if (lane == 0) loads[1] = n + 1;
        }
      } while (!dead && pc.next(a));
      tell(false);
      if (dead && lane == 0) {   // copies under way land before the block ends: all begun, of K perhaps one more than of V
        const uint32_t k = loads[0], v = loads[1];
        for (uint32_t x = k > RK ? k - RK : 0; x < k; ++x) mbar_wait(&k_full[x % RK], (x / RK) & 1);
        for (uint32_t x = v > RV ? v - RV : 0; x < v; ++x) mbar_wait(&v_full[x % RV], (x / RV) & 1);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    // ---- softmax group g, this thread's row
    const int g = warp >> 2, row = threadIdx.x & 127;
    const uint32_t lane0 = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t ts = tmem + 128 * g + lane0, tp = ts + kWeights<D>, to = ts + 256;
    const float scale = fmaxf(fabsf(a.scale_log2), 0x1p-126f);   // above 0, so that -inf stays -inf
    // The group's first warp issues its products, one elected lane of it; what is uniform for the warp (tm, gg) is
    // made so for the compiler, so that the descriptors live in uniform registers.
    const bool issuer = (warp & 3) == 0;
    const uint32_t gg = __shfl_sync(0xffffffffu, (uint32_t)g, 0);
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0) + 128 * gg;   // S; O 256 columns on
    constexpr uint32_t pv = mma_shape<T>(kTile, D, true);
    // a negative scale negates the queries, so that the softmax knows positive ones only
    const uint32_t qk = mma_shape<T>(kTile, kKeys, false) | (a.scale_log2 < 0.f ? 1u << 13 : 0u);
    const uint64_t q_desc = tile_desc(shared_addr(qs) + gg * QB, 16, 1024);
    uint32_t begun[2] = {0, 0};   // loads, as last seen
    // Queries (0) or a half of the weights (1, 2) to the issuing warp: the others do not wait, but a dead one, whose other
    // waits are over, does, so that no warp is ever a round ahead.
    auto hand_over = [&](int what) {
      if (issuer || dead) asm volatile("bar.sync %0, 128;" ::"r"(1 + 3 * g + what) : "memory");
      else asm volatile("bar.arrive %0, 128;" ::"r"(1 + 3 * g + what) : "memory");
    };
    // tile x of K (0) or V (1) is there
    auto landed = [&](int kv, uint32_t x, uint64_t* full, uint32_t parity) {
      for (int spin = 0; begun[kv] <= x && !dead; ++spin) {
        begun[kv] = __shfl_sync(0xffffffffu, loads[kv], 0);
        dead = spin > lb::kSpinLimit;
      }
      if (!dead) dead = !__all_sync(0xffffffffu, mbar_wait(full, parity));
      tc_after();
    };
    uint32_t turns = 0;   // waits on p_free
    // tile x: S = Q K^T; `after`: behind a PV of the same piece
    auto score = [&](uint32_t x, bool after) {
      landed(0, x, &k_full[x % RK], (x / RK) & 1);
      if (!kWeights<D> && after && !dead) {
        dead = !__all_sync(0xffffffffu, mbar_wait(&p_free[gg], turns++ & 1));
        tc_after();
      }
      const uint64_t k = tile_desc(shared_addr(ks) + x % RK * KB, 16, 1024);
      if (elect_one()) {
#pragma unroll
        for (int c = 0; c < D / 16; ++c)
          mma_ss(tm, q_desc + ((c >> 2) * QHALF + (c & 3) * 32) / 16, k + ((c >> 2) * KHALF + (c & 3) * 32) / 16, qk, c > 0);
        tc_commit(&s_full[gg]);
      }
      __syncwarp();
    };
    // tile x, half of its keys: O (+)= P V; `once`: nobody else reads the tile
    auto weigh = [&](uint32_t x, bool add, bool once, bool last, int half) {
      if (!half) landed(1, x, &v_full[x % RV], (x / RV) & 1);
      else tc_after();
      const uint64_t v = tile_desc(shared_addr(vs) + x % RV * KB, KHALF, 1024);
      if (elect_one()) {
#pragma unroll
        for (int c = 0; c < kKeys / 32; ++c)
          mma_ts(tm + 256, tm + kWeights<D> + 8 * (c + 4 * half), v + (c + 4 * half) * 2048 / 16, pv, add || c + half > 0);
        if (half) {
          tc_commit(&v_free[x % RV]);
          if (once) mbar_arrive(&v_free[x % RV]);
          if (last) tc_commit(&o_full[gg]);
          else if (!kWeights<D>) tc_commit(&p_free[gg]);
        }
      }
      __syncwarp();
    };
    uint32_t steps = 0, pieces = 0;
    auto steps_of = [&](const Piece<ManyCut>& x) {   // of this group
      const int tiles = x.t1 - x.t0;
      return x.rows_left() > kTile ? tiles : (tiles - g + 1) / 2;
    };
    auto row_of = [&](const Piece<ManyCut>& x) {     // of this thread, among the key set's
      return x.r * ManyCut::kRows + (x.rows_left() > kTile ? g * kTile : 0) + row;
    };
    // The group's queries for a piece, under way: the products that read the last ones are done by then.
    auto load_queries = [&](const Piece<ManyCut>& x) {
      if (steps_of(x) > 0) {
        const int at = row_of(x), tok = a.by_group(at);
        const bool in = at < x.rows;
        const unsigned char* src =
            in ? a.q + (long long)(x.first + tok) * a.q_token + (long long)(x.h * a.group + at - tok * a.group) * a.q_head
               : a.q;
        const uint32_t dst = shared_addr(qs + g * QB) + row * 128;
#pragma unroll
        for (int c = 0; c < D / 8; ++c)
          copy16(dst + (c >> 3) * QHALF + (((c & 7) ^ (row & 7)) << 4), src + (in ? 16 * c : 0), in ? 16 : 0);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    // The i-th piece; false after the last.  The wait outlasts all those of the loading warp, which tells of an end in
    // any case.
    auto hear = [&](uint32_t i, Piece<ManyCut>& x) -> bool {
      bool ok = false;
      for (int k = 0; k < 16 && !ok; ++k) ok = mbar_wait(&msg_full[i & 1], (i >> 1) & 1);
      if (!__all_sync(0xffffffffu, ok)) {
        dead = true;
        return false;
      }
      x = msg[i & 1];
      const bool valid = msg_valid[i & 1] != 0;
      __syncwarp();
      if (lane == 0) mbar_arrive(&msg_free[i & 1]);
      return valid;
    };
    uint32_t heard = 0;
    Piece<ManyCut> pc;
    bool more = hear(heard++, pc);
    if (more) load_queries(pc);
    while (more) {
      const int tiles = pc.t1 - pc.t0, mine = steps_of(pc);
      const bool wide = pc.rows_left() > kTile;
      const int at = row_of(pc);
      const int lim = at < pc.rows ? pc.sees(a.by_group(at)) : 0;
      float m = -INFINITY, l = 0.f;
      if (mine > 0) {
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        async_fence();
        hand_over(0);
        if (issuer) score(n + (wide ? 0 : g), false);
        for (int j = 0; j < mine; ++j, ++steps) {
          const int tile = wide ? j : 2 * j + g;
          const int key = (pc.t0 + tile) * kKeys;
          if (!dead && !mbar_wait(&s_full[g], steps & 1)) dead = true;
          dead = __any_sync(0xffffffffu, dead);
          tc_after();
          uint32_t s[kKeys];
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_load32(ts + 32 * c, s + 32 * c);
          if ((threadIdx.x & 127) == 0) {   // the products that made these scores have read the K tile
            mbar_arrive(&k_free[(n + tile) % RK]);
            if (!wide) mbar_arrive(&k_free[(n + tile) % RK]);
          }
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_load_wait(s + 32 * c);
          if (__any_sync(0xffffffffu, key + kKeys > lim)) {
#pragma unroll
            for (int i = 0; i < kKeys; ++i)
              if (key + i >= lim) s[i] = 0xff800000u;   // -inf
          }
          // four chains each, so that their latency is covered with two warps a scheduler
          float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int i = 0; i < kKeys; i += 8)
#pragma unroll
            for (int c = 0; c < 4; ++c)
              tops[c] = max3(tops[c], __uint_as_float(s[i + 2 * c]), __uint_as_float(s[i + 2 * c + 1]));
          const float top = scale * max3(max3(tops[0], tops[1], tops[2]), tops[3], -INFINITY);
          const bool raise = !(top <= m + kRaise);   // also if a score is NaN
          if (__any_sync(0xffffffffu, raise)) {
            const float to_m = top < INFINITY ? top : NAN;   // inf - inf is none either
            const float f = raise ? exp2_fast(m - to_m) : 1.f;
            if (raise) m = to_m;
            l *= f;
            if (j > 0) {   // rare: small steps, as the scores fill the registers
#pragma unroll 1
              for (int c = 0; c < D; c += 8) {
                uint32_t o[8];
                tmem_load8(to + c, o);
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                tmem_store8(to + c, o);
              }
            }
          }
          if (pc.len - key < kKeys) {   // V rows past the end (both groups of a wide segment write the same zeros)
            const uint32_t x = n + tile;
            landed(1, x, &v_full[x % RV], (x / RV) & 1);
            if (row >= pc.len - key) {
#pragma unroll
              for (int c = 0; c < D / 8; ++c)
                *reinterpret_cast<uint4*>(vs + x % RV * KB + (c >> 3) * KHALF + row * 128 + (c & 7) * 16) =
                    make_uint4(0, 0, 0, 0);
            }
            async_fence();
          }
          const float base = m == -INFINITY ? 0.f : m;
          const uint64_t scale2 = pair(scale, scale), base2 = pair(-base, -base);
          uint64_t sums[4] = {0, 0, 0, 0};
#pragma unroll
          for (int half = 0; half < 2; ++half) {
#pragma unroll
            for (int i0 = 32 * half; i0 < 32 * half + 32; i0 += 8) {
              // eight pairs at a time, and no more in flight: the scores fill the registers
              asm volatile("" ::: "memory");
              uint64_t x[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) x[i] = fma2(pair(s[2 * (i0 + i)], s[2 * (i0 + i) + 1]), scale2, base2);
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                float2 e = split(x[i]);
                e = make_float2(exp2_fast(e.x), exp2_fast(e.y));
                sums[i & 3] = add2(sums[i & 3], pair(e.x, e.y));
                s[i0 + i] = Mma<T>::pack(e.x, e.y);
              }
            }
            tmem_store32(tp + 32 * half, s + 32 * half);
            tmem_store_wait();
            tc_before();
            hand_over(1 + half);
            if (issuer) {
              weigh(n + tile, j > 0, !wide, j + 1 == mine, half);
              if (half && j + 1 < mine) score(n + tile + (wide ? 1 : 2), true);
            }
          }
          const float2 sum = split(add2(add2(sums[0], sums[1]), add2(sums[2], sums[3])));
          l += sum.x + sum.y;
        }
      }
      Piece<ManyCut> nx;
      more = hear(heard++, nx);
      if (more) load_queries(nx);
      if (mine > 0) {
        if (!dead && !mbar_wait(&o_full[g], pieces++ & 1)) dead = true;
        dead = __any_sync(0xffffffffu, dead);
        tc_after();
      }
      // ---- the partial: rows of one way, or two ways of the same rows
      const unsigned first = pc.row0 + blockIdx.x * ManyCut::kRows, to_row = first + g * kTile + row;
      const bool keep = at < pc.rows && first <= (unsigned)(a.n_rows - ManyCut::kRows);
      if (keep) a.ml[to_row] = make_float2(m, l);
      if (mine > 0) {
        float* dst = a.part + (long long)to_row * D;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          tmem_load32(to + 32 * c, o);
          tmem_load_wait(o);
          if (keep)
#pragma unroll
            for (int i = 0; i < 32; i += 8) store32(dst + 32 * c + i, o + i);
        }
        tc_before();
      }
      n += tiles;
      pc = nx;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    if (dead && issuer) {   // products under way end before the block does (in a block that is well, o_full said so)
      if (elect_one()) tc_commit(&quiet[gg]);
      __syncwarp();
      mbar_wait(&quiet[gg], 0);
    }
  }
  if (dead) bad |= lb::kStatusTimeout;
  if (bad) atomicOr(a.status, bad);
  __syncwarp();
  tc_before();
  __syncthreads();
  if (warp == 9) {
    tc_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

// ------------------------------------------------------------------ the join

// Where a key set's partials are: of one launch of a partial kernel.
struct Source {
  const PlanHead* head;
  const SeqPlan* seqs;
  const float2* ml;
  const float* part;
  int few;                    // of few_rows_kernel, else of many_rows_kernel
  int n_rows;
};
struct JoinArgs {
  Source set[2];   // the own keys', the prefix's (head null: no prefix)
  unsigned char* out;
  long long out_token, out_head;   // bytes
  int n, n_tokens, heads, group;
  Divisor by_group;
};

// A block per token, or several where there are few tokens: finds the token's
// sequence; then each warp takes a query head at a time, weighs the row's
// partials of both key sets and writes the output.  Bound by latency at decode
// sizes: the plan is one round of loads, the first six partials another.
template <class T, int D>
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ JoinArgs a) {
  constexpr int E = D / 32;
  const int t = blockIdx.x, lane = threadIdx.x & 31;
  __shared__ SeqPlan s_plan;
  __shared__ int s_found;   // the token's sequence: the last one that has it, if starts descend and several do
  if (threadIdx.x == 0) s_found = -1;
  __syncthreads();
  lb::dependent_begin();
  PlanHead head[2];
  head[0] = *a.set[0].head;
  head[1] = a.set[1].head ? *a.set[1].head : PlanHead{1, 0, 0, 0, 0, 0, 0, 0};
  int mine = -1;
  SeqPlan has{};
#pragma unroll 1
  for (int i = threadIdx.x; i < a.n; i += blockDim.x) {
    const SeqPlan s = a.set[0].seqs[i];
    if (t >= s.first && t < s.first + s.count) {
      has = s;
      mine = i;
    }
  }
  if (mine >= 0) atomicMax(&s_found, mine);
  __syncthreads();
  if (mine >= 0 && mine == s_found) s_plan = has;
  __syncthreads();
  if (s_found < 0 || head[0].width == 0 || head[1].width == 0) return;
  const SeqPlan s = s_plan;
#pragma unroll 1
  for (int h = blockIdx.y * 8 + (threadIdx.x >> 5); h < a.heads * a.group; h += 8 * gridDim.y) {
    const int kv = a.by_group(h), sub = h - kv * a.group;

    // rows first[w], first[w] + step[w], ... (count[w] of them) of the work memory are the row's partials in key set w
    int first[2] = {0, 0}, step[2] = {1, 1}, count[2] = {0, 0};
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const Source& S = a.set[w];
      if (!S.head) continue;
      const bool few = S.few;
      const int tile = few ? FewCut::kRows : ManyCut::kRows;
      auto extent_of = [&](int tiles, int left) {
        return few ? extent<FewCut>(tiles, left) : extent<ManyCut>(tiles, left);
      };
      // the row's segment: units ua .. ua + ext - 1
      int row, left, r, ua, ext, before;   // before: stored rows before the head's
      if (w) {
        row = (t - head[1].t0) * a.group + sub;
        if ((unsigned)row >= (unsigned)head[1].p_rows) continue;   // starts descend
        r = few ? row / FewCut::kRows : row / ManyCut::kRows;
        left = head[1].p_rows - r * tile;
        ua = kv * head[1].p_head + r * extent_of(head[1].p_kt, tile);
        ext = extent_of(head[1].p_kt, left);
        before = kv * (few ? stored_rows<FewCut>(head[1].p_rows) : stored_rows<ManyCut>(head[1].p_rows));
      } else {
        const int rows = s.count * a.group;
        row = (t - s.first) * a.group + sub;
        r = few ? row / FewCut::kRows : row / ManyCut::kRows;
        left = rows - r * tile;
        auto own = [&](int i) {
          return extent_of(few ? own_tiles<FewCut>(a.by_group, rows, s.len, s.before, i)
                               : own_tiles<ManyCut>(a.by_group, rows, s.len, s.before, i), rows - i * tile);
        };
        int units = 0;   // of the head's row tiles before this one
        if (r > 0) {
#pragma unroll 1
          for (int i = lane; i < r; i += 32) units += own(i);
          units = __reduce_add_sync(0xffffffffu, units);
        }
        ua = s.units_before + kv * s.head + units;
        ext = own(r);
        before = s.rows_before + kv * (few ? stored_rows<FewCut>(rows) : stored_rows<ManyCut>(rows));
      }
      if (ext == 0) continue;
      const unsigned width = (unsigned)head[w].width;
      const int c0 = (unsigned)ua / width, c1 = (unsigned)(ua + ext - 1) / width;
      // one partial a block, in a narrow tile of many_rows_kernel two ways of it; tiles before the row's are full
      first[w] = before + row + c0 * tile;
      const bool ways = !few && left <= 128;
      step[w] = ways ? tile / 2 : tile;
      count[w] = ways ? 2 * (c1 - c0 + 1) : c1 - c0 + 1;
    }
    float acc[E] = {}, m = -INFINITY, l = 0.f;
    const int total = count[0] + count[1];
    constexpr int kAtOnce = 6;
#pragma unroll 1
    for (int i0 = 0; i0 < total; i0 += kAtOnce) {
      float2 p[kAtOnce];
      float v[kAtOnce][E];
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        const int k = i0 + i, w = k >= count[0];
        const int x = first[w] + (k - (w ? count[0] : 0)) * step[w];
        p[i] = make_float2(-INFINITY, 0.f);
        if (k < total && (unsigned)x < (unsigned)a.set[w].n_rows) {
          p[i] = a.set[w].ml[x];
          const float* src = a.set[w].part + (long long)x * D + lane * E;
          if constexpr (E == 4) {
            const float4 z = *reinterpret_cast<const float4*>(src);
            v[i][0] = z.x, v[i][1] = z.y, v[i][2] = z.z, v[i][3] = z.w;
          } else {
            const float2 z = *reinterpret_cast<const float2*>(src);
            v[i][0] = z.x, v[i][1] = z.y;
          }
        }
      }
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        if (p[i].x == -INFINITY) continue;   // nothing seen; what stands in its row need not have been written
        const float now = fmaxf(m, p[i].x);
        const float f0 = exp2_fast(m - now), f1 = exp2_fast(p[i].x - now);
        m = now;
        l = l * f0 + p[i].y * f1;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = acc[e] * f0 + v[i][e] * f1;
      }
    }
    const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
    T r[E];
#pragma unroll
    for (int e = 0; e < E; ++e) r[e] = (T)(acc[e] * inv);
    unsigned char* dst = a.out + (long long)t * a.out_token + (long long)h * a.out_head + lane * E * 2;
    if constexpr (E == 4) *reinterpret_cast<uint2*>(dst) = *reinterpret_cast<const uint2*>(r);
    else *reinterpret_cast<uint32_t*>(dst) = *reinterpret_cast<const uint32_t*>(r);
  }
}

// ------------------------------------------------------------------ host

int sm_count() {
  static lb::PerDevice slot;
  int v = 148;
  const int dev = lb::current_device();
  if (dev < 0) return 148;
  const int e = slot.get(dev, v, [&](int& out) -> int {
    return cudaDeviceGetAttribute(&out, cudaDevAttrMultiProcessorCount, dev);
  });
  return e || v < 1 ? 148 : v;
}

size_t up(size_t v) { return (v + 255) / 256 * 256; }

// Work memory of one launch: [head][sequences][ml][partials], for `rows` stored
// rows and a further tile for every block's beginning within a segment.
struct Region {
  int blocks, few;   // blocks 0: no such launch
  long long rows;
  size_t seqs, ml, part, bytes;
};
Region region(int tile, int blocks, int64_t rows, int n, int D) {
  Region g;
  g.blocks = blocks;
  g.few = tile == kFewRows;
  g.rows = rows + (int64_t)tile * blocks;
  g.seqs = up(sizeof(PlanHead));
  g.ml = g.seqs + up(sizeof(SeqPlan) * (size_t)n);
  g.part = g.ml + up(sizeof(float2) * (size_t)g.rows);
  g.bytes = g.part + up(sizeof(float) * (size_t)g.rows * D);
  return g;
}

// Which launch takes what: the rows that read a key set decide.  A sequence's
// own keys go to the few-rows kernel if one tile of it holds its rows: 0.65 to
// 0.97 of the many-rows kernel's time for 4 to 64 sequences of 100 to 8000 keys,
// 2 and 8 heads of 128 (16 rows).  Two tiles read the keys twice, which only a
// batch with little to read takes lightly: 24 and 32 rows, up to 32 sequences x
// heads, 0.66 to 0.97 (1.2 at 4000 to 8000 keys); 128 and 512 of them, 0.98 to
// 1.5.  The prefix goes there only if one tile holds its rows (32 rows over 64000
// keys: 103 us and 63), though over a short one two cost less than the other
// kernel's beginning (2000 keys: 15 and 20; 8192: 25 and 25); how long it is, is
// known on the device alone.  So are the tokens of each sequence: most_q decides
// by what the caller knows, and either kernel takes any number, so the work
// memory has room for any division of the batch's tokens.
constexpr int kFewSegments = 32;   // sequences x heads of a batch with little to read
struct Split {
  bool few_prefix, few_own, many_prefix, many_own;
  Region few, many;
};
Split split_of(int heads, int group, int n_tokens, int n, int most_q, bool with_prefix, int D) {
  Split s{};
  const int64_t p_rows = (int64_t)n_tokens * group, o_rows = (int64_t)most_q * group;
  s.few_prefix = with_prefix && p_rows <= kFewRows;
  s.many_prefix = with_prefix && !s.few_prefix;
  s.few_own = o_rows <= ((int64_t)n * heads <= kFewSegments ? 2 * kFewRows : kFewRows);
  s.many_own = !s.few_own;
  // Stored rows at most: one for each query row, and in the many-rows kernel 128 more for a narrow last tile, which
  // the prefix and every sequence may have.
  if (s.few_prefix || s.few_own)
    s.few = region(kFewRows, 2 * sm_count(), heads * p_rows * ((int)s.few_prefix + (int)s.few_own), n, D);
  if (s.many_prefix || s.many_own)
    s.many = region(ManyCut::kRows, sm_count(),
                    heads * ((s.many_prefix ? p_rows + 128 : 0) + (s.many_own ? p_rows + 128ll * std::min(n, n_tokens) : 0)),
                    n, D);
  return s;
}

template <class K>
cudaError_t allow_smem(K kern, lb::PerDevice& slot, int bytes) {
  int v = 0;
  return static_cast<cudaError_t>(slot.get(lb::current_device(), v, [&](int& out) -> int {
    out = 1;
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  }));
}

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
  static const EncodeFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeFn>(p);
  }();
  return fn;
}

// A plane as (width, rows of a page, heads, pages); a copy brings 64 columns
// of a page's rows, 128 at most, into 128-byte rows with the 128-byte swizzle.
lb_status plane_map(const lb_cache& c, const lb_plane& P, CUtensorMap* map) {
  const EncodeFn fn = encode_fn();
  if (!fn) return lb::cuda_fail(cudaErrorNotSupported);
  const int64_t row = 2 * P.width;
  auto stride = [&](int64_t s, int64_t extent) -> cuuint64_t { return (cuuint64_t)(extent > 1 ? 2 * s : row); };
  const cuuint64_t dim[4] = {(cuuint64_t)P.width, (cuuint64_t)c.page_size, (cuuint64_t)P.heads, (cuuint64_t)c.n_pages};
  const cuuint64_t st[3] = {stride(P.stride_row, c.page_size), stride(P.stride_head, P.heads),
                            stride(P.stride_page, c.n_pages)};
  const cuuint32_t box[4] = {64, (cuuint32_t)std::min(c.page_size, kKeys), 1, 1}, one[4] = {1, 1, 1, 1};
  const CUresult r = fn(map, P.dt == LB_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
                        P.data, dim, st, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? LB_OK : LB_ERR_SHAPE;   // strides that the copy engine does not take
}

template <class T, int D>
cudaError_t launch(const Split& s, const AttendArgs& few, const AttendArgs& many, const CUtensorMap& k,
                   const CUtensorMap& v, const JoinArgs& join, cudaStream_t st) {
  static lb::PerDevice few_smem, many_smem;
  cudaError_t e = cudaSuccess;
  if (s.many.blocks) {
    e = allow_smem(many_rows_kernel<T, D>, many_smem, kManySmem<D>);
    if (e != cudaSuccess) return e;
    e = lb::launch_dependent_on(st, many_rows_kernel<T, D>, dim3(s.many.blocks), kManyThreads, kManySmem<D>, many, k, v);
  }
  if (e == cudaSuccess && s.few.blocks) {
    e = allow_smem(few_rows_kernel<T, D>, few_smem, kFewSmem<D>);
    if (e != cudaSuccess) return e;
    e = lb::launch_dependent_on(st, few_rows_kernel<T, D>, dim3(s.few.blocks), kFewThreads, kFewSmem<D>, few);
  }
  if (e != cudaSuccess) return e;
  // blocks of a token: eight an SM in all, of eight heads each at least
  const int y = std::min(lb::ceil_div(join.heads * join.group, 8), std::max(1, 148 * 8 / join.n_tokens));
  return lb::launch_dependent_on(st, join_kernel<T, D>, dim3(join.n_tokens, y), 256, 0, join);
}

lb_status check_attend(const lb_cache* c, int k, int heads_q, int n_tokens, int n, int most_q) {
  const lb_status r = lb::check_cache(c);
  if (r != LB_OK) return r;
  if (k < 0 || k >= c->n_planes) return LB_ERR_ARG;
  const lb_plane& K = c->planes[k];
  if (K.dt != LB_F16 && K.dt != LB_BF16) return LB_ERR_UNSUPPORTED;
  if (K.width != 64 && K.width != 128) return LB_ERR_UNSUPPORTED;
  if (K.heads < 1 || heads_q < 1 || heads_q % K.heads || heads_q > 4096) return LB_ERR_SHAPE;
  if (n < 1 || n > 4096 || n_tokens < 0 || most_q < 1) return LB_ERR_SHAPE;
  // units, rows and keys are counted in 31 bits
  if ((int64_t)n_tokens * heads_q > 1 << 22 || (int64_t)c->max_pages * c->page_size > 1 << 24) return LB_ERR_SHAPE;
  return LB_OK;
}

}  // namespace

extern "C" {

size_t littlebit_cache_attend_work(const lb_cache* c, int k, int heads_q, int n_tokens, int n, int most_q,
                                   int with_prefix) {
  if (check_attend(c, k, heads_q, n_tokens, n, most_q) != LB_OK) return 0;
  const lb_plane& K = c->planes[k];
  const Split s = split_of(K.heads, heads_q / K.heads, n_tokens, n, std::min(most_q, std::max(n_tokens, 1)),
                           with_prefix != 0, K.width);
  return s.few.bytes + s.many.bytes;
}

lb_status littlebit_cache_attend(const lb_cache* c, int k, int v, const lb_rows* q, int n_tokens,
                                 const int32_t* slots, const int32_t* starts, int n, int prefix, int most_q,
                                 float scale, const lb_rows* out, void* work, size_t work_bytes, void* stream) {
  if (!q || !out) return LB_ERR_ARG;
  lb_status r = check_attend(c, k, q->heads, n_tokens, n, most_q);
  if (r != LB_OK || (r = lb::check_list(c, slots, starts, n, n_tokens, prefix)) != LB_OK) return r;
  if ((r = lb::check_cache_plane(c, k)) != LB_OK || (r = lb::check_cache_plane(c, v)) != LB_OK) return r;
  const lb_plane &K = c->planes[k], &V = c->planes[v];
  if (V.dt != K.dt) return LB_ERR_ARG;
  if (V.heads != K.heads || V.width != K.width || q->width != K.width) return LB_ERR_SHAPE;
  if (out->heads != q->heads || out->width != q->width) return LB_ERR_SHAPE;
  if ((r = lb::check_token_rows(q, K.dt)) != LB_OK || (r = lb::check_token_rows(out, K.dt)) != LB_OK) return r;
  const float scale_log2 = scale * 1.4426950408889634f;   // scores are taken in units of log 2
  if (!std::isfinite(scale_log2)) return LB_ERR_ARG;
  if (n_tokens == 0) return LB_OK;
  if (!work) return LB_ERR_ARG;
  if (reinterpret_cast<uintptr_t>(work) % 256) return LB_ERR_ALIGN;
  const int D = K.width, group = q->heads / K.heads;
  most_q = std::min(most_q, n_tokens);
  const Split s = split_of(K.heads, group, n_tokens, n, most_q, prefix >= 0, D);
  if (work_bytes < s.few.bytes + s.many.bytes) return LB_ERR_SHAPE;
  CUtensorMap map_k{}, map_v{};
  if (s.many.blocks && ((r = plane_map(*c, K, &map_k)) != LB_OK || (r = plane_map(*c, V, &map_v)) != LB_OK)) return r;
  unsigned* status = nullptr;
  cudaError_t e = lb::touch_cache_status(&status);
  if (e != cudaSuccess) return lb::cuda_fail(e);

  AttendArgs a{};
  a.k = PlaneArg{static_cast<const unsigned char*>(K.data), 2 * K.stride_page, 2 * K.stride_head, 2 * K.stride_row};
  a.v = PlaneArg{static_cast<const unsigned char*>(V.data), 2 * V.stride_page, 2 * V.stride_head, 2 * V.stride_row};
  a.q = static_cast<const unsigned char*>(q->data);
  a.q_token = 2 * q->stride_token;
  a.q_head = 2 * q->stride_head;
  a.table = c->table;
  a.table_stride = c->table_stride;
  a.length = c->length;
  a.n_pages = c->n_pages;
  while ((1 << a.page_shift) < c->page_size) ++a.page_shift;
  a.n_slots = c->n_slots;
  a.max_pages = c->max_pages;
  a.slots = slots;
  a.starts = starts;
  a.n = n;
  a.n_tokens = n_tokens;
  a.prefix = prefix;
  a.heads = K.heads;
  a.group = group;
  a.by_group = lb::divisor(group);
  a.scale_log2 = scale_log2;
  a.status = status;
  JoinArgs j{};
  auto place = [&](const Region& g, unsigned char* w, bool own, bool with_prefix) {
    AttendArgs x = a;
    x.do_prefix = with_prefix;
    x.do_own = own;
    x.head = reinterpret_cast<PlanHead*>(w);
    x.seqs = reinterpret_cast<SeqPlan*>(w + g.seqs);
    x.ml = reinterpret_cast<float2*>(w + g.ml);
    x.part = reinterpret_cast<float*>(w + g.part);
    x.n_rows = (int)g.rows;
    const Source src{x.head, x.seqs, x.ml, x.part, g.few, (int)g.rows};
    if (own) j.set[0] = src;
    if (with_prefix) j.set[1] = src;
    return x;
  };
  unsigned char* w = static_cast<unsigned char*>(work);
  AttendArgs few = place(s.few, w, s.few_own, s.few_prefix);
  few.after_many = s.many.blocks > 0;
  const AttendArgs many = place(s.many, w + s.few.bytes, s.many_own, s.many_prefix);
  j.out = static_cast<unsigned char*>(out->data);
  j.out_token = 2 * out->stride_token;
  j.out_head = 2 * out->stride_head;
  j.n = n;
  j.n_tokens = n_tokens;
  j.heads = K.heads;
  j.group = group;
  j.by_group = a.by_group;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (K.dt == LB_F16)
    e = D == 128 ? launch<__half, 128>(s, few, many, map_k, map_v, j, st)
                 : launch<__half, 64>(s, few, many, map_k, map_v, j, st);
  else
    e = D == 128 ? launch<__nv_bfloat16, 128>(s, few, many, map_k, map_v, j, st)
                 : launch<__nv_bfloat16, 64>(s, few, many, map_k, map_v, j, st);
  return e == cudaSuccess ? LB_OK : lb::cuda_fail(e);
}

}  // extern "C"
