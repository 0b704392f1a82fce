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
// Work.  A segment is (K and V head, tile of query rows, key set); a unit is
// one key tile of one segment.  The query rows of a tile are (token, query
// head of the group) pairs, so that a K and V head is read once for its whole
// group.  The units of all segments lie in a row, and block c of G (the
// grid, or U if that is less) takes units [U c / G, U (c + 1) / G): every block gets the same amount to within one
// unit, whatever the lengths.  A block writes one fp32 partial for each segment
// that it touches, at slot segment + c (unique, since along the row of units
// one of the two grows from partial to partial), and join_kernel adds a row's
// partials in the order of their blocks: the result does not depend on timing.
// The lengths are read on the device, so a captured graph follows a growing
// cache.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "lb_internal.h"

namespace {

constexpr unsigned kStatusIndex = 1u << LB_ERR_INDEX;

// A plane of one cache, strides in bytes.
struct PlaneArg {
  const unsigned char* data;
  long long stride_page, stride_head, stride_row;
};

// What both the partial kernels and the join know of a launch.
struct PlanHead {
  long long units;       // all units of the launch
  int t0, t1;            // tokens of the batch
  int p_segs, p_kt, p_rt;   // prefix: segments, key tiles and row tiles a segment
  int pad;
};
struct SeqPlan {
  long long units_before;   // units of the launch before this sequence's (the prefix's included)
  int segs_before;          // segments before this sequence's (the prefix's included)
  int first, count;         // tokens
  int kt, rt;               // key tiles and row tiles a segment
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
  int n, n_tokens, prefix, most_q;
  int heads, group;            // K and V heads; query heads of each
  float scale_log2;
  int do_prefix, do_own;       // which key sets this launch takes
  PlanHead* head;              // written by block 0 for the join
  SeqPlan* seqs;
  float2* ml;                  // [slot][rows_alloc] maximum (times log2 e) and sum
  float* part;                 // [slot][rows_alloc][D]
  int rows_alloc, n_partials;
  unsigned* status;
};

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t shared_addr(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// ------------------------------------------------------------------ the plan

struct Seq {
  int first, count;   // tokens of the batch (count cut to most_q)
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
  const long long cap = (long long)a.max_pages << a.page_shift;
  s.len = ok ? (int)min((long long)max(a.length[s.slot], 0), cap) : 0;
  s.before = s.len - (end - s.first);
  s.count = min(end - s.first, a.most_q);
  return s;
}

template <int ROWS, int KEYS>
__device__ __forceinline__ void seq_tiles(const AttendArgs& a, const Seq& s, int& rt, int& kt) {
  rt = (s.count * a.group + ROWS - 1) / ROWS;
  kt = (int)(((long long)s.len + KEYS - 1) / KEYS);
}

// Where a block begins: the totals, and the sequence (or the prefix: -1) its first unit lies in.
struct Begin {
  long long units, u0, u1;   // all units; this block's
  int p_segs, p_kt, p_rt, t0;
  int p_len;
  int seq;                   // sequence of u0; -1: the prefix
  long long seq_u;           // units before it
  int seq_segs;              // segments before it
};

// Run by the whole block (THREADS threads).  Two sweeps over the sequences,
// THREADS at a time: the total, then the place of u0.  Block 0 leaves the
// plan for join_kernel.
template <int THREADS, int ROWS, int KEYS>
__device__ __forceinline__ Begin plan_block(const AttendArgs& a, long long* sm /* THREADS/32 * 2 + 4 */) {
  constexpr int W = THREADS / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  Begin b;
  b.t0 = min(max(a.starts[0], 0), a.n_tokens);
  const int t1 = min(max(a.starts[a.n], b.t0), a.n_tokens);
  b.p_segs = b.p_kt = b.p_rt = b.p_len = 0;
  if (a.do_prefix) {
    const long long cap = (long long)a.max_pages << a.page_shift;
    b.p_len = (int)min((long long)max(a.length[a.prefix], 0), cap);
    b.p_rt = (int)(((long long)(t1 - b.t0) * a.group + ROWS - 1) / ROWS);
    b.p_kt = (int)(((long long)b.p_len + KEYS - 1) / KEYS);
    b.p_segs = b.p_rt * a.heads;
  }
  const long long p_units = (long long)b.p_segs * b.p_kt;
  long long* warp_u = sm;
  long long* warp_s = sm + W;
  long long* found = sm + 2 * W;   // sequence, units before, segments before
  long long total = p_units;
  for (int pass = 0; pass < 2; ++pass) {
    if (pass == 1) {
      b.units = total;
      // with fewer units than blocks the last blocks have none: a block inside a segment always has a unit
      const long long blocks = min((long long)gridDim.x, total);
      b.u0 = blockIdx.x < blocks ? total * blockIdx.x / blocks : total;
      b.u1 = blockIdx.x < blocks ? total * (blockIdx.x + 1) / blocks : total;
      b.seq = -1;
      b.seq_u = 0;
      b.seq_segs = 0;
      if (blockIdx.x == 0 && tid == 0) *a.head = PlanHead{total, b.t0, t1, b.p_segs, b.p_kt, b.p_rt, 0};
      if (b.u0 < p_units || b.u0 >= b.u1) break;
    }
    long long u = p_units;
    long long segs = b.p_segs;
    if (a.do_own)
      for (int i0 = 0; i0 < a.n; i0 += THREADS) {
        const int i = i0 + tid;
        int rt = 0, kt = 0;
        Seq s{};
        if (i < a.n) {
          s = load_seq(a, i);
          seq_tiles<ROWS, KEYS>(a, s, rt, kt);
          if (s.slot != -1 && (s.slot < 0 || s.slot >= a.n_slots) && blockIdx.x == 0)
            atomicOr(a.status, kStatusIndex);
        }
        const long long mine = (long long)rt * kt * a.heads, mine_s = (long long)rt * a.heads;
        long long xu = mine, xs = mine_s;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const long long yu = __shfl_up_sync(0xffffffffu, xu, d), ys = __shfl_up_sync(0xffffffffu, xs, d);
          if (lane >= d) {
            xu += yu;
            xs += ys;
          }
        }
        __syncthreads();
        if (lane == 31) {
          warp_u[warp] = xu;
          warp_s[warp] = xs;
        }
        __syncthreads();
        long long before_u = u + xu - mine, before_s = segs + xs - mine_s;
        for (int w = 0; w < W; ++w) {
          if (w < warp) {
            before_u += warp_u[w];
            before_s += warp_s[w];
          }
          u += warp_u[w];
          segs += warp_s[w];
        }
        if (pass == 0) {
          if (blockIdx.x == 0 && i < a.n) a.seqs[i] = SeqPlan{before_u, (int)before_s, s.first, s.count, kt, rt, 0};
        } else if (i < a.n && b.u0 >= before_u && b.u0 < before_u + mine) {
          found[0] = i;
          found[1] = before_u;
          found[2] = before_s;
        }
      }
    total = u;
    if (pass == 1) {
      __syncthreads();
      b.seq = (int)found[0];
      b.seq_u = found[1];
      b.seq_segs = (int)found[2];
    }
  }
  return b;
}

// Walks a block's units in order.  Every warp keeps its own (the values are
// the same in all of them).
template <int ROWS, int KEYS>
struct Walk {
  int seq;        // -1: the prefix
  int h, r, t;    // head, row tile, key tile
  int rt, kt;
  int seg;        // segment number
  int first, count, len, before;
  const int* row; // page table row

  __device__ __forceinline__ void enter(const AttendArgs& a, const Begin& b) {
    if (seq < 0) {
      rt = b.p_rt;
      kt = b.p_kt;
      first = b.t0;
      count = 0;
      len = before = b.p_len;
      row = a.table + a.prefix * a.table_stride;
    } else {
      const Seq s = load_seq(a, seq);
      seq_tiles<ROWS, KEYS>(a, s, rt, kt);
      first = s.first;
      count = s.count;
      len = s.len;
      before = s.before;
      row = a.table + s.slot * a.table_stride;
    }
  }
  __device__ __forceinline__ void start(const AttendArgs& a, const Begin& b) {
    seq = b.seq;
    enter(a, b);
    const long long off = b.u0 - b.seq_u;
    const int s = (int)(off / kt);
    t = (int)(off - (long long)s * kt);
    h = s / rt;
    r = s - h * rt;
    seg = b.seq_segs + s;
  }
  __device__ __forceinline__ void next(const AttendArgs& a, const Begin& b) {
    if (++t < kt) return;
    t = 0;
    ++seg;
    if (++r < rt) return;
    r = 0;
    if (++h < a.heads) return;
    h = 0;
    do {
      if (++seq >= a.n) {
        seq = a.n;
        return;
      }
      enter(a, b);
      if (kt == 0) seg += rt * a.heads;   // no keys: its segments have no units
    } while (kt == 0 || rt == 0);
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
// shared memory when a segment ends.
constexpr int kFewRows = 16, kFewKeys = 64, kFewThreads = 128;

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
  __shared__ long long plan_sm[12];
  __shared__ float2 stat[4][16];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, c = lane & 3;
  const Begin b = plan_block<kFewThreads, kFewRows, kFewKeys>(a, plan_sm);
  if (b.u0 >= b.u1) return;
  const uint32_t ring = shared_addr(smem) + warp * S * kFewStage<D>;
  float* joined = reinterpret_cast<float*>(smem + 4 * S * kFewStage<D>);
  using W = Walk<kFewRows, kFewKeys>;

  // ---- loads: page numbers one unit ahead of the copies, copies S - 1 units ahead of the products
  W lw;
  lw.start(a, b);
  long long l_left = b.u1 - b.u0;
  int page[2] = {0, 0};
  auto fetch_pages = [&]() {
    const int key = lw.t * kFewKeys + 16 * warp;
#pragma unroll
    for (int i = 0; i < 2; ++i) page[i] = key + 8 * i < lw.len ? lw.row[(key + 8 * i) >> a.page_shift] : 0;
  };
  fetch_pages();
  unsigned bad = 0;
  auto issue = [&](int stage) {
    if (l_left > 0) {
      const int key = lw.t * kFewKeys + 16 * warp;
      if (key < lw.len) {
        const uint32_t dst = ring + stage * kFewStage<D>;
        const long long head_k = lw.h * a.k.stride_head, head_v = lw.h * a.v.stride_head;
#pragma unroll
        for (int i = 0; i < CH / 2; ++i) {
          const int row = (i * 32 + lane) / CH, ch = lane % CH;
          const int p = page[row >> 3];
          const bool in = (unsigned)p < (unsigned)a.n_pages;
          if (!in) bad = kStatusIndex;
          const bool use = in && key + row < lw.len;
          const long long off = use ? (key + row) & ((1 << a.page_shift) - 1) : 0;
          const long long pg = use ? p : 0;
          const uint32_t at = dst + row * (2 * D) + ((ch ^ (row & 7)) << 4);
          copy16(at, a.k.data + pg * a.k.stride_page + off * a.k.stride_row + head_k + 16 * ch, use ? 16 : 0);
          copy16(at + 32 * D, a.v.data + pg * a.v.stride_page + off * a.v.stride_row + head_v + 16 * ch, use ? 16 : 0);
        }
      }
      if (--l_left > 0) {
        lw.next(a, b);
        fetch_pages();
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int s = 0; s < S - 1; ++s) issue(s);

  W w;
  w.start(a, b);
  long long left = b.u1 - b.u0;
  uint32_t qf[D / 16][4];
  float o[D / 8][4];
  float m[2], l[2];
  int lim[2];   // keys that rows g and g + 8 see
  int stage = 0;
  bool fresh = true;
  while (left > 0) {
    asm volatile("cp.async.wait_group %0;" ::"n"(S - 2) : "memory");
    __syncwarp();
    issue(stage == 0 ? S - 1 : stage - 1);
    if (fresh) {   // a new segment: its query rows
      fresh = false;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int row = w.r * kFewRows + g + 8 * i;
        const int tok = row / a.group;
        const int n_tok = w.seq < 0 ? 0x7fffffff : w.count;
        const bool in = tok < n_tok && w.first + tok < a.n_tokens;
        lim[i] = in ? (w.seq < 0 ? w.len : min(w.len, w.before + tok + 1)) : 0;
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
    const int key = w.t * kFewKeys + 16 * warp;
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
          top[e >> 1] = fmaxf(top[e >> 1], s[n][e]);
        }
      float alpha[2], base[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 1));
        top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 2));
        const float now = fmaxf(m[i], top[i]);
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
    --left;
    const bool last = w.t + 1 == w.kt || left == 0;
    if (last) {
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
        for (int x = 0; x < 4; ++x) top = fmaxf(top, stat[x][g + 8 * i].x);
        f[i] = top == -INFINITY ? 0.f : exp2_fast(m[i] - top);
      }
      const int slot = w.seg + (int)blockIdx.x;
      const int rows_here = w.seq < 0 ? (a.n_tokens - w.first) * a.group : w.count * a.group;
      const int rows = slot < a.n_partials ? min(min(kFewRows, a.rows_alloc), rows_here - w.r * kFewRows) : 0;
      if (threadIdx.x < rows) {
        float top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int x = 0; x < 4; ++x) top = fmaxf(top, stat[x][threadIdx.x].x);
        if (top != -INFINITY)
#pragma unroll
          for (int x = 0; x < 4; ++x) sum += exp2_fast(stat[x][threadIdx.x].x - top) * stat[x][threadIdx.x].y;
        a.ml[(long long)slot * a.rows_alloc + threadIdx.x] = make_float2(top, sum);
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
            *reinterpret_cast<float4*>(a.part + ((long long)slot * a.rows_alloc + row) * D + half * 64 + col) = v;
          }
        }
        __syncthreads();
      }
      fresh = true;
    }
    if (left > 0) w.next(a, b);
  }
  if (bad) atomicOr(a.status, bad);
}

// ------------------------------------------------------------------ the join

// Where a key set's partials are: of one launch of a partial kernel.
struct Source {
  const PlanHead* head;
  const SeqPlan* seqs;
  const float2* ml;
  const float* part;
  int rows, rows_alloc, blocks, n_partials;   // query rows of a tile; blocks of the launch
};
struct JoinArgs {
  Source prefix, own;   // head null: no such key set
  unsigned char* out;
  long long out_token, out_head;   // bytes
  int n, n_tokens, heads, group;
};

// One warp per (token, query head): finds the token's sequence, weighs the
// row's partials of both key sets and writes the output.
template <class T, int D>
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ JoinArgs a) {
  constexpr int E = D / 32;
  const int t = blockIdx.x, lane = threadIdx.x & 31;
  const int h = blockIdx.y * 8 + (threadIdx.x >> 5);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __shared__ int s_seq;
  if (threadIdx.x == 0) s_seq = -1;
  __syncthreads();
  for (int i = threadIdx.x; i < a.n; i += blockDim.x) {
    const int first = a.own.seqs[i].first, count = a.own.seqs[i].count;
    if (t >= first && t < first + count) s_seq = i;
  }
  __syncthreads();
  const int seq = s_seq;
  if (seq < 0 || h >= a.heads * a.group) return;
  const int kv = h / a.group, sub = h - kv * a.group;
  float acc[E] = {}, m = -INFINITY, l = 0.f;

  auto add = [&](const Source& S, int seg, long long ua, int kt, int row) {
    if (kt <= 0) return;
    const long long U = S.head->units, G = min((long long)S.blocks, U);
    const int c0 = (int)(((ua + 1) * G - 1) / U), c1 = (int)(((ua + kt) * G - 1) / U);
    for (int c = c0; c <= c1; ++c) {
      const long long at = (long long)(seg + c) * S.rows_alloc + row;
      if (seg + c >= S.n_partials) continue;
      const float2 p = S.ml[at];
      float v[E];
      if constexpr (E == 4) {
        const float4 x = *reinterpret_cast<const float4*>(S.part + at * D + lane * 4);
        v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
      } else {
        const float2 x = *reinterpret_cast<const float2*>(S.part + at * D + lane * 2);
        v[0] = x.x, v[1] = x.y;
      }
      if (p.x == -INFINITY) continue;   // nothing seen
      const float now = fmaxf(m, p.x);
      const float f0 = exp2_fast(m - now), f1 = exp2_fast(p.x - now);
      m = now;
      l = l * f0 + p.y * f1;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = acc[e] * f0 + v[e] * f1;
    }
  };
  if (a.prefix.head) {
    const PlanHead H = *a.prefix.head;
    const int row = (t - H.t0) * a.group + sub;
    const int seg = kv * H.p_rt + row / a.prefix.rows;
    add(a.prefix, seg, (long long)seg * H.p_kt, H.p_kt, row % a.prefix.rows);
  }
  if (a.own.head) {
    const SeqPlan s = a.own.seqs[seq];
    const int row = (t - s.first) * a.group + sub;
    const int k = kv * s.rt + row / a.own.rows;
    add(a.own, s.segs_before + k, s.units_before + (long long)k * s.kt, s.kt, row % a.own.rows);
  }
  const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
  T r[E];
#pragma unroll
  for (int e = 0; e < E; ++e) r[e] = (T)(acc[e] * inv);
  unsigned char* dst = a.out + (long long)t * a.out_token + (long long)h * a.out_head + lane * E * 2;
  if constexpr (E == 4) *reinterpret_cast<uint2*>(dst) = *reinterpret_cast<const uint2*>(r);
  else *reinterpret_cast<uint32_t*>(dst) = *reinterpret_cast<const uint32_t*>(r);
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

// Work memory of one launch: [head][sequences][ml][partials].
struct Region {
  int blocks, rows, rows_alloc;
  long long partials;
  size_t seqs, ml, part, bytes;
};
Region region(int rows, int blocks, int64_t segs, int64_t most_rows, int n, int D) {
  Region g;
  g.blocks = blocks;
  g.rows = rows;
  g.rows_alloc = (int)std::min<int64_t>(rows, most_rows);
  g.partials = segs + blocks;
  g.seqs = up(sizeof(PlanHead));
  g.ml = g.seqs + up(sizeof(SeqPlan) * (size_t)n);
  g.part = g.ml + up(sizeof(float2) * (size_t)g.partials * g.rows_alloc);
  g.bytes = g.part + up(sizeof(float) * (size_t)g.partials * g.rows_alloc * D);
  return g;
}

// Segments of the two key sets at most, with tiles of `rows` query rows.
int64_t prefix_segs(int64_t heads, int64_t group, int64_t tokens, int rows) {
  return heads * ((tokens * group + rows - 1) / rows);
}
int64_t own_segs(int64_t heads, int64_t group, int64_t tokens, int64_t n, int64_t most_q, int rows) {
  const int64_t one = (most_q * group + rows - 1) / rows;
  return heads * std::min(n * one, n + (tokens * group + rows - 1) / rows);
}

Region few_region(int heads, int group, int n_tokens, int n, int most_q, bool with_prefix, int D) {
  const int64_t segs = (with_prefix ? prefix_segs(heads, group, n_tokens, kFewRows) : 0) +
                       own_segs(heads, group, n_tokens, n, most_q, kFewRows);
  const int64_t most = (int64_t)group * std::max(with_prefix ? n_tokens : 0, most_q);
  return region(kFewRows, 2 * sm_count(), segs, most, n, D);
}

template <class K>
cudaError_t allow_smem(K kern, lb::PerDevice& slot, int bytes) {
  int v = 0;
  return static_cast<cudaError_t>(slot.get(lb::current_device(), v, [&](int& out) -> int {
    out = 1;
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  }));
}

template <class T, int D>
cudaError_t launch(const AttendArgs& few, int blocks, const JoinArgs& join, cudaStream_t st) {
  static lb::PerDevice smem;
  cudaError_t e = allow_smem(few_rows_kernel<T, D>, smem, kFewSmem<D>);
  if (e != cudaSuccess) return e;
  few_rows_kernel<T, D><<<blocks, kFewThreads, kFewSmem<D>, st>>>(few);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  join_kernel<T, D><<<dim3(join.n_tokens, lb::ceil_div(join.heads * join.group, 8)), 256, 0, st>>>(join);
  return cudaGetLastError();
}

lb_status check_attend(const lb_cache* c, int k, int heads_q, int n_tokens, int n, int most_q) {
  const lb_status r = lb::check_cache(c);
  if (r != LB_OK) return r;
  if (k < 0 || k >= c->n_planes) return LB_ERR_ARG;
  const lb_plane& K = c->planes[k];
  if (K.dt != LB_F16 && K.dt != LB_BF16) return LB_ERR_UNSUPPORTED;
  if (K.width != 64 && K.width != 128) return LB_ERR_UNSUPPORTED;
  if (K.heads < 1 || heads_q < 1 || heads_q % K.heads || heads_q > 4096) return LB_ERR_SHAPE;
  if (n < 1 || n > 4096 || n_tokens < 0 || n_tokens > 1 << 20 || most_q < 1) return LB_ERR_SHAPE;
  return LB_OK;
}

}  // namespace

extern "C" {

size_t littlebit_cache_attend_work(const lb_cache* c, int k, int heads_q, int n_tokens, int n, int most_q,
                                   int with_prefix) {
  if (check_attend(c, k, heads_q, n_tokens, n, most_q) != LB_OK) return 0;
  const lb_plane& K = c->planes[k];
  return few_region(K.heads, heads_q / K.heads, n_tokens, n, std::min(most_q, std::max(n_tokens, 1)),
                    with_prefix != 0, K.width).bytes;
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
  if (!(scale == scale) || std::isinf(scale)) return LB_ERR_ARG;
  if (n_tokens == 0) return LB_OK;
  if (!work) return LB_ERR_ARG;
  if (reinterpret_cast<uintptr_t>(work) % 256) return LB_ERR_ALIGN;
  const int D = K.width, group = q->heads / K.heads;
  most_q = std::min(most_q, n_tokens);
  const Region g = few_region(K.heads, group, n_tokens, n, most_q, prefix >= 0, D);
  if (work_bytes < g.bytes) return LB_ERR_SHAPE;
  unsigned* status = nullptr;
  cudaError_t e = lb::touch_cache_status(&status);
  if (e != cudaSuccess) return lb::cuda_fail(e);

  unsigned char* w = static_cast<unsigned char*>(work);
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
  a.most_q = most_q;
  a.heads = K.heads;
  a.group = group;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.do_prefix = prefix >= 0;
  a.do_own = 1;
  a.head = reinterpret_cast<PlanHead*>(w);
  a.seqs = reinterpret_cast<SeqPlan*>(w + g.seqs);
  a.ml = reinterpret_cast<float2*>(w + g.ml);
  a.part = reinterpret_cast<float*>(w + g.part);
  a.rows_alloc = g.rows_alloc;
  a.n_partials = (int)g.partials;
  a.status = status;
  JoinArgs j{};
  const Source s{a.head, a.seqs, a.ml, a.part, g.rows, g.rows_alloc, g.blocks, (int)g.partials};
  j.own = s;
  if (prefix >= 0) j.prefix = s;
  j.out = static_cast<unsigned char*>(out->data);
  j.out_token = 2 * out->stride_token;
  j.out_head = 2 * out->stride_head;
  j.n = n;
  j.n_tokens = n_tokens;
  j.heads = K.heads;
  j.group = group;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (K.dt == LB_F16)
    e = D == 128 ? launch<__half, 128>(a, g.blocks, j, st) : launch<__half, 64>(a, g.blocks, j, st);
  else
    e = D == 128 ? launch<__nv_bfloat16, 128>(a, g.blocks, j, st) : launch<__nv_bfloat16, 64>(a, g.blocks, j, st);
  return e == cudaSuccess ? LB_OK : lb::cuda_fail(e);
}

}  // extern "C"
