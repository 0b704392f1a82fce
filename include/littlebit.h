/*
 * littlebit.h -- C ABI of the B200 (sm_100a) LittleBit linear-layer library.
 *
 * The layer (Samsung LittleBit article, aifrontier.co.jp, section 2, the
 * "latent factorisation", "three scales" and "residual compensation" bullets)
 * approximates a weight W (d_out x d_in) as
 *     W  ~=  sum_p  diag(h_p) . U_p . diag(l_p) . V_p^T . diag(g_p)
 * with U_p in {+-1}^(d_out x s), V_p in {+-1}^(d_in x s), fp16 row scale h
 * (length d_out), column scale g (length d_in) and latent scale l (length s);
 * p runs over one path, or two when residual compensation is on, and the
 * outputs of the paths are added.  W is never formed: the forward is
 *     y = sum_p  h_p (.) ( U_p ( l_p (.) ( V_p^T ( g_p (.) x ) ) ) ).
 * Storage per layer is the effective bit width of the LittleBit-2 column
 * (physicalainews.jp, chapter 1): [s(a+b+16) + 16(a+b)] / (ab) bits per
 * weight, or [2s(a+b+16) + 32(a+b)] / (ab) with the residual path.
 *
 * Conventions for every entry point
 * ---------------------------------
 *  - Pointers named *_dev are CUDA device pointers on the current device;
 *    everything else is host memory.  The caller owns every buffer it passes.
 *  - `stream` is a cudaStream_t passed as void* (NULL = legacy default
 *    stream).  Device work is enqueued on it and the call returns without
 *    waiting; the return value reports only what the host can check
 *    (arguments, alignment, shapes, launch errors).
 *  - The library keeps workspaces per (device, stream) -- descriptor tables
 *    and the latent-vector scratch of the forward; one each for the prefill
 *    part and each 16-row decode group of a call, and for each chunk of a
 *    host-buffer call -- allocated on first use with cudaMalloc, grown when
 *    needed and freed by littlebit_release().  Calls enqueued on the same
 *    stream are ordered; calls on different streams use different workspaces.
 *  - No entry point falls back to the CPU: without a usable CUDA device the
 *    call returns LB_ERR_CUDA.
 */
#ifndef LITTLEBIT_H
#define LITTLEBIT_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  LB_OK = 0,
  LB_ERR_ARG = 1,         /* null pointer, bad enum, bad count */
  LB_ERR_ALIGN = 2,       /* a pointer is not aligned as documented */
  LB_ERR_SHAPE = 3,       /* a dimension is outside what the kernels accept */
  LB_ERR_CUDA = 4,        /* a CUDA runtime call failed (see littlebit_last_cuda_error) */
  LB_ERR_TIMEOUT = 5,     /* a bounded device wait ran out (littlebit_device_status) */
  LB_ERR_UNSUPPORTED = 6, /* a valid request this build does not implement */
  LB_ERR_RANGE = 7,       /* a value left the range of the format it is held in (littlebit_device_status) */
  LB_ERR_PAGES = 8,       /* a paged cache had no free page, or a slot no room, for what was asked (littlebit_device_status) */
  LB_ERR_INDEX = 9        /* an index in device memory lay outside its cache, or a slot was not free (littlebit_device_status) */
} lb_status;

typedef enum { LB_F16 = 0, LB_BF16 = 1, LB_F32 = 2, LB_I8 = 3 } lb_dtype;

/* Which factor a packed buffer holds (see the layout below). */
typedef enum { LB_ROLE_V = 0, LB_ROLE_U = 1 } lb_role;

/*
 * Packed factor layout ("sign-plane tiles")
 * -----------------------------------------
 * A factor is viewed as a +-1 matrix F with R rows and K columns, the rows
 * being the outputs of the pass that reads it and K its contraction:
 *   LB_ROLE_V:  F[j][i] = V[i][j],  R = s,      K = d_in
 *   LB_ROLE_U:  F[o][j] = U[o][j],  R = d_out,  K = s
 * F is cut into tiles of TR x TK = 4096 elements (512 bytes):
 *   LB_ROLE_V: TR = 16,  TK = 256          LB_ROLE_U: TR = 128, TK = 32
 * R and K are zero-padded to whole tiles (padding bits are 0).  Tile (rb, kt)
 * starts at byte 512 * (rb * (Kpad / TK) + kt).  Within a tile, lane
 * L = 0..31 owns bytes 16L..16L+15 as four little-endian uint32 words
 * w_0..w_3.  With g = L / 4 and c = L % 4, bit n = 8m + q (m = 0..3,
 * q = 0..7) of w_r is the sign of element (row, k):
 *   LB_ROLE_V:  row = 16 rb + g + 8 (r % 2),         k = 256 kt + 32 q + 16 (r / 2) + 4 c + m
 *   LB_ROLE_U:  row = 128 rb + 16 q + g + 8 (r % 2), k = 32 kt + 16 (r / 2) + 4 c + m
 * and it is 1 exactly when F[row][k] < 0, i.e. sign(0) is +1.
 * Why: each lane's 16 bytes are one 128-bit load, and masking a word with
 * 0x01010101 << q leaves, byte by byte, the int8 A fragment of one
 * m16n8k32 tensor-core product for rows/columns block q (values 0 or 2^q),
 * so the decode kernels feed sign bits to the tensor cores with one logic op
 * per four signs and no unpacking.
 */

/* Bytes of a packed factor with `rows` x `cols` logical elements (R x K above). */
size_t littlebit_packed_bytes(lb_role role, int rows, int cols);

/* Effective bits per weight (LittleBit-2 column, chapter 1); host-only math. */
double littlebit_eff_bits(int d_in, int d_out, int s, int residual);

/*
 * Pack the signs of a real (or +-1) factor into the layout above: the
 * binarisation of the factors to +-1 (Samsung LittleBit article, section 2,
 * the "latent factorisation" and "Dual-SVID initialisation" bullets;
 * LittleBit-2 column, chapter 2: sign(U), sign(V)), stored one bit per sign.
 *   src_dev : factor in its natural orientation, n_long x s elements of type
 *             dt (LB_F16, LB_BF16, LB_F32 or LB_I8); element (a, j) is read at
 *             src_dev[a * stride_long + j * stride_s] (strides in elements).
 *             Role V: n_long = d_in (V is d_in x s); role U: n_long = d_out.
 *   dst_dev : littlebit_packed_bytes(role, R, K) bytes, 16-byte aligned;
 *             every byte is written (padding bits 0).
 * A NaN has no sign to keep and is packed as +1 (bit 0).
 * Errors: LB_ERR_ARG (null, bad dtype/role), LB_ERR_SHAPE (n_long or s < 1),
 * LB_ERR_ALIGN (dst not 16-byte aligned), LB_ERR_CUDA.
 */
lb_status littlebit_pack_signs(const void* src_dev, lb_dtype dt, int n_long, int s,
                               int64_t stride_long, int64_t stride_s, lb_role role,
                               void* dst_dev, void* stream);

/*
 * Inverse of littlebit_pack_signs (a test and inspection aid): the packed
 * factor at src_dev (littlebit_packed_bytes(role, R, K) bytes, 16-byte
 * aligned) back to +-1 values in its natural orientation, n_long x s int8,
 * row-major (element (a, j) at dst_dev[a * s + j]; role V: n_long = d_in,
 * role U: n_long = d_out).  Padding bits are not read.
 * Errors: LB_ERR_ARG (null, bad role), LB_ERR_SHAPE (n_long or s < 1),
 * LB_ERR_ALIGN (src not 16-byte aligned), LB_ERR_CUDA.
 */
lb_status littlebit_unpack_signs(const void* src_dev, lb_role role, int n_long, int s, int8_t* dst_dev,
                                 void* stream);

/* One path of a layer: device pointers, all owned by the caller. */
typedef struct lb_path {
  const void* V_bits;    /* packed LB_ROLE_V factor, 16-byte aligned */
  const void* U_bits;    /* packed LB_ROLE_U factor, 16-byte aligned */
  const uint16_t* h;     /* fp16 [d_out] row (output) scale, 16-byte aligned */
  const uint16_t* g;     /* fp16 [d_in]  column (input) scale, 16-byte aligned */
  const uint16_t* l;     /* fp16 [s]     latent scale */
} lb_path;

typedef struct lb_layer {
  int d_in;              /* multiple of 256, >= 256 */
  int d_out;             /* multiple of 128, >= 128 */
  int s;                 /* latent rank, 1 .. 1024 */
  int residual;          /* 0: path[0] only; 1: path[0] + path[1], same s */
  lb_path path[2];
} lb_layer;

/*
 * y = forward(x) for one layer (formula at the top of this file).
 *   x_dev : batch x d_in row-major activations, y_dev : batch x d_out.
 *   Decode (1 <= batch <= 16): x and y are fp16 (xdt = LB_F16); four kernel
 *   launches (input quantisation, latent pass, finalize, output pass), int8
 *   tensor-core products with int32 accumulation, fp32 scaling.
 *   Prefill (batch a multiple of 128, batch * d_in <= 2^30): xdt = LB_F16 or
 *   LB_BF16, y of the same type -- fp16 tcgen05 tensor-core path, see
 *   littlebit_linear_forward_many.
 *   Any other batch above 16 (fp16 only, batch * d_in <= 2^30): the leading
 *   multiple of 128 rows take the prefill path and the remaining rows the
 *   decode path in groups of at most 16 (the weights stream once per group).
 *   x_dev and y_dev must be 16-byte aligned; every other pointer as in lb_path.
 * Errors: LB_ERR_ARG, LB_ERR_ALIGN, LB_ERR_SHAPE, LB_ERR_UNSUPPORTED (a dtype
 * the batch's path does not take: bf16 below 128 rows or off a multiple of
 * 128, f32 or i8 activations), LB_ERR_CUDA.
 */
lb_status littlebit_linear_forward(const lb_layer* layer, const void* x_dev, void* y_dev,
                                   int batch, lb_dtype xdt, void* stream);

/*
 * The same forward for n independent layers (each with its own input and
 * output buffer, e.g. every linear layer of a model stack), done by the same
 * launches for the whole list (decode: the four passes; prefill: operand
 * preparation and two grouped GEMM launches per group of layers),
 * so that the weights of all layers stream from HBM back to back.  layers, xs,
 * ys are host arrays of length n.
 *
 * The library keeps a workspace per (device, stream) and remembers the last
 * call's arguments on it (the layer structs and the x and y pointers): a call
 * that repeats them enqueues kernels and events only -- no allocation, no
 * host-to-device copy -- and may therefore be captured into a CUDA graph, on
 * the same stream as an earlier eager call with the same arguments.  Kernels
 * read the pointed-to data when they run, so new contents at the same
 * addresses are picked up.
 */
lb_status littlebit_linear_forward_many(const lb_layer* layers, int n, const void* const* xs,
                                        void* const* ys, int batch, lb_dtype xdt, void* stream);

/*
 * littlebit_linear_forward_many, and in addition, on the decode path, records
 * events[i] (cudaEvent_t values passed as void*; a NULL entry is skipped) on
 * `stream` right after kernel launch i, for i < n_events <= 3: 0 = input
 * quantisation, 1 = latent pass, 2 = finalize (the output pass is last), so
 * that a caller can time each kernel with CUDA events.  The prefill path
 * records none; a batch split into groups records them in its first decode
 * group.  events may be NULL when n_events is 0.
 */
lb_status littlebit_linear_forward_many_timed(const lb_layer* layers, int n, const void* const* xs,
                                              void* const* ys, int batch, lb_dtype xdt, void* stream,
                                              void* const* events, int n_events);

/*
 * littlebit_linear_forward_many with the activations in HOST memory (no
 * counterpart in the pages; a transport wrapper around the same forward).
 *   x_host: the n layers' inputs back to back -- layer i's batch x d_in[i]
 *     row-major matrix starts at element sum_{j<i} batch * d_in[j] -- in xdt
 *     (2-byte elements).  y_host: the outputs the same way with d_out (y has
 *     x's dtype).  Both are caller-owned host memory.
 *   n_chunks (>= 1; at most min(n, 64) are used): the stack is cut into that
 *     many consecutive groups of layers of about equal bytes.  Group c's input
 *     copy, its forward and its output copy are chained by events on two
 *     library-owned copy streams and `stream`, so that copies of one group
 *     overlap the kernels of its neighbours.  Page-locked host buffers
 *     (cudaHostAlloc / cudaHostRegister) are needed for that overlap; with
 *     pageable memory the result is the same but the copies serialise.
 * Device copies of the whole stack's x and y are held per (device, stream)
 * until littlebit_release().  Both copy streams start after the work already
 * enqueued on `stream`, and `stream` continues only after the last output
 * copy, so y_host is complete once `stream` has been synchronised (the host
 * buffers must stay untouched until then).  Not for CUDA-graph capture by the
 * caller.  With page-locked buffers, the second of consecutive calls with the
 * same layers, batch, dtype, chunk count and host buffers captures the call's
 * copies and kernels as a CUDA graph, and later such calls replay it with one
 * launch; a host-buffer call with other arguments on `stream`, or
 * littlebit_release(), drops it.
 * Batch, dtype and layer rules, and errors, as littlebit_linear_forward_many;
 * LB_ERR_ARG also for NULL host pointers or n_chunks < 1.
 */
lb_status littlebit_linear_forward_many_host(const lb_layer* layers, int n, const void* x_host, void* y_host,
                                             int batch, lb_dtype xdt, int n_chunks, void* stream);

/*
 * The latent cache (Samsung LittleBit article, section 4, the KV-cache bullet:
 * because a K or V projection is factorised, the r-wide latent can be cached
 * in place of the d-wide projection).  The forward splits at t'_p = l_p (.)
 * V_p^T (g_p (.) x):
 *   littlebit_latent_forward:  x rows -> cache rows [t'_1 | t'_2]
 *   littlebit_latent_expand:   cache rows -> y = sum_p h_p (.) U_p t'_p
 * so that latent_expand(latent_forward(x)) is the layer's output up to the
 * rounding of the cache to fp16.
 * A cache row holds npaths*s fp16 values, path p at columns p*s .. p*s+s-1;
 * rows are littlebit_latent_row_elems(s, residual) elements apart (npaths*s
 * rounded up to a multiple of 8, so every row starts on 16 bytes).  For the
 * Llama-2-7B 4096x4096 projection at 0.1 BPW (s = 188, one path) a row is 192
 * values against 4096 for the projection itself: 21.3x smaller.
 */

/* Elements between cache rows of a layer of rank s (0 for an invalid s). */
int littlebit_latent_row_elems(int s, int residual);

/*
 * Cache rows of n layers' inputs: ts[i] (batch x littlebit_latent_row_elems
 * fp16, 16-byte aligned, caller-owned) receives layer i's latents of xs[i]
 * (batch x d_in, xdt).  Batch and dtype rules as littlebit_linear_forward_many
 * (decode: the input quantisation, latent pass and finalize kernels; prefill:
 * operand preparation and the first tcgen05 GEMM, whose epilogue writes the
 * rows).  Errors as littlebit_linear_forward_many.
 */
lb_status littlebit_latent_forward(const lb_layer* layers, int n, const void* const* xs, void* const* ts,
                                   int batch, lb_dtype xdt, void* stream);

/*
 * Projections rebuilt from cache rows: ys[i] (rows x d_out, ydt) = sum_p h_p
 * (.) U_p t'_p for the rows x littlebit_latent_row_elems fp16 cache rows at
 * ts[i].  rows <= 16: the cache rows are quantised to the output pass's 16-bit
 * operand (finalize kernel) and the output pass runs (ydt = LB_F16); rows a
 * multiple of 128: the rows are laid out as the second tcgen05 GEMM's operand
 * and that GEMM runs (ydt = LB_F16 or LB_BF16); other counts split as the
 * forward does.  Errors as littlebit_linear_forward_many.
 */
lb_status littlebit_latent_expand(const lb_layer* layers, int n, const void* const* ts, void* const* ys, int rows,
                                  lb_dtype ydt, void* stream);

/*
 * Initialisation of a path from real factors (the step before the forward).
 * The caller supplies the rank-s truncated SVD of the weight (any library
 * routine), split evenly: U' = U_s sqrt(S_s) (d_out x s) and V' = V_s sqrt(S_s)
 * (d_in x s), fp32 row-major on the device.
 *
 * littlebit_init_dual_svid (Samsung LittleBit article, section 2, the
 * Dual-SVID bullet: the factors' signs are the binary factors and rank-1
 * approximations of their magnitudes give the scales):
 *   U_bits_dev, V_bits_dev <- the packed signs of U', V' (sign(0) = +1; sizes
 *     littlebit_packed_bytes(LB_ROLE_U, d_out, s) and (LB_ROLE_V, s, d_in));
 *   |U'| ~ a_U b_U^T and |V'| ~ a_V b_V^T, the best rank-1 fits (top singular
 *     pairs, non-negative), found by `iters` power steps (1..1000; 32 is
 *     ample for factors of a truncated SVD);
 *   h_dev <- a_U / mean(a_U) (d_out fp16), g_dev <- a_V / mean(a_V) (d_in fp16),
 *   l_dev <- (mean(a_U) b_U) (.) (mean(a_V) b_V) (s fp16).
 * Shapes as lb_layer; every pointer 16-byte aligned (l_dev 2).  Scratch is
 * allocated and freed stream-ordered on `stream` (cudaMallocAsync).
 * For residual compensation the second path is the same initialisation of
 * the SVD of W - W_hat_1 (article section 2, residual-compensation bullet).
 *
 * littlebit_joint_itq (LittleBit-2 column, chapter 2, "solution 1"): X_dev
 * holds the stacked factors [U'; V'] (n_rows = d_out + d_in rows of s fp32);
 * `iters` (0..1000; the column's default is 50) alternations of
 * B = sign(X R) and R = the orthogonal Procrustes solution (the polar factor
 * of X^T B, by 30 Newton-Schulz steps) are run from R_dev (r_given = 1) or
 * from the identity (r_given = 0); on return R_dev holds R (s x s fp32) and
 * X_dev holds X R, i.e. U' R and V' R, whose product is U' V'^T.  Run it
 * before littlebit_init_dual_svid.  fp32 products on the CUDA cores; scratch
 * stream-ordered as above.
 * Errors: LB_ERR_ARG, LB_ERR_SHAPE, LB_ERR_ALIGN, LB_ERR_CUDA.
 */
lb_status littlebit_init_dual_svid(const float* Uf_dev, const float* Vf_dev, int d_out, int d_in, int s, int iters,
                                   void* U_bits_dev, void* V_bits_dev, uint16_t* h_dev, uint16_t* g_dev,
                                   uint16_t* l_dev, void* stream);
lb_status littlebit_joint_itq(float* X_dev, int n_rows, int s, int iters, float* R_dev, int r_given, void* stream);

/*
 * The decode forward of littlebit_linear_forward (one layer, 1 <= batch <= 16,
 * fp16 x and y) for callers that cannot let the library allocate device
 * memory: for example a process whose device memory is reserved up front by
 * its own allocator, or a latency-critical loop that cannot absorb the
 * device-wide synchronisation of cudaMalloc/cudaFree.  The pages describe no
 * such interface; it has no counterpart in them.
 *   - Allocates nothing.  Its scratch is one fixed 1 MiB device array inside
 *     the library, held by every GPU that loads the library until the process
 *     exits.  A layer whose scratch does not fit returns LB_ERR_SHAPE; per
 *     path it needs, for n = ceil(d_in/2048) input slices and r = 1 at batch 1,
 *     else 4*ceil(batch/4): n quantised input slices of 64*ceil(batch/4) +
 *     4096*r bytes, 4*ceil(n/4) * batch * 16*ceil(s/16) fp32 partial sums,
 *     and the t' bytes (about 2*r*s).
 *   - The first call on a device, with that device current, looks up the
 *     array's device address (cudaGetSymbolAddress) and zeroes its status
 *     word on `stream`; make that first call before any stream capture.
 *   - Every call shares the array and the array keeps the last call's
 *     contents; each call writes every region its kernels read before they
 *     read it.  Calls whose work overlaps on the GPU (other streams, other
 *     host threads) race on it and give wrong results: serialise them.
 *   - Device-side error bits (a bounded wait that gave up, a non-finite
 *     input) collect in the array's status word until littlebit_device_status
 *     reads and clears them.
 * Arguments, alignment and other errors as littlebit_linear_forward.
 */
lb_status littlebit_linear_forward_noalloc(const lb_layer* layer, const void* x_dev, void* y_dev,
                                           int batch, lb_dtype xdt, void* stream);

/*
 * The paged cache: rows of many sequences in pages, and the operators of a
 * serving step around them -- rotary positions, rows written to and read from
 * pages, page bookkeeping, and attention.  (The pages of the method describe
 * the latent rows that such a cache may hold, Samsung LittleBit article,
 * section 4, the KV-cache bullet; these operators have no counterpart in them.)
 *
 * A cache has n_pages pages of page_size rows (a power of two, 8..1024).  A
 * plane holds one row of `heads` x `width` values per cached token: K or V of
 * one layer, or a layer's latent rows (heads = 1, width =
 * littlebit_latent_row_elems).  Element (page, head, row, c) of a plane is at
 * data[page * stride_page + head * stride_head + row * stride_row + c]
 * (strides in elements, any order).  All planes share the page numbers.
 *   table  [n_slots][table_stride]  pages of each sequence slot, in order;
 *          max_pages (<= table_stride) entries are used, -1 where none
 *   length [n_slots]                tokens held by each slot
 *   refs   [n_pages]                slots that hold the page; 0: free
 * The arrays are device memory of the caller; an empty cache has table = -1,
 * length = 0, refs = 0.  Row r of the whole cache is row r % page_size of
 * page r / page_size; the `where` arrays below hold such numbers.
 *
 * Everything the bookkeeping calls decide lies in device memory, so a serving
 * step of them may be captured into a CUDA graph.  They allocate the
 * lowest-numbered free pages, in the order of the lists given.  What cannot be
 * done is left out as a whole (a sequence is not extended, a child not made),
 * takes nothing from what follows it in the list, and raises a bit in the cache status word of the device, which
 * littlebit_device_status returns: LB_ERR_PAGES, no free page or no room in
 * max_pages; LB_ERR_INDEX, a slot, page or row number outside the cache, a
 * slot twice in one list, a fork into a slot that holds tokens, starts that
 * descend or lie outside the step's tokens (they are cut to what there is).  A slot number
 * of -1 in a list is padding and skipped.  Lists take up to 4096 entries.
 * Calls that change one cache, and those that read it beside them, must be
 * ordered by the caller.  Alignment: every
 * plane's and row tensor's base on 16 bytes, strides and row sizes multiples
 * of 16 bytes.  None of these calls allocates device memory or waits for the
 * device; their kernels use programmatic dependent launch and begin with a wait
 * for all work before them on the stream.
 */
typedef struct lb_plane {
  void* data;
  int64_t stride_page, stride_head, stride_row;   /* elements */
  int heads, width;
  lb_dtype dt;
} lb_plane;

typedef struct lb_cache {
  const lb_plane* planes;   /* host array, 1..1024 planes */
  int n_planes;
  int n_pages, page_size, n_slots, max_pages;
  int64_t table_stride;
  int32_t* table;
  int32_t* length;
  int32_t* refs;
} lb_cache;

/* Rows of tokens: element (t, head, c) at data[t * stride_token + head * stride_head + c] (strides in elements). */
typedef struct lb_rows {
  void* data;
  int64_t stride_token, stride_head;
  int heads, width;
} lb_rows;

/*
 * Rotary positions.  Pair i of a head (i < rotary_dim / 2) is turned by the
 * angle pos * f_i, f_i = base^(-2i / rotary_dim) radians per token:
 *   (a, b) -> scale * (a cos - b sin, b cos + a sin),
 * with (a, b) at elements (i, i + rotary_dim/2), or (2i, 2i + 1) if
 * `interleaved`; elements from rotary_dim on are left alone.  inverse = 1
 * turns by the opposite angle: the transposed map, i.e. the gradient's.
 * phases holds f_i / 2 pi as 64-bit fractions of a turn, so that pos * phase
 * modulo 2^64 is the angle, without loss at any position.
 */
typedef struct lb_rotary {
  const uint64_t* phases;   /* device, rotary_dim / 2 */
  int rotary_dim;           /* multiple of 16, at most the width of the rows */
  int interleaved;
  float scale;
} lb_rotary;

/*
 * Host: the phases of f_i, stretched for a context `factor` times as long.
 * original = 0: every f_i is divided by factor.  original > 0: a pair that
 * makes turns = original * f_i / 2 pi turns over the original context keeps
 * f_i where turns >= fast, gets f_i / factor where turns <= slow, and in
 * between the mix keep * f_i + (1 - keep) * f_i / factor, keep = (turns - slow)
 * / (fast - slow), or with log_ramp = 1 the same ramp in log(turns).
 * Errors: LB_ERR_ARG (null, base or factor not positive, fast <= slow with
 * original > 0, slow <= 0 with log_ramp), LB_ERR_SHAPE (rotary_dim not a
 * positive even number).
 */
lb_status littlebit_rotary_phases(int rotary_dim, double base, double factor, double original, double slow,
                                  double fast, int log_ramp, uint64_t* phases_host);

/*
 * Rotates n tensors (1..8) of n_tokens rows of one dtype (LB_F16, LB_BF16,
 * LB_F32) in one launch: dst[i] = rotated src[i]; dst[i].data may be
 * src[i].data with the same strides.  positions_dev: int32 per token, any sign.
 * Angles are exact, cos and sin fp32, one rounding to the dtype.
 * Errors: LB_ERR_ARG, LB_ERR_SHAPE, LB_ERR_ALIGN, LB_ERR_CUDA.
 */
lb_status littlebit_rotary(const lb_rows* src, const lb_rows* dst, int n, int n_tokens, lb_dtype dt,
                           const int32_t* positions_dev, const lb_rotary* rope, int inverse, void* stream);

/*
 * Makes room for new tokens: sequence i of the list (slot slots_dev[i]) grows
 * by starts_dev[i + 1] - starts_dev[i] tokens, the tokens starts[i] ..
 * starts[i + 1] - 1 of the step (starts: n + 1 ascending int32).  Pages are
 * taken, table, length and refs updated, and for each of the n_tokens tokens
 *   where_dev[t]     <- its row in the cache (int64), -1 if it has none
 *   positions_dev[t] <- its index in its sequence, plus the length of slot
 *                       `prefix` if that is >= 0 (-1 with where = -1)
 * One launch.  A sequence whose last page is shared must not grow (forks own
 * their last, partly filled page, so extending a fork never meets one).
 */
lb_status littlebit_cache_extend(const lb_cache* c, const int32_t* slots_dev, const int32_t* starts_dev, int n,
                                 int n_tokens, int prefix, int64_t* where_dev, int32_t* positions_dev, void* stream);

/*
 * where and positions, as above, of tokens that the cache holds: the tokens
 * starts[i] .. starts[i + 1] - 1 are tokens first_dev[i], first_dev[i] + 1, ...
 * of slot slots[i] (first_dev null: from the slot's first token on).
 */
lb_status littlebit_cache_locate(const lb_cache* c, const int32_t* slots_dev, const int32_t* starts_dev,
                                 const int32_t* first_dev, int n, int n_tokens, int prefix, int64_t* where_dev,
                                 int32_t* positions_dev, void* stream);

/*
 * Writes the rows of n_tokens tokens into n planes (1..7, host list of plane
 * numbers): rows[i] goes to plane planes[i] at row where_dev[t]; a token with
 * where -1 is skipped.  Planes whose bit i is set in `rotated` get the rows
 * rotated (rope, positions_dev).  q, if not null, is rotated into q_out by the
 * same launch (every token, also skipped ones).  All of one dtype, that of the
 * planes: LB_F16, LB_BF16 or LB_F32.  One launch.  Two tokens of one row leave
 * either's values there.
 */
lb_status littlebit_cache_write(const lb_cache* c, const int* planes, const lb_rows* rows, int n, int n_tokens,
                                const int64_t* where_dev, const lb_rotary* rope, const int32_t* positions_dev,
                                unsigned int rotated, const lb_rows* q, const lb_rows* q_out, void* stream);

/* The other way: rows[i] <- the rows where_dev[t] of plane planes[i]; rows of
 * tokens with where -1 are left as they were.  E.g. latent rows for
 * littlebit_latent_expand. */
lb_status littlebit_cache_read(const lb_cache* c, const int* planes, const lb_rows* rows, int n, int n_tokens,
                               const int64_t* where_dev, void* stream);

/*
 * Slot children[i] becomes a copy of slot parents[i]: it shares the parent's
 * full pages (refs + 1) and gets a page of its own for a partly filled last
 * one, into which the rows held are copied, in every plane.  Children must be
 * empty.  A parent whose last, partly filled page is a number outside the cache
 * is refused; such a number among its full pages is handed on and reported.
 * A parent may be named many times.  work_dev:
 * littlebit_cache_fork_work(n) bytes, 16-byte aligned.  Two launches (one more
 * for every further 64 planes).
 */
size_t littlebit_cache_fork_work(int n);
lb_status littlebit_cache_fork(const lb_cache* c, const int32_t* parents_dev, const int32_t* children_dev, int n,
                               void* work_dev, void* stream);

/* Empties the slots: their pages lose a reference, their table rows become -1.
 * Empty slots, and a slot named twice, are fine.  One launch. */
lb_status littlebit_cache_free(const lb_cache* c, const int32_t* slots_dev, int n, void* stream);

/*
 * Moves the pages in use to the lowest numbers: with L pages in use, the k-th
 * one at or above L moves to the k-th free one below L, in every plane, and
 * table and refs follow.  The new tables go to table_out (strided as table)
 * and refs_out, which may be the cache's own arrays; otherwise those, and the
 * rows they lead to, stay good for work under way until a page is taken
 * again.  count_dev <- L.  work_dev: littlebit_cache_compact_work(n_pages)
 * bytes, 16-byte aligned.  Two launches (as littlebit_cache_fork).
 */
size_t littlebit_cache_compact_work(int n_pages);
lb_status littlebit_cache_compact(const lb_cache* c, int32_t* table_out, int32_t* refs_out, int32_t* count_dev,
                                  void* work_dev, void* stream);

/* Copies page src_dev[i] to page dst_dev[i] in every plane, i < n (n up to
 * 2^20).  No page may be both a source and a destination of one call, or a
 * destination twice.  Tables are not touched. */
lb_status littlebit_cache_copy(const lb_cache* c, const int32_t* src_dev, const int32_t* dst_dev, int n,
                               void* stream);

/*
 * Attention of new tokens over the cache, for a batch whose sequences share a
 * prefix:
 *   out[t, h] = sum_j w_j v_j / sum_j w_j,   w_j = exp(scale * q[t, h] . k_j)
 * over the tokens j of slot `prefix` (all of them; none if prefix is -1) and
 * the tokens of t's own slot up to t itself.  Sequence i of the list has the
 * tokens starts[i] .. starts[i + 1] - 1 of q, which are the last tokens of
 * slot slots[i]; rows of q in no sequence are left out and their rows of out
 * left as they were.  A token that sees nothing (prefix and slot empty) gets
 * zeros.  K is plane k, V plane v (fp16 or bf16, equal shape, width 64 or
 * 128); q and out have their dtype, q.heads a multiple of the planes' heads:
 * query head h reads head h / (q.heads / heads).  most_q (1 at least): the
 * tokens of the longest sequence as far as the caller knows them; it decides
 * which kernel takes the sequences' own keys (up to 16 rows of tokens x query
 * heads of one K and V head, 32 in small batches: the one for few rows).
 * Sequences longer or shorter than that come out the same but for rounding.
 * The prefix is read and multiplied once for the whole batch.  Scores, sums
 * and outputs are accumulated in fp32; the weights are rounded to the dtype
 * for the product with V (half a step of each; of fp16's smallest at most 2^-25
 * of the row's largest), the outputs once at the end.  Rows past a
 * sequence's end are never used, whatever they hold.  (A non-finite V of a
 * token may reach the outputs of earlier tokens of the same call and
 * sequence, whose weight for it is zero.)
 * Two or three launches.  Limits: n_tokens * q.heads <= 2^22, max_pages *
 * page_size <= 2^24 tokens; the planes' strides must be positive multiples of 16
 * bytes below 2^40.  A page number outside the cache counts as a page of zeros
 * and raises LB_ERR_INDEX; a slot outside it has no tokens and raises it too,
 * and so has -1, without a report: such rows see the prefix alone.  A call of
 * more work than 2^31 key tiles (of 128 query rows x 128 keys, or 16 x 64) does
 * nothing and raises LB_ERR_INDEX.
 * work_dev: littlebit_cache_attend_work bytes, 256-byte aligned, needed until
 * the call's launches are done; calls that may overlap need their own.
 * Errors: LB_ERR_ARG (also a scale that is not below 2.3e38 in magnitude),
 * LB_ERR_SHAPE, LB_ERR_ALIGN, LB_ERR_UNSUPPORTED (dtype or width), LB_ERR_CUDA.
 */
size_t littlebit_cache_attend_work(const lb_cache* c, int k, int heads_q, int n_tokens, int n, int most_q,
                                   int with_prefix);
lb_status littlebit_cache_attend(const lb_cache* c, int k, int v, const lb_rows* q, int n_tokens,
                                 const int32_t* slots_dev, const int32_t* starts_dev, int n, int prefix, int most_q,
                                 float scale, const lb_rows* out, void* work_dev, size_t work_bytes, void* stream);

/*
 * (Host helpers below: no counterpart in the pages.)
 * Waits for `stream`, then returns in *status the device-side error bits that
 * the forward kernels enqueued on it have raised since the last call, and
 * clears them.  Bit (1 << LB_ERR_TIMEOUT) means a bounded wait for a bulk copy
 * into shared memory gave up (the outputs of that call are not valid).
 * Bit (1 << LB_ERR_RANGE) means a value could not be held in the format the
 * kernels keep it in, so the outputs of that call hold inf or NaN: an input
 * x that is inf or NaN (decode and prefill), a bf16 input beyond fp16's
 * finite range (|x| > 65504; prefill converts x to fp16), or a latent value
 * t' = l (.) t, or an fp16 output y, beyond fp16's range (prefill).
 * The word of littlebit_linear_forward_noalloc on the current device is read
 * and cleared too (its calls may be on any stream: synchronise them first), and
 * likewise the word of the paged cache's calls on the current device, whose
 * bits are (1 << LB_ERR_PAGES), (1 << LB_ERR_INDEX) and, from its attention,
 * (1 << LB_ERR_TIMEOUT) (see there).
 * *status is 0 when nothing was raised.  Errors: LB_ERR_ARG, LB_ERR_CUDA.
 */
lb_status littlebit_device_status(void* stream, unsigned int* status);

/*
 * Exercises the error path that every bounded device wait of the library
 * takes when it gives up, without any fault or hang: enqueues on `stream` one
 * kernel of one warp that polls an mbarrier that nothing completes, `polls`
 * times (each poll may suspend for up to about 1 us; 1000 polls last about a
 * millisecond), and then raises bit (1 << LB_ERR_TIMEOUT) in the status word
 * of the (device, stream) workspace.  It issues no copy, so nothing is left
 * in flight.  The next littlebit_device_status on the stream reports the bit
 * and clears it; the stream and its workspace remain usable.  Allocates the
 * workspace's status word if no forward has run on the stream yet.
 * Errors: LB_ERR_ARG (polls outside 1 .. 4194304), LB_ERR_CUDA.
 */
lb_status littlebit_check_wait_timeout(void* stream, int polls);

/* Free every workspace of every device, with its side stream and events, and
 * the device copies, copy streams and events of the host-buffer stack call
 * (call with no work in flight on any stream the library was given). */
void littlebit_release(void);

/* Human-readable name of a status code (static string). */
const char* littlebit_status_string(lb_status st);

/* Text of the last CUDA error seen by this thread (static per thread). */
const char* littlebit_last_cuda_error(void);

#ifdef __cplusplus
}
#endif

#endif /* LITTLEBIT_H */
