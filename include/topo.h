/*
 * topo.h -- C ABI of the batched generated-topology library for MI355X (gfx950).
 *
 * The library builds, for a batch of B sparse voxel grids at once, the topology
 * of a generated grid: coarsen by 2/4/8, refine by 2/4/8, box-dilate [-1,1]^3,
 * pad {-1,0}^3 or {0,1}^3, and the k3s2 transposed-conv target (refine by 2 then
 * pad {-1,0}^3). Each grid is a three-level tree of 8^3 leaves (512-bit active
 * masks), 16^3-leaf lower nodes, 32^3-lower upper nodes and one root tile per
 * upper node, stored in the canonical x-major tree order. One pass runs over all
 * source leaves of all members, with one host readback of node counts.
 *
 * Source of the operations and outputs: the fvdb-core pages
 *   - "Generated-topology grid construction dominates per-iteration
 *     ConvolutionPlan cost" (issue page): Summary, Root cause, Suggested direction;
 *   - "Batched leaf-mask topology construction for generated conv grids"
 *     (PR page): section 1 (one emission pass, canonical order, dedup, one
 *     readback, batched writers, empty members, multi-pass factors 4 and 8),
 *     section 2 (box-dilate passes, pads, k3s2 transpose), Test plan.
 *
 * Conventions (all entry points):
 *   - Pointers named d_* are HIP device pointers; h_* are host pointers.
 *   - `stream` is a hipStream_t (NULL = the legacy default stream). All device
 *     work is enqueued on it; device outputs become valid in stream order.
 *   - Every entry point validates its arguments on the host before any launch.
 *     On any non-TC_OK status, *out is set to NULL, nothing is leaked and
 *     tc_last_error() returns a message for the calling thread.
 *   - int32 overflow of an output coordinate is detected on the device, by the
 *     kernels that compute the output nodes, and reported at the pass's one
 *     readback (TC_ERR_OVERFLOW, no batch), before any output is allocated.
 *   - The kernels that write a batch's leaf masks check their indices; a failed
 *     check (a library defect, never an input property) is reported as
 *     TC_ERR_INTERNAL: by the pass itself when it ends on the readback of the
 *     batch's headers (small batches, see tc_build_batched_topology), else by
 *     the first call that blocks on the batch afterwards (tc_batch_voxel_total,
 *     tc_batch_read_headers, tc_enumerate_ijk, tc_build_kernel_map, or a pass
 *     that reads it), and by every later one.
 *   - Calls on different streams or threads are independent. A tc_grid_batch is
 *     immutable after creation and may be read concurrently.
 *   - Coordinates are int32 voxel indices; counts are int32 (nodes) or int64
 *     (voxels).
 */
#ifndef TOPO_H
#define TOPO_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define TC_ABI_VERSION 1

typedef enum tc_status {
  TC_OK = 0,
  TC_ERR_INVALID_ARG = 1,  /* bad pointer, op, factor, B < 1, bad offsets, capacity */
  TC_ERR_OVERFLOW = 2,     /* an output voxel coordinate would leave int32 */
  TC_ERR_ALLOC = 3,        /* the allocator (or the HIP pool) returned no memory */
  TC_ERR_HIP = 4,          /* a HIP runtime call failed; message has the HIP error */
  TC_ERR_UNSUPPORTED = 5,  /* e.g. a factor that is not a power of two */
  TC_ERR_INTERNAL = 6      /* a device-side consistency check failed */
} tc_status;

/* Operations (PR page sections 1 and 2).
 *   TC_OP_COARSEN     factor 2, 4 or 8: { floor(v / f) }         (conv_grid k2s2 for f = 2)
 *   TC_OP_REFINE      factor 2, 4 or 8: { f*v + d, d in [0,f)^3 } (conv_transpose_grid k2s2)
 *   TC_OP_DILATE      factor 1: Minkowski sum with [-1,1]^3       (conv_grid k3s1)
 *   TC_OP_PAD_NEG     factor 1: Minkowski sum with {-1,0}^3
 *   TC_OP_PAD_POS     factor 1: Minkowski sum with {0,1}^3
 *   TC_OP_CONV_T_K3S2 factor 2: refine by 2, then TC_OP_PAD_NEG   (conv_transpose_grid k3s2)
 *   TC_OP_CONV_S1     factor K in [1,8]: Minkowski sum with [-floor(K/2), floor((K-1)/2)]^3
 *                     (conv_grid, kernel K, stride 1)
 *   TC_OP_CONV_T_S1   factor K in [1,8]: Minkowski sum with [-floor((K-1)/2), floor(K/2)]^3
 *                     (conv_transpose_grid, kernel K, stride 1)
 * Factors 4 and 8 (and k3s2) run chained x2 passes, each with its own readback.
 * The kernel-K ops run as sequences of TC_OP_DILATE / TC_OP_PAD_* passes (PR page
 * section 2; K in {2,3,4,5} in its test plan): the kernel's offsets are
 * [-floor((K-1)/2), floor(K/2)] per axis, the transposed conv scatters to them and
 * the conv gathers from them; K = 1 returns a copy of the source.
 * Coarsening rounds toward minus infinity. */
typedef enum tc_op {
  TC_OP_COARSEN = 1,
  TC_OP_REFINE = 2,
  TC_OP_DILATE = 3,
  TC_OP_PAD_NEG = 4,
  TC_OP_PAD_POS = 5,
  TC_OP_CONV_T_K3S2 = 6,
  TC_OP_CONV_S1 = 7,
  TC_OP_CONV_T_S1 = 8
} tc_op;

/* Caller-supplied device allocator. When an entry point is given one, all the
 * device memory of that call comes from it: the output batch's buffer (one
 * allocation per output batch, returned through `free` by tc_batch_free), the
 * scratch arrays of the passes and the intermediate batches of chained passes.
 * `alloc` returns a device pointer usable on `stream`, aligned to at least 256
 * bytes, or NULL on failure (the call then fails with TC_ERR_ALLOC, *out is NULL
 * and nothing is leaked). `free` receives the same pointer, byte count and
 * stream. Both are called from the thread that calls into the library (or, for
 * cached scratch, from the thread of a later call or of tc_scratch_release).
 * Scratch blocks are not freed at the end of a call: the library caches them
 * per (device, stream, allocator) and hands them to the next call with the
 * same key, so a steady stream of passes makes no allocator calls beyond its
 * outputs; tc_scratch_release returns the idle ones through `free`.
 * Passing a NULL tc_allocator* makes the library take all of this from the
 * device's stream-ordered pool (hipMallocAsync on the call's stream), with
 * the same caching. */
typedef struct tc_allocator {
  void* (*alloc)(void* ctx, size_t bytes, void* stream);
  void (*free)(void* ctx, void* ptr, size_t bytes, void* stream);
  void* ctx;
} tc_allocator;

typedef struct tc_grid_batch tc_grid_batch; /* opaque, owned by the caller */

/* Per-grid header (PR page section 1: every grid gets mGridIndex = g,
 * mGridCount = B, its node counts and its bbox). 80 bytes, device resident. */
typedef struct tc_grid_header {
  int32_t grid_index;   /* g */
  int32_t grid_count;   /* B */
  int32_t upper_count;  /* upper nodes (= root tiles) of this grid */
  int32_t lower_count;
  int32_t leaf_count;
  int32_t upper_begin;  /* batch-global index of the grid's first upper node */
  int32_t lower_begin;
  int32_t leaf_begin;
  int64_t voxel_count;
  int64_t voxel_begin;  /* batch-global index of the grid's first voxel */
  int32_t bbox_min[3];  /* inclusive index-space bbox of active voxels; an empty */
  int32_t bbox_max[3];  /* grid has min = INT32_MAX and max = INT32_MIN */
  int32_t reserved[2];
} tc_grid_header;

/* Device arrays of a batch, all inside one allocation (`buffer`), in canonical
 * order: grids in order; inside a grid root tiles by signed x-major tile
 * coordinate, then x-major child offsets. Layouts:
 *   upper_origin int32[N2][4]  x, y, z (multiple of 4096), grid
 *   upper_key    uint64[N2]    (Tx+2^19)<<40 | (Ty+2^19)<<20 | (Tz+2^19), T = origin/4096
 *   upper_first  int32[N2]     index of the first child lower node
 *   upper_mask   uint64[N2][512] child bit (x*32+y)*32+z of the lower inside the upper
 *   lower_origin int32[N1][4]  x, y, z (multiple of 128), parent upper index
 *   lower_first  int32[N1]     index of the first child leaf
 *   lower_mask   uint64[N1][64]  child bit (x*16+y)*16+z of the leaf inside the lower
 *   lower_prefix uint16[N1][64]  active children in words < w
 *   leaf_origin  int32[L][4]   x, y, z (multiple of 8), grid
 *   leaf_parent  int32[L]      parent lower index
 *   leaf_mask    uint64[L][8]  voxel bit n = x*64 + y*8 + z (word x, bit y*8+z)
 *   leaf_prefix  uint64[L]     seven 9-bit fields; field w-1 = voxels in words < w
 *   leaf_offset  int64[L]      0-based index of the leaf's first voxel in its grid
 * Node indices are batch-global. */
typedef struct tc_batch_info {
  int32_t grid_count;
  int32_t upper_count;
  int32_t lower_count;
  int32_t leaf_count;
  const int32_t* h_upper_counts; /* [B], host, valid for the batch's lifetime */
  const int32_t* h_lower_counts;
  const int32_t* h_leaf_counts;
  const void* d_buffer;
  size_t buffer_bytes;
  const tc_grid_header* d_headers;
  const int32_t* d_upper_origin;
  const uint64_t* d_upper_key;
  const int32_t* d_upper_first;
  const uint64_t* d_upper_mask;
  const int32_t* d_lower_origin;
  const int32_t* d_lower_first;
  const uint64_t* d_lower_mask;
  const uint16_t* d_lower_prefix;
  const int32_t* d_leaf_origin;
  const int32_t* d_leaf_parent;
  const uint64_t* d_leaf_mask;
  const uint64_t* d_leaf_prefix;
  const int64_t* d_leaf_offset;
} tc_batch_info;

/* Library version of this header; a caller checks it equals TC_ABI_VERSION. */
int32_t tc_abi_version(void);

/* Static text for a status code. */
const char* tc_status_string(tc_status status);

/* Message describing the calling thread's most recent non-TC_OK status. */
const char* tc_last_error(void);

/* Builds a batch of B grids from int32 voxel rows (the ijk front-end; PR page,
 * Measurements: follow-up ijk emission front-end, and Test plan: expected
 * topologies built from ijk).
 *   d_ijk      int32[N][3] device, N = h_offsets[B]; may be NULL when N = 0.
 *   h_offsets  int64[B+1] host: member g owns rows [h_offsets[g], h_offsets[g+1]);
 *              h_offsets[0] = 0, non-decreasing. N >= 2^30 is TC_ERR_UNSUPPORTED.
 *   Duplicate rows collapse; row order is irrelevant.
 * Blocks on a few small readbacks. *out is owned by the caller. */
tc_status tc_batch_from_ijk(const int32_t* d_ijk, const int64_t* h_offsets, int32_t grid_count,
                            const tc_allocator* allocator, void* stream, tc_grid_batch** out);

/* Builds a batch from float32 points (the points front-end beside the ijk
 * front-end; PR page, Measurements, follow-ups).
 *   d_xyz         float32[N][3] device, N = h_offsets[B]; may be NULL when N = 0.
 *   h_offsets     int64[B+1] host, as for tc_batch_from_ijk.
 *   h_voxel_size  float32[B][3] host, finite and > 0; h_origin float32[B][3] host, finite.
 *   mode          0: the voxel whose centre is nearest to the point, per axis
 *                    floor(x + 1/2) with x = (p - origin) / voxel_size computed in
 *                    float32 (a tie goes to the larger index);
 *                 1: the 8 voxels floor(x) + {0,1}^3 around the point.
 * Duplicates collapse. A point whose x is not finite is TC_ERR_INVALID_ARG, an
 * index outside int32 TC_ERR_OVERFLOW. More than 2^30 voxel rows (N, or 8N in
 * mode 1) is TC_ERR_UNSUPPORTED. Blocks on a few small readbacks. */
tc_status tc_batch_from_points(const float* d_xyz, const int64_t* h_offsets, int32_t grid_count,
                              const float* h_voxel_size, const float* h_origin, int32_t mode,
                              const tc_allocator* allocator, void* stream, tc_grid_batch** out);

/* One batched pass (or a chain of passes) over every member of `src`
 * (PR page section 1: emission, sorts, dedup, single readback, one allocation,
 * writers; section 2: box-dilate and pads; factors 4, 8 and k3s2 chain passes).
 *   op      a tc_op; factor as documented at tc_op.
 * `src` is borrowed and never modified. Blocks exactly once per pass, on one
 * readback; on return the host counts in tc_batch_info are valid and device
 * arrays are valid in stream order. Small batches (an output laid out by
 * capacities that fits in 32 MiB: at most 8 / 1 / 27 / 8 output leaves per
 * source leaf for refine / coarsen / dilate / pads, the tile and lower
 * candidates for the nodes, at most 1024 members and 262144 leaf slots) take
 * their one allocation after the node, marking and count launches, with no
 * readback before it, and read back all headers at the end (the voxel total is
 * then known too); their arrays sit at capacity offsets
 * inside the buffer and buffer_bytes is the capacity. Larger batches read the
 * per-grid node counts back first and allocate exactly.
 * Returns TC_ERR_OVERFLOW (and no batch) when any output voxel would leave int32,
 * TC_ERR_UNSUPPORTED for a non-power-of-two refine/coarsen factor. */
tc_status tc_build_batched_topology(const tc_grid_batch* src, int32_t op, int32_t factor,
                                    const tc_allocator* allocator, void* stream,
                                    tc_grid_batch** out);

/* Several generated targets of one source in one call (PR page section 1: the
 * per-iteration plan builds every target of a source; section 2: the box ops
 * and the k3s2 chain). Equivalent to n_ops calls of tc_build_batched_topology,
 * op h_ops[i] with factor h_factors[i] into out[i], on the same stream and
 * allocator, but the small-batch passes of consecutive ops are enqueued back to
 * back: each keeps its header readback pending, in a pinned host block of its
 * own, and the call waits once, at the end, for all of them (a chain's
 * intermediate passes still wait for their own counts).
 *   n_ops      >= 1; h_ops, h_factors int32[n_ops] host; out tc_grid_batch*[n_ops]
 *              host, every entry set (NULL on failure).
 * On return every out[i] is as tc_build_batched_topology leaves it. Validation
 * of every (op, factor) happens before any launch; an error in any op frees
 * every batch the call made and reports that op's status (its index in the
 * message when n_ops > 1). */
tc_status tc_build_batched_topology_many(const tc_grid_batch* src, int32_t n_ops, const int32_t* h_ops,
                                         const int32_t* h_factors, const tc_allocator* allocator,
                                         void* stream, tc_grid_batch** out);

/* Masked refine (PR page, test plan: masked refine): the voxels of `src` whose
 * keep flag is zero are dropped, the rest are refined by `factor` (2, 4 or 8),
 * as tc_build_batched_topology(TC_OP_REFINE) would refine the pruned batch.
 *   d_keep  device array of n_keep bytes, one per voxel of src in enumeration
 *           order (grid by grid, the order tc_enumerate_ijk writes); non-zero
 *           keeps the voxel. Read only; the caller keeps ownership.
 *   n_keep  must equal src's voxel total (tc_batch_voxel_total), else
 *           TC_ERR_INVALID_ARG; d_keep may be NULL only when it is 0.
 * Other arguments and the result as for tc_build_batched_topology. Blocks on the
 * voxel total (if not yet known), one flag check and the passes' readbacks. */
tc_status tc_build_masked_refine(const tc_grid_batch* src, const uint8_t* d_keep, int64_t n_keep,
                                 int32_t factor, const tc_allocator* allocator, void* stream,
                                 tc_grid_batch** out);

/* Counts (host) and device array pointers of a batch. Never blocks. */
tc_status tc_batch_get_info(const tc_grid_batch* batch, tc_batch_info* out);

/* Copies the B headers to host memory h_out (tc_grid_header[B]); this blocks on
 * `stream` (one small readback). Voxel counts and bboxes live only on the device
 * until this is called. */
tc_status tc_batch_read_headers(const tc_grid_batch* batch, tc_grid_header* h_out, void* stream);

/* Total voxel count of the batch (blocks like tc_batch_read_headers the first
 * time; cached afterwards). */
tc_status tc_batch_voxel_total(const tc_grid_batch* batch, int64_t* h_total, void* stream);

/* Writes the jagged voxel enumeration: d_ijk_out int32[V][3] device, V = voxel
 * total, grid after grid, each grid in canonical order (test plan: ijk.jdata);
 * member g's rows start at headers[g].voxel_begin. `capacity` is the row capacity
 * of d_ijk_out; fewer than V rows is TC_ERR_INVALID_ARG. Enqueues one kernel
 * (after a voxel-total readback the first time). */
tc_status tc_enumerate_ijk(const tc_grid_batch* batch, int32_t* d_ijk_out, int64_t capacity,
                           void* stream);

/* tc_enumerate_ijk of n batches in one launch (up to eight per launch, so a
 * group of small batches fills the device once instead of n times): batch j's
 * rows go to d_ijk_outs[j] (int32[V_j][3] device, capacities[j] >= V_j rows;
 * 16-byte aligned outputs take the vector stores). A NULL output is allowed for
 * a batch without voxels.
 *   n           >= 1; batches, d_ijk_outs, capacities: host arrays of n entries.
 * Every argument is checked before the launch. */
tc_status tc_enumerate_ijk_many(int32_t n, const tc_grid_batch* const* batches, int32_t* const* d_ijk_outs,
                                const int64_t* capacities, void* stream);

/* Kernel map of a convolution plan between two batches with the same member
 * count (issue page "Generated-topology grid construction dominates
 * per-iteration ConvolutionPlan cost", Measurements: a plan builds a k3 s1 map
 * on one topology and a k2s2 transposed-conv map; the layout is this library's).
 *   src, dst     source (input) and target (output) batches; read only.
 *   kernel_size  K in [1, 8]; offsets O_K = [-floor((K-1)/2), floor(K/2)] per
 *                axis, the same offset box as TC_OP_CONV_S1 / TC_OP_CONV_T_S1.
 *   stride       S in {1, 2} (others: TC_ERR_UNSUPPORTED).
 *   transposed   0: conv, target o reads source S*o + d;
 *                1: transposed conv, target o reads source (o - d)/S when S
 *                divides o - d in every component.
 *   d_out        device int32[V_dst][K^3]: row j = target voxel j in the order of
 *                tc_enumerate_ijk(dst), column k = offset d taken x-major,
 *                k = ((dx-lo)*K + (dy-lo))*K + (dz-lo) with lo = -floor((K-1)/2);
 *                the entry is the index (in the order of tc_enumerate_ijk(src))
 *                of the same member's source voxel, or -1. Owned by the caller.
 *   capacity     int32 entries available at d_out; fewer than V_dst * K^3 is
 *                TC_ERR_INVALID_ARG (d_out may be NULL only when that is 0).
 * Different member counts, K outside [1, 8] or S < 1 are TC_ERR_INVALID_ARG; a
 * source of more than INT32_MAX voxels is TC_ERR_UNSUPPORTED. Blocks on the two
 * voxel totals (if not yet known), then enqueues two kernels on `stream`. */
tc_status tc_build_kernel_map(const tc_grid_batch* src, const tc_grid_batch* dst, int32_t kernel_size,
                              int32_t stride, int32_t transposed, int32_t* d_out, int64_t capacity,
                              void* stream);

/* Kernel map with no allocation, for callers that cannot allocate device
 * memory (code under HIP graph capture, tight serving loops, harnesses that
 * forbid hipMalloc). Arguments, output and errors as for tc_build_kernel_map;
 * it calls no hipMalloc, hipFree or other allocating routine, and reads the
 * voxel totals back into host stack memory when they are not yet known.
 * Scratch: a static device array of 64 MiB per GPU, loaded with the library
 * and held by every GPU it runs on until the process ends (its device address
 * is looked up on the first call on each device). The call needs
 *   256-byte aligned: 1 KiB per source upper node + 8 bytes per target leaf and
 *   window slot (8 to 64 slots, 27 for k3 s1) + 8 bytes per target leaf;
 * beyond 64 MiB it returns TC_ERR_UNSUPPORTED before any launch and writes
 * nothing. Every call on one GPU uses the same array, and no kernel relies on
 * what an earlier call left there: calls on one stream are ordered, but calls
 * that overlap on one GPU (other streams, other threads) race on it. */
tc_status tc_build_kernel_map_noalloc(const tc_grid_batch* src, const tc_grid_batch* dst, int32_t kernel_size,
                                      int32_t stride, int32_t transposed, int32_t* d_out, int64_t capacity,
                                      void* stream);

/* ---------------------------------------------------------------------------
 * Operators on feature rows. A voxel of a batch is one row of a feature matrix,
 * row j being voxel j of tc_enumerate_ijk; a kernel map's entries are rows of
 * its source's features. Any other matrix with one row per token is taken alike.
 *
 * Conventions: matrices are row-major with unit channel stride; an input's
 * `*_stride` is the distance between rows in elements (at least 0: a stride of
 * 0 repeats one row), outputs without a stride are contiguous. No alignment
 * beyond the element's own is required; 8-bit rows and weights on 16-byte boundaries
 * take shorter paths to the same results. Nothing is allocated and nothing blocks: the calls may be
 * captured into a HIP graph. An output may not overlap an input, except where
 * said. A pointer whose array is empty may be NULL. Channels are 1 to 2^20. */
typedef enum tc_dtype { TC_F32 = 0, TC_F16 = 1, TC_BF16 = 2 } tc_dtype;

/* Root-mean-square norm of every row with the residual's addition (training form):
 *   h = x + r, rounded to dtype; s = 1 / sqrt(mean(h^2) + eps); out = h s w, rounded to dtype.
 * The norm is that of the rounded h. The sum of the squares is a 32-bit float, or a 64-bit one where
 * the squares near the ends of 32 bits, so every finite row has its norm; s is a 32-bit float (infinite
 * only where 1 / sqrt(...) leaves its range: rows below 2^-128 with an eps as small, whose out is right
 * all the same).
 *   d_x         dtype[n_rows][channels], x_stride.
 *   d_residual  dtype[n_rows][channels], residual_stride, or NULL (h = x).
 *   d_weight    weight_dtype[channels] (TC_F32, or dtype), or NULL (ones).
 *   eps         finite, >= 0.
 *   d_sum       dtype[n_rows][channels]: h, or NULL. With contiguous rows it may
 *               be d_x or d_residual itself.
 *   d_out       dtype[n_rows][channels].
 *   d_rstd      float[n_rows]: s, or NULL. */
tc_status tc_rms_norm(const void* d_x, int64_t x_stride, const void* d_residual, int64_t residual_stride,
                      const void* d_weight, int32_t weight_dtype, int64_t n_rows, int32_t channels, int32_t dtype,
                      float eps, void* d_sum, void* d_out, float* d_rstd, void* stream);

/* The same norm with an output in 8 bits and a scale for each row (serving form):
 *   p = h w, a = max over the row of |p|; q = p * (127 / a) rounded to nearest even;
 *   scale = a s / 127, so that q * scale stands for h s w.
 * p is exact in 64 bits and the norm's factor s cancels out of q, so q is the same
 * integer in any implementation that follows the line above in 64 bits.
 * A row with a = 0 has q = 0 and scale = 0; a row with an infinity or NaN in p has
 * q = 0 and scale = NaN. Other arguments as for tc_rms_norm.
 *   d_q      int8[n_rows][channels], in [-127, 127].
 *   d_scale  float[n_rows]. */
tc_status tc_rms_norm_i8(const void* d_x, int64_t x_stride, const void* d_residual, int64_t residual_stride,
                         const void* d_weight, int32_t weight_dtype, int64_t n_rows, int32_t channels, int32_t dtype,
                         float eps, void* d_sum, int8_t* d_q, float* d_scale, void* stream);

/* Gradient of tc_rms_norm. With dy the gradient of out, dh that of h by its other
 * uses (the residual stream), g = dy w and u = h s:
 *   grad_x = s (g - u mean(g u)) + dh, rounded to dtype: the gradient of x, and of r alike;
 *   grad_weight = sum over rows of dy u, a 32-bit float sum in an order that
 *   only n_rows, channels and dtype decide.
 *   d_grad_out   dtype[n_rows][channels], grad_out_stride.
 *   d_grad_sum   dh, dtype[n_rows][channels], grad_sum_stride, or NULL (zeros).
 *   d_h          h as tc_rms_norm left it (x where there is no residual), h_stride.
 *   d_rstd       float[n_rows]: s as tc_rms_norm left it.
 *   d_grad_x     dtype[n_rows][channels], or NULL. With contiguous rows it may be
 *                d_grad_sum itself.
 *   d_grad_weight float[channels], or NULL (not both NULL). Zeros without rows.
 *   d_workspace  tc_rms_norm_backward_workspace(n_rows, channels) bytes, 16-byte
 *                aligned, read and written in stream order; may be NULL when
 *                d_grad_weight is. */
tc_status tc_rms_norm_backward(const void* d_grad_out, int64_t grad_out_stride, const void* d_grad_sum,
                               int64_t grad_sum_stride, const void* d_h, int64_t h_stride, const void* d_weight,
                               int32_t weight_dtype, const float* d_rstd, int64_t n_rows, int32_t channels,
                               int32_t dtype, void* d_grad_x, float* d_grad_weight, void* d_workspace,
                               int64_t workspace_bytes, void* stream);

/* Bytes of d_workspace; 0 for arguments that tc_rms_norm_backward refuses. */
int64_t tc_rms_norm_backward_workspace(int64_t n_rows, int32_t channels);

/* Product of 8-bit rows with 8-bit weights, scales per row and per output channel:
 *   out[m][n] = x_scale[m] * w_scale[n] * sum_c x[m][c] w[n][c] + bias[n], rounded to out_dtype.
 * The sum is exact (int32); the rest is 32-bit float.
 *   d_x        int8[n_rows][c_in], x_stride; d_x_scale float[n_rows].
 *   d_w        int8[c_out][c_in], w_stride;  d_w_scale float[c_out].
 *   d_bias     float[c_out], or NULL.
 *   c_in       1 to 131071 (more could leave int32: TC_ERR_UNSUPPORTED).
 *   d_out      out_dtype[n_rows][c_out], out_stride >= c_out elements. */
tc_status tc_matmul_i8(const int8_t* d_x, int64_t x_stride, const float* d_x_scale, const int8_t* d_w,
                       int64_t w_stride, const float* d_w_scale, const float* d_bias, int64_t n_rows, int32_t c_out,
                       int32_t c_in, int32_t out_dtype, void* d_out, int64_t out_stride, void* stream);

/* The same product over a kernel map: the convolution a map of tc_build_kernel_map
 * stands for, with the rows in 8 bits:
 *   out[j][n] = w_scale[n] * sum_t x_scale[i] * sum_c x[i][c] w[t][n][c] + bias[n], i = map[j][t],
 * rounded to out_dtype; a tap whose entry lies outside [0, n_src) adds nothing.
 * Sums over channels are exact (int32), the sum over taps is a 32-bit float sum
 * in an order that only the sizes decide.
 *   d_x       int8[n_src][c_in], x_stride; d_x_scale float[n_src].
 *   d_map     int32[n_dst][taps], taps in [1, 512].
 *   d_w       int8[taps][c_out][c_in], contiguous; d_w_scale float[c_out].
 * n_src is at most INT32_MAX. Other arguments as for tc_matmul_i8. */
tc_status tc_sparse_conv_i8(const int8_t* d_x, int64_t x_stride, const float* d_x_scale, int64_t n_src,
                            const int32_t* d_map, int64_t n_dst, int32_t taps, const int8_t* d_w,
                            const float* d_w_scale, const float* d_bias, int32_t c_out, int32_t c_in,
                            int32_t out_dtype, void* d_out, int64_t out_stride, void* stream);

/* Layer norm of every row with the residual's addition (training form):
 *   h = x + r, rounded to dtype; m = mean(h), s = 1 / sqrt(mean((h - m)^2) + eps);
 *   out = (h - m) s w + b, rounded to dtype.
 * The norm is that of the rounded h. m is a 64-bit sum, held as two floats, so that rows far from zero keep
 * the digits of their spread; the squares' sum is a 32-bit float, or a 64-bit one where the squares near the
 * ends of 32 bits, so every finite row has its norm.
 *   d_x         dtype[n_rows][channels], x_stride.
 *   d_residual  dtype[n_rows][channels], residual_stride, or NULL (h = x).
 *   d_weight    weight_dtype[channels] (TC_F32, or dtype), or NULL (ones).
 *   d_bias      bias_dtype[channels] (TC_F32, or dtype), or NULL (zeros).
 *   eps         finite, >= 0.
 *   d_sum       dtype[n_rows][channels]: h, or NULL. With contiguous rows it may
 *               be d_x or d_residual itself.
 *   d_out       dtype[n_rows][channels].
 *   d_mean      float[n_rows]: m rounded to 32 bits, or NULL.
 *   d_rstd      float[n_rows]: s (infinite where it leaves 32 bits), or NULL. */
tc_status tc_layer_norm(const void* d_x, int64_t x_stride, const void* d_residual, int64_t residual_stride,
                        const void* d_weight, int32_t weight_dtype, const void* d_bias, int32_t bias_dtype,
                        int64_t n_rows, int32_t channels, int32_t dtype, float eps, void* d_sum, void* d_out,
                        float* d_mean, float* d_rstd, void* stream);

/* Gradient of tc_layer_norm. With dy the gradient of out, dh that of h by its other
 * uses (the residual stream), g = dy w and u = (h - m) s:
 *   grad_x = s (g - mean(g) - u mean(g u)) + dh, rounded to dtype: the gradient of x, and of r alike;
 *   grad_weight = sum over rows of dy u, grad_bias = sum over rows of dy: 32-bit float sums in an order
 *   that only n_rows, channels and dtype decide.
 * m is h's mean as the row has it; d_mean, its rounding to 32 bits, is where the sums start from. A row whose s is
 * infinite (a spread below 2^-128 with eps = 0) makes its grad_x and all of grad_weight NaN.
 *   d_grad_out    dtype[n_rows][channels], grad_out_stride.
 *   d_grad_sum    dh, dtype[n_rows][channels], grad_sum_stride, or NULL (zeros).
 *   d_h           h as tc_layer_norm left it (x where there is no residual), h_stride.
 *   d_mean, d_rstd  float[n_rows] as tc_layer_norm left them.
 *   d_grad_x      dtype[n_rows][channels], or NULL. With contiguous rows it may be
 *                 d_grad_sum itself.
 *   d_grad_weight, d_grad_bias  float[channels], or NULL (not all three NULL). Zeros without rows.
 *   d_workspace   tc_layer_norm_backward_workspace(n_rows, channels) bytes, 16-byte
 *                 aligned, read and written in stream order; may be NULL when
 *                 d_grad_weight and d_grad_bias are. */
tc_status tc_layer_norm_backward(const void* d_grad_out, int64_t grad_out_stride, const void* d_grad_sum,
                                 int64_t grad_sum_stride, const void* d_h, int64_t h_stride, const void* d_weight,
                                 int32_t weight_dtype, const float* d_mean, const float* d_rstd, int64_t n_rows,
                                 int32_t channels, int32_t dtype, void* d_grad_x, float* d_grad_weight,
                                 float* d_grad_bias, void* d_workspace, int64_t workspace_bytes, void* stream);

/* Bytes of d_workspace; 0 for arguments that tc_layer_norm_backward refuses. */
int64_t tc_layer_norm_backward_workspace(int64_t n_rows, int32_t channels);

/* Rotary positions: the pairs of every head of a row are turned by angles that the row's
 * integer coordinates decide (a voxel's x, y, z as tc_enumerate_ijk gives them, or a token's time,
 * height and width). Pair i of an axis a has the angle t = positions[row][a] * freqs[i] radians:
 *   (x1, x2) -> (x1 cos t - x2 sin t, x1 sin t + x2 cos t), rounded to dtype;
 * with `inverse` by -t, which is the gradient too. Any coordinate and finite frequency: angles are
 * reduced in 64 bits, and cos and sin are off by at most 2^-23.
 *   d_x          dtype[n_rows][heads][dim] with unit stride in a head, x_row_stride and
 *                x_head_stride elements between rows and heads (at least 0). dim 2 to 4096, heads 1 to 2^20.
 *   d_positions  int32[n_rows][n_axes], position_stride elements between rows (at least 0).
 *   h_sections   host int32[n_axes], n_axes 1 to 4: how many pairs each axis turns, one axis's pairs after
 *                another's (an axis may have none); together `pairs`, 1 to dim / 2.
 *   d_freqs      float[pairs]: radians for a step along the pair's axis.
 *   interleaved  1: pair i is channels 2 i and 2 i + 1; 0: channels i and pairs + i.
 *                Channels from 2 * pairs on are copied.
 *   d_out        dtype[n_rows][heads][dim] with its own strides; rows and heads may not overlap
 *                one another. It may be d_x itself, with the same strides, or else share no element with it
 *                (other parts of the same rows, heads or rows between its own). An overlap is refused, and so are
 *                different strides of the two that interleave more than 2^18 times. */
tc_status tc_rotary(const void* d_x, int64_t x_row_stride, int64_t x_head_stride, int64_t n_rows, int32_t heads,
                    int32_t dim, int32_t dtype, const int32_t* d_positions, int64_t position_stride, int32_t n_axes,
                    const int32_t* h_sections, const float* d_freqs, int32_t interleaved, int32_t inverse, void* d_out,
                    int64_t out_row_stride, int64_t out_head_stride, void* stream);

/* Rows in microscaled 4 bits: blocks of 32 channels under one power of two (the last
 * block of a row may have fewer). A value is sign, two bits of exponent and one of
 * mantissa: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives (codes 0 to 7, 8 to 15). Of a block with the largest
 * magnitude a:
 *   E = max(floor(log2 a) - 2, -127), or -127 for a = 0; q = x 2^-E rounded to nearest even, at most 6;
 *   scale = E + 127, so that q 2^(scale - 127) stands for x.
 * A block with an infinity or NaN has q = 0 and scale = 255, which stands for NaN.
 *   d_x      dtype[n_rows][channels], x_stride.
 *   d_q      uint8[n_rows][ceil(channels / 2)], contiguous: channel 2 i in the low four bits of byte i, 2 i + 1
 *            in the high ones (0 beyond an odd number of channels).
 *   d_scale  uint8[n_rows][ceil(channels / 32)], contiguous. */
tc_status tc_quantise_mx4(const void* d_x, int64_t x_stride, int64_t n_rows, int32_t channels, int32_t dtype,
                          uint8_t* d_q, uint8_t* d_scale, void* stream);

/* The values that such rows stand for, rounded to out_dtype (NaN under a scale of 255; a value beyond out_dtype's
 * range is infinite).
 *   d_q      uint8[n_rows][ceil(channels / 2)], q_stride bytes; d_scale uint8[n_rows][ceil(channels / 32)],
 *            scale_stride bytes.
 *   d_out    out_dtype[n_rows][channels], contiguous. */
tc_status tc_dequantise_mx4(const uint8_t* d_q, int64_t q_stride, const uint8_t* d_scale, int64_t scale_stride,
                            int64_t n_rows, int32_t channels, int32_t out_dtype, void* d_out, void* stream);

/* Product of such rows with such weights:
 *   out[m][n] = sum over blocks of 2^(x_scale + w_scale - 254) sum_c x[m][c] w[n][c] + bias[n], rounded to out_dtype.
 * Sums are 32-bit floats in an order that only the sizes, alignments and strides decide. A scale of 255 makes the outputs that its block
 * goes into NaN. Sums beyond 32 bits are infinite, or NaN.
 *   d_x      uint8[n_rows][ceil(c_in / 2)], x_stride bytes; d_x_scale uint8[n_rows][ceil(c_in / 32)],
 *            x_scale_stride bytes. The high bits of the last byte of an odd c_in may hold anything.
 *   d_w      uint8[c_out][ceil(c_in / 2)], w_stride; d_w_scale uint8[c_out][ceil(c_in / 32)], w_scale_stride.
 *   d_bias   float[c_out], or NULL.
 *   d_out    out_dtype[n_rows][c_out], out_stride >= c_out elements. */
tc_status tc_matmul_mx4(const uint8_t* d_x, int64_t x_stride, const uint8_t* d_x_scale, int64_t x_scale_stride,
                        const uint8_t* d_w, int64_t w_stride, const uint8_t* d_w_scale, int64_t w_scale_stride,
                        const float* d_bias, int64_t n_rows, int32_t c_out, int32_t c_in, int32_t out_dtype,
                        void* d_out, int64_t out_stride, void* stream);

/* Cached device memory: every call takes its scratch arrays (and the buffers
 * of intermediate batches) from blocks cached process-wide per device, stream
 * and allocator, and keeps them for the next call with the same key (reuse is
 * ordered by that stream, so none is waited for). At most 24 idle blocks and
 * 8 GiB of idle bytes stay cached; beyond that the least recently used are
 * freed. tc_batch_free likewise keeps the buffer of a batch built without an
 * allocator (up to 64 buffers, 4 GiB) for the next batch on the same device
 * and stream. tc_scratch_release synchronizes the device, then frees every idle
 * scratch block (through its allocator's `free`, or to the device's pool) and
 * every cached batch buffer; later calls allocate again. Blocks in use by a
 * concurrent call are kept. Fails only with a HIP error. */
tc_status tc_scratch_release(void);

/* Releases the batch's device buffer (through the allocator it was created with,
 * stream-ordered on its creation stream) and the handle. NULL is ignored. */
void tc_batch_free(tc_grid_batch* batch);

/* Testing hook for the TC_ERR_INTERNAL path above: the next batch that the
 * calling thread builds (from ijk, from points, or as the output or an
 * intermediate of a pass) behaves as if its leaf-mask writers had flagged
 * `bits` (1 or 2; 0 cancels). That batch is written normally and its flags are
 * read back with its voxel total, so the error surfaces where a real one
 * would. Bits outside [0, 3] are TC_ERR_INVALID_ARG. */
tc_status tc_debug_inject_flags(int32_t bits);

/* Testing hook for the large-batch form of the box ops' leaf gather: while `on`
 * is 1, the calling thread's dilate and pad passes read their source arrays
 * through 64-bit addresses, as they do by themselves when a source array is
 * 2 GiB or more; 0 restores the default (32-bit buffer offsets below that
 * size). Results are the same either way. Values other than 0 and 1 are
 * TC_ERR_INVALID_ARG. */
tc_status tc_debug_wide_loads(int32_t on);

/* Kernel timing for measurement: while enabled, every launch of a kernel whose
 * name is in `kernel_names` (comma-separated __global__ function names, e.g.
 * "k_leaf_gather,k_enumerate"; "*" selects every kernel) is bracketed by HIP
 * events on the stream it is launched on. tc_profile_read() waits for those
 * events and returns the summed milliseconds and launch count of one kernel
 * since tc_profile_enable(). Not thread-safe against concurrent passes. */
tc_status tc_profile_enable(const char* kernel_names);
tc_status tc_profile_read(const char* kernel_name, double* h_total_ms, int64_t* h_launches);
tc_status tc_profile_disable(void);

#ifdef __cplusplus
}
#endif

#endif /* TOPO_H */
