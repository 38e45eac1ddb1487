/*
 * vg.h — C ABI of the GB300 (sm_103a) submanifold sparse 3D convolution library
 * (libvoxelgemm.so).
 *
 * The operator is the submanifold convolution of "Contribution Tasks —
 * JeffreyXiang/FlexGEMM", §一 (positioning) and §二 (architecture map; "how one
 * call flows through the modules"; key types and functions table):
 * sparse_submanifold_conv3d(feats, coords, shape, weight, bias) evaluates a
 * 3x3x3 convolution only at the active voxels, through a neighbour map that is
 * built once from a coordinate hash map and reused by the forward and the
 * backward pass (the page's neighbor_cache).  The kernel interface in "From
 * CUDA to Triton: Triton JIT and autotuning", §六 6.2 (signature of
 * sparse_submanifold_conv_fwd_masked_implicit_gemm_kernel) fixes V = 27 taps,
 * a uint32 neighbour table, a row order (sorted_idx) and a contraction over
 * V * Ci.
 *
 * Conventions used by every call below:
 *  - tap k <-> offset (dx,dy,dz) in {-1,0,1}^3 with k = 9(dx+1) + 3(dy+1) + (dz+1);
 *    k = 13 is the centre and o_{26-k} = -o_k.
 *  - nbr[i][k] = j when voxel j sits at coord_i + o_k in the same batch element,
 *    else VG_NONE; mask[i] bit k is set iff nbr[i][k] != VG_NONE.  A neighbour
 *    outside the grid is absent (no wrap, no padding).  Row indices are the
 *    caller's row order.
 *  - forward:  out[i][co] = bias[co] + sum_k sum_ci W[k][ci][co] * feats[nbr[i][k]][ci]
 *    input gradient:  dX[j] = sum over (i,k) with nbr[i][k] = j of W_k dY[i]
 *    weight gradient: dW[k][ci][co] = sum_i f[nbr[i][k]][ci] * dY[i][co];  db = sum_i dY[i]
 *  - Every pointer argument is a DEVICE pointer (cudaMalloc'd or equivalent),
 *    row-major and contiguous, owned by the caller; the library allocates no
 *    memory and keeps no global state.  `stream` is a cudaStream_t (NULL = the
 *    legacy default stream).  Calls are stream-ordered and asynchronous unless
 *    stated otherwise.
 *  - Argument errors are detected on the host before anything is launched and
 *    returned as a status code; nothing is written in that case.
 *  - Accumulation is fp32 on every path; outputs are rounded to the input
 *    dtype with round-to-nearest-even.
 *  - N < 2^31 rows.
 */
#ifndef VOXEL_GEMM_VG_H
#define VOXEL_GEMM_VG_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define VG_API __attribute__((visibility("default")))
#else
#define VG_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

/* ---- status codes ---------------------------------------------------------------- */
#define VG_OK                       0
#define VG_ERR_INVALID_ARG          1  /* null pointer, bad size, misaligned pointer     */
#define VG_ERR_COORD_OUT_OF_RANGE   2  /* a coordinate outside [0,B)x[0,X)x[0,Y)x[0,Z)    */
#define VG_ERR_DUPLICATE_COORD      3  /* two rows with the same (b,x,y,z)               */
#define VG_ERR_HASH_FULL            4  /* the voxel hash table overflowed                */
#define VG_ERR_UNSUPPORTED          5  /* channel counts/dtype/flags this build does not run */
#define VG_ERR_WORKSPACE_TOO_SMALL  6  /* ws_bytes below the matching *_workspace_bytes() */
#define VG_ERR_CUDA                 7  /* a CUDA runtime call or launch failed           */
#define VG_ERR_DEVICE_TIMEOUT       8  /* a bounded device-side wait gave up (kernel returned early) */

/* ---- element types ---------------------------------------------------------------- */
#define VG_F32   0
#define VG_F16   1
#define VG_BF16  2

/* ---- flags -------------------------------------------------------------------------- */
#define VG_KEY32            0x1u   /* force 32-bit hash keys (needs B*X*Y*Z < 2^32)    */
#define VG_KEY64            0x2u   /* force 64-bit hash keys                            */
#define VG_ORDER_HILBERT    0x4u   /* row order from the Hilbert code instead of Morton  */
/* Map-build flags: how the probe finds a voxel's neighbours.  The hash table
 * is the pages' method.  The column index counts the voxels of every (b, x, y)
 * column, prefix-sums the counts, stores each column's voxels sorted by z, and
 * searches a voxel's 9 neighbouring columns for z - 1, z, z + 1; it needs
 * B*X*Y <= 2^28.  By default the column index is used when the hash table would
 * exceed 64 MiB (so would not stay in the GPU's L2) and B*X*Y <= 8 N + 2^20;
 * VG_MAP_HASH or VG_MAP_COLUMNS forces one (both: VG_ERR_INVALID_ARG;
 * VG_MAP_COLUMNS on a larger grid: VG_ERR_UNSUPPORTED).  The map, the row order
 * and the tiles are identical either way. */
#define VG_MAP_HASH         0x8u
#define VG_MAP_COLUMNS      0x40u
/* Testing aid: size the hash table below N so that the overflow path
 * (VG_ERR_HASH_FULL) can be exercised from the host. */
#define VG_TEST_SMALL_HASH  0x100u
/* Convolution flag: fp32 features may run on the tensor cores as TF32 (inputs
 * read with a 10-bit mantissa, products accumulated in fp32), as the pages'
 * allow_tf32 switch does ("From CUDA to Triton: Triton JIT and autotuning",
 * §六 6.2: allow_tf32 is part of the autotune key and of the kernel arguments).
 * Applies to fp32 with Cin and Cout multiples of 32 (forward, input gradient and
 * weight gradient); otherwise, and without the flag, fp32 runs on the exact FFMA
 * path. */
#define VG_ALLOW_TF32       0x10u
/* Convolution flag: on the tensor-core paths, keep one work unit per (128-row
 * tile, output-channel block) even when there are fewer such units than SMs.
 * By default a small problem (the pages' inference benchmark case: few voxels)
 * cuts each unit's taps into up to 6 groups that run on separate SMs and writes
 * fp32 partial sums, which a second kernel adds in group order (deterministic)
 * before the bias and the rounding; this flag turns that off, for comparisons.
 * Results agree within rounding either way. */
#define VG_NO_SMALL_N_SPLIT 0x20u

#define VG_NONE 0xFFFFFFFFu        /* missing neighbour in nbr                          */
#define VG_TILE_ROWS 128           /* rows per tile of the sorted order (tile masks)    */

/* Human-readable name of a status code (static string). */
VG_API const char* vg_strerror(int status);

/* Library version as 10000*major + 100*minor + patch. */
VG_API int vg_version(void);

/* ======================================================================================
 * Neighbour map (hash build, 27-tap probe, valid-tap mask, Morton row order, tile masks)
 * Follows the page's hashmap_insert_3d_idx_as_val + subm_neighbor_map +
 * migemm_neighmap_pp steps ("Contribution Tasks — JeffreyXiang/FlexGEMM", §二,
 * module table rows kernels.cuda.hash and kernels.cuda.spconv; init_hashmap picks
 * uint32 or uint64 keys by grid volume).  Reading taken: 64-bit keys iff
 * B*X*Y*Z >= 2^30, unless VG_KEY32/VG_KEY64 forces the width; the map itself is
 * identical either way, and identical again when a column index replaces the
 * hash table (VG_MAP_HASH).
 * ====================================================================================== */

/* Bytes of device workspace vg_nbrmap_build needs for these sizes and flags
 * (0 if the arguments are invalid).  The workspace is the neighbour cache: it
 * holds the hash table (or the column index), the sorted row order and the per-tile masks, and must
 * stay alive and unmodified while convolutions use the map. */
VG_API size_t vg_nbrmap_workspace_bytes(int64_t N, int B, int X, int Y, int Z, unsigned flags);

/* Build the neighbour map of N voxels.
 *   coords  [N][4] int32 (b,x,y,z), 16-byte aligned
 *   ws      workspace of >= vg_nbrmap_workspace_bytes(...) bytes, 256-byte aligned
 *   nbr     [N][27] uint32 output (original row order), mask [N] uint32 output
 * Asynchronous: argument errors are returned at once; data-dependent errors
 * (out-of-range or duplicate coordinates, hash overflow) are recorded on the
 * device in ws and returned by vg_nbrmap_status().  The convolution calls read
 * that record on the device and write nothing when the map is bad. */
VG_API int vg_nbrmap_build(const int32_t* coords, int64_t N, int B, int X, int Y, int Z,
                    unsigned flags, void* ws, size_t ws_bytes,
                    uint32_t* nbr, uint32_t* mask, void* stream);

/* Synchronises `stream` and returns the data-dependent status of the last build
 * into ws (VG_OK, VG_ERR_COORD_OUT_OF_RANGE, VG_ERR_DUPLICATE_COORD,
 * VG_ERR_HASH_FULL or VG_ERR_DEVICE_TIMEOUT when a bounded wait of the sort
 * gave up; the first in that order if several apply). */
VG_API int vg_nbrmap_status(const void* ws, void* stream);

/* Device pointers into a built workspace (no device access, no sync):
 *   sorted_idx [N] uint32 — row r of the processing order is voxel sorted_idx[r]
 *                (the page's sorted_idx).  Stable sort by the key
 *                ((m >> F) << (27 + G)) | (mask << G) | ((m & (2^F - 1)) >> (F - G)),
 *                where m = (b << 3L) | bit-interleave(x, y, z) is the Morton code
 *                (with VG_ORDER_HILBERT: m = (b << 3L) | Hilbert code of (x, y, z) with
 *                L bits, as vg_encode_seq computes it),
 *                L = ceil(log2(max(X,Y,Z))), F = min(3L, 30) and G = min(F, 6),
 *                lowered to 32 - 27 - (bits of m above F) when that makes the
 *                whole key fit 32 bits (4 radix passes instead of 5):
 *                batch element (or 1024^3-voxel Morton block of a larger grid),
 *                then the valid-tap mask, then the
 *                top G fine Morton bits (at most a 4x4x4 split of the block), then the
 *                input order (stable).
 *   tile_mask  [ceil(N/128)] uint32 — OR of mask over sorted rows [128t, 128t+128) */
VG_API const uint32_t* vg_nbrmap_sorted_idx(const void* ws);
VG_API const uint32_t* vg_nbrmap_tile_mask(const void* ws, int64_t N);
/*   sorted_nbr [ceil(N/128)*128][27] uint32 — sorted_nbr[r][k] = nbr[sorted_idx[r]][k],
 *                rows past N are VG_NONE (the map in processing order, so a tile's
 *                neighbour lists are one contiguous 13.5 KB block). */
VG_API const uint32_t* vg_nbrmap_sorted_nbr(const void* ws, int64_t N);

/* Host-only description of the build plan (no device work):
 *   info[0] = how neighbours are looked up: 0 hash table with 32-bit keys, 1 hash
 *   table with 64-bit keys, 2 column index (see VG_MAP_HASH); info[1] = significant bits of the
 *   sort key above, info[2] = radix-sort passes, info[3] = kernels launched by
 *   vg_nbrmap_build (memsets not counted).
 *   sm_count: SMs of the device the plan is for; 0 = the current device's (the
 *   launch grids and the workspace size follow the SM count; without any CUDA
 *   device, 0 plans for 152 SMs).  Returns VG_OK or VG_ERR_INVALID_ARG. */
VG_API int vg_nbrmap_describe(int64_t N, int B, int X, int Y, int Z, unsigned flags, int sm_count,
                              int info[4]);

/* ======================================================================================
 * Convolution (forward, input gradient, weight/bias gradient)
 * The masked implicit GEMM of "From CUDA to Triton: Triton JIT and autotuning",
 * §六 6.2 (kernel arguments input, weight, bias, neighbor, sorted_idx, output;
 * contraction V * Ci) and its backward ("Contribution Tasks — JeffreyXiang/FlexGEMM",
 * §二 call flow: the backward reuses the neighbour cache and returns feats.grad
 * and weight.grad).
 *   dtype: VG_F32 (fp32 FFMA path; with VG_ALLOW_TF32 and Cin, Cout multiples
 *          of 32 all three passes run on the tensor cores as TF32), VG_F16 or
 *          VG_BF16 (tensor-core path when Cin and Cout are
 *          multiples of 64, CUDA-core path otherwise).
 *   Cin and Cout must be multiples of 8 (VG_ERR_UNSUPPORTED otherwise); flags
 *   is 0 or a combination of VG_ALLOW_TF32 and VG_NO_SMALL_N_SPLIT (other bits:
 *   VG_ERR_UNSUPPORTED); the conv workspace size depends on the flags.
 *   feats [N][Cin], weight [27][Cin][Cout], bias [Cout] (or NULL), out [N][Cout],
 *   all of `dtype`, 16-byte aligned.
 *   nbr_ws/nbr/mask: a map built by vg_nbrmap_build for the same N.
 *   conv_ws: >= vg_conv_workspace_bytes(...) bytes, 256-byte aligned; holds the
 *   repacked weights, split-K partial sums, dY in processing order (16-bit
 *   tensor-core path with Cout >= 128, and TF32) and a device error record.  Calls that may overlap on
 *   the GPU (different streams) need their own conv_ws each; they may share
 *   nbr_ws/nbr/mask, which conv calls only read.
 * ====================================================================================== */

/* Bytes of conv workspace needed by vg_subm_conv3d_fwd/bwd for these sizes. */
VG_API size_t vg_conv_workspace_bytes(int64_t N, int Cin, int Cout, int dtype, unsigned flags);

/* Host-only description of the convolution plan (no device work):
 *   info[0] = 1 on the 16-bit tensor-core path, 2 when the fp32 passes run on the
 *   tensor cores as TF32, else 0, info[1] = split-K chunks of the weight
 *   gradient, info[2] = kernels launched by a forward call, info[3] = kernels
 *   launched by a backward call producing all three gradients (memsets not
 *   counted).  sm_count as in vg_nbrmap_describe (the split-K chunk count and
 *   the workspace size follow it; vg_conv_workspace_bytes and the conv calls
 *   use the current device's).  Returns VG_OK or the status vg_subm_conv3d_fwd
 *   would return for these sizes. */
VG_API int vg_conv_describe(int64_t N, int Cin, int Cout, int dtype, unsigned flags, int sm_count,
                            int info[4]);

VG_API int vg_subm_conv3d_fwd(const void* nbr_ws, const uint32_t* nbr, const uint32_t* mask, int64_t N,
                       int dtype, const void* feats, const void* weight, const void* bias,
                       void* out, int Cin, int Cout, unsigned flags,
                       void* conv_ws, size_t conv_ws_bytes, void* stream);

/* Backward.  grad_out [N][Cout]; outputs grad_feats [N][Cin], grad_weight
 * [27][Cin][Cout], grad_bias [Cout]; each output may be NULL to skip it.
 * grad_weight is reduced over split-K chunks in a fixed order (bitwise
 * deterministic run to run). */
VG_API int vg_subm_conv3d_bwd(const void* nbr_ws, const uint32_t* nbr, const uint32_t* mask, int64_t N,
                       int dtype, const void* grad_out, const void* feats, const void* weight,
                       void* grad_feats, void* grad_weight, void* grad_bias,
                       int Cin, int Cout, unsigned flags,
                       void* conv_ws, size_t conv_ws_bytes, void* stream);

/* Synchronises `stream` and returns VG_ERR_DEVICE_TIMEOUT if a kernel of the
 * most recent vg_subm_conv3d_fwd/bwd call on conv_ws gave up a bounded
 * device-side wait (its outputs are then incomplete), else VG_OK.  Every
 * fwd/bwd call clears this record when it starts. */
VG_API int vg_conv_status(void* conv_ws, void* stream);


/* ======================================================================================
 * Regular sparse convolution: strided (down-sampling) and transposed (up-sampling)
 * "Contribution Tasks — JeffreyXiang/FlexGEMM", §二 module table and key functions:
 * sparse_conv3d and kernels.cuda.spconv sparse_neighbor_map -- a convolution whose
 * output sites differ from its input sites.  The pages give no formula; the reading
 * taken is the convolution torch's dense conv3d computes on the densified grid, kept
 * at the output sites whose window holds an active input:
 *   kernel K in {2, 3} per axis (padding 0 for K = 2, 1 for K = 3), stride s in {1, 2};
 *   output grid Xo = (X + 2p - K) / s + 1 (floor), likewise Yo, Zo, same batch count;
 *   tap k = (tx*K + ty)*K + tz <-> offset d_k = (tx - p, ty - p, tz - p), taps = K^3;
 *   output site o is active iff an input sits at s*o + d_k for some k;
 *   output rows are numbered in ascending linear key ((b*Xo + x)*Yo + y)*Zo + z.
 * Strided forward:    out[o] = bias + sum_k W_k^T f[down[o][k]]         (f: input sites)
 * Transposed forward: out[j] = bias + sum_k W_k^T g[up[j][k]]           (g: output sites)
 *   (the dense equivalent is conv_transpose3d with the same K, s, p, output at the input sites)
 * W is [taps][Cin][Cout].  The backward passes run the same kernels as the
 * submanifold convolution (input gradient through the other map with W_k
 * transposed, weight gradient split-K with a fixed-order reduce).
 * ====================================================================================== */

/* A built regular-convolution map: host struct filled by vg_sparse_map_build.  Every
 * pointer points into the map workspace (device memory) and stays valid while it does. */
typedef struct {
    int64_t n_in;               /* input sites (rows of coords)                          */
    int64_t n_out;              /* output sites                                          */
    int kernel, stride, taps;   /* taps = kernel^3                                        */
    int out_grid[4];            /* B, Xo, Yo, Zo                                          */
    const void* side_in;        /* row order and tiles of the input sites (device)        */
    const void* side_out;       /* row order and tiles of the output sites (device)       */
    const uint32_t* down;       /* [n_out][27]: input row at stride*o + d_k, else VG_NONE */
    const uint32_t* down_mask;  /* [n_out]: bit k set iff down[o][k] is valid             */
    const uint32_t* up;         /* [n_in][27]: output row o with stride*o + d_k = coord   */
    const uint32_t* up_mask;    /* [n_in]                                                 */
    const int32_t* coords_out;  /* [n_out][4] (b, x, y, z) in the output grid             */
} vg_sparse_map;

/* Bytes of map workspace for N input sites (0 if the arguments are invalid); flags:
 * 0 or VG_ORDER_HILBERT.  Sized for the largest possible number of output sites. */
VG_API size_t vg_sparse_map_workspace_bytes(int64_t N, int B, int X, int Y, int Z, int kernel, int stride,
                                            unsigned flags);
/* Build the map of N input sites coords [N][4] (device, int32, 16-byte aligned) into
 * ws (device, 256-byte aligned).  SYNCHRONISES `stream`: the number of output sites
 * is data-dependent and returned in map->n_out.  Returns VG_OK, an argument error,
 * VG_ERR_COORD_OUT_OF_RANGE / VG_ERR_DUPLICATE_COORD for bad input sites (map->n_out
 * is then 0 and convolutions on the map write nothing), VG_ERR_HASH_FULL or
 * VG_ERR_DEVICE_TIMEOUT. */
VG_API int vg_sparse_map_build(const int32_t* coords, int64_t N, int B, int X, int Y, int Z, int kernel,
                               int stride, unsigned flags, void* ws, size_t ws_bytes, vg_sparse_map* map,
                               void* stream);
/* Conv workspace for a pass on `map` (transposed = 0: strided, input sites -> output
 * sites; 1: transposed, output sites -> input sites), as vg_conv_workspace_bytes. */
VG_API size_t vg_sparse_conv_workspace_bytes(const vg_sparse_map* map, int transposed, int Cin, int Cout,
                                             int dtype, unsigned flags);
/* Forward.  transposed = 0: feats [n_in][Cin] -> out [n_out][Cout];  transposed = 1:
 * feats [n_out][Cin] -> out [n_in][Cout].  Conventions, dtypes, flags and errors as
 * vg_subm_conv3d_fwd; asynchronous. */
VG_API int vg_sparse_conv3d_fwd(const vg_sparse_map* map, int transposed, int dtype, const void* feats,
                                const void* weight, const void* bias, void* out, int Cin, int Cout,
                                unsigned flags, void* conv_ws, size_t conv_ws_bytes, void* stream);
/* Backward: grad_out has the forward output's rows, grad_feats the forward input's;
 * grad_weight [taps][Cin][Cout], grad_bias [Cout]; each output may be NULL. */
VG_API int vg_sparse_conv3d_bwd(const vg_sparse_map* map, int transposed, int dtype, const void* grad_out,
                                const void* feats, const void* weight, void* grad_feats, void* grad_weight,
                                void* grad_bias, int Cin, int Cout, unsigned flags, void* conv_ws,
                                size_t conv_ws_bytes, void* stream);

/* ======================================================================================
 * Serialisation: space-filling-curve codes of voxel coordinates
 * "Contribution Tasks — JeffreyXiang/FlexGEMM", §二 module table (kernels.cuda.serialize:
 * z_order_encode/decode, hilbert_encode/decode) and the ops layer's
 * encode_seq/decode_seq(coords, shape, mode).  The pages give the names only; the
 * reading taken: code = (b << 3*bits) | curve(x, y, z) for x, y, z in [0, 2^bits).
 *   VG_CURVE_ZORDER:  bit j of x, y, z at bit 3j+2, 3j+1, 3j of the curve part.
 *   VG_CURVE_HILBERT: J. Skilling's Hilbert curve ("Programming the Hilbert curve",
 *                     AIP Conf. Proc. 707, 2004): consecutive codes are face
 *                     neighbours; its transposed index is interleaved like a z-order
 *                     code, x before y before z at each level.
 * The neighbour-map build can use either curve for its row order (VG_ORDER_HILBERT).
 * ====================================================================================== */
#define VG_CURVE_ZORDER  0
#define VG_CURVE_HILBERT 1

/* codes[i] (uint64, device) of coords[i] = (b,x,y,z) (int32 [N][4], device, 16-byte
 * aligned), bits in [0, 20].  A row whose x, y or z lies outside [0, 2^bits), or whose
 * b is negative or does not fit above the curve bits (b >= 2^(63 - 3*bits)), gets
 * the code 0xFFFFFFFFFFFFFFFF.  Asynchronous; VG_ERR_INVALID_ARG for bad sizes,
 * modes or pointers. */
VG_API int vg_encode_seq(const int32_t* coords, int64_t N, int bits, int mode, uint64_t* codes, void* stream);
/* The inverse: coords[i] = (b,x,y,z) of codes[i] (the bits above 3*bits are b). */
VG_API int vg_decode_seq(const uint64_t* codes, int64_t N, int bits, int mode, int32_t* coords, void* stream);

/* ======================================================================================
 * Data-parallel gradient exchange
 * The pages describe a single-GPU operator library and have no multi-GPU step.
 * When several processes each run the convolution on their own batch elements
 * with replicated weights, their weight and bias gradients must be summed; this
 * call is the arithmetic of that exchange, done in a fixed order so that every
 * process ends with the same bits run after run.  Moving the gradients between
 * processes (an all-gather) is the caller's.
 * ====================================================================================== */

/* out[i] = round(parts[0][i] + parts[1][i] + ... + parts[nparts-1][i]) with the
 * additions done in fp32 in index order (left to right) and one round-to-nearest-
 * even to `dtype` at the end.  parts: [nparts][count] contiguous, out: [count],
 * both of `dtype` and aligned to its size; out may not overlap parts.
 * Asynchronous on `stream`; VG_ERR_INVALID_ARG for nparts <= 0, count < 0, an
 * unknown dtype, or null/misaligned pointers. */
VG_API int vg_sum_ordered(const void* parts, int nparts, int64_t count, int dtype, void* out, void* stream);

/* ======================================================================================
 * Forward pass without a caller-provided workspace.
 * The paper has no counterpart to this call.  It is for callers that cannot
 * allocate device memory: plug-ins hosted by a runtime that owns all device memory
 * and forbids allocation after start-up, and hot paths that cannot afford the
 * device-wide synchronisation of cudaMalloc/cudaFree.
 * Arguments and output are those of vg_subm_conv3d_fwd without conv_ws: the scratch
 * (repacked weight tiles and the error word) is a fixed __device__ array of
 * 8 MiB + 256 B inside the library, which every GPU that loads the library holds
 * until the process exits.  The call runs the same kernels as vg_subm_conv3d_fwd
 * with VG_NO_SMALL_N_SPLIT (it has no room for split partial sums), so the
 * output is bit-identical to that call's.  A kernel that gives up a bounded wait
 * is reported by vg_subm_conv3d_fwd_noalloc_status(), not by this call's
 * return value (which covers argument and launch errors only).
 *  - Returns VG_ERR_WORKSPACE_TOO_SMALL when the repacked weights (27*Cin*Cout*2
 *    bytes on the tensor-core path: 16-bit dtype, Cin and Cout multiples of 64)
 *    exceed 8 MiB, e.g. Cin = Cout = 512.
 *  - Allocates nothing.  The first call on each device looks up the array's device
 *    address (cudaGetSymbolAddress) and keeps it once the lookup succeeds.
 *  - Every call uses the same array, which keeps the previous call's contents: calls
 *    that can overlap on the GPU (other streams, other host threads) race on it and
 *    must be serialised by the caller.
 * ====================================================================================== */
VG_API int vg_subm_conv3d_fwd_noalloc(const void* nbr_ws, const uint32_t* nbr, const uint32_t* mask,
                                      int64_t N, int dtype, const void* feats, const void* weight,
                                      const void* bias, void* out, int Cin, int Cout, unsigned flags,
                                      void* stream);

/* Device-side status of the most recent vg_subm_conv3d_fwd_noalloc call on the
 * current device.  The paper has no counterpart to this call either: it reads
 * the error word that the no-allocation forward keeps in its fixed array, so a
 * caller without a conv workspace can still learn that a kernel gave up a
 * bounded wait.  Synchronises `stream` (the stream of that call), then reads and
 * clears the word.  Returns VG_ERR_DEVICE_TIMEOUT if a kernel of that call gave
 * up (its output is then incomplete), VG_OK otherwise, VG_ERR_CUDA if the array's
 * address cannot be looked up or the copy fails.  Allocates nothing. */
VG_API int vg_subm_conv3d_fwd_noalloc_status(void* stream);

/* ======================================================================================
 * Attention-block operators
 * The pages stop at the convolution; the models that use it put blocks between the
 * convolutions in which the voxel tokens attend to an encoder's states (an image's or a
 * text's), and train both.  The calls below are that block's own arithmetic: the norm and
 * rotation of queries and keys, the attention, and the optimizer step.
 * ====================================================================================== */

/* Rows of heads: element (row, head, i) of a [rows][heads][head_dim] tensor lies at
 * data + row * row_stride + head * head_stride + i (strides in elements).  Tokens may
 * come first (row_stride = heads * head_dim or more, as in a packed projection) or heads
 * (head_stride = rows * row_stride).  data is 16-byte aligned and both strides are
 * multiples of 16 bytes and at least head_dim; the elements of an output do not overlap. */
typedef struct {
    void* data;
    int64_t row_stride, head_stride;
} vg_heads;

/* --------------------------------------------------------------------------------------
 * Norm of queries and keys for each head and rotary positions with up to three axes, in one
 * pass (neither q nor k is read twice; either may be absent, with 0 heads).
 *   n = x / sqrt(mean_i x_i^2 + eps) * weight            (skipped with VG_QK_NO_NORM)
 *   pair p of axis a turns by t = (float)coords[row][1 + a] * freqs[p]:
 *   (y0, y1) = (n0 cos t - n1 sin t, n0 sin t + n1 cos t)
 * Axis a owns axis_pairs[a] consecutive pairs, axis 0 first; pairs beyond their sum are not
 * turned.  Pair p is elements (2p, 2p + 1), or (p, p + head_dim/2) with VG_ROPE_HALVES.
 * coords is the neighbour map's [N][4] int32 (b, x, y, z), or (b, time, height, width) of
 * another encoder's tokens; column 0 is not used.  coords and freqs NULL: norm alone.
 * Weights are [heads][head_dim] ([head_dim] with VG_QK_SHARED_WEIGHT), of `dtype`, 16-byte
 * aligned; NULL: ones.  head_dim is a multiple of 8, at most 256; 0 < heads <= 4096 in all.
 * Sums and angles are fp32; outputs are rounded once.  The forward may run in place
 * (an output with its input's data and strides).
 * -------------------------------------------------------------------------------------- */
#define VG_ROPE_HALVES      0x200u
#define VG_QK_NO_NORM       0x400u
#define VG_QK_SHARED_WEIGHT 0x800u

VG_API int vg_qk_norm_rope_fwd(int64_t N, int heads_q, int heads_k, int head_dim, int dtype, const vg_heads* q,
                               const vg_heads* k, const void* q_weight, const void* k_weight,
                               const int32_t* coords, const float* freqs, const int axis_pairs[3], double eps,
                               unsigned flags, const vg_heads* q_out, const vg_heads* k_out, void* stream);
/* Bytes of workspace of the backward pass (0 if the arguments are invalid). */
VG_API size_t vg_qk_norm_rope_workspace_bytes(int64_t N, int heads_q, int heads_k, int head_dim);
/* Gradients of the forward's inputs q, k (the unnormed ones; not read with VG_QK_NO_NORM)
 * and of its weights, summed over the rows (and over the heads that share a weight) in a
 * fixed order.  grad_q_weight / grad_k_weight NULL: not wanted.  ws: 256-byte aligned,
 * needed when a weight gradient is wanted. */
VG_API int vg_qk_norm_rope_bwd(int64_t N, int heads_q, int heads_k, int head_dim, int dtype, const vg_heads* q,
                               const vg_heads* k, const void* q_weight, const void* k_weight,
                               const int32_t* coords, const float* freqs, const int axis_pairs[3], double eps,
                               unsigned flags, const vg_heads* grad_q_out, const vg_heads* grad_k_out,
                               const vg_heads* grad_q, const vg_heads* grad_k, void* grad_q_weight,
                               void* grad_k_weight, void* ws, size_t ws_bytes, void* stream);

/* --------------------------------------------------------------------------------------
 * Cross attention: the tokens of each sample attend to that sample's encoder states.
 *   out = softmax(scale q k^T) v over the sample's valid keys; lse = log sum exp(scale q k^T).
 * Sample b has the query rows [q_offsets[b], q_offsets[b+1]) and the key rows
 * [k_offsets[b], k_offsets[b+1]), of which the first k_lens[b] are valid (k_lens NULL: all).
 * Rows past the valid ones are never used, whatever they hold; their gradients are zero.  A
 * sample without valid keys gives out = 0 and lse = -inf, and takes no part in any gradient.
 * heads_q is a multiple of heads_k: query head h reads key head h / (heads_q / heads_k), and
 * the gradient of a key head is the sum over its query heads.
 *   dtype VG_F16 / VG_BF16: tensor cores, fp32 softmax and sums, the scores' weights (and
 *   their gradients) rounded to dtype before the second product.  In fp16 those gradients have a
 *   scale of their own for each query in grad_q, and for each sample in grad_k.
 *   VG_F32: fp32 multiply-adds throughout.
 *   head_dim is a multiple of 8, at most 128; scale > 0 and finite; lse is [heads_q][n_q].
 * With few query rows the keys are cut into parts that run side by side, with few keys the
 * queries (backward); parts are joined in a fixed order, so every result is the same from
 * run to run.
 * -------------------------------------------------------------------------------------- */
typedef struct {
    int64_t n_q, n_k;            /* rows of q, of k and v: q_offsets[batch], k_offsets[batch]  */
    int batch, heads_q, heads_k, head_dim, dtype;
    float scale;
    const int32_t* q_offsets;    /* [batch + 1], device                                       */
    const int32_t* k_offsets;    /* [batch + 1], device                                       */
    const int32_t* k_lens;       /* [batch], device, or NULL                                   */
} vg_attn;

/* Bytes of workspace (0 if the arguments are invalid; the offset pointers are not looked
 * at).  backward: 1 for a workspace that vg_cross_attn_bwd takes too. */
VG_API size_t vg_cross_attn_workspace_bytes(const vg_attn* a, int backward);
/* ws: 256-byte aligned; its first 4 bytes, the error record, are zero before the first
 * call.  lse may be NULL.  Asynchronous.  Offsets or lengths that are no partition of the
 * rows are found on the device: nothing is written and vg_cross_attn_status says so. */
VG_API int vg_cross_attn_fwd(const vg_attn* a, const vg_heads* q, const vg_heads* k, const vg_heads* v,
                             const vg_heads* out, float* lse, void* ws, size_t ws_bytes, void* stream);
/* out and lse are the forward's. */
VG_API int vg_cross_attn_bwd(const vg_attn* a, const vg_heads* q, const vg_heads* k, const vg_heads* v,
                             const vg_heads* out, const float* lse, const vg_heads* grad_out, const vg_heads* grad_q,
                             const vg_heads* grad_k, const vg_heads* grad_v, void* ws, size_t ws_bytes,
                             void* stream);
/* Synchronises `stream`; VG_ERR_INVALID_ARG if a call on ws found bad offsets,
 * VG_ERR_DEVICE_TIMEOUT if a bounded device-side wait gave up, else VG_OK.  Clears the record. */
VG_API int vg_cross_attn_status(void* ws, void* stream);

/* --------------------------------------------------------------------------------------
 * AdamW step over many tensors at once.
 *   g = grad * grad_scale
 *   m = m * beta1 + g * c1,  v = v * beta2 + (g * g) * c2
 *   p = p * decay - (m / (sqrt(v) * root + eps)) * rate
 * p is master where given (param, which is then not read, gets p rounded to its dtype), else
 * param.  c1 = 1 - beta1, c2 = 1 - beta2, decay = 1 - lr weight_decay, root = 1 / sqrt(1 - beta2^step)
 * and rate = lr / (1 - beta1^step) are computed in 64 bits and rounded once to fp32, as are
 * beta1, beta2, eps and grad_scale; every operation above is one fp32 rounding, in the order written.
 * state_bits 32: m and v are fp32 [n].  state_bits 8: m and v are codes, uint8 [n], with
 * one fp32 scale for every VG_ADAMW_BLOCK elements in m_scale and v_scale [ceil(n/256)];
 * codes 0 with any scale are zero states.  Scales are powers of two.  A code c stands for
 *   m: (c & 128 ? -1 : 1) * x * scale, a = c & 127: x = a / 512 below 8, else
 *      (1 + (a & 7)/8) 2^((a >> 3) - 7); 127 is NaN;
 *   v: (x * scale)^2, x = 0 at c = 0, else (1 + ((c - 1) & 15)/16) 2^((c - 1) >> 4); 255 is NaN.
 * New states take the nearest value (ties to even mantissas; a positive v never becomes
 * zero); a state that is not finite is held as NaN.  The step itself uses the moments
 * before they are rounded.
 * -------------------------------------------------------------------------------------- */
#define VG_ADAMW_BLOCK 256

typedef struct {
    void* param;            /* [n] of dtype, updated                                   */
    const void* grad;       /* [n] of dtype                                            */
    float* master;          /* [n] or NULL, updated                                    */
    void* m;                /* [n] fp32 or codes, updated                              */
    void* v;
    float* m_scale;         /* [ceil(n / 256)], 8-bit states only, updated             */
    float* v_scale;
    int64_t n;
    double weight_decay;
    int dtype;
} vg_adamw_tensor;

/* tensors: HOST array of `count` (read before the call returns; the pointers in it are
 * device pointers).  step counts from 1.  Asynchronous; one launch for up to 384 tensors.
 * Pointers aligned to 16 bytes (codes: 8) take the wide path, others are served element by
 * element. */
VG_API int vg_adamw_step(const vg_adamw_tensor* tensors, int count, int state_bits, int64_t step, double lr,
                         double beta1, double beta2, double eps, double grad_scale, void* stream);
/* out[i] = the value that 8-bit state code i stands for; second: 0 for m, 1 for v. */
VG_API int vg_adamw_decode(const uint8_t* codes, const float* scales, int64_t n, int second, float* out,
                           void* stream);

/* ======================================================================================
 * Recurrent-block operators
 * The other block that networks put between the convolutions mixes the voxel tokens along a
 * space-filling curve (the order of vg_encode_seq's codes): s + dropout(scan(project(norm(s)))),
 * with the residual stream s.  The calls below are its norm, its recurrence and its dropout.
 * ====================================================================================== */

/* Rows of channels: element (row, c) lies at data + row * row_stride + c (stride in elements, a
 * multiple of 16 bytes, at least the channel count and below 2^30; data 16-byte aligned).  Channel counts
 * are multiples of 8.  An output may take the place of an input of its own type (the same data
 * and stride); otherwise it overlaps no other operand. */
typedef struct {
    void* data;
    int64_t row_stride;
} vg_rows;

/* --------------------------------------------------------------------------------------
 * Layer norm of each row.
 *   z = (x - mean) * rstd,  y = z * weight + bias,  rstd = 1 / sqrt(mean((x - mean)^2) + eps)
 * weight and bias are [C] of `dtype`, 16-byte aligned; NULL: ones, zeros.  stats [N][2] fp32 is
 * (mean, rstd), 8-byte aligned; the forward's may be NULL.  C is a multiple of 8, at most 8192.
 * Statistics and sums are fp32 (squares of the differences from the mean); outputs are rounded
 * once.  Backward, with g = grad_y * weight:
 *   grad_x = (g - mean(g) - z * mean(g z)) * rstd  (+ grad_skip, if that is not NULL: the
 *            gradient that reaches x past the norm, as in a residual stream)
 *   grad_weight = sum over rows of grad_y z,  grad_bias = sum of grad_y, in a fixed order.
 * grad_weight and grad_bias may be NULL (not wanted); ws, 256-byte aligned, is needed unless both are.
 * -------------------------------------------------------------------------------------- */
VG_API int vg_layer_norm_fwd(int64_t N, int C, int dtype, const vg_rows* x, const void* weight, const void* bias,
                             double eps, const vg_rows* y, float* stats, void* stream);
/* Bytes of workspace of the backward pass (0 if the arguments are invalid). */
VG_API size_t vg_layer_norm_workspace_bytes(int64_t N, int C);
VG_API int vg_layer_norm_bwd(int64_t N, int C, int dtype, const vg_rows* x, const void* weight, const float* stats,
                             const vg_rows* grad_y, const vg_rows* grad_skip, const vg_rows* grad_x,
                             void* grad_weight, void* grad_bias, void* ws, size_t ws_bytes, void* stream);

/* --------------------------------------------------------------------------------------
 * Gated linear recurrence of each channel along each sequence.
 *   a_t = sigmoid(gate_t),  h_t = a_t h_{t-1} + (1 - a_t) x_t,  out_t = h_t
 * With VG_SCAN_FREE_INPUT, h_t = a_t h_{t-1} + x_t.  Sequence b visits the positions
 * [offsets[b], offsets[b+1]) upwards, or downwards with VG_SCAN_REVERSE; position p is row
 * order[p] of gate, x and out (order NULL: row p), where order is a permutation of the rows
 * (for instance the order of their codes along a curve).  h_{-1} is first[b] (NULL: zeros);
 * last[b] (NULL: not wanted) receives the state after the last token, first[b] itself where
 * there are no tokens.  first and last are fp32 [batch][C], 16-byte aligned, and do not overlap.
 * States and sums are fp32; outputs are rounded once.  A token that is not finite makes its
 * channel's states up to the end of its sequence infinite or NaN, and touches nothing else.
 * The positions are cut into parts that run side by side; they are joined in a fixed order, so every
 * result is the same from run to run.
 * Backward: lam_t = grad_out_t + a_{t+1} lam_{t+1}, with grad_last[b] in place of the last term at
 * the last token;
 *   grad_x = (1 - a) lam (VG_SCAN_FREE_INPUT: lam),  grad_first = a_0 lam_0,
 *   grad_gate = a (1 - a) (h_{t-1} - x) lam (VG_SCAN_FREE_INPUT: a (1 - a) h_{t-1} lam).
 * -------------------------------------------------------------------------------------- */
#define VG_SCAN_REVERSE    0x1000u
#define VG_SCAN_FREE_INPUT 0x2000u

typedef struct {
    int64_t n;                   /* rows: offsets[batch]                                       */
    int channels, batch, dtype;
    unsigned flags;
    const int32_t* offsets;      /* [batch + 1], device                                        */
    const int32_t* order;        /* [n], device, or NULL                                       */
} vg_scan;

/* Bytes of workspace of vg_gated_scan_fwd and _bwd (0 if the arguments are invalid; the pointers, flags
 * and batch make no difference).  No less for more rows of as many channels: a workspace for the most rows
 * serves calls of fewer.  Calls that may overlap on the GPU need a workspace each. */
VG_API size_t vg_gated_scan_workspace_bytes(const vg_scan* s);
/* Rows of `carries` (fp32 [rows][C], 16-byte aligned), the states that the forward pass keeps for
 * the backward pass: one for every 16 positions. */
VG_API int64_t vg_gated_scan_carry_rows(int64_t n);
/* ws: 256-byte aligned; its first 4 bytes, the error record, are zero before the first call.
 * carries may be NULL (no backward pass will follow).  Asynchronous.  Offsets that are no partition of the
 * positions are found on the device: nothing is written and vg_gated_scan_status says so.  An
 * entry of order that is no row is reported the same way: nothing is read or written for its
 * token, and its sequence's results are undefined. */
VG_API int vg_gated_scan_fwd(const vg_scan* s, const vg_rows* gate, const vg_rows* x, const float* first,
                             const vg_rows* out, float* last, float* carries, void* ws, size_t ws_bytes,
                             void* stream);
/* carries is the forward's; grad_last and grad_first [batch][C] fp32 may be NULL. */
VG_API int vg_gated_scan_bwd(const vg_scan* s, const vg_rows* gate, const vg_rows* x, const float* first,
                             const float* carries, const vg_rows* grad_out, const float* grad_last,
                             const vg_rows* grad_gate, const vg_rows* grad_x, float* grad_first, void* ws,
                             size_t ws_bytes, void* stream);
/* One token of each of n sequences: state [n][C] (fp32, 16-byte aligned) is h_{t-1} before and h_t
 * after the call; flags: 0 or VG_SCAN_FREE_INPUT. */
VG_API int vg_gated_scan_step(int64_t n, int C, int dtype, unsigned flags, const vg_rows* gate, const vg_rows* x,
                              float* state, const vg_rows* out, void* stream);
/* Synchronises `stream`; VG_ERR_INVALID_ARG if a call on ws found bad offsets or a bad order, else
 * VG_OK.  Clears the record. */
VG_API int vg_gated_scan_status(void* ws, void* stream);

/* --------------------------------------------------------------------------------------
 * Dropout into the residual stream; the mask is computed where it is needed and never stored.
 *   out[i] = residual[i] + (keep_i ? x[i] / (1 - p) : 0);  backward: grad_x[i] = keep_i ? grad_out[i] / (1 - p) : 0
 *   (residual's gradient is grad_out itself)
 * keep_i is w_i >= round(p 2^32), where w_i is word i mod 4 of Philox 4x32 with ten rounds (J. K.
 * Salmon, M. A. Moraes, R. O. Dror, D. E. Shaw, "Parallel random numbers: as easy as 1, 2, 3",
 * SC 2011) at key (low, high word of rng[0]) and counter (low, high word of i / 4, low word of
 * rng[1], call).  rng is on the DEVICE: rng[0] is the seed, rng[1] the step, which a captured
 * graph can count up itself; `call` tells apart the calls of one step.  The mask depends on
 * nothing else, so the backward pass takes the same three.  0 <= p <= 1 - 2^-32.  x, residual
 * (or NULL) and out are n contiguous elements; out may be x or residual itself.  Pointers aligned
 * to 16 bytes take the wide path, others are served element by element.
 * -------------------------------------------------------------------------------------- */
VG_API int vg_dropout_add_fwd(int64_t n, int dtype, const void* x, const void* residual, double p,
                              const uint64_t* rng, uint32_t call, void* out, void* stream);
VG_API int vg_dropout_add_bwd(int64_t n, int dtype, const void* grad_out, double p, const uint64_t* rng,
                              uint32_t call, void* grad_x, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* VOXEL_GEMM_VG_H */
