// Internal launcher interface between the C-ABI layer (api.cpp) and the
// kernel translation units.  Not part of the public ABI.
#pragma once

#include <cuda.h>  // CUtensorMap (type only)
#include <cuda_runtime.h>
#include <stdint.h>
#include <stddef.h>
#include <algorithm>
#include <atomic>

namespace fp8lin {

// Host-side launch counter (defined in api.cpp).
void count_launch();

// Brackets one kernel launch with CUDA events on its stream while kernel
// timing is enabled (fp8_profile_begin/end); also counts the launch.
// bytes/flops: the launch's algorithmic HBM traffic and floating-point work;
// m, n, k: its problem shape (GEMM M, N, K; quantizer rows, columns; glue
// element count), which keeps launches of one kernel on different shapes
// apart in the timing records.
class LaunchScope {
 public:
  LaunchScope(const char *name, cudaStream_t st, double bytes, double flops, int64_t m = 0,
              int64_t n = 0, int64_t k = 0);
  ~LaunchScope();

 private:
  int rec_ = -1;
  cudaStream_t st_;
};

// Tensorwise quantization keeps one fp32 partial amax per CTA of its first
// pass in the caller's workspace; at most this many.
constexpr int kMaxPartials = 1024;

int num_sms();

// Kernel launches allow programmatic dependent launch (the kernel may be
// scheduled while the previous kernel on the stream drains; each kernel waits
// for it in pdl_wait or pdl_wait_then_release before touching global memory,
// see common.cuh) unless the
// environment sets FP8LIN_PDL=0 when the library first launches.
bool pdl_enabled();

// Blocks of `kernel` (threads per block, no dynamic shared memory) that fit on
// one SM of the current device, cached per device in per_dev[64].  Grids of
// grid-stride kernels are sized to this many blocks per SM: under overlapped
// launch the blocks are placed on SMs in the order the previous kernel frees
// them, and a smaller grid would crowd onto the first SMs freed.
template <typename Kernel>
int blocks_per_sm(Kernel kernel, int threads, std::atomic<int> *per_dev) {
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64) return 1;
  if (per_dev[dev] == 0) {
    int n = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, 0) != cudaSuccess || n < 1)
      n = 1;
    per_dev[dev] = n;
  }
  return per_dev[dev];
}

// overlap = false: a plain launch (the kernel starts once the previous one on
// the stream has completed).
template <typename... KArgs, typename... Args>
cudaError_t launch_kernel_as(bool overlap, void (*kernel)(KArgs...), dim3 grid, dim3 block,
                             size_t smem, cudaStream_t st, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = overlap && pdl_enabled() ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}
template <typename... KArgs, typename... Args>
cudaError_t launch_kernel(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                          cudaStream_t st, Args... args) {
  return launch_kernel_as(true, kernel, grid, block, smem, st, args...);
}
int tensorwise_partials_count(int64_t rows, int64_t cols);

// mode: 0 tensorwise, 1 1x128 blocks, 2 128x128 tiles; fmt: fp8_format.
// Tensorwise with amax_done: the first pass already wrote `partials`
// (launch_amax_partials on the same tensor); only the cast runs.  rows need
// not be a multiple of 16 here: out_col then has rows of rows rounded up to
// 16 bytes, filled up with zeros.
cudaError_t launch_quantize(const void *x, int64_t rows, int64_t cols, int mode, int fmt,
                            uint8_t *out_row, uint8_t *out_col, float *row_scale,
                            float *row_scale_inv, float *col_scale, float *col_scale_inv,
                            float *partials, cudaStream_t st, bool amax_done = false);
// Tensorwise first pass alone: tensorwise_partials_count(rows, cols) partial maxima.
cudaError_t launch_amax_partials(const void *x, int64_t rows, int64_t cols, float *partials,
                                 cudaStream_t st);

// Delayed scaling: cast with the scale of the history's maximum, then write
// this tensor's amax to hist[step % hist_len] (partials: >= 2 x SMs floats).
cudaError_t launch_quantize_delayed(const void *x, int64_t rows, int64_t cols, int fmt,
                                    uint8_t *out_row, uint8_t *out_col, float *scale,
                                    float *scale_inv, float *hist, int hist_len, int64_t step,
                                    float *partials, cudaStream_t st);

// Fused GELU (bwd = 0: A = GELU(H), E4M3) or GELU backward (bwd = 1:
// dH = H * GELU'(H2) with H = dA, E5M2) with the 1x128 quantizer.
cudaError_t launch_gelu_quantize(const void *H, const void *H2, int64_t rows, int64_t cols,
                                 int bwd, uint8_t *out_row, uint8_t *out_col, float *row_scale,
                                 float *row_scale_inv, float *col_scale, float *col_scale_inv,
                                 cudaStream_t st);

// TMA descriptor of a bf16 [rows, cols] row-major tensor (row stride cols,
// 16-byte aligned base) for box_rows x box_cols boxes, no swizzle, zeros read
// outside the tensor.
bool make_bf16_tile_map(CUtensorMap *m, const void *base, int64_t rows, int64_t cols, int box_rows,
                        int box_cols);
// Reads and clears the quantizer kernels' device status word (0 = ok).
cudaError_t quant_read_status(unsigned *status);

// FP8 GEMM (tcgen05).  scaling: fp8_scaling.  ws may be null when
// gemm_workspace_bytes() is 0.  a_rows != 0 (tensor scaling only): A is given
// transposed, [a_rows, M] with M contiguous, and is zero from row a_rows to K.
size_t gemm_workspace_bytes(int64_t M, int64_t N, int64_t K, int scaling);
cudaError_t launch_gemm(const uint8_t *A, int a_fmt, const float *a_sinv, const uint8_t *B,
                        int b_fmt, const float *b_sinv, int64_t M, int64_t N, int64_t K,
                        int scaling, void *C, void *ws, cudaStream_t st, int64_t a_rows = 0);
// Launches the bounded-wait probe (a wait nobody satisfies; limit_ns <= 1 s).
cudaError_t launch_wait_timeout_probe(uint64_t limit_ns, cudaStream_t st);
// Reads and clears the GEMM kernels' device status word (0 = ok).
cudaError_t gemm_read_status(unsigned *status, cudaStream_t st);

// Operand and output tiles of the GEMM kernels: u8 [rows, cols] boxes of
// box_rows rows x 128 bytes, and bf16 [rows, cols] boxes of 32 rows x 64
// columns, both 128-byte swizzled.
bool make_u8_map(CUtensorMap *m, const void *base, int64_t rows, int64_t cols, int box_rows);
bool make_bf16_slab_map(CUtensorMap *m, void *base, int64_t rows, int64_t cols);

// Root-mean-square norm (norm.cu).  cols: a multiple of 16, at most
// kMaxNormCols (a row is held in the registers of one CTA).
constexpr int64_t kMaxNormCols = 16384;
cudaError_t launch_rmsnorm_rows(const void *x, const void *res, const void *w, int w_f32,
                                int64_t rows, int64_t cols, float eps, void *r, float *rstd,
                                float *rstd_lo, void *y, uint8_t *row, float *row_scale, float *row_scale_inv,
                                cudaStream_t st);
cudaError_t launch_rmsnorm_cols(const void *r, const float *rstd, const float *rstd_lo,
                                const void *w, int w_f32, int64_t rows, int64_t cols, uint8_t *col, float *col_scale,
                                float *col_scale_inv, cudaStream_t st);
// partials: norm_bwd_ctas(rows, cols) x cols floats.
int norm_bwd_ctas(int64_t rows, int64_t cols);
cudaError_t launch_rmsnorm_bwd(const void *dy, const void *dr, const void *r, const float *rstd,
                               const void *w, int w_f32, int64_t rows, int64_t cols, void *dx,
                               float *dw, float *partials, cudaStream_t st);
cudaError_t norm_read_status(unsigned *status);

// Gated feed-forward (gated.cu).  Any number of tokens N; G and U null: no
// backward pass follows.  x not null (where gated_takes_bf16): the tokens in
// bf16, xq and x_sinv unused.
cudaError_t launch_gated_fwd(const uint8_t *xq, const float *x_sinv, const uint8_t *wq,
                             const float *w_sinv, int64_t N, int64_t K, int64_t F, bool block,
                             int act, void *H, void *G, void *U, cudaStream_t st,
                             const void *x = nullptr);
bool gated_takes_bf16(int64_t N, int64_t K, int64_t F, bool block);
// Activation quantizer (E4M3) for few tokens in one launch, with the bytes and
// scales of launch_quantize; col may be null.
bool gated_quantizes_few(int64_t N, int64_t K, bool block);
cudaError_t launch_gated_quantize_few(const void *x, int64_t N, int64_t K, bool block, uint8_t *row,
                                      uint8_t *col, float *row_scale_inv, float *col_scale,
                                      float *col_scale_inv, cudaStream_t st);
// dG and dU, E5M2, as one [N, 2F] tensor; block scaling: its transpose [2F, N
// rounded up to 16] too.  Tensor scaling: no transpose (col and col_scale_inv
// unused), row_scale_inv takes the one scale, partials kMaxPartials floats.
cudaError_t launch_gated_bwd_quantize(const void *dH, const void *G, const void *U, int64_t N,
                                      int64_t F, bool block, int act, uint8_t *row, uint8_t *col,
                                      float *row_scale_inv, float *col_scale_inv, float *partials,
                                      cudaStream_t st);
cudaError_t gated_read_status(unsigned *status);

// Gradient clipping (clip.cu): one chunk of one tensor.
struct ClipChunk {
  const void *src;
  void *dst;
  int32_t n;    // elements
  int32_t f32;  // 1: fp32, 0: bf16
};
// Sets of at most 16 chunks of 2048 elements take one launch (few: the table is
// cut so).
constexpr int kClipFewChunks = 16, kClipFewElements = 2048;
int clip_ctas(int64_t chunks);  // partial sums the first pass writes
// write = false: the norm alone.
cudaError_t launch_clip(const ClipChunk *table, int64_t chunks, bool few, double in_bytes, double elements,
                        bool write, float max_norm, float *norm, float *partials, cudaStream_t st);

// Routing (route.cu): logits [T, E] bf16 or fp32, bias fp32 [E] or null; E <= kMaxExperts,
// k and groups <= 32.  per, per_magic and groups_pow2 are filled in by the launch.
constexpr int kMaxExperts = 1024, kMaxChoices = 32;
struct RouteArgs {
  const void *logits;
  const float *bias;
  int64_t T;
  int E, k, groups, kept, top;
  int f32, sigmoid, renorm, vec;
  float scale;
  int per;             // experts of a group
  unsigned per_magic;  // e * per_magic >> 20 = e / per
  int groups_pow2;
};
cudaError_t launch_route_fwd(RouteArgs a, float *weights, int *experts, cudaStream_t st);
cudaError_t launch_route_bwd(RouteArgs a, const float *dweights, const float *weights, const int *experts,
                             void *dlogits, cudaStream_t st);

// An expert with tokens: its rows in the experts' order, and the work (of one item of
// the weight's rows, in the units of list_work) of all experts before it.  Behind the
// last one an entry that has `from` alone, up to the count of lists that there might be.
struct W4List {
  int e, first, count, from;
};
// Rows in the experts' order (rows.cu).  hist: E x order_chunks(slots) ints,
// unused for one chunk.  lists: [most + 1], for products of `tile` tokens at a time.
int order_chunks(int64_t slots);
cudaError_t launch_expert_order(const int *experts, int64_t slots, int E, int align, int *counts, int *offsets,
                                int *position, int *order, int *hist, cudaStream_t st,
                                W4List *lists = nullptr, int most = 0, int tile = 0);
cudaError_t launch_rows_gather(const void *x, int64_t T, int64_t C, int k, int E, int align, const int *counts,
                               const int *offsets, const int *position, void *xs, cudaStream_t st);
cudaError_t launch_rows_combine(const void *z, const int *position, const float *weights, int64_t T, int64_t C, int k,
                                void *y, cudaStream_t st);
cudaError_t launch_rows_combine_bwd(const void *dy, const void *z, const int *position, const float *weights, int64_t T,
                                    int64_t C, int k, int E, int align, const int *counts, const int *offsets, void *dz,
                                    float *dweights, cudaStream_t st);

// 4-bit weights (w4.cu).  One weight: experts null, T tokens.  A stack: `experts`
// the slots' experts [T k], order/offsets/counts their rows in the experts'
// order (null for one token, whose slots are the rows); tokens: x has a row per
// token, else per row of that order.
struct W4Args {
  const uint8_t *codes;   // [E, rows, K / 2]
  const uint16_t *scale;  // bf16 [E, rows, ceil(K / group)]
  const uint8_t *zero;    // the same shape, or null: 8
  const void *x;
  void *out;              // gated: bf16 [P, N]; else bf16, or (out_f32) fp32 [planes, P, N]
  void *part;             // fp32 [planes, P, rows], with more than one
  const int *experts, *order, *offsets, *counts;
  const W4List *lists;     // with order: [min(E, P) + 1]
  int T, P, E, k, tokens;  // P: output rows (T, or the slots)
  int N, rows, K, group;   // N outputs; rows = 2 N when gated
  int gated, act, out_f32;
  int groups, cluster;  // filled in by the launch
  unsigned per_block;   // 2^32 / blocks
};
// How a product is cut: n-tiles of 8 tokens, parts of K, warps (256 of K each)
// and blocks to a part; planes: partial sums that are left for a second kernel (1:
// none, the parts are added within the launch).  tokens: as many as a list may be
// expected to have; lists: weights; side: blocks of tokens that read the weight side by
// side; P: output rows; joined: the caller adds the planes.
struct W4Plan {
  int nt, parts, warps, blocks, planes;
  bool wide;  // w4_wide.cu; its planes are always added after
};
// Tokens of one weight that a block takes: 8, 16 or 32.
int w4_block_tokens(int N, int K, bool gated, int64_t T);
W4Plan w4_plan(int N, int K, int group, bool gated, int tokens, int lists, int side, int64_t P, bool joined);
// Whether w4_wide.cu takes a product of so many weights (of all lists) and tokens (of a
// list in the mean).
bool w4_is_wide(int64_t weights, int K, int64_t tokens, int lists);
// The same for w4_wide.cu, and its launch: sums over the parts into a.part, x [P, K].
W4Plan w4_wide_plan(int N, int K, bool gated, int tokens, int lists, int64_t P);
cudaError_t launch_w4_wide(const W4Args &a, const W4Plan &p, int lists, cudaStream_t st);
cudaError_t w4_wide_read_status(unsigned *status);
// lists: as many experts as may have a token; one weight: blocks of 8 nt tokens.  Sums
// the planes unless out_f32.
cudaError_t launch_w4_product(W4Args a, const W4Plan &p, int lists, cudaStream_t st);
cudaError_t launch_w4_join(const float *z, const int *experts, const int *position, const float *weights, int64_t T,
                           int64_t N, int k, int E, int planes, void *y, cudaStream_t st);
cudaError_t launch_w4_quantize(const void *w, int64_t rows, int64_t K, int group, uint8_t *codes, void *scale,
                               uint8_t *zero, cudaStream_t st);

cudaError_t launch_gelu_fwd(const void *H, void *A, int64_t n, cudaStream_t st);
cudaError_t launch_gelu_bwd(const void *dA, const void *H, void *dH, int64_t n, cudaStream_t st);
cudaError_t launch_grad_accumulate(float *acc, const void *dW, int64_t n, cudaStream_t st);

}  // namespace fp8lin
