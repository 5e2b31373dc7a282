// Kernel parameter blocks and launchers shared by the C-ABI layer and the
// kernel translation units of libvce.  Not part of the public interface.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace vce {

struct CeFwdParams {
  const void* logits;
  int64_t d1, ls0, ls1, V;
  const int64_t* targets;
  int64_t ts0, ts1;
  float eps;
  int64_t ignore_idx;
  float* loss_tok;
  float* stats;
  float* entropy;  // optional (N)
  int64_t v0;      // first vocabulary column of the row (0 unless sharded)
  float* partial;  // shard mode: (N, 4) partial statistics instead of loss/stats
  float* partial_w;  // shard mode, optional: (N) entropy statistic w of the shard
};

struct CeMergeParams {
  const float* partials;    // (n_shards, N, 4)
  const float* partials_w;  // with entropy: (n_shards, N)
  int64_t n_shards, N, d1;
  const int64_t* targets;
  int64_t ts0, ts1, V, ignore_idx;  // V: the full vocabulary
  float eps;
  float* loss_tok;
  float* stats;
  float* entropy;  // optional (N), needs partials_w
};

struct CeMeanParams {
  const float* loss_tok;
  const int64_t* targets;
  int64_t N, d1, ts0, ts1, ignore_idx;
  float* loss_mean;
  int32_t* n_valid;
};

struct CeBwdParams {
  const void* logits;
  void* grad;
  int64_t d1, ls0, ls1, V;
  const int64_t* targets;
  int64_t ts0, ts1;
  const float* stats;
  const int32_t* n_valid;
  const float* grad_output;
  const float* entropy;       // with grad_entropy: the forward's entropy (N)
  const float* grad_entropy;  // optional (N): adds grad_entropy[r] dH/dz
  float eps;
  int reduce_loss;
  int64_t ignore_idx;
  int64_t v0, Vg;  // the row holds columns v0 .. v0 + V - 1 of Vg (0, V unless sharded)
  int splits = 1;  // workgroups per row (set by the launcher)
};

hipError_t launch_ce_forward(const CeFwdParams& p, int dtype, int64_t N, hipStream_t stream);
hipError_t launch_ce_mean(const CeMeanParams& p, hipStream_t stream);
hipError_t launch_ce_merge_shards(const CeMergeParams& p, hipStream_t stream);

struct ShiftParams {
  const int64_t* targets;
  int64_t d0, d1, ts0, ts1, N, ignore_idx;
  int seq_axis;
  int64_t* out;
};
hipError_t launch_shift_targets(const ShiftParams& p, hipStream_t stream);
hipError_t launch_ce_backward(const CeBwdParams& p, int dtype, int64_t N, hipStream_t stream);
// One-pass forward + backward (rows of at most 512 x 32 16-byte vectors: see ce_fb_fits).
bool ce_fb_fits(int dtype, int64_t V);
hipError_t launch_ce_forward_backward(const CeFwdParams& f, const CeBwdParams& b, int dtype,
                                      int64_t N, hipStream_t stream);

// ---- fused linear cross-entropy ----------------------------------------------

// Workspace plan of the linear form for an (M, H, V) problem.
struct LcePlan {
  int64_t M, H, V;
  int64_t Mp;          // M rounded up to the token tile
  int64_t n_vtiles;    // vocabulary tiles of the forward
  int64_t chunk;       // vocabulary rows per backward chunk (multiple of the tile)
  int64_t n_chunks;
  int64_t ldz;         // row stride (elements) of the dZ chunk buffer
  size_t off_part;     // forward: per-tile partials and target logits
  size_t off_dz, off_dx;  // backward: dZ of one chunk, FP32 dX accumulator
  size_t off_dz2;         // second dZ buffer (BF16 form, several chunks), else off_dz
  size_t fwd_bytes;       // what the forward alone uses (from offset 0)
  size_t total;
  // FP32 inputs: X and W split into BF16 hi and lo planes in the workspace
  // (lo plane right after its hi plane), dZ in two planes, no accumulator
  // (dX is FP32 and accumulates in place)
  bool f32;
  size_t off_xs, off_ws;  // hi planes of X and W
  size_t xplane, wplane;  // bytes per plane
  int64_t dzplane;        // elements from the hi plane of dZ to its lo plane
};

bool lce_make_plan(int64_t M, int64_t H, int64_t V, LcePlan* plan, bool f32 = false);

struct LceFwdArgs {
  const void* X;
  const void* W;
  const int64_t* targets;
  float eps;
  int reduce_loss;
  int64_t ignore_idx;
  float* loss_tok;
  float* loss_mean;
  float* stats;
  int32_t* n_valid;
  float* entropy;  // optional (M)
  char* ws;
  int64_t v0;      // vocabulary index of W's first row (0 unless sharded)
  float* partial;  // shard mode: (M, 4) local statistics instead of loss/stats
  float* partial_w;  // shard mode, optional: (M) entropy statistic w of the shard
  float scale = 1.0f;  // logits = scale X W^T (scale > 0)
};

struct LceBwdArgs {
  const void* X;
  const void* W;
  const int64_t* targets;
  const float* stats;
  const int32_t* n_valid;
  const float* grad_output;
  const float* entropy;       // with grad_entropy: the forward's entropy (M)
  const float* grad_entropy;  // optional (M)
  float eps;
  int reduce_loss;
  int64_t ignore_idx;
  void* dX;
  void* dW;
  char* ws;
  int64_t v0, Vg;  // W holds vocabulary rows v0 .. v0 + V - 1 of Vg (0, V unless sharded)
  float scale = 1.0f;  // logits = scale X W^T (scale > 0)
};

hipError_t launch_lce_forward(const LcePlan& plan, const LceFwdArgs& a, hipStream_t stream);
hipError_t launch_lce_backward(const LcePlan& plan, const LceBwdArgs& a, hipStream_t stream);
hipError_t launch_gemm_bf16(const void* P, int64_t ldp, int p_dim, const void* Q, int64_t ldq,
                            int q_dim, int64_t rows, int64_t cols, int64_t K, float* C,
                            int64_t ldc, hipStream_t stream);

// A grid of n workgroups in two dimensions: one dimension holds fewer than 2^32
// threads.  Workgroup blockIdx.y * gridDim.x + blockIdx.x; those at or past n
// have nothing to do.
inline dim3 grid2(int64_t n) {
  const int64_t x = n < ((int64_t)1 << 21) ? n : ((int64_t)1 << 21);
  return dim3((unsigned)x, (unsigned)((n + x - 1) / x));
}

// ---- residual + RMS norm -------------------------------------------------------

struct RmsFwdParams {
  const void* x;
  const void* residual;  // optional
  int64_t M, ldx, ldr;
  int H;
  const void* weight;
  int wdtype;
  float w0, eps;
  void* y;          // (M, H), the norm's output (not with q)
  uint8_t* q;       // (M, H) E4M3 and (M, H / 32) scale bytes instead of y
  uint8_t* scales;
  void* h;          // optional (M, H): x + residual
  float* rstd;      // optional (M)
};

struct RmsBwdParams {
  const void* dy;
  const void* h;
  int64_t M;
  int H;
  const void* weight;
  int wdtype;
  float w0;
  const float* rstd;
  const void* dh;  // optional (M, H)
  void* dx;
  // up to rms_bwd_parts(M) shares of dw, rms_share_width(H) apart; NULL without dweight
  float* partial;
  float* dweight;  // optional (H)
};

bool rms_width_ok(int64_t H);
int rms_bwd_parts(int64_t M);  // at most
// A share of dw starts on a cache line, whatever H is.
__host__ __device__ inline int64_t rms_share_width(int64_t H) { return (H + 31) / 32 * 32; }
hipError_t launch_rms_forward(const RmsFwdParams& p, int dtype, bool mx, hipStream_t stream);
hipError_t launch_rms_backward(RmsBwdParams p, int dtype, hipStream_t stream);

// ---- microscaled formats -------------------------------------------------------

struct MxQuantParams {
  const void* x;
  int64_t rows, K, ldx;
  uint8_t* q;
  uint8_t* scales;
  bool small = false;  // thread index fits 31 bits (set by the launcher)
};

struct MxDequantParams {
  const uint8_t* q;
  const uint8_t* scales;
  void* out;
  int64_t n8 = 0;  // groups of 8 values (set by the launcher)
};

hipError_t launch_mx_quantize(const MxQuantParams& p, int dtype, int fmt, hipStream_t stream);
hipError_t launch_mx_dequantize(MxDequantParams p, int64_t n, int fmt, int dtype,
                                hipStream_t stream);

struct MxGemmParams {
  const uint8_t *x, *xs, *w, *ws;  // values and scales of X (M, K) and W (V, K)
  int64_t M, K, V;
  float scale;
  void* out;    // (M, V), row i at element i * ldo
  int64_t ldo;
  bool wide = false;  // four logits may be stored at once (set by the launcher)
};

bool mx_logits_size_ok(int64_t M, int64_t V);
hipError_t launch_mx_logits(MxGemmParams p, int x_format, int w_format, int dtype,
                            hipStream_t stream);

// ---- drawing a token -----------------------------------------------------------

// A row that sample_pick_kernel has left to the kernels after it: the bin of
// distances lo .. hi that holds its threshold, the weight before the bin, the
// row's weight, and the number of the bin's tokens listed so far.
struct SampleState {
  uint32_t what;
  float lo, hi;
  uint32_t n;
  unsigned long long above, mass;
};

struct SampleParams {
  const void* logits;
  int64_t d1, ls0, ls1, V;
  const float* temperature;  // each optional (N) except u
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  const float* u;
  int64_t* token;
  float* logprob;  // optional (N)
  // set by the launcher: the weights' fixed point and polynomial, and the
  // workspace's parts
  enum { kT = 1, kK = 2, kP = 4, kM = 8 };
  int has = 0;  // which of the optional parameters are given
  double magic = 0.0, unit = 0.0, inv_v = 0.0;
  double poly[9] = {};
  uint32_t rows = 0;
  int segs = 0;                             // segments per row
  float* group_max = nullptr;               // (N, segs, 256)
  float* seg_max = nullptr;                 // (N, segs)
  // the others only for rows that LDS does not hold whole
  unsigned long long* seg_sum = nullptr;    // (N, segs)
  unsigned long long* hist = nullptr;       // (N, 2048)
  SampleState* state = nullptr;             // (N), NULL where every row is done in one kernel
  uint32_t* done = nullptr;                 // (N, 2): workgroups of the row past each kernel
};

// Rows times segments stay below 2^31.
bool sample_size_ok(int64_t N, int64_t V);
size_t sample_workspace_bytes(int64_t N, int64_t V);
hipError_t launch_sample(SampleParams p, int dtype, int64_t N, void* workspace,
                         hipStream_t stream);

}  // namespace vce
