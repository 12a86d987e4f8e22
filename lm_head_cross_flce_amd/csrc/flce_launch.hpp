// Internal launch interface between the C-ABI host code and the kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace flce {

// Launch timing: while the calling thread's timing log is on (the C-ABI's
// flce_timing_start), records a HIP event on st and tags it with `kernel`,
// the kernel just launched (null: the start of an entry point's launches).
// Does nothing otherwise.
void mark_launch(hipStream_t st, const char* kernel);

// Every kernel launch of the library: the launch, then its timing mark.
#define FLCE_LAUNCH(kernel, grid, block, shmem, stream, ...)                 \
  do {                                                                      \
    hipLaunchKernelGGL(kernel, grid, block, shmem, stream, __VA_ARGS__);    \
    ::flce::mark_launch(stream, #kernel);                                   \
  } while (0)

enum Reduction { kNone = 0, kSum = 1, kMean = 2 };
enum DxMode { kDxFirst = 0, kDxAccum = 1, kDxLast = 2, kDxOnly = 3 };

struct FwdLaunch {
  const void* x; const void* W; const void* b; const int64_t* targets;
  int N, H, V;            // V: rows of W (a shard's rows for the shard forward)
  int NT, P, VT;          // token tiles, vocabulary phases, vocabulary tiles
  int64_t vocab_start;    // global index of W's row 0; targets are global indices
  int64_t ignore_index;
  float eps, eps_over_v, s;
  float logit_scale;      // logits are logit_scale * (x W^T + b)
  int reduction;
  void* partials;         // float4 [P][N]
  float* rowloss;         // [N]
  float* loss;            // [1] or [N]
  float* lse;             // [N]
  int64_t* n_valid;       // [1]
  float* stats;           // shard forward: float4 [N] {m, d, sum z, z_y} over the shard's rows
  float* zloss;           // optional: the z-loss term alone, [1] or [N] like loss; null if not wanted
  float* rowzl;           // [N] per-row z-loss terms (workspace), used when zloss is set
  // Fused schedule, chunk forward only: every logit of the chunk is kept as
  // e = exp(z - m_h) in the input dtype, m_h the max over the token's 128
  // rows of the tile that one wave holds.
  void* ebuf;             // [N][lde]
  int64_t lde;            // row stride of ebuf in elements (VT * 256)
  float* mref;            // [N][VT][2]: m_h per token, vocabulary tile and half tile
};

struct BwdLaunch {
  const void* x; const void* W; const void* b; const int64_t* targets;
  int N, H, V;            // V: rows of W (a shard's rows for the shard backward)
  int NT;
  int64_t vocab_start;    // global index of W's row 0; targets are global indices
  int64_t ignore_index;
  float eps, eps_over_v, s;
  float logit_scale;      // logits are logit_scale * (x W^T + b)
  int reduction;
  int accumulate;         // add dx, dW, db to what the outputs hold
  const float* lse; const int64_t* n_valid; const float* grad;
  void* coef;             // float4 [N]
  int* yv;                // [N]
  void* slab; int64_t ldS;
  float* dx_acc;          // [dx_split][N][H] fp32; with split_acc, uint16 [N][H]
  int dx_split;           // input-gradient K split: parts of each slab's columns, one accumulator each
  // 16-bit inputs, one part, several slabs: each fp32 accumulator value is
  // held as its high 16 bits in dx itself and its low 16 bits in dx_acc (the
  // last slab writes the rounded result over the high halves).
  int split_acc;
  float* dbp;             // [NT][ldS]: per token tile db partials of the current slab; null if no db
  float* gscale;          // fp16 inputs: {S, 1/S}, the dlogits slab's power-of-two scale; null otherwise
  void* dx; void* dW; void* db;
};

// Fused schedule, one chunk: the kept e values turned into dlogits in place.
struct FusedDz {
  void* ebuf; int64_t lde;
  const float* mref;      // [N][VT][2]
  const void* coef;       // float4 [N] from bwd_coef_kernel (with the fp16 slab scale)
  const int* yv;          // [N] target rows, -1 if ignored
  int N, V, VT;           // the chunk's tokens, vocabulary rows, vocabulary tiles
  float* dbp;             // [ceil(N / 256)][lde]: fp32 column sums per 256 tokens; null if no db
  const float* gscale;    // fp16: {S, 1/S}; the coefficients, so the stored dlogits, carry S; null otherwise
};

// dtype: 0 = fp32, 1 = bf16, 2 = fp16.  Each returns the launch error code.
hipError_t launch_forward(const FwdLaunch& a, int dtype, hipStream_t st);
// Shard forward: logits statistics of W's rows only, merged over phases into a.stats.
hipError_t launch_shard_forward(const FwdLaunch& a, int dtype, hipStream_t st);
// Merge of a.P shards' statistics (a.partials = float4 [P][N]) into lse, loss and the count.
hipError_t launch_merge(const FwdLaunch& a, hipStream_t st);
hipError_t launch_bwd_prepare(const BwdLaunch& a, hipStream_t st);
// dz_ready: the slab already holds the slab's dlogits (and, with want_db,
// the db partials in a.dbp), so the recompute is skipped.
hipError_t launch_bwd_slab(const BwdLaunch& a, int dtype, int vs, int width, int dx_mode, bool want_db,
                           bool dz_ready, hipStream_t st);
// dx = the sum of the a.dx_split fp32 accumulators (plus dx's old values when
// a.accumulate), written in dx's dtype.
hipError_t launch_bwd_dx_finalize(const BwdLaunch& a, int dtype, hipStream_t st);

// Fused schedule (gradients formed in the forward pass, one token chunk at a
// time).  launch_fused_count: the non-ignored count into a.n_valid before the
// first chunk.  launch_fused_forward: the chunk's logits tiles, statistics
// and kept e values, then the per-row lse and loss (a.* point at the chunk's
// rows).  launch_fused_dz: dlogits in place (and db column sums).
// launch_fused_products: the chunk's dx rows (K = the whole vocabulary) and
// its dW contribution, added to dW unless first (or a.accumulate) says to
// overwrite.  launch_fused_db: db accumulated in fp32 over the chunks
// (first: overwrite), and, with last, written to db in its dtype (added to
// it when accumulate).  launch_finalize: the reduced loss over all rows.
hipError_t launch_fused_count(const FwdLaunch& a, hipStream_t st);
hipError_t launch_fused_forward(const FwdLaunch& a, int dtype, hipStream_t st);
hipError_t launch_fused_dz(const FusedDz& f, int dtype, hipStream_t st);
hipError_t launch_fused_products(const BwdLaunch& a, int dtype, bool first, hipStream_t st);
hipError_t launch_fused_db(const float* dbp, int rows, int64_t lde, float* dbacc, int V, bool first, bool last,
                           void* db, int dtype, bool accumulate, hipStream_t st);
hipError_t launch_finalize(const FwdLaunch& a, hipStream_t st);
// Forward keeping the first slab's logits (e values in head.ebuf, maxima in
// head.mref) for the backward: head covers W's rows [0, head.V) with head.P
// phases, rest the remaining rest.V rows (vocab_start = head.V) with rest.P
// phases whose partials follow head's; then the merge and the final loss.
hipError_t launch_forward_keep(const FwdLaunch& head, const FwdLaunch& rest, int dtype, hipStream_t st);

// ---------------------------------------------------------------------------
// Feed-forward operators: the linear layer (nmat = 1) and the gated product
// (nmat = 2, weights 0 = gate, 1 = up).
// ---------------------------------------------------------------------------

enum Activation { kActNone = 0, kActRelu = 1, kActGelu = 2, kActGeluTanh = 3, kActSilu = 4, kActSigmoid = 5 };

// Most tokens that the few-token kernel takes.  16-bit: above 4 the 64 x 64
// tiles are as fast or faster (F=12288, H=4096 gated: 4 tokens 37.5 us against
// 35.2, 16 tokens 45 against 36); below, a small product spares the join's
// launch (F=1024, H=4096: 5.3 us against 8.3).  fp32: its MFMA is slow enough for
// the tiles to lose up to 16 tokens (gated 83 us against 117).
constexpr int skinny_tokens(int dtype) { return dtype == 0 ? 16 : 4; }
constexpr int kSkinnyMost = 16;

// Rows of H elements that are no whole 16-byte pieces (H % 8 != 0): x [rows[0]]
// and the weights copied to dst, one after the other, as rows of the padded
// width with zeros.
struct LayerPad {
  const void* src[3]; int64_t rows[3];
  int H, width;
  void* dst;
};

struct LayerFwd {
  const void* x; const void* W[2]; const void* b[2];   // rows of H elements (padded: H % 8 == 0)
  const void* residual;   // [N][F] added to the output, or null; may be y itself
  void* y;                // [N][F]
  float* z[2];            // [N][F] pre-activations kept for the backward (linear: z[0]), or null
  int N, H, F, act, nmat;
  int tile;               // S of the 32 S x 32 S output tiles: 8 (16-bit only), 4 or 2; 0: the few-token kernel
  int TM, TN;             // token tiles, feature tiles (gated: 16 S features each)
  int parts, kc;          // K split: parts of kc columns of x each
  float* part;            // parts > 1: [parts][N][ldp] fp32 sums; gated: u's at column ldp / 2
  int64_t ldp;            // nmat * F rounded up to 8
};

struct LayerBwd {
  const void* x; const void* W[2];
  const float* z[2];      // kept pre-activations (linear with kActNone: null)
  const void* dy;         // [N][F]
  int N, H, F, act, nmat; // x, W: rows of H elements (padded: H % 8 == 0)
  int Hout;               // dx, dW: rows of Hout elements
  void* dz;               // [N][ldz]: dz, zero from column F on; gated: dg, then du from column segk
  int64_t ldz;
  int segk;               // K (columns of dz) where weight 1 starts; past every K when nmat == 1
  bool dz_is_dy;          // dz is dy itself (no activation, F % 8 == 0): only its column sums are needed
  float* dbp; int64_t ldb;   // [db_blocks][ldb] fp32 partial column sums; null if no db
  int db_blocks, db_rows;    // token rows per block
  void* db[2];
  void* dx; int dx_tile, dx_parts, dx_kc;   // dx_tile and dw_tile, where neither is 8, are the same
  void* dW[2]; int dw_tile, dw_parts, dw_kc;
  float* dx_part; float* dw_part;   // split products: [parts][N][Hout], [parts][mats written][F][Hout]
};

hipError_t launch_layer_pad(const LayerPad& a, int dtype, hipStream_t st);
hipError_t launch_layer_forward(const LayerFwd& a, int dtype, hipStream_t st);
hipError_t launch_layer_backward(const LayerBwd& a, int dtype, hipStream_t st);

// ---------------------------------------------------------------------------
// Gradient norm and clipping
// ---------------------------------------------------------------------------

constexpr int kNormTensors = 96;             // tensors of one launch: their table fits in the kernel arguments

struct NormTable {
  const void* in[kNormTensors];
  void* out[kNormTensors];          // clipping: where the scaled gradients go (in[] itself when in place)
  int64_t n[kNormTensors];          // elements
  int64_t end[kNormTensors];        // chunks of this tensor and the ones before it
  uint8_t dtype[kNormTensors];
  int count;
  int chunk_bytes;                  // gradient bytes of one chunk: a power of two, 4096 or more
  int in_place;                     // out is in for every tensor
};

// parts partial sums of squares (or maxima) of the table's tensors, one per
// workgroup.  stream: read past the memory-side cache.
hipError_t launch_grad_norm(const NormTable& t, bool inf_norm, bool stream, double* part, int parts, hipStream_t st);
// The norm of `parts` partials, or *given, to norm_out (if set), and the table's tensors scaled by it.
hipError_t launch_grad_clip(const NormTable& t, bool inf_norm, const double* part, int parts, const float* given,
                            float* norm_out, float max_norm, int blocks, hipStream_t st);

}  // namespace flce
