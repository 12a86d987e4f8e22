// C-ABI entry points of the FLCE library: argument validation, workspace
// layout and the launch sequence.  No allocation and no host synchronisation:
// everything is enqueued on the caller's stream.
#include <algorithm>
#include <cmath>
#include <cstdlib>
#include <cstring>
#include <mutex>
#include <numeric>
#include <vector>

#include "flce.h"
#include "flce_launch.hpp"

namespace {

constexpr int kCUs = 256;                      // MI355X compute units
constexpr int kTile = 256;
constexpr size_t kAlign = 256;
constexpr size_t kSlabCapBytes = size_t(1) << 30;
constexpr size_t kSlabTargetBytes = size_t(256) << 20;
constexpr size_t kScratchBytes = FLCE_FORWARD_SCRATCH_BYTES;   // flce_forward_noalloc's static scratch

size_t align_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }
int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

struct Geometry {
  int NT, VT, P;
  int64_t slab_cols;
  int dx_split;
  size_t off_partials, off_rowloss, off_rowzl, fwd_total;
  size_t off_slab, off_dxacc, off_dbp, off_coef, off_yv, off_gscale, bwd_total;
  // Kept first slab (flce_forward_keep / flce_backward_kept): the forward's
  // kept-value schedule covers W's rows [0, width0) (VT0 tiles, P0 phases),
  // the plain forward the other VT - VT0 tiles (P1 phases); the keep buffer
  // holds the slab [N][slab_cols] in the input dtype at 0 and the maxima
  // [N][VT0][2] fp32 at off_kmref.
  int64_t width0;
  int VT0, P0, P1;
  size_t off_kmref, keep_total;
};

flce_status check_shape(int64_t N, int64_t H, int64_t V, int dtype) {
  if (N < 1 || H < 1 || V < 1) return FLCE_ERR_INVALID_ARGUMENT;
  if (dtype != FLCE_F32 && dtype != FLCE_BF16 && dtype != FLCE_F16) return FLCE_ERR_UNSUPPORTED;
  if (N > (int64_t(1) << 30) || V > (int64_t(1) << 30) || H > (int64_t(1) << 20)) return FLCE_ERR_UNSUPPORTED;
  if (H % 8 != 0) return FLCE_ERR_UNSUPPORTED;
  return FLCE_OK;
}

// Vocabulary slab width for the backward: the wider of (a) enough vocabulary
// tiles that the dW contraction of one slab (H/256 x slab/256 output tiles)
// fills every CU twice (once when the fp32 dx accumulator is under 128 MiB)
// and (b) the widest slab within 256 MiB whose dW tiles fill whole rounds of
// 256 CUs; capped at 1 GiB.  Every slab after the first costs one
// read-modify-write pass over the fp32 dx accumulator (N x H x 8 bytes),
// which all CUs make at the same moment, so wider slabs save HBM time when
// the accumulator is large; when it is small, a narrower slab is faster (at
// N=16384, H=1024, V=256000: 16384 columns instead of 32768, backward -1.7%,
// as more of the slab is still cached when dx and dW read it).  (b) gives the
// Llama-3-sized head (N=8192, H=4096, V=128256) 16384 columns, with all extra
// memory at 9.7% of its fp32 logits.
// FLCE_SLAB_COLS (a positive multiple of 256; the caller's memory knob) or
// else FLCE_DEBUG_SLAB_COLS (the tests force many slabs with it) overrides it.
int64_t slab_cols(int64_t N, int64_t H, int64_t V, int dtype) {
  const int64_t es = dtype == FLCE_F32 ? 4 : 2;
  const int64_t vmax = cdiv(V, kTile) * kTile;
  for (const char* name : {"FLCE_SLAB_COLS", "FLCE_DEBUG_SLAB_COLS"}) {
    if (const char* env = std::getenv(name)) {
      const long long c = std::atoll(env);
      if (c > 0 && c % kTile == 0) return c < vmax ? c : vmax;
    }
  }
  const int64_t th = cdiv(H, kTile);
  const bool small_acc = (size_t)N * (size_t)H * 4 < (size_t(128) << 20);
  int64_t want = cdiv((small_acc ? 1 : 2) * kCUs, th) * kTile;
  const int64_t round_cols = kTile * (kCUs / std::gcd((int64_t)kCUs, th));   // whole dW rounds
  const int64_t by_bytes = (int64_t)(kSlabTargetBytes / (size_t)(N * es)) / round_cols * round_cols;
  if (by_bytes > want) want = by_bytes;
  int64_t cap = (int64_t)(kSlabCapBytes / (size_t)(N * es)) / kTile * kTile;
  if (cap < kTile) cap = kTile;
  int64_t c = want < cap ? want : cap;
  return c < vmax ? c : vmax;
}

// Input-gradient K split.  The dx product has cdiv(N, 256) x cdiv(H, 256)
// output tiles, one workgroup each; when that is at most half the CUs, each
// slab's columns are split into parts that run side by side, each adding into
// its own fp32 accumulator, and the parts are summed once after the last slab.
// At most 8 parts of at least 512 columns.  The Llama-3-sized head (512
// tiles) never splits; N=4096, H=2048 (128 tiles) splits in two.
int dx_split(int64_t N, int64_t H, int64_t slab_cols) {
  const int64_t tiles = cdiv(N, kTile) * cdiv(H, kTile);
  if (2 * tiles > kCUs) return 1;
  int64_t p = kCUs / tiles;
  if (p > slab_cols / 512) p = slab_cols / 512;
  if (p > 8) p = 8;
  return p < 2 ? 1 : (int)p;
}

// Where the backward accumulates dx over the slabs.  Several K parts: one
// fp32 [N][H] accumulator each, summed once at the end.  One part and several
// slabs: fp32 inputs accumulate in dx itself; 16-bit inputs keep each fp32
// value's high half in dx and its low half in an [N][H] 16-bit array (exact:
// the value is the two halves' bits).  One slab: no accumulator.
bool dx_in_place(int64_t V, int64_t slab_cols, int parts) { return parts <= 1 && cdiv(V, slab_cols) > 1; }

size_t dx_acc_bytes(int64_t N, int64_t H, int64_t V, int dtype, int64_t slab_cols, int parts) {
  if (parts > 1) return (size_t)parts * N * H * 4;
  if (!dx_in_place(V, slab_cols, parts) || dtype == FLCE_F32) return 0;
  return (size_t)N * H * 2;
}

// Forward phases for NT token tiles: enough that the grid (token tiles x
// phases) fills the CUs, and at least 8 (see geometry), at most VT.
int fwd_phases(int NT, int VT) {
  int P = kCUs / NT;
  if (P < 8) P = 8;
  if (P > VT) P = VT;
  return P;
}

// with_dx_acc: the backward keeps its own fp32 dx accumulator (the shard
// backward accumulates into the caller's buffer instead).  kept: the layouts
// of flce_forward_keep and flce_backward_kept (the forward's partials cover
// both of its launches' phases; the backward's slab is the keep buffer).
Geometry geometry(int64_t N, int64_t H, int64_t V, int dtype, int has_bias, bool with_dx_acc = true,
                  bool kept = false) {
  Geometry g{};
  const int64_t es = dtype == FLCE_F32 ? 4 : 2;
  g.NT = (int)cdiv(N, kTile);
  g.VT = (int)cdiv(V, kTile);
  g.slab_cols = slab_cols(N, H, V, dtype);
  g.width0 = g.slab_cols < V ? g.slab_cols : V;
  g.VT0 = (int)cdiv(g.width0, kTile);
  g.P0 = fwd_phases(g.NT, g.VT0);
  g.P1 = g.VT > g.VT0 ? fwd_phases(g.NT, g.VT - g.VT0) : 0;
  // Forward phases: enough that the grid (token tiles x phases) fills the CUs,
  // and at least 8, so that each XCD's 32 concurrent tiles are 4 token tiles
  // x 8 vocabulary tiles (12 operand panels per round; 16 x 2 at N=32768
  // would stream 18) and take x's copies first.  Past 256 workgroups the grid
  // runs in rounds.  N=32768, H=2048, V=128000: 8 phases instead of 2, forward
  // -3.7% (same-box A/B).
  const int P = fwd_phases(g.NT, g.VT);
  g.P = P;
  size_t off = 0;
  g.off_partials = off;
  off = align_up(off + (size_t)(kept ? g.P0 + g.P1 : P) * N * 16);
  g.off_rowloss = off;
  off = align_up(off + (size_t)N * 4);
  g.off_rowzl = off;
  off = align_up(off + (size_t)N * 4);
  g.fwd_total = off;

  g.dx_split = with_dx_acc ? dx_split(N, H, g.slab_cols) : 1;
  off = 0;
  g.off_slab = off;
  if (!kept) off = align_up(off + (size_t)N * g.slab_cols * es);
  g.off_dxacc = off;
  if (with_dx_acc) off = align_up(off + dx_acc_bytes(N, H, V, dtype, g.slab_cols, g.dx_split));
  g.off_dbp = off;
  if (has_bias) off = align_up(off + (size_t)g.NT * g.slab_cols * 4);
  g.off_coef = off;
  off = align_up(off + (size_t)N * 16);
  g.off_yv = off;
  off = align_up(off + (size_t)N * 4);
  g.off_gscale = off;   // fp16: the dlogits slab's scale {S, 1/S}
  if (dtype == FLCE_F16) off = align_up(off + 8);
  g.bwd_total = off;

  g.off_kmref = align_up((size_t)N * g.slab_cols * es);
  g.keep_total = align_up(g.off_kmref + (size_t)N * g.VT0 * 2 * 4);
  return g;
}

// Fused schedule (gradients formed in the forward pass, one token chunk at a
// time).  Workspace: the chunk's kept logits [chunk][VT * 256] in the input
// dtype (turned into dlogits in place), their per-(token, tile, half) maxima,
// the chunk forward's per-phase partials, per-row losses of all N tokens,
// per-token coefficients, the dx product's K-split accumulators, and db's
// per-256-token column sums and fp32 running total.  Sized for the largest
// chunk and for the shorter last chunk, whichever needs more.
struct FusedGeometry {
  int64_t chunk;
  int VT;
  int64_t lde;
  size_t off_partials, off_rowloss, off_rowzl, off_e, off_mref, off_coef, off_yv, off_dxacc, off_dbp, off_dbacc,
      off_gscale, total;
};

FusedGeometry fused_geometry(int64_t N, int64_t H, int64_t V, int dtype, int has_bias, int64_t chunk) {
  FusedGeometry g{};
  const int64_t es = dtype == FLCE_F32 ? 4 : 2;
  g.chunk = chunk < N ? chunk : N;
  g.VT = (int)cdiv(V, kTile);
  g.lde = (int64_t)g.VT * kTile;
  const int64_t nchunks = cdiv(N, g.chunk);
  const int64_t sizes[2] = {g.chunk, N - (nchunks - 1) * g.chunk};
  size_t part = 0, dxacc = 0;
  for (int64_t c : sizes) {
    const int NTc = (int)cdiv(c, kTile);
    const size_t p = (size_t)fwd_phases(NTc, g.VT) * c * 16;
    const int split = dx_split(c, H, g.lde);
    const size_t a = split > 1 ? (size_t)split * c * H * 4 : 0;
    if (p > part) part = p;
    if (a > dxacc) dxacc = a;
  }
  size_t off = 0;
  g.off_partials = off;
  off = align_up(off + part);
  g.off_rowloss = off;
  off = align_up(off + (size_t)N * 4);
  g.off_rowzl = off;
  off = align_up(off + (size_t)N * 4);
  g.off_e = off;
  off = align_up(off + (size_t)g.chunk * g.lde * es);
  g.off_mref = off;
  off = align_up(off + (size_t)g.chunk * g.VT * 2 * 4);
  g.off_coef = off;
  off = align_up(off + (size_t)g.chunk * 16);
  g.off_yv = off;
  off = align_up(off + (size_t)g.chunk * 4);
  g.off_dxacc = off;
  off = align_up(off + dxacc);
  g.off_dbp = off;
  if (has_bias) off = align_up(off + (size_t)cdiv(g.chunk, kTile) * g.lde * 4);
  g.off_dbacc = off;
  if (has_bias) off = align_up(off + (size_t)V * 4);
  g.off_gscale = off;
  if (dtype == FLCE_F16) off = align_up(off + 8);
  g.total = off;
  return g;
}

// Default chunk: the fewest chunks whose workspace fits in what the recompute
// schedule uses for the same problem (forward plus backward workspace: the
// two schedules then compare at equal extra memory), then balanced, in
// multiples of 256 tokens.  At least 256 tokens.
int64_t fused_default_chunk(int64_t N, int64_t H, int64_t V, int dtype, int has_bias) {
  const Geometry r = geometry(N, H, V, dtype, has_bias);
  const size_t budget = r.fwd_total + r.bwd_total;
  int64_t best = kTile;
  for (int64_t c = cdiv(N, kTile) * kTile; c >= kTile; c -= kTile) {
    if (fused_geometry(N, H, V, dtype, has_bias, c).total <= budget) {
      best = c;
      break;
    }
  }
  const int64_t nchunks = cdiv(N, best);
  return cdiv(cdiv(N, nchunks), kTile) * kTile;
}

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

flce_status check_options(float eps, float s, int reduction) {
  if (!(eps >= 0.f && eps <= 1.f)) return FLCE_ERR_INVALID_ARGUMENT;
  if (!(s >= 0.f) || !std::isfinite(s)) return FLCE_ERR_INVALID_ARGUMENT;
  if (reduction != FLCE_REDUCTION_NONE && reduction != FLCE_REDUCTION_SUM && reduction != FLCE_REDUCTION_MEAN)
    return FLCE_ERR_INVALID_ARGUMENT;
  return FLCE_OK;
}

flce_status check_shard(int64_t V_shard, int64_t vocab_start, int64_t V_total) {
  if (vocab_start < 0 || V_total < 1 || V_total > (int64_t(1) << 30)) return FLCE_ERR_INVALID_ARGUMENT;
  if (vocab_start + V_shard > V_total) return FLCE_ERR_INVALID_ARGUMENT;
  return FLCE_OK;
}

flce_status check_inputs(const void* x, const void* W, const void* b, const int64_t* targets, int dtype) {
  if (!x || !W || !targets) return FLCE_ERR_INVALID_ARGUMENT;
  if (!aligned(x, 16) || !aligned(W, 16) || !aligned(targets, 8)) return FLCE_ERR_INVALID_ARGUMENT;
  if (b && !aligned(b, dtype == FLCE_F32 ? 4 : 2)) return FLCE_ERR_INVALID_ARGUMENT;
  return FLCE_OK;
}

// Backward launch sequence shared by the full and the shard entry points:
// per-token coefficients, then per slab the recompute, dx and dW (+ db)
// launches.  dx_out_fp32: dx is the fp32 accumulator itself (a.dx_acc),
// never cast; accumulate: it already holds a partial sum to add to.
// kmref (flce_backward_kept): the slab buffer a.slab already holds slab 0's
// kept values e and kmref their maxima; slab 0's dlogits are made from them in
// place (and its db partials written) instead of being recomputed.
flce_status run_backward(flce::BwdLaunch& a, const Geometry& g, int64_t V, int dtype, bool want_db,
                         bool dx_out_fp32, bool accumulate, hipStream_t s, const float* kmref = nullptr) {
  (void)hipGetLastError();
  flce::mark_launch(s, nullptr);
  if (flce::launch_bwd_prepare(a, s) != hipSuccess) return FLCE_ERR_HIP;
  if (kmref) {
    flce::FusedDz fd{};
    fd.ebuf = a.slab; fd.lde = a.ldS;
    fd.mref = kmref;
    fd.coef = a.coef; fd.yv = a.yv;
    fd.N = a.N; fd.V = (int)g.width0; fd.VT = g.VT0;
    fd.dbp = want_db ? a.dbp : nullptr;
    fd.gscale = nullptr;   // db partials of dz * S, as the recompute writes them (1/S is applied in their sum)
    if (flce::launch_fused_dz(fd, dtype, s) != hipSuccess) return FLCE_ERR_HIP;
  }
  const int64_t cols = g.slab_cols;
  const int64_t nslab = cdiv(V, cols);
  // dx accumulated in place (see dx_acc_bytes): fp32 dx is its own
  // accumulator, which the caller's-buffer modes below handle.
  const bool in_place = !dx_out_fp32 && a.dx && dx_in_place(V, cols, a.dx_split);
  const bool fp32_in_place = in_place && dtype == FLCE_F32;
  if (fp32_in_place) a.dx_acc = (float*)a.dx;
  a.split_acc = in_place && dtype != FLCE_F32;
  for (int64_t k = 0; k < nslab; ++k) {
    const int64_t vs = k * cols;
    const int64_t width = (V - vs) < cols ? (V - vs) : cols;
    int mode = flce::kDxAccum;
    if (dx_out_fp32 || fp32_in_place) {
      if (k == 0 && !(accumulate || (fp32_in_place && a.accumulate))) mode = flce::kDxFirst;
    } else if (a.dx_split > 1) {
      mode = k == 0 ? flce::kDxFirst : flce::kDxAccum;   // the parts' sum is written below
    } else if (nslab == 1) {
      mode = flce::kDxOnly;
    } else if (k == 0) {
      mode = flce::kDxFirst;
    } else if (k == nslab - 1) {
      mode = flce::kDxLast;
    }
    if (flce::launch_bwd_slab(a, dtype, (int)vs, (int)width, mode, want_db, kmref && k == 0, s) != hipSuccess)
      return FLCE_ERR_HIP;
  }
  if (a.dx && !dx_out_fp32 && a.dx_split > 1 && flce::launch_bwd_dx_finalize(a, dtype, s) != hipSuccess)
    return FLCE_ERR_HIP;
  return FLCE_OK;
}

flce_options default_options() {
  flce_options o{};
  o.logit_scale = 1.f;
  o.accumulate = 0;
  o.z_loss = nullptr;
  return o;
}

// Host-side checks of a forward call (no HIP call).
flce_status check_forward(const void* x, const void* W, const void* b, const int64_t* targets, int64_t N,
                          int64_t H, int64_t V, int dtype, float eps, float s, int reduction, const flce_options& o,
                          const float* loss, const float* lse, const int64_t* n_valid) {
  if (!std::isfinite(o.logit_scale)) return FLCE_ERR_INVALID_ARGUMENT;
  if (o.z_loss && !aligned(o.z_loss, 4)) return FLCE_ERR_INVALID_ARGUMENT;
  flce_status st = check_shape(N, H, V, dtype);
  if (st != FLCE_OK) return st;
  if ((st = check_options(eps, s, reduction)) != FLCE_OK) return st;
  if ((st = check_inputs(x, W, b, targets, dtype)) != FLCE_OK) return st;
  if (!loss || !lse || !n_valid || !aligned(loss, 4) || !aligned(lse, 4) || !aligned(n_valid, 8))
    return FLCE_ERR_INVALID_ARGUMENT;
  return FLCE_OK;
}

// The forward's launches, with its per-phase partials and per-row losses in
// ws (g.fwd_total bytes, laid out by geometry()).
flce_status forward_into(const Geometry& g, const void* x, const void* W, const void* b, const int64_t* targets,
                         int64_t N, int64_t H, int64_t V, int dtype, float eps, float s, int64_t ignore_index,
                         int reduction, const flce_options& o, float* loss, float* lse, int64_t* n_valid, char* ws,
                         hipStream_t stream) {
  flce::FwdLaunch a{};
  a.x = x; a.W = W; a.b = b; a.targets = targets;
  a.N = (int)N; a.H = (int)H; a.V = (int)V;
  a.NT = g.NT; a.P = g.P; a.VT = g.VT;
  a.ignore_index = ignore_index;
  a.eps = eps;
  a.eps_over_v = (float)((double)eps / (double)V);
  a.s = s;
  a.reduction = reduction;
  a.logit_scale = o.logit_scale;
  a.partials = ws + g.off_partials;
  a.rowloss = (float*)(ws + g.off_rowloss);
  a.rowzl = (float*)(ws + g.off_rowzl);
  a.zloss = o.z_loss;
  a.loss = loss; a.lse = lse; a.n_valid = n_valid;
  (void)hipGetLastError();
  flce::mark_launch(stream, nullptr);
  if (flce::launch_forward(a, dtype, stream) != hipSuccess) return FLCE_ERR_HIP;
  return FLCE_OK;
}

// flce_forward_keep's launches: the kept-value forward over W's first
// g.width0 rows, writing e and its maxima into keep, and the plain forward
// over the rest, then one merge.
flce_status forward_keep_into(const Geometry& g, const void* x, const void* W, const void* b,
                              const int64_t* targets, int64_t N, int64_t H, int64_t V, int dtype, float eps, float s,
                              int64_t ignore_index, int reduction, const flce_options& o, float* loss, float* lse,
                              int64_t* n_valid, char* keep, char* ws, hipStream_t stream) {
  const int64_t es = dtype == FLCE_F32 ? 4 : 2;
  flce::FwdLaunch head{};
  head.x = x; head.W = W; head.b = b; head.targets = targets;
  head.N = (int)N; head.H = (int)H; head.V = (int)g.width0;
  head.NT = g.NT; head.P = g.P0; head.VT = g.VT0;
  head.ignore_index = ignore_index;
  head.eps = eps;
  head.eps_over_v = (float)((double)eps / (double)V);
  head.s = s;
  head.reduction = reduction;
  head.logit_scale = o.logit_scale;
  head.partials = ws + g.off_partials;
  head.rowloss = (float*)(ws + g.off_rowloss);
  head.rowzl = (float*)(ws + g.off_rowzl);
  head.zloss = o.z_loss;
  head.loss = loss; head.lse = lse; head.n_valid = n_valid;
  head.ebuf = keep;
  head.lde = g.slab_cols;
  head.mref = (float*)(keep + g.off_kmref);
  flce::FwdLaunch rest = head;
  rest.V = (int)(V - g.width0);
  if (rest.V > 0) {
    rest.W = (const char*)W + g.width0 * H * es;
    rest.b = b ? (const char*)b + g.width0 * es : nullptr;
    rest.VT = g.VT - g.VT0;
    rest.P = g.P1;
    rest.vocab_start = g.width0;
    rest.partials = ws + g.off_partials + (size_t)g.P0 * N * 16;
    rest.ebuf = nullptr;
    rest.mref = nullptr;
  }
  (void)hipGetLastError();
  flce::mark_launch(stream, nullptr);
  if (flce::launch_forward_keep(head, rest, dtype, stream) != hipSuccess) return FLCE_ERR_HIP;
  return FLCE_OK;
}

// ---------------------------------------------------------------------------
// Launch timing log (flce_timing_*).  Per host thread: a fixed set of events
// created by flce_timing_start, recorded in order by mark_launch until the
// set is used up.
// ---------------------------------------------------------------------------
struct TimingLog {
  bool on = false;
  size_t used = 0;
  std::vector<hipEvent_t> ev;
  std::vector<const char*> tag;
  std::vector<int> launch_mark;   // mark index that ends each logged launch
};
thread_local TimingLog g_tlog;

void timing_clear(TimingLog& t) {
  for (hipEvent_t e : t.ev) (void)hipEventDestroy(e);
  t.ev.clear();
  t.tag.clear();
  t.launch_mark.clear();
  t.used = 0;
  t.on = false;
}

// ---------------------------------------------------------------------------
// Static forward scratch (flce_forward_noalloc).  Each GPU holds its own copy
// of this array at its own address for the life of the process; host code
// uses only the address hipGetSymbolAddress returns for a device (the array's
// name on the host is a stand-in, not a device address).  The address is
// looked up once per device, with that device current, and cached.  The
// forward writes every byte it later reads (each phase's partials for every
// token, each row's loss), so nothing needs clearing between calls.
// ---------------------------------------------------------------------------

static __device__ __align__(256) char scratch[kScratchBytes];

constexpr int kMaxDevices = 64;
std::mutex g_scratch_mu;
char* g_scratch_ptr[kMaxDevices] = {};

// The scratch array of the device that `stream` belongs to, which must be the
// current device (the symbol lookup is made with that device current).
flce_status scratch_on_stream_device(hipStream_t stream, char** out) {
  int cur = -1;
  if (hipGetDevice(&cur) != hipSuccess || cur < 0 || cur >= kMaxDevices) return FLCE_ERR_HIP;
  if (stream) {
    hipDevice_t sd = -1;
    if (hipStreamGetDevice(stream, &sd) != hipSuccess) return FLCE_ERR_HIP;
    if (sd != cur) return FLCE_ERR_INVALID_ARGUMENT;
  }
  std::lock_guard<std::mutex> lock(g_scratch_mu);
  if (!g_scratch_ptr[cur]) {
    void* p = nullptr;
    if (hipGetSymbolAddress(&p, HIP_SYMBOL(scratch)) != hipSuccess || !p) return FLCE_ERR_HIP;
    g_scratch_ptr[cur] = (char*)p;
  }
  *out = g_scratch_ptr[cur];
  return FLCE_OK;
}

flce_status backward_impl(const void* x, const void* W, const void* b, const int64_t* targets, int64_t N, int64_t H,
                          int64_t V, flce_dtype dtype, float label_smoothing, float z_loss_scale, int64_t ignore_index,
                          flce_reduction reduction, const flce_options* opts, const float* lse, const int64_t* n_valid,
                          const float* grad_loss, void* dx, void* dW, void* db, void* keep, size_t keep_bytes,
                          void* workspace, size_t workspace_bytes, hipStream_t stream);

}  // namespace

namespace flce {
void mark_launch(hipStream_t st, const char* kernel) {
  TimingLog& t = g_tlog;
  if (!t.on || t.used >= t.ev.size()) return;
  if (hipEventRecord(t.ev[t.used], st) != hipSuccess) {
    t.on = false;
    return;
  }
  t.tag[t.used] = kernel;
  if (kernel && t.used > 0) t.launch_mark.push_back((int)t.used);
  ++t.used;
}
}  // namespace flce

extern "C" {

flce_status flce_timing_start(int capacity) {
  if (capacity < 2 || capacity > (1 << 20)) return FLCE_ERR_INVALID_ARGUMENT;
  TimingLog& t = g_tlog;
  timing_clear(t);
  t.ev.resize((size_t)capacity, nullptr);
  t.tag.assign((size_t)capacity, nullptr);
  for (int i = 0; i < capacity; ++i) {
    // timing only: no system-scope fence (cache writeback) at each record
    if (hipEventCreateWithFlags(&t.ev[(size_t)i], hipEventDisableSystemFence) != hipSuccess) {
      t.ev.resize((size_t)i);
      timing_clear(t);
      return FLCE_ERR_HIP;
    }
  }
  t.on = true;
  return FLCE_OK;
}

flce_status flce_timing_stop(void) {
  g_tlog.on = false;
  return FLCE_OK;
}

int64_t flce_timing_count(void) { return (int64_t)g_tlog.launch_mark.size(); }

flce_status flce_timing_read(int64_t index, const char** kernel, float* ms) {
  const TimingLog& t = g_tlog;
  if (index < 0 || index >= (int64_t)t.launch_mark.size() || !kernel || !ms) return FLCE_ERR_INVALID_ARGUMENT;
  const int j = t.launch_mark[(size_t)index];
  if (hipEventSynchronize(t.ev[(size_t)j]) != hipSuccess) return FLCE_ERR_HIP;
  if (hipEventElapsedTime(ms, t.ev[(size_t)j - 1], t.ev[(size_t)j]) != hipSuccess) return FLCE_ERR_HIP;
  *kernel = t.tag[(size_t)j];
  return FLCE_OK;
}

flce_status flce_timing_clear(void) {
  timing_clear(g_tlog);
  return FLCE_OK;
}

const char* flce_status_string(flce_status status) {
  switch (status) {
    case FLCE_OK: return "ok";
    case FLCE_ERR_INVALID_ARGUMENT: return "invalid argument";
    case FLCE_ERR_UNSUPPORTED: return "unsupported dtype or shape";
    case FLCE_ERR_WORKSPACE_TOO_SMALL: return "workspace too small";
    case FLCE_ERR_HIP: return "HIP launch failed";
    case FLCE_ERR_SCRATCH_TOO_SMALL: return "problem needs more forward scratch than the static buffer holds";
    default: return "unknown status";
  }
}

int64_t flce_backward_slab_cols(int64_t N, int64_t H, int64_t V, flce_dtype dtype) {
  if (check_shape(N, H, V, dtype) != FLCE_OK) return 0;
  return slab_cols(N, H, V, dtype);
}

flce_status flce_workspace_size(int64_t N, int64_t H, int64_t V, flce_dtype dtype, int has_bias, flce_reduction reduction,
                                size_t* fwd_bytes, size_t* bwd_bytes) {
  flce_status st = check_shape(N, H, V, dtype);
  if (st != FLCE_OK) return st;
  st = check_options(0.f, 0.f, reduction);
  if (st != FLCE_OK) return st;
  const Geometry g = geometry(N, H, V, dtype, has_bias);
  if (fwd_bytes) *fwd_bytes = g.fwd_total;
  if (bwd_bytes) *bwd_bytes = g.bwd_total;
  return FLCE_OK;
}

flce_status flce_forward(const void* x, const void* W, const void* b, const int64_t* targets, int64_t N,
                         int64_t H, int64_t V, flce_dtype dtype, float label_smoothing, float z_loss_scale,
                         int64_t ignore_index, flce_reduction reduction, float* loss, float* lse, int64_t* n_valid,
                         void* workspace, size_t workspace_bytes, hipStream_t stream) {
  return flce_forward_ex(x, W, b, targets, N, H, V, dtype, label_smoothing, z_loss_scale, ignore_index, reduction,
                         nullptr, loss, lse, n_valid, workspace, workspace_bytes, stream);
}

flce_status flce_forward_ex(const void* x, const void* W, const void* b, const int64_t* targets, int64_t N,
                            int64_t H, int64_t V, flce_dtype dtype, float label_smoothing, float z_loss_scale,
                            int64_t ignore_index, flce_reduction reduction, const flce_options* opts, float* loss, float* lse,
                            int64_t* n_valid, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  const flce_options o = opts ? *opts : default_options();
  flce_status st = check_forward(x, W, b, targets, N, H, V, dtype, label_smoothing, z_loss_scale, reduction, o,
                                 loss, lse, n_valid);
  if (st != FLCE_OK) return st;
  const Geometry g = geometry(N, H, V, dtype, b != nullptr);
  if (workspace_bytes < g.fwd_total) return FLCE_ERR_WORKSPACE_TOO_SMALL;
  if (!workspace || !aligned(workspace, 16)) return FLCE_ERR_INVALID_ARGUMENT;
  return forward_into(g, x, W, b, targets, N, H, V, dtype, label_smoothing, z_loss_scale, ignore_index, reduction,
                      o, loss, lse, n_valid, (char*)workspace, (hipStream_t)stream);
}

flce_status flce_forward_noalloc(const void* x, const void* W, const void* b, const int64_t* targets, int64_t N,
                                 int64_t H, int64_t V, flce_dtype dtype, float label_smoothing, float z_loss_scale,
                                 int64_t ignore_index, flce_reduction reduction, const flce_options* opts, float* loss,
                                 float* lse, int64_t* n_valid, hipStream_t stream) {
  const flce_options o = opts ? *opts : default_options();
  flce_status st = check_forward(x, W, b, targets, N, H, V, dtype, label_smoothing, z_loss_scale, reduction, o,
                                 loss, lse, n_valid);
  if (st != FLCE_OK) return st;
  const Geometry g = geometry(N, H, V, dtype, b != nullptr);
  if (g.fwd_total > kScratchBytes) return FLCE_ERR_SCRATCH_TOO_SMALL;
  char* ws = nullptr;
  if ((st = scratch_on_stream_device((hipStream_t)stream, &ws)) != FLCE_OK) return st;
  return forward_into(g, x, W, b, targets, N, H, V, dtype, label_smoothing, z_loss_scale, ignore_index, reduction,
                      o, loss, lse, n_valid, ws, (hipStream_t)stream);
}

flce_status flce_backward(const void* x, const void* W, const void* b, const int64_t* targets, int64_t N,
                          int64_t H, int64_t V, flce_dtype dtype, float label_smoothing, float z_loss_scale,
                          int64_t ignore_index, flce_reduction reduction, const float* lse, const int64_t* n_valid,
                          const float* grad_loss, void* dx, void* dW, void* db, void* workspace,
                          size_t workspace_bytes, hipStream_t stream) {
  return flce_backward_ex(x, W, b, targets, N, H, V, dtype, label_smoothing, z_loss_scale, ignore_index, reduction,
                          nullptr, lse, n_valid, grad_loss, dx, dW, db, workspace, workspace_bytes, stream);
}

flce_status flce_backward_ex(const void* x, const void* W, const void* b, const int64_t* targets, int64_t N,
                             int64_t H, int64_t V, flce_dtype dtype, float label_smoothing, float z_loss_scale,
                             int64_t ignore_index, flce_reduction reduction, const flce_options* opts, const float* lse,
                             const int64_t* n_valid, const float* grad_loss, void* dx, void* dW, void* db,
                             void* workspace, size_t workspace_bytes, hipStream_t stream) {
  return backward_impl(x, W, b, targets, N, H, V, dtype, label_smoothing, z_loss_scale, ignore_index, reduction, opts,
                       lse, n_valid, grad_loss, dx, dW, db, nullptr, 0, workspace, workspace_bytes, stream);
}

flce_status flce_keep_workspace_size(int64_t N, int64_t H, int64_t V, flce_dtype dtype, int has_bias,
                                     flce_reduction reduction, size_t* fwd_bytes, size_t* keep_bytes,
                                     size_t* bwd_bytes) {
  flce_status st = check_shape(N, H, V, dtype);
  if (st != FLCE_OK) return st;
  st = check_options(0.f, 0.f, reduction);
  if (st != FLCE_OK) return st;
  const Geometry g = geometry(N, H, V, dtype, has_bias, true, true);
  if (fwd_bytes) *fwd_bytes = g.fwd_total;
  if (keep_bytes) *keep_bytes = g.keep_total;
  if (bwd_bytes) *bwd_bytes = g.bwd_total;
  return FLCE_OK;
}

flce_status flce_forward_keep(const void* x, const void* W, const void* b, const int64_t* targets, int64_t N,
                              int64_t H, int64_t V, flce_dtype dtype, float label_smoothing, float z_loss_scale,
                              int64_t ignore_index, flce_reduction reduction, const flce_options* opts, float* loss,
                              float* lse, int64_t* n_valid, void* keep, size_t keep_bytes, void* workspace,
                              size_t workspace_bytes, hipStream_t stream) {
  const flce_options o = opts ? *opts : default_options();
  flce_status st = check_forward(x, W, b, targets, N, H, V, dtype, label_smoothing, z_loss_scale, reduction, o,
                                 loss, lse, n_valid);
  if (st != FLCE_OK) return st;
  const Geometry g = geometry(N, H, V, dtype, b != nullptr, true, true);
  if (workspace_bytes < g.fwd_total || keep_bytes < g.keep_total) return FLCE_ERR_WORKSPACE_TOO_SMALL;
  if (!workspace || !aligned(workspace, 16) || !keep || !aligned(keep, 16)) return FLCE_ERR_INVALID_ARGUMENT;
  return forward_keep_into(g, x, W, b, targets, N, H, V, dtype, label_smoothing, z_loss_scale, ignore_index,
                           reduction, o, loss, lse, n_valid, (char*)keep, (char*)workspace, (hipStream_t)stream);
}

flce_status flce_backward_kept(const void* x, const void* W, const void* b, const int64_t* targets, int64_t N,
                               int64_t H, int64_t V, flce_dtype dtype, float label_smoothing, float z_loss_scale,
                               int64_t ignore_index, flce_reduction reduction, const flce_options* opts,
                               const float* lse, const int64_t* n_valid, const float* grad_loss, void* keep,
                               size_t keep_bytes, void* dx, void* dW, void* db, void* workspace,
                               size_t workspace_bytes, hipStream_t stream) {
  if (!keep) return FLCE_ERR_INVALID_ARGUMENT;
  return backward_impl(x, W, b, targets, N, H, V, dtype, label_smoothing, z_loss_scale, ignore_index, reduction, opts,
                       lse, n_valid, grad_loss, dx, dW, db, keep, keep_bytes, workspace, workspace_bytes, stream);
}

}  // extern "C"

namespace {

// flce_backward_ex, and with keep != NULL flce_backward_kept.
flce_status backward_impl(const void* x, const void* W, const void* b, const int64_t* targets, int64_t N, int64_t H,
                          int64_t V, flce_dtype dtype, float label_smoothing, float z_loss_scale, int64_t ignore_index,
                          flce_reduction reduction, const flce_options* opts, const float* lse, const int64_t* n_valid,
                          const float* grad_loss, void* dx, void* dW, void* db, void* keep, size_t keep_bytes,
                          void* workspace, size_t workspace_bytes, hipStream_t stream) {
  const flce_options o = opts ? *opts : default_options();
  if (!std::isfinite(o.logit_scale)) return FLCE_ERR_INVALID_ARGUMENT;
  flce_status st = check_shape(N, H, V, dtype);
  if (st != FLCE_OK) return st;
  if ((st = check_options(label_smoothing, z_loss_scale, reduction)) != FLCE_OK) return st;
  if ((st = check_inputs(x, W, b, targets, dtype)) != FLCE_OK) return st;
  if (!lse || !n_valid || !grad_loss) return FLCE_ERR_INVALID_ARGUMENT;
  if (!aligned(lse, 4) || !aligned(n_valid, 8) || !aligned(grad_loss, 4)) return FLCE_ERR_INVALID_ARGUMENT;
  if ((dx && !aligned(dx, 16)) || (dW && !aligned(dW, 16))) return FLCE_ERR_INVALID_ARGUMENT;
  if (db && !aligned(db, dtype == FLCE_F32 ? 4 : 2)) return FLCE_ERR_INVALID_ARGUMENT;
  const bool kept = keep != nullptr;
  const Geometry g = geometry(N, H, V, dtype, b != nullptr, true, kept);
  if (workspace_bytes < g.bwd_total || (kept && keep_bytes < g.keep_total)) return FLCE_ERR_WORKSPACE_TOO_SMALL;
  if (!workspace || !aligned(workspace, 16) || (kept && !aligned(keep, 16))) return FLCE_ERR_INVALID_ARGUMENT;
  const bool want_db = b != nullptr && db != nullptr;
  if (!dx && !dW && !want_db) return FLCE_OK;

  char* ws = (char*)workspace;
  flce::BwdLaunch a{};
  a.x = x; a.W = W; a.b = b; a.targets = targets;
  a.N = (int)N; a.H = (int)H; a.V = (int)V;
  a.NT = g.NT;
  a.ignore_index = ignore_index;
  a.eps = label_smoothing;
  a.eps_over_v = (float)((double)label_smoothing / (double)V);
  a.s = z_loss_scale;
  a.logit_scale = o.logit_scale;
  a.reduction = reduction;
  a.accumulate = o.accumulate != 0;
  a.lse = lse; a.n_valid = n_valid; a.grad = grad_loss;
  a.coef = ws + g.off_coef;
  a.yv = (int*)(ws + g.off_yv);
  a.slab = kept ? (char*)keep : ws + g.off_slab;
  a.ldS = g.slab_cols;
  a.dx_acc = (float*)(ws + g.off_dxacc);
  a.dx_split = g.dx_split;
  a.dbp = want_db ? (float*)(ws + g.off_dbp) : nullptr;
  a.gscale = dtype == FLCE_F16 ? (float*)(ws + g.off_gscale) : nullptr;
  a.dx = dx; a.dW = dW; a.db = want_db ? db : nullptr;

  return run_backward(a, g, V, dtype, want_db, false, false, (hipStream_t)stream,
                      kept ? (const float*)((char*)keep + g.off_kmref) : nullptr);
}

}  // namespace

extern "C" {

flce_status flce_fused_workspace_size(int64_t N, int64_t H, int64_t V, flce_dtype dtype, int has_bias,
                                      int64_t chunk_tokens, int64_t* chunk_used, size_t* bytes) {
  flce_status st = check_shape(N, H, V, dtype);
  if (st != FLCE_OK) return st;
  if (chunk_tokens < 0 || chunk_tokens % kTile != 0) return FLCE_ERR_INVALID_ARGUMENT;
  const int64_t chunk = chunk_tokens ? chunk_tokens : fused_default_chunk(N, H, V, dtype, has_bias);
  const FusedGeometry g = fused_geometry(N, H, V, dtype, has_bias, chunk);
  if (chunk_used) *chunk_used = g.chunk;
  if (bytes) *bytes = g.total;
  return FLCE_OK;
}

flce_status flce_fused_forward_backward(const void* x, const void* W, const void* b, const int64_t* targets,
                                        int64_t N, int64_t H, int64_t V, flce_dtype dtype, float label_smoothing,
                                        float z_loss_scale, int64_t ignore_index, flce_reduction reduction,
                                        const flce_options* opts, const float* grad_loss, int64_t chunk_tokens,
                                        float* loss, float* lse, int64_t* n_valid, void* dx, void* dW, void* db,
                                        void* workspace, size_t workspace_bytes, hipStream_t stream) {
  const flce_options o = opts ? *opts : default_options();
  flce_status st = check_forward(x, W, b, targets, N, H, V, dtype, label_smoothing, z_loss_scale, reduction, o,
                                 loss, lse, n_valid);
  if (st != FLCE_OK) return st;
  if (!grad_loss || !aligned(grad_loss, 4)) return FLCE_ERR_INVALID_ARGUMENT;
  if ((dx && !aligned(dx, 16)) || (dW && !aligned(dW, 16))) return FLCE_ERR_INVALID_ARGUMENT;
  if (db && !aligned(db, dtype == FLCE_F32 ? 4 : 2)) return FLCE_ERR_INVALID_ARGUMENT;
  if (chunk_tokens < 0 || chunk_tokens % kTile != 0) return FLCE_ERR_INVALID_ARGUMENT;
  const int64_t chunk = chunk_tokens ? chunk_tokens : fused_default_chunk(N, H, V, dtype, b != nullptr);
  const FusedGeometry g = fused_geometry(N, H, V, dtype, b != nullptr, chunk);
  if (workspace_bytes < g.total) return FLCE_ERR_WORKSPACE_TOO_SMALL;
  if (!workspace || !aligned(workspace, 16)) return FLCE_ERR_INVALID_ARGUMENT;
  const bool want_db = b != nullptr && db != nullptr;
  const bool grads = dx || dW || want_db;
  const int64_t es = dtype == FLCE_F32 ? 4 : 2;
  const bool none = reduction == FLCE_REDUCTION_NONE;
  char* ws = (char*)workspace;
  float* gscale = dtype == FLCE_F16 ? (float*)(ws + g.off_gscale) : nullptr;

  flce::FwdLaunch base{};
  base.W = W; base.b = b;
  base.H = (int)H; base.V = (int)V; base.VT = g.VT;
  base.ignore_index = ignore_index;
  base.eps = label_smoothing;
  base.eps_over_v = (float)((double)label_smoothing / (double)V);
  base.s = z_loss_scale;
  base.reduction = reduction;
  base.logit_scale = o.logit_scale;
  base.n_valid = n_valid;
  (void)hipGetLastError();
  flce::mark_launch(stream, nullptr);
  // The mean's count is needed by the first chunk's dlogits.
  flce::FwdLaunch cnt = base;
  cnt.targets = targets;
  cnt.N = (int)N;
  if (grads && flce::launch_fused_count(cnt, stream) != hipSuccess) return FLCE_ERR_HIP;
  for (int64_t c0 = 0; c0 < N; c0 += g.chunk) {
    const int nc = (int)((N - c0) < g.chunk ? (N - c0) : g.chunk);
    const int NTc = (int)cdiv(nc, kTile);
    const bool first = c0 == 0, last = c0 + nc >= N;
    flce::FwdLaunch fa = base;
    fa.x = (const char*)x + c0 * H * es;
    fa.targets = targets + c0;
    fa.N = nc;
    fa.NT = NTc;
    fa.P = fwd_phases(NTc, g.VT);
    fa.partials = ws + g.off_partials;
    fa.rowloss = (float*)(ws + g.off_rowloss) + c0;
    fa.rowzl = (float*)(ws + g.off_rowzl) + c0;
    fa.zloss = o.z_loss ? (none ? o.z_loss + c0 : o.z_loss) : nullptr;
    fa.loss = none ? loss + c0 : loss;
    fa.lse = lse + c0;
    fa.ebuf = ws + g.off_e;
    fa.lde = g.lde;
    fa.mref = (float*)(ws + g.off_mref);
    if (flce::launch_fused_forward(fa, dtype, stream) != hipSuccess) return FLCE_ERR_HIP;
    if (!grads) continue;
    flce::BwdLaunch ba{};
    ba.x = fa.x; ba.W = W; ba.b = b; ba.targets = targets + c0;
    ba.N = nc; ba.H = (int)H; ba.V = (int)V; ba.NT = NTc;
    ba.ignore_index = ignore_index;
    ba.eps = label_smoothing;
    ba.eps_over_v = base.eps_over_v;
    ba.s = z_loss_scale;
    ba.logit_scale = o.logit_scale;
    ba.reduction = reduction;
    ba.accumulate = o.accumulate != 0;
    ba.lse = lse + c0; ba.n_valid = n_valid;
    ba.grad = none ? grad_loss + c0 : grad_loss;
    ba.coef = ws + g.off_coef;
    ba.yv = (int*)(ws + g.off_yv);
    ba.slab = ws + g.off_e;
    ba.ldS = g.lde;
    ba.dx_acc = (float*)(ws + g.off_dxacc);
    ba.dx_split = dx_split(nc, H, g.lde);
    ba.gscale = gscale;
    ba.dx = dx ? (char*)dx + c0 * H * es : nullptr;
    ba.dW = dW;
    ba.db = nullptr;
    if (flce::launch_bwd_prepare(ba, stream) != hipSuccess) return FLCE_ERR_HIP;
    flce::FusedDz fd{};
    fd.ebuf = ws + g.off_e; fd.lde = g.lde;
    fd.mref = (const float*)(ws + g.off_mref);
    fd.coef = ba.coef; fd.yv = ba.yv;
    fd.N = nc; fd.V = (int)V; fd.VT = g.VT;
    fd.dbp = want_db ? (float*)(ws + g.off_dbp) : nullptr;
    fd.gscale = gscale;
    if (flce::launch_fused_dz(fd, dtype, stream) != hipSuccess) return FLCE_ERR_HIP;
    if (want_db && flce::launch_fused_db(fd.dbp, NTc, g.lde, (float*)(ws + g.off_dbacc), (int)V, first, last, db,
                                         dtype, o.accumulate != 0, stream) != hipSuccess)
      return FLCE_ERR_HIP;
    if ((dx || dW) && flce::launch_fused_products(ba, dtype, first, stream) != hipSuccess) return FLCE_ERR_HIP;
  }
  flce::FwdLaunch fin = base;
  fin.targets = targets;
  fin.N = (int)N;
  fin.rowloss = (float*)(ws + g.off_rowloss);
  fin.rowzl = (float*)(ws + g.off_rowzl);
  fin.zloss = o.z_loss;
  fin.loss = loss;
  if (flce::launch_finalize(fin, stream) != hipSuccess) return FLCE_ERR_HIP;
  return FLCE_OK;
}

flce_status flce_shard_workspace_size(int64_t N, int64_t H, int64_t V_shard, flce_dtype dtype, int has_bias,
                                      size_t* fwd_bytes, size_t* merge_bytes, size_t* bwd_bytes) {
  flce_status st = check_shape(N, H, V_shard, dtype);
  if (st != FLCE_OK) return st;
  const Geometry g = geometry(N, H, V_shard, dtype, has_bias, false);
  if (fwd_bytes) *fwd_bytes = g.fwd_total;
  if (merge_bytes) *merge_bytes = align_up((size_t)N * 4);
  if (bwd_bytes) *bwd_bytes = g.bwd_total;
  return FLCE_OK;
}

flce_status flce_shard_forward(const void* x, const void* W_shard, const void* b_shard, const int64_t* targets,
                               int64_t N, int64_t H, int64_t V_shard, int64_t vocab_start, int64_t V_total,
                               flce_dtype dtype, float label_smoothing, int64_t ignore_index, float* stats,
                               void* workspace, size_t workspace_bytes, hipStream_t stream) {
  flce_status st = check_shape(N, H, V_shard, dtype);
  if (st != FLCE_OK) return st;
  if ((st = check_shard(V_shard, vocab_start, V_total)) != FLCE_OK) return st;
  if ((st = check_options(label_smoothing, 0.f, FLCE_REDUCTION_MEAN)) != FLCE_OK) return st;
  if ((st = check_inputs(x, W_shard, b_shard, targets, dtype)) != FLCE_OK) return st;
  if (!stats || !aligned(stats, 16)) return FLCE_ERR_INVALID_ARGUMENT;
  const Geometry g = geometry(N, H, V_shard, dtype, b_shard != nullptr, false);
  if (workspace_bytes < g.fwd_total) return FLCE_ERR_WORKSPACE_TOO_SMALL;
  if (!workspace || !aligned(workspace, 16)) return FLCE_ERR_INVALID_ARGUMENT;

  char* ws = (char*)workspace;
  flce::FwdLaunch a{};
  a.x = x; a.W = W_shard; a.b = b_shard; a.targets = targets;
  a.N = (int)N; a.H = (int)H; a.V = (int)V_shard;
  a.NT = g.NT; a.P = g.P; a.VT = g.VT;
  a.vocab_start = vocab_start;
  a.ignore_index = ignore_index;
  a.eps = label_smoothing;
  a.logit_scale = 1.f;
  a.partials = ws + g.off_partials;
  a.stats = stats;
  (void)hipGetLastError();
  flce::mark_launch((hipStream_t)stream, nullptr);
  if (flce::launch_shard_forward(a, dtype, (hipStream_t)stream) != hipSuccess) return FLCE_ERR_HIP;
  return FLCE_OK;
}

flce_status flce_shard_merge(const float* stats, int64_t num_shards, const int64_t* targets, int64_t N,
                             int64_t V_total, float label_smoothing, float z_loss_scale, int64_t ignore_index,
                             flce_reduction reduction, float* loss, float* lse, int64_t* n_valid, void* workspace,
                             size_t workspace_bytes, hipStream_t stream) {
  if (N < 1 || N > (int64_t(1) << 30) || V_total < 1 || V_total > (int64_t(1) << 30)) return FLCE_ERR_INVALID_ARGUMENT;
  if (num_shards < 1 || num_shards > (int64_t(1) << 20)) return FLCE_ERR_INVALID_ARGUMENT;
  flce_status st = check_options(label_smoothing, z_loss_scale, reduction);
  if (st != FLCE_OK) return st;
  if (!stats || !aligned(stats, 16) || !targets || !aligned(targets, 8)) return FLCE_ERR_INVALID_ARGUMENT;
  if (!loss || !lse || !n_valid || !aligned(loss, 4) || !aligned(lse, 4) || !aligned(n_valid, 8))
    return FLCE_ERR_INVALID_ARGUMENT;
  if (workspace_bytes < align_up((size_t)N * 4)) return FLCE_ERR_WORKSPACE_TOO_SMALL;
  if (!workspace || !aligned(workspace, 16)) return FLCE_ERR_INVALID_ARGUMENT;

  flce::FwdLaunch a{};
  a.targets = targets;
  a.N = (int)N;
  a.P = (int)num_shards;
  a.ignore_index = ignore_index;
  a.eps = label_smoothing;
  a.eps_over_v = (float)((double)label_smoothing / (double)V_total);
  a.s = z_loss_scale;
  a.logit_scale = 1.f;
  a.reduction = reduction;
  a.partials = const_cast<float*>(stats);
  a.rowloss = (float*)workspace;
  a.loss = loss; a.lse = lse; a.n_valid = n_valid;
  (void)hipGetLastError();
  flce::mark_launch((hipStream_t)stream, nullptr);
  if (flce::launch_merge(a, (hipStream_t)stream) != hipSuccess) return FLCE_ERR_HIP;
  return FLCE_OK;
}

flce_status flce_shard_backward(const void* x, const void* W_shard, const void* b_shard, const int64_t* targets,
                                int64_t N, int64_t H, int64_t V_shard, int64_t vocab_start, int64_t V_total,
                                flce_dtype dtype, float label_smoothing, float z_loss_scale, int64_t ignore_index,
                                flce_reduction reduction, const float* lse, const int64_t* n_valid, const float* grad_loss,
                                float* dx_partial, int accumulate_dx, void* dW_shard, void* db_shard,
                                void* workspace, size_t workspace_bytes, hipStream_t stream) {
  flce_status st = check_shape(N, H, V_shard, dtype);
  if (st != FLCE_OK) return st;
  if ((st = check_shard(V_shard, vocab_start, V_total)) != FLCE_OK) return st;
  if ((st = check_options(label_smoothing, z_loss_scale, reduction)) != FLCE_OK) return st;
  if ((st = check_inputs(x, W_shard, b_shard, targets, dtype)) != FLCE_OK) return st;
  if (!lse || !n_valid || !grad_loss) return FLCE_ERR_INVALID_ARGUMENT;
  if (!aligned(lse, 4) || !aligned(n_valid, 8) || !aligned(grad_loss, 4)) return FLCE_ERR_INVALID_ARGUMENT;
  if ((dx_partial && !aligned(dx_partial, 16)) || (dW_shard && !aligned(dW_shard, 16))) return FLCE_ERR_INVALID_ARGUMENT;
  if (db_shard && !aligned(db_shard, dtype == FLCE_F32 ? 4 : 2)) return FLCE_ERR_INVALID_ARGUMENT;
  const Geometry g = geometry(N, H, V_shard, dtype, b_shard != nullptr, false);
  if (workspace_bytes < g.bwd_total) return FLCE_ERR_WORKSPACE_TOO_SMALL;
  if (!workspace || !aligned(workspace, 16)) return FLCE_ERR_INVALID_ARGUMENT;
  const bool want_db = b_shard != nullptr && db_shard != nullptr;
  if (!dx_partial && !dW_shard && !want_db) return FLCE_OK;

  char* ws = (char*)workspace;
  flce::BwdLaunch a{};
  a.x = x; a.W = W_shard; a.b = b_shard; a.targets = targets;
  a.N = (int)N; a.H = (int)H; a.V = (int)V_shard;
  a.NT = g.NT;
  a.vocab_start = vocab_start;
  a.ignore_index = ignore_index;
  a.eps = label_smoothing;
  a.eps_over_v = (float)((double)label_smoothing / (double)V_total);
  a.s = z_loss_scale;
  a.logit_scale = 1.f;
  a.reduction = reduction;
  a.lse = lse; a.n_valid = n_valid; a.grad = grad_loss;
  a.coef = ws + g.off_coef;
  a.yv = (int*)(ws + g.off_yv);
  a.slab = ws + g.off_slab;
  a.ldS = g.slab_cols;
  a.dx_acc = dx_partial;
  a.dbp = want_db ? (float*)(ws + g.off_dbp) : nullptr;
  a.gscale = dtype == FLCE_F16 ? (float*)(ws + g.off_gscale) : nullptr;
  a.dx = dx_partial; a.dW = dW_shard; a.db = want_db ? db_shard : nullptr;
  return run_backward(a, g, V_shard, dtype, want_db, true, accumulate_dx != 0, (hipStream_t)stream);
}

}  // extern "C"

// ---------------------------------------------------------------------------
// Linear layer and gated product
// ---------------------------------------------------------------------------

namespace {

// How a product of M x N outputs over K is cut: output tiles of 32 S x 32 S
// (S = 8, 16-bit only; 4; 2) and parts of K.
struct Cut {
  int S, parts;
  double ns;
};

// Depth of a part: the 64-deep copy block divides it, so every part starts on
// a block.
int64_t part_depth(int64_t K, int64_t parts) { return parts > 1 ? cdiv(cdiv(K, parts), 64) * 64 : K; }

// The cut with the least estimated time, in ns, of the busiest CU's q tiles:
//   q * per_tile + K * max(alone, q * shared) + fixed,
// `alone` a tile's time per K when nothing else is on its CU (the latency of
// its loop) and `shared` what a tile costs a full CU.  A split adds a launch and
// the fp32 partial sums' way out and back.  Fitted to bf16 and fp32 runs of 16
// shapes from 100 x 64 x 64 to 517 x 20480 x 4096 at each S (no bias, no
// activation): within a fifth of most, and it picks the fastest or one within
// 15% of it.  Some of them, us at S = 8 / 4 / 2: 300 x 700 x 500 20.4 / 8.4 / 5.0,
// 1024 x 4096 x 1024 23.5 / 16.3 / 10.8, 2048 x 4096 x 1024 35.6 / 17.4 / 24.1,
// 4096 x 4096 x 4096 90 / 120 / 175; fp32 at S = 4 / 2: 100 x 64 x 64 3.9 / 1.3,
// 300 x 700 x 500 16.8 / 11.3, 4096 x 4096 x 1024 167 / 218.
struct TileCost {
  int S;
  double alone, shared, per_tile, fixed;
};
constexpr TileCost kCost16[] = {{8, 20.0, 20.0, 7000.0, 0.0}, {4, 10.5, 7.3, 500.0, 1000.0}, {2, 8.0, 2.7, 200.0, 800.0}};
constexpr TileCost kCost32[] = {{4, 55.0, 41.0, 700.0, 2500.0}, {2, 24.0, 15.0, 200.0, 1000.0}};
constexpr double kJoinNs = 1500.0, kJoinNsPerByte = 0.235e-3;

// FLCE_DEBUG_LAYER_TILE: the tests run every S (2, 4, 8) on every shape with it,
// and 1 the few-token kernel wherever it fits.
int forced_tile() {
  const char* env = std::getenv("FLCE_DEBUG_LAYER_TILE");
  return env ? std::atoi(env) : 0;
}

// only: the S to use (0: any).
Cut product_cut(int64_t M, int64_t N, int64_t K, int dtype, int only = 0) {
  Cut best{only ? only : 2, 1, 1e300};
  if (M < 1 || N < 1) return best;
  const int forced = forced_tile();
  double least = 0.0;
  auto consider = [&](const TileCost& t) {
    if ((forced == 2 || forced == 4 || (forced == 8 && dtype != FLCE_F32)) && t.S != forced) return;
    const int64_t tiles = cdiv(M, 32 * t.S) * cdiv(N, 32 * t.S);
    for (int64_t parts : {1, 2, 3, 4, 6, 8, 12, 16}) {
      if (t.S == 2 && tiles * parts >= (int64_t(1) << 23)) return;   // a launch has fewer than 2^32 threads
      const int64_t kc = part_depth(K, parts);
      if (parts > 1 && (kc < 256 || cdiv(K, kc) != parts)) continue;
      const double q = (double)cdiv(tiles * parts, kCUs);
      const double loop = (double)kc * (t.S == 8 ? q * t.shared : std::max(t.alone, q * t.shared));
      double ns = t.fixed + q * t.per_tile + loop;
      if (parts > 1) ns += kJoinNs + kJoinNsPerByte * 4.0 * (double)parts * (double)M * (double)N;
      if (least == 0.0 || ns < least) {
        least = ns;
        best = {t.S, (int)parts, ns};
      }
    }
  };
  if (dtype == FLCE_F32) {
    for (const TileCost& t : kCost32) consider(t);
  } else {
    for (const TileCost& t : kCost16) consider(t);
  }
  return best;
}

struct LayerGeometry {
  int64_t Hp;          // H rounded up to 8: the width of the rows that the kernels read
  size_t pad_bytes;    // padded copies of x and the weights (none when Hp == H), first in both workspaces
  int fwd_tile, TM, TN, fwd_parts;
  int64_t kc, ldp;
  size_t fwd_total;
  bool dz_is_dy;
  int64_t ldz, segk;
  int db_blocks, db_rows;
  int64_t ldb;
  int dx_tile, dx_parts, dw_tile, dw_parts;
  int64_t dx_kc, dw_kc;
  size_t off_dbp, off_part, off_dw_part, bwd_total;
};

LayerGeometry layer_geometry(int64_t N, int64_t Hout, int64_t F, int dtype, int act, int nmat) {
  LayerGeometry g{};
  const int64_t es = dtype == FLCE_F32 ? 4 : 2;
  const int64_t H = cdiv(Hout, 8) * 8;
  g.Hp = H;
  g.pad_bytes = H == Hout ? 0 : align_up((size_t)(N + nmat * F) * H * es);
  Cut fwd = product_cut(N, nmat * F, H, dtype);
  const int forced = forced_tile();
  if (forced == 1 ? N <= flce::kSkinnyMost : forced == 0 && N <= flce::skinny_tokens(dtype)) fwd = {0, 1, 0.0};
  g.fwd_tile = fwd.S;
  g.TM = fwd.S ? (int)cdiv(N, 32 * fwd.S) : 0;
  g.TN = fwd.S ? (int)cdiv(F, 32 * fwd.S / nmat) : 0;
  g.fwd_parts = fwd.parts;
  g.kc = part_depth(H, g.fwd_parts);
  g.ldp = nmat * cdiv(F, 8) * 8;
  g.fwd_total = g.pad_bytes + (g.fwd_parts > 1 ? align_up((size_t)g.fwd_parts * N * g.ldp * 4) : 0);

  // dz: rows padded to 16-byte pieces; the gated product's two halves each to
  // a whole 64-deep copy block, so that no block of the dx product straddles
  // the weights.
  g.dz_is_dy = nmat == 1 && act == FLCE_ACT_NONE && F % 8 == 0;
  g.segk = nmat == 2 ? cdiv(F, 64) * 64 : int64_t(1) << 30;
  g.ldz = nmat == 2 ? 2 * g.segk : cdiv(F, 8) * 8;
  size_t off = g.pad_bytes + (g.dz_is_dy ? 0 : align_up((size_t)N * g.ldz * es));
  // Column sums, and dz with them: at most 64 blocks of tokens, 16 tokens each at
  // least (gated, N=1037, F=2731: 11.8 us in 44 blocks of 24, 19.5 in 17 of 64).
  g.db_rows = (int)(cdiv(cdiv(N, 64), 8) * 8);
  if (g.db_rows < 16) g.db_rows = 16;
  g.db_blocks = (int)cdiv(N, g.db_rows);
  g.ldb = nmat * F;
  g.off_dbp = off;
  off = align_up(off + (size_t)g.db_blocks * g.ldb * 4);
  // Two small products share a launch, and with it their tiles' size.
  Cut cx = product_cut(H, N, g.ldz, dtype), cw = product_cut(H, nmat * F, N, dtype);
  if (cx.S < 8 && cw.S < 8 && cx.S != cw.S) {
    const Cut x4 = product_cut(H, N, g.ldz, dtype, 4), w4 = product_cut(H, nmat * F, N, dtype, 4);
    const Cut x2 = product_cut(H, N, g.ldz, dtype, 2), w2 = product_cut(H, nmat * F, N, dtype, 2);
    const bool two = x2.ns + w2.ns < x4.ns + w4.ns;
    cx = two ? x2 : x4;
    cw = two ? w2 : w4;
  }
  g.dx_tile = cx.S;
  g.dx_parts = cx.parts;
  g.dw_tile = cw.S;
  g.dw_parts = cw.parts;
  g.dx_kc = part_depth(g.ldz, g.dx_parts);
  g.dw_kc = part_depth(N, g.dw_parts);
  g.off_part = off;
  off = align_up(off + (g.dx_parts > 1 ? (size_t)g.dx_parts * N * Hout * 4 : 0));
  g.off_dw_part = off;
  g.bwd_total = align_up(off + (g.dw_parts > 1 ? (size_t)g.dw_parts * nmat * F * Hout * 4 : 0));
  return g;
}

flce_status check_layer(int64_t N, int64_t H, int64_t F, int dtype, int act, int nmat) {
  if (N < 0 || H < 1 || F < 1) return FLCE_ERR_INVALID_ARGUMENT;
  if (act < FLCE_ACT_NONE || act > FLCE_ACT_SIGMOID) return FLCE_ERR_INVALID_ARGUMENT;
  if (dtype != FLCE_F32 && dtype != FLCE_BF16 && dtype != FLCE_F16) return FLCE_ERR_UNSUPPORTED;
  if (N > (int64_t(1) << 30) || H > (int64_t(1) << 20) || F > (int64_t(1) << (nmat == 2 ? 19 : 20)))
    return FLCE_ERR_UNSUPPORTED;
  const int64_t wide = H > F ? H : F;   // every plane of output tiles fits in an int
  if (cdiv(N, 64) * cdiv(wide, 32) > (int64_t(1) << 27) || cdiv(F, 32) * cdiv(H, 64) > (int64_t(1) << 27))
    return FLCE_ERR_UNSUPPORTED;
  return FLCE_OK;
}

bool bad_tensor(const void* p, size_t align, bool required) { return p ? !aligned(p, align) : required; }

// x and the weights as the kernels read them: themselves, or padded copies in
// the workspace.
bool pad_rows(const LayerGeometry& g, const void* x, const void* const (&W)[2], int64_t N, int64_t H, int64_t F, int dtype,
              int nmat, char* ws, hipStream_t stream, const void*& xo, const void* (&Wo)[2]) {
  xo = x;
  for (int m = 0; m < nmat; ++m) Wo[m] = W[m];
  if (g.Hp == H) return true;
  const int64_t row = g.Hp * (dtype == FLCE_F32 ? 4 : 2);
  const flce::LayerPad p{{x, W[0], W[1]}, {N, F, nmat == 2 ? F : 0}, (int)H, (int)g.Hp, ws};
  xo = ws;
  for (int m = 0; m < nmat; ++m) Wo[m] = ws + (N + m * F) * row;
  return flce::launch_layer_pad(p, dtype, stream) == hipSuccess;
}

// The entry points' shared parts: nmat = 1 is the linear layer, 2 the gated product.
flce_status layer_forward(const void* x, const void* const (&W)[2], const void* const (&b)[2], const void* residual,
                          int64_t N, int64_t H, int64_t F, int dtype, int act, int nmat, void* y, float* const (&z)[2],
                          void* workspace, size_t workspace_bytes, hipStream_t stream) {
  const flce_status st = check_layer(N, H, F, dtype, act, nmat);
  if (st != FLCE_OK) return st;
  const size_t es = dtype == FLCE_F32 ? 4 : 2;
  const bool rows = N > 0;   // without rows the token tensors may be null
  if (bad_tensor(x, 16, rows) || bad_tensor(y, 16, rows) || bad_tensor(residual, 16, false)) return FLCE_ERR_INVALID_ARGUMENT;
  for (int m = 0; m < nmat; ++m)
    if (bad_tensor(W[m], 16, true) || bad_tensor(b[m], es, false) || bad_tensor(z[m], 16, false))
      return FLCE_ERR_INVALID_ARGUMENT;
  if (nmat == 2 && (z[0] == nullptr) != (z[1] == nullptr)) return FLCE_ERR_INVALID_ARGUMENT;
  const LayerGeometry g = layer_geometry(N, H, F, dtype, act, nmat);
  if (workspace_bytes < g.fwd_total) return FLCE_ERR_WORKSPACE_TOO_SMALL;
  if (bad_tensor(workspace, 16, g.fwd_total > 0)) return FLCE_ERR_INVALID_ARGUMENT;
  if (!rows) return FLCE_OK;
  char* ws = (char*)workspace;
  flce::LayerFwd a{};
  (void)hipGetLastError();
  flce::mark_launch(stream, nullptr);
  if (!pad_rows(g, x, W, N, H, F, dtype, nmat, ws, stream, a.x, a.W)) return FLCE_ERR_HIP;
  for (int m = 0; m < nmat; ++m) {
    a.b[m] = b[m];
    a.z[m] = z[m];
  }
  a.residual = residual;
  a.y = y;
  a.N = (int)N; a.H = (int)g.Hp; a.F = (int)F;
  a.act = act; a.nmat = nmat;
  a.tile = g.fwd_tile; a.TM = g.TM; a.TN = g.TN;
  a.parts = g.fwd_parts; a.kc = (int)g.kc;
  a.part = (float*)(ws + g.pad_bytes); a.ldp = g.ldp;
  return flce::launch_layer_forward(a, dtype, stream) == hipSuccess ? FLCE_OK : FLCE_ERR_HIP;
}

flce_status layer_backward(const void* x, const void* const (&W)[2], const float* const (&z)[2], const void* dy,
                           int64_t N, int64_t H, int64_t F, int dtype, int act, int nmat, void* dx,
                           void* const (&dW)[2], void* const (&db)[2], void* workspace, size_t workspace_bytes,
                           hipStream_t stream) {
  const flce_status st = check_layer(N, H, F, dtype, act, nmat);
  if (st != FLCE_OK) return st;
  const size_t es = dtype == FLCE_F32 ? 4 : 2;
  const bool rows = N > 0;
  const bool need_z = rows && (nmat == 2 || act != FLCE_ACT_NONE);
  if (bad_tensor(x, 16, rows) || bad_tensor(dy, 16, rows) || bad_tensor(dx, 16, false)) return FLCE_ERR_INVALID_ARGUMENT;
  for (int m = 0; m < nmat; ++m)
    if (bad_tensor(W[m], 16, true) || bad_tensor(z[m], 16, need_z) || bad_tensor(dW[m], 16, false) ||
        bad_tensor(db[m], es, false))
      return FLCE_ERR_INVALID_ARGUMENT;
  const LayerGeometry g = layer_geometry(N, H, F, dtype, act, nmat);
  if (workspace_bytes < g.bwd_total) return FLCE_ERR_WORKSPACE_TOO_SMALL;
  if (bad_tensor(workspace, 16, g.bwd_total > 0)) return FLCE_ERR_INVALID_ARGUMENT;
  const bool want_db = db[0] || db[1];
  if (!dx && !dW[0] && !dW[1] && !want_db) return FLCE_OK;
  char* ws = (char*)workspace;
  flce::LayerBwd a{};
  (void)hipGetLastError();
  flce::mark_launch(stream, nullptr);
  if (!pad_rows(g, x, W, N, H, F, dtype, nmat, ws, stream, a.x, a.W)) return FLCE_ERR_HIP;
  a.dy = dy;
  for (int m = 0; m < nmat; ++m) {
    a.z[m] = z[m];
    a.dW[m] = dW[m];
    a.db[m] = db[m];
  }
  a.N = (int)N; a.H = (int)g.Hp; a.F = (int)F;
  a.Hout = (int)H;
  a.act = act; a.nmat = nmat;
  a.dz_is_dy = g.dz_is_dy;
  a.dz = g.dz_is_dy ? const_cast<void*>(dy) : ws + g.pad_bytes;
  a.ldz = g.ldz; a.segk = (int)g.segk;
  a.dbp = want_db ? (float*)(ws + g.off_dbp) : nullptr;
  a.ldb = g.ldb; a.db_blocks = g.db_blocks; a.db_rows = g.db_rows;
  a.dx = dx; a.dx_tile = g.dx_tile; a.dx_parts = g.dx_parts; a.dx_kc = (int)g.dx_kc;
  a.dw_tile = g.dw_tile; a.dw_parts = g.dw_parts; a.dw_kc = (int)g.dw_kc;
  a.dx_part = (float*)(ws + g.off_part);
  a.dw_part = (float*)(ws + g.off_dw_part);
  return flce::launch_layer_backward(a, dtype, stream) == hipSuccess ? FLCE_OK : FLCE_ERR_HIP;
}

// ---------------------------------------------------------------------------
// Gradient norm and clipping
// ---------------------------------------------------------------------------

// Workgroups over all launches of one call (each launch has at least one): 4
// per CU, all resident at once, keep enough loads in flight, and the partials
// stay few enough for every workgroup of the clipping pass to add them up.
constexpr int64_t kNormBlocks = 4 * kCUs;

// Past this many gradient bytes the norm's loads leave nothing in the 256 MB
// memory-side cache.  Below, the clipping pass finds there what the norm has read;
// above, little of it is left by then, and making room for it costs more.  bf16,
// norm + clipping pass, us, keeping / not: 128 MB 52 + 41 / 24 + 79, 192 MB 74 + 70
// / 32 + 104, 1 GB 232 + 382 / 156 + 435.
constexpr double kNormStreamBytes = 160.0 * (1 << 20);

double norm_bytes_read(const int64_t* numels, const flce_dtype* dtypes, int64_t count) {
  double bytes = 0.0;
  for (int64_t i = 0; i < count; ++i) bytes += (double)numels[i] * (dtypes[i] == FLCE_F32 ? 4.0 : 2.0);
  return bytes;
}

// Bytes of a chunk: about 8 chunks a workgroup balance them, but 16 KB where
// that still makes one each (four 16-byte loads of each thread in flight); 4 KB
// at least, 256 KB at most.
int64_t norm_chunk_bytes(double bytes) {
  int64_t chunk = 4096;
  while (chunk < (int64_t(1) << 18) &&
         bytes > (double)chunk * (chunk < 16384 ? 1.0 : 8.0) * (double)kNormBlocks)
    chunk *= 2;
  return chunk;
}

// A tensor's chunks of work: whole chunks counted from its first 16-byte boundary.
int64_t norm_chunks(const void* p, int64_t n, int64_t es, int64_t chunk) {
  if (n == 0) return 0;
  int64_t head = (int64_t)((16 - ((uintptr_t)p & 15)) & 15) / es;
  if (head > n) head = n;
  const int64_t c = cdiv(n - head, chunk / es);
  return c > 0 ? c : 1;
}

int64_t norm_launches(int64_t count) { return cdiv(count, flce::kNormTensors); }

int64_t dtype_bytes(int dtype) { return dtype == FLCE_F32 ? 4 : 2; }

flce_status check_norm(const void* const* grads, const int64_t* numels, const flce_dtype* dtypes, int64_t count) {
  if (count < 0 || count > (int64_t(1) << 20)) return FLCE_ERR_INVALID_ARGUMENT;
  if (count > 0 && (!grads || !numels || !dtypes)) return FLCE_ERR_INVALID_ARGUMENT;
  for (int64_t i = 0; i < count; ++i) {
    if (dtypes[i] != FLCE_F32 && dtypes[i] != FLCE_BF16 && dtypes[i] != FLCE_F16) return FLCE_ERR_UNSUPPORTED;
    if (numels[i] < 0 || numels[i] > (int64_t(1) << 40)) return FLCE_ERR_INVALID_ARGUMENT;
    if (numels[i] > 0 && (!grads[i] || !aligned(grads[i], dtype_bytes(dtypes[i])))) return FLCE_ERR_INVALID_ARGUMENT;
  }
  return FLCE_OK;
}

// No byte that clipping writes may belong to another tensor, read or written:
// workgroups of both would race.  (A tensor's out may be its own gradient.)
flce_status check_disjoint(const void* const* grads, void* const* outs, const int64_t* numels, const flce_dtype* dtypes,
                           int64_t count) {
  struct Range {
    uintptr_t lo, hi;
    bool written;
  };
  std::vector<Range> r;
  r.reserve(outs ? 2 * count : count);
  for (int64_t i = 0; i < count; ++i) {
    if (numels[i] == 0) continue;
    const uintptr_t bytes = (uintptr_t)(numels[i] * dtype_bytes(dtypes[i]));
    const uintptr_t in = (uintptr_t)grads[i], out = outs ? (uintptr_t)outs[i] : in;
    if (outs && (!outs[i] || !aligned(outs[i], dtype_bytes(dtypes[i])))) return FLCE_ERR_INVALID_ARGUMENT;
    if (out != in) r.push_back({in, in + bytes, false});
    r.push_back({out, out + bytes, true});
  }
  std::sort(r.begin(), r.end(), [](const Range& a, const Range& b) { return a.lo < b.lo; });
  uintptr_t end = 0, wend = 0;   // furthest end of all ranges so far, and of the written ones
  for (const Range& v : r) {
    if (v.lo < (v.written ? end : wend)) return FLCE_ERR_INVALID_ARGUMENT;
    end = std::max(end, v.hi);
    if (v.written) wend = std::max(wend, v.hi);
  }
  return FLCE_OK;
}

// Launch table l of a call: tensors [l * kNormTensors, ...).  Returns its chunks.
int64_t norm_table(flce::NormTable& t, const void* const* grads, void* const* outs, const int64_t* numels,
                   const flce_dtype* dtypes, int64_t count, int64_t l, int64_t chunk) {
  t.chunk_bytes = (int)chunk;
  const int64_t i0 = l * flce::kNormTensors;
  t.count = (int)std::min<int64_t>(flce::kNormTensors, count - i0);
  t.in_place = 1;
  int64_t end = 0;
  for (int k = 0; k < t.count; ++k) {
    const int64_t i = i0 + k;
    t.in[k] = grads[i];
    t.out[k] = outs ? outs[i] : const_cast<void*>(grads[i]);
    if (t.out[k] != t.in[k] && numels[i] > 0) t.in_place = 0;
    t.n[k] = numels[i];
    t.dtype[k] = (uint8_t)dtypes[i];
    end += norm_chunks(grads[i], numels[i], dtype_bytes(dtypes[i]), chunk);
    t.end[k] = end;
  }
  return end;
}

// norm_out and the scaled gradients.  grads without out and clip = false: the norm alone.
// given: the norm to scale by.
flce_status run_grad_norm(const void* const* grads, void* const* outs, const int64_t* numels, const flce_dtype* dtypes,
                          int64_t count, float max_norm, bool inf_norm, const float* given, bool clip, float* norm_out,
                          double* part, hipStream_t stream) {
  const int64_t launches = norm_launches(count);
  const double bytes = norm_bytes_read(numels, dtypes, count);
  const int64_t chunk = norm_chunk_bytes(bytes);
  int64_t total = 0;
  for (int64_t i = 0; i < count; ++i) total += norm_chunks(grads[i], numels[i], dtype_bytes(dtypes[i]), chunk);
  auto blocks_of = [&](int64_t chunks) -> int {   // this launch's share of the workgroups
    if (total <= kNormBlocks) return (int)std::max<int64_t>(1, chunks);
    return (int)std::max<int64_t>(1, (int64_t)((double)kNormBlocks * (double)chunks / (double)total));
  };
  (void)hipGetLastError();
  flce::mark_launch(stream, nullptr);
  flce::NormTable t;
  int parts = 0;
  if (!given) {
    for (int64_t l = 0; l < launches; ++l) {
      const int blocks = blocks_of(norm_table(t, grads, outs, numels, dtypes, count, l, chunk));
      if (flce::launch_grad_norm(t, inf_norm, bytes > kNormStreamBytes, part + parts, blocks, stream) != hipSuccess) return FLCE_ERR_HIP;
      parts += blocks;
    }
  }
  if (!clip || launches == 0) {   // the norm alone
    t.count = 0;
    t.in_place = 1;
    if (!norm_out) return FLCE_OK;
    return flce::launch_grad_clip(t, inf_norm, part, parts, given, norm_out, max_norm, 1, stream) == hipSuccess
               ? FLCE_OK : FLCE_ERR_HIP;
  }
  for (int64_t l = 0; l < launches; ++l) {
    const int blocks = blocks_of(norm_table(t, grads, outs, numels, dtypes, count, l, chunk));
    if (flce::launch_grad_clip(t, inf_norm, part, parts, given, l == 0 ? norm_out : nullptr, max_norm, blocks, stream) !=
        hipSuccess)
      return FLCE_ERR_HIP;
  }
  return FLCE_OK;
}

size_t norm_bytes(int64_t count) { return align_up((size_t)(kNormBlocks + norm_launches(count)) * sizeof(double)); }

// Host memory for the overlap check is the one thing a call may fail to get.
flce_status grad_norm_call(const void* const* grads, void* const* outs, const int64_t* numels, const flce_dtype* dtypes,
                           int64_t count, float max_norm, float norm_type, const float* given, bool clip, float* norm_out,
                           void* workspace, size_t workspace_bytes, hipStream_t stream) noexcept {
  const flce_status st = check_norm(grads, numels, dtypes, count);
  if (st != FLCE_OK) return st;
  const bool inf_norm = std::isinf(norm_type) && norm_type > 0.f;
  if (!inf_norm && norm_type != 2.f) return FLCE_ERR_UNSUPPORTED;
  if (clip && !(max_norm >= 0.f)) return FLCE_ERR_INVALID_ARGUMENT;
  if (bad_tensor(norm_out, 4, !given) || bad_tensor(given, 4, false)) return FLCE_ERR_INVALID_ARGUMENT;
  if (!given) {
    if (workspace_bytes < norm_bytes(count)) return FLCE_ERR_WORKSPACE_TOO_SMALL;
    if (bad_tensor(workspace, 16, true)) return FLCE_ERR_INVALID_ARGUMENT;
  }
  if (clip) {
    try {
      const flce_status so = check_disjoint(grads, outs, numels, dtypes, count);
      if (so != FLCE_OK) return so;
    } catch (...) {
      return FLCE_ERR_HIP;
    }
  }
  return run_grad_norm(grads, outs, numels, dtypes, count, max_norm, inf_norm, given, clip, norm_out, (double*)workspace,
                       stream);
}

}  // namespace

extern "C" {

flce_status flce_linear_workspace_size(int64_t N, int64_t H, int64_t F, flce_dtype dtype, flce_activation activation,
                                       size_t* fwd_bytes, size_t* bwd_bytes) {
  const flce_status st = check_layer(N, H, F, dtype, activation, 1);
  if (st != FLCE_OK) return st;
  const LayerGeometry g = layer_geometry(N, H, F, dtype, activation, 1);
  if (fwd_bytes) *fwd_bytes = g.fwd_total;
  if (bwd_bytes) *bwd_bytes = g.bwd_total;
  return FLCE_OK;
}

flce_status flce_linear_forward(const void* x, const void* W, const void* b, const void* residual, int64_t N, int64_t H,
                                int64_t F, flce_dtype dtype, flce_activation activation, void* y, float* z,
                                void* workspace, size_t workspace_bytes, hipStream_t stream) {
  return layer_forward(x, {W, nullptr}, {b, nullptr}, residual, N, H, F, dtype, activation, 1, y, {z, nullptr},
                       workspace, workspace_bytes, stream);
}

flce_status flce_linear_backward(const void* x, const void* W, const float* z, const void* dy, int64_t N, int64_t H,
                                 int64_t F, flce_dtype dtype, flce_activation activation, void* dx, void* dW, void* db,
                                 void* workspace, size_t workspace_bytes, hipStream_t stream) {
  return layer_backward(x, {W, nullptr}, {z, nullptr}, dy, N, H, F, dtype, activation, 1, dx, {dW, nullptr},
                        {db, nullptr}, workspace, workspace_bytes, stream);
}

flce_status flce_glu_workspace_size(int64_t N, int64_t H, int64_t F, flce_dtype dtype, size_t* fwd_bytes,
                                    size_t* bwd_bytes) {
  const flce_status st = check_layer(N, H, F, dtype, FLCE_ACT_NONE, 2);
  if (st != FLCE_OK) return st;
  const LayerGeometry g = layer_geometry(N, H, F, dtype, FLCE_ACT_NONE, 2);
  if (fwd_bytes) *fwd_bytes = g.fwd_total;
  if (bwd_bytes) *bwd_bytes = g.bwd_total;
  return FLCE_OK;
}

flce_status flce_glu_forward(const void* x, const void* Wg, const void* Wu, const void* bg, const void* bu, int64_t N,
                             int64_t H, int64_t F, flce_dtype dtype, flce_activation activation, void* h, float* g,
                             float* u, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  return layer_forward(x, {Wg, Wu}, {bg, bu}, nullptr, N, H, F, dtype, activation, 2, h, {g, u}, workspace,
                       workspace_bytes, stream);
}

flce_status flce_glu_backward(const void* x, const void* Wg, const void* Wu, const float* g, const float* u,
                              const void* dh, int64_t N, int64_t H, int64_t F, flce_dtype dtype,
                              flce_activation activation, void* dx, void* dWg, void* dWu, void* dbg, void* dbu,
                              void* workspace, size_t workspace_bytes, hipStream_t stream) {
  return layer_backward(x, {Wg, Wu}, {g, u}, dh, N, H, F, dtype, activation, 2, dx, {dWg, dWu}, {dbg, dbu}, workspace,
                        workspace_bytes, stream);
}

flce_status flce_grad_norm_workspace_size(int64_t count, size_t* bytes) {
  if (count < 0 || count > (int64_t(1) << 20)) return FLCE_ERR_INVALID_ARGUMENT;
  if (bytes) *bytes = norm_bytes(count);
  return FLCE_OK;
}

flce_status flce_grad_norm(const void* const* grads, const int64_t* numels, const flce_dtype* dtypes, int64_t count,
                           float norm_type, float* norm, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  return grad_norm_call(grads, nullptr, numels, dtypes, count, 0.f, norm_type, nullptr, false, norm, workspace,
                        workspace_bytes, stream);
}

flce_status flce_clip_grad_norm(const void* const* grads, void* const* outs, const int64_t* numels,
                                const flce_dtype* dtypes, int64_t count, float max_norm, float norm_type, float* norm,
                                void* workspace, size_t workspace_bytes, hipStream_t stream) {
  return grad_norm_call(grads, outs, numels, dtypes, count, max_norm, norm_type, nullptr, true, norm, workspace,
                        workspace_bytes, stream);
}

flce_status flce_clip_grads_with_norm(const void* const* grads, void* const* outs, const int64_t* numels,
                                      const flce_dtype* dtypes, int64_t count, float max_norm, const float* norm,
                                      hipStream_t stream) {
  if (!norm) return FLCE_ERR_INVALID_ARGUMENT;
  return grad_norm_call(grads, outs, numels, dtypes, count, max_norm, 2.f, norm, true, nullptr, nullptr, 0, stream);
}

}  // extern "C"
