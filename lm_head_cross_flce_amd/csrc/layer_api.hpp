// Host side of the linear layer and the gated product: argument checks, tile and
// split choice, workspace layout, entry points.  Included once, by flce_api.hip.
#pragma once

namespace {

// A tensor of a call (p null or no bytes: absent).
struct Memory {
  const void* p;
  size_t bytes;
  bool written;
};

// Whether a tensor that the call writes shares a byte with another of them:
// workgroups of both would race.
bool clash(const Memory* m, int count) {
  for (int i = 0; i < count; ++i)
    for (int j = 0; j < i; ++j) {
      if (!m[i].p || !m[j].p || !m[i].bytes || !m[j].bytes || !(m[i].written || m[j].written)) continue;
      const uintptr_t a = (uintptr_t)m[i].p, b = (uintptr_t)m[j].p;
      if (a < b + m[j].bytes && b < a + m[i].bytes) return true;
    }
  return false;
}

// How a product of M x N outputs over K is cut: output tiles of 32 S x 32 S
// (S = 8, 16-bit only; 4; 2) and parts of K.
struct Cut {
  int S, parts;
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
// and 1 the few-token kernel wherever it fits.  Read once a call; 0 for anything
// else.
int forced_tile() {
  const char* env = std::getenv("FLCE_DEBUG_LAYER_TILE");
  const int s = env ? std::atoi(env) : 0;
  return s == 1 || s == 2 || s == 4 || s == 8 ? s : 0;
}

// forced: from forced_tile.  only: the S to use (0: any).
Cut product_cut(int64_t M, int64_t N, int64_t K, int dtype, int forced, int only = 0) {
  if (M < 1 || N < 1) return {only ? only : 2, 1};   // nothing to form
  Cut best{only ? only : 2, 1};
  double least = 0.0;
  auto consider = [&](const TileCost& t) {
    if (only && t.S != only) return;
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
        best = {t.S, (int)parts};
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
  const int forced = forced_tile();
  Cut fwd = product_cut(N, nmat * F, H, dtype, forced);
  if (forced == 1 ? N <= flce::kSkinnyMost : forced == 0 && N <= flce::skinny_tokens(dtype)) fwd = {0, 1};
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
  // Two small products share a launch, and with it their tiles' size: where their
  // own picks differ, S = 4 with the splits costed for it.  (Of 70 such shapes,
  // N to 4096, H and F to 8192, all types, S = 4 took 1-2% more than the faster of
  // both on average and 16% at worst; the size whose times add up to less, 4% and
  // 57%, as the products fill each other's rounds.)  It holds for a call that asks
  // for one gradient alone too, which so has the same bits as beside the other.
  Cut cx = product_cut(H, N, g.ldz, dtype, forced), cw = product_cut(H, nmat * F, N, dtype, forced);
  if (cx.S < 8 && cw.S < 8 && cx.S != cw.S) {
    cx = product_cut(H, N, g.ldz, dtype, forced, 4);
    cw = product_cut(H, nmat * F, N, dtype, forced, 4);
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
  const size_t nf = (size_t)N * F * es, fh = (size_t)F * H * es;
  const Memory mem[] = {{x, (size_t)N * H * es, false}, {W[0], fh, false}, {W[1], fh, false},
                        {b[0], F * es, false}, {b[1], F * es, false}, {residual == y ? nullptr : residual, nf, false},
                        {y, nf, true}, {z[0], (size_t)N * F * 4, true}, {z[1], (size_t)N * F * 4, true},
                        {workspace, g.fwd_total, true}};
  if (clash(mem, 10)) return FLCE_ERR_INVALID_ARGUMENT;
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
  const size_t nh = (size_t)N * H * es, fh = (size_t)F * H * es, kept = need_z ? (size_t)N * F * 4 : 0;
  const Memory mem[] = {{x, nh, false}, {W[0], fh, false}, {W[1], fh, false}, {z[0], kept, false}, {z[1], kept, false},
                        {dy, (size_t)N * F * es, false}, {dx, nh, true}, {dW[0], fh, true}, {dW[1], fh, true},
                        {db[0], F * es, true}, {db[1], F * es, true}, {workspace, g.bwd_total, true}};
  if (clash(mem, 12)) return FLCE_ERR_INVALID_ARGUMENT;
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

}  // extern "C"

#include "layer_norm_api.hpp"
#include "layer_mx_api.hpp"
#include "layer_sample_api.hpp"
