// Host side of the microscaled tensors: argument checks, tile and split choice,
// workspace layout, entry points.  Included once, at the end of layer_api.hpp.
#pragma once

#include "layer_norm_api.hpp"

namespace {

flce_status check_mx(int64_t R, int64_t C, int dtype, int format) {
  if (R < 0 || C < 1 || bad_format(format)) return FLCE_ERR_INVALID_ARGUMENT;
  if (dtype != FLCE_F32 && dtype != FLCE_BF16 && dtype != FLCE_F16) return FLCE_ERR_UNSUPPORTED;
  if (R > (int64_t(1) << 30) || C > (int64_t(1) << 20)) return FLCE_ERR_UNSUPPORTED;
  return FLCE_OK;
}

flce_status mx_convert(const void* x, void* y, uint8_t* codes, uint8_t* scales, int64_t R, int64_t C, int dtype, int format,
                       bool quantize, hipStream_t stream) {
  const flce_status st = check_mx(R, C, dtype, format);
  if (st != FLCE_OK) return st;
  const void* plain = quantize ? x : y;
  if (bad_tensor(plain, 16, R > 0) || bad_tensor(codes, 16, R > 0) || bad_tensor(scales, 4, R > 0)) return FLCE_ERR_INVALID_ARGUMENT;
  if (R == 0) return FLCE_OK;
  const Memory mem[] = {{plain, (size_t)R * C * type_bytes(dtype), !quantize}, {codes, R * mx_code_bytes(C, format), quantize},
                        {scales, R * mx_scale_bytes(C), quantize}};
  if (clash(mem, 3)) return FLCE_ERR_INVALID_ARGUMENT;
  flce::MxConvert a{};
  a.x = x; a.y = y; a.codes = codes; a.scales = scales;
  a.R = R; a.C = (int)C; a.Cp = (int)mx_cols(C);
  a.format = format;
  (void)hipGetLastError();
  flce::mark_launch(stream, nullptr);
  return (quantize ? flce::launch_mx_quantize(a, dtype, stream) : flce::launch_mx_dequantize(a, dtype, stream)) == hipSuccess
             ? FLCE_OK : FLCE_ERR_HIP;
}

struct MxGeometry {
  int tile, TM, TN, parts;   // tile 0: the few-token kernel, parts waves to a group of features; 1: its wide form
  int64_t kc, ldp;
  size_t total;
};

// Most tokens of the few-token kernels: 4 (16 tokens, 4096 -> 12288: 22 us, 18 in tiles), or 16 where a wave of 64
// features fills the card three times (e4m3, 4096 -> 128256: 62 us for one token, 72 for 16; tiles 88 for 17).
constexpr int64_t kMxFew = 4, kMxWideFew = 16;

// The tests' override of the tile, or 0.
int forced_mx_tile() {
  const char* env = std::getenv("FLCE_DEBUG_MX_TILE");
  const int s = env ? std::atoi(env) : 0;
  return s == 2 || s == 4 || s == 8 ? s : 0;
}

// The cut with the least estimated time, in us, of the busiest CU's q tiles, as product_cut has it:
//   q * per_tile + steps * max(alone, q * shared) + 4, a step 128 columns of K,
// by runs of 200 x 8192 x 8192, 517 x 4000 x 10241, 1024 x 4096 x 4096, 2048 and 8192 x 4096 x 12288 and
// 4096 x 8192 x 8192 at each tile, within a seventh of them then.  The kernels' times, us at S = 8 / 4 / 2:
// 8192 x 4096 x 12288 e2m1 206 / 334 / 448, e4m3 293 / 514 / 725; 517 x 4000 x 10241 e4m3 46 (with its join) / 43 / 59;
// 1024 x 4096 x 4096 e2m1 28 / 22 / 25.
struct MxCost {
  int S;
  double per_tile, alone, shared;
};
constexpr MxCost kMxCost[2][3] = {{{8, 6.7, 1.24, 1.24}, {4, 2.9, 0.87, 0.54}, {2, 0.2, 0.30, 0.27}},    // e4m3
                                  {{8, 6.8, 0.83, 0.83}, {4, 2.4, 0.66, 0.335}, {2, 0.3, 0.25, 0.147}}};   // e2m1
constexpr double kMxOddRows = 14.0;   // a 256-row tile's epilogue where F % 8 != 0

MxGeometry mx_geometry(int64_t N, int64_t K, int64_t F, int format, int dtype) {
  MxGeometry g{};
  const int64_t Kp = mx_cols(K), steps = Kp / 128;
  const int forced = forced_mx_tile();
  const bool exact = dtype == FLCE_F32 && format == FLCE_MX_E4M3;
  // The wide few-token kernel and the 256-row tile move scales in runs of 512 columns; neither expands operands.
  const bool runs = Kp >= 512 && !exact;
  const bool wide = runs && F >= 64 * 3 * kCUs;
  if (N <= (wide ? kMxWideFew : kMxFew) && !forced) {
    g.tile = wide ? 1 : 0;
    // enough waves for every CU, each with K of its own to walk
    g.parts = 1;
    while (g.parts < 8 && cdiv(F, 16) * g.parts < 8 * kCUs && steps >= 2 * g.parts) g.parts *= 2;
    g.kc = Kp;
    return g;
  }
  double least = 0.0;
  for (const MxCost& c : kMxCost[format == FLCE_MX_E2M1]) {
    if (c.S == 8 && !runs) continue;
    if (forced && c.S != (forced == 8 && !runs ? 4 : forced)) continue;
    const int64_t TM = cdiv(N, 32 * c.S), TN = cdiv(F, 32 * c.S);
    for (int64_t parts : {1, 2, 4, 8}) {
      const int64_t kc = cdiv(cdiv(Kp, parts), 256) * 256;
      if (parts > 1 && (kc < 512 || cdiv(Kp, kc) != parts)) continue;
      const double q = (double)cdiv(TM * TN * parts, kCUs), depth = (double)(parts > 1 ? kc : Kp) / 128.0;
      const double slow = exact ? 1.7 : 1.0;   // (1024 x 4096 x 4096: 2.2 and 2.4 times at S = 4 and 2)
      double us = q * (c.per_tile + (c.S == 8 && parts == 1 && F % 8 != 0 ? kMxOddRows : 0.0)) +
                  slow * depth * std::max(c.alone, q * c.shared) + 4.0;
      if (parts > 1) us += 3.0 + 8.0 * (double)parts * (double)N * (double)F / 4e6;   // the sums' way out and back
      if (least == 0.0 || us < least) {
        least = us;
        g.tile = c.S;
        g.TM = (int)TM;
        g.TN = (int)TN;
        g.parts = (int)parts;
        g.kc = parts > 1 ? kc : Kp;
      }
    }
  }
  g.ldp = cdiv(F, 8) * 8;
  g.total = g.parts > 1 ? align_up((size_t)g.parts * N * g.ldp * 4) : 0;
  return g;
}

flce_status check_mx_linear(int64_t N, int64_t K, int64_t F, int dtype, int format, int act) {
  if (N < 0 || K < 1 || F < 1 || bad_format(format)) return FLCE_ERR_INVALID_ARGUMENT;
  if (act < FLCE_ACT_NONE || act > FLCE_ACT_SIGMOID) return FLCE_ERR_INVALID_ARGUMENT;
  if (dtype != FLCE_F32 && dtype != FLCE_BF16 && dtype != FLCE_F16) return FLCE_ERR_UNSUPPORTED;
  if (N > (int64_t(1) << 30) || K > (int64_t(1) << 20) || F > (int64_t(1) << 20)) return FLCE_ERR_UNSUPPORTED;
  if (cdiv(N, 64) * cdiv(F, 64) > (int64_t(1) << 22)) return FLCE_ERR_UNSUPPORTED;   // a launch has fewer than 2^32 threads
  return FLCE_OK;
}

}  // namespace

extern "C" {

flce_status flce_mx_quantize(const void* x, int64_t R, int64_t C, flce_dtype dtype, flce_mx_format format, uint8_t* codes,
                             uint8_t* scales, hipStream_t stream) {
  return mx_convert(x, nullptr, codes, scales, R, C, dtype, format, true, stream);
}

flce_status flce_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t R, int64_t C, flce_mx_format format,
                               flce_dtype dtype, void* y, hipStream_t stream) {
  return mx_convert(nullptr, y, const_cast<uint8_t*>(codes), const_cast<uint8_t*>(scales), R, C, dtype, format, false, stream);
}

flce_status flce_mx_linear_workspace_size(int64_t N, int64_t K, int64_t F, flce_mx_format x_format, flce_dtype dtype,
                                          size_t* bytes) {
  const flce_status st = check_mx_linear(N, K, F, dtype, x_format, FLCE_ACT_NONE);
  if (st != FLCE_OK) return st;
  if (bytes) *bytes = mx_geometry(N, K, F, x_format, dtype).total;
  return FLCE_OK;
}

flce_status flce_mx_linear(const uint8_t* x, const uint8_t* x_scales, flce_mx_format x_format, const uint8_t* W,
                           const uint8_t* W_scales, const void* b, const void* residual, int64_t N, int64_t K, int64_t F,
                           flce_dtype dtype, flce_activation activation, void* y, void* workspace, size_t workspace_bytes,
                           hipStream_t stream) {
  const flce_status st = check_mx_linear(N, K, F, dtype, x_format, activation);
  if (st != FLCE_OK) return st;
  const size_t es = type_bytes(dtype);
  const bool rows = N > 0;
  if (bad_tensor(x, 16, rows) || bad_tensor(x_scales, 4, rows) || bad_tensor(W, 16, true) || bad_tensor(W_scales, 4, true) ||
      bad_tensor(b, es, false) || bad_tensor(residual, 16, false) || bad_tensor(y, 16, rows))
    return FLCE_ERR_INVALID_ARGUMENT;
  const MxGeometry g = mx_geometry(N, K, F, x_format, dtype);
  if (workspace_bytes < g.total) return FLCE_ERR_WORKSPACE_TOO_SMALL;
  if (bad_tensor(workspace, 16, g.total > 0)) return FLCE_ERR_INVALID_ARGUMENT;
  if (!rows) return FLCE_OK;
  const size_t nf = (size_t)N * F * es;
  const Memory mem[] = {{x, N * mx_code_bytes(K, x_format), false}, {x_scales, N * mx_scale_bytes(K), false},
                        {W, F * mx_code_bytes(K, FLCE_MX_E2M1), false}, {W_scales, F * mx_scale_bytes(K), false},
                        {b, (size_t)F * es, false}, {residual == y ? nullptr : residual, nf, false}, {y, nf, true},
                        {workspace, g.total, true}};
  if (clash(mem, 8)) return FLCE_ERR_INVALID_ARGUMENT;
  flce::MxLinear a{};
  a.x = x; a.xs = x_scales; a.W = W; a.Ws = W_scales;
  a.b = b; a.residual = residual; a.y = y;
  a.N = (int)N; a.F = (int)F; a.Kp = (int)mx_cols(K);
  a.format = x_format;
  a.act = activation;
  a.tile = g.tile; a.TM = g.TM; a.TN = g.TN;
  a.parts = g.parts; a.kc = (int)g.kc;
  a.part = (float*)workspace; a.ldp = g.ldp;
  (void)hipGetLastError();
  flce::mark_launch(stream, nullptr);
  return flce::launch_mx_linear(a, dtype, stream) == hipSuccess ? FLCE_OK : FLCE_ERR_HIP;
}

}  // extern "C"
