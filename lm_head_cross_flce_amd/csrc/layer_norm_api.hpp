// Host side of the root-mean-square norm: argument checks, geometry, entry points.
// Included once, at the end of layer_api.hpp.
#pragma once

#include "layer_launch.hpp"

namespace {

flce_status check_norm_shape(int64_t N, int64_t H, int dtype) {
  if (N < 0 || H < 1) return FLCE_ERR_INVALID_ARGUMENT;
  if (dtype != FLCE_F32 && dtype != FLCE_BF16 && dtype != FLCE_F16) return FLCE_ERR_UNSUPPORTED;
  if (N > (int64_t(1) << 30) || H > (int64_t(1) << 20)) return FLCE_ERR_UNSUPPORTED;
  return FLCE_OK;
}

size_t type_bytes(int dtype) { return dtype == FLCE_F32 ? 4 : 2; }

// Columns of a microscaled tensor's rows, and their code bytes.
int64_t mx_cols(int64_t C) { return cdiv(C, flce::kMxPad) * flce::kMxPad; }
size_t mx_code_bytes(int64_t C, int format) { return (size_t)mx_cols(C) / (format == FLCE_MX_E2M1 ? 2 : 1); }
size_t mx_scale_bytes(int64_t C) { return (size_t)mx_cols(C) / flce::kMxBlock; }
bool bad_format(int format) { return format != FLCE_MX_E4M3 && format != FLCE_MX_E2M1; }

// Workgroups of the backward, each with sums of its own for dweight: 4 a CU of 256 threads, or
// one of 1024.  (8192 x 4096 bf16: 1024 workgroups 59 us and 6 for adding their sums, 512 87 and
// 4.5, 2048 62 and 10; 2000 x 16000: 256 58 and 5, 1024 68 and 12.)  Up to 1024 columns
// a workgroup has four rows or more at once, and 512 are enough (16384 x 512 fp32).  Of these as many
// as have equally many rows (1037 x 4096 bf16: 519 workgroups 12.5 us and 4.5, 1024, thirteen of them with
// two rows, 14.7 and 6.1).
int64_t norm_parts(int64_t N, int64_t H) {
  if (H > flce::kNormMost) return std::min<int64_t>(N, 64);
  const int lanes = flce::norm_lanes((int)H, false);
  const int64_t groups = cdiv(N, flce::norm_rows(lanes)), most = lanes == 1024 ? 256 : lanes == 256 ? 1024 : 512;
  return groups ? cdiv(groups, cdiv(groups, most)) : 0;
}
size_t norm_bwd_bytes(int64_t N, int64_t H) { return align_up((size_t)norm_parts(N, H) * H * 4); }

// y, or codes and scales.
flce_status norm_forward(const void* x, const void* residual, const void* weight, int64_t N, int64_t H, int dtype, float eps,
                         int format, void* y, uint8_t* codes, uint8_t* scales, void* h, float* rstd, hipStream_t stream) {
  const flce_status st = check_norm_shape(N, H, dtype);
  if (st != FLCE_OK) return st;
  if (!(eps >= 0.f) || std::isinf(eps)) return FLCE_ERR_INVALID_ARGUMENT;
  const bool mx = format >= 0;
  if (mx && bad_format(format)) return FLCE_ERR_INVALID_ARGUMENT;
  const bool rows = N > 0;
  const size_t es = type_bytes(dtype), nh = (size_t)N * H * es;
  if (bad_tensor(x, 16, rows) || bad_tensor(residual, 16, false) || bad_tensor(weight, es, false) || bad_tensor(h, 16, false) ||
      bad_tensor(rstd, 4, false))
    return FLCE_ERR_INVALID_ARGUMENT;
  if (mx ? bad_tensor(codes, 16, rows) || bad_tensor(scales, 4, rows) : bad_tensor(y, 16, rows)) return FLCE_ERR_INVALID_ARGUMENT;
  if (h && !residual) return FLCE_ERR_INVALID_ARGUMENT;   // it would be x
  if (!rows) return FLCE_OK;
  const bool in_place = h == x || h == residual;   // each thread writes where it has read
  const Memory mem[] = {{h == x ? nullptr : x, nh, false}, {h == residual ? nullptr : residual, nh, false},
                        {weight, (size_t)H * es, false}, {h, nh, true}, {mx ? nullptr : y, nh, true},
                        {codes, mx ? N * mx_code_bytes(H, format) : 0, true}, {scales, mx ? N * mx_scale_bytes(H) : 0, true},
                        {rstd, (size_t)N * 4, true}};
  if (clash(mem, 8)) return FLCE_ERR_INVALID_ARGUMENT;
  // x and the residual in part the same memory: one of them is written in place, so the other's rows would change
  if (in_place && x != residual) {
    const Memory both[] = {{x, nh, true}, {residual, nh, false}};
    if (clash(both, 2)) return FLCE_ERR_INVALID_ARGUMENT;
  }
  flce::NormFwd a{};
  a.x = x; a.residual = residual; a.weight = weight;
  a.h = h; a.y = y; a.codes = codes; a.scales = scales; a.rstd = rstd;
  a.N = N; a.H = (int)H; a.Hp = (int)mx_cols(H);
  a.format = format;
  a.eps = eps;
  const int lanes = flce::norm_lanes(mx ? a.Hp : a.H, mx);
  a.blocks = (int)std::min<int64_t>(cdiv(N, flce::norm_rows(lanes)), lanes == 1024 ? 512 : 2048);
  (void)hipGetLastError();
  flce::mark_launch(stream, nullptr);
  return flce::launch_rms_norm_forward(a, dtype, stream) == hipSuccess ? FLCE_OK : FLCE_ERR_HIP;
}

}  // namespace

extern "C" {

flce_status flce_rms_norm_forward(const void* x, const void* residual, const void* weight, int64_t N, int64_t H,
                                  flce_dtype dtype, float eps, void* y, void* h, float* rstd, hipStream_t stream) {
  return norm_forward(x, residual, weight, N, H, dtype, eps, -1, y, nullptr, nullptr, h, rstd, stream);
}

flce_status flce_rms_norm_mx_forward(const void* x, const void* residual, const void* weight, int64_t N, int64_t H,
                                     flce_dtype dtype, float eps, flce_mx_format format, uint8_t* codes, uint8_t* scales,
                                     void* h, float* rstd, hipStream_t stream) {
  if (bad_format(format)) return FLCE_ERR_INVALID_ARGUMENT;
  return norm_forward(x, residual, weight, N, H, dtype, eps, format, nullptr, codes, scales, h, rstd, stream);
}

flce_status flce_rms_norm_workspace_size(int64_t N, int64_t H, flce_dtype dtype, size_t* bwd_bytes) {
  const flce_status st = check_norm_shape(N, H, dtype);
  if (st != FLCE_OK) return st;
  if (bwd_bytes) *bwd_bytes = norm_bwd_bytes(N, H);
  return FLCE_OK;
}

flce_status flce_rms_norm_backward(const void* h, const void* weight, const float* rstd, const void* dy, const void* dh,
                                   int64_t N, int64_t H, flce_dtype dtype, void* dx, void* dweight, void* workspace,
                                   size_t workspace_bytes, hipStream_t stream) {
  const flce_status st = check_norm_shape(N, H, dtype);
  if (st != FLCE_OK) return st;
  const bool rows = N > 0;
  const size_t es = type_bytes(dtype), nh = (size_t)N * H * es;
  if (bad_tensor(h, 16, rows) || bad_tensor(weight, es, false) || bad_tensor(rstd, 4, rows) || bad_tensor(dy, 16, rows) ||
      bad_tensor(dh, 16, false) || bad_tensor(dx, 16, false) || bad_tensor(dweight, es, false))
    return FLCE_ERR_INVALID_ARGUMENT;
  const size_t bytes = dweight ? norm_bwd_bytes(N, H) : 0;
  if (workspace_bytes < bytes) return FLCE_ERR_WORKSPACE_TOO_SMALL;
  if (bad_tensor(workspace, 16, bytes > 0)) return FLCE_ERR_INVALID_ARGUMENT;
  if (!dx && !dweight) return FLCE_OK;
  const Memory mem[] = {{h, nh, false}, {weight, (size_t)H * es, false}, {rstd, (size_t)N * 4, false},
                        {dx == dy ? nullptr : dy, nh, false}, {dx == dh ? nullptr : dh, nh, false}, {dx, nh, true},
                        {dweight, (size_t)H * es, true}, {workspace, bytes, true}};
  if (clash(mem, 8)) return FLCE_ERR_INVALID_ARGUMENT;
  // rows too long for the registers are read again for dweight, after dx
  if (dx && dx == dy && dweight && H > flce::kNormMost) return FLCE_ERR_INVALID_ARGUMENT;
  if ((dx == dy || dx == dh) && dx && dh && dy != dh) {
    const Memory both[] = {{dy, nh, true}, {dh, nh, false}};
    if (clash(both, 2)) return FLCE_ERR_INVALID_ARGUMENT;
  }
  if (!rows && !dweight) return FLCE_OK;
  flce::NormBwd a{};
  a.h = h; a.weight = weight; a.rstd = rstd; a.dy = dy; a.dh = dh;
  a.dx = rows ? dx : nullptr; a.dweight = dweight;
  a.part = (float*)workspace;
  a.N = N; a.H = (int)H;
  a.parts = (int)norm_parts(N, H);
  (void)hipGetLastError();
  flce::mark_launch(stream, nullptr);
  return flce::launch_rms_norm_backward(a, dtype, stream) == hipSuccess ? FLCE_OK : FLCE_ERR_HIP;
}

}  // extern "C"
