// Host side of the sampler: argument checks, workspace layout, entry points.
// Included once, at the end of layer_api.hpp.
#pragma once

#include "layer_launch.hpp"

namespace {

struct SampleGeometry {
  int64_t slices, groups;
  size_t off_top, off_sum, off_bin, off_hist, total;
};

SampleGeometry sample_geometry(int64_t N, int64_t V) {
  SampleGeometry g{};
  if (V <= flce::kOneLaunchTokens) return g;
  g.slices = cdiv(V, flce::kSliceTokens);
  g.groups = cdiv(V, flce::kGroupTokens);
  g.off_top = align_up((size_t)N * g.groups * 4);
  g.off_sum = align_up(g.off_top + (size_t)N * g.slices * 4);
  g.off_bin = align_up(g.off_sum + (size_t)N * g.slices * 8);
  g.off_hist = align_up(g.off_bin + (size_t)N * g.slices * 4);
  g.total = align_up(g.off_hist + (size_t)N * g.slices * flce::kHistBins * 8);
  return g;
}

flce_status check_sample(int64_t N, int64_t V, int dtype) {
  if (N < 0 || V < 1) return FLCE_ERR_INVALID_ARGUMENT;
  if (dtype != FLCE_F32 && dtype != FLCE_BF16 && dtype != FLCE_F16) return FLCE_ERR_UNSUPPORTED;
  // a launch has fewer than 2^32 threads: 1024 a row, 256 a slice
  if (N >= (int64_t(1) << 22) || V > (int64_t(1) << 30) || N * cdiv(V, flce::kSliceTokens) >= (int64_t(1) << 24))
    return FLCE_ERR_UNSUPPORTED;
  return FLCE_OK;
}

}  // namespace

extern "C" {

flce_status flce_sample_workspace_size(int64_t N, int64_t V, flce_dtype dtype, size_t* bytes) {
  const flce_status st = check_sample(N, V, dtype);
  if (st != FLCE_OK) return st;
  if (bytes) *bytes = N > 0 ? sample_geometry(N, V).total : 0;
  return FLCE_OK;
}

flce_status flce_sample(const void* logits, const float* u, int64_t N, int64_t V, flce_dtype dtype,
                        const flce_sampling* params, int64_t* tokens, void* workspace, size_t workspace_bytes,
                        hipStream_t stream) {
  const flce_status st = check_sample(N, V, dtype);
  if (st != FLCE_OK) return st;
  if (!params) return FLCE_ERR_INVALID_ARGUMENT;
  const bool rows = N > 0;
  if (bad_tensor(logits, 16, rows) || bad_tensor(u, 4, rows) || bad_tensor(tokens, 8, rows) ||
      bad_tensor(params->temperatures, 4, false) || bad_tensor(params->top_ks, 8, false) ||
      bad_tensor(params->top_ps, 4, false) || bad_tensor(params->min_ps, 4, false))
    return FLCE_ERR_INVALID_ARGUMENT;
  if (!rows) return FLCE_OK;
  const SampleGeometry g = sample_geometry(N, V);
  if (workspace_bytes < g.total) return FLCE_ERR_WORKSPACE_TOO_SMALL;
  if (bad_tensor(workspace, 16, g.total > 0)) return FLCE_ERR_INVALID_ARGUMENT;
  const size_t n4 = (size_t)N * 4;
  const Memory mem[] = {{logits, (size_t)N * V * type_bytes(dtype), false}, {u, n4, false},
                        {params->temperatures, n4, false}, {params->top_ks, 2 * n4, false}, {params->top_ps, n4, false},
                        {params->min_ps, n4, false}, {tokens, 2 * n4, true}, {workspace, g.total, true}};
  if (clash(mem, 8)) return FLCE_ERR_INVALID_ARGUMENT;
  flce::Sample a{};
  a.logits = logits; a.u = u;
  a.temperature = params->temperatures; a.top_k = params->top_ks; a.top_p = params->top_ps; a.min_p = params->min_ps;
  a.temperature0 = params->temperature; a.top_k0 = params->top_k; a.top_p0 = params->top_p; a.min_p0 = params->min_p;
  a.tokens = tokens;
  a.N = N; a.V = (int)V;
  a.slices = (int)g.slices; a.groups = (int)g.groups;
  char* ws = (char*)workspace;
  a.group_top = (uint32_t*)ws;
  a.slice_top = (uint32_t*)(ws + g.off_top);
  a.slice_sum = (double*)(ws + g.off_sum);
  a.slice_bin = (int*)(ws + g.off_bin);
  a.hist = (unsigned long long*)(ws + g.off_hist);
  a.hist_shift = 40;   // a bin's V elements under 2^(1/8) each, in 63 bits
  while ((double)V * 1.2 * (double)(1ull << a.hist_shift) > 4e18) --a.hist_shift;
  (void)hipGetLastError();
  flce::mark_launch(stream, nullptr);
  return flce::launch_sample(a, dtype, stream) == hipSuccess ? FLCE_OK : FLCE_ERR_HIP;
}

}  // extern "C"
