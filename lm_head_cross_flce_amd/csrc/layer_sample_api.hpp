// Host side of the sampler: argument checks and entry point.  Included once, at the
// end of layer_api.hpp.
#pragma once

#include "layer_launch.hpp"

extern "C" {

flce_status flce_sample(const void* logits, const float* u, int64_t N, int64_t V, flce_dtype dtype,
                        const flce_sampling* params, int64_t* tokens, hipStream_t stream) {
  if (N < 0 || V < 1 || !params) return FLCE_ERR_INVALID_ARGUMENT;
  if (dtype != FLCE_F32 && dtype != FLCE_BF16 && dtype != FLCE_F16) return FLCE_ERR_UNSUPPORTED;
  if (N > (int64_t(1) << 22) || V > (int64_t(1) << 30)) return FLCE_ERR_UNSUPPORTED;   // a workgroup of 1024 threads a row
  const bool rows = N > 0;
  if (bad_tensor(logits, 16, rows) || bad_tensor(u, 4, rows) || bad_tensor(tokens, 8, rows) ||
      bad_tensor(params->temperatures, 4, false) || bad_tensor(params->top_ks, 8, false) ||
      bad_tensor(params->top_ps, 4, false) || bad_tensor(params->min_ps, 4, false))
    return FLCE_ERR_INVALID_ARGUMENT;
  if (!rows) return FLCE_OK;
  const size_t n4 = (size_t)N * 4;
  const Memory mem[] = {{logits, (size_t)N * V * (dtype == FLCE_F32 ? 4 : 2), false}, {u, n4, false},
                        {params->temperatures, n4, false}, {params->top_ks, 2 * n4, false}, {params->top_ps, n4, false},
                        {params->min_ps, n4, false}, {tokens, 2 * n4, true}};
  if (clash(mem, 7)) return FLCE_ERR_INVALID_ARGUMENT;
  flce::Sample a{};
  a.logits = logits; a.u = u;
  a.temperature = params->temperatures; a.top_k = params->top_ks; a.top_p = params->top_ps; a.min_p = params->min_ps;
  a.temperature0 = params->temperature; a.top_k0 = params->top_k; a.top_p0 = params->top_p; a.min_p0 = params->min_p;
  a.tokens = tokens;
  a.N = N; a.V = (int)V;
  (void)hipGetLastError();
  flce::mark_launch(stream, nullptr);
  return flce::launch_sample(a, dtype, stream) == hipSuccess ? FLCE_OK : FLCE_ERR_HIP;
}

}  // extern "C"
