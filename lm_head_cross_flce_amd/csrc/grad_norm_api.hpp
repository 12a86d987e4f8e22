// Host side of the gradient norm and clipping: argument checks, chunks, launch
// tables, entry points.  Included once, by flce_api.hip.
#pragma once

#include "layer_api.hpp"   // clash

namespace {

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

// Nor may the norm (written, or given and read by every workgroup) or the
// workspace share memory with a tensor, beyond a given norm with what is only read.
flce_status check_scalars(const void* const* grads, void* const* outs, const int64_t* numels, const flce_dtype* dtypes,
                          int64_t count, bool clip, const float* given, const float* norm_out, const void* workspace,
                          size_t workspace_bytes) {
  Memory m[] = {{given, 4, false}, {norm_out, 4, true}, {workspace, workspace_bytes, true}, {}};
  if (clash(m, 3)) return FLCE_ERR_INVALID_ARGUMENT;
  auto meets = [&](const void* p, size_t bytes, bool written) {
    m[3] = {p, bytes, written};
    return clash(m, 4);
  };
  for (int64_t i = 0; i < count; ++i) {
    const size_t bytes = (size_t)(numels[i] * dtype_bytes(dtypes[i]));
    const void* out = outs ? outs[i] : grads[i];
    if (meets(grads[i], bytes, clip && out == grads[i]) || (clip && out != grads[i] && meets(out, bytes, true)))
      return FLCE_ERR_INVALID_ARGUMENT;
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
  const flce_status sc = check_scalars(grads, outs, numels, dtypes, count, clip, given, norm_out, given ? nullptr : workspace,
                                       given ? 0 : norm_bytes(count));
  if (sc != FLCE_OK) return sc;
  return run_grad_norm(grads, outs, numels, dtypes, count, max_norm, inf_norm, given, clip, norm_out, (double*)workspace,
                       stream);
}

}  // namespace

extern "C" {

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
