// Global gradient norm over many tensors, and clipping.
//
//   norm = (sum over tensors and elements of g^2)^(1/2)   or   max |g|
//   out  = g min(1, max_norm / (norm + 1e-6))
//
// HBM bounds both passes.  The tensors' addresses and sizes travel in the
// kernel arguments (a table of up to kNormTensors), so the library copies
// nothing to the device and a captured graph holds them.  A launch's tensors
// are cut into chunks of 4 KB or more (more in a large call); a workgroup takes
// a run of consecutive chunks, so it looks its first tensor up once and then
// walks the table.
// Sums of squares are kept in fp64: one element's square can pass fp32's
// range, and the fp64 additions cost less than the loads they hide under.
// Every workgroup leaves one partial and adds are made in a fixed order, so a
// norm is the same bit for bit at every call.
#include "flce_device.hpp"
#include "flce_launch.hpp"

namespace flce {

namespace {

// NaN stays: it compares false with everything.
__device__ __forceinline__ float max_nan(float a, float b) { return (b > a || b != b) ? b : a; }

template <bool INF> struct NormAcc {
  double s;
  float m;
  __device__ __forceinline__ void add(float v) {
    if constexpr (INF) m = max_nan(m, fabsf(v));
    else s = fma((double)v, (double)v, s);
  }
  __device__ __forceinline__ void merge(const NormAcc& o) {
    if constexpr (INF) m = max_nan(m, o.m);
    else s += o.s;
  }
};

// Sum (or max) over the workgroup's 256 threads, in every thread.
template <bool INF> __device__ __forceinline__ NormAcc<INF> block_reduce(NormAcc<INF> a) {
  __shared__ NormAcc<INF> red[4];
#pragma unroll
  for (int mask = 1; mask < 64; mask <<= 1) {
    NormAcc<INF> o{};
    if constexpr (INF) o.m = __shfl_xor(a.m, mask);
    else o.s = __shfl_xor(a.s, mask);
    a.merge(o);
  }
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = a;
  __syncthreads();
  a = red[0];
#pragma unroll
  for (int i = 1; i < 4; ++i) a.merge(red[i]);
  return a;
}

// Unpacks 16 bytes (8 or 4 elements).
template <class T> struct Vec {
  static constexpr int kN = 16 / sizeof(T);
  float v[kN];
  __device__ __forceinline__ explicit Vec(u32x4 w) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 4) v[i] = __uint_as_float(w[i]);
      else {
        v[2 * i] = h16_to_f32<T>(w[i]);
        v[2 * i + 1] = h16_to_f32<T>(w[i] >> 16);
      }
    }
  }
  __device__ __forceinline__ u32x4 scaled(float c) const {
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 4) w[i] = __float_as_uint(v[i] * c);
      else w[i] = pack2<T>(v[2 * i] * c, v[2 * i + 1] * c);
    }
    return w;
  }
};
template <class T> __device__ __forceinline__ float one(const T* p) {
  if constexpr (sizeof(T) == 4) return *(const float*)p;
  else return h16_to_f32<T>(*(const uint16_t*)p);
}
template <class T> __device__ __forceinline__ void put(T* p, float v) {
  if constexpr (sizeof(T) == 4) *(float*)p = v;
  else *(uint16_t*)p = (uint16_t)(pack2<T>(v, 0.f) & 0xffffu);
}

// Chunk c of an n-element tensor at p: the elements up to p's first 16-byte
// boundary (head) belong to chunk 0, and the chunks count from there.
struct Span {
  int64_t head, lo, hi;   // [lo, hi): the chunk's elements; chunk 0 also has [0, head)
};
template <class T> __device__ __forceinline__ Span span_of(const T* p, int64_t n, int64_t c, int chunk_bytes) {
  const int64_t CH = chunk_bytes / (int)sizeof(T);
  Span s;
  s.head = ((16 - ((uintptr_t)p & 15)) & 15) / sizeof(T);
  s.head = s.head < n ? s.head : n;
  s.lo = s.head + c * CH;
  s.hi = s.lo + CH < n ? s.lo + CH : n;
  return s;
}

// One chunk into the accumulator: 16 bytes a thread, 4 loads in flight.
// STREAM: loads that leave nothing in the memory-side cache.
template <class T, bool INF, bool STREAM>
__device__ __forceinline__ void norm_chunk(NormAcc<INF>& a, const T* p, int64_t n, int64_t c, int chunk_bytes) {
  const Span s = span_of(p, n, c, chunk_bytes);
  const int tid = threadIdx.x;
  if (c == 0 && tid < s.head) a.add(one(p + tid));
  constexpr int V = Vec<T>::kN;
  const int64_t len = s.hi > s.lo ? s.hi - s.lo : 0;
  const int nv = (int)(len / V);
  const u32x4* q = (const u32x4*)(p + s.lo);
  auto fetch = [&](int i) { return STREAM ? __builtin_nontemporal_load(q + i) : q[i]; };
  int i = tid;
  for (; i + 768 < nv; i += 1024) {
    u32x4 w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = fetch(i + 256 * k);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const Vec<T> v(w[k]);
#pragma unroll
      for (int e = 0; e < V; ++e) a.add(v.v[e]);
    }
  }
  for (; i < nv; i += 256) {
    const Vec<T> v(fetch(i));
#pragma unroll
    for (int e = 0; e < V; ++e) a.add(v.v[e]);
  }
  const int64_t t = s.lo + (int64_t)nv * V + tid;
  if (t < s.hi) a.add(one(p + t));
}

template <class T>
__device__ __forceinline__ void clip_chunk(const T* p, T* d, int64_t n, int64_t c, int chunk_bytes, float coef) {
  const Span s = span_of(p, n, c, chunk_bytes);
  const int tid = threadIdx.x;
  constexpr int V = Vec<T>::kN;
  if (c == 0 && tid < s.head) put(d + tid, one(p + tid) * coef);
  const int64_t len = s.hi > s.lo ? s.hi - s.lo : 0;
  const int nv = ((uintptr_t)(d + s.lo) & 15) == 0 ? (int)(len / V) : 0;   // out aligned like p, or one by one
  const u32x4* q = (const u32x4*)(p + s.lo);
  u32x4* o = (u32x4*)(d + s.lo);
  int i = tid;
  for (; i + 768 < nv; i += 1024) {
    u32x4 w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = q[i + 256 * k];
#pragma unroll
    for (int k = 0; k < 4; ++k) o[i + 256 * k] = Vec<T>(w[k]).scaled(coef);
  }
  for (; i < nv; i += 256) o[i] = Vec<T>(q[i]).scaled(coef);
  for (int64_t t = s.lo + (int64_t)nv * V + tid; t < s.hi; t += 256) put(d + t, one(p + t) * coef);
}

// The tensor that holds chunk c: the number of tensors whose chunks end at or
// before it, counted by all lanes at once (a search through the table would
// wait for a load from the kernel arguments at each step).
__device__ __forceinline__ int find_tensor(const NormTable& t, int64_t c) {
  static_assert(kNormTensors <= 128, "two entries a lane");
  const int lane = threadIdx.x & 63;
  const bool a = lane < t.count && t.end[lane] <= c;
  const bool b = lane + 64 < t.count && t.end[lane + 64 < kNormTensors ? lane + 64 : 0] <= c;
  return __popcll(__ballot(a)) + __popcll(__ballot(b));
}

}  // namespace

template <bool INF, bool STREAM> __global__ void __launch_bounds__(256) grad_norm_kernel(NormTable t, double* part) {
  const int64_t total = t.count ? t.end[t.count - 1] : 0;
  const int64_t c0 = total * blockIdx.x / gridDim.x, c1 = total * (blockIdx.x + 1) / gridDim.x;
  NormAcc<INF> a{};
  int k = c0 < c1 ? find_tensor(t, c0) : 0;
  for (int64_t c = c0; c < c1; ++c) {
    while (t.end[k] <= c) ++k;
    const int64_t cc = c - (k ? t.end[k - 1] : 0);
    if (t.dtype[k] == 1) norm_chunk<uint16_t, INF, STREAM>(a, (const uint16_t*)t.in[k], t.n[k], cc, t.chunk_bytes);
    else if (t.dtype[k] == 2) norm_chunk<_Float16, INF, STREAM>(a, (const _Float16*)t.in[k], t.n[k], cc, t.chunk_bytes);
    else norm_chunk<float, INF, STREAM>(a, (const float*)t.in[k], t.n[k], cc, t.chunk_bytes);
  }
  a = block_reduce(a);
  if (threadIdx.x == 0) part[blockIdx.x] = INF ? (double)a.m : a.s;
}

// Every workgroup adds the partials up itself (a few KB from L2, cheaper than
// another launch), in the same order.  given: the norm comes from there
// instead.  norm_out: written by workgroup 0.
template <bool INF> __global__ void __launch_bounds__(256) grad_clip_kernel(NormTable t, const double* part, int parts,
                                                                            const float* given, float* norm_out,
                                                                            float max_norm) {
  float norm;
  double nd;
  if (given) {
    norm = *given;
    nd = norm;
  } else {
    NormAcc<INF> a{};
    for (int i = threadIdx.x; i < parts; i += 256) {
      NormAcc<INF> o{};
      if constexpr (INF) o.m = (float)part[i];
      else o.s = part[i];
      a.merge(o);
    }
    a = block_reduce(a);
    nd = INF ? (double)a.m : sqrt(a.s);
    norm = (float)nd;
  }
  if (norm_out && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = norm;
  if (t.count == 0) return;
  const double cd = (double)max_norm / (nd + 1e-6);
  const float coef = cd > 1.0 ? 1.f : (float)cd;   // NaN stays
  if (coef == 1.f && t.in_place) return;           // every gradient keeps its value
  // The run of chunks that this workgroup of the norm's launch read, last one
  // first: those are still in the memory-side cache.
  const int64_t total = t.end[t.count - 1];
  const int64_t c0 = total * blockIdx.x / gridDim.x, c1 = total * (blockIdx.x + 1) / gridDim.x;
  int k = c0 < c1 ? find_tensor(t, c1 - 1) : 0;
  for (int64_t c = c1 - 1; c >= c0; --c) {
    while (k && t.end[k - 1] > c) --k;
    const int64_t cc = c - (k ? t.end[k - 1] : 0);
    if (t.dtype[k] == 1) clip_chunk((const uint16_t*)t.in[k], (uint16_t*)t.out[k], t.n[k], cc, t.chunk_bytes, coef);
    else if (t.dtype[k] == 2) clip_chunk((const _Float16*)t.in[k], (_Float16*)t.out[k], t.n[k], cc, t.chunk_bytes, coef);
    else clip_chunk((const float*)t.in[k], (float*)t.out[k], t.n[k], cc, t.chunk_bytes, coef);
  }
}

hipError_t launch_grad_norm(const NormTable& t, bool inf_norm, bool stream, double* part, int parts, hipStream_t st) {
  const dim3 grid(parts), blk(256);
  if (inf_norm && stream) FLCE_LAUNCH((grad_norm_kernel<true, true>), grid, blk, 0, st, t, part);
  else if (inf_norm) FLCE_LAUNCH((grad_norm_kernel<true, false>), grid, blk, 0, st, t, part);
  else if (stream) FLCE_LAUNCH((grad_norm_kernel<false, true>), grid, blk, 0, st, t, part);
  else FLCE_LAUNCH((grad_norm_kernel<false, false>), grid, blk, 0, st, t, part);
  return hipGetLastError();
}

hipError_t launch_grad_clip(const NormTable& t, bool inf_norm, const double* part, int parts, const float* given,
                            float* norm_out, float max_norm, int blocks, hipStream_t st) {
  if (inf_norm) FLCE_LAUNCH((grad_clip_kernel<true>), dim3(blocks), dim3(256), 0, st, t, part, parts, given, norm_out, max_norm);
  else FLCE_LAUNCH((grad_clip_kernel<false>), dim3(blocks), dim3(256), 0, st, t, part, parts, given, norm_out, max_norm);
  return hipGetLastError();
}

}  // namespace flce
