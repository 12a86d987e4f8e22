// Sampling a token from each row of logits: temperature, top-k, top-p, min-p, and the
// draw from a given uniform number.
//
//   w_j = exp((z_j - max) / T), tokens ranked by z from the largest, equal ones by index
//   top-k: the first k;  top-p: of those, each whose predecessors' w is less than p times
//   their sum;  min-p: of those, w_j >= min_p
//   token = the first in the vocabulary's order at which the kept w add up to more than u
//   times their sum
//
// Weights are formed in double and added as whole numbers of 2^-s, s as large as
// keeps a row's sum under 2^63 (46 at 128256 tokens): a whole sum does not depend on
// its order, so atomics may form it, and every comparison with it is exact.  The
// rounding, 2^-47 of the largest weight a token, is far under what a float32 u can
// tell apart.
#include "layer_device.hpp"
#include "layer_launch.hpp"

namespace flce {

typedef unsigned long long u64;

// Order of the values as whole numbers; -0 is 0.  Every NaN is above +infinity or below -infinity.
__device__ __forceinline__ uint32_t value_key(float v) {
  const uint32_t b = __float_as_uint(v + 0.f);
  return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) { return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu)); }
constexpr uint32_t kKeyInf = 0xff800000u, kKeyMinusInf = 0x007fffffu;

// A row's weights as whole numbers.
struct Weigh {
  float top;
  double inv_t, unit, min_w;   // unit: 2^s
  __device__ __forceinline__ double real(float z) const {
    // equal to the largest: 1, also where that is infinite; masked: 0, whatever T
    return z == top ? 1.0 : z == -INFINITY || top == INFINITY ? 0.0 : exp(((double)z - (double)top) * inv_t);
  }
  __device__ __forceinline__ u64 operator()(float z) const { return (u64)rint(real(z) * unit); }
  __device__ __forceinline__ u64 kept(float z) const {
    const double w = real(z);
    return w >= min_w ? (u64)rint(w * unit) : 0;
  }
};

constexpr int kRowThreads = 1024, kRowWaves = kRowThreads / 64;
constexpr int kBins = 2048, kUnits = 2048;   // the units of a row: runs of 512 tokens, or of more in long rows

__device__ __forceinline__ u64 wave_scan(u64 v, int lane) {
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const u64 t = __shfl_up(v, d);
    if (lane >= d) v += t;
  }
  return v;
}

struct RowLds {
  u64 hist[kBins];
  u64 wave[kRowWaves];
  u64 mass[kUnits];
  uint32_t same[kUnits];
  u64 found_above;
  uint32_t found, key[kRowWaves];
};

// Sum of v over threads before this one, and over all of them.
__device__ __forceinline__ u64 block_scan(u64 v, u64& all, RowLds& L) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const u64 in = wave_scan(v, lane);
  __syncthreads();
  if (lane == 63) L.wave[wave] = in;
  __syncthreads();
  u64 before = in - v;
  all = 0;
#pragma unroll
  for (int w = 0; w < kRowWaves; ++w) {
    if (w < wave) before += L.wave[w];
    all += L.wave[w];
  }
  return before;
}

// The bin, from the last one down, in which the sum of the bins passes `want` (from 1
// to their whole sum), and the sum of the bins above it.
__device__ __forceinline__ uint32_t find_bin(u64 want, u64& above, RowLds& L) {
  const int t = threadIdx.x, hi = kBins - 1 - 2 * t;
  const u64 a = L.hist[hi], b = L.hist[hi - 1];
  u64 all;
  const u64 before = block_scan(a + b, all, L);
  if (before < want && before + a + b >= want) {
    const bool first = before + a >= want;
    L.found = first ? hi : hi - 1;
    L.found_above = first ? before : before + a;
  }
  __syncthreads();
  above = L.found_above;
  return L.found;
}

// f(value, index) over the row's tokens from first to last, 8 a lane at a time, by all threads.
template <class T, class F> __device__ __forceinline__ void each_token(const T* z, int V, F&& f) {
  for (int j = threadIdx.x * 8; j < V; j += kRowThreads * 8) {
    float v[8];
    load_some<T, 8>(z + j, V - j, v);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (j + e < V) f(v[e], j + e);
  }
}

// The key at which, from the largest down, the sum of `count(value)` reaches want, and the
// sum above that key.  skip: values whose key is below it count nothing; at it, `at_skip` in all.
template <class T, class F>
__device__ __forceinline__ uint32_t find_key(const T* z, int V, u64 want, u64& above, uint32_t skip, u64 at_skip, F&& count,
                                             RowLds& L) {
  constexpr int kLevels = sizeof(T) == 2 ? 2 : 3;   // 16-bit values' keys have their lowest 16 bits alike
  uint32_t prefix = 0;
  above = 0;
#pragma unroll 1
  for (int level = 0; level < kLevels; ++level) {
    const int shift = level == 0 ? 21 : level == 1 ? 10 : 0, bits = level == 2 ? 10 : 11;
    __syncthreads();
    for (int i = threadIdx.x; i < kBins; i += kRowThreads) L.hist[i] = 0;
    __syncthreads();
    each_token(z, V, [&](float v, int) {
      const uint32_t k = value_key(v);
      if (k <= skip || (level > 0 && (k >> (shift + bits)) != prefix)) return;
      atomicAdd(&L.hist[(k >> shift) & ((1u << bits) - 1)], count(v));
    });
    if (threadIdx.x == 0 && at_skip && (level == 0 || (skip >> (shift + bits)) == prefix))
      atomicAdd(&L.hist[(skip >> shift) & ((1u << bits) - 1)], at_skip);
    __syncthreads();
    u64 a;
    const uint32_t bin = find_bin(want - above, a, L);
    above += a;
    prefix = (prefix << bits) | bin;
  }
  // a 16-bit value's key ends in 10 bits of 0 or 1, as its sign bit has it
  return sizeof(T) == 2 ? (prefix << 10) | ((prefix >> 21) ? 0u : 0x3ffu) : prefix;
}

// One row a workgroup, read from memory in every pass.
template <class T> __global__ void __launch_bounds__(kRowThreads) sample_kernel(Sample a) {
  __shared__ RowLds L;
  const int64_t row = blockIdx.x;
  const T* z = (const T*)a.logits + row * a.V;
  const int V = a.V, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  // the largest key; a NaN of either sign stands above all
  uint32_t top = 0;
  each_token(z, V, [&](float v, int) { top = max(top, v != v ? 0xffffffffu : value_key(v)); });
#pragma unroll
  for (int d = 1; d < 64; d *= 2) top = max(top, (uint32_t)__shfl_xor((int)top, d));
  if (lane == 0) L.key[wave] = top;
  __syncthreads();
  for (int w = 0; w < kRowWaves; ++w) top = max(top, L.key[w]);
  if (top > kKeyInf || top <= kKeyMinusInf) {   // a NaN, or no token left
    if (tid == 0) a.tokens[row] = -1;
    return;
  }
  const float T0 = a.temperature ? a.temperature[row] : a.temperature0;
  const int64_t k = a.top_k ? a.top_k[row] : a.top_k0;
  const float p = a.top_p ? a.top_p[row] : a.top_p0, mp = a.min_p ? a.min_p[row] : a.min_p0, u = a.u[row];
  const bool greedy = !(T0 > 0.f);
  const int s = 62 - (V > 2 ? 32 - __clz(V - 1) : 1);   // V 2^s <= 2^62
  const Weigh w{key_value(top), greedy ? 0.0 : 1.0 / (double)T0, (double)(1ull << s), mp > 0.f ? (double)fminf(mp, 1.f) : 0.0};

  // Tokens above key `cut` are kept and the first `ties` at it.
  uint32_t cut = 0;
  u64 ties = 0;
  if (greedy) {
    cut = top;
    ties = 1;
  } else {
    if (k > 0 && k < V) {
      u64 above;
      cut = find_key(z, V, (u64)k, above, 0u, 0ull, [](float) { return 1ull; }, L);
      ties = (u64)k - above;
    }
    if (p < 1.f) {
      u64 sum = 0, all;
      each_token(z, V, [&](float v, int) { sum += value_key(v) > cut ? w(v) : 0; });
      block_scan(sum, all, L);
      const u64 at_cut = cut ? ties * w(key_value(cut)) : 0;
      all += at_cut;
      const double want = p > 0.f ? ceil((double)p * (double)all) : 0.0;
      if (want < 1.0) {
        cut = top;
        ties = 1;
      } else {
        u64 above;
        const u64 target = min((u64)want, all);
        const uint32_t c = find_key(z, V, target, above, cut, at_cut, w, L);
        const u64 each = w(key_value(c));
        const u64 need = (target - above + each - 1) / each;
        ties = c == cut ? min(ties, need) : need;
        cut = c;
      }
    }
  }

  // Kept weight and tokens at the cut of each unit.
  const int unit = 512 * ((V + 512 * kUnits - 1) / (512 * kUnits)), units = (V + unit - 1) / unit;
  for (int i = wave; i < units; i += kRowWaves) {
    u64 m = 0;
    uint32_t same = 0;
    for (int j = i * unit + lane * 8; j < min(V, (i + 1) * unit); j += 512) {
      float v[8];
      load_some<T, 8>(z + j, V - j, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (j + e >= V) continue;
        const uint32_t key = value_key(v[e]);
        if (key > cut) m += w.kept(v[e]);
        same += key == cut;
      }
    }
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      m += __shfl_xor(m, d);
      same += __shfl_xor(same, d);
    }
    if (lane == 0) {
      L.mass[i] = m;
      L.same[i] = same;
    }
  }
  __syncthreads();
  const u64 each = cut ? (greedy ? 1 : w.kept(key_value(cut))) : 0;
  // Each thread two units: their kept weight with the ties that the units before leave them.
  u64 m[2] = {0, 0}, n[2] = {0, 0}, all;
#pragma unroll
  for (int h = 0; h < 2; ++h)
    if (2 * tid + h < units) n[h] = L.same[2 * tid + h];
  u64 before = block_scan(n[0] + n[1], all, L);
  u64 used[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    used[h] = min(before, ties);
    const u64 take = min(n[h], ties - used[h]);
    if (2 * tid + h < units) m[h] = L.mass[2 * tid + h] + take * each;
    before += n[h];
  }
  before = block_scan(m[0] + m[1], all, L);
  const double spot = u > 0.f ? floor((double)u * (double)all) : 0.0;
  const u64 want = spot < (double)all ? min((u64)spot, all - 1) : all - 1;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (before <= want && want < before + m[h]) {
      L.found = 2 * tid + h;
      L.found_above = before;
      L.mass[0] = used[h];
    }
    before += m[h];
  }
  __syncthreads();
  // The first wave walks the unit, 512 tokens at a time.
  if (wave > 0) return;
  const int i = L.found;
  u64 done = L.found_above, taken = L.mass[0];
  for (int j0 = i * unit; j0 < min(V, (i + 1) * unit); j0 += 512) {
    const int j = j0 + lane * 8;
    float v[8];
    load_some<T, 8>(z + j, V - j, v);
    u64 same = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) same += j + e < V && value_key(v[e]) == cut;
    const u64 scan = wave_scan(same, lane);
    u64 tie = taken + scan - same, weight[8], sum = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      weight[e] = 0;
      if (j + e >= V) continue;
      const uint32_t key = value_key(v[e]);
      if (key > cut) weight[e] = w.kept(v[e]);
      else if (key == cut && tie++ < ties) weight[e] = each;
      sum += weight[e];
    }
    const u64 in = wave_scan(sum, lane);
    u64 at = done + in - sum;
    if (at <= want && want < at + sum) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (at <= want && want < at + weight[e]) a.tokens[row] = j + e;
        at += weight[e];
      }
    }
    done += __shfl(in, 63);
    taken += __shfl(scan, 63);
    if (done > want) break;
  }
}

hipError_t launch_sample(const Sample& a, int dtype, hipStream_t st) {
  const dim3 grid((unsigned)a.N), blk(kRowThreads);
  if (dtype == 1) FLCE_LAUNCH((sample_kernel<uint16_t>), grid, blk, 0, st, a);
  else if (dtype == 2) FLCE_LAUNCH((sample_kernel<_Float16>), grid, blk, 0, st, a);
  else FLCE_LAUNCH((sample_kernel<float>), grid, blk, 0, st, a);
  return hipGetLastError();
}

}  // namespace flce
