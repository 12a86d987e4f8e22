// Sampling a token from each row of logits: temperature, top-k, top-p, min-p, and the
// draw from a given uniform number.
//
//   w_j = exp((z_j - max) / T), tokens ranked by z from the largest, equal ones by index
//   top-k: the first k;  top-p: of those, each whose predecessors' w is less than p times
//   their sum;  min-p: of those, w_j >= min_p
//   token = the first in the vocabulary's order at which the kept w add up to more than u
//   times their sum
//
// The logits are read once, by as many workgroups as they fill: each takes 8192 tokens
// and leaves their largest, the largest of every 32, and, for rows that need it, the sum
// of their w and, for top-p, its histogram.  Then one workgroup a row finds the tokens
// that can be kept from these alone: the k-th of the groups' largest is not above the
// k-th token, and a histogram says in which bin top-p's nucleus ends.
// It reads these tokens' groups only, and ranks and draws among at most 4096 tokens in
// LDS.  A nucleus of more tokens is drawn from by the histograms (sample_nucleus); what
// else keeps more goes through sample_whole, which reads the row several times.  Rows of
// up to 8192 tokens take one launch: their workgroup finds the groups' largest itself.
//
// HBM bounds the first launch (256 rows of 128256 fp32 logits, 131 MB: 28 us where no
// sums are asked for, 55 with them, 56 to 63 with histograms, whose LDS atomics bound it); the
// second is a chain of barriers and scans in one workgroup a row, 5 us (largest logit), 11
// (top-k 50), 16 (with top-p and min-p), 20 (a nucleus of under 4096 tokens) to 56 (one of
// 20000) and 64 (62000), and up to 71 with all CUs at work.  Rows that go through
// sample_whole take 126 (top-k 5000) and 129 (z / T past the histograms' reach).
//
// Weights are formed in double, to 2^-45.  Where tokens are ranked, they are added as whole
// numbers of 2^-s of the largest, s as large as keeps a row's sum under 2^62: such a
// sum does not depend on its order, so atomics may form it, and every comparison with it
// is exact.  A float32 u tells 2^-24 of the sum apart; all roundings together stay under it:
//   - up to V = 2^18 tokens s = 62 - ceil(log2 V) (45 at 128256): V 2^-(s + 1) <= 2^-27;
//   - in longer rows a list of at most 4096 tokens has s = 44: 2^12 2^-45 = 2^-33;
//   - in a longer row that sample_whole walks, 32 times the weights of the groups' largest
//     bound the sum, and are at most 32 times it.  With that bound in [2^(e - 1), 2^e) s is
//     62 - e: each rounding is 2^-57 of the sum at most, and n tokens kept from the largest
//     down have n / V of it, so all are V 2^-57 <= 2^-27 of what is kept.  (Of the sum itself
//     it would be V 2^-62, for another pass over the row: 5.6 -> 8.0 ms at 8.4 million tokens.)
//   - a histogram's bin holds whole numbers of 2^-40 (2^-38 at 8 million tokens) of the
//     weight at its lower edge, so each weight to 2^-39 of itself.
#include "layer_device.hpp"
#include "layer_launch.hpp"

namespace flce {

typedef unsigned long long u64;

// Order of the values as whole numbers; -0 is 0.
__device__ __forceinline__ uint32_t value_key(float v) {
  const uint32_t b = __float_as_uint(v + 0.f);
  return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) { return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu)); }
constexpr uint32_t kKeyInf = 0xff800000u, kKeyMinusInf = 0x007fffffu, kKeyNan = 0xffffffffu;

// 2^f, |f| <= 1/2, to 2^-45.6: the polynomial of degree 9 through it at the ten Chebyshev
// points (computed in 50 digits).
__device__ __forceinline__ double pow2_near(double f) {
  double p = 1.0205905413765595e-07;
  p = fma(p, f, 1.325964524488711e-06);
  p = fma(p, f, 1.5252672924850737e-05);
  p = fma(p, f, 0.0001540343375125101);
  p = fma(p, f, 0.0013333558200794592);
  p = fma(p, f, 0.009618129193934313);
  p = fma(p, f, 0.05550410866465167);
  p = fma(p, f, 0.2402265069564034);
  p = fma(p, f, 0.6931471805599462);
  return fma(p, f, 1.0000000000000135);
}
// 2^x for x <= 0.  Under 2^-65 it is 0: 2^30 tokens of such a weight would not add 2^-34 of
// the largest.
__device__ __forceinline__ double pow2_negative(double x) {
  const double n = rint(x);
  return x < -65.0 ? 0.0 : __builtin_ldexp(pow2_near(x - n), (int)n);
}
constexpr int kNoBins = -2000000000;   // the first bin of a slice that has no histogram: past every other's bins
constexpr double kLog2eDouble = 1.4426950408889634;
__device__ __forceinline__ double exp_bin(int bins) { return pow2_negative(0.125 * kLog2eDouble * bins); }   // e^(bins / 8), bins <= 0

// Weights relative to a value that is not below any.  unit: 2^s (see above).
struct Weigh {
  float top;
  double scale, unit, min_w;   // scale: log2(e) / T
  __device__ __forceinline__ double real(float z) const {
    // equal to the largest: 1, also where that is infinite; masked: 0, whatever T
    return z == top ? 1.0 : z == -INFINITY || top == INFINITY ? 0.0 : pow2_negative(((double)z - (double)top) * scale);
  }
  __device__ __forceinline__ u64 operator()(float z) const { return (u64)rint(real(z) * unit); }
  __device__ __forceinline__ u64 kept(float z) const {
    const double w = real(z);
    return w >= min_w ? (u64)rint(w * unit) : 0;
  }
};

// A row's parameters.
struct RowParams {
  float T, p, min_p, u;
  int64_t k;   // 0: off
  __device__ __forceinline__ void load(const Sample& a, int64_t row) {
    T = a.temperature ? a.temperature[row] : a.temperature0;
    p = a.top_p ? a.top_p[row] : a.top_p0;
    min_p = a.min_p ? a.min_p[row] : a.min_p0;
    k = a.top_k ? a.top_k[row] : a.top_k0;
    if (k <= 0 || k >= a.V) k = 0;
    u = a.u[row];
  }
  __device__ __forceinline__ bool greedy() const { return !(T > 0.f); }
  __device__ __forceinline__ bool needs_sum() const { return !greedy() && k == 0; }
  // top-p over the whole row; a p that is not above 0 keeps the first token alone
  __device__ __forceinline__ bool needs_histogram() const { return needs_sum() && p < 1.f && p > 0.f; }
};

// Histograms of w: bins of an eighth in z / T, so that all slices' bins fall together; a
// slice keeps the kHistBins below its largest.  A bin holds whole numbers of 2^-s of
// exp(z / T) over its value at the bin's lower edge.
struct Bins {
  double scale;   // bins of a unit of z
  // Whether z / T is small enough for a largest logit z (to 2^-41).  Slices' own may be twice as far from 0, so one that
  // has no histogram lies 4096 below any row's largest that has.
  static __device__ __forceinline__ bool fits(float top, float T, double most) { return fabs((double)top / (double)T) < most; }
  __device__ __forceinline__ double place(float z) const { return (double)z * scale; }
  __device__ __forceinline__ int bin(float z) const { return z > -INFINITY ? (int)fmax(floor(place(z)), -1e9) : -1000000000; }
  // the weight over that at its bin's lower edge, from 1 to e^(1/8)
  __device__ __forceinline__ double over(float z) const {
    const double x = place(z);
    return pow2_near((x - floor(x)) * (0.125 * kLog2eDouble));
  }
};

// v moved over the wave's lanes by a DPP control, 0 where none comes in.
template <int CTRL, int ROWS, class V> __device__ __forceinline__ V moved(V v) {
  if constexpr (sizeof(V) == 8) {
    typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
    u32x2_t t = __builtin_bit_cast(u32x2_t, v);
    t[0] = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)t[0], CTRL, ROWS, 0xF, false);
    t[1] = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)t[1], CTRL, ROWS, 0xF, false);
    return __builtin_bit_cast(V, t);
  } else {
    return (V)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, false);
  }
}
// Inclusive scans over the 16 lanes of a row and over the wave; f's identity is 0.
template <class V, class F> __device__ __forceinline__ V row_scan(V v, F&& f) {
  v = f(v, moved<0x111, 0xF>(v));   // from 1, 2, 4 and 8 lanes below
  v = f(v, moved<0x112, 0xF>(v));
  v = f(v, moved<0x114, 0xF>(v));
  return f(v, moved<0x118, 0xF>(v));
}
template <class V, class F> __device__ __forceinline__ V wave_scan(V v, F&& f) {
  v = row_scan(v, f);
  v = f(v, moved<0x142, 0xA>(v));   // a row's last lane to rows 1 and 3, lane 31 to rows 2 and 3
  return f(v, moved<0x143, 0xC>(v));
}
template <class V> __device__ __forceinline__ V lane_of(V v, int lane) {
  if constexpr (sizeof(V) == 8) {
    typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
    u32x2_t t = __builtin_bit_cast(u32x2_t, v);
    t[0] = (uint32_t)__builtin_amdgcn_readlane((int)t[0], lane);
    t[1] = (uint32_t)__builtin_amdgcn_readlane((int)t[1], lane);
    return __builtin_bit_cast(V, t);
  } else {
    return (V)__builtin_amdgcn_readlane((int)v, lane);
  }
}
struct Add {
  template <class V> __device__ __forceinline__ V operator()(V x, V y) const { return x + y; }
};
struct Max {
  __device__ __forceinline__ uint32_t operator()(uint32_t x, uint32_t y) const { return max(x, y); }
};
template <class V, class F> __device__ __forceinline__ V wave_all(V v, F&& f) { return lane_of(wave_scan(v, f), 63); }

// ---------------------------------------------------------------------------
// The pass over the logits
// ---------------------------------------------------------------------------

// Slice j of a row: 8192 tokens, 32 a thread in four runs of 8; four lanes hold a
// group of 32 consecutive ones.
template <class T> __global__ void __launch_bounds__(256) sample_slice_kernel(Sample a) {
  __shared__ uint32_t red[4];
  __shared__ double sums[4];
  __shared__ u64 hist[kHistBins];
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.x / a.slices;
  const int j = (int)(blockIdx.x - row * a.slices), base = j * kSliceTokens;
  const T* z = (const T*)a.logits + row * a.V + base;
  RowParams r;
  r.load(a, row);
  const int left = a.V - base;
  float v[4][8];
  uint32_t top = 0;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const int at = c * 2048 + tid * 8;
    load_some<T, 8>(z + at, left - at, v[c]);
    uint32_t g = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (at + e < left) g = max(g, v[c][e] != v[c][e] ? kKeyNan : value_key(v[c][e]));
      else v[c][e] = -INFINITY;
    g = max(g, (uint32_t)__shfl_xor((int)g, 1));
    g = max(g, (uint32_t)__shfl_xor((int)g, 2));
    if ((tid & 3) == 0 && at < left) a.group_top[row * a.groups + (base + at) / kGroupTokens] = g;
    top = max(top, g);
  }
  top = wave_all(top, Max());
  if ((tid & 63) == 0) red[tid >> 6] = top;
  __syncthreads();
  top = max(max(red[0], red[1]), max(red[2], red[3]));
  if (tid == 0) a.slice_top[row * a.slices + j] = top;
  if (!r.needs_sum()) return;
  double s = 0.0;
  const bool some = top <= kKeyInf && top > kKeyMinusInf;
  if (r.needs_histogram()) {   // its bins' sum stands for the sum
    int64_t at = row * a.slices + j;
    const float zt = some ? key_value(top) : 0.f;
    const bool fits = some && Bins::fits(zt, r.T, 8192.0);
    const Bins b{8.0 / (double)r.T};
    const int base_bin = fits ? b.bin(zt) - (kHistBins - 1) : kNoBins;
    if (tid == 0) a.slice_bin[at] = base_bin;
    if (!fits) return;
    for (int i = tid; i < kHistBins; i += 256) hist[i] = 0;
    __syncthreads();
    const double unit = (double)(1ull << a.hist_shift);
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int i = b.bin(v[c][e]) - base_bin;
        if (i >= 0) atomicAdd(&hist[i], (u64)rint(b.over(v[c][e]) * unit));
      }
    __syncthreads();
    for (int i = tid; i < kHistBins; i += 256) a.hist[at * kHistBins + i] = hist[i];
    return;
  }
  if (some) {
    const Weigh w{key_value(top), kLog2eDouble / (double)r.T, 1.0, 0.0};
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int e = 0; e < 8; ++e) s += w.real(v[c][e]);
  }
  s = wave_all(s, Add());
  if ((tid & 63) == 0) sums[tid >> 6] = s;
  __syncthreads();
  if (tid == 0) a.slice_sum[row * a.slices + j] = (sums[0] + sums[1]) + (sums[2] + sums[3]);
}

// ---------------------------------------------------------------------------
// One workgroup a row
// ---------------------------------------------------------------------------

constexpr int kRowThreads = 1024, kRowWaves = kRowThreads / 64;
constexpr int kBins = 2048, kMost = 4096, kGroups = 8192;
constexpr int kNucleusMost = 8192, kMaxSlices = 1024;
constexpr int kUnitTokens = 1 << 18;   // of more tokens the unit of weights does not depend on their number
constexpr int kUnits = 2048;   // sample_whole: runs of 512 tokens, or of more in long rows

struct RowLds {
  u64 wave[2][kRowWaves];
  u64 found_above, carried;
  uint32_t found;
  u64 hist[kBins];   // zero between find_key's uses
  int base[kMaxSlices];   // the slices' first bins
  union {
    struct {
      uint32_t group[kGroups];      // largest key of each group; then the groups that pass, in order
      u64 token[kMost];             // key << 32 | index
      u64 weight[kMost];
    } list;
    struct {
      u64 token[kNucleusMost];   // key << 32 | index
      double slice[kMaxSlices];
      u64 extra[kMaxSlices];
      uint32_t equal[kMaxSlices];
    } nucleus;
    struct {
      u64 mass[kUnits];
      uint32_t same[kUnits];
    } whole;
  };
};

// A row's workgroup.  The waves' results lie in LDS by turns in two places, so one
// barrier is enough for each sum.
struct Row {
  RowLds& m;
  int turn;
};

// f over v (8 bytes) of the threads before this one, and of all of them.
template <class V> __device__ __forceinline__ V block_scan(V v, V& all, Row& L) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const V in = wave_scan(v, Add());
  u64* place = L.m.wave[L.turn ^= 1];
  if (lane == 63) place[wave] = __builtin_bit_cast(u64, in);
  __syncthreads();
  const V waves = row_scan(__builtin_bit_cast(V, place[lane & 15]), Add());
  all = lane_of(waves, 15);
  const V before = wave ? lane_of(waves, wave - 1) : V(0);
  return before + moved<0x138, 0xF>(in);   // the lane below's
}
// The largest of a and of b over all threads.
__device__ __forceinline__ void block_max(uint32_t& a, uint32_t& b, Row& L) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  a = wave_scan(a, Max());
  b = wave_scan(b, Max());
  u64* place = L.m.wave[L.turn ^= 1];
  if (lane == 63) place[wave] = (u64)a << 32 | b;
  __syncthreads();
  const u64 w = place[lane & 15];
  a = lane_of(row_scan((uint32_t)(w >> 32), Max()), 15);
  b = lane_of(row_scan((uint32_t)w, Max()), 15);
}
__device__ __forceinline__ uint32_t block_max(uint32_t v, Row& L) {
  uint32_t none = 0;
  block_max(v, none, L);
  return v;
}

// The key at which, from the largest down, the sum of the weights reaches want, and the sum
// above that key; 0 if want is more than their whole sum.  each(f) calls f(key, weight)
// for every element, among all threads; keys lie in [lo, hi].  Each level splits the
// keys' range into 2048 bins; coarse: the first level's bin's lowest key.
template <class F>
__device__ __forceinline__ uint32_t find_key(uint32_t lo, uint32_t hi, u64 want, u64& above, F&& each, Row& L, bool coarse = false) {
  above = 0;
#pragma unroll 1
  while (true) {
    const int bits = hi > lo ? 32 - __clz((int)(hi - lo)) : 0, shift = bits > 11 ? bits - 11 : 0;
    each([&](uint32_t k, u64 w) {
      if (k >= lo && k <= hi && w) atomicAdd(&L.m.hist[(k - lo) >> shift], w);
    });
    __syncthreads();
    // thread t has bins 2047 - 2 t and the one below it, and leaves them empty
    const int top = kBins - 1 - 2 * (int)threadIdx.x;
    const u64 a = L.m.hist[top], b = L.m.hist[top - 1];
    L.m.hist[top] = 0;
    L.m.hist[top - 1] = 0;
    u64 all;
    const u64 before = above + block_scan(a + b, all, L);
    if (above + all < want) return 0;
    if (before < want && before + a + b >= want) {
      const bool first = before + a >= want;
      L.m.found = first ? top : top - 1;
      L.m.found_above = first ? before : before + a;
    }
    __syncthreads();
    above = L.m.found_above;
    lo += L.m.found << shift;
    if (shift == 0 || coarse) return lo;
    hi = min(hi, lo + ((1u << shift) - 1));
  }
}

// What of `ties` equal tokens of weight `each` top-p keeps: the sum before them is above,
// and those whose predecessors' sum is under want stay (at least one does).
__device__ __forceinline__ u64 ties_needed(u64 want, u64 above, u64 each) { return (want - above + each - 1) / each; }

// top-p's sum that predecessors have to stay under, a whole number: at least 1, or 0 if only the
// first token is kept.
__device__ __forceinline__ u64 nucleus(float p, double all) {
  const double want = p > 0.f ? ceil((double)p * all) : 0.0;
  return want < 1.0 ? 0 : (u64)want;
}

// Which of the kept weights' sum the draw has to pass: u times it, under it.
__device__ __forceinline__ u64 spot(float u, u64 all) {
  const double s = u > 0.f ? floor((double)u * (double)all) : 0.0;
  return s < (double)all ? min((u64)s, all - 1) : all - 1;
}

// f(value, index) over the row's tokens, 8 a lane at a time, by all threads.
template <class T, class F> __device__ __forceinline__ void each_token(const T* z, int V, F&& f) {
  for (int j = threadIdx.x * 8; j < V; j += kRowThreads * 8) {
    float v[8];
    load_some<T, 8>(z + j, V - j, v);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (j + e < V) f(v[e], j + e);
  }
}

// Tokens of the row that stay, in order, as (key << 32 | index) in list: of runs of 8 tokens, run c from at(c) on (in
// order), those that keep(value, index) says.  Returns their number; of more than MOST only that.
//
// Each wave takes a stretch of the runs and writes what it finds to a 16th of the list; the parts are then moved
// together.  If a wave finds more than its part holds, all walk a second time and write to the final places.
template <class T, int MOST, class At, class Keep>
__device__ __forceinline__ uint32_t collect(const T* z, int V, int runs, u64* list, At&& at, Keep&& keep, Row& L) {
  constexpr int U = 2;   // runs a lane has under way
  constexpr uint32_t kPart = MOST / kRowWaves;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int share = (runs + 64 * U * kRowWaves - 1) / (64 * U * kRowWaves) * (64 * U);
  const int c0 = min(runs, wave * share), c1 = min(runs, c0 + share);
  // to list[first + i] for i under `room`; returns how many there are
  auto walk = [&](uint32_t first, uint32_t room) {
    uint32_t n = 0;
#pragma unroll 1
    for (int c = c0; c < c1; c += 64 * U) {
      float v[U][8];
      int j[U];
#pragma unroll
      for (int q = 0; q < U; ++q) {
        const int run = c + 64 * q + lane;
        j[q] = run < c1 ? at(run) : V;
        load_some<T, 8>(z + min(j[q], V), V - j[q], v[q]);
      }
#pragma unroll
      for (int q = 0; q < U; ++q) {
        uint32_t hits = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) hits |= (uint32_t)(j[q] + e < V && keep(v[q][e], j[q] + e)) << e;
        if (!__ballot(hits != 0)) continue;
        const uint32_t own = (uint32_t)__popc(hits), in = wave_scan(own, Add());
        uint32_t i = n + in - own;
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (hits >> e & 1) {
            if (i < room) list[first + i] = (u64)value_key(v[q][e]) << 32 | (uint32_t)(j[q] + e);
            ++i;
          }
        n += lane_of(in, 63);
      }
    }
    return n;
  };
  __syncthreads();
  const uint32_t n = walk(wave * kPart, kPart);
  // the waves' numbers, and what the ones before have
  u64 total;
  const uint32_t start = (uint32_t)lane_of(block_scan((u64)(lane == 0 ? n : 0u), total, L), 0);
  if (total > MOST) return (uint32_t)min(total, (u64)0xffffffffu);
  const bool over = block_max(n, L) > kPart;
  if (over) {
    walk(start, MOST);
    __syncthreads();
    return (uint32_t)total;
  }
  u64 own[kPart / 64];
#pragma unroll
  for (uint32_t k = 0; k < kPart / 64; ++k) own[k] = list[wave * kPart + 64 * k + lane];
  __syncthreads();
#pragma unroll
  for (uint32_t k = 0; k < kPart / 64; ++k)
    if (64 * k + lane < n) list[start + 64 * k + lane] = own[k];
  __syncthreads();
  return (uint32_t)total;
}

// A row with any number of tokens to keep, read from memory in every pass.
template <class T>
__device__ __forceinline__ void sample_whole(const Sample& a, int64_t row, const RowParams& r, Weigh w, uint32_t top, Row& L) {
  const T* z = (const T*)a.logits + row * a.V;
  const int V = a.V, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  if (V > kUnitTokens) {   // the unit by a bound on the row's sum: 32 at least, under 2^36
    double own = 0.0, bound;
    for (int i = tid; i < a.groups; i += kRowThreads) own += w.real(key_value(a.group_top[row * a.groups + i]));
    block_scan(own, bound, L);
    w.unit = __builtin_ldexp(1.0, 61 - ilogb(kGroupTokens * bound));
  }
  // Tokens above key `cut` are kept and the first `ties` at it.
  uint32_t cut = 0;
  u64 ties = 0;
  if (r.k) {
    u64 above;
    cut = find_key(kKeyMinusInf, top, (u64)r.k, above, [&](auto&& f) { each_token(z, V, [&](float v, int) { f(value_key(v), 1ull); }); }, L);
    ties = (u64)r.k - above;
  }
  if (r.p < 1.f) {
    u64 sum = 0, all;
    each_token(z, V, [&](float v, int) { sum += value_key(v) > cut ? w(v) : 0; });
    block_scan(sum, all, L);
    const u64 at_cut = cut ? ties * w(key_value(cut)) : 0;
    all += at_cut;
    const u64 want = min(nucleus(r.p, (double)all), all);
    if (want == 0) {
      cut = top;
      ties = 1;
    } else {
      u64 above;
      const uint32_t was = cut;
      cut = find_key(max(cut, kKeyMinusInf), top, want, above, [&](auto&& f) {
        each_token(z, V, [&](float v, int) {
          const uint32_t k = value_key(v);
          if (k > was) f(k, w(v));
        });
        if (tid == 0 && at_cut) f(was, at_cut);
      }, L);
      const u64 need = ties_needed(want, above, w(key_value(cut)));
      ties = cut == was ? min(ties, need) : need;
    }
  }
  __syncthreads();

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
    m = wave_all(m, Add());
    same = wave_all(same, Add());
    if (lane == 0) {
      L.m.whole.mass[i] = m;
      L.m.whole.same[i] = same;
    }
  }
  __syncthreads();
  const u64 each = cut ? w.kept(key_value(cut)) : 0;
  // Each thread two units: their kept weight with the ties that the units before leave them.
  u64 m[2] = {0, 0}, n[2] = {0, 0}, all;
#pragma unroll
  for (int h = 0; h < 2; ++h)
    if (2 * tid + h < units) n[h] = L.m.whole.same[2 * tid + h];
  u64 before = block_scan(n[0] + n[1], all, L);
  u64 used[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    used[h] = min(before, ties);
    if (2 * tid + h < units) m[h] = L.m.whole.mass[2 * tid + h] + min(n[h], ties - used[h]) * each;
    before += n[h];
  }
  before = block_scan(m[0] + m[1], all, L);
  const u64 want = spot(r.u, all);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (before <= want && want < before + m[h]) {
      L.m.found = 2 * tid + h;
      L.m.found_above = before;
      L.m.carried = used[h];
    }
    before += m[h];
  }
  __syncthreads();
  // The first wave walks the unit, 512 tokens at a time.
  if (wave > 0) return;
  const int i = L.m.found;
  u64 done = L.m.found_above, taken = L.m.carried;
  for (int j0 = i * unit; j0 < min(V, (i + 1) * unit); j0 += 512) {
    const int j = j0 + lane * 8;
    float v[8];
    load_some<T, 8>(z + j, V - j, v);
    u64 same = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) same += j + e < V && value_key(v[e]) == cut;
    const u64 scan = wave_scan(same, Add());
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
    const u64 in = wave_scan(sum, Add());
    u64 at = done + in - sum;
    if (at <= want && want < at + sum) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (at <= want && want < at + weight[e]) a.tokens[row] = j + e;
        at += weight[e];
      }
    }
    done += lane_of(in, 63);
    taken += lane_of(scan, 63);
    if (done > want) break;
  }
}

// A row that nothing is cut off from: the slice in which u times the whole sum lies, then the token in it.  The
// sums are doubles in a fixed order; where their rounding leaves the spot past a slice's last token, that is taken.
template <class T>
__device__ __forceinline__ void sample_slices(const Sample& a, int64_t row, const RowParams& r, const Weigh& w, Row& L) {
  const T* z = (const T*)a.logits + row * a.V;
  const int tid = threadIdx.x;
  // thread t takes slices per t .. per (t + 1) - 1
  const int per = (a.slices + kRowThreads - 1) / kRowThreads;
  auto mass = [&](int j) {
    const uint32_t top = a.slice_top[row * a.slices + j];
    return top <= kKeyMinusInf ? 0.0 : a.slice_sum[row * a.slices + j] * w.real(key_value(top));
  };
  double own = 0.0, all;
  for (int j = tid * per; j < min(a.slices, (tid + 1) * per); ++j) own += mass(j);
  double before = block_scan(own, all, L);
  const double u = r.u > 0.f ? (double)r.u : 0.0, want = u * all;
  // the last slice with any weight, should the spot lie past all
  uint32_t last = 0;
  double b = before;
  for (int j = tid * per; j < min(a.slices, (tid + 1) * per); ++j) {
    const double m = mass(j);
    if (m > 0.0) last = j + 1;
    b += m;
  }
  last = block_max(last, L);
  if (tid == 0) L.m.found = 0;
  __syncthreads();
  // the first slice at whose end the sum is past the spot
  b = before;
  for (int j = tid * per; j < min(a.slices, (tid + 1) * per); ++j) {
    const double m = mass(j);
    if (m > 0.0 && b + m > want) {
      atomicMax(&L.m.found, 0x80000000u - (uint32_t)j);
      break;
    }
    b += m;
  }
  __syncthreads();
  const bool past = L.m.found == 0;
  const int j = past ? (int)last - 1 : (int)(0x80000000u - L.m.found);
  // what the slices before it add up to, as its thread had it
  __syncthreads();
  if (tid == j / per) {
    double s = before;
    for (int i = tid * per; i < j; ++i) s += mass(i);
    L.m.found_above = __builtin_bit_cast(u64, s);
  }
  __syncthreads();
  const double rest = past ? INFINITY : want - __builtin_bit_cast(double, L.m.found_above);
  // 8 tokens a thread
  const int at = j * kSliceTokens + tid * 8;
  float v[8];
  load_some<T, 8>(z + at, a.V - at, v);
  double q[8], sum = 0.0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    q[e] = at + e < a.V ? w.real(v[e]) : 0.0;
    sum += q[e];
  }
  double whole;
  double cum = block_scan(sum, whole, L);
  uint32_t first = 0, end = 0;   // as 2^31 less the index, and the index + 1
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    cum += q[e];
    if (q[e] > 0.0) {
      end = at + e + 1;
      if (cum > rest && first == 0) first = 0x80000000u - (uint32_t)(at + e);
    }
  }
  first = block_max(first, L);
  end = block_max(end, L);
  if (tid == 0) a.tokens[row] = first ? (int64_t)(0x80000000u - first) : (int64_t)end - 1;
}

// Where top-p's nucleus ends, from the histograms of the row's slices.
struct Nucleus {
  int top_bin, last;   // it ends in bin top_bin - last
  double sum;          // of w, relative to the largest token's
  double rest;         // what that bin has to give, relative to top_bin's lower edge, in 2^-hist_shift
};
// False: z / T is too large for histograms, or the row has too many slices (or a sum's rounding fell between two bins).
__device__ __forceinline__ bool find_nucleus(const Sample& a, int64_t row, const RowParams& r, float top, Nucleus& n, Row& L) {
  if (a.slices > kMaxSlices || !Bins::fits(top, r.T, 4096.0)) return false;
  const int tid = threadIdx.x, J = a.slices;
  const Bins b{8.0 / (double)r.T};
  n.top_bin = b.bin(top);
  const u64* H = a.hist + row * J * kHistBins;
  if (tid < J) L.m.base[tid] = a.slice_bin[row * J + tid];
  if (tid == 0) L.m.found = kHistBins;
  __syncthreads();
  // Thread t sums bin top_bin - t over the slices: a whole number of at most 2^62.  Bins are weighted relative to
  // top_bin's lower edge.
  u64 count = 0;
  if (tid < kHistBins)
#pragma unroll 4
    for (int j = 0; j < J; ++j) {
      const int base = L.m.base[j], i = n.top_bin - tid - base;
      if (i >= 0 && i < kHistBins) count += H[(int64_t)j * kHistBins + i];
    }
  const double mass = (double)count * exp_bin(-tid);
  double all;
  const double before = block_scan(mass, all, L), need = (double)r.p * all;
  if (count && before < need && before + mass >= need) {
    L.m.found = tid;
    L.m.found_above = __builtin_bit_cast(u64, before);
  }
  __syncthreads();
  n.last = L.m.found;
  n.rest = need - __builtin_bit_cast(double, L.m.found_above);
  n.sum = all / (b.over(top) * (double)(1ull << a.hist_shift));
  return n.last < kHistBins;
}

// top-p (and min-p) over a row whose nucleus has more tokens than the list holds: the tokens of the bin in which it ends
// are listed and ranked, and the slice that the draw falls into is read once more.  False: the bin has too many tokens.
template <class T>
__device__ __forceinline__ bool sample_nucleus(const Sample& a, int64_t row, const RowParams& r, const Weigh& w, const Nucleus& nuc, Row& L) {
  const T* z = (const T*)a.logits + row * a.V;
  const int V = a.V, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, J = a.slices;
  const Bins b{8.0 / (double)r.T};
  const int top_bin = nuc.top_bin;
  const double unit = (double)(1ull << a.hist_shift);
  const u64* H = a.hist + row * J * kHistBins;
  int last = nuc.last;
  double all;
  __syncthreads();
  // min-p may end higher up: then it alone cuts the bin in which it does
  bool ranked = true;
  if (w.min_w > 0.0) {
    const double x = b.place(w.top) + 8.0 * log(w.min_w), f = floor(x);
    if (x - f < 1e-6 || x - f > 1.0 - 1e-6) return false;   // an edge that rounding could move
    if (top_bin - (int)f < last) {
      last = top_bin - (int)f;
      ranked = false;
    }
  }
  const int edge = top_bin - last;   // the bin itself

  // Its tokens, in order.
  const float lo = (float)(((double)edge - 0.01) / b.scale), hi = (float)(((double)edge + 1.01) / b.scale);   // around it
  const uint32_t found = collect<T, kNucleusMost>(z, V, (V + 7) / 8, L.m.nucleus.token, [](int c) { return 8 * c; },
                                                  [&](float v, int) {
                                                    const bool near = v >= lo && v <= hi;
                                                    return __ballot(near) ? near && b.bin(v) == edge : false;
                                                  }, L);
  if (found > kNucleusMost) return false;
  const int listed = (int)found;
  auto key_of = [&](int i) { return (uint32_t)(L.m.nucleus.token[i] >> 32); };
  auto weight = [&](uint32_t key) { return (u64)rint(b.over(key_value(key)) * unit); };
  uint32_t cut = 0;
  u64 ties = 0;
  if (ranked && listed > 0) {
    u64 own = 0, sum;
    uint32_t most = 0, least = 0;
    for (int i = tid; i < listed; i += kRowThreads) {
      own += weight(key_of(i));
      most = max(most, key_of(i));
      least = max(least, ~key_of(i));
    }
    block_scan(own, sum, L);
    most = block_max(most, L);
    least = ~block_max(least, L);
    const double want_real = ceil(nuc.rest / exp_bin(-last));
    const u64 want = min(want_real < 1.0 ? 1ull : (u64)want_real, sum);
    u64 above;
    cut = find_key(least, most, want, above, [&](auto&& f) {
      for (int i = tid; i < listed; i += kRowThreads) f(key_of(i), weight(key_of(i)));
    }, L);
    ties = ties_needed(want, above, weight(cut));
  }
  auto passes = [&](uint32_t key) { return w.min_w == 0.0 || w.real(key_value(key)) >= w.min_w; };

  // Kept mass of each slice: its bins above, and the listed tokens that stay.
  __syncthreads();
  if (tid < J) {
    L.m.nucleus.extra[tid] = 0;
    L.m.nucleus.equal[tid] = 0;
  }
  __syncthreads();
  {
    // ties in order: thread t has tokens per t .. per (t + 1) - 1 of the list
    const int per = (listed + kRowThreads - 1) / kRowThreads;
    u64 same = 0, none;
    for (int i = tid * per; i < min(listed, (tid + 1) * per); ++i) same += key_of(i) == cut;
    u64 tie = block_scan(same, none, L);
    for (int i = tid * per; i < min(listed, (tid + 1) * per); ++i) {
      const uint32_t k = key_of(i);
      const int j = (int)((uint32_t)L.m.nucleus.token[i] / kSliceTokens);
      bool keep = k > cut;
      if (k == cut) {
        atomicAdd(&L.m.nucleus.equal[j], 1u);
        keep = tie++ < ties;
      }
      if (keep && passes(k)) atomicAdd(&L.m.nucleus.extra[j], weight(k));
    }
  }
  __syncthreads();
  // a wave a slice
  for (int j = wave; j < J; j += kRowWaves) {
    const int base = L.m.base[j];
    double m = 0.0;
    if (base != kNoBins)
      for (int i = lane; i < kHistBins; i += 64)
        if (base + i > edge) m += (double)H[(int64_t)j * kHistBins + i] * exp_bin(base + i - top_bin);
    m = wave_all(m, Add());
    if (lane == 0) L.m.nucleus.slice[j] = m + (double)L.m.nucleus.extra[j] * exp_bin(-last);
  }
  __syncthreads();
  double own = tid < J ? L.m.nucleus.slice[tid] : 0.0, kept;
  const u64 equal = tid < J ? L.m.nucleus.equal[tid] : 0;
  const double sum_before = block_scan(own, kept, L);
  u64 equals;
  const u64 equal_before = block_scan(equal, equals, L);
  const double spot = (r.u > 0.f ? (double)r.u : 0.0) * kept;
  uint32_t at = block_max(own > 0.0 && sum_before + own > spot ? kMaxSlices - tid : 0, L);
  const uint32_t end = block_max(own > 0.0 ? tid + 1 : 0, L);
  if (end == 0) return false;   // not reached: the largest token is kept
  const bool past = at == 0;
  const int slice = past ? (int)end - 1 : kMaxSlices - (int)at;
  __syncthreads();
  if (tid == slice) {
    L.m.found_above = __builtin_bit_cast(u64, sum_before);
    L.m.carried = equal_before;
  }
  __syncthreads();
  const double left = past ? INFINITY : spot - __builtin_bit_cast(double, L.m.found_above);
  u64 tie = L.m.carried;
  // 8 tokens a thread
  const int t0 = slice * kSliceTokens + tid * 8;
  float v[8];
  load_some<T, 8>(z + t0, V - t0, v);
  u64 same = 0, none;
#pragma unroll
  for (int e = 0; e < 8; ++e) same += t0 + e < V && value_key(v[e]) == cut;
  tie += block_scan(same, none, L);
  double q[8], sum = 0.0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    q[e] = 0.0;
    if (t0 + e >= V) continue;
    const int bin = b.bin(v[e]);
    const uint32_t k = value_key(v[e]);
    bool keep = bin > edge;
    if (bin == edge) {
      keep = k > cut || (k == cut && tie < ties);
      keep = keep && passes(k);
    }
    tie += k == cut;
    if (keep) q[e] = rint(b.over(v[e]) * unit) * exp_bin(bin - top_bin);
    sum += q[e];
  }
  double cum = block_scan(sum, all, L);
  uint32_t token = 0, tail = 0;   // as 2^31 less the index, and the index + 1
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    cum += q[e];
    if (q[e] > 0.0) {
      tail = t0 + e + 1;
      if (cum > left && token == 0) token = 0x80000000u - (uint32_t)(t0 + e);
    }
  }
  token = block_max(token, L);
  tail = block_max(tail, L);
  if (tid == 0) a.tokens[row] = token ? (int64_t)(0x80000000u - token) : (int64_t)tail - 1;
  return true;
}

// GROUPS: the groups' largest come from sample_slice_kernel; else the workgroup finds them.
template <class T, bool GROUPS> __global__ void __launch_bounds__(kRowThreads) sample_row_kernel(Sample a) {
  __shared__ RowLds lds;
  Row L{lds, 0};
  const int64_t row = blockIdx.x;
  const T* z = (const T*)a.logits + row * a.V;
  const int V = a.V, tid = threadIdx.x, lane = tid & 63;
  RowParams r;
  r.load(a, row);
  L.m.hist[tid] = 0;
  L.m.hist[tid + kRowThreads] = 0;
  // Groups of `size` tokens, so many that their largest fit in LDS.
  int size = kGroupTokens;
  while ((V + size - 1) / size > kGroups) size *= 2;
  const int groups = (V + size - 1) / size, merge = size / kGroupTokens;
  uint32_t top = 0, under = 0;   // under: the complement of the least group that a mask left
  if constexpr (GROUPS) {
    for (int i = tid; i < groups; i += kRowThreads) {
      uint32_t g = 0;
      for (int m = i * merge; m < min(a.groups, (i + 1) * merge); ++m) g = max(g, a.group_top[row * a.groups + m]);
      L.m.list.group[i] = g;
      top = max(top, g);
      under = max(under, g > kKeyMinusInf ? ~g : 0u);
    }
  } else {
    for (int j0 = 0; j0 < V; j0 += kRowThreads * 8) {
      const int j = j0 + tid * 8;
      float v[8];
      load_some<T, 8>(z + j, V - j, v);
      uint32_t g = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (j + e < V) g = max(g, v[e] != v[e] ? kKeyNan : value_key(v[e]));
      g = max(g, (uint32_t)__shfl_xor((int)g, 1));
      g = max(g, (uint32_t)__shfl_xor((int)g, 2));
      if ((tid & 3) == 0 && j < V) L.m.list.group[j / kGroupTokens] = g;
      top = max(top, g);
      under = max(under, g > kKeyMinusInf && j < V ? ~g : 0u);
    }
  }
  block_max(top, under, L);
  if (top > kKeyInf || top <= kKeyMinusInf) {   // a NaN, or no token left
    if (tid == 0) a.tokens[row] = -1;
    return;
  }
  const int most = min(V, kUnitTokens), s = 62 - (most > 2 ? 32 - __clz(most - 1) : 1);   // most 2^s <= 2^62
  const Weigh w{key_value(top), kLog2eDouble / (double)r.T, (double)(1ull << s),
                r.min_p > 0.f ? (double)fminf(r.min_p, 1.f) : 0.0};

  if (r.greedy() || r.p <= 0.f) {   // the first token of the first group that has the largest
    uint32_t g = 0;
    for (int i = tid; i < groups; i += kRowThreads)
      if (L.m.list.group[i] == top) g = max(g, (uint32_t)(kGroups - i));
    g = kGroups - block_max(g, L);
    if (tid >= 64) return;
    for (int j0 = (int)g * size; j0 < V; j0 += 64) {
      const int j = j0 + lane;
      const u64 hit = __ballot(j < V && value_key(load1<T>(z + min(j, V - 1))) == top);
      if (hit) {
        if (lane == 0) a.tokens[row] = j0 + __ffsll((long long)hit) - 1;
        return;
      }
    }
    return;
  }

  // Every token that can be kept has a key of at least `low`.
  uint32_t low = 0;
  double whole = 0.0;   // the row's sum of w, for top-p without top-k
  Nucleus nuc;
  bool binned = false;  // top-p's end is known from histograms
  if (r.k) {
    // a key that k of the groups' largest reach, and few more
    if (r.k <= groups) {
      u64 above;
      low = find_key(~under, top, (u64)r.k, above, [&](auto&& f) {
        for (int g = tid; g < groups; g += kRowThreads) f(L.m.list.group[g], 1ull);
      }, L, true);
    }
  } else {
    if (GROUPS && !(r.p < 1.f) && w.min_w == 0.0) return sample_slices<T>(a, row, r, w, L);
    if (w.top == INFINITY) {
      low = kKeyInf;
      if (r.p < 1.f) {   // the sum is a number of tokens
        u64 own = 0, all;
        each_token(z, V, [&](float v, int) { own += v == INFINITY; });
        block_scan(own, all, L);
        whole = (double)all;
      }
    } else {
      double cut = w.min_w > 0.0 ? (double)w.top + (double)r.T * log(w.min_w) : -INFINITY;   // no token under it is kept
      if (r.p < 1.f) {
        if constexpr (GROUPS) {
          if (!find_nucleus(a, row, r, w.top, nuc, L)) return sample_whole<T>(a, row, r, w, top, L);
          binned = true;
          whole = nuc.sum;
          cut = fmax(cut, (double)(nuc.top_bin - nuc.last) * ((double)r.T * 0.125));
        } else {
          double own = 0.0;
          each_token(z, V, [&](float v, int) { own += w.real(v); });
          block_scan(own, whole, L);
          cut = fmax(cut, (double)w.top + (double)r.T * log(fmin((1.0 - (double)r.p) * whole / V, 1.0)));
        }
      }
      // with a margin for the rounding of all this
      cut -= 1e-6 * (fabs(cut) + fabs((double)w.top)) + 1e-9 * (double)r.T;
      if (cut > -3e38) low = value_key(fminf((float)cut, w.top));
    }
  }
  low = max(low, kKeyMinusInf + 1);   // masked tokens have no weight

  // The groups that have such tokens, in order, in place: thread t looks at `per` consecutive ones.
  const int per = (groups + kRowThreads - 1) / kRowThreads;
  uint32_t pass = 0;   // bits: at most 8 groups a thread
  __syncthreads();
  for (int i = 0; i < per; ++i)
    if (tid * per + i < groups && L.m.list.group[tid * per + i] >= low) pass |= 1u << i;
  u64 found;
  u64 at = block_scan((u64)__popc(pass), found, L);
  __syncthreads();
  for (int i = 0; i < per; ++i)
    if (pass >> i & 1) L.m.list.group[at++] = tid * per + i;
  __syncthreads();
  // Of so many groups' tokens the list would hardly hold those that stay (independent ones: 3% of the row's).
  if (binned && found * 20 > (u64)groups * 13) {
    if (!sample_nucleus<T>(a, row, r, w, nuc, L)) sample_whole<T>(a, row, r, w, top, L);   // (its list lies where the groups did)
    return;
  }
  // Their tokens, in order.
  const int runs = size / 8, shift = 31 - __clz(runs);
  const uint32_t total = collect<T, kMost>(z, V, (int)found << shift, L.m.list.token,
                                           [&](int c) { return (int)L.m.list.group[c >> shift] * size + (c & (runs - 1)) * 8; },
                                           [&](float v, int) { return value_key(v) >= low; }, L);
  if (total > kMost) {
    if (binned && sample_nucleus<T>(a, row, r, w, nuc, L)) return;
    return sample_whole<T>(a, row, r, w, top, L);
  }
  for (int i = tid; i < (int)total; i += kRowThreads) L.m.list.weight[i] = w(key_value((uint32_t)(L.m.list.token[i] >> 32)));
  __syncthreads();

  // Tokens above key `cut` are kept and the first `ties` at it.
  const int count = (int)total;
  auto key_at = [&](int i) { return (uint32_t)(L.m.list.token[i] >> 32); };
  uint32_t cut = 0;
  u64 ties = 0;
  if (r.k && r.k < count) {
    u64 above;
    cut = find_key(low, top, (u64)r.k, above, [&](auto&& f) {
      for (int i = tid; i < count; i += kRowThreads) f(key_at(i), 1ull);
    }, L);
    ties = (u64)r.k - above;
  }
  if (r.p < 1.f) {
    u64 sum = 0, all;
    for (int i = tid; i < count; i += kRowThreads)
      if (key_at(i) > cut) sum += L.m.list.weight[i];
    block_scan(sum, all, L);
    const u64 at_cut = cut ? ties * w(key_value(cut)) : 0;
    all += at_cut;
    const u64 want = min(nucleus(r.p, r.k ? (double)all : whole * w.unit), all);
    if (want == 0) {
      cut = top;
      ties = 1;
    } else {
      u64 above;
      const uint32_t was = cut;
      cut = find_key(low, top, want, above, [&](auto&& f) {
        for (int i = tid; i < count; i += kRowThreads)
          if (key_at(i) > was) f(key_at(i), L.m.list.weight[i]);
        if (tid == 0 && at_cut) f(was, at_cut);
      }, L);
      const u64 need = ties_needed(want, above, w(key_value(cut)));
      ties = cut == was ? min(ties, need) : need;
    }
  }
  // The draw: thread t has tokens 4 t .. 4 t + 3 of the list.
  u64 same = 0, none;
#pragma unroll
  for (int e = 0; e < 4; ++e) same += 4 * tid + e < count && key_at(4 * tid + e) == cut;
  u64 tie = block_scan(same, none, L);
  u64 weight[4], sum = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int i = 4 * tid + e;
    weight[e] = 0;
    if (i >= count) continue;
    const uint32_t k = key_at(i);
    if (k > cut || (k == cut && tie++ < ties))
      weight[e] = w.min_w == 0.0 || w.real(key_value(k)) >= w.min_w ? L.m.list.weight[i] : 0;
    sum += weight[e];
  }
  u64 all;
  u64 before = block_scan(sum, all, L);
  const u64 want = spot(r.u, all);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (before <= want && want < before + weight[e]) a.tokens[row] = (uint32_t)L.m.list.token[4 * tid + e];
    before += weight[e];
  }
}

template <class T> static hipError_t sample_launch(const Sample& a, hipStream_t st) {
  if (a.slices) {
    FLCE_LAUNCH((sample_slice_kernel<T>), dim3((unsigned)(a.N * a.slices)), dim3(256), 0, st, a);
    FLCE_LAUNCH((sample_row_kernel<T, true>), dim3((unsigned)a.N), dim3(kRowThreads), 0, st, a);
  } else {
    FLCE_LAUNCH((sample_row_kernel<T, false>), dim3((unsigned)a.N), dim3(kRowThreads), 0, st, a);
  }
  return hipGetLastError();
}

hipError_t launch_sample(const Sample& a, int dtype, hipStream_t st) {
  return dtype == 1 ? sample_launch<uint16_t>(a, st) : dtype == 2 ? sample_launch<_Float16>(a, st) : sample_launch<float>(a, st);
}

}  // namespace flce
