// Root-mean-square norm with the residual's addition, and its gradients:
//
//   h = x + residual,  n = h rstd,  rstd = (mean_c h^2 + eps)^-1/2,  y = n w
//   dn = dy w,  dx = dresidual = dh + rstd (dn - n mean_c(dn n)),  dw = sum_rows dy n
//
// Each row is read once and stays in its lanes' registers between the sum and the
// scaling, so HBM bounds all of them: the forward reads x and the residual and
// writes h and y, the backward reads h, dy and dh and writes dx.  Sums are fp32; y
// is formed from the fp32 sum h, before h is rounded to the tensors' type, so it
// takes one rounding (an output in 8 or 4 bits comes from the fp32 y).
//
// The backward reads h as it was written: the residual stream in the tensors' type.
// In bf16 that rounding takes the gradients' error from 1.6e-3 (their own rounding
// included) to 2.4e-3; an fp32 copy of h, 8 bytes an element more between forward and
// backward, would take half as long again.  Without a residual h is x and nothing is lost.
//
// A row lies in 8, 64, 256 or 1024 lanes, so that a lane has one to four runs of 8
// columns; longer rows (over 16384 columns) are read twice.  8192 x 4096 bf16: forward
// 47 us (5.7 TB/s of reads and writes), backward 61 (4.4) and 6 for dweight's sums.
#include "layer_mx_device.hpp"

namespace flce {

// Sum over a row's lanes.  Rows of several waves meet in LDS; the two halves of
// red take turns, so one barrier a row is enough.
template <int LANES> __device__ __forceinline__ float row_sum(float v, float* red, int& turn) {
#pragma unroll
  for (int d = 1; d < (LANES < 64 ? LANES : 64); d *= 2) v += __shfl_xor(v, d);
  if constexpr (LANES > 64) {
    constexpr int W = LANES / 64;
    float* r = red + turn * W;
    if ((threadIdx.x & 63) == 0) r[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) v += r[w];
    turn ^= 1;
  }
  return v;
}

// m^-1/2, with a Newton step whose residual 1 - m r^2 is formed from both parts of m r: within 0.51 of the last place
// (1 / sqrtf: twice that).  Where that residual is no number, m is 0 or infinite and r is the limit.
__device__ __forceinline__ float inverse_root(float m) {
  const float r = rsqrtf(m), t = m * r, low = fmaf(m, r, -t);
  const float e = fmaf(-low, r, fmaf(-t, r, 1.f));
  return e == e ? fmaf(0.5f * r, e, r) : r;
}

constexpr int norm_threads(int lanes) { return lanes < 256 ? 256 : lanes; }

// Eight columns, of which `left` are inside the row.  VEC: H % 8 == 0, so all or
// none are (the partial runs' branches cost the long rows their registers).
template <class T, bool VEC> __device__ __forceinline__ void load_run(const T* p, int left, float (&v)[8]) {
  if constexpr (VEC) {
    if (left > 0) {
      load_vec<T, 8>(p, v);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = 0.f;
    }
  } else {
    load_some<T, 8>(p, left, v);
  }
}
template <class T, bool VEC> __device__ __forceinline__ void store_run(T* p, int left, const float (&v)[8]) {
  if constexpr (VEC) {
    if (left > 0) store_vec<T, 8>(p, v);
  } else {
    store_some<T, 8>(p, left, v);
  }
}

// C runs of 8 columns a lane.  OUT: -1 y, else a microscaled format.
template <class T, int OUT, int LANES, int C, bool VEC>
__global__ void __launch_bounds__(norm_threads(LANES)) norm_fwd_kernel(NormFwd a) {
  constexpr int RB = norm_threads(LANES) / LANES;
  __shared__ float red[2 * (LANES > 64 ? LANES / 64 : 1)];
  int turn = 0;
  const int lane = threadIdx.x % LANES, sub = threadIdx.x / LANES;
  float w[C][8];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int col = (c * LANES + lane) * 8;
#pragma unroll
    for (int e = 0; e < 8; ++e) w[c][e] = 1.f;
    if (a.weight) load_run<T, VEC>((const T*)a.weight + col, a.H - col, w[c]);
  }
  const float inv = 1.f / (float)a.H;
  for (int64_t r0 = (int64_t)blockIdx.x * RB; r0 < a.N; r0 += (int64_t)gridDim.x * RB) {
    const int64_t row = r0 + sub, base = row * a.H;
    const bool live = row < a.N;
    float v[C][8];
    float s = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = (c * LANES + lane) * 8, left = live ? a.H - col : 0;
      load_run<T, VEC>((const T*)a.x + base + col, left, v[c]);
      if (a.residual) {
        float t[8];
        load_run<T, VEC>((const T*)a.residual + base + col, left, t);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[c][e] += t[e];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) s = fmaf(v[c][e], v[c][e], s);
    }
    s = row_sum<LANES>(s, red, turn);
    const float rstd = inverse_root(fmaf(s, inv, a.eps));
    if (live && lane == 0 && a.rstd) a.rstd[row] = rstd;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = (c * LANES + lane) * 8, left = live ? a.H - col : 0;
      if (a.h) store_run<T, VEC>((T*)a.h + base + col, left, v[c]);
      float y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = v[c][e] * rstd * w[c][e];
      if constexpr (OUT < 0) {
        store_run<T, VEC>((T*)a.y + base + col, left, y);
      } else {
        // columns past H are zeros, also where rstd is infinite
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = e < left ? y[e] : 0.f;
        mx_store8<OUT>(a.codes, a.scales, row, live ? a.Hp : 0, col, y);
      }
    }
  }
}

// Rows longer than the registers: read twice.  Each element's last read is by the
// thread that writes it, so h may be x or the residual here too.
template <class T, int OUT> __global__ void __launch_bounds__(1024) norm_fwd_long_kernel(NormFwd a) {
  __shared__ float red[32];
  int turn = 0;
  const float inv = 1.f / (float)a.H;
  auto load = [&](int64_t base, int col, float (&v)[8]) {
    load_some<T, 8>((const T*)a.x + base + col, a.H - col, v);
    if (a.residual) {
      float t[8];
      load_some<T, 8>((const T*)a.residual + base + col, a.H - col, t);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] += t[e];
    }
  };
  for (int64_t row = blockIdx.x; row < a.N; row += gridDim.x) {
    const int64_t base = row * a.H;
    float s = 0.f;
    for (int col = threadIdx.x * 8; col < a.H; col += 8192) {
      float v[8];
      load(base, col, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) s = fmaf(v[e], v[e], s);
    }
    s = row_sum<1024>(s, red, turn);
    const float rstd = inverse_root(fmaf(s, inv, a.eps));
    if (threadIdx.x == 0 && a.rstd) a.rstd[row] = rstd;
    const int width = OUT < 0 ? a.H : a.Hp;
    for (int col = threadIdx.x * 8; col < width; col += 8192) {
      float v[8], w[8];
      load(base, col, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = 1.f;
      if (a.weight) load_some<T, 8>((const T*)a.weight + col, a.H - col, w);
      if (a.h) store_some<T, 8>((T*)a.h + base + col, a.H - col, v);
      float y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = v[e] * rstd * w[e];
      if constexpr (OUT < 0) {
        store_some<T, 8>((T*)a.y + base + col, a.H - col, y);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = col + e < a.H ? y[e] : 0.f;
        mx_store8<OUT>(a.codes, a.scales, row, a.Hp, col, y);
      }
    }
  }
}

// A group of lanes keeps its rows' sums of dy n for dweight in registers; the groups of a
// workgroup add theirs in LDS, and norm_dw_kernel the workgroups', all in a fixed order.
// (A sum for each group: 4096 rows of 1024 columns had 2048 of them, 8 us to add up.)
template <class T, int LANES, int C, bool VEC>
__global__ void __launch_bounds__(norm_threads(LANES)) norm_bwd_kernel(NormBwd a) {
  constexpr int RB = norm_threads(LANES) / LANES;
  __shared__ float red[2 * (LANES > 64 ? LANES / 64 : 1)];
  int turn = 0;
  const int lane = threadIdx.x % LANES, sub = threadIdx.x / LANES;
  float dw[C][8] = {};
  const float inv = 1.f / (float)a.H;
  for (int64_t r0 = (int64_t)blockIdx.x * RB; r0 < a.N; r0 += (int64_t)a.parts * RB) {
    const int64_t row = r0 + sub, base = row * a.H;
    const bool live = row < a.N;
    const float rstd = live ? a.rstd[row] : 0.f;
    float n[C][8], d[C][8];
    float s = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = (c * LANES + lane) * 8, left = live ? a.H - col : 0;
      load_run<T, VEC>((const T*)a.h + base + col, left, n[c]);
      load_run<T, VEC>((const T*)a.dy + base + col, left, d[c]);
      float w[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = 1.f;
      if (a.weight) load_run<T, VEC>((const T*)a.weight + col, a.H - col, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        n[c][e] = e < left ? n[c][e] * rstd : 0.f;
        dw[c][e] = fmaf(d[c][e], n[c][e], dw[c][e]);
        d[c][e] *= w[e];
        s = fmaf(d[c][e], n[c][e], s);
      }
    }
    if (a.dx) {
      s = row_sum<LANES>(s, red, turn) * inv;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int col = (c * LANES + lane) * 8, left = live ? a.H - col : 0;
        float t[8] = {};
        if (a.dh) load_run<T, VEC>((const T*)a.dh + base + col, left, t);
#pragma unroll
        for (int e = 0; e < 8; ++e) t[e] = fmaf(rstd, fmaf(-s, n[c][e], d[c][e]), t[e]);
        store_run<T, VEC>((T*)a.dx + base + col, left, t);
      }
    }
  }
  if (a.dweight) {
    if constexpr (RB > 1) {
      __shared__ float group[RB - 1][C][LANES][9];   // 9: lanes start on different banks
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (sub > 0) group[sub - 1][c][lane][e] = dw[c][e];
      __syncthreads();
      if (sub > 0) return;
#pragma unroll
      for (int c = 0; c < C; ++c)
        for (int g = 0; g < RB - 1; ++g)
#pragma unroll
          for (int e = 0; e < 8; ++e) dw[c][e] += group[g][c][lane][e];
    }
    float* p = a.part + (int64_t)blockIdx.x * a.H;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = (c * LANES + lane) * 8;
      store_run<float, VEC>(p + col, a.H - col, dw[c]);
    }
  }
}

template <class T> __global__ void __launch_bounds__(1024) norm_bwd_long_kernel(NormBwd a) {
  __shared__ float red[32];
  int turn = 0;
  const float inv = 1.f / (float)a.H;
  for (int64_t row = blockIdx.x; row < a.N; row += gridDim.x) {
    const int64_t base = row * a.H;
    const float rstd = a.rstd[row];
    float s = 0.f;
    auto load = [&](int col, float (&n)[8], float (&d)[8]) {
      load_some<T, 8>((const T*)a.h + base + col, a.H - col, n);
      load_some<T, 8>((const T*)a.dy + base + col, a.H - col, d);
      float w[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = 1.f;
      if (a.weight) load_some<T, 8>((const T*)a.weight + col, a.H - col, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        n[e] = col + e < a.H ? n[e] * rstd : 0.f;
        d[e] *= w[e];
      }
    };
    for (int col = threadIdx.x * 8; col < a.H; col += 8192) {
      float n[8], d[8];
      load(col, n, d);
#pragma unroll
      for (int e = 0; e < 8; ++e) s = fmaf(d[e], n[e], s);
    }
    s = row_sum<1024>(s, red, turn) * inv;
    for (int col = threadIdx.x * 8; col < a.H; col += 8192) {
      float n[8], d[8], t[8] = {};
      load(col, n, d);
      if (a.dh) load_some<T, 8>((const T*)a.dh + base + col, a.H - col, t);
#pragma unroll
      for (int e = 0; e < 8; ++e) t[e] = fmaf(rstd, fmaf(-s, n[e], d[e]), t[e]);
      store_some<T, 8>((T*)a.dx + base + col, a.H - col, t);
    }
  }
}

// Long rows: sums of dy n over rows blockIdx.y, + parts, ... for 2048 columns.
template <class T> __global__ void __launch_bounds__(256) norm_dw_long_kernel(NormBwd a) {
  const int col = (blockIdx.x * 256 + threadIdx.x) * 8;
  if (col >= a.H) return;
  float dw[8] = {};
  for (int64_t row = blockIdx.y; row < a.N; row += a.parts) {
    float n[8], d[8];
    const float rstd = a.rstd[row];
    load_some<T, 8>((const T*)a.h + row * a.H + col, a.H - col, n);
    load_some<T, 8>((const T*)a.dy + row * a.H + col, a.H - col, d);
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[e] = fmaf(d[e], n[e] * rstd, dw[e]);
  }
  store_some<float, 8>(a.part + (int64_t)blockIdx.y * a.H + col, a.H - col, dw);
}

// dweight from the groups' sums: 64 columns a workgroup, 16 threads a column.
template <class T> __global__ void __launch_bounds__(1024) norm_dw_kernel(NormBwd a) {
  __shared__ float red[16][64];
  const int c = threadIdx.x & 63, g = threadIdx.x >> 6, col = blockIdx.x * 64 + c;
  float s = 0.f;
  if (col < a.H) {
#pragma unroll 8
    for (int p = g; p < a.parts; p += 16) s += a.part[(int64_t)p * a.H + col];
  }
  red[g][c] = s;
  __syncthreads();
  if (g == 0 && col < a.H) {
    s = 0.f;
#pragma unroll
    for (int k = 0; k < 16; ++k) s += red[k][c];
    store1<T>((T*)a.dweight + col, s);
  }
}

// f(lanes, runs of 8 columns a lane) for rows of H columns.
template <bool MX, class F> static void with_row(int H, F&& f) {
  const int lanes = norm_lanes(H, MX), runs = (H + 8 * lanes - 1) / (8 * lanes);
  using std::integral_constant;
  if constexpr (!MX) {
    if (lanes == 8) return f(integral_constant<int, 8>{}, integral_constant<int, 1>{});
  }
  if (lanes == 64) {
    if (runs == 1) return f(integral_constant<int, 64>{}, integral_constant<int, 1>{});
    return f(integral_constant<int, 64>{}, integral_constant<int, 2>{});
  }
  if (lanes == 256) {
    if (runs == 1) return f(integral_constant<int, 256>{}, integral_constant<int, 1>{});
    if (runs == 2) return f(integral_constant<int, 256>{}, integral_constant<int, 2>{});
    return f(integral_constant<int, 256>{}, integral_constant<int, 4>{});
  }
  f(integral_constant<int, 1024>{}, integral_constant<int, 2>{});
}

template <class T, int OUT> static void norm_forward(const NormFwd& a, hipStream_t st) {
  const int width = OUT < 0 ? a.H : a.Hp;
  if (width > kNormMost) {
    FLCE_LAUNCH((norm_fwd_long_kernel<T, OUT>), dim3(a.blocks), dim3(1024), 0, st, a);
    return;
  }
  with_row<(OUT >= 0)>(width, [&](auto lanes, auto runs) {
    const dim3 grid(a.blocks), blk(norm_threads(lanes.value));
    if (a.H % 8 == 0) FLCE_LAUNCH((norm_fwd_kernel<T, OUT, lanes.value, runs.value, true>), grid, blk, 0, st, a);
    else FLCE_LAUNCH((norm_fwd_kernel<T, OUT, lanes.value, runs.value, false>), grid, blk, 0, st, a);
  });
}

template <class T> static hipError_t norm_forward_t(const NormFwd& a, hipStream_t st) {
  if (!a.codes) norm_forward<T, -1>(a, st);
  else if (a.format == kMxE4M3) norm_forward<T, kMxE4M3>(a, st);
  else norm_forward<T, kMxE2M1>(a, st);
  return hipGetLastError();
}

template <class T> static hipError_t norm_backward_t(const NormBwd& a, hipStream_t st) {
  if (a.H > kNormMost) {
    if (a.dx) {
      const int blocks = (int)(a.N < 1024 ? a.N : 1024);
      FLCE_LAUNCH((norm_bwd_long_kernel<T>), dim3(blocks), dim3(1024), 0, st, a);
    }
    if (a.dweight && a.N > 0) FLCE_LAUNCH((norm_dw_long_kernel<T>), dim3((a.H + 2047) / 2048, a.parts), dim3(256), 0, st, a);
  } else if (a.N > 0) {
    with_row<false>(a.H, [&](auto lanes, auto runs) {
      const dim3 grid(a.parts), blk(norm_threads(lanes.value));
      if (a.H % 8 == 0) FLCE_LAUNCH((norm_bwd_kernel<T, lanes.value, runs.value, true>), grid, blk, 0, st, a);
      else FLCE_LAUNCH((norm_bwd_kernel<T, lanes.value, runs.value, false>), grid, blk, 0, st, a);
    });
  }
  if (a.dweight) FLCE_LAUNCH((norm_dw_kernel<T>), dim3((a.H + 63) / 64), dim3(1024), 0, st, a);
  return hipGetLastError();
}

hipError_t launch_rms_norm_forward(const NormFwd& a, int dtype, hipStream_t st) {
  return dtype == 1 ? norm_forward_t<uint16_t>(a, st) : dtype == 2 ? norm_forward_t<_Float16>(a, st) : norm_forward_t<float>(a, st);
}
hipError_t launch_rms_norm_backward(const NormBwd& a, int dtype, hipStream_t st) {
  return dtype == 1 ? norm_backward_t<uint16_t>(a, st) : dtype == 2 ? norm_backward_t<_Float16>(a, st)
                                                                    : norm_backward_t<float>(a, st);
}

}  // namespace flce
