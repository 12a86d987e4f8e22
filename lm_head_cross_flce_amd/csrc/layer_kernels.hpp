// Kernels of the linear layer, y = act(x W^T + b) + residual, and of the gated
// product, h = act(x Wg^T + bg) * (x Wu^T + bu), with their gradients, for one
// element type T (each type is its own translation unit).
//
// Many tokens: the products run on MFMA tiles of one of three sizes, with the activation, product and residual in the epilogue,
// while the accumulators are still in registers.  MFMA bounds them.
// Few tokens: every weight is read once for a few rows of x, so HBM bounds the
// call and a kernel that streams weights past them runs instead.
#pragma once

#include "layer_device.hpp"

namespace flce {

// Eight elements of a padded row a thread.
template <class T> __global__ void __launch_bounds__(256) layer_pad_kernel(LayerPad a) {
  const int pieces = a.width / 8;
  const int64_t all = (a.rows[0] + a.rows[1] + a.rows[2]) * pieces;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < all; i += (int64_t)gridDim.x * 256) {
    int64_t row = i / pieces;
    const int h = (int)(i - row * pieces) * 8;
    const T* src = (const T*)a.src[0];
    if (row >= a.rows[0]) {
      row -= a.rows[0];
      src = (const T*)a.src[1];
      if (row >= a.rows[1]) {
        row -= a.rows[1];
        src = (const T*)a.src[2];
      }
    }
    float v[8];
    load_some<T, 8>(src + row * a.H + h, a.H - h, v);
    store_vec<T, 8>((T*)a.dst + i * 8, v);
  }
}

template <class T> static hipError_t layer_pad(const LayerPad& a, hipStream_t st) {
  const int64_t blocks = ((a.rows[0] + a.rows[1] + a.rows[2]) * (a.width / 8) + 255) / 256;
  FLCE_LAUNCH((layer_pad_kernel<T>), dim3((unsigned)(blocks < 4096 ? blocks : 4096)), dim3(256), 0, st, a);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Forward, tiles
// ---------------------------------------------------------------------------

// Workgroup w computes tiles w, w + grid, ... of the tokens x features plane
// (times the K parts).  Tokens are the MFMA rows and features its columns, in
// weight_row's order: a lane holds S consecutive features of a token (gated:
// S / 2 of g and the same of u), so a token's features of a wave are written as
// 16 adjacent pieces.  S = 8: 16-byte pieces (gated: 8), and the next tile's
// first copies run under the epilogue.  S = 4, 2: one tile a workgroup.
//
// SPLIT: the sums go to a.part in fp32 and layer_join_fwd_kernel does the rest.
template <class T, int S, int ACT, bool GLU, bool SPLIT>
__global__ void __launch_bounds__(kThreads, (Tile<T, S>::kPerCu)) layer_fwd_kernel(LayerFwd a) {
  constexpr int M = Tile<T, S>::M;
  constexpr int FT = GLU ? M / 2 : M;   // features of a tile
  constexpr int C = GLU ? S / 2 : S;    // consecutive features of a lane
  // The wave's index as a scalar: the epilogue's descriptors start at its rows,
  // and one made from a vector register costs a loop over the lanes at each store.
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1, g = lane >> 4, c = lane & 15;
  const int tiles = a.TM * a.TN, total = tiles * a.parts;
  int n0, f0, k0;
  auto place = [&](int t) {
    const int part = SPLIT ? t / tiles : 0;
    int tm, tn;
    tile_coords(t - part * tiles, tiles, a.TM, a.TN, tm, tn);
    n0 = tm * M;
    f0 = tn * FT;
    k0 = part * a.kc;
  };
  auto opa = [&]() { return Opnd<T>{(const T*)a.x + k0, a.H, a.N, min(a.kc, a.H - k0)}; };
  auto opb = [&]() { return Opnd<T>{(const T*)a.W[0] + k0, a.H, a.F, min(a.kc, a.H - k0)}; };
  int t = blockIdx.x;
  place(t);
  const bool vec = S == 8 && a.F % C == 0;   // every lane's run is whole and aligned to its size
  auto tile = [&](auto& acc, int n0, int f0, int part, const float (&b0)[C], const float (&b1)[C]) {
    // Value (i, r) of a lane is token n0w + 4 g + 16 i + r.  In an aligned tile
    // its byte offset is the lane's (token 4 g, or kOOB for a token past N) plus
    // the wave's (16 i + r tokens), from a descriptor at the wave's first token: at
    // most 128 * ld * 4.
    const int n0w = n0 + wm * 16 * S, f = f0 + (wn * 16 + c) * C;
    const int64_t ld = SPLIT ? a.ldp : a.F;
    const int left = (SPLIT ? (int)(GLU ? a.ldp / 2 : a.ldp) : a.F) - f;   // features of this lane's run inside the row
    const int lim = left > 0 ? a.N - n0w - 4 * g : 0;
    const uint32_t lane0 = (uint32_t)(4 * g * (int)ld + f);
    auto offset = [&](int i, int r, uint32_t es) -> uint32_t { return 16 * i + r < lim ? lane0 * es : kOOB; };
    auto wave_offset = [&](int i, int r, int es) -> int { return (16 * i + r) * (int)ld * es; };
    const int64_t base = ((int64_t)part * a.N + n0w) * ld;
    auto rows = [&](auto whole) {   // whole: vec, as a constant
      constexpr bool kVec = whole.value;
      constexpr int ES = sizeof(T);
      const bool res = !GLU && !SPLIT && a.residual != nullptr, keep = !SPLIT && a.z[0] != nullptr;
      __amdgpu_buffer_rsrc_t ry, rr, rz0, rz1;
      if constexpr (kVec) {
        ry = make_rsrc((const T*)a.y + base);
        rr = make_rsrc((const T*)a.residual + base);
        rz0 = make_rsrc((SPLIT ? a.part : a.z[0]) + base);
        rz1 = make_rsrc((SPLIT ? a.part + a.ldp / 2 : a.z[1]) + base);
      }
      unrolled<S>([&](auto block) {
        constexpr int i = block.value;
        float rs[4][C];
        if constexpr (!GLU && !SPLIT) {
          if (res) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              if constexpr (kVec) buf_load_vec<T, C>(rr, offset(i, r, ES), wave_offset(i, r, ES), rs[r]);
              else if (16 * i + r < lim)
                load_some<T, C>((const T*)a.residual + base + lane0 + (16 * i + r) * ld, left, rs[r]);
            }
          }
        }
        f32x4 z[S];
#pragma unroll
        for (int j = 0; j < S; ++j) z[j] = block_sums<S>(acc[i][j]);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          float z0[C], z1[C], v[C];
#pragma unroll
          for (int e = 0; e < C; ++e) {
            z0[e] = z[e][r] + (SPLIT ? 0.f : b0[e]);
            z1[e] = z[S - C + e][r] + (SPLIT ? 0.f : b1[e]);
            if constexpr (!SPLIT) {
              v[e] = act_fwd<T, ACT>(z0[e]);
              if constexpr (GLU) v[e] *= z1[e];
              else if (res) v[e] += rs[r][e];
            }
          }
          if constexpr (kVec) {
            if (SPLIT || keep) {
              buf_store_vec<float, C>(rz0, offset(i, r, 4), wave_offset(i, r, 4), z0);
              if constexpr (GLU) buf_store_vec<float, C>(rz1, offset(i, r, 4), wave_offset(i, r, 4), z1);
            }
            if constexpr (!SPLIT) buf_store_vec<T, C>(ry, offset(i, r, ES), wave_offset(i, r, ES), v);
          } else if (16 * i + r < lim) {
            const int64_t o = base + lane0 + (16 * i + r) * ld;
            if (SPLIT || keep) {
              store_some<float, C>((SPLIT ? a.part : a.z[0]) + o, left, z0);
              if constexpr (GLU) store_some<float, C>((SPLIT ? a.part + a.ldp / 2 : a.z[1]) + o, left, z1);
            }
            if constexpr (!SPLIT) store_some<T, C>((T*)a.y + o, left, v);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      });
    };
    if constexpr (S == 8 && SPLIT) {
      rows(std::true_type{});   // rows of the partial sums are padded to 8 columns
    } else if constexpr (S == 8) {
      if (vec) rows(std::true_type{});
      else rows(std::false_type{});
    } else {
      rows(std::false_type{});
    }
  };
  auto biases = [&](float (&b0)[C], float (&b1)[C]) {
    const int f = f0 + (wn * 16 + c) * C;
#pragma unroll
    for (int e = 0; e < C; ++e) {
      b0[e] = (!SPLIT && a.b[0] && f + e < a.F) ? load1<T>((const T*)a.b[0] + f + e) : 0.f;
      b1[e] = (!SPLIT && GLU && a.b[1] && f + e < a.F) ? load1<T>((const T*)a.b[1] + f + e) : 0.f;
    }
  };
  float b0[C], b1[C];
  if constexpr (S == 8) {
    typedef typename std::conditional<GLU, DmaGlu, Dma<true>>::type DB;
    FLCE_LDS(L, T);
    TileCopy<true, true, Dma<true>, DB> tc;
    auto begin = [&]() {
      const Opnd<T> A = opa(), B = opb();
      tc.da.init(A, n0, tid);
      if constexpr (GLU) tc.db.init(B.p, (const T*)a.W[1] + k0, B.ld, a.F, f0, tid);
      else tc.db.init(B, f0, tid, 2);
      tc.begin(A, B, L, tid);
    };
    begin();
    __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0<0>());   // the mainloop's first wait allows for an epilogue's stores
    Acc acc;
    while (true) {
      const Opnd<T> A = opa(), B = opb();
      const int n0c = n0, f0c = f0, part = SPLIT ? t / tiles : 0;
      biases(b0, b1);
      // Each tile's epilogue stores at least 32 times per wave after the next tile's first copies.
      gemm_tile_bf16_run<true, true, 32>(acc, A, B, A.kext, L, tid, tc);
      t += gridDim.x;
      const bool more = t < total;
      if (more) {
        place(t);
        begin();
      }
      acc_drain();
      tile(acc, n0c, f0c, part, b0, b1);
      if (!more) break;
      if (!SPLIT && !vec) __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0<0>());   // lanes past the row stored nothing
    }
  } else {
    biases(b0, b1);
    f32x4 acc[S][S];
    const Opnd<T> A = opa(), B = opb();
    RowCopy<T, S, false, false> ca;
    RowCopy<T, S, true, GLU> cb;
    ca.init(A.p, nullptr, A.ld, a.N, n0, tid);
    cb.init(B.p, (const T*)a.W[1] + k0, B.ld, a.F, f0, tid);
    SMALL_LDS(L, T, S);
    if constexpr (sizeof(T) == 2) gemm_small<T, S, RowFrag<S>, RowFrag<S>>(acc, ca, A.kext, cb, B.kext, A.kext, L, tid);
    else gemm_small_f32<S>(acc, ca, A.kext, cb, B.kext, A.kext, L, tid);
    tile(acc, n0, f0, SPLIT ? t / tiles : 0, b0, b1);
  }
}

// The epilogue of a split forward: thread i takes 8 features of one token.
template <class T, int ACT, bool GLU> __global__ void __launch_bounds__(256) layer_join_fwd_kernel(LayerFwd a) {
  const int F8 = (a.F + 7) / 8;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < (int64_t)a.N * F8; i += (int64_t)gridDim.x * 256) {
    const int n = (int)(i / F8), f = (int)(i - (int64_t)n * F8) * 8;
    const int left = min(8, a.F - f);
    float z0[8] = {}, z1[8] = {}, v[8];
    for (int p = 0; p < a.parts; ++p) {
      const float* s = a.part + ((int64_t)p * a.N + n) * a.ldp + f;
      load_vec<float, 8>(s, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) z0[e] += v[e];
      if constexpr (GLU) {
        load_vec<float, 8>(s + a.ldp / 2, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) z1[e] += v[e];
      }
    }
    const int64_t o = (int64_t)n * a.F + f;
    float rs[8] = {}, t[8];
    if (!GLU && a.residual) load_some<T, 8>((const T*)a.residual + o, left, rs);
    if (a.b[0]) {
      load_some<T, 8>((const T*)a.b[0] + f, left, t);
#pragma unroll
      for (int e = 0; e < 8; ++e) z0[e] += t[e];
    }
    if (GLU && a.b[1]) {
      load_some<T, 8>((const T*)a.b[1] + f, left, t);
#pragma unroll
      for (int e = 0; e < 8; ++e) z1[e] += t[e];
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      v[e] = act_fwd<T, ACT>(z0[e]);
      v[e] = GLU ? v[e] * z1[e] : v[e] + rs[e];
    }
    if (a.z[0]) store_some<float, 8>(a.z[0] + o, left, z0);
    if (GLU && a.z[1]) store_some<float, 8>(a.z[1] + o, left, z1);
    store_some<T, 8>((T*)a.y + o, left, v);
  }
}

// ---------------------------------------------------------------------------
// Forward, few tokens
// ---------------------------------------------------------------------------

constexpr int kSkinnyWaves = 8;

// Workgroup b computes features 16 b .. 16 b + 15 of at most 16 tokens.  Its 8
// waves split K; each loads its weight rows straight into registers (no two
// waves share a weight, so LDS would only add a hop) with two groups of 4 loads
// of each weight in flight, and x's rows through the caches.  The waves' sums
// meet in LDS and are added in wave order.  HBM bounds it: one token, H=4096,
// F=12288 bf16, gated: 39 us, 5.1 TB/s of weights.
template <class T, bool GLU>
__global__ void __launch_bounds__(64 * kSkinnyWaves) layer_fwd_skinny_kernel(LayerFwd a) {
  constexpr int R = GLU ? 2 : 1, ES = sizeof(T);
  constexpr int kStep = 64 / ES;   // K of one step: 16 bytes in each of the 4 lane groups
  constexpr int kU = 4;
  __shared__ f32x4 red[kSkinnyWaves][R][64];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = lane >> 4, rl = lane & 15, f0 = blockIdx.x * 16;
  // Rows past F or N repeat the last one: their sums are not stored.
  const uint32_t offw = (uint32_t)min(rl, a.F - 1 - f0) * (uint32_t)(a.H * ES) + 16u * g;
  const uint32_t offx = (uint32_t)min(rl, a.N - 1) * (uint32_t)(a.H * ES) + 16u * g;
  __amdgpu_buffer_rsrc_t rw[R];
#pragma unroll
  for (int r = 0; r < R; ++r) rw[r] = make_rsrc((const T*)a.W[r] + (int64_t)f0 * a.H);
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(a.x);

  const int steps = (a.H + kStep - 1) / kStep, per = (steps + kSkinnyWaves - 1) / kSkinnyWaves;
  const int s0 = wave * per, s1 = min(steps, s0 + per);
  const int klim = min(s1 * kStep, a.H) - g * (16 / ES);   // step s of this lane is inside K when s * kStep < klim
  f32x4 acc[R] = {};
  u32x4 w[2][kU][R], x[2][kU];
  auto load = [&](int h, int s) {
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const bool in = (s + u) * kStep < klim;
      const int so = 64 * (s + u);
#pragma unroll
      for (int r = 0; r < R; ++r)
        w[h][u][r] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rw[r], in ? offw : kOOB, so, 0));
      x[h][u] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rx, in ? offx : kOOB, so, 0));
    }
  };
  auto mma = [&](int h) {
#pragma unroll
    for (int u = 0; u < kU; ++u)
#pragma unroll
      for (int r = 0; r < R; ++r) mma_frag<T>(acc[r], w[h][u][r], x[h][u]);
  };
  load(0, s0);
  for (int s = s0; s < s1; s += 2 * kU) {
    load(1, s + kU);
    mma(0);
    load(0, s + 2 * kU);
    mma(1);
  }
#pragma unroll
  for (int r = 0; r < R; ++r) red[wave][r][lane] = acc[r];
  __syncthreads();
  // Element (token n, feature f) sits in lane 16 (f / 4) + n, value f % 4.
  const int f = tid & 15, n = tid >> 4;
  if (n >= a.N || f0 + f >= a.F) return;
  float z[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    z[r] = 0.f;
#pragma unroll
    for (int q = 0; q < kSkinnyWaves; ++q) z[r] += ((const float*)&red[q][r][16 * (f >> 2) + n])[f & 3];
    if (a.b[r]) z[r] += load1<T>((const T*)a.b[r] + f0 + f);
  }
  const int64_t o = (int64_t)n * a.F + f0 + f;
  float v = act_fwd_rt<T>(a.act, z[0]);
  if constexpr (GLU) v *= z[R - 1];
  else if (a.residual) v += load1<T>((const T*)a.residual + o);
  if (a.z[0]) {
    a.z[0][o] = z[0];
    if constexpr (GLU) a.z[1][o] = z[R - 1];
  }
  store1<T>((T*)a.y + o, v);
}

// f.operator()<ACT>() for the activation.
template <class F> static void with_act(int act, F&& f) {
  switch (act) {
    case kActRelu: return f(std::integral_constant<int, kActRelu>{});
    case kActGelu: return f(std::integral_constant<int, kActGelu>{});
    case kActGeluTanh: return f(std::integral_constant<int, kActGeluTanh>{});
    case kActSilu: return f(std::integral_constant<int, kActSilu>{});
    case kActSigmoid: return f(std::integral_constant<int, kActSigmoid>{});
    default: return f(std::integral_constant<int, kActNone>{});
  }
}

// f(integral_constant<int, S>) for the tile.
template <class T, class F> static void with_tile(int s, F&& f) {
  if constexpr (sizeof(T) == 2) {
    if (s == 8) return f(std::integral_constant<int, 8>{});
  }
  if (s == 4) return f(std::integral_constant<int, 4>{});
  return f(std::integral_constant<int, 2>{});
}

template <class T, bool GLU> static void launch_fwd(const LayerFwd& a, hipStream_t st) {
  if (a.tile == 0) {
    FLCE_LAUNCH((layer_fwd_skinny_kernel<T, GLU>), dim3((a.F + 15) / 16), dim3(64 * kSkinnyWaves), 0, st, a);
    return;
  }
  const int total = a.TM * a.TN * a.parts;
  const dim3 grid(a.tile < 8 || total < kPersistGrid ? total : kPersistGrid), blk(kThreads);
  with_tile<T>(a.tile, [&](auto tile) {
    constexpr int S = tile.value;
    if (a.parts > 1) {
      FLCE_LAUNCH((layer_fwd_kernel<T, S, kActNone, GLU, true>), grid, blk, 0, st, a);
    } else {
      with_act(a.act, [&](auto act) {
        FLCE_LAUNCH((layer_fwd_kernel<T, S, act.value, GLU, false>), grid, blk, 0, st, a);
      });
    }
  });
  if (a.parts > 1) {
    const int64_t blocks = ((int64_t)a.N * ((a.F + 7) / 8) + 255) / 256;
    const dim3 gj((unsigned)(blocks < 4096 ? blocks : 4096));
    with_act(a.act, [&](auto act) { FLCE_LAUNCH((layer_join_fwd_kernel<T, act.value, GLU>), gj, dim3(256), 0, st, a); });
  }
}

// ---------------------------------------------------------------------------
// Backward
// ---------------------------------------------------------------------------

// dz = dy act'(z), or dg = dh u act'(g) and du = dh act(g), into a.dz, and
// their column sums over a.db_rows tokens into a.dbp.  Thread (column group,
// row) = (tid % 32, tid / 32) walks its block's tokens 8 rows apart.  The sums
// take the values before they are rounded to T.
// dz is rounded because it is an operand of T's matrix products: a second part
// would double them (gated, N=8192, H=4096, F=12288: 2.3 of the pass's 3.8 ms).  It is the
// whole of what 16-bit gradients lose beside their own rounding: relative error
// 2.35e-3 against the formula in bf16, 1.66e-3 with dz in fp32, 2.35e-3 for the
// formula in 64 bits with dz rounded; fp16 2.9e-4, 2.1e-4 and 2.9e-4.
template <class T, int ACT, bool GLU> __global__ void __launch_bounds__(256) layer_dz_kernel(LayerBwd a) {
  constexpr int R = GLU ? 2 : 1;
  const int tid = threadIdx.x, f = (blockIdx.x * 32 + (tid & 31)) * 8;
  const int n1 = min(a.N, (int)(blockIdx.y + 1) * a.db_rows);
  const int left = a.F - f;
  const int width = GLU ? a.segk : (int)a.ldz;   // columns of one weight in dz
  float sum[R][8] = {};
  if (f < width) {
#pragma unroll 2
    for (int n = blockIdx.y * a.db_rows + (tid >> 5); n < n1; n += 8) {
      const int64_t o = (int64_t)n * a.F + f;
      float dy[8], z0[8] = {}, z1[8] = {}, d[R][8];
      load_some<T, 8>((const T*)a.dy + o, left, dy);
      if (ACT != kActNone || GLU) load_some<float, 8>(a.z[0] + o, left, z0);
      if (GLU) load_some<float, 8>(a.z[1] + o, left, z1);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float v;
        d[0][e] = act_bwd<T, ACT>(z0[e], GLU ? dy[e] * z1[e] : dy[e], v);
        if (GLU) d[R - 1][e] = dy[e] * v;
#pragma unroll
        for (int r = 0; r < R; ++r) sum[r][e] += d[r][e];
      }
      if (!a.dz_is_dy) {
#pragma unroll
        for (int r = 0; r < R; ++r) store_vec<T, 8>((T*)a.dz + (int64_t)n * a.ldz + r * a.segk + f, d[r]);
      }
    }
  }
  if (!a.dbp) return;
  __shared__ float red[R][8][256];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int e = 0; e < 8; ++e) red[r][tid >> 5][8 * (tid & 31) + e] = sum[r][e];
  __syncthreads();
  const int col = blockIdx.x * 256 + tid;
  if (col >= a.F) return;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    float s = 0.f;
#pragma unroll
    for (int q = 0; q < 8; ++q) s += red[r][q][tid];
    a.dbp[blockIdx.y * a.ldb + r * (a.ldb / R) + col] = s;
  }
}

// db[m][f] = the blocks' sums added in block order.
template <class T> __device__ __forceinline__ void column_sum(const LayerBwd& a, int m, int f) {
  const float* p = a.dbp + m * (a.ldb / a.nmat) + f;
  float s = 0.f;
#pragma unroll 8
  for (int b = 0; b < a.db_blocks; ++b) s += p[b * a.ldb];
  store1<T>((T*)a.db[m] + f, s);
}

// db of the weights whose gradient no launch of layer_dw_kernel forms.
template <class T> __global__ void __launch_bounds__(256) layer_db_kernel(LayerBwd a) {
  const int f = blockIdx.x * 256 + threadIdx.x, m = blockIdx.y;
  if (f < a.F && a.db[m] && !a.dW[m]) column_sum<T>(a, m, f);
}

// A lane's values of C[h][row]: four consecutive h of the rows row0 + 16 j (to
// rows), at h0 + 16 i, into a [rows][width] matrix of E.
template <class E, int S, class A>
__device__ __forceinline__ void store_rows(const A& acc, E* out, int width, int row0, int rows, int h0) {
  auto all = [&](auto whole) {   // whole: width % 4 == 0, as a constant
    unrolled<S>([&](auto col) {
      constexpr int j = col.value;
      const int row = row0 + 16 * j;
      E* p = out + (int64_t)row * width;
      unrolled<S>([&](auto block) {
        constexpr int i = block.value;
        const f32x4 z = block_sums<S>(acc[i][j]);
        const int h = h0 + 16 * i;
        if (row < rows && h < width) {
          const float v[4] = {z[0], z[1], z[2], z[3]};
          if constexpr (whole.value) store_vec<E, 4>(p + h, v);
          else store_some<E, 4>(p + h, width - h, v);
        }
      });
    });
  };
  if (width % 4 == 0) all(std::true_type{});
  else all(std::false_type{});
}

// Where a workgroup stands in one of the two gradient products.
//   dx[n][h] = sum over the rows f of W (gated: of Wg, then of Wu) of dz[n][f] W[f][h]: C[h][n]
//   dW[f][h] = sum_n dz[n][f] x[n][h]: C[h][f]
// so a lane holds four consecutive h of a row.  Workgroup w computes tile w % G
// over part w / G of K.  dW: column tile tn belongs to weight m0 (tn < TF) or
// the next.  That is told by a compare: a division put the descriptors'
// addresses into vector registers, which costs a loop over the lanes at every
// copy (N=8192, H=4096, 24576 rows took 1463 us so, 1127 now).
struct GradTile {
  int h0, c0, k0, part, m, second;   // second: 1 for the next weight (dW)
};
template <int S> __device__ __forceinline__ GradTile dx_place(const LayerBwd& a, int w, int TH, int TM) {
  const int G = TH * TM, part = a.dx_parts > 1 ? w / G : 0;
  int tm, tn;
  tile_coords(w - part * G, G, TH, TM, tm, tn);
  return {tm * 32 * S, tn * 32 * S, part * a.dx_kc, part, 0, 0};
}
template <int S> __device__ __forceinline__ GradTile dw_place(const LayerBwd& a, int w, int TH, int TF, int m0, int mats) {
  const int G = TH * TF * mats, part = a.dw_parts > 1 ? w / G : 0;
  int tm, tn;
  tile_coords(w - part * G, G, TH, TF * mats, tm, tn);
  const int second = tn >= TF ? 1 : 0;
  return {tm * 32 * S, (tn - second * TF) * 32 * S, part * a.dw_kc, part, m0 + second, second};
}

// The tile's sums to the gradient, or to its part's fp32 partial sums.
template <class T, int S, class A>
__device__ __forceinline__ void store_dx(const LayerBwd& a, const GradTile& t, const A& acc, int tid) {
  const int lane = tid & 63, wave = tid >> 6;
  const int n = t.c0 + (wave & 1) * 16 * S + (lane & 15), h = t.h0 + (wave >> 1) * 16 * S + 4 * (lane >> 4);
  if (a.dx_parts > 1) store_rows<float, S>(acc, a.dx_part + (int64_t)t.part * a.N * a.Hout, a.Hout, n, a.N, h);
  else store_rows<T, S>(acc, (T*)a.dx, a.Hout, n, a.N, h);
}
template <class T, int S, class A>
__device__ __forceinline__ void store_dw(const LayerBwd& a, const GradTile& t, int mats, const A& acc, int tid) {
  const int lane = tid & 63, wave = tid >> 6;
  const int f = t.c0 + (wave & 1) * 16 * S + (lane & 15), h = t.h0 + (wave >> 1) * 16 * S + 4 * (lane >> 4);
  if (a.dw_parts > 1)
    store_rows<float, S>(acc, a.dw_part + ((int64_t)t.part * mats + t.second) * a.F * a.Hout, a.Hout, f, a.F, h);
  else store_rows<T, S>(acc, (T*)a.dW[t.m], a.Hout, f, a.F, h);
}

// The first H tile's workgroups of dW also finish db for their columns.
template <class T, int S> __device__ __forceinline__ void finish_db(const LayerBwd& a, const GradTile& t, int tid) {
  if (t.h0 == 0 && t.part == 0 && a.db[t.m] && tid < 32 * S && t.c0 + tid < a.F) column_sum<T>(a, t.m, t.c0 + tid);
}

// S = 8: one launch a product.
template <class T> __global__ void __launch_bounds__(kThreads, 1) layer_dx_kernel(LayerBwd a, int TH, int TM) {
  const int tid = threadIdx.x;
  const GradTile t = dx_place<8>(a, blockIdx.x, TH, TM);
  const int K = max(1, min(a.dx_kc, (int)a.ldz - t.k0));
  FLCE_LDS(L, T);
  const Opnd<T> A{(const T*)a.W[0], a.H, a.H, K};   // K only: rows past F read zeros
  const Opnd<T> B{(const T*)a.dz + t.k0, a.ldz, a.N, (int)a.ldz - t.k0};
  Acc acc;
  TileCopy<false, true, DmaSeg, Dma<true>> tc;
  tc.da.d.init(A, t.h0, tid);
  tc.da.s = SegRows{{a.W[0], a.W[1]}, a.H, a.F, a.segk, t.k0};
  tc.da.m0 = t.h0;
  tc.db.init(B, t.c0, tid);
  tc.begin(A, B, L, tid);
  gemm_tile_bf16_run<false, true>(acc, A, B, K, L, tid, tc);
  acc_drain();
  store_dx<T, 8>(a, t, acc, tid);
}
template <class T>
__global__ void __launch_bounds__(kThreads, 1) layer_dw_kernel(LayerBwd a, int TH, int TF, int m0, int mats) {
  const int tid = threadIdx.x;
  const GradTile t = dw_place<8>(a, blockIdx.x, TH, TF, m0, mats);
  const int K = max(0, min(a.dw_kc, a.N - t.k0)), width = a.nmat == 2 ? a.segk : (int)a.ldz;
  finish_db<T, 8>(a, t, tid);
  FLCE_LDS(L, T);
  const Opnd<T> A{(const T*)a.x + (int64_t)t.k0 * a.H, a.H, a.H, K};
  const Opnd<T> B{(const T*)a.dz + (int64_t)t.k0 * a.ldz + (int64_t)t.m * a.segk, a.ldz, width, K};
  Acc acc;
  gemm_tile<T, false, false>(acc, A, t.h0, B, t.c0, max(K, 1), L, tid);   // K >= 1: no token sums zeros
  acc_drain();
  store_dw<T, 8>(a, t, mats, acc, tid);
}

// S = 4, 2: both products in one launch, dx in the first gx workgroups: small
// products leave CUs idle, which the other's workgroups take, and the host
// launches less (N=785, H=1216, F=192 bf16, forward and backward: 41.6 us with a
// launch each, 32.8 so).
template <class T, int S>
__global__ void __launch_bounds__(kThreads, (Tile<T, S>::kPerCu)) layer_grads_kernel(LayerBwd a, int gx, int TH, int TM,
                                                                                   int TF, int m0, int mats) {
  const int tid = threadIdx.x;
  SMALL_LDS(L, T, S);
  f32x4 acc[S][S];
  if ((int)blockIdx.x < gx) {
    const GradTile t = dx_place<S>(a, blockIdx.x, TH, TM);
    const int K = max(1, min(a.dx_kc, (int)a.ldz - t.k0));
    ColCopy<T, S> ca;
    RowCopy<T, S, false, false> cb;
    ca.init(SegRows{{a.W[0], a.W[1]}, a.H, a.F, a.segk, t.k0}, a.H, t.h0, tid);
    cb.init((const T*)a.dz + t.k0, nullptr, a.ldz, a.N, t.c0, tid);
    if constexpr (sizeof(T) == 2) gemm_small<T, S, ColFrag<S>, RowFrag<S>>(acc, ca, K, cb, (int)a.ldz - t.k0, K, L, tid);
    else gemm_small_f32<S>(acc, ca, K, cb, (int)a.ldz - t.k0, K, L, tid);
    store_dx<T, S>(a, t, acc, tid);
  } else {
    const GradTile t = dw_place<S>(a, blockIdx.x - gx, TH, TF, m0, mats);
    const int K = max(0, min(a.dw_kc, a.N - t.k0)), width = a.nmat == 2 ? a.segk : (int)a.ldz;
    finish_db<T, S>(a, t, tid);
    const T* x = (const T*)a.x + (int64_t)t.k0 * a.H;
    const T* dz = (const T*)a.dz + (int64_t)t.k0 * a.ldz + (int64_t)t.m * a.segk;
    ColCopy<T, S> ca, cb;
    ca.init(SegRows{{x, x}, a.H, K, 1 << 30, 0}, a.H, t.h0, tid);
    cb.init(SegRows{{dz, dz}, a.ldz, K, 1 << 30, 0}, width, t.c0, tid);
    if constexpr (sizeof(T) == 2) gemm_small<T, S, ColFrag<S>, ColFrag<S>>(acc, ca, K, cb, K, K, L, tid);
    else gemm_small_f32<S>(acc, ca, K, cb, K, K, L, tid);
    store_dw<T, S>(a, t, mats, acc, tid);
  }
}

// Split products' parts added in part order: blockIdx.y is dx, dW of the first
// weight written, dW of the next.  Four values a thread.
template <class T> struct Join {
  const float* part[3];
  int64_t n[3], stride[3];   // values, and from one part to the next
  int parts[3];
  T* out[3];
};
template <class T> __global__ void __launch_bounds__(256) layer_join_kernel(Join<T> a) {
  const int y = blockIdx.y;
  const float* s = a.part[y];
  const int64_t n = a.n[y];
  for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4; i < n; i += (int64_t)gridDim.x * 1024) {
    const int left = (int)min((int64_t)4, n - i);
    float v[4], t[4];
    load_some<float, 4>(s + i, left, v);
    for (int p = 1; p < a.parts[y]; ++p) {
      load_some<float, 4>(s + p * a.stride[y] + i, left, t);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] += t[e];
    }
    store_some<T, 4>(a.out[y] + i, left, v);
  }
}

template <class T, bool GLU> static void launch_dz(const LayerBwd& a, hipStream_t st) {
  const int width = GLU ? a.segk : (int)a.ldz;
  const dim3 grid((width + 255) / 256, a.db_blocks);
  with_act(a.act, [&](auto act) { FLCE_LAUNCH((layer_dz_kernel<T, act.value, GLU>), grid, dim3(256), 0, st, a); });
}

template <class T> static void launch_bwd(const LayerBwd& a, hipStream_t st) {
  const dim3 blk(kThreads);
  if (a.N > 0 && (!a.dz_is_dy || a.db[0] || a.db[1])) {
    if (a.nmat == 2) launch_dz<T, true>(a, st);
    else launch_dz<T, false>(a, st);
  }
  if ((a.db[0] && !a.dW[0]) || (a.db[1] && !a.dW[1]))
    FLCE_LAUNCH((layer_db_kernel<T>), dim3((a.F + 255) / 256, a.nmat), dim3(256), 0, st, a);
  auto tiles = [](int n, int s) { return (n + 32 * s - 1) / (32 * s); };
  const bool dx = a.dx && a.N > 0, dw = a.dW[0] || a.dW[1];
  const int m0 = a.dW[0] ? 0 : 1, mats = (a.dW[0] && a.dW[1]) ? 2 : 1;
  Join<T> join{};
  int joins = 0;
  int64_t most = 0;
  if (dx && a.dx_parts > 1) {
    const int64_t n = (int64_t)a.N * a.Hout;
    join.part[0] = a.dx_part; join.n[0] = join.stride[0] = n; join.parts[0] = a.dx_parts; join.out[0] = (T*)a.dx;
    joins = 1;
    most = n;
  }
  for (int k = 0; dw && a.dw_parts > 1 && k < mats; ++k, ++joins) {
    const int64_t n = (int64_t)a.F * a.Hout;
    join.part[joins] = a.dw_part + k * n; join.n[joins] = n; join.stride[joins] = mats * n;
    join.parts[joins] = a.dw_parts; join.out[joins] = (T*)a.dW[m0 + k];
    most = most > n ? most : n;
  }
  // dx_tile and dw_tile, where neither is 8, are the same.
  auto small = [&](auto tile, bool with_dx, bool with_dw) {
    constexpr int S = tile.value;
    if constexpr (S < 8) {
      const int TH = tiles(a.H, S), TM = tiles(a.N, S), TF = tiles(a.F, S);
      const int gx = with_dx ? TH * TM * a.dx_parts : 0, gw = with_dw ? TH * TF * mats * a.dw_parts : 0;
      FLCE_LAUNCH((layer_grads_kernel<T, S>), dim3(gx + gw), blk, 0, st, a, gx, TH, TM, TF, m0, mats);
    }
  };
  const bool dx8 = a.dx_tile == 8, dw8 = a.dw_tile == 8;
  if constexpr (sizeof(T) == 2) {
    if (dx && dx8) FLCE_LAUNCH((layer_dx_kernel<T>), dim3(tiles(a.H, 8) * tiles(a.N, 8) * a.dx_parts), blk, 0, st, a, tiles(a.H, 8), tiles(a.N, 8));
    if (dw && dw8) FLCE_LAUNCH((layer_dw_kernel<T>), dim3(tiles(a.H, 8) * tiles(a.F, 8) * mats * a.dw_parts), blk, 0, st, a, tiles(a.H, 8), tiles(a.F, 8), m0, mats);
  }
  if ((dx && !dx8) || (dw && !dw8))
    with_tile<T>(dx8 ? a.dw_tile : a.dx_tile, [&](auto tile) { small(tile, dx && !dx8, dw && !dw8); });
  if (joins) {
    const int64_t blocks = ((most + 3) / 4 + 255) / 256;
    FLCE_LAUNCH((layer_join_kernel<T>), dim3((unsigned)(blocks < 2048 ? blocks : 2048), joins), dim3(256), 0, st, join);
  }
}

template <class T> static hipError_t layer_forward(const LayerFwd& a, hipStream_t st) {
  if (a.nmat == 2) launch_fwd<T, true>(a, st);
  else launch_fwd<T, false>(a, st);
  return hipGetLastError();
}
template <class T> static hipError_t layer_backward(const LayerBwd& a, hipStream_t st) {
  launch_bwd<T>(a, st);
  return hipGetLastError();
}

}  // namespace flce
