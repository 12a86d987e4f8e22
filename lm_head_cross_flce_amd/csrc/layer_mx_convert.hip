// Microscaled quantisation and its inverse.  Both are bound by HBM: a lane takes 8
// columns, the four lanes of a block find its largest magnitude among themselves,
// and every byte is read and written once.  12288 x 4096 bf16 to e2m1: 23.5 us
// (5.4 TB/s), back 20 (6.3, some of it in the memory-side cache); to e4m3 27.6 (5.5), back 23 (6.6).
#include "layer_mx_device.hpp"

namespace flce {

// Lane's place: 8 columns of a row, in 32 bits where the count allows it.
template <class I, class F> __device__ __forceinline__ void each_run(const MxConvert& a, F&& f) {
  const I runs = (I)(a.Cp / 8), all = (I)a.R * runs;
  for (I i = (I)blockIdx.x * 256 + threadIdx.x; i < all; i += (I)gridDim.x * 256) {
    const I row = i / runs;
    f((int64_t)row, (int)(i - row * runs) * 8);
  }
}

template <class T, int FMT, class I> __global__ void __launch_bounds__(256) mx_quantize_kernel(MxConvert a) {
  each_run<I>(a, [&](int64_t row, int col) {
    float v[8];
    load_some<T, 8>((const T*)a.x + row * a.C + col, a.C - col, v);
    mx_store8<FMT>(a.codes, a.scales, row, a.Cp, col, v);
  });
}

template <class T, int FMT, class I> __global__ void __launch_bounds__(256) mx_dequantize_kernel(MxConvert a) {
  each_run<I>(a, [&](int64_t row, int col) {
    if (col >= a.C) return;
    const uint32_t s = a.scales[row * (a.Cp / kMxBlock) + col / kMxBlock];
    float v[8];
    if constexpr (FMT == kMxE4M3) {
      const u32x2 c = *(const u32x2*)(a.codes + row * a.Cp + col);
      mx_decode8<FMT>(c[0], c[1], s, v);
    } else {
      mx_decode8<FMT>(*(const uint32_t*)(a.codes + row * (a.Cp / 2) + col / 2), 0u, s, v);
    }
    store_some<T, 8>((T*)a.y + row * a.C + col, a.C - col, v);
  });
}

template <class F> static hipError_t with_format(const MxConvert& a, int dtype, F&& f) {
  const int64_t all = a.R * (a.Cp / 8), blocks = (all + 255) / 256;
  const dim3 grid((unsigned)(blocks < 16384 ? blocks : 16384));
  // past 2^31 runs (and a grid's stride) the index needs 64 bits
  const bool wide = all > (int64_t(1) << 31);
  auto types = [&](auto t, auto fmt) {
    if (wide) f(t, fmt, int64_t{}, grid);
    else f(t, fmt, uint32_t{}, grid);
  };
  auto formats = [&](auto t) {
    if (a.format == kMxE4M3) types(t, std::integral_constant<int, kMxE4M3>{});
    else types(t, std::integral_constant<int, kMxE2M1>{});
  };
  if (dtype == 1) formats(uint16_t{});
  else if (dtype == 2) formats(_Float16{});
  else formats(float{});
  return hipGetLastError();
}

hipError_t launch_mx_quantize(const MxConvert& a, int dtype, hipStream_t st) {
  return with_format(a, dtype, [&](auto t, auto fmt, auto i, dim3 grid) {
    FLCE_LAUNCH((mx_quantize_kernel<decltype(t), fmt.value, decltype(i)>), grid, dim3(256), 0, st, a);
  });
}
hipError_t launch_mx_dequantize(const MxConvert& a, int dtype, hipStream_t st) {
  return with_format(a, dtype, [&](auto t, auto fmt, auto i, dim3 grid) {
    FLCE_LAUNCH((mx_dequantize_kernel<decltype(t), fmt.value, decltype(i)>), grid, dim3(256), 0, st, a);
  });
}

}  // namespace flce
