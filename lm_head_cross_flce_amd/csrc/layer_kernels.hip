// Dispatch of the feed-forward operators to their element types' kernels
// (layer_kernels.hpp, one translation unit per type).
#include "flce_launch.hpp"

namespace flce {

hipError_t layer_pad_bf16(const LayerPad& a, hipStream_t st);
hipError_t layer_forward_bf16(const LayerFwd& a, hipStream_t st);
hipError_t layer_pad_f16(const LayerPad& a, hipStream_t st);
hipError_t layer_forward_f16(const LayerFwd& a, hipStream_t st);
hipError_t layer_pad_f32(const LayerPad& a, hipStream_t st);
hipError_t layer_forward_f32(const LayerFwd& a, hipStream_t st);
hipError_t layer_backward_bf16(const LayerBwd& a, hipStream_t st);
hipError_t layer_backward_f16(const LayerBwd& a, hipStream_t st);
hipError_t layer_backward_f32(const LayerBwd& a, hipStream_t st);

hipError_t launch_layer_pad(const LayerPad& a, int dtype, hipStream_t st) {
  return dtype == 1 ? layer_pad_bf16(a, st) : dtype == 2 ? layer_pad_f16(a, st) : layer_pad_f32(a, st);
}
hipError_t launch_layer_forward(const LayerFwd& a, int dtype, hipStream_t st) {
  return dtype == 1 ? layer_forward_bf16(a, st) : dtype == 2 ? layer_forward_f16(a, st) : layer_forward_f32(a, st);
}
hipError_t launch_layer_backward(const LayerBwd& a, int dtype, hipStream_t st) {
  return dtype == 1 ? layer_backward_bf16(a, st) : dtype == 2 ? layer_backward_f16(a, st) : layer_backward_f32(a, st);
}

}  // namespace flce
