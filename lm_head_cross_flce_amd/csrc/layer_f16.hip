// The feed-forward operators' kernels for f16 tensors.
#include "layer_kernels.hpp"

namespace flce {

hipError_t layer_pad_f16(const LayerPad& a, hipStream_t st) { return layer_pad<_Float16>(a, st); }
hipError_t layer_forward_f16(const LayerFwd& a, hipStream_t st) { return layer_forward<_Float16>(a, st); }
hipError_t layer_backward_f16(const LayerBwd& a, hipStream_t st) { return layer_backward<_Float16>(a, st); }

}  // namespace flce
