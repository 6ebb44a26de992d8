// Rotary positions: f16 storage.
#include "rotary.cuh"
namespace mt {
MT_DEFINE_ROTARY(__half, f16)
}  // namespace mt
