// Rotary positions: bf16 storage.
#include "rotary.cuh"
namespace mt {
MT_DEFINE_ROTARY(__nv_bfloat16, bf16)
}  // namespace mt
