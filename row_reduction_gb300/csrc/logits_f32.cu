// Logits: f32 storage.
#include "logits.cuh"
namespace mt {
MT_DEFINE_LOGITS(float, f32)
}  // namespace mt
