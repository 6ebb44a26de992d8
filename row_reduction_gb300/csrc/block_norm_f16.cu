// Norms around a block: f16 storage.
#include "block_norm.cuh"
namespace mt {
MT_DEFINE_BLOCK_NORM(__half, f16)
}  // namespace mt
