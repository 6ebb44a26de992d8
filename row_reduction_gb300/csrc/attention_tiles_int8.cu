// Attention over the cache, prompts on tensor memory: int8 codes.
#include "attention_tiles.cuh"
namespace mt {
MT_DEFINE_ATTENTION_TILES(launch_attention_tiles_int8, true)
}  // namespace mt
