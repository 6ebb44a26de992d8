// Attention over the cache, prompts on tensor memory: e4m3 codes.
#include "attention_tiles.cuh"
namespace mt {
MT_DEFINE_ATTENTION_TILES(launch_attention_tiles_e4m3, false)
}  // namespace mt
