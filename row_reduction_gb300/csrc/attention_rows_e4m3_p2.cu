// Attention over the cache, many rows: e4m3 codes, FP16 and FP32 queries.
#include "attention_rows.cuh"
namespace mt {
MT_DEFINE_ATTENTION_ROWS(launch_attention_rows_e4m3_p2, false, 2)
}  // namespace mt
