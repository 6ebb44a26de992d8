// Attention over the cache, many rows: e4m3 codes, BF16 queries.
#include "attention_rows.cuh"
namespace mt {
MT_DEFINE_ATTENTION_ROWS(launch_attention_rows_e4m3_p1, false, 1)
}  // namespace mt
