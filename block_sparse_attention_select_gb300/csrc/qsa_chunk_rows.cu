// Dense attention over the paged K/V cache for few rows: the kernel is in
// qsa_chunk_rows.cuh.
#include "qsa_chunk_rows.cuh"

namespace qsa {

int32_t chunk_rows_part_rows(int32_t rows, int32_t group)
{
    return static_cast<int32_t>(std::min<int64_t>(CR_ROWS, static_cast<int64_t>(rows) * group));
}

size_t chunk_rows_workspace_bytes(int32_t rows, int32_t group, int32_t head_dim)
{
    return ws_o<CR_ROWS, CHUNK_MAX_CTAS>() + size_t{2} * CHUNK_MAX_CTAS * chunk_rows_part_rows(rows, group) * head_dim * 4;
}

int32_t chunk_rows_box(int32_t page_tokens) { return std::min(page_tokens, CR_TILE); }

int launch_chunk_rows(const ChunkParams &p, const void *tk, const void *tv, int sms, bool overlap, void *stream)
{
    return launch_rows_for<RowsGeometry>(p, tk, tv, sms, overlap, false, static_cast<cudaStream_t>(stream));
}

}  // namespace qsa
