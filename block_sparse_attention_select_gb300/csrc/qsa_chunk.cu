// Dense attention of new tokens over the paged K/V cache by pairs of SMs: the
// kernel is in qsa_chunk_pair.cuh.
#include "qsa_chunk_pair.cuh"

namespace qsa {

int32_t chunk_part_rows(int32_t rows, int32_t group)
{
    return static_cast<int32_t>(std::min<int64_t>(CH_ROWS, static_cast<int64_t>(rows) * group));
}

size_t chunk_workspace_bytes(int32_t rows, int32_t group, int32_t head_dim)
{
    return ws_o<CH_ROWS, CHUNK_MAX_PAIRS>() + size_t{2} * CHUNK_MAX_PAIRS * chunk_part_rows(rows, group) * head_dim * 4;
}

// Tensor maps of K and V: `row` bytes of a token and `chunks` such rows, of `box`
// tokens, per copy.
void chunk_boxes(int32_t head_dim, int32_t page_tokens, bool e4m3, ChunkBox *k, ChunkBox *v)
{
    k->row = 128;
    k->box = std::min(page_tokens, CH_TILE / 2);
    k->chunks = k->box == CH_TILE / 2 ? head_dim * (e4m3 ? 1 : 2) / k->row : 1;
    v->row = e4m3 ? head_dim / 2 : 128;
    v->box = std::min(page_tokens, CH_TILE);
    v->chunks = v->box == CH_TILE ? head_dim / 2 * (e4m3 ? 1 : 2) / v->row : 1;
}

int launch_chunk(const ChunkParams &p, const void *tk, const void *tv, int sms, bool overlap, void *stream)
{
    return launch_pairs_for<PairGeometry>(p, tk, tv, sms, overlap, false, static_cast<cudaStream_t>(stream));
}

}  // namespace qsa
