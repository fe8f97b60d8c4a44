// Definitions shared by the chunk kernels (rope_append.cu, chunk_attn.cu) and the C-ABI layer.
#pragma once

#include "mfa_internal.cuh"

namespace mfa {

// The chunk attention's tensor maps of one sequence: as KvSeq's, with boxes of 64 rows. They
// follow the KvSeq entries of a table of mfa_chunk_table_bytes bytes; the first reserved word
// of an entry is the distance in bytes to its own (0: the table has none), so that a
// description of fewer sequences than the table was made for finds them too.
struct alignas(128) KvChunkMaps {
  CUtensorMap k;
  CUtensorMap v;
};
constexpr int kChunkBoxRows = 64;
__device__ __forceinline__ bool has_chunk_maps(const KvSeq& s) { return s.reserved[0] != 0; }
__device__ __forceinline__ const KvChunkMaps* chunk_maps(const KvSeq& s) {
  return reinterpret_cast<const KvChunkMaps*>(reinterpret_cast<const uint8_t*>(&s) + s.reserved[0]);
}
inline void set_chunk_maps(KvSeq& s, int batch, int b) {
  s.reserved[0] = static_cast<int32_t>(sizeof(KvSeq) * (batch - b) + sizeof(KvChunkMaps) * b);
}

// The chunk attention's partials follow the workspace of the other calls: its work is cut
// into contiguous ranges over pairs of SMs, and a range has at most two items that do not
// cover their tile, its first and its last (chunk_attn.cu), so two slots of 256 rows -- 4
// tokens x 64 heads, running maximum and sum and the 256 accumulators of each, fp32 -- per
// pair, and the merge's 8 bytes a pair.
constexpr int kChunkRows = 256;
constexpr size_t kChunkPartialFloats = (size_t)kChunkRows * (2 + kHeadDim);
inline int chunk_grid_for(int num_sms) { return num_sms / 2; }
inline size_t chunk_ws_bytes(const WsLayout& L, int num_sms) {
  return L.total + (size_t)chunk_grid_for(num_sms) *
                       (2 * kChunkPartialFloats * sizeof(float) + sizeof(int2));
}

struct RopeAppendArgs {
  const uint16_t* q;        // [n_rows, 64, 256] bf16, or null (append only)
  uint16_t* q_out;
  const uint16_t* k;        // row t at k + t * k_ld
  const uint16_t* v;
  int k_ld, v_ld;
  const float* table;       // [max_pos, rot_dim]: cosines, then sines
  int max_pos, rot_dim;     // rot_dim 0: no rotation
  int interleaved;
  const int32_t* positions; // [axes, n_rows], or null: the cache row
  uint8_t pair_axis[kHeadDim / 2];
  const KvSeq* kv;
  int kv_dtype;
  float k_scale, v_scale;
  const int32_t* q_start;   // [batch + 1]
  const int32_t* seq_lens;  // [batch]
  int batch, n_rows;
  uint32_t* err;
};
cudaError_t launch_rope_append(const RopeAppendArgs& a, cudaStream_t s);

struct ChunkAttnArgs {
  const uint16_t* q;        // [n_rows, 64, 256] bf16
  const KvSeq* kv;          // device table
  int kv_dtype, page_size;
  float k_scale, v_scale;   // FP8 only
  const int32_t* q_start;   // [batch + 1]
  const int32_t* seq_lens;  // [batch]
  int batch, n_rows;
  float scale;
  uint16_t* out;            // [n_rows, 64, 256] bf16
  float* partials;          // two slots of kChunkPartialFloats per pair
  int2* info;               // [pairs]: the split tile that begins in a pair, for the merge
  uint32_t* err;
  int pairs;                // CTA pairs of the grid
};
// q_map and out_map cover q and out as [n_rows * 64 rows, 256] bf16, boxes of [64 rows x 64
// dims], 128-byte swizzle.
cudaError_t launch_chunk_attn(const CUtensorMap& q_map, const CUtensorMap& out_map,
                              const ChunkAttnArgs& a, cudaStream_t s);
// CTA pairs that can be resident on the current device at once (0 on an error).
int chunk_attn_pairs(const ChunkAttnArgs& a);

}  // namespace mfa
