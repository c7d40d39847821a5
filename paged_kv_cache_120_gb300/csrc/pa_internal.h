// Internal declarations shared by libpa's translation units.
#pragma once

#include <cstdarg>
#include <cstddef>
#include <cstdint>

#include "../../include/pa.h"

namespace pa {

// Record a message for pa_last_error() on the calling thread; returns `code`.
int set_error(int code, const char *fmt, ...);

// Read and clear the prefill kernels' device error word (PA_DEVERR_* bits)
// on the current device. Returns a cudaError_t value (0 on success).
int prefill_take_device_error(int *bits);

// The same for pa_build_step and for the rotary write.
int step_take_device_error(int *bits);
int rope_take_device_error(int *bits);

// Cross attention of a few rows (arguments checked by the caller): whether
// the decode kernels' ragged form takes the shape, the workspace it needs,
// and the call.
bool cross_rows_fit(int num_seqs, int max_seqlen_q, int num_q_heads, int num_kv_heads, int block_size);
int cross_rows_workspace(int num_seqs, int max_seqlen_q, int num_q_heads, int num_kv_heads, int head_size, int dtype, bool fp8,
                         size_t *bytes);
int cross_rows(const char *who, void *out, const void *query, const void *kv_cache, const int32_t *block_tables,
               int max_blocks_per_seq, const int32_t *cu_seqlens_q, const int32_t *kv_lens, int num_seqs, int total_q,
               int max_seqlen_q, float scale, int num_q_heads, int num_kv_heads, int head_size, int num_blocks,
               int block_size, int dtype, bool fp8, float k_scale, float v_scale, void *workspace, size_t workspace_bytes,
               unsigned flags, pa_stream_t stream);

}  // namespace pa
