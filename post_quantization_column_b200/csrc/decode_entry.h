// decode_entry.h — the decode-step operators' entry points for a caller that knows the device of every
// pointer: those of include/awq_search.h with that device first. awq_decode.cu defines them and
// decode_binding.cpp calls them; both include this, so that an argument changed in one is an error
// in the other.
#pragma once

#include "../../include/awq_search.h"

extern "C" {
int awq_rms_norm_on(int device, const void* X, int x_dtype, int64_t x_stride, const void* residual, int r_dtype,
                    int64_t r_stride, void* residual_out, int64_t ro_stride, const void* weight, int w_dtype, int64_t M,
                    int64_t K, float eps, void* out, int out_dtype, float* out_scales, awq_stream_t stream);
int awq_kv_append_on(int device, const void* q, int64_t q_token_stride, int64_t q_head_stride, const void* k,
                     int64_t k_token_stride, int64_t k_head_stride, const void* v, int64_t v_token_stride,
                     int64_t v_head_stride, int in_dtype, int64_t T, int Hq, void* q_out, int q_dtype,
                     const int32_t* positions, const int32_t* seqs, const double* freqs, int rotary_dim, int interleaved,
                     float magnitude, const awq_paged_cache* cache, int32_t* status, awq_stream_t stream);
int awq_paged_attention_on(int device, const void* q, int64_t q_seq_stride, int64_t q_head_stride, int q_dtype, int Hq,
                           const awq_paged_cache* cache, const int32_t* lengths, float scale, void* out,
                           void* workspace, int64_t workspace_bytes, int32_t* status, awq_stream_t stream);
}
