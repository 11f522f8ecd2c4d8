// sequence_launch.h -- host-side interface between the sequence calls' ABI
// (sequence_abi.cu) and their kernels.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "mbrs_sequence.h"

namespace mbrs {
namespace seq {

// Checked by the ABI: sizes, strides, alignment, overlaps.  overlap, here and
// below: softmax_set_launch_overlap's setting.
cudaError_t launch_append(const softmax_append_args_t &a, int overlap, cudaStream_t stream);

// Attention.  Both launchers take the workspace the ABI has checked against
// the bytes below.
struct AttnCall {
    softmax_sequence_args_t a;
    bool paged;
    void *workspace;
    int sms;
    int64_t wait_ns;
    int starve;  // a test hook (softmax_attention_set_wait_test)
    int overlap;
    cudaStream_t stream;
};

// k_seq_rows.cu: a block of few query rows against a stretch of keys
int64_t rows_workspace_bytes(const softmax_sequence_args_t &a, int sms);
cudaError_t launch_rows(const AttnCall &c);
cudaError_t read_clear_rows_error_word(unsigned int *word);

// k_seq_tiles.cu: tiles of many query rows on the tensor cores
int64_t tiles_workspace_bytes(const softmax_sequence_args_t &a, int sms);
cudaError_t launch_tiles(const AttnCall &c);
cudaError_t read_clear_tiles_error_word(unsigned int *word);

// sequence_abi.cu: both kernels' words
cudaError_t read_clear_sequence_error_word(unsigned int *word);

}  // namespace seq
}  // namespace mbrs
