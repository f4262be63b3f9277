// spa_errors.h - the device error words of the translation units that have no host call of their own to
// read them (see spa_device.cuh), read and cleared together.
#pragma once
#include <cuda_runtime.h>

namespace spa {

// Address of a unit's word on the current device.
cudaError_t indexer_error_word(int** word);
cudaError_t latent_cache_error_word(int** word);
cudaError_t latent_decode_error_word(int** word);
cudaError_t latent_prefill_error_word(int** word);

// The OR of those words on the current device, which are cleared: one kernel and one copy, whatever their
// number, where a read and a clear of each are two blocking copies a word.
cudaError_t collect_error_words(int* value);

}  // namespace spa
