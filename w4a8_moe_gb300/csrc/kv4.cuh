// Key/value cache of 4 bits: launch parameters (kv4.cu, kv4_attn.cu).
//
// A row is one head of one token: D codes of 4 bits, the even value of a byte in
// its low half, and with them two bf16 numbers, the step s and the least value m;
// a code c stands for c s + m.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "kv8.cuh"

namespace w4a8 {

cudaError_t launch_kv4_write(const Kv8Rows& a, const uint16_t* k, const uint16_t* v, const int32_t* slots,
                             uint8_t* k_cache, uint8_t* v_cache, uint32_t* k_scale, uint32_t* v_scale, cudaStream_t s);
cudaError_t launch_kv4_read(const Kv8Rows& a, const uint8_t* k_cache, const uint8_t* v_cache, const uint32_t* k_scale,
                            const uint32_t* v_scale, const int32_t* slots, uint16_t* k, uint16_t* v, cudaStream_t s);

// Decode attention: the rows of the batch are query tokens, each with its own
// length (`lens`). The scale pointers of the base are those of the pairs above.
struct Kv4Attn : Kv8Attn {
    int per_tile;   // tokens of a sequence that a tile of rows holds
};
cudaError_t launch_kv4_attn(const Kv4Attn& a, int D, int num_sms, cudaStream_t s);

}  // namespace w4a8
