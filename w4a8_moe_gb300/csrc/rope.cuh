// Norm and rotation of queries and keys: launch parameters (rope.cu).
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "kv8.cuh"

namespace w4a8 {

constexpr int kRopeMostD = 256;

struct Rope {
    const uint16_t* q;   // bf16 [T, Hq, D], [T, Hkv, D]; rows *_stride elements apart
    const uint16_t* k;
    const uint16_t* v;   // read only where a cache is written
    int64_t q_stride, k_stride, v_stride;
    int T, Hq, Hkv, D, rot;
    const int32_t* positions;
    const uint64_t* turns;   // [rot / 2] turns per position, times 2^64
    float magnitude;
    int interleaved;
    const uint16_t* q_weight;   // bf16 [D], null: no norm
    const uint16_t* k_weight;
    float eps, inv_d;   // 1 / D
    uint16_t* q_out;
    uint16_t* k_out;   // null where a cache is written
    int64_t q_out_stride, k_out_stride;
    // the cache, where one is written
    const int32_t* slots;
    uint8_t* k_cache;
    uint8_t* v_cache;
    float* k_scale;
    float* v_scale;
    int num_slots, page_shift, per_token;
    float min_scale;
    int tokens, slice;   // tokens of a block, rows (heads) of each
};
// Where `to_cache` is set the keys and values go into the cache, else the keys to k_out.
cudaError_t launch_rope(const Rope& a, bool to_cache, int num_sms, cudaStream_t s);

}  // namespace w4a8
