// Page tables and slots of a step's new tokens: launch parameters (pages.cu).
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

namespace w4a8 {

constexpr int kPagesMostSeqs = 4096;   // their prefix sums live in shared memory

struct PagePool {
    int32_t* table;   // [B, max_pages], rows `stride` apart
    int64_t stride;
    int max_pages;
    int32_t* stack;   // [num_pages] pages that nobody has, the top last
    int32_t* count;   // [1] how many
    int num_pages, page_shift;
    uint32_t* err;
    uint32_t* ticket;   // blocks that have read the lengths and the count; zero between calls
};
struct PagesExtend {
    PagePool p;
    int B, T;              // sequences; tokens that the outputs have room for
    const int32_t* lens;
    const int32_t* add;    // new tokens of each sequence
    int32_t* starts;       // [B + 1]
    int32_t* seqs;         // [T] and the next three
    int32_t* positions;
    int32_t* seen;
    int32_t* slots;
    int32_t* lens_out;     // may be lens
};
struct PagesTruncate {
    PagePool p;
    int B;
    const int32_t* lens;
    const int32_t* keep;
    int32_t* lens_out;   // may be lens or keep
};
cudaError_t launch_pages_extend(const PagesExtend& a, int num_sms, cudaStream_t s);
cudaError_t launch_pages_truncate(const PagesTruncate& a, int num_sms, cudaStream_t s);

}  // namespace w4a8
