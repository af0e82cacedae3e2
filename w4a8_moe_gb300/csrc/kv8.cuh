// Shared pieces of the FP8 key/value cache kernels (kv8.cu, kv8_attn.cu):
// launch parameters, the work split of the attention, E4M3 -> f16 conversion.
#pragma once
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace w4a8 {

constexpr uint32_t kErrBitIndex = 2u;  // a page index or a length was out of range

// ---- cache: E4M3 codes [num_pages, Hkv, page_size, D], page_size = 1 << page_shift.
struct Kv8Rows {            // arguments of the write and the read
    int T, Hkv, D;
    int num_slots;          // num_pages * page_size
    int page_shift;
    int per_token;          // scales: 0 one per head, 1 one per token and head
    float min_scale;
    int64_t k_stride, v_stride;   // elements between two tokens' rows
};
cudaError_t launch_kv8_write(const Kv8Rows& a, const uint16_t* k, const uint16_t* v, const int32_t* slots,
                             uint8_t* k_cache, uint8_t* v_cache, float* k_scale, float* v_scale, cudaStream_t s);
cudaError_t launch_kv8_read(const Kv8Rows& a, const uint8_t* k_cache, const uint8_t* v_cache, const float* k_scale,
                            const float* v_scale, const int32_t* slots, uint16_t* k, uint16_t* v, cudaStream_t s);

// ---- attention
constexpr int kKv8MaxBatch = 4096;  // the split's prefix sums live in shared memory
constexpr int kKv8Unit = 16;        // keys per unit of the split (a unit never crosses a page)
constexpr int kKv8MaxWarps = 152 * 16;   // warps the units are divided over, at most

struct Kv8Attn {
    const uint16_t* q;
    int64_t q_stride;
    int B, Hq, Hkv, group;
    const uint8_t* k_cache;
    const uint8_t* v_cache;
    const float* k_scale;
    const float* v_scale;
    int num_pages, page_shift;
    const int32_t* prefix_pages;
    int prefix_len;
    const int32_t* page_table;
    int64_t table_stride;
    int max_pages;
    const int32_t* lens;
    float sm_scale, cap;
    int tiles;          // row tiles of a sequence's query heads that share a kv head
    int ptiles;         // row tiles of the whole batch over the prefix (0: no prefix here)
    float* part_o;      // [slot][row of the tile][D], not divided by the sum
    float2* part_ml;    // [slot][row of the tile]: reference exponent (log2), sum
    uint32_t* err;
    uint16_t* out;
    float* lse;
    int warps;          // that the units go to
    int free_warps;     // of them those that need not wait for the tiled prefix
    int spread;         // warps up to which the units are spread by twos
    float free_us;      // that the others wait, about
    int beside;         // a tiled prefix runs beside
    int* cum;           // [B + 1] prefix sums of the sequences' units, left for the join
};
// The prefix on the tensor cores: CTAs of (kv head, 256 rows, a range of key
// tiles); part_* [split][kv head][row] as above.
constexpr int kKv8PrefixCtas = 152;  // SMs the workspace is sized for
constexpr int kKv8MaxSplits = 64;
struct Kv8Prefix {
    int tiles;            // 128-key tiles of the prefix
    int row_pairs;        // pairs of 128-row tiles
    int splits, tiles_per_split;
    float us;             // about how long it takes
    float* part_o;
    float2* part_ml;
};
int kv8_prefix_most_splits(int Hkv, int rows, int prefix_len);
int64_t kv8_prefix_most_rows(int Hkv, int rows, int prefix_len);
Kv8Prefix kv8_prefix_plan(int Hkv, int rows, int prefix_len, int D, float tile_us, int64_t own_max, int num_sms);
cudaError_t launch_kv8_prefix(const Kv8Attn& a, const Kv8Prefix& p, int D, int per_token, cudaStream_t s);
bool kv8_prefix_tiled(int Hkv, int rows, int prefix_len);
int kv8_attn_row_tile(int group);
void kv8_attn_layout(const Kv8Attn& a, const Kv8Prefix& p, int D, int num_sms, int* blocks_per_sm, int* warps_a_row);
cudaError_t launch_kv8_attn(const Kv8Attn& a, const Kv8Prefix& p, int D, int per_token, int num_sms, cudaStream_t s);

// Two E4M3 codes (low byte first) to two f16 values: exact for every code.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t pair)
{
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(pair)));
    return r;
}

// Four codes to two registers of two.
__device__ __forceinline__ void e4m3x4_to_f16x4(uint32_t w, uint32_t& lo, uint32_t& hi)
{
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}

// A softmax weight goes into the second product in f16, relative to its row's
// running reference. The reference is raised only when a weight would pass
// 2^kWeightMost over it, and then to 2^kWeightTop under the largest one. So the
// heaviest key of a piece stands 2^kWeightTop over f16's 1 at least, a weight loses
// bits only below 2^-22 of that one, and none of them loses more than 2^-33 of it:
// many light keys beside one that has nearly all of the weight, but no value, still
// add up right. What is left above is for the maximum to grow without the
// accumulators being rescaled (kWeightTop 7 / 8 / 10, us: 128 sequences over 32768
// tokens 101.7 / 102.2 / 103.8, 256 over 65536 260.6 / 261.4 / 264.2).
constexpr float kWeightTop = 8.0f;
constexpr float kWeightMost = 15.0f;
// Per-token scales: what is compared, and what goes into f16, is the weight times
// its value's scale (the reference then carries the values' size too, and drops out
// of o / l), the largest of these products of single keys; a key whose values are
// all zero has none. Smaller scales count as kLeastScale there, which keeps the
// weights themselves inside fp32: 2^100 where the reference was raised, 2^107 at
// most, added up over the keys of a piece.
constexpr float kLeastScale = 0x1p-92f;
constexpr float kLeastScaleLog2 = -92.0f;

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ex2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// Untiled copy global -> shared, counted on an mbarrier; 16-byte addresses and size.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t at)
{
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
    return v;
}
// Two fp32 operations in one instruction.
struct F2 {
    uint64_t v;
    __device__ __forceinline__ F2(float lo, float hi) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi)); }
    __device__ __forceinline__ explicit F2(uint64_t x) : v(x) {}
    __device__ __forceinline__ float lo() const { return __uint_as_float(static_cast<uint32_t>(v)); }
    __device__ __forceinline__ float hi() const { return __uint_as_float(static_cast<uint32_t>(v >> 32)); }
};
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a.v), "l"(b.v), "l"(c.v));
    return F2(r);
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a.v), "l"(b.v));
    return F2(r);
}
__device__ __forceinline__ F2 add2(F2 a, F2 b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a.v), "l"(b.v));
    return F2(r);
}
__device__ __forceinline__ float rcp(float x)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

}  // namespace w4a8
