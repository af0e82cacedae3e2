// FP8 key/value cache: quantizing the keys and values of a call's tokens into
// their slots, and reading slots back as bf16.
//
// "ROCm: enable trillion-parameter MoE models with INT4-FP8 single node",
// config.json quantization_config (kv_cache_scheme: FP8, static scale;
// min_kv_scale): the KV8 of W4A8KV8.
#include "internal.h"
#include "kv8.cuh"
#include "ptx.cuh"

namespace w4a8 {

namespace {

constexpr int kRowThreads = 256;

// A row is one (token, keys or values, head): D values. A lane takes 8 values
// (16 bytes of bf16) out of each of two halves of the row, so D / 16 lanes
// share a row and every load and store of a warp covers whole 32-byte sectors.
// Rows are numbered token first, then keys / values, then head: a warp's rows
// are neighbours in the bf16 tensors.
struct RowAt {
    int t, h;
    bool is_v;
    bool live;
    int64_t slot;
};
template <int D>
__device__ __forceinline__ RowAt row_at(const Kv8Rows& a, const int32_t* __restrict__ slots)
{
    RowAt r;
    const int64_t row = (static_cast<int64_t>(blockIdx.x) * kRowThreads + threadIdx.x) / (D / 16);
    const int64_t per = 2 * a.Hkv;
    r.t = static_cast<int>(row / per);
    const int rem = static_cast<int>(row - r.t * per);
    r.is_v = rem >= a.Hkv;
    r.h = r.is_v ? rem - a.Hkv : rem;
    r.live = r.t < a.T;
    r.slot = r.live ? __ldg(slots + r.t) : -1;
    return r;
}
__device__ __forceinline__ int64_t cache_row(const Kv8Rows& a, int64_t slot, int h)
{
    const int64_t page = slot >> a.page_shift;
    const int64_t off = slot & ((1 << a.page_shift) - 1);
    return ((page * a.Hkv + h) << a.page_shift) + off;
}

}  // namespace

// code = E4M3(x / s): fp32 division, round to nearest even, saturating; a NaN
// keeps the NaN code. Per-token scales come from the row itself:
// s = max(max over the finite |x| / 448, min_scale), 1 where that is 0.
template <int D>
__global__ void __launch_bounds__(kRowThreads) kv8_write_kernel(const __grid_constant__ Kv8Rows a,
                                                                const uint16_t* __restrict__ k,
                                                                const uint16_t* __restrict__ v,
                                                                const int32_t* __restrict__ slots,
                                                                uint8_t* __restrict__ k_cache,
                                                                uint8_t* __restrict__ v_cache,
                                                                float* __restrict__ k_scale,
                                                                float* __restrict__ v_scale)
{
    constexpr int L = D / 16;
    const RowAt r = row_at<D>(a, slots);
    const int lane = threadIdx.x % L;
    const bool ok = r.live && r.slot >= 0 && r.slot < a.num_slots;
    const uint16_t* src = r.is_v ? v + r.t * a.v_stride : k + r.t * a.k_stride;
    uint4 raw[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    if (ok) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            raw[i] = __ldg(reinterpret_cast<const uint4*>(src + static_cast<int64_t>(r.h) * D) + i * L + lane);
    }
    float x[2][8];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t u[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[i][2 * j] = __uint_as_float(u[j] << 16);
            x[i][2 * j + 1] = __uint_as_float(u[j] & 0xFFFF0000u);
        }
    }
    float s;
    float* scale = r.is_v ? v_scale : k_scale;
    if (a.per_token) {
        float amax = 0.0f;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float m = fabsf(x[i][j]);
                amax = m < __int_as_float(0x7F800000) ? fmaxf(amax, m) : amax;
            }
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1)
            amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
        s = fmaxf(__fdiv_rn(amax, 448.0f), a.min_scale);
        s = s == 0.0f ? 1.0f : s;
    } else {
        s = ok ? __ldg(scale + r.h) : 1.0f;
    }
    if (!ok)
        return;
    const int64_t at = cache_row(a, r.slot, r.h);
    uint8_t* dst = (r.is_v ? v_cache : k_cache) + at * D;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint32_t c[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            c[j] = cvt_e4m3x2(__fdiv_rn(x[i][2 * j + 1], s), __fdiv_rn(x[i][2 * j], s));
        *(reinterpret_cast<uint2*>(dst) + i * L + lane) = make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
    }
    if (a.per_token && lane == 0)
        scale[at] = s;
}

// x = bf16(dec(code) * s); rows whose slot is out of range are zero.
template <int D>
__global__ void __launch_bounds__(kRowThreads) kv8_read_kernel(const __grid_constant__ Kv8Rows a,
                                                               const uint8_t* __restrict__ k_cache,
                                                               const uint8_t* __restrict__ v_cache,
                                                               const float* __restrict__ k_scale,
                                                               const float* __restrict__ v_scale,
                                                               const int32_t* __restrict__ slots,
                                                               uint16_t* __restrict__ k, uint16_t* __restrict__ v)
{
    constexpr int L = D / 16;
    const RowAt r = row_at<D>(a, slots);
    if (!r.live)
        return;
    const int lane = threadIdx.x % L;
    uint2 raw[2] = {make_uint2(0, 0), make_uint2(0, 0)};
    float s = 0.0f;
    if (r.slot >= 0 && r.slot < a.num_slots) {
        const int64_t at = cache_row(a, r.slot, r.h);
        const uint2* src = reinterpret_cast<const uint2*>((r.is_v ? v_cache : k_cache) + at * D);
#pragma unroll
        for (int i = 0; i < 2; ++i)
            raw[i] = __ldg(src + i * L + lane);
        s = __ldg((r.is_v ? v_scale : k_scale) + (a.per_token ? at : r.h));
    }
    uint16_t* dst = (r.is_v ? v + r.t * a.v_stride : k + r.t * a.k_stride) + static_cast<int64_t>(r.h) * D;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t w[4] = {raw[i].x & 0xFFFFu, raw[i].x >> 16, raw[i].y & 0xFFFFu, raw[i].y >> 16};
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t h2 = e4m3x2_to_f16x2(w[j]);
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
            o[j] = static_cast<uint32_t>(float_to_bf16_bits(f.x * s)) |
                   (static_cast<uint32_t>(float_to_bf16_bits(f.y * s)) << 16);
        }
        *(reinterpret_cast<uint4*>(dst) + i * L + lane) = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

static unsigned row_blocks(const Kv8Rows& a)
{
    const int64_t threads = static_cast<int64_t>(a.T) * a.Hkv * 2 * (a.D / 16);
    return static_cast<unsigned>((threads + kRowThreads - 1) / kRowThreads);
}

cudaError_t launch_kv8_write(const Kv8Rows& a, const uint16_t* k, const uint16_t* v, const int32_t* slots,
                             uint8_t* k_cache, uint8_t* v_cache, float* k_scale, float* v_scale, cudaStream_t s)
{
    if (a.D == 128)
        kv8_write_kernel<128><<<row_blocks(a), kRowThreads, 0, s>>>(a, k, v, slots, k_cache, v_cache, k_scale, v_scale);
    else
        kv8_write_kernel<64><<<row_blocks(a), kRowThreads, 0, s>>>(a, k, v, slots, k_cache, v_cache, k_scale, v_scale);
    return cudaGetLastError();
}

cudaError_t launch_kv8_read(const Kv8Rows& a, const uint8_t* k_cache, const uint8_t* v_cache, const float* k_scale,
                            const float* v_scale, const int32_t* slots, uint16_t* k, uint16_t* v, cudaStream_t s)
{
    if (a.D == 128)
        kv8_read_kernel<128><<<row_blocks(a), kRowThreads, 0, s>>>(a, k_cache, v_cache, k_scale, v_scale, slots, k, v);
    else
        kv8_read_kernel<64><<<row_blocks(a), kRowThreads, 0, s>>>(a, k_cache, v_cache, k_scale, v_scale, slots, k, v);
    return cudaGetLastError();
}

}  // namespace w4a8
