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

// A row is one (token, head), its keys and its values: D values each. A lane
// takes 8 values (16 bytes of bf16) out of each half of both, so D / 16 lanes
// share a row, every load and store of a warp covers whole 32-byte sectors, and
// a lane has all of its loads in flight together after the slot's.
struct RowAt {
    int t, h;
    bool live;
    int64_t slot;
};
template <int D>
__device__ __forceinline__ RowAt row_at(const Kv8Rows& a, const int32_t* __restrict__ slots)
{
    RowAt r;
    const int64_t row = (static_cast<int64_t>(blockIdx.x) * kRowThreads + threadIdx.x) / (D / 16);
    const unsigned n = static_cast<unsigned>(row);   // T * Hkv < 2^31, and the grid ends less than a block behind
    r.t = static_cast<int>(n / static_cast<unsigned>(a.Hkv));
    r.h = static_cast<int>(n - static_cast<unsigned>(r.t) * a.Hkv);
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

// E4M3(x / s) of 16 values, the quotient rounded to fp32 first (as the format's
// definition here says). A correctly rounded fp32 division of every value is
// most of the call's arithmetic, so the quotient is taken as q = x * (1 / s):
// that is within 2^-22 of x / s, which changes the code only where a rounding
// boundary of E4M3 lies that close to q. Boundaries have the low 20 bits
// 0x80000 (4 significant bits and a half) or, below 2^-6, 0 (odd multiples of
// 2^-10); a thread with any q within 4 units of either divides. With s a power
// of two the product is exact and none needs it; where 1 / s could leave the
// normal range all divide. Measured at 32768 tokens of 8 heads: see
// kv8_write_kernel.
__device__ __forceinline__ void encode16(const float (&x)[2][8], float s, uint32_t (&c)[2][4])
{
    const uint32_t sb = __float_as_uint(s);
    const bool plain = sb - 0x04000000u < 0x78000000u;   // 2^-119 <= s < 2^121
    const bool power = (sb & 0x7FFFFFu) == 0;
    const float r = __fdiv_rn(1.0f, s);
    uint32_t nearest = 0x7FFFFu;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float lo = x[i][2 * j] * r, hi = x[i][2 * j + 1] * r;
            nearest = min(nearest, (__float_as_uint(lo) + 4u) & 0x7FFFFu);
            nearest = min(nearest, (__float_as_uint(hi) + 4u) & 0x7FFFFu);
            c[i][j] = cvt_e4m3x2(hi, lo);
        }
    if (!plain || (nearest <= 8u && !power)) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                c[i][j] = cvt_e4m3x2(__fdiv_rn(x[i][2 * j + 1], s), __fdiv_rn(x[i][2 * j], s));
    }
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
    uint4 raw[2][2];
#pragma unroll
    for (int y = 0; y < 2; ++y) {
        const uint16_t* src = (y ? v + r.t * a.v_stride : k + r.t * a.k_stride) + static_cast<int64_t>(r.h) * D;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            raw[y][i] = ok ? __ldg(reinterpret_cast<const uint4*>(src) + i * L + lane) : make_uint4(0, 0, 0, 0);
    }
    const int64_t at = ok ? cache_row(a, r.slot, r.h) : 0;
#pragma unroll
    for (int y = 0; y < 2; ++y) {
        float x[2][8];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t u[4] = {raw[y][i].x, raw[y][i].y, raw[y][i].z, raw[y][i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[i][2 * j] = __uint_as_float(u[j] << 16);
                x[i][2 * j + 1] = __uint_as_float(u[j] & 0xFFFF0000u);
            }
        }
        float s;
        float* scale = y ? v_scale : k_scale;
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
        if (ok) {
            uint32_t c[2][4];
            encode16(x, s, c);
            uint2* dst = reinterpret_cast<uint2*>((y ? v_cache : k_cache) + at * D);
#pragma unroll
            for (int i = 0; i < 2; ++i)
                dst[i * L + lane] = make_uint2(c[i][0] | (c[i][1] << 16), c[i][2] | (c[i][3] << 16));
            if (a.per_token && lane == 0)
                scale[at] = s;
        }
    }
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
    uint2 raw[2][2] = {{make_uint2(0, 0), make_uint2(0, 0)}, {make_uint2(0, 0), make_uint2(0, 0)}};
    float s[2] = {0.0f, 0.0f};
    if (r.slot >= 0 && r.slot < a.num_slots) {
        const int64_t at = cache_row(a, r.slot, r.h);
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            const uint2* src = reinterpret_cast<const uint2*>((y ? v_cache : k_cache) + at * D);
#pragma unroll
            for (int i = 0; i < 2; ++i)
                raw[y][i] = __ldg(src + i * L + lane);
            s[y] = __ldg((y ? v_scale : k_scale) + (a.per_token ? at : r.h));
        }
    }
#pragma unroll
    for (int y = 0; y < 2; ++y) {
        uint16_t* dst = (y ? v + r.t * a.v_stride : k + r.t * a.k_stride) + static_cast<int64_t>(r.h) * D;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t w[4] = {raw[y][i].x & 0xFFFFu, raw[y][i].x >> 16, raw[y][i].y & 0xFFFFu, raw[y][i].y >> 16};
            uint32_t o[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t h2 = e4m3x2_to_f16x2(w[j]);
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
                o[j] = static_cast<uint32_t>(float_to_bf16_bits(f.x * s[y])) |
                       (static_cast<uint32_t>(float_to_bf16_bits(f.y * s[y])) << 16);
            }
            *(reinterpret_cast<uint4*>(dst) + i * L + lane) = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
}

static unsigned row_blocks(const Kv8Rows& a)
{
    const int64_t threads = static_cast<int64_t>(a.T) * a.Hkv * (a.D / 16);
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
