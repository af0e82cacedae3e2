// Key/value cache of 4 bits: quantizing the keys and values of a call's tokens into
// their slots, and reading slots back as bf16.
//
// "ROCm: enable trillion-parameter MoE models with INT4-FP8 single node",
// config.json quantization_config (int4_experts; kv_cache_scheme): the KV8 of
// W4A8KV8 taken down to the width of its weights, one scale per token and head.
//
//   m = min x,  s = bf16((max x - min x) / 15),  c = clamp(rint((x - m) / s), 0, 15)
// m is one of the row's own bf16 values, so it is kept without a rounding.
#include <math.h>

#include "internal.h"
#include "kv4.cuh"
#include "ptx.cuh"

namespace w4a8 {

namespace {

constexpr int kRowThreads = 128;

// A row's keys and values, D of each; D / 16 lanes share it, 16 values of both a
// lane: 32 bytes of bf16 and 8 bytes of codes, whole sectors for the warp.
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

// Codes of 16 values: rint((x - m) / s) in 0..15, the difference and the quotient
// rounded to fp32 each. The quotient is q = d r with r = 1 / s correctly rounded and
// one correction, q + (d - q s) r, which rounds like the division where nothing
// under- or overflows (Markstein 1990, as in the FP8 cache's encoder): 2^-60 <= s <
// 2^60, and |d| <= 15.06 s for every value of the row; differences below 2^-11 s have
// the code 0 either way. Other rows divide halves, which cannot overflow.
__device__ __forceinline__ uint2 encode_row16(const float (&x)[16], bool finite, float m, float s)
{
    uint32_t c[16];
    const bool plain = finite && s >= 8.6736174e-19f && s < 1.1529215e18f && fabsf(m) < 1.1529215e18f;
    if (plain) {
        const float r = __frcp_rn(s);
        const F2 r2(r, r), s2(-s, -s), m2(-m, -m);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const F2 d = add2(F2(x[2 * j], x[2 * j + 1]), m2), q = mul2(d, r2);
            const F2 y = fma2(fma2(q, s2, d), r2, q);
            c[2 * j] = static_cast<uint32_t>(min(max(__float2int_rn(y.lo()), 0), 15));
            c[2 * j + 1] = static_cast<uint32_t>(min(max(__float2int_rn(y.hi()), 0), 15));
        }
    } else {
#pragma unroll
        for (int j = 0; j < 16; ++j)
            c[j] = s > 0.0f ? static_cast<uint32_t>(
                                  min(max(__float2int_rn(__fdiv_rn(0.5f * x[j] - 0.5f * m, 0.5f * s)), 0), 15))
                            : 0;
    }
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 16; ++j)
        w[j / 8] |= c[j] << (4 * (j % 8));
    return make_uint2(w[0], w[1]);
}

}  // namespace

template <int D>
__global__ void __launch_bounds__(kRowThreads) kv4_write_kernel(const __grid_constant__ Kv8Rows a,
                                                                const uint16_t* __restrict__ k,
                                                                const uint16_t* __restrict__ v,
                                                                const int32_t* __restrict__ slots,
                                                                uint8_t* __restrict__ k_cache,
                                                                uint8_t* __restrict__ v_cache,
                                                                uint32_t* __restrict__ k_scale,
                                                                uint32_t* __restrict__ v_scale)
{
    constexpr int L = D / 16;
    grid_dep_wait();
    const RowAt r = row_at<D>(a, slots);
    const int lane = threadIdx.x % L;
    uint4 raw[2][2];   // read whatever the slot is: the loads need not wait for it
#pragma unroll
    for (int y = 0; y < 2; ++y) {
        const uint16_t* src = (y ? v + r.t * a.v_stride : k + r.t * a.k_stride) + static_cast<int64_t>(r.h) * D;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            raw[y][i] = r.live ? __ldg(reinterpret_cast<const uint4*>(src) + lane * 2 + i) : make_uint4(0, 0, 0, 0);
    }
    const bool ok = r.live && r.slot >= 0 && r.slot < a.num_slots;
    const int64_t at = ok ? cache_row(a.page_shift, a.Hkv, r.slot, r.h) : 0;
#pragma unroll
    for (int y = 0; y < 2; ++y) {
        float x[16];
        unpack16(raw[y], x);
        // over the finite values; a NaN anywhere leaves the row without numbers
        float lo = INFINITY, hi = -INFINITY, odd = 0.0f;   // odd: NaN where a value is not finite
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            lo = fminf(lo, x[i]);
            hi = fmaxf(hi, x[i]);
            odd += 0.0f * x[i];
        }
        const bool finite = odd == 0.0f;
        if (__any_sync(0xFFFFFFFFu, !finite)) {
            lo = INFINITY, hi = -INFINITY, odd = 0.0f;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                if (fabsf(x[i]) < INFINITY)
                    lo = fminf(lo, x[i]), hi = fmaxf(hi, x[i]);
                odd = isnan(x[i]) ? x[i] : odd;
            }
        }
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) {
            lo = fminf(lo, __shfl_xor_sync(0xFFFFFFFFu, lo, o));
            hi = fmaxf(hi, __shfl_xor_sync(0xFFFFFFFFu, hi, o));
            odd += __shfl_xor_sync(0xFFFFFFFFu, odd, o);
        }
        if (hi < lo)   // nothing finite
            lo = hi = 0.0f;
        uint16_t s_bits = float_to_bf16_bits(__fdiv_rn(0.5f * hi - 0.5f * lo, 7.5f));   // halves cannot overflow
        uint16_t m_bits = float_to_bf16_bits(lo);   // exact
        if (isnan(odd))
            s_bits = m_bits = 0x7FC0u;
        if (ok) {
            uint8_t* dst = (y ? v_cache : k_cache) + at * (D / 2);
            *(reinterpret_cast<uint2*>(dst) + lane) =
                isnan(odd) ? make_uint2(0, 0) : encode_row16(x, finite, lo, bf16_bits_to_float(s_bits));
            if (lane == 0)
                (y ? v_scale : k_scale)[at] = s_bits | (static_cast<uint32_t>(m_bits) << 16);
        }
    }
}

// x = bf16(c s + m); rows whose slot is out of range are zero.
template <int D>
__global__ void __launch_bounds__(kRowThreads) kv4_read_kernel(const __grid_constant__ Kv8Rows a,
                                                               const uint8_t* __restrict__ k_cache,
                                                               const uint8_t* __restrict__ v_cache,
                                                               const uint32_t* __restrict__ k_scale,
                                                               const uint32_t* __restrict__ v_scale,
                                                               const int32_t* __restrict__ slots,
                                                               uint16_t* __restrict__ k, uint16_t* __restrict__ v)
{
    constexpr int L = D / 16;
    grid_dep_wait();
    const RowAt r = row_at<D>(a, slots);
    if (!r.live)
        return;
    const int lane = threadIdx.x % L;
    uint2 raw[2] = {make_uint2(0, 0), make_uint2(0, 0)};
    uint32_t pair[2] = {0, 0};
    if (r.slot >= 0 && r.slot < a.num_slots) {
        const int64_t at = cache_row(a.page_shift, a.Hkv, r.slot, r.h);
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            raw[y] = __ldg(reinterpret_cast<const uint2*>((y ? v_cache : k_cache) + at * (D / 2)) + lane);
            pair[y] = __ldg((y ? v_scale : k_scale) + at);
        }
    }
#pragma unroll
    for (int y = 0; y < 2; ++y) {
        const float s = __uint_as_float(pair[y] << 16), m = __uint_as_float(pair[y] & 0xFFFF0000u);
        uint16_t* dst = (y ? v + r.t * a.v_stride : k + r.t * a.k_stride) + static_cast<int64_t>(r.h) * D;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t w = i ? raw[y].y : raw[y].x;
            uint32_t o[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float x0 = fmaf(static_cast<float>((w >> (8 * j)) & 15u), s, m);
                const float x1 = fmaf(static_cast<float>((w >> (8 * j + 4)) & 15u), s, m);
                o[j] = static_cast<uint32_t>(float_to_bf16_bits(x0)) |
                       (static_cast<uint32_t>(float_to_bf16_bits(x1)) << 16);
            }
            *(reinterpret_cast<uint4*>(dst) + lane * 2 + i) = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
}

static unsigned row_blocks(const Kv8Rows& a)
{
    const int64_t threads = static_cast<int64_t>(a.T) * a.Hkv * (a.D / 16);
    return static_cast<unsigned>((threads + kRowThreads - 1) / kRowThreads);
}

cudaError_t launch_kv4_write(const Kv8Rows& a, const uint16_t* k, const uint16_t* v, const int32_t* slots,
                             uint8_t* k_cache, uint8_t* v_cache, uint32_t* k_scale, uint32_t* v_scale, cudaStream_t s)
{
    return launch_dependent(a.D == 128 ? kv4_write_kernel<128> : kv4_write_kernel<64>, dim3(row_blocks(a)),
                            dim3(kRowThreads), 0, s, a, k, v, slots, k_cache, v_cache, k_scale, v_scale);
}

cudaError_t launch_kv4_read(const Kv8Rows& a, const uint8_t* k_cache, const uint8_t* v_cache, const uint32_t* k_scale,
                            const uint32_t* v_scale, const int32_t* slots, uint16_t* k, uint16_t* v, cudaStream_t s)
{
    return launch_dependent(a.D == 128 ? kv4_read_kernel<128> : kv4_read_kernel<64>, dim3(row_blocks(a)),
                            dim3(kRowThreads), 0, s, a, k_cache, v_cache, k_scale, v_scale, slots, k, v);
}

}  // namespace w4a8
