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

// A row's keys and values, D of each; D / 16 lanes share it, a lane taking 8 values
// (16 bytes of bf16, 4 of codes) out of each half of both, so that every load and
// store of a warp covers whole 32-byte sectors.
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
// 2^60, and 0 <= d <= 15.06 s for every value of a row, as s is at most 2^-8 off;
// differences below 2^-11 s have the code 0 either way. Such a quotient rounds to 0..15
// by itself, and added to 1.5 * 2^23 it does so into the sum's lowest bits, where codes
// are put together by multiplying by 16. Other rows divide halves, which cannot
// overflow.
__device__ __forceinline__ uint2 encode_row16(const float (&x)[16], bool finite, float m, float s)
{
    uint32_t w[2];
    const bool plain = finite && s >= 8.6736174e-19f && s < 1.1529215e18f && fabsf(m) < 1.1529215e18f;
    if (plain) {
        const float r = __frcp_rn(s);
        const F2 r2(r, r), s2(-s, -s), m2(-m, -m), round2(12582912.0f, 12582912.0f);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t sum = 0;
#pragma unroll
            for (int j = 3; j >= 0; --j) {
                const F2 d = add2(F2(x[8 * i + 2 * j], x[8 * i + 2 * j + 1]), m2), q = mul2(d, r2);
                const F2 y = add2(fma2(fma2(q, s2, d), r2, q), round2);
                sum = sum * 256 + __float_as_uint(y.hi()) * 16 + __float_as_uint(y.lo());
            }
            w[i] = sum - 0x4B400000u * 0x11111111u;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            w[i] = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float y = __fdiv_rn(0.5f * x[8 * i + j] - 0.5f * m, 0.5f * s);
                w[i] |= s > 0.0f ? static_cast<uint32_t>(min(max(__float2int_rn(y), 0), 15)) << (4 * j) : 0;
            }
        }
    }
    return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b)   // NaN where one of them is
{
    asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(a) : "r"(b));
    return a;
}
// The largest value of a row (high half) and the largest of its negatives (low half),
// 16 values here and those of the other lanes; NaN where a value is.
template <int L>
__device__ __forceinline__ uint32_t bounds(const uint4 (&raw)[2])
{
    const uint32_t u[8] = {raw[0].x, raw[0].y, raw[0].z, raw[0].w, raw[1].x, raw[1].y, raw[1].z, raw[1].w};
    uint32_t hi = u[0], lo = u[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) {
        hi = max_bf16x2(hi, u[i]);
        asm("min.NaN.bf16x2 %0, %0, %1;" : "+r"(lo) : "r"(u[i]));
    }
    lo ^= 0x80008000u;
    uint32_t r = max_bf16x2(prmt(lo, hi, 0x5410), prmt(lo, hi, 0x7632));
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1)
        r = max_bf16x2(r, __shfl_xor_sync(0xFFFFFFFFu, r, o));
    return r;
}

}  // namespace

// 32768 tokens of 8 heads of 128 (172 MB): 34.3 us, 5.0 TB/s or 74 % of a copy's rate;
// the arithmetic of 16 codes, some 200 instructions a lane, bounds it as much as memory
// does (with a conversion and two bounds for each code 35.5 us, 12 blocks an SM 34.3 / as
// many as registers would leave, 10, 35.5). 256 tokens take 2.7 us.
template <int D>
__global__ void __launch_bounds__(kRowThreads, 12) kv4_write_kernel(const __grid_constant__ Kv8Rows a,
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
            raw[y][i] = r.live ? __ldg(reinterpret_cast<const uint4*>(src) + i * L + lane) : make_uint4(0, 0, 0, 0);
    }
    const bool ok = r.live && r.slot >= 0 && r.slot < a.num_slots;
    const int64_t at = ok ? cache_row(a.page_shift, a.Hkv, r.slot, r.h) : 0;
#pragma unroll
    for (int y = 0; y < 2; ++y) {
        float x[16];
        unpack16(raw[y], x);
        const uint32_t ends = bounds<L>(raw[y]);
        float lo = -__uint_as_float(ends << 16), hi = __uint_as_float(ends & 0xFFFF0000u), odd = 0.0f;
        const bool finite = fabsf(lo) < INFINITY && fabsf(hi) < INFINITY;   // all of the row
        if (__any_sync(0xFFFFFFFFu, !finite)) {
            // over the finite values; a NaN anywhere leaves the row without numbers
            lo = INFINITY, hi = -INFINITY;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                if (fabsf(x[i]) < INFINITY)
                    lo = fminf(lo, x[i]), hi = fmaxf(hi, x[i]);
                odd = isnan(x[i]) ? x[i] : odd;
            }
#pragma unroll
            for (int o = L / 2; o > 0; o >>= 1) {
                lo = fminf(lo, __shfl_xor_sync(0xFFFFFFFFu, lo, o));
                hi = fmaxf(hi, __shfl_xor_sync(0xFFFFFFFFu, hi, o));
                odd += __shfl_xor_sync(0xFFFFFFFFu, odd, o);
            }
        }
        if (hi < lo)   // nothing finite
            lo = hi = 0.0f;
        uint16_t s_bits = float_to_bf16_bits(__fdiv_rn(0.5f * hi - 0.5f * lo, 7.5f));   // halves cannot overflow
        uint16_t m_bits = float_to_bf16_bits(lo);   // exact
        if (isnan(odd))
            s_bits = m_bits = 0x7FC0u;
        if (ok) {
            uint32_t* dst = reinterpret_cast<uint32_t*>((y ? v_cache : k_cache) + at * (D / 2));
            const uint2 c = isnan(odd) ? make_uint2(0, 0) : encode_row16(x, finite, lo, bf16_bits_to_float(s_bits));
            dst[lane] = c.x;
            dst[L + lane] = c.y;
            if (lane == 0)
                (y ? v_scale : k_scale)[at] = s_bits | (static_cast<uint32_t>(m_bits) << 16);
        }
    }
}

// x = bf16(c s + m); rows whose slot is out of range are zero. Bound by memory: the same
// 32768 tokens 30.2 us, 5.7 TB/s, 83 % of a copy's rate (37.6 us with 16 values in a row
// to a lane, whose stores cover half sectors).
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
    uint32_t raw[2][2] = {{0, 0}, {0, 0}}, pair[2] = {0, 0};
    if (r.slot >= 0 && r.slot < a.num_slots) {
        const int64_t at = cache_row(a.page_shift, a.Hkv, r.slot, r.h);
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            const uint32_t* src = reinterpret_cast<const uint32_t*>((y ? v_cache : k_cache) + at * (D / 2));
            raw[y][0] = __ldg(src + lane);
            raw[y][1] = __ldg(src + L + lane);
            pair[y] = __ldg((y ? v_scale : k_scale) + at);
        }
    }
#pragma unroll
    for (int y = 0; y < 2; ++y) {
        const float s = __uint_as_float(pair[y] << 16), m = __uint_as_float(pair[y] & 0xFFFF0000u);
        uint16_t* dst = (y ? v + r.t * a.v_stride : k + r.t * a.k_stride) + static_cast<int64_t>(r.h) * D;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t w = raw[y][i];
            uint32_t o[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                // 2^23 + c has c in its lowest bits
                const F2 c = add2(F2(__uint_as_float(0x4B000000u | ((w >> (8 * j)) & 15u)),
                                     __uint_as_float(0x4B000000u | ((w >> (8 * j + 4)) & 15u))),
                                  F2(-8388608.0f, -8388608.0f));
                const F2 v = fma2(c, F2(s, s), F2(m, m));
                o[j] = pack_bf16(v.lo(), v.hi());
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
