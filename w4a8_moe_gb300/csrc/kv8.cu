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

constexpr int kRowThreads = 128;   // (writing 32768 tokens, us: 64 34.0, 128 32.0, 256 32.6)
constexpr float kInv448Hi = static_cast<float>(1.0 / 448.0);
constexpr float kInv448Lo = static_cast<float>(1.0 / 448.0 - static_cast<double>(kInv448Hi));

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

// E4M3(x / s) of 16 values, the quotient rounded to fp32 first. A division of
// every value would be most of the call's arithmetic; here it is q = x r with
// r = 1 / s correctly rounded, then q + (q s - x) (-r) by two fused multiply-adds,
// which is the correctly rounded quotient where nothing under- or overflows
// (P. Markstein, "Computation of elementary functions on the IBM RISC System/6000
// processor", 1990). With 2^-60 <= s < 2^60 and finite values below 2^60 s that
// holds for every quotient above 2^-11, and smaller ones have the code 0 either
// way; other rows divide. The residual is taken with that sign so that a zero
// keeps its own: q s - x is +0 for x = -0, and +0 (-r) + (-0) is -0.
__device__ __forceinline__ void encode16(const uint4 (&raw)[2], float top, float s, uint2 (&c)[2])
{
    const float r = __frcp_rn(s);
    const bool plain = s >= 8.6736174e-19f && s < 1.1529215e18f && top < s * 1.1529215e18f;
    const F2 r2(-r, -r), s2(s, s);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t u[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
        uint32_t e[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float lo = __uint_as_float(u[j] << 16), hi = __uint_as_float(u[j] & 0xFFFF0000u);
            if (plain) {
                const F2 x(-lo, -hi), q = mul2(x, r2);
                const F2 t = fma2(fma2(q, s2, x), r2, q);
                e[j] = cvt_e4m3x2(t.hi(), t.lo());
            } else {
                e[j] = cvt_e4m3x2(__fdiv_rn(hi, s), __fdiv_rn(lo, s));
            }
        }
        c[i] = make_uint2(e[0] | (e[1] << 16), e[2] | (e[3] << 16));
    }
}

// The largest magnitude of 16 bf16 values, as bits: not finite from 0x7F80 on.
__device__ __forceinline__ uint32_t top16(const uint4 (&raw)[2])
{
    constexpr uint32_t m = 0x7FFF7FFFu;
    const uint32_t a = __vmaxu2(__vmaxu2(raw[0].x & m, raw[0].y & m), __vmaxu2(raw[0].z & m, raw[0].w & m));
    const uint32_t b = __vmaxu2(__vmaxu2(raw[1].x & m, raw[1].y & m), __vmaxu2(raw[1].z & m, raw[1].w & m));
    const uint32_t t = __vmaxu2(a, b);
    return max(t >> 16, t & 0xFFFFu);
}
// The same over the finite ones.
__device__ __forceinline__ uint32_t top16_finite(const uint4 (&raw)[2])
{
    uint32_t top = 0;
    for (int i = 0; i < 2; ++i) {
        const uint32_t u[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
        for (int j = 0; j < 8; ++j) {
            const uint32_t m = (u[j >> 1] >> (j & 1 ? 16 : 0)) & 0x7FFFu;
            top = m < 0x7F80u ? max(top, m) : top;
        }
    }
    return top;
}
// Over the lanes of a row.
template <int L>
__device__ __forceinline__ uint32_t row_top(uint32_t top)
{
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1)
        top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    return top;
}

}  // namespace

// Bound by memory: 32768 tokens of 8 heads of 128 with per-token scales (203.6
// MB) take 32.0 us, 6.4 TB/s or 94 % of a copy's rate, three sets of tensors in
// turn (with the loads behind the slot's 35.0; with streaming loads, `.cs`, 33.0);
// 32 tokens take 2.1 us, a launch and two dependent loads.
//
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
    const int64_t at = ok ? cache_row(a, r.slot, r.h) : 0;
#pragma unroll
    for (int y = 0; y < 2; ++y) {
        float* scale = y ? v_scale : k_scale;
        uint32_t top = top16(raw[y]);
        float s;
        if (a.per_token) {
            top = row_top<L>(top);
            uint32_t finite = top;
            if (__any_sync(0xFFFFFFFFu, top >= 0x7F80u))
                finite = row_top<L>(top16_finite(raw[y]));
            // s = the row's largest / 448: its product with 1 / 448 kept in two
            // parts rounds like the quotient (compared for every bf16 value)
            const float amax = __uint_as_float(finite << 16);
            s = fmaf(amax, kInv448Hi, amax * kInv448Lo);
            if (finite < 0x1800u)   // below 2^-79 the second part may be no normal number
                s = __fdiv_rn(amax, 448.0f);
            s = fmaxf(s, a.min_scale);
            s = s == 0.0f ? 1.0f : s;
        } else {
            s = r.live ? __ldg(scale + r.h) : 1.0f;
        }
        if (ok) {
            uint2 c[2];
            encode16(raw[y], __uint_as_float(top << 16), s, c);
            uint2* dst = reinterpret_cast<uint2*>((y ? v_cache : k_cache) + at * D);
            dst[lane] = c[0];
            dst[L + lane] = c[1];
            if (a.per_token && lane == 0)
                scale[at] = s;
        }
    }
}

// x = bf16(dec(code) * s); rows whose slot is out of range are zero. The same
// 32768 tokens: 31.8 us, 6.4 TB/s, 95 % of a copy's rate.
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
    grid_dep_wait();
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
    return launch_dependent(a.D == 128 ? kv8_write_kernel<128> : kv8_write_kernel<64>, dim3(row_blocks(a)),
                            dim3(kRowThreads), 0, s, a, k, v, slots, k_cache, v_cache, k_scale, v_scale);
}

cudaError_t launch_kv8_read(const Kv8Rows& a, const uint8_t* k_cache, const uint8_t* v_cache, const float* k_scale,
                            const float* v_scale, const int32_t* slots, uint16_t* k, uint16_t* v, cudaStream_t s)
{
    return launch_dependent(a.D == 128 ? kv8_read_kernel<128> : kv8_read_kernel<64>, dim3(row_blocks(a)),
                            dim3(kRowThreads), 0, s, a, k_cache, v_cache, k_scale, v_scale, slots, k, v);
}

}  // namespace w4a8
