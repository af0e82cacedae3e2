// Per-head norms and the rotation of queries and keys by their positions, with
// the result as bf16 or, keys and values, straight into the FP8 cache.
//
// "ROCm: enable trillion-parameter MoE models with INT4-FP8 single node",
// config.json (rotary attention; kv_cache_scheme FP8): what a layer does between
// its QKV projection and the KV8 cache.
//
//   y = x * rsqrt(mean(x^2) + eps) * w           (where a norm is asked for)
//   (a, b) -> magnitude * (a cos t - b sin t, b cos t + a sin t),  t = position * f_i
// for the pairs (i, i + rot / 2) or (2i, 2i + 1) of the first rot values of a head.
#include "internal.h"
#include "rope.cuh"

namespace w4a8 {

namespace {

constexpr int kThreads = 128;

__device__ __forceinline__ uint4 pack8(const float* x)
{
    uint32_t u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        u[j] = static_cast<uint32_t>(float_to_bf16_bits(x[2 * j])) |
               (static_cast<uint32_t>(float_to_bf16_bits(x[2 * j + 1])) << 16);
    return make_uint4(u[0], u[1], u[2], u[3]);
}

template <int L>
__device__ __forceinline__ float row_sum(float x)
{
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1)
        x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
    return x;
}
template <int L>
__device__ __forceinline__ float row_max(float x)
{
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1)
        x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, o));
    return x;
}

}  // namespace

// L lanes share a row (one head of one token), 16 values each, in two runs of 8:
// a rotating lane has both halves of 8 pairs, so nothing is exchanged but the sum
// of squares (and the largest value of a row that finds its own scale), every
// load and store is 16 bytes, and a row may be written over itself.
//
// The angle. A table holds f_i / 2 pi as 64-bit fractions of a turn; times the
// position, modulo 2^64, is the exact fraction of the turn that the position comes
// to, whatever its size, where an fp32 angle would be off by 2^-24 of all its
// turns (a tenth of a radian at a position of a million). Its upper 32 bits go
// through sincospif. That is some 40 instructions a pair, the largest part of a
// row's arithmetic, so a group of lanes keeps its 8 sines and cosines for several
// heads of its token.
template <int L, bool INTER, bool CACHE>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ Rope a)
{
    grid_dep_wait();
    const int lane = threadIdx.x % L;
    const int t = blockIdx.x * (kThreads / L) + threadIdx.x / L;
    const int n_q = a.Hq, n_k = a.Hq + a.Hkv, n = CACHE ? n_k + a.Hkv : n_k;
    const int r0 = blockIdx.y * a.slice, r1 = min(r0 + a.slice, n);
    const bool live = t < a.T && lane * 16 < a.D;
    const bool turning = live && lane * 16 < a.rot;
    // the lane's two runs of 8 values
    const int at0 = !INTER && turning ? lane * 8 : lane * 16;
    const int at1 = !INTER && turning ? lane * 8 + a.rot / 2 : lane * 16 + 8;

    auto load = [&](int r, uint4(&raw)[2]) {
        raw[0] = raw[1] = make_uint4(0, 0, 0, 0);
        if (live && r < r1) {
            const uint16_t* src = r < n_q   ? a.q + t * a.q_stride + static_cast<int64_t>(r) * a.D
                                  : r < n_k ? a.k + t * a.k_stride + static_cast<int64_t>(r - n_q) * a.D
                                            : a.v + t * a.v_stride + static_cast<int64_t>(r - n_k) * a.D;
            raw[0] = *reinterpret_cast<const uint4*>(src + at0);
            raw[1] = *reinterpret_cast<const uint4*>(src + at1);
        }
    };
    uint4 next[2];
    load(r0, next);

    int64_t slot = -1;
    if (CACHE && t < a.T)
        slot = __ldg(a.slots + t);
    float cs[8], sn[8];
    if (r0 < n_k && turning) {
        const int64_t pos = __ldg(a.positions + t);
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            const ulonglong2 f = __ldg(reinterpret_cast<const ulonglong2*>(a.turns + lane * 8 + j));
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const uint64_t turn = static_cast<uint64_t>(pos) * (e ? f.y : f.x);
                sincospif(static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f, &sn[j + e], &cs[j + e]);
                sn[j + e] *= a.magnitude;
                cs[j + e] *= a.magnitude;
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            cs[j] = 1.0f, sn[j] = 0.0f;
    }

    const uint16_t* weight_of = nullptr;
    float w[16];
    for (int r = r0; r < r1; ++r) {
        float x[16];
        unpack16(next, x);
        load(r + 1, next);
        const uint16_t* weight = r < n_q ? a.q_weight : r < n_k ? a.k_weight : nullptr;
        if (weight) {
            if (weight != weight_of) {
                weight_of = weight;
                uint4 raw[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
                if (live) {
                    raw[0] = __ldg(reinterpret_cast<const uint4*>(weight + at0));
                    raw[1] = __ldg(reinterpret_cast<const uint4*>(weight + at1));
                }
                unpack16(raw, w);
            }
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < 16; ++i)
                sum = fmaf(x[i], x[i], sum);
            sum = row_sum<L>(sum);
            const float f = rsqrtf(sum / static_cast<float>(a.D) + a.eps);
#pragma unroll
            for (int i = 0; i < 16; ++i)
                x[i] = x[i] * f * w[i];
        }
        if (turning && r < n_k) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int i0 = INTER ? 2 * j : j, i1 = INTER ? 2 * j + 1 : j + 8;
                const float lo = x[i0], hi = x[i1];
                x[i0] = fmaf(lo, cs[j], -hi * sn[j]);
                x[i1] = fmaf(hi, cs[j], lo * sn[j]);
            }
        }
        if (!CACHE || r < n_q) {
            if (live) {
                uint16_t* dst = r < n_q ? a.q_out + t * a.q_out_stride + static_cast<int64_t>(r) * a.D
                                        : a.k_out + t * a.k_out_stride + static_cast<int64_t>(r - n_q) * a.D;
                *reinterpret_cast<uint4*>(dst + at0) = pack8(x);
                *reinterpret_cast<uint4*>(dst + at1) = pack8(x + 8);
            }
            continue;
        }
        // ---- into the cache, as kv8_write does with bf16 rows
        const bool is_k = r < n_k;
        const int h = is_k ? r - n_q : r - n_k;
        const bool ok = live && slot >= 0 && slot < a.num_slots;
        const int64_t row = ok ? cache_row(a.page_shift, a.Hkv, slot, h) : 0;
        float* scale = is_k ? a.k_scale : a.v_scale;
        float top = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i)
            top = fmaxf(top, fabsf(x[i]));   // (passes over NaN)
        float s;
        if (a.per_token) {
            top = row_max<L>(top);
            float finite = top;
            if (__any_sync(0xFFFFFFFFu, top > 3.4028235e38f)) {
                finite = 0.0f;
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    finite = fmaxf(finite, fabsf(x[i]) <= 3.4028235e38f ? fabsf(x[i]) : 0.0f);
                finite = row_max<L>(finite);
            }
            s = fmaxf(__fdiv_rn(finite, 448.0f), a.min_scale);
            s = s == 0.0f ? 1.0f : s;
        } else {
            s = __ldg(scale + h);
        }
        if (ok) {
            uint2 c[2];
            encode16(x, top, s, c);
            uint8_t* dst = (is_k ? a.k_cache : a.v_cache) + row * a.D;
            *reinterpret_cast<uint2*>(dst + at0) = c[0];
            *reinterpret_cast<uint2*>(dst + at1) = c[1];
            if (a.per_token && lane == 0)
                scale[row] = s;
        }
    }
}

template <int L, bool CACHE>
static cudaError_t launch(const Rope& a, cudaStream_t s)
{
    const int rows = a.Hq + (CACHE ? 2 : 1) * a.Hkv, tokens = kThreads / L;
    const dim3 grid((a.T + tokens - 1) / tokens, (rows + a.slice - 1) / a.slice);
    return launch_dependent(a.interleaved ? rope_kernel<L, true, CACHE> : rope_kernel<L, false, CACHE>, grid,
                            dim3(kThreads), 0, s, a);
}

cudaError_t launch_rope(Rope a, bool to_cache, int num_sms, cudaStream_t s)
{
    const int L = a.D <= 64 ? 4 : a.D <= 128 ? 8 : 16;
    const int64_t rows = a.Hq + (to_cache ? 2 : 1) * a.Hkv;
    // rows that a group of lanes takes: one until the GPU is full of groups, then up to 8
    const int64_t lanes = rows * a.T * L;
    a.slice = static_cast<int>(min(max(lanes / (static_cast<int64_t>(num_sms) * 1024), int64_t{1}), int64_t{8}));
    a.slice = static_cast<int>(rows / max(rows / a.slice, int64_t{1}));
    if ((rows + a.slice - 1) / a.slice > 65535)
        a.slice = static_cast<int>((rows + 65534) / 65535);
    if (to_cache)
        return L == 4 ? launch<4, true>(a, s) : launch<8, true>(a, s);
    return L == 4 ? launch<4, false>(a, s) : L == 8 ? launch<8, false>(a, s) : launch<16, false>(a, s);
}

}  // namespace w4a8
