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
constexpr int kMostTokens = 4;   // of a block

__device__ __forceinline__ uint4 pack8(const float* x)
{
    return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}

// Cosine and sine of turn / 2^64 turns. The nearest quarter is taken off in whole
// numbers and the rest (an eighth at most) converted once, so that however near an
// angle is to a quarter's end its sine there keeps all of a float's digits. (The upper
// 32 bits alone are off by 2^-32 of a turn, which is 0.4 % of the first position's sine
// of a pair that turns by 210 of them.)
__device__ __forceinline__ float2 cos_sin(uint64_t turn)
{
    const uint32_t quarter = static_cast<uint32_t>((turn + (uint64_t{1} << 61)) >> 62);
    float s, c;
    sincospif(__ll2float_rn(static_cast<int64_t>(turn - (static_cast<uint64_t>(quarter) << 62))) * 0x1p-63f, &s, &c);
    const float x = quarter & 1 ? -s : c, y = quarter & 1 ? c : s;
    return quarter & 2 ? make_float2(-x, -y) : make_float2(x, y);
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

// Bound by memory: 32768 tokens of 32 + 8 heads of 128 with norms (671 MB) take 103
// us, 6.5 TB/s or 96 % of a copy's rate, 8192 of them 30.3 us, 82 % (a launch and the
// first rows' way are 4 us of it); 32768 tokens of 48 query and 8 kv heads into the
// cache (1009 MB) 164 us, 91 %. 32 tokens take 2.1 us, into the cache 2.6.
//
// L lanes share a row (one head of one token), 16 values each, in two runs of 8:
// a rotating lane has both halves of 8 pairs, so nothing is exchanged but the sum
// of squares (and the largest value of a row that finds its own scale), every
// load and store is 16 bytes, and a row may be written over itself.
//
// The angle. A table holds f_i / 2 pi as 64-bit fractions of a turn; times the
// position, modulo 2^64, is the exact fraction of the turn that the position comes
// to, whatever its size, where an fp32 angle would be off by 2^-24 of all its
// turns (a tenth of a radian at a position of a million). The nearest quarter is taken
// off it, the rest goes through sincospif. That is dozens of instructions a pair, a third of a row's
// arithmetic, so a block makes the sines and cosines of its tokens once, in shared
// memory, while its first rows are on their way (made by each group of lanes for its
// own heads: 37.5 us for the 8192 tokens). Shared memory holds what a lane reads in one
// instruction as the lanes lie, so that none of its reads conflict (43.4 us with norms
// and interleaved pairs before). One block a range of tokens for as long as the kernel
// runs, without new blocks, was slower: 188 us into the cache.
template <int L, bool INTER, bool CACHE>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ Rope a)
{
    constexpr int G = kThreads / L;   // rows at once
    extern __shared__ __align__(16) float table[];   // [tokens][2][rot / 2] cosines, sines, in fours of the lanes
    __shared__ uint4 weights[2][2][L];               // of the norms: queries' and keys', a lane's two runs
    __shared__ int64_t slot_of[kMostTokens];
    grid_dep_wait();
    const int lane = threadIdx.x % L, group = threadIdx.x / L;
    const int t0 = blockIdx.x * a.tokens, tokens = min(a.tokens, a.T - t0);
    const int n_q = a.Hq, n_k = a.Hq + a.Hkv, n = CACHE ? n_k + a.Hkv : n_k;
    const int first = blockIdx.y * a.slice, rows = min(a.slice, n - first);   // of each token
    const bool mine = lane * 16 < a.D, turning = lane * 16 < a.rot;
    // the lane's two runs of 8 values
    const int at0 = !INTER && turning ? lane * 8 : lane * 16;
    const int at1 = !INTER && turning ? lane * 8 + a.rot / 2 : lane * 16 + 8;

    // the group's next row: token (of the block's; from `tokens` on there is none) and r
    int next_token = 0, next_r = group;
    uint4 next[2];
    auto fetch = [&]() {
        while (next_r >= rows) {
            next_r -= rows;
            ++next_token;
        }
        next[0] = next[1] = make_uint4(0, 0, 0, 0);
        if (mine && next_token < tokens) {
            const int r = first + next_r;
            const int64_t t = t0 + next_token;
            const uint16_t* src = r < n_q   ? a.q + t * a.q_stride + static_cast<int64_t>(r) * a.D
                                  : r < n_k ? a.k + t * a.k_stride + static_cast<int64_t>(r - n_q) * a.D
                                            : a.v + t * a.v_stride + static_cast<int64_t>(r - n_k) * a.D;
            next[0] = *reinterpret_cast<const uint4*>(src + at0);
            next[1] = *reinterpret_cast<const uint4*>(src + at1);
        }
    };
    fetch();

    const int half = a.rot / 2;
    for (int i = threadIdx.x; i < tokens * half; i += kThreads) {
        const int token = i / half, j = i - token * half;
        const int64_t pos = __ldg(a.positions + t0 + token);
        const uint64_t turn = static_cast<uint64_t>(pos) * __ldg(a.turns + j);
        const float2 cs = cos_sin(turn);
        float* to = table + token * a.rot + (j / 4 % 2) * (half / 2) + j / 8 * 4 + j % 4;
        to[0] = cs.x * a.magnitude;
        to[half] = cs.y * a.magnitude;
    }
    const bool norms = a.q_weight || a.k_weight;
    if (threadIdx.x < 2 * L) {   // the lanes of the first groups load their runs of the queries' and the keys' weights
        const uint16_t* weight = threadIdx.x < L ? a.q_weight : a.k_weight;
        if (weight && mine) {
            weights[threadIdx.x / L][0][lane] = __ldg(reinterpret_cast<const uint4*>(weight + at0));
            weights[threadIdx.x / L][1][lane] = __ldg(reinterpret_cast<const uint4*>(weight + at1));
        }
    }
    if (CACHE && threadIdx.x < tokens)
        slot_of[threadIdx.x] = __ldg(a.slots + t0 + threadIdx.x);
    __syncthreads();

    for (int left = tokens * rows; left > 0; left -= G) {
        float x[16];
        unpack16(next, x);
        const int token = next_token, r = first + next_r;
        const bool there = token < tokens, live = mine && there;
        next_r += G;
        fetch();
        if (norms) {
            F2 sum2(0.0f, 0.0f);
#pragma unroll
            for (int j = 0; j < 16; j += 2)
                sum2 = fma2(F2(x[j], x[j + 1]), F2(x[j], x[j + 1]), sum2);
            const float sum = row_sum<L>(sum2.lo() + sum2.hi());
            if (live && (r < n_q ? a.q_weight : r < n_k ? a.k_weight : nullptr)) {
                const float mean = fmaf(sum, a.inv_d, a.eps);
                float f = rsqrtf(mean);   // two units off at most: a Newton step takes it to half of one
                if (mean >= 0x1p-100f && mean < 0x1p120f)
                    f = fmaf(0.5f * f, fmaf(-mean * f, f, 1.0f), f);
                const uint4 raw[2] = {weights[r < n_q ? 0 : 1][0][lane], weights[r < n_q ? 0 : 1][1][lane]};
                float w[16];
                unpack16(raw, w);
#pragma unroll
                for (int j = 0; j < 16; j += 2) {
                    const F2 y = mul2(mul2(F2(x[j], x[j + 1]), F2(f, f)), F2(w[j], w[j + 1]));
                    x[j] = y.lo(), x[j + 1] = y.hi();
                }
            }
        }
        if (turning && r < n_k && there) {
            const float* cosines = table + token * a.rot + lane * 4;
#pragma unroll
            for (int j = 0; j < 8; j += 4) {   // four pairs
                const float4 c4 = *reinterpret_cast<const float4*>(cosines + j / 4 * (half / 2));
                const float4 s4 = *reinterpret_cast<const float4*>(cosines + j / 4 * (half / 2) + half);
                const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
                if (INTER) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float lo = x[2 * (j + i)], hi = x[2 * (j + i) + 1];
                        x[2 * (j + i)] = fmaf(lo, c[i], -hi * s[i]);
                        x[2 * (j + i) + 1] = fmaf(hi, c[i], lo * s[i]);
                    }
                } else {   // (the pairs' first values are neighbours, and their second ones)
#pragma unroll
                    for (int i = j; i < j + 4; i += 2) {
                        const F2 lo(x[i], x[i + 1]), hi(x[8 + i], x[9 + i]);
                        const F2 cc(c[i - j], c[i - j + 1]), ss(s[i - j], s[i - j + 1]);
                        const F2 y0 = fma2(hi, mul2(ss, F2(-1.0f, -1.0f)), mul2(lo, cc)), y1 = fma2(lo, ss, mul2(hi, cc));
                        x[i] = y0.lo(), x[i + 1] = y0.hi(), x[8 + i] = y1.lo(), x[9 + i] = y1.hi();
                    }
                }
            }
        }
        if (live && (!CACHE || r < n_q)) {
            const int64_t t = t0 + token;
            uint16_t* dst = r < n_q ? a.q_out + t * a.q_out_stride + static_cast<int64_t>(r) * a.D
                                    : a.k_out + t * a.k_out_stride + static_cast<int64_t>(r - n_q) * a.D;
            *reinterpret_cast<uint4*>(dst + at0) = pack8(x);
            *reinterpret_cast<uint4*>(dst + at1) = pack8(x + 8);
        }
        if (!CACHE || !__any_sync(0xFFFFFFFFu, r >= n_q))
            continue;
        // ---- into the cache, as kv8_write does with bf16 rows
        float top = 0.0f;
#pragma unroll
        for (int j = 0; j < 16; ++j)
            top = fmaxf(top, fabsf(x[j]));   // (passes over NaN)
        float finite = 0.0f;
        if (a.per_token) {
            top = row_max<L>(top);
            finite = top;
            if (__any_sync(0xFFFFFFFFu, top > 3.4028235e38f)) {
                finite = 0.0f;
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    finite = fmaxf(finite, fabsf(x[j]) <= 3.4028235e38f ? fabsf(x[j]) : 0.0f);
                finite = row_max<L>(finite);
            }
        }
        const int64_t slot = live ? slot_of[token] : -1;
        if (r >= n_q && slot >= 0 && slot < a.num_slots) {
            const bool is_k = r < n_k;
            const int h = is_k ? r - n_q : r - n_k;
            const int64_t at = cache_row(a.page_shift, a.Hkv, slot, h);
            float* scale = is_k ? a.k_scale : a.v_scale;
            float s;
            if (a.per_token) {
                s = fmaxf(__fdiv_rn(finite, 448.0f), a.min_scale);
                s = s == 0.0f ? 1.0f : s;
                if (lane == 0)
                    scale[at] = s;
            } else {
                s = __ldg(scale + h);
            }
            const Encoder encode(top, s);
            uint32_t c[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                c[j] = encode.two(x[4 * j], x[4 * j + 1]) | (encode.two(x[4 * j + 2], x[4 * j + 3]) << 16);
            uint8_t* dst = (is_k ? a.k_cache : a.v_cache) + at * a.D;
            *reinterpret_cast<uint2*>(dst + at0) = make_uint2(c[0], c[1]);
            *reinterpret_cast<uint2*>(dst + at1) = make_uint2(c[2], c[3]);
        }
    }
}

template <int L, bool CACHE>
static cudaError_t launch(Rope a, int num_sms, cudaStream_t s)
{
    constexpr int G = kThreads / L;
    a.inv_d = 1.0f / static_cast<float>(a.D);
    const int rows = a.Hq + (CACHE ? 2 : 1) * a.Hkv;
    // A block for one token, or for several where they are many (angles are made once
    // a block and 16 blocks an SM keep it busy); few tokens are spread over the SMs by
    // their rows.
    const int64_t passes = static_cast<int64_t>(a.T) * ((rows + G - 1) / G), each = static_cast<int64_t>(num_sms) * 16;
    a.tokens = static_cast<int>(min(max(passes / each, int64_t{1}), int64_t{kMostTokens}));
    a.slice = passes < each ? G : rows;
    const dim3 grid((a.T - 1) / a.tokens + 1, (rows + a.slice - 1) / a.slice);
    return launch_dependent(a.interleaved ? rope_kernel<L, true, CACHE> : rope_kernel<L, false, CACHE>, grid,
                            dim3(kThreads), a.tokens * a.rot * static_cast<int>(sizeof(float)), s, a);
}

cudaError_t launch_rope(const Rope& a, bool to_cache, int num_sms, cudaStream_t s)
{
    if (to_cache)
        return a.D <= 64 ? launch<4, true>(a, num_sms, s) : launch<8, true>(a, num_sms, s);
    return a.D <= 64    ? launch<4, false>(a, num_sms, s)
           : a.D <= 128 ? launch<8, false>(a, num_sms, s)
                        : launch<16, false>(a, num_sms, s);
}

}  // namespace w4a8
