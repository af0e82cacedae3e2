// Decode attention over the FP8 key/value cache: the sequences' own tokens,
// short shared prefixes, and the join of all partial results.
//
// "ROCm: enable trillion-parameter MoE models with INT4-FP8 single node",
// config.json (kv_cache_scheme FP8; 48 query and 8 key/value heads): the
// attention that reads the KV8 cache of a W4A8KV8 checkpoint.
//
// One query token per sequence. Query head h uses kv head h / group; its keys
// are the prefix's, which all sequences share, and then its sequence's own:
//   s_j = sm_scale * q . k_j       (cap > 0: cap * tanh(s_j / cap))
//   out = sum_j e^{s_j} v_j / sum_j e^{s_j},   lse = log sum_j e^{s_j}
// The sum is cut into pieces; a piece keeps, for each of its rows, a reference
// exponent m (log2), l = sum 2^{x_j - m} and o = sum 2^{x_j - m} v_j, with
// x = s * log2(e), and kv8_join_kernel adds pieces up under their largest m.
#include <math.h>

#include "internal.h"
#include "kv8.cuh"
#include "ptx.cuh"

namespace w4a8 {

namespace {

constexpr int kWarps = 4;
constexpr float kLog2e = 1.4426950408889634f;
// The reference exponent of a row is raised only when a score passes it by
// this much: 2^{x - m} then stays below 2^8, far inside f16, and the row's
// accumulators are hardly ever rescaled. With per-token scales the f16 operand
// is 2^{x - m} * vs, so what is compared is x + log2(the largest vs at hand):
// m then carries the values' size too, and drops out of o / l.
constexpr float kSlack = 8.0f;

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
// D[16x8] += A[16x16] B[16x8], f16 operands, fp32 accumulators.
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Codes are read once: keep them out of L1.
__device__ __forceinline__ uint4 ld_codes16(const uint8_t* p)
{
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}
__device__ __forceinline__ uint2 ld_codes8(const uint8_t* p)
{
    uint2 v;
    asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
    return v;
}

// ---------------------------------------------------------------------------
// The split. A pair is (rows, keys): first the prefix's pairs (kv head, row
// tile of the whole batch), then the sequences' (sequence, kv head, row tile of
// the group). The keys of a pair are cut into units of 16, all units stand in
// one line in pair order, and CTA c of n takes units [U c / n, U (c + 1) / n):
// equal work however ragged the lengths are. The piece of pair p done by CTA c
// is stored in slot p + c: along the line p + c rises with every piece, so no
// two share a slot, and a reader finds a pair's slots from U and n alone.
// ---------------------------------------------------------------------------
struct Line {
    int64_t U;      // units
    int n;          // CTAs with units
    int up;         // units of a prefix pair
    int pairs_p;    // prefix pairs
    int64_t own;    // first unit of the sequences' pairs
    int hr;         // pairs of a sequence
};
__device__ __forceinline__ int seq_len(const Kv8Attn& a, int b)
{
    return a.max_pages ? min(max(__ldg(a.lens + b), 0), a.max_pages << a.page_shift) : 0;
}
__device__ __forceinline__ int seq_units(const Kv8Attn& a, int b)
{
    return (seq_len(a, b) + kKv8Unit - 1) / kKv8Unit;
}
__device__ __forceinline__ Line make_line(const Kv8Attn& a, int64_t seq_total)
{
    Line l;
    l.hr = a.Hkv * a.tiles;
    l.pairs_p = a.Hkv * a.ptiles;
    l.up = (a.prefix_len + kKv8Unit - 1) / kKv8Unit;
    l.own = static_cast<int64_t>(l.pairs_p) * l.up;
    l.U = l.own + seq_total * l.hr;
    const int64_t n = (l.U + kKv8MinUnits - 1) / kKv8MinUnits;
    l.n = static_cast<int>(n < a.ctas ? n : a.ctas);
    return l;
}
__device__ __forceinline__ int64_t cta_begin(const Line& l, int c) { return l.U * c / l.n; }
__device__ __forceinline__ int cta_of(const Line& l, int64_t u) { return static_cast<int>(((u + 1) * l.n - 1) / l.U); }

// One unit's codes as a thread holds them: for S = Q K^T two n-tiles of 8 keys
// (this thread: key g of each, chunk c of its D values); for O^T = V^T P^T
// four keys (2c, 2c+1, 2c+8, 2c+9), chunk g of their D values. Neither needs
// shared memory: which d a fragment register stands for is free as long as q
// and o use the same order, so every thread reads contiguous bytes.
template <int D>
struct Codes {
    uint4 k[2][D / 64];
    uint32_t v[4][D / 32];
    float ks[4], vs[4];   // scales of keys 2c, 2c+1, 2c+8, 2c+9 (per-token scales only)
};

template <int D, bool TOK>
__device__ __forceinline__ void load_unit(Codes<D>& x, const Kv8Attn& a, int h, int page, int key0, int len, int g, int c)
{
    const int off = key0 & ((1 << a.page_shift) - 1);
    const int64_t row = ((static_cast<int64_t>(page) * a.Hkv + h) << a.page_shift) + off;
    const uint8_t* kb = a.k_cache + row * D;
    const uint8_t* vb = a.v_cache + row * D;
    const int live = len - key0;   // keys of this unit that exist (may pass 16)
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int j = 0; j < D / 64; ++j)
            x.k[t][j] = t * 8 + g < live ? ld_codes16(kb + (t * 8 + g) * D + (j * 4 + c) * 16) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int key = c * 2 + (i & 1) + (i >> 1) * 8;
        if (D == 128) {
            const uint4 w = key < live ? ld_codes16(vb + key * D + g * 16) : make_uint4(0, 0, 0, 0);
            x.v[i][0] = w.x, x.v[i][1] = w.y, x.v[i][D / 32 - 2] = w.z, x.v[i][D / 32 - 1] = w.w;
        } else {
            const uint2 w = key < live ? ld_codes8(vb + key * D + g * 8) : make_uint2(0, 0);
            x.v[i][0] = w.x, x.v[i][1] = w.y;
        }
        if (TOK) {
            x.ks[i] = key < live ? __ldg(a.k_scale + row + key) : 0.0f;
            x.vs[i] = key < live ? __ldg(a.v_scale + row + key) : 0.0f;
        }
    }
}

}  // namespace

// Row tile: 8 rows where the group fits, else 16 (two column tiles of O^T).
int kv8_attn_row_tile(int group) { return group <= 8 ? 8 : 16; }

// A CTA walks its units piece by piece. Its four warps take units in turn, each
// with its own running reference and sums, and join them through shared memory
// at the piece's end.
template <int D, int NT, bool TOK>
__global__ void __launch_bounds__(kWarps * 32) kv8_attn_kernel(const __grid_constant__ Kv8Attn a)
{
    constexpr int R = 8 * NT;      // rows of a tile
    constexpr int KS = D / 16;     // k-steps of Q K^T = m-tiles of O^T
    extern __shared__ __align__(16) uint8_t smem[];
    float* so = reinterpret_cast<float*>(smem);                    // [warp][row][D]
    float* sm = so + kWarps * R * D;                               // [warp][row]
    float* sl = sm + kWarps * R;                                   // [warp][row]
    int* cum = reinterpret_cast<int*>(sl + kWarps * R);            // [B + 1]
    __shared__ int warp_sum[kWarps];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;

    // prefix sums of the sequences' units
    int carry = 0;
    for (int b0 = 0; b0 < a.B; b0 += kWarps * 32) {
        const int b = b0 + tid;
        const int n = b < a.B ? seq_units(a, b) : 0;
        if (blockIdx.x == 0 && b < a.B && a.max_pages &&
            static_cast<unsigned>(__ldg(a.lens + b)) > static_cast<unsigned>(a.max_pages << a.page_shift))
            set_error(a.err, kErrBitIndex);
        int s = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int t = __shfl_up_sync(0xFFFFFFFFu, s, o);
            s += lane >= o ? t : 0;
        }
        if (lane == 31)
            warp_sum[warp] = s;
        __syncthreads();
        int base = carry;
        for (int w = 0; w < warp; ++w)
            base += warp_sum[w];
        if (b < a.B)
            cum[b] = base + s - n;
        for (int w = 0; w < kWarps; ++w)
            carry += warp_sum[w];
        __syncthreads();
    }
    if (tid == 0)
        cum[a.B] = carry;
    __syncthreads();

    const Line line = make_line(a, carry);
    const int cta = blockIdx.x;
    if (cta >= line.n)
        return;
    int64_t u = cta_begin(line, cta);
    const int64_t u_end = cta_begin(line, cta + 1);

    while (u < u_end) {
        // ---- the piece at u
        int h, row0, len, b = 0, pair;
        int64_t first, last;   // the pair's units
        const int32_t* pages;
        int n_pages;
        const bool prefix = u < line.own;
        if (prefix) {
            pair = static_cast<int>(u / line.up);
            h = pair / a.ptiles;
            row0 = (pair % a.ptiles) * R;
            len = a.prefix_len;
            first = static_cast<int64_t>(pair) * line.up;
            last = first + line.up;
            pages = a.prefix_pages;
            n_pages = (a.prefix_len + (1 << a.page_shift) - 1) >> a.page_shift;
        } else {
            const int64_t rel = u - line.own;
            int lo = 0, hi = a.B;   // the last b with cum[b] * hr <= rel
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (static_cast<int64_t>(cum[mid]) * line.hr <= rel)
                    lo = mid;
                else
                    hi = mid;
            }
            b = lo;
            const int n = cum[b + 1] - cum[b];
            const int64_t start = static_cast<int64_t>(cum[b]) * line.hr;
            const int j = static_cast<int>((rel - start) / n);
            h = j / a.tiles;
            row0 = (j % a.tiles) * R;
            len = seq_len(a, b);
            first = line.own + start + static_cast<int64_t>(j) * n;
            last = first + n;
            pages = a.page_table + b * a.table_stride;
            n_pages = a.max_pages;
            pair = line.pairs_p + b * line.hr + j;
        }
        const int64_t stop = last < u_end ? last : u_end;
        const int ua = static_cast<int>(u - first), ub = static_cast<int>(stop - first);
        const int rows = min(R, (prefix ? a.B * a.group : a.group) - row0);

        // ---- queries: f16 fragments of q * 2^-e with e from the row's largest
        // element. bf16 has 8 significant bits and f16 11, so only elements
        // below 2^-16 of the row's largest lose anything, and what they lose is
        // at most 2^-25 of it: the size of one fp32 rounding of the product.
        uint32_t qa[KS][2 * NT];
        float qs[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int r = row0 + t * 8 + g;
            uint4 raw[D / 32];
            if (t * 8 + g < rows) {
                const int qb = prefix ? r / a.group : b;
                const int qh = h * a.group + (prefix ? r % a.group : r);
                const uint16_t* src = a.q + qb * a.q_stride + static_cast<int64_t>(qh) * D;
#pragma unroll
                for (int j = 0; j < D / 64; ++j) {
                    raw[2 * j] = __ldg(reinterpret_cast<const uint4*>(src + (j * 4 + c) * 16));
                    raw[2 * j + 1] = __ldg(reinterpret_cast<const uint4*>(src + (j * 4 + c) * 16) + 1);
                }
            } else {
#pragma unroll
                for (int j = 0; j < D / 32; ++j)
                    raw[j] = make_uint4(0, 0, 0, 0);
            }
            uint32_t top = 0;
#pragma unroll
            for (int j = 0; j < D / 32; ++j) {
                const uint32_t w[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    top = max(top, max((w[i] >> 16) & 0x7FFFu, w[i] & 0x7FFFu));
            }
            top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
            top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
            const int ex = static_cast<int>(top >> 7);
            const int e = top == 0 || ex == 255 ? 0 : max(ex, 1) - 127;
            const float down = ldexpf(1.0f, -e);
            float f = ldexpf(a.sm_scale, e);
            if (!TOK)
                f *= __ldg(a.k_scale + h);
            qs[t] = a.cap > 0.0f ? f / a.cap : f * kLog2e;
#pragma unroll
            for (int j = 0; j < D / 32; ++j) {   // 8 values: two k-steps' two registers each
                const uint32_t w[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    qa[2 * j + (i >> 1)][(i & 1) * NT + t] =
                        pack_f16(__uint_as_float(w[i] << 16) * down, __uint_as_float(w[i] & 0xFFFF0000u) * down);
            }
        }

        float o[KS][NT][4];
#pragma unroll
        for (int j = 0; j < KS; ++j)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    o[j][t][i] = 0.0f;
        float m[NT], l[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t)
            m[t] = -INFINITY, l[t] = 0.0f;

        Codes<D> x;
        auto fetch = [&](int unit) {
            const int key0 = unit * kKv8Unit;
            const int idx = key0 >> a.page_shift;
            int page = idx < n_pages ? __ldg(pages + idx) : -1;
            if (static_cast<unsigned>(page) >= static_cast<unsigned>(a.num_pages)) {
                set_error(a.err, kErrBitIndex);
                page = 0;
            }
            load_unit<D, TOK>(x, a, h, page, key0, len, g, c);
        };
        for (int unit = ua + warp; unit < ub; unit += kWarps) {
            fetch(unit);
            // ---- S = Q K^T
            float s[2][4];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    s[t][i] = 0.0f;
#pragma unroll
                for (int j = 0; j < D / 64; ++j) {
                    const uint32_t w[4] = {x.k[t][j].x, x.k[t][j].y, x.k[t][j].z, x.k[t][j].w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t b0 = e4m3x2_to_f16x2(w[i] & 0xFFFFu), b1 = e4m3x2_to_f16x2(w[i] >> 16);
                        const uint32_t* qf = qa[j * 4 + i];
                        mma_f16(s[t], qf[0], NT == 2 ? qf[1] : 0u, qf[NT], NT == 2 ? qf[2 * NT - 1] : 0u, b0, b1);
                    }
                }
            }
            // ---- scores in log2 units; keys past the end are -inf
            const int live = len - unit * kKv8Unit;
            float lift = 0.0f;   // log2 of the unit's largest value scale
            if (TOK) {
                float top = fmaxf(fmaxf(fabsf(x.vs[0]), fabsf(x.vs[1])), fmaxf(fabsf(x.vs[2]), fabsf(x.vs[3])));
                top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
                lift = fmaxf(log2f(top), -100.0f);
            }
            bool grow = false;
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int i = 0; i < 2 * NT; ++i) {
                    float f = s[t][i] * qs[i >> 1];
                    if (TOK)
                        f *= x.ks[t * 2 + (i & 1)];
                    if (a.cap > 0.0f) {   // tanh y = 1 - 2 / (1 + e^{2y})
                        const float e = ex2(f * (2.0f * kLog2e));
                        f = (a.cap * kLog2e) * (1.0f - __fdividef(2.0f, 1.0f + e));
                        if (e > 1e30f)
                            f = a.cap * kLog2e;
                    }
                    f = t * 8 + c * 2 + (i & 1) < live ? f : -INFINITY;
                    s[t][i] = f;
                    grow = grow || f + lift > m[i >> 1] + kSlack;
                }
            if (__any_sync(0xFFFFFFFFu, grow)) {
                float f[NT];
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    float top = fmaxf(fmaxf(s[0][2 * t], s[0][2 * t + 1]), fmaxf(s[1][2 * t], s[1][2 * t + 1]));
                    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2)) + lift;
                    const float to = fmaxf(m[t], top);
                    f[t] = to == -INFINITY ? 1.0f : ex2(m[t] - to);
                    m[t] = to;
                    l[t] *= f[t];
                }
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const float f0 = __shfl_sync(0xFFFFFFFFu, f[t], c * 8);
                    const float f1 = __shfl_sync(0xFFFFFFFFu, f[t], c * 8 + 4);
#pragma unroll
                    for (int j = 0; j < KS; ++j) {
                        o[j][t][0] *= f0, o[j][t][1] *= f1;
                        o[j][t][2] *= f0, o[j][t][3] *= f1;
                    }
                }
            }
            // ---- P^T and O^T += V^T P^T
            uint32_t pb[NT][2];
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const float ref = m[t] == -INFINITY ? 0.0f : m[t];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float p0 = ex2(s[k][2 * t] - ref), p1 = ex2(s[k][2 * t + 1] - ref);
                    l[t] += p0 + p1;
                    if (TOK) {
                        p0 *= x.vs[2 * k];
                        p1 *= x.vs[2 * k + 1];
                    }
                    pb[t][k] = pack_f16(p0, p1);
                }
            }
#pragma unroll
            for (int w = 0; w < D / 32; ++w)
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const uint32_t sel = half ? 0x7362u : 0x5140u;
                    const uint32_t lo = prmt(x.v[0][w], x.v[1][w], sel), hi = prmt(x.v[2][w], x.v[3][w], sel);
                    const uint32_t a0 = e4m3x2_to_f16x2(lo & 0xFFFFu), a1 = e4m3x2_to_f16x2(lo >> 16);
                    const uint32_t a2 = e4m3x2_to_f16x2(hi & 0xFFFFu), a3 = e4m3x2_to_f16x2(hi >> 16);
#pragma unroll
                    for (int t = 0; t < NT; ++t)
                        mma_f16(o[w * 2 + half][t], a0, a1, a2, a3, pb[t][0], pb[t][1]);
                }
        }

        // ---- the warps' results, joined in a fixed order
        const float vscale = TOK ? 1.0f : __ldg(a.v_scale + h);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            l[t] += __shfl_xor_sync(0xFFFFFFFFu, l[t], 1);
            l[t] += __shfl_xor_sync(0xFFFFFFFFu, l[t], 2);
            if (c == 0) {
                sm[warp * R + t * 8 + g] = m[t];
                sl[warp * R + t * 8 + g] = l[t];
            }
#pragma unroll
            for (int j = 0; j < KS; ++j) {
                float* dst = so + (warp * R + t * 8 + c * 2) * D + g * (D / 8) + 2 * j;
                *reinterpret_cast<float2*>(dst) = make_float2(o[j][t][0] * vscale, o[j][t][2] * vscale);
                *reinterpret_cast<float2*>(dst + D) = make_float2(o[j][t][1] * vscale, o[j][t][3] * vscale);
            }
        }
        __syncthreads();
        const int64_t slot = pair + cta;
        for (int i = tid; i < rows * (D / 4); i += kWarps * 32) {
            const int r = i / (D / 4), d = (i % (D / 4)) * 4;
            float top = sm[r];
#pragma unroll
            for (int w = 1; w < kWarps; ++w)
                top = fmaxf(top, sm[w * R + r]);
            const float ref = top == -INFINITY ? 0.0f : top;
            float4 acc = make_float4(0, 0, 0, 0);
            float sum = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float f = ex2(sm[w * R + r] - ref);
                const float4 v = *reinterpret_cast<const float4*>(so + (w * R + r) * D + d);
                acc.x += v.x * f, acc.y += v.y * f, acc.z += v.z * f, acc.w += v.w * f;
                sum += sl[w * R + r] * f;
            }
            *reinterpret_cast<float4*>(a.part_o + (slot * R + r) * D + d) = acc;
            if (d == 0)
                a.part_ml[slot * R + r] = make_float2(top, sum);
        }
        __syncthreads();
        u = stop;
    }
}

// One CTA per (sequence, query head) adds up the pieces of its row. Warps take
// pieces in turn, a lane D / 32 values, all loads of a warp's pieces in flight
// together; the warps' sums are joined in a fixed order.
constexpr int kJoinWarps = 4;
template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32) kv8_join_kernel(const __grid_constant__ Kv8Attn a,
                                                                   const __grid_constant__ Kv8Prefix p, int R)
{
    constexpr int V = D / 32;
    const int b = blockIdx.x, qh = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int h = qh / a.group, gi = qh % a.group;
    __shared__ int part[2][kJoinWarps];
    __shared__ float so[kJoinWarps][D];
    __shared__ float2 sml[kJoinWarps];
    int before = 0, all = 0;
    for (int i = tid; i < a.B; i += kJoinWarps * 32) {
        const int n = seq_units(a, i);
        all += n;
        before += i < b ? n : 0;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        before += __shfl_xor_sync(0xFFFFFFFFu, before, o);
        all += __shfl_xor_sync(0xFFFFFFFFu, all, o);
    }
    if (lane == 0)
        part[0][warp] = before, part[1][warp] = all;
    __syncthreads();
    before = all = 0;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w)
        before += part[0][w], all += part[1][w];
    const Line line = make_line(a, all);

    // the row's pieces: [0, n0) of the tiled prefix, [n0, n1) of the untiled one, [n1, n2) of its own keys
    const int row = b * a.group + gi;
    const int n0 = p.splits;
    int n1 = n0, n2, c_pre = 0, c_own = 0, pair_pre = 0, pair_own = 0;
    if (a.ptiles) {
        pair_pre = h * a.ptiles + row / R;
        const int64_t first = static_cast<int64_t>(pair_pre) * line.up;
        c_pre = cta_of(line, first);
        n1 += cta_of(line, first + line.up - 1) - c_pre + 1;
    }
    n2 = n1;
    const int units = seq_units(a, b);
    if (units) {
        const int j = h * a.tiles + gi / R;
        pair_own = line.pairs_p + b * line.hr + j;
        const int64_t first = line.own + static_cast<int64_t>(before) * line.hr + static_cast<int64_t>(j) * units;
        c_own = cta_of(line, first);
        n2 += cta_of(line, first + units - 1) - c_own + 1;
    }
    float top = -INFINITY, sum = 0.0f, acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i)
        acc[i] = 0.0f;
#pragma unroll 4
    for (int k = warp; k < n2; k += kJoinWarps) {
        const float* o;
        const float2* mlp;
        if (k < n0) {
            const int64_t at = (static_cast<int64_t>(k) * a.Hkv + h) * a.B * a.group + row;
            o = p.part_o + at * D;
            mlp = p.part_ml + at;
        } else {
            const int64_t at = k < n1 ? static_cast<int64_t>(pair_pre + c_pre + k - n0) * R + row % R
                                      : static_cast<int64_t>(pair_own + c_own + k - n1) * R + gi % R;
            o = a.part_o + at * D;
            mlp = a.part_ml + at;
        }
        const float2 ml = *mlp;
        float v[V];
        if (V == 4) {
            const float4 w = *(reinterpret_cast<const float4*>(o) + lane);
            v[0] = w.x, v[1] = w.y, v[V - 2] = w.z, v[V - 1] = w.w;
        } else {
            const float2 w = *(reinterpret_cast<const float2*>(o) + lane);
            v[0] = w.x, v[1] = w.y;
        }
        const float to = fmaxf(top, ml.x);
        const float ref = to == -INFINITY ? 0.0f : to;
        const float f0 = ex2(top - ref), f1 = ex2(ml.x - ref);
#pragma unroll
        for (int i = 0; i < V; ++i)
            acc[i] = acc[i] * f0 + v[i] * f1;
        sum = sum * f0 + ml.y * f1;
        top = to;
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
        so[warp][lane * V + i] = acc[i];
    if (lane == 0)
        sml[warp] = make_float2(top, sum);
    __syncthreads();
    if (tid >= D / 2)
        return;
    top = sml[0].x;
#pragma unroll
    for (int w = 1; w < kJoinWarps; ++w)
        top = fmaxf(top, sml[w].x);
    const float ref = top == -INFINITY ? 0.0f : top;
    float x = 0.0f, y = 0.0f;
    sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) {
        const float f = ex2(sml[w].x - ref);
        x += so[w][2 * tid] * f;
        y += so[w][2 * tid + 1] * f;
        sum += sml[w].y * f;
    }
    const bool empty = top == -INFINITY && sum == 0.0f;
    const int64_t head = static_cast<int64_t>(b) * a.Hq + qh;
    x = empty ? 0.0f : x / sum;
    y = empty ? 0.0f : y / sum;
    *reinterpret_cast<uint32_t*>(a.out + head * D + 2 * tid) =
        static_cast<uint32_t>(float_to_bf16_bits(x)) | (static_cast<uint32_t>(float_to_bf16_bits(y)) << 16);
    if (a.lse && tid == 0)
        a.lse[head] = empty ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
}

template <int D, int NT, bool TOK>
static cudaError_t launch_pieces(const Kv8Attn& a, cudaStream_t s)
{
    const int smem = (kWarps * 8 * NT * (D + 2) + a.B + 1) * 4;
    auto kern = kv8_attn_kernel<D, NT, TOK>;
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess)
            return e;
    }
    kern<<<a.ctas, kWarps * 32, smem, s>>>(a);
    return cudaGetLastError();
}

// Rows of the batch over the prefix from which the tensor-core kernel takes it.
bool kv8_prefix_tiled(int rows) { return rows > 16; }

cudaError_t launch_kv8_attn(const Kv8Attn& in, const Kv8Prefix& p, int D, int per_token, int num_sms, cudaStream_t s)
{
    Kv8Attn a = in;
    const int R = kv8_attn_row_tile(a.group);
    a.ctas = num_sms * (R == 8 ? 3 : 2);
    a.ctas = a.ctas < kKv8MaxCtas ? a.ctas : kKv8MaxCtas;
    cudaError_t e;
    if (p.splits) {
        e = launch_kv8_prefix(a, p, D, per_token, s);
        if (e != cudaSuccess)
            return e;
    }
    if (a.max_pages || a.ptiles) {
        if (D == 128)
            e = R == 8 ? (per_token ? launch_pieces<128, 1, true>(a, s) : launch_pieces<128, 1, false>(a, s))
                       : (per_token ? launch_pieces<128, 2, true>(a, s) : launch_pieces<128, 2, false>(a, s));
        else
            e = R == 8 ? (per_token ? launch_pieces<64, 1, true>(a, s) : launch_pieces<64, 1, false>(a, s))
                       : (per_token ? launch_pieces<64, 2, true>(a, s) : launch_pieces<64, 2, false>(a, s));
        if (e != cudaSuccess)
            return e;
    }
    const dim3 grid(a.B, a.Hq);
    if (D == 128)
        kv8_join_kernel<128><<<grid, kJoinWarps * 32, 0, s>>>(a, p, R);
    else
        kv8_join_kernel<64><<<grid, kJoinWarps * 32, 0, s>>>(a, p, R);
    return cudaGetLastError();
}

}  // namespace w4a8
