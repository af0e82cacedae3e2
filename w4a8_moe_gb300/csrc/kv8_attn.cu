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

constexpr int kWarps = 4;    // per CTA; they share nothing but the prefix sums
constexpr int kStages = 2;   // units in flight per warp
constexpr int kDescs = 64;   // unit descriptors held per warp (two batches of 32)
constexpr float kMostWeight = 0x1p15f;   // 2^kWeightMost
constexpr float kLowest = -3.4028235e38f;   // the reference of a row without keys

// D[16x8] += A[16x16] B[16x8], f16 operands, fp32 accumulators.
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Thread (g, c) of an 8 x 8 matrix of f16 holds row g, columns 2c and 2c + 1:
// the same of its transpose.
__device__ __forceinline__ uint32_t transpose8(uint32_t x)
{
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
__device__ __forceinline__ float lds32(uint32_t at)
{
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(at));
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t at)
{
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at));
    return v;
}

// ---------------------------------------------------------------------------
// The split. A pair is (rows, keys): first the prefix's pairs (kv head, row
// tile of the whole batch), then the sequences' (sequence, kv head, row tile of
// the group). The keys of a pair are cut into units of 16 and all units stand in
// one line in pair order. Warp w of n takes units [U w / n, U (w + 1) / n): equal
// work however ragged the lengths are. Beside a tiled prefix, which holds SMs,
// the warps that run at once get a longer share than those that start after it
// (make_line). The piece of pair p done by warp w is stored in slot p + w: along
// the line p + w rises with every piece, so no two share a slot, and a reader
// finds a pair's slots from the shares' bounds alone.
// ---------------------------------------------------------------------------
struct Line {
    int64_t U;      // units
    int64_t U1;     // of them for the first n1 warps
    int n1, n;      // warps with units
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
// Warps for so many units. Two units are in flight at once, so a second pair of
// them costs a warp another latency (one sequence of 8 heads and 64 keys: 8.4 us
// against 7.0); more pieces cost the join (256 of 48 heads and 60 keys: 22.6 us by
// twos, 18.9 by fours). So few units are spread by twos, up to `spread` warps, and
// more by fours, up to all warps.
__host__ __device__ __forceinline__ int warps_for(int64_t units, int spread, int most)
{
    const int u = units < 1 << 16 ? static_cast<int>(units) : 1 << 16;
    return min(max(min((u + 1) >> 1, spread), u >> 2), most);
}
__device__ __forceinline__ Line make_line(const Kv8Attn& a, int64_t seq_total)
{
    Line l;
    l.hr = a.Hkv * a.tiles;
    l.pairs_p = a.Hkv * a.ptiles;
    l.up = (a.prefix_len + kKv8Unit - 1) / kKv8Unit;
    l.own = static_cast<int64_t>(l.pairs_p) * l.up;
    l.U = l.own + seq_total * l.hr;
    l.U1 = l.U;
    const int late = a.warps - a.free_warps;
    if (late > 0) {
        // Rounded step by step: the writer and the reader of the pieces have to
        // come to the same bounds, so nothing may be contracted in one of them.
        const float unit_us = 1.6f, start_us = 3.0f;   // of a warp
        const float work = __fmul_rn(unit_us, static_cast<float>(l.U)), free = static_cast<float>(a.free_warps);
        if (work > __fmul_rn(free, __fadd_rn(a.free_us, start_us))) {
            // the free warps work for free_us + y, the late ones for y less their start
            const float rest = __fadd_rn(work, -__fmul_rn(free, a.free_us));
            const float y = __fdiv_rn(__fadd_rn(rest, __fmul_rn(start_us, static_cast<float>(late))),
                                      static_cast<float>(a.warps));
            const int64_t u1 = static_cast<int64_t>(__fdiv_rn(__fmul_rn(free, __fadd_rn(a.free_us, y)), unit_us));
            l.U1 = u1 < l.U ? u1 : l.U;
        }
    }
    l.n1 = warps_for(l.U1, a.spread, a.free_warps);
    l.n = l.n1 + (late > 0 ? warps_for(l.U - l.U1, a.spread, late) : 0);
    return l;
}
// (32-bit division where the numbers allow it: warps are fewer than 2^12.)
__device__ __forceinline__ int64_t share(int64_t units, int i, int n)
{
    return units < 1 << 20 ? static_cast<uint32_t>(units) * static_cast<uint32_t>(i) / static_cast<uint32_t>(n)
                           : units * i / n;
}
__device__ __forceinline__ int share_of(int64_t units, int64_t u, int n)
{
    return units < 1 << 20 ? static_cast<int>((static_cast<uint32_t>(u + 1) * static_cast<uint32_t>(n) - 1) /
                                              static_cast<uint32_t>(units))
                           : static_cast<int>(((u + 1) * n - 1) / units);
}
__device__ __forceinline__ int64_t warp_begin(const Line& l, int w)
{
    return w < l.n1 ? share(l.U1, w, l.n1) : l.U1 + (l.n > l.n1 ? share(l.U - l.U1, w - l.n1, l.n - l.n1) : 0);
}
__device__ __forceinline__ int warp_of(const Line& l, int64_t u)
{
    return u < l.U1 ? share_of(l.U1, u, l.n1) : l.n1 + share_of(l.U - l.U1, u - l.U1, l.n - l.n1);
}

// A unit as its warp meets it, found by one lane for each of 32 units ahead.
struct __align__(16) Unit {
    int64_t row;    // cache row (page, head, offset) of its first key
    int pair;
    int live_last;  // keys that exist (1..16), and 256 where the pair ends
};
__device__ __forceinline__ Unit find_unit(const Kv8Attn& a, const Line& line, const int* cum, int64_t u)
{
    Unit x;
    int h, len, n_pages, k;
    const int32_t* pages;
    bool last;
    if (u < line.own) {
        x.pair = static_cast<int>(u / line.up);
        k = static_cast<int>(u - static_cast<int64_t>(x.pair) * line.up);
        h = x.pair / a.ptiles;
        len = a.prefix_len;
        last = k == line.up - 1;
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
        const unsigned n = cum[lo + 1] - cum[lo];
        const int64_t in = rel - static_cast<int64_t>(cum[lo]) * line.hr;
        int j;
        if (in <= 0xFFFFFFFFll) {
            j = static_cast<int>(static_cast<uint32_t>(in) / n);
            k = static_cast<int>(static_cast<uint32_t>(in) - j * n);
        } else {
            j = static_cast<int>(in / n);
            k = static_cast<int>(in - static_cast<int64_t>(j) * n);
        }
        h = j / a.tiles;
        len = seq_len(a, lo);
        last = k == static_cast<int>(n) - 1;
        pages = a.page_table + lo * a.table_stride;
        n_pages = a.max_pages;
        x.pair = line.pairs_p + lo * line.hr + j;
    }
    const int key0 = k * kKv8Unit;
    const int idx = key0 >> a.page_shift;
    int page = idx < n_pages ? __ldg(pages + idx) : -1;
    if (static_cast<unsigned>(page) >= static_cast<unsigned>(a.num_pages)) {
        set_error(a.err, kErrBitIndex);
        page = 0;
    }
    x.row = ((static_cast<int64_t>(page) * a.Hkv + h) << a.page_shift) + (key0 & ((1 << a.page_shift) - 1));
    x.live_last = min(len - key0, kKv8Unit) | (last ? 256 : 0);
    return x;
}

template <int D>
struct Ring {   // one warp's shared memory
    static constexpr int kCodes = kKv8Unit * D;               // bytes of K or V codes of a unit
    static constexpr int kStage = 2 * kCodes + 2 * kKv8Unit * 4;   // K, V, their scales
    static constexpr int desc = kStages * kStage;
    static constexpr int bars = desc + kDescs * 16;
    static constexpr int total = (bars + kStages * 8 + 127) / 128 * 128;   // bulk copies want 16 bytes
};

}  // namespace

// Row tile: 8 rows where the group fits, else 16 (two column tiles of O^T).
int kv8_attn_row_tile(int group) { return group <= 8 ? 8 : 16; }

// Bound by memory: 32 sequences of 4096-8192 keys (416 MB) at 5.7 TB/s, 84 % of a
// copy's rate, with 16 warps an SM, each on one unit with the next two on their
// way. Short sequences are bound by the chain lengths -> page -> codes -> result,
// some 5 us.
//
// Every warp walks its own units, with a ring of bulk copies kStages units
// ahead (across piece boundaries), and stores a piece's result from registers.
// Both products have the rows as their N: S^T = K Q^T with 16 keys as M and
// O^T = V^T P^T with D as M, so no MMA row is idle for groups of 8. Fragments
// come straight from the linear copies: which d a fragment register stands for
// is free as long as q and o use the same order, so every thread reads
// contiguous bytes: of K keys g and g + 8, chunks c of their D values; of V keys
// 2c, 2c+1, 2c+8, 2c+9, chunk g. P^T passes from the first product's layout to
// the second's by an 8 x 8 transpose. A thread's rows are 2c and 2c + 1 in both,
// so the running statistics need no exchange.
template <int D, int NT, bool TOK, int PER_SM>
__global__ void __launch_bounds__(kWarps * 32, PER_SM) kv8_attn_kernel(const __grid_constant__ Kv8Attn a)
{
    using S = Ring<D>;
    constexpr int R = 8 * NT;      // rows of a tile
    constexpr int KS = D / 16;     // k-steps of Q K^T = m-tiles of O^T
    extern __shared__ __align__(128) uint8_t smem[];
    int* cum = reinterpret_cast<int*>(smem + kWarps * S::total);   // [B + 1]
    __shared__ int warp_sum[kWarps];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
    if (!a.beside)
        grid_dep_wait();   // else what came before the tiled prefix is done, and the prefix is not needed
    grid_dep_launch();     // the join reads the lengths only until this kernel has ended

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
        if (b < a.B) {
            cum[b] = base + s - n;
            if (blockIdx.x == 0)
                a.cum[b] = base + s - n;
        }
        for (int w = 0; w < kWarps; ++w)
            carry += warp_sum[w];
        __syncthreads();
    }
    if (tid == 0) {
        cum[a.B] = carry;
        if (blockIdx.x == 0)
            a.cum[a.B] = carry;
    }
    const uint32_t ring = smem_u32(smem) + warp * S::total;
    if (lane < kStages)
        mbar_init(ring + S::bars + lane * 8, 1);
    fence_mbar_init();
    __syncthreads();

    const Line line = make_line(a, carry);
    // few units: one warp on each SM before a second; the first CTAs run first, and
    // the late ones go on from the last warp of theirs that has a share
    const int first = a.free_warps / kWarps, block = static_cast<int>(blockIdx.x);
    int me = block < first ? warp * first + block : line.n1 + (block - first) * kWarps + warp;
    if (block < first && me >= line.n1)
        me = line.n;
    const int64_t u_begin = me < line.n ? warp_begin(line, me) : 0;
    const int units = me < line.n ? static_cast<int>(warp_begin(line, me + 1) - u_begin) : 0;
    Unit* descs = reinterpret_cast<Unit*>(smem + warp * S::total + S::desc);

    // unit i of this warp into its ring slot; batches of 32 descriptors ahead of it
    auto issue = [&](int i) {
        if (i >= units)
            return;
        if (i % 32 == 0) {
            if (i + lane < units)
                descs[(i + lane) % kDescs] = find_unit(a, line, cum, u_begin + i + lane);
            __syncwarp();
        }
        if (lane == 0) {
            const int64_t row = descs[i % kDescs].row;
            const uint32_t dst = ring + (i % kStages) * S::kStage, bar = ring + S::bars + (i % kStages) * 8;
            mbar_arrive_expect_tx(bar, TOK ? S::kStage : 2 * S::kCodes);
            bulk_load(dst, a.k_cache + row * D, S::kCodes, bar);
            bulk_load(dst + S::kCodes, a.v_cache + row * D, S::kCodes, bar);
            if (TOK) {
                bulk_load(dst + 2 * S::kCodes, a.k_scale + row, kKv8Unit * 4, bar);
                bulk_load(dst + 2 * S::kCodes + kKv8Unit * 4, a.v_scale + row, kKv8Unit * 4, bar);
            }
        }
    };
#pragma unroll
    for (int i = 0; i < kStages; ++i)
        issue(i);

    uint32_t qb[KS][NT][2];
    float qs[NT][2], o[KS][NT][4], m[NT][2], l[NT][2];
    int rows = 0, h = 0;
    bool fresh = true;
    for (int i = 0; i < units; ++i) {
        const int pair = descs[i % kDescs].pair, live_last = descs[i % kDescs].live_last;
        const int live = live_last & 255;
        if (fresh) {
            // ---- a new piece. Queries: f16 fragments of q * 2^-e with e from
            // the row's largest element. bf16 has 8 significant bits and f16
            // 11, so only elements below 2^-16 of the row's largest lose
            // anything, and what they lose is at most 2^-25 of it: the size of
            // one fp32 rounding of the product.
            int b = 0, row0;
            const bool prefix = pair < line.pairs_p;
            if (prefix) {
                h = pair / a.ptiles;
                row0 = (pair % a.ptiles) * R;
                rows = min(R, a.B * a.group - row0);
            } else {
                b = (pair - line.pairs_p) / line.hr;
                const int j = (pair - line.pairs_p) % line.hr;
                h = j / a.tiles;
                row0 = (j % a.tiles) * R;
                rows = min(R, a.group - row0);
            }
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
                    for (int e = 0; e < 4; ++e)
                        top = max(top, max((w[e] >> 16) & 0x7FFFu, w[e] & 0x7FFFu));
                }
                top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
                top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
                const int ex = static_cast<int>(top >> 7);
                const int e = top == 0 || ex == 255 ? 0 : max(ex, 1) - 127;
                const float down = ldexpf(1.0f, -e);
                float f = ldexpf(a.sm_scale, e);
                if (!TOK)
                    f *= __ldg(a.k_scale + h);
                f = a.cap > 0.0f ? f / a.cap * (2.0f * kLog2e) : f * kLog2e;
#pragma unroll
                for (int y = 0; y < 2; ++y) {   // of the rows 2c, 2c + 1
                    qs[t][y] = __shfl_sync(0xFFFFFFFFu, f, c * 8 + y * 4);
                    m[t][y] = kLowest;
                    l[t][y] = 0.0f;
                }
#pragma unroll
                for (int j = 0; j < D / 32; ++j) {   // 8 values: two k-steps' two registers each
                    const uint32_t w[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        qb[2 * j + (k >> 1)][t][k & 1] =
                            pack_f16(__uint_as_float(w[k] << 16) * down, __uint_as_float(w[k] & 0xFFFF0000u) * down);
                }
            }
#pragma unroll
            for (int j = 0; j < KS; ++j)
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        o[j][t][k] = 0.0f;
            fresh = false;
        }

        // ---- the unit's codes into registers, and its slot to the next copy
        const uint32_t at = ring + (i % kStages) * S::kStage;
        if (!__all_sync(0xFFFFFFFFu, mbar_wait(ring + S::bars + (i % kStages) * 8, (i / kStages) & 1))) {
            set_error(a.err, kErrBitTimeout);
            for (int j = i + 1; j < min(i + kStages, units); ++j)   // copies in flight end before the warp does
                mbar_wait(ring + S::bars + (j % kStages) * 8, (j / kStages) & 1);
            break;
        }
        uint4 xk[2][D / 64];
        uint32_t xv[4][D / 32];
        float ks[2], vs[2];   // scales of keys g, g + 8
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int j = 0; j < D / 64; ++j)
                xk[t][j] = lds128(at + (t * 8 + g) * D + (j * 4 + c) * 16);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int key = c * 2 + (k & 1) + (k >> 1) * 8;
            if (D == 128) {
                const uint4 w = lds128(at + S::kCodes + key * D + g * 16);
                xv[k][0] = w.x, xv[k][1] = w.y, xv[k][D / 32 - 2] = w.z, xv[k][D / 32 - 1] = w.w;
            } else {
                const uint2 w = lds64(at + S::kCodes + key * D + g * 8);
                xv[k][0] = w.x, xv[k][1] = w.y;
            }
        }
        if (TOK) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                ks[x] = lds32(at + 2 * S::kCodes + (x * 8 + g) * 4);
                vs[x] = lds32(at + 2 * S::kCodes + (kKv8Unit + x * 8 + g) * 4);
            }
        }
        if (live < kKv8Unit) {   // what lies behind the last key may be no number
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (c * 2 + (k & 1) + (k >> 1) * 8 >= live) {
#pragma unroll
                    for (int w = 0; w < D / 32; ++w)
                        xv[k][w] = 0;
                }
#pragma unroll
            for (int x = 0; x < 2; ++x)
                if (TOK && x * 8 + g >= live)
                    ks[x] = 0.0f, vs[x] = 0.0f;
        }
        __syncwarp();
        issue(i + kStages);

        // ---- S^T = K Q^T: s[t][2 x + y] is key g + 8 x, row 8 t + 2c + y
        float s[NT][4];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                s[t][k] = 0.0f;
#pragma unroll
        for (int j = 0; j < D / 64; ++j) {
            const uint32_t w0[4] = {xk[0][j].x, xk[0][j].y, xk[0][j].z, xk[0][j].w};
            const uint32_t w1[4] = {xk[1][j].x, xk[1][j].y, xk[1][j].z, xk[1][j].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                uint32_t a0, a1, a2, a3;
                e4m3x4_to_f16x4(w0[k], a0, a2);
                e4m3x4_to_f16x4(w1[k], a1, a3);
#pragma unroll
                for (int t = 0; t < NT; ++t)
                    mma_f16(s[t], a0, a1, a2, a3, qb[j * 4 + k][t][0], qb[j * 4 + k][t][1]);
            }
        }
        // ---- scores in log2 units (cap * tanh(y) = cap * (1 - 2 / (1 + e^{2y})),
        // qs holding 2 log2(e) / cap); keys past the end are -inf
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                // (rounded once: the reference and the weights see the same score)
                s[t][k] = TOK ? __fmul_rn(s[t][k] * qs[t][k & 1], ks[k >> 1]) : __fmul_rn(s[t][k], qs[t][k & 1]);
            }
        if (a.cap > 0.0f) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    s[t][k] = fmaf(-2.0f * kLog2e * a.cap, rcp(1.0f + ex2(s[t][k])), kLog2e * a.cap);
        }
        if (live < kKv8Unit) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    s[t][k] = (k >> 1) * 8 + g < live ? s[t][k] : -INFINITY;
        }
        // ---- weights under the reference as it stands; where one would come
        // near f16's end the reference is raised and they are taken again
        float p[NT][4];
        auto weigh = [&]() {
            float top = 0.0f;
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    p[t][k] = ex2(s[t][k] - m[t][k & 1]);
                    // (the second bound holds a weight in range where its value's scale is 0)
                    top = fmaxf(top, TOK ? p[t][k] * fmaxf(fabsf(vs[k >> 1]), kLeastScale) : p[t][k]);
                }
            return top;
        };
        if (__any_sync(0xFFFFFFFFu, weigh() > kMostWeight)) {
            float lift[2] = {0.0f, 0.0f};   // log2 of the value scales of keys g, g + 8
            if (TOK) {
                // values of a key that are all zero add nothing, whatever their scale
                // (kv8_write gives them 1): 0 then, so that they lead no reference
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    uint32_t any = 0;
#pragma unroll
                    for (int w = 0; w < D / 32; ++w)
                        any |= xv[k][w];
                    const uint32_t lanes = __ballot_sync(0xFFFFFFFFu, (any & 0x7F7F7F7Fu) != 0);
                    if ((g & 1) == (k & 1) && !(lanes & (0x11111111u << (g >> 1))))
                        vs[k >> 1] = 0.0f;
                }
#pragma unroll
                for (int x = 0; x < 2; ++x)
                    lift[x] = fmaxf(log2f(fabsf(vs[x])), kLeastScaleLog2);
            }
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    float top = TOK ? fmaxf(s[t][y] + lift[0], s[t][2 + y] + lift[1]) : fmaxf(s[t][y], s[t][2 + y]);
#pragma unroll
                    for (int x = 4; x < 32; x <<= 1)
                        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, x));
                    const float to = fmaxf(m[t][y], top - kWeightTop);
                    const float f = ex2(m[t][y] - to);
                    m[t][y] = to;
                    l[t][y] *= f;
#pragma unroll
                    for (int j = 0; j < KS; ++j) {
                        o[j][t][y] *= f;
                        o[j][t][2 + y] *= f;
                    }
                }
            weigh();
        }
        // ---- P^T and O^T += V^T P^T
        uint32_t pb[NT][2];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                l[t][0] += p[t][2 * x];
                l[t][1] += p[t][2 * x + 1];
                pb[t][x] = transpose8(TOK ? pack_f16(p[t][2 * x] * vs[x], p[t][2 * x + 1] * vs[x])
                                          : pack_f16(p[t][2 * x], p[t][2 * x + 1]));
            }
#pragma unroll
        for (int w = 0; w < D / 32; ++w)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const uint32_t sel = half ? 0x7362u : 0x5140u;
                uint32_t a0, a1, a2, a3;
                e4m3x4_to_f16x4(prmt(xv[0][w], xv[1][w], sel), a0, a1);
                e4m3x4_to_f16x4(prmt(xv[2][w], xv[3][w], sel), a2, a3);
#pragma unroll
                for (int t = 0; t < NT; ++t)
                    mma_f16(o[w * 2 + half][t], a0, a1, a2, a3, pb[t][0], pb[t][1]);
            }

        // ---- the piece ends with its pair or with the warp's units
        if ((live_last & 256) || i + 1 == units) {
            const float vscale = TOK ? 1.0f : __ldg(a.v_scale + h);
            const int64_t slot = static_cast<int64_t>(pair) + me;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
#pragma unroll
                for (int y = 0; y < 2; ++y) {
#pragma unroll
                    for (int x = 4; x < 32; x <<= 1)
                        l[t][y] += __shfl_xor_sync(0xFFFFFFFFu, l[t][y], x);
                    if (g == 0 && t * 8 + c * 2 + y < rows)
                        a.part_ml[slot * R + t * 8 + c * 2 + y] = make_float2(m[t][y], l[t][y]);
                }
                float* dst = a.part_o + (slot * R + t * 8 + c * 2) * D + g * (D / 8);
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    if (t * 8 + c * 2 + e < rows) {
#pragma unroll
                        for (int j = 0; j < KS; j += 2)
                            *reinterpret_cast<float4*>(dst + e * D + 2 * j) =
                                make_float4(o[j][t][e] * vscale, o[j][t][2 + e] * vscale, o[j + 1][t][e] * vscale,
                                            o[j + 1][t][2 + e] * vscale);
                    }
            }
            fresh = true;
        }
    }
    grid_dep_wait();   // the join after this kernel also reads what the one before it wrote
}

// Adds up the pieces of a (sequence, query head): W warps take them in turn, or,
// where there are very many rows, half a warp (W = 0). The fewer rows, the more
// warps take one: with few rows each has many pieces, and only their number hides
// the loads' latency, which is what bounds this; with very many rows the warps of
// others do, and each takes few registers.
constexpr int kJoinCta = 4;      // warps of a CTA where a row has one or less
constexpr int kJoinSums = 128;   // sequences up to which a warp sums their units itself
template <int D, int W>
__global__ void __launch_bounds__((W > 1 ? W : kJoinCta) * 32) kv8_join_kernel(const __grid_constant__ Kv8Attn a,
                                                                         const __grid_constant__ Kv8Prefix p, int R)
{
    constexpr int L = W ? 32 : 16;                  // lanes of a row
    constexpr int V = D / L, F = V >= 4 ? 4 : 2;    // values of a lane, in groups of F that stand L F apart
    constexpr int S = W ? W : 1;                    // strides over the pieces
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid % L;
    const int head = W > 1 ? blockIdx.x : blockIdx.x * (kJoinCta * 32 / L) + tid / L;   // b * Hq + query head
    const int first_piece = W > 1 ? warp : 0;
    const bool there = head < a.B * a.Hq;
    const int b = there ? head / a.Hq : 0, qh = there ? head - b * a.Hq : 0, h = qh / a.group, gi = qh - h * a.group;
    // units before the sequence's and all of them: a short sum over the lengths
    // while the kernel before is still at work, else what it left
    const bool sum_here = a.B <= kJoinSums;
    int before = 0, units = 0, all = 0;
    if (sum_here) {
        for (int i = lane; i < a.B; i += L) {
            const int n = seq_units(a, i);
            all += n;
            before += i < b ? n : 0;
            units += i == b ? n : 0;
        }
#pragma unroll
        for (int x = L / 2; x > 0; x >>= 1) {
            all += __shfl_xor_sync(0xFFFFFFFFu, all, x);
            before += __shfl_xor_sync(0xFFFFFFFFu, before, x);
            units += __shfl_xor_sync(0xFFFFFFFFu, units, x);
        }
    } else {
        grid_dep_wait();
        if (a.max_pages) {
            before = a.cum[b];
            units = a.cum[b + 1] - before;
            all = a.cum[a.B];
        }
    }
    const Line line = make_line(a, all);

    // the row's pieces: [0, n0) of the tiled prefix, [n0, n1) of the untiled one, [n1, n2) of its own keys
    const int row = b * a.group + gi;
    const int n0 = p.splits;
    int n1 = n0, n2;
    int64_t at_pre = 0, at_own = 0;   // the first piece's row, minus its number times R
    if (a.ptiles) {
        const int pair = h * a.ptiles + row / R;
        const int64_t first = static_cast<int64_t>(pair) * line.up;
        const int w = warp_of(line, first);
        n1 += warp_of(line, first + line.up - 1) - w + 1;
        at_pre = static_cast<int64_t>(pair + w - n0) * R + row % R;
    }
    n2 = n1;
    if (units) {
        const int j = h * a.tiles + gi / R;
        const int64_t first = line.own + static_cast<int64_t>(before) * line.hr + static_cast<int64_t>(j) * units;
        const int w = warp_of(line, first);
        n2 += warp_of(line, first + units - 1) - w + 1;
        at_own = static_cast<int64_t>(line.pairs_p + b * line.hr + j + w - n1) * R + gi % R;
    }
    n2 = there ? n2 : 0;
    if (sum_here)
        grid_dep_wait();
    // Lane i of a row finds piece first_piece + S i and its weight; then every
    // lane reads its values of all of them. Nothing that is read waits for
    // anything but the kernel before. (Both halves of a warp go round together.)
    const int most = W ? n2 : max(n2, __shfl_xor_sync(0xFFFFFFFFu, n2, 16));
    float top = -INFINITY, sum = 0.0f, acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i)
        acc[i] = 0.0f;
    for (int k0 = first_piece; k0 < most; k0 += L * S) {
        const int k = k0 + S * lane;
        const float* src = a.part_o;
        float2 ml = make_float2(-INFINITY, 0.0f);
        if (k < n2) {
            const bool tiled = k < n0;
            const int64_t at = tiled ? (static_cast<int64_t>(k) * a.Hkv + h) * a.B * a.group + row
                                     : (k < n1 ? at_pre : at_own) + static_cast<int64_t>(k) * R;
            src = (tiled ? p.part_o : a.part_o) + at * D;
            ml = (tiled ? p.part_ml : a.part_ml)[at];
        }
        const int n = min(L, (n2 - k0 + S - 1) / S), rounds = min(L, (most - k0 + S - 1) / S);
        // Pieces whose values are on their way together: many where the rows are few (64
        // sequences over 8192, 8 / 12 / 16 / 20: 29.7 / 28.6 / 27.9 / 28.1 us), else few, so
        // that more rows fit an SM (100 of 48 heads and 60 own keys, 4 / 3 / 2 10.8 / 10.6 / 10.3).
        constexpr int kAhead = W ? 16 : D == 128 ? 2 : 6;
        float v[kAhead][V];
        auto fetch = [&](int j0) {
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const float* from = reinterpret_cast<const float*>(
                    __shfl_sync(0xFFFFFFFFu, reinterpret_cast<unsigned long long>(src), (j0 + j) % L, L));
                if (j0 + j < n) {
#pragma unroll
                    for (int i = 0; i < V; i += F) {
                        const float* x = from + (i / F * L + lane) * F;
                        if (F == 4) {
                            const float4 w = *reinterpret_cast<const float4*>(x);
                            v[j][i] = w.x, v[j][i + 1] = w.y, v[j][i + F - 2] = w.z, v[j][i + F - 1] = w.w;
                        } else {
                            const float2 w = *reinterpret_cast<const float2*>(x);
                            v[j][i] = w.x, v[j][i + 1] = w.y;
                        }
                    }
                }
            }
        };
        fetch(0);
        float best = ml.x;
#pragma unroll
        for (int x = L / 2; x > 0; x >>= 1)
            best = fmaxf(best, __shfl_xor_sync(0xFFFFFFFFu, best, x));
        const float to = fmaxf(top, best);
        const float ref = to == -INFINITY ? 0.0f : to;
        const float f0 = ex2(top - ref), f1 = ex2(ml.x - ref);
        float l = ml.y * f1;
#pragma unroll
        for (int x = L / 2; x > 0; x >>= 1)
            l += __shfl_xor_sync(0xFFFFFFFFu, l, x);
        sum = sum * f0 + l;
        top = to;
#pragma unroll
        for (int i = 0; i < V; ++i)
            acc[i] *= f0;
        for (int j0 = 0; j0 < rounds; j0 += kAhead) {
            if (j0 > 0)
                fetch(j0);
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const float f = __shfl_sync(0xFFFFFFFFu, f1, (j0 + j) % L, L);
                if (j0 + j < n) {
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        acc[i] += v[j][i] * f;
                }
            }
        }
    }
    if (W > 1) {
        __shared__ float so[S][D];
        __shared__ float2 sml[S];
#pragma unroll
        for (int i = 0; i < V; ++i)
            so[warp][i * L + lane] = acc[i];
        if (lane == 0)
            sml[warp] = make_float2(top, sum);
        __syncthreads();
        if (warp > 0)
            return;
#pragma unroll
        for (int w = 1; w < S; ++w)
            top = fmaxf(top, sml[w].x);
        const float ref = top == -INFINITY ? 0.0f : top;
        sum = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i)
            acc[i] = 0.0f;
#pragma unroll
        for (int w = 0; w < S; ++w) {
            const float f = ex2(sml[w].x - ref);
            sum += sml[w].y * f;
#pragma unroll
            for (int i = 0; i < V; ++i)
                acc[i] += so[w][i * L + lane] * f;
        }
    }
    if (!there)
        return;
    const bool empty = sum == 0.0f;
    uint16_t* dst = a.out + static_cast<int64_t>(head) * D;
#pragma unroll
    for (int i = 0; i < V; i += F) {
        uint32_t r[F / 2];
#pragma unroll
        for (int j = 0; j < F; j += 2)
            r[j / 2] = static_cast<uint32_t>(float_to_bf16_bits(empty ? 0.0f : acc[i + j] / sum)) |
                       (static_cast<uint32_t>(float_to_bf16_bits(empty ? 0.0f : acc[i + j + 1] / sum)) << 16);
        uint16_t* x = dst + (i / F * L + lane) * F;
        if (F == 4)
            *reinterpret_cast<uint2*>(x) = make_uint2(r[0], r[F / 2 - 1]);
        else
            *reinterpret_cast<uint32_t*>(x) = r[0];
    }
    if (a.lse && lane == 0)
        a.lse[head] = empty ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
}

static int ring_smem(int D, int B) { return kWarps * (D == 128 ? Ring<128>::total : Ring<64>::total) + (B + 1) * 4; }

template <int D, int NT, bool TOK, int PER_SM>
static cudaError_t launch_pieces(const Kv8Attn& a, cudaStream_t s)
{
    const int smem = ring_smem(D, a.B);
    auto kern = kv8_attn_kernel<D, NT, TOK, PER_SM>;
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess)
            return e;
    }
    return launch_dependent(kern, dim3(a.warps / kWarps), dim3(kWarps * 32), smem, s, a);
}

template <int D, int NT, int PER_SM>
static cudaError_t launch_pieces(const Kv8Attn& a, int per_token, cudaStream_t s)
{
    return per_token ? launch_pieces<D, NT, true, PER_SM>(a, s) : launch_pieces<D, NT, false, PER_SM>(a, s);
}

// Units of the sequences' own keys if they fill their page tables: what the host can know of them.
static int64_t most_units(const Kv8Attn& a)
{
    return static_cast<int64_t>(a.B) * a.Hkv * a.tiles * ((a.max_pages << a.page_shift) / kKv8Unit);
}

// Warps that take a row of the join (0: half a warp). Several warps pay while a row
// may have many pieces and all of the rows' blocks fit the SMs at once: 8 up to 2
// rows an SM, 4 up to 4 (7 with D 64), 2 up to 8. `pieces` is what the page tables
// allow, an upper bound: inside those limits a row of few pieces loses little by
// too many warps, but beyond them much. us in all, own keys alone but for the last:
//   576 rows (12 sequences of 48 heads), 4 / 2 / 1: 60 own keys 8.7 / 8.6 / 8.3,
//     1-4000 20.7 / 21.8 / 23.9; 840 (30 of 28) 11.2 / 8.9 / 8.5, 24.8 / 23.0 / 24.3
//   1024 of D 64 (64 of 16), 4 / 2 / 1: 9.9 / 10.1 / 9.9, 14.1 / 15.7 / 18.8; 1120
//     (70 of 16) 12.1 / 10.1 / 9.9, 16.9 / 15.8 / 18.5
//   1280 (10 of 128), 2 / 1: 12.6 / 10.4, 31.0 / 29.5
//   over a prefix, 8 / 4: 272 of D 64 over 4999 tokens and 1-2000 own keys 12.0 /
//     13.9; 320 over 9000 and 60 17.3 / 15.0, 576 over 20000 25.5 / 22.4
// Half a warp a row where rows are very many, 1 / half: 4800 of 60 own keys 13.8 /
// 10.5, of 1-1000 36.7 / 34.6; 2400 11.6 / 11.5, 19.5 / 23.3.
static int join_warps(const Kv8Attn& a, const Kv8Prefix& p, int D, int num_sms)
{
    const int heads = a.B * a.Hq, pairs = a.B * a.Hkv * a.tiles;
    const int pieces = p.splits + warps_for(most_units(a), a.spread, a.warps) / pairs;
    if (heads <= num_sms || (pieces > 16 && heads <= 2 * num_sms))
        return 8;
    if (heads <= 2 * num_sms || ((pieces > 16 || p.splits > 8) && heads <= 4 * num_sms) ||
        (pieces > 24 && D == 64 && heads <= 7 * num_sms))
        return 4;
    if (pieces > 12 && heads <= 8 * num_sms)
        return 2;
    return heads > 18 * num_sms ? 0 : 1;
}

template <int D>
static cudaError_t launch_join(const Kv8Attn& a, const Kv8Prefix& p, int R, int num_sms, cudaStream_t s)
{
    const int heads = a.B * a.Hq, warps = join_warps(a, p, D, num_sms);
    if (warps > 1)
        return launch_dependent(warps == 8   ? kv8_join_kernel<D, 8>
                                : warps == 4 ? kv8_join_kernel<D, 4>
                                             : kv8_join_kernel<D, 2>,
                                dim3(heads), dim3(warps * 32), 0, s, a, p, R);
    const int rows = kJoinCta * (warps ? 1 : 2);   // of a CTA
    return launch_dependent(warps ? kv8_join_kernel<D, 1> : kv8_join_kernel<D, 0>, dim3((heads + rows - 1) / rows),
                            dim3(kJoinCta * 32), 0, s, a, p, R);
}

// Whether the tensor-core kernel takes the prefix. It costs a third launch and
// whole SMs; without it every 8 rows read the prefix again, from L2, at the cost
// of a unit of a sequence's own keys. 48 query and 8 kv heads, 16 sequences of up
// to 64 own keys, us without / with: 512 prefix tokens (3072 such units) 13.3 /
// 13.8, 1024 15.5 / 13.9, 2048 22.6 / 14.5; one sequence of 48 query heads (6 rows)
// 16384 tokens (8192 units) 21.7 / 19.0, 65536 47.6 / 50.8.
bool kv8_prefix_tiled(int Hkv, int rows, int prefix_len)
{
    const int64_t units = static_cast<int64_t>(Hkv) * ((rows + 7) / 8) * ((prefix_len + kKv8Unit - 1) / kKv8Unit);
    return units > 3072;
}

// How the units are shared out (a.warps to a.spread); blocks an SM of their kernel.
static int lay_out(Kv8Attn& a, const Kv8Prefix& p, int D, int num_sms)
{
    const int R = kv8_attn_row_tile(a.group);
    const int64_t pairs = static_cast<int64_t>(a.Hkv) * (a.ptiles + static_cast<int64_t>(a.B) * a.tiles);
    // As many as registers allow, but for 16 rows of D 128, which spill at three: three
    // only where the tables allow very many units and the sequences are many too. 16
    // query and 1 kv heads, us at two / three: 40 sequences of 1-4000 own keys 16.9 /
    // 18.9, 64 of 8000 39.3 / 42.1, 100 of 1-4000 25.0 / 27.6, of 8000 55.7 / 51.9, 256
    // of 8000 124 / 114.
    const bool two = R == 16 && D == 128 && (most_units(a) < 40000 || pairs < 96);
    const int fit = 228 * 1024 / (ring_smem(D, a.B) + 1024);   // CTAs an SM holds: by registers, by shared memory
    const int blocks = min(R == 8 ? 4 : two ? 2 : 3, fit), per_sm = blocks * kWarps;
    a.warps = num_sms * per_sm;
    // a CTA of the tiled prefix takes a whole SM; the others' warps can start at once
    const int taken = p.splits * a.Hkv * p.row_pairs;
    a.free_warps = taken ? max(num_sms - taken, 0) * per_sm : a.warps;
    a.free_us = p.us;
    a.warps = min(a.warps, kKv8MaxWarps);
    a.free_warps = min(a.free_warps, kKv8MaxWarps);
    // by twos up to 128 pieces a pair (one sequence of 16 heads and 30000 keys, 937 / 468
    // pieces: 27.2 / 16.6 us) and 1536 warps (64 of 8 heads and 1000 keys, 1024 / 1536 /
    // 2048: 12.6 / 12.2 / 13.3), or 2048 where a pair then has 8 pieces at most
    a.spread = static_cast<int>(min(max(min(8 * pairs, int64_t{2048}), int64_t{1536}), 128 * pairs));
    return blocks;
}

void kv8_attn_layout(const Kv8Attn& in, const Kv8Prefix& p, int D, int num_sms, int* blocks_per_sm, int* warps_a_row)
{
    Kv8Attn a = in;
    *blocks_per_sm = lay_out(a, p, D, num_sms);
    *warps_a_row = join_warps(a, p, D, num_sms);
}

cudaError_t launch_kv8_attn(const Kv8Attn& in, const Kv8Prefix& p, int D, int per_token, int num_sms, cudaStream_t s)
{
    Kv8Attn a = in;
    const int R = kv8_attn_row_tile(a.group);
    const bool two = lay_out(a, p, D, num_sms) == 2;
    cudaError_t e;
    if (p.splits) {
        e = launch_kv8_prefix(a, p, D, per_token, s);
        if (e != cudaSuccess)
            return e;
    }
    if (a.max_pages || a.ptiles) {
        a.beside = p.splits > 0;
        if (D == 128)
            e = R == 8 ? launch_pieces<128, 1, 4>(a, per_token, s)
                : two  ? launch_pieces<128, 2, 2>(a, per_token, s)
                       : launch_pieces<128, 2, 3>(a, per_token, s);
        else
            e = R == 8 ? launch_pieces<64, 1, 4>(a, per_token, s) : launch_pieces<64, 2, 3>(a, per_token, s);
        if (e != cudaSuccess)
            return e;
    }
    return D == 128 ? launch_join<128>(a, p, R, num_sms, s) : launch_join<64>(a, p, R, num_sms, s);
}

}  // namespace w4a8
