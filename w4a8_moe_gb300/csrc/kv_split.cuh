// The split of the decode attention's work between warps, shared by the caches of
// 8 and of 4 bits (kv8_attn.cu, kv4_attn.cu) and by the join of their pieces.
#pragma once
#include "kv8.cuh"
#include "ptx.cuh"

namespace w4a8 {

constexpr float kMostWeight = 0x1p15f;   // 2^kWeightMost
constexpr int kPlaceUnits = 8;   // units of a warp from which on shares may go by its block's place
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
// the group). The keys of a pair are cut into units (of 16 keys, or 32 with 4 bits) and all units stand in
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
    int places;     // shares by the blocks' places on their SM (1: equal shares)
};
__device__ __forceinline__ int seq_len(const Kv8Attn& a, int b)
{
    return a.max_pages ? min(max(__ldg(a.lens + b), 0), a.max_pages << a.page_shift) : 0;
}
__device__ __forceinline__ int seq_units(const Kv8Attn& a, int b, int unit_shift)
{
    return static_cast<int>((static_cast<unsigned>(seq_len(a, b)) + (1u << unit_shift) - 1) >> unit_shift);
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
__device__ __forceinline__ Line make_line(const Kv8Attn& a, int64_t seq_total, int unit_shift)
{
    Line l;
    l.hr = a.Hkv * a.tiles;
    l.pairs_p = a.Hkv * a.ptiles;
    l.up = (a.prefix_len + (1 << unit_shift) - 1) >> unit_shift;
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
    l.places = a.places > 1 && l.U >= kPlaceUnits * static_cast<int64_t>(a.warps) ? a.places : 1;
    return l;
}
// An SM's schedulers let the warps of its first block go before those of its second
// and so on. With equal shares the last ones end much later, and alone: 64 sequences
// of 8192-16384 keys of 4 bits, the four blocks' warps after 100, 113, 129 and 145 us,
// the memory being busy for the first 100 and half idle then. Where units are many the
// shares therefore go by the block's place, in the proportions of
// Kv8Attn::place_weight: the n / places warps of each place stand together in the line.
__device__ __forceinline__ int64_t weight_before(const Kv8Attn& a, const Line& l, int w)   // of w warps
{
    const int per = l.n / l.places, place = min(w / per, l.places - 1);
    int64_t sum = static_cast<int64_t>(w - place * per) * a.place_weight[place];
    for (int p = 0; p < place; ++p)
        sum += static_cast<int64_t>(per) * a.place_weight[p];
    return sum;
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
template <bool PLACES = false>
__device__ __forceinline__ int64_t warp_begin(const Kv8Attn& a, const Line& l, int w)
{
    if (PLACES && l.places > 1)
        return l.U * weight_before(a, l, w) / weight_before(a, l, l.n);
    return w < l.n1 ? share(l.U1, w, l.n1) : l.U1 + (l.n > l.n1 ? share(l.U - l.U1, w - l.n1, l.n - l.n1) : 0);
}
template <bool PLACES = false>
__device__ __forceinline__ int warp_of(const Kv8Attn& a, const Line& l, int64_t u)
{
    if (PLACES && l.places > 1) {   // the last w whose begin, rounded down, is u or less
        const int per = l.n / l.places;
        int64_t rest = ((u + 1) * weight_before(a, l, l.n) - 1) / l.U;
        int place = 0;
        for (; place < l.places - 1 && rest >= static_cast<int64_t>(per) * a.place_weight[place]; ++place)
            rest -= static_cast<int64_t>(per) * a.place_weight[place];
        return place * per + static_cast<int>(min(rest / a.place_weight[place], static_cast<int64_t>(per - 1)));
    }
    return u < l.U1 ? share_of(l.U1, u, l.n1) : l.n1 + share_of(l.U - l.U1, u - l.U1, l.n - l.n1);
}

// Prefix sums of the sequences' units into `cum` [B + 1] (block 0 also leaves them
// for the join); returns their sum. Lengths out of range set the error word. By a
// block of WARPS warps, which a barrier has to follow before cum[B] is read.
template <int WARPS>
__device__ __forceinline__ int sum_units(const Kv8Attn& a, int* cum, int* warp_sum)
{
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int carry = 0;
    for (int b0 = 0; b0 < a.B; b0 += WARPS * 32) {
        const int b = b0 + tid;
        const int n = b < a.B ? seq_units(a, b, kKv8UnitShift) : 0;
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
        for (int w = 0; w < WARPS; ++w)
            carry += warp_sum[w];
        __syncthreads();
    }
    if (tid == 0) {
        cum[a.B] = carry;
        if (blockIdx.x == 0)
            a.cum[a.B] = carry;
    }
    return carry;
}

}  // namespace w4a8
