// Decode attention over the key/value cache of 4 bits.
//
// "ROCm: enable trillion-parameter MoE models with INT4-FP8 single node",
// config.json (48 query and 8 key/value heads): the attention of kv8_attn.cu for a
// cache of the weights' width.
//
// A key is k_j = s_j c_j + m_j with codes c_j in 0..15, a value v_j = t_j d_j + n_j:
//   x_j = sm_scale * (s_j (q . c_j) + m_j sum(q))       (cap > 0: cap * tanh(x_j / cap))
//   out = (sum_j (e^{x_j} t_j) d_j + sum_j e^{x_j} n_j) / sum_j e^{x_j}
// so the matrix products run over the codes, and the least values are one number a
// key. The split between warps, the pieces and their join are those of the FP8 cache.
#include <math.h>

#include "internal.h"
#include "kv4.cuh"
#include "kv_split.cuh"

namespace w4a8 {

namespace {

constexpr int kWarps = 4;    // per CTA; they share nothing but the prefix sums
constexpr int kUnitShift = kKv4UnitShift;
constexpr int kUnit = 1 << kUnitShift;   // keys
constexpr int kSub = kUnit / 16;         // of them in one product
constexpr int kDescs = 64;   // unit descriptors held per warp (two batches of 32)

// A unit as its warp meets it, found by one lane for each of 32 units ahead.
struct __align__(16) Unit {
    int64_t row[2];   // cache rows (page, head, offset) of its first and its seventeenth key
    int pair;
    int live_last;    // keys that exist (1..32), 256 where the pair ends, 512 where a token does not see all of them
    int key0;
    int tokens;       // that the pair's rows belong to
};

template <int D>
struct Ring {   // one warp's shared memory
    static constexpr int kStages = 2;             // units in flight
    static constexpr int kCodes = kUnit * D / 2;  // bytes of K or V codes of a unit
    static constexpr int kStage = 2 * kCodes + 2 * kUnit * 4;   // K, V, their scales
    static constexpr int desc = kStages * kStage;
    static constexpr int total = (desc + kDescs * static_cast<int>(sizeof(Unit)) + 127) / 128 * 128;
};

__device__ __forceinline__ int64_t page_row(const Kv4Attn& a, const int32_t* pages, int h, int key)
{
    const int idx = key >> a.page_shift;
    int page = idx < a.max_pages ? __ldg(pages + idx) : -1;
    if (static_cast<unsigned>(page) >= static_cast<unsigned>(a.num_pages)) {
        set_error(a.err, kErrBitIndex);
        page = 0;
    }
    return cache_row(a.page_shift, a.Hkv, (static_cast<int64_t>(page) << a.page_shift) + (key & ((1 << a.page_shift) - 1)),
                     h);
}
// Prefix sums of the sequences' units into `cum` [B + 1] (block 0 also leaves them
// for the join); returns their sum. Lengths out of range set the error word. By a
// block of WARPS warps, which a barrier has to follow before cum is read: a thread
// takes some sequences in a row, so that the block meets once (4096 sequences 61.6 ->
// 56.0 us, 1024 59.0 -> 55.2 against WARPS * 32 at a time).
template <int WARPS>
__device__ __forceinline__ int sum_lengths(const Kv8Attn& a, int* cum, int* warp_sum)
{
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int per = (a.B + WARPS * 32 - 1) / (WARPS * 32), b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
    int n = 0;
#pragma unroll 4
    for (int b = b0; b < b1; ++b) {
        n += seq_units(a, b, kUnitShift);
        if (blockIdx.x == 0 && a.max_pages &&
            static_cast<unsigned>(__ldg(a.lens + b)) > static_cast<unsigned>(a.max_pages << a.page_shift))
            set_error(a.err, kErrBitIndex);
    }
    int s = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xFFFFFFFFu, s, o);
        s += lane >= o ? t : 0;
    }
    if (lane == 31)
        warp_sum[warp] = s;
    __syncthreads();
    int base = s - n, total = 0;
    for (int w = 0; w < WARPS; ++w) {
        base += w < warp ? warp_sum[w] : 0;
        total += warp_sum[w];
    }
    for (int b = b0; b < b1; ++b) {
        cum[b] = base;
        if (blockIdx.x == 0)
            a.cum[b] = base;
        base += seq_units(a, b, kUnitShift);
    }
    if (tid == 0) {
        cum[a.B] = total;
        if (blockIdx.x == 0)
            a.cum[a.B] = total;
    }
    return total;
}

// Several tokens of a sequence share a tile of rows where they are neighbours in the
// batch: each run of tokens with one sequence is cut into tiles of up to per_tile
// tokens, and the first of a tile stands for it in the line. Prefix sums of the tiles'
// units as sum_lengths has them (0 for the others), and, from block 0, whose tile each
// token is in.
template <int WARPS>
__device__ __forceinline__ int sum_tiles(const Kv4Attn& a, int* cum, int* warp_sum)
{
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    __shared__ int warp_start[WARPS];
    int carry = 0, carry_start = 0;
    for (int b0 = 0; b0 < a.B; b0 += WARPS * 32) {
        const int b = b0 + tid;
        const int seq = b < a.B ? __ldg(a.seqs + b) : 0;
        // where the token's run starts: the last boundary up to it
        int start = b < a.B && (b == 0 || __ldg(a.seqs + b - 1) != seq) ? b : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1)
            start = max(start, __shfl_up_sync(0xFFFFFFFFu, start, min(o, lane)));
        if (lane == 31)
            warp_start[warp] = start;
        __syncthreads();
        start = max(start, carry_start);
        for (int w = 0; w < warp; ++w)
            start = max(start, warp_start[w]);
        for (int w = 0; w < WARPS; ++w)
            carry_start = max(carry_start, warp_start[w]);
        const int in_tile = (b - start) % a.per_tile;
        int n = 0;
        if (b < a.B) {
            if (blockIdx.x == 0) {
                a.lead[b] = b - in_tile;
                if (static_cast<unsigned>(__ldg(a.lens + b)) > static_cast<unsigned>(a.max_pages << a.page_shift))
                    set_error(a.err, kErrBitIndex);
            }
            if (in_tile == 0)
                for (int j = 0; j < a.per_tile && b + j < a.B && __ldg(a.seqs + b + j) == seq; ++j)
                    n = max(n, seq_units(a, b + j, kUnitShift));
        }
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

template <bool MULTI>
__device__ __forceinline__ Unit find_unit(const Kv4Attn& a, const Line& line, const int* cum, int64_t u)
{
    int lo = 0, hi = a.B;   // the last b with cum[b] * hr <= u
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (static_cast<int64_t>(cum[mid]) * line.hr <= u)
            lo = mid;
        else
            hi = mid;
    }
    const unsigned n = cum[lo + 1] - cum[lo];
    const int64_t in = u - static_cast<int64_t>(cum[lo]) * line.hr;
    int j, k;
    if (in <= 0xFFFFFFFFll) {
        j = static_cast<int>(static_cast<uint32_t>(in) / n);
        k = static_cast<int>(static_cast<uint32_t>(in) - j * n);
    } else {
        j = static_cast<int>(in / n);
        k = static_cast<int>(in - static_cast<int64_t>(j) * n);
    }
    int seq = lo;
    if (a.seqs) {
        seq = __ldg(a.seqs + lo);
        if (static_cast<unsigned>(seq) >= static_cast<unsigned>(a.num_seqs)) {
            set_error(a.err, kErrBitIndex);
            seq = 0;
        }
    }
    const int h = j / a.tiles, key0 = k << kUnitShift;
    const int32_t* pages = a.page_table + seq * a.table_stride;
    Unit x;
    x.key0 = key0;
    x.tokens = 1;
    int len = seq_len(a, lo), least = len;
    if (MULTI)
        for (; x.tokens < a.per_tile && lo + x.tokens < a.B && __ldg(a.seqs + lo + x.tokens) == __ldg(a.seqs + lo); ++x.tokens) {
            const int other = seq_len(a, lo + x.tokens);
            len = max(len, other), least = min(least, other);
        }
    x.pair = lo * line.hr + j;
    x.row[0] = page_row(a, pages, h, key0);
    // a page of 16 ends inside the unit, and the next may not exist
    x.row[1] = a.page_shift >= kUnitShift ? x.row[0] + 16 : len - key0 > 16 ? page_row(a, pages, h, key0 + 16) : x.row[0];
    x.live_last = min(len - key0, kUnit) | (k == static_cast<int>(n) - 1 ? 256 : 0) | (least - key0 < kUnit ? 512 : 0);
    return x;
}

__device__ __forceinline__ void copy16(uint32_t to, const void* from)
{
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}

}  // namespace

// Bound by instructions and memory alike: 64 sequences of 8192-16384 keys, 32 query and
// 8 kv heads (857 MB) take 143 us, 6.0 TB/s or 88 % of a copy's rate, with the units'
// arithmetic left out 129 us; a unit is 477 instructions of a warp, 176 of them the
// masks below (integer instructions, which go at half the rate), 32 matrix products.
// Short sequences are bound by the chain lengths -> page -> codes -> result -> join,
// some 7 us.
//
// Fragments. An f16 whose bits are 0000 0000 0000 cccc is the subnormal number
// c 2^-24, and one with the code four bits up is c 2^-20; the tensor cores take
// subnormals as they are, so codes become operands by a mask, two to a register,
// without any conversion. The powers of two are taken out again where it costs
// nothing: of a key's codes in the queries that meet them (2^14 or 2^10 times the
// query, whose largest element stands in [1, 2)), of a value's in the result.
//   word of 8 codes: & 000F000F -> codes 0, 4; & 00F000F0 -> 1, 5; shifted by 8 -> 2, 6 and 3, 7
// Which d a fragment register stands for is free as long as q and o use the same
// order. Both products have the rows as their N: S^T = K Q^T with 16 keys as M and
// O^T = V^T P^T with D as M. A thread reads, of K's keys g and g + 8, chunk c of
// their D codes, and of V's keys 2c, 2c + 1, 2c + 8, 2c + 9 (the pairs of an operand
// register), chunk g. So that these reads meet no bank twice, the upper four of eight
// keys are taken in the order 5 4 7 6, and rows of D 128, two of which cover the banks,
// have the halves of every other two exchanged.
template <int D, int NT, bool MULTI, int PER_SM>
__global__ void __launch_bounds__(kWarps * 32, PER_SM) kv4_attn_kernel(const __grid_constant__ Kv4Attn a)
{
    using S = Ring<D>;
    constexpr int kStages = S::kStages;
    constexpr int R = 8 * NT;      // rows of a tile
    constexpr int KS = D / 16;     // k-steps of Q K^T = m-tiles of O^T
    constexpr int WK = D / 32;     // words of a thread's chunk of a key: 8 codes each
    constexpr int WV = D / 64;     // and of a value
    extern __shared__ __align__(128) uint8_t smem[];
    int* cum = reinterpret_cast<int*>(smem + kWarps * S::total);   // [B + 1]
    __shared__ int warp_sum[kWarps];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
    const int swap_g = g ^ (g >> 2), swap_c = c >> 1;   // keys in the order 0 1 2 3 5 4 7 6 (see above)
    grid_dep_wait();
    grid_dep_launch();     // the join reads the lengths only until this kernel has ended
    const int total = MULTI ? sum_tiles<kWarps>(a, cum, warp_sum) : sum_lengths<kWarps>(a, cum, warp_sum);
    const uint32_t ring = smem_u32(smem) + warp * S::total;
    __syncthreads();

    const Line line = make_line(a, total, kUnitShift);
    // Few units: one warp on each SM before a second. Very many: a block takes one of the
    // shares for its place on the SM, and where those are gone one of another place's
    // (which block does a share changes no result). There are as many shares as blocks,
    // so one is found, unless the workspace's header was not zero.
    int place = 0, block = blockIdx.x;
    const int sms = gridDim.x / line.places;
    if (line.places > 1) {
        __shared__ int mine;
        if (tid == 0) {
            unsigned slot;
            asm volatile("mov.u32 %0, %warpid;" : "=r"(slot));
            int p = min(static_cast<int>(slot) / kWarps, line.places - 1), tries = 0;
            unsigned ticket;
            while ((ticket = atomicAdd(a.tickets + p, 1u)) >= static_cast<unsigned>(sms) && ++tries < line.places)
                p = p + 1 < line.places ? p + 1 : 0;
            if (tries == line.places)
                set_error(a.err, kErrBitIndex);
            mine = tries == line.places ? blockIdx.x : p * sms + ticket;
        }
        __syncthreads();
        place = mine / sms;
        block = mine - place * sms;
    }
    const int me = (place * kWarps + warp) * sms + block;
    const int64_t u_begin = me < line.n ? warp_begin<true>(a, line, me) : 0;
    const int units = me < line.n ? static_cast<int>(warp_begin<true>(a, line, me + 1) - u_begin) : 0;
    Unit* descs = reinterpret_cast<Unit*>(smem + warp * S::total + S::desc);

    // unit i of this warp into its ring slot; batches of 32 descriptors ahead of it.
    // (Every call is one group of copies, empty behind the last unit.)
    auto issue = [&](int i) {
        if (i < units) {
            if (i % 32 == 0) {
                if (i + lane < units)
                    descs[(i + lane) % kDescs] = find_unit<MULTI>(a, line, cum, u_begin + i + lane);
                __syncwarp();
            }
            const Unit& x = descs[i % kDescs];
            const uint32_t stage = ring + (i % kStages) * S::kStage;
            const uint32_t to = stage + (D == 128 ? lane ^ (lane >> 2 & 2) : lane) * 16;
#pragma unroll
            for (int p = 0; p < 2; ++p) {   // 16 keys
                const int64_t from = x.row[p] * (D / 2) + lane * 16;
#pragma unroll
                for (int j = 0; j < D / 64; ++j) {
                    copy16(to + p * 8 * D + j * 512, a.k_cache + from + j * 512);
                    copy16(to + S::kCodes + p * 8 * D + j * 512, a.v_cache + from + j * 512);
                }
            }
            if (lane < 16)   // four pairs of numbers of a key or a value each
                copy16(stage + 2 * S::kCodes + lane * 16, (lane & 8 ? a.v_scale : a.k_scale) + x.row[(lane >> 2) & 1] + (lane & 3) * 4);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < kStages; ++i)
        issue(i);

    uint32_t qb[KS][NT][2];
    float qs[NT][2], qm[NT][2], o[KS][NT][4], m[NT][2];
    F2 l2[NT], ln2[NT];   // sums of the weights, and of weights times least values, of rows 2c and 2c + 1
    int rows = 0, sees[NT][2];   // MULTI: keys that rows 2c and 2c + 1 see
    bool fresh = true;
    for (int i = 0; i < units; ++i) {
        const int pair = descs[i % kDescs].pair, live_last = descs[i % kDescs].live_last;
        const int live = live_last & 255;
        if (fresh) {
            // ---- a new piece. Queries: f16 fragments of q * 2^-e, e from the row's
            // largest element, times the powers above. bf16 has 8 significant bits,
            // so only elements below 2^-27 of the largest lose anything, 2^-35 of it.
            const int b = pair / line.hr, j = pair % line.hr;
            const int h = j / a.tiles, row0 = (j % a.tiles) * R;   // (MULTI: one tile)
            rows = MULTI ? descs[i % kDescs].tokens * a.group : min(R, a.group - row0);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const int r = row0 + t * 8 + g;
                uint4 raw[D / 32];
                if (t * 8 + g < rows) {
                    const int token = MULTI ? r / a.group : 0;
                    const uint16_t* src = a.q + (b + token) * a.q_stride +
                                          static_cast<int64_t>(h * a.group + r - token * a.group) * D + c * (D / 4);
#pragma unroll
                    for (int w = 0; w < WK; ++w)
                        raw[w] = __ldg(reinterpret_cast<const uint4*>(src) + w);
                } else {
#pragma unroll
                    for (int w = 0; w < WK; ++w)
                        raw[w] = make_uint4(0, 0, 0, 0);
                }
                uint32_t top = 0;
#pragma unroll
                for (int w = 0; w < WK; ++w) {
                    const uint32_t x[4] = {raw[w].x, raw[w].y, raw[w].z, raw[w].w};
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        top = max(top, max((x[e] >> 16) & 0x7FFFu, x[e] & 0x7FFFu));
                }
                top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
                top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
                const int ex = static_cast<int>(top >> 7);
                const int e = top == 0 || ex == 255 ? 0 : max(ex, 1) - 127;
                const float down = ldexpf(1.0f, -e);
                float sum = 0.0f;   // of q * 2^-e
#pragma unroll
                for (int w = 0; w < WK; ++w) {
                    const uint32_t x[4] = {raw[w].x, raw[w].y, raw[w].z, raw[w].w};
                    float y[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        y[k] = __uint_as_float(k & 1 ? x[k / 2] & 0xFFFF0000u : x[k / 2] << 16) * down;
                        sum += y[k];
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float f = k & 1 ? 0x1p10f : 0x1p14f;
                        qb[2 * w + (k >> 1)][t][k & 1] = pack_f16(y[k] * f, y[k + 4] * f);
                    }
                }
                sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
                sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 2);
                float f = ldexpf(a.sm_scale, e);
                f = a.cap > 0.0f ? f / a.cap * (2.0f * kLog2e) : f * kLog2e;
#pragma unroll
                for (int y = 0; y < 2; ++y) {   // of the rows 2c, 2c + 1
                    qs[t][y] = __shfl_sync(0xFFFFFFFFu, f, c * 8 + y * 4);
                    qm[t][y] = __shfl_sync(0xFFFFFFFFu, f * sum, c * 8 + y * 4);
                    m[t][y] = kLowest;
                    if (MULTI) {
                        const int token = (t * 8 + 2 * c + y) / a.group;
                        sees[t][y] = t * 8 + 2 * c + y < rows ? seq_len(a, b + token) : 0;
                    }
                }
                l2[t] = ln2[t] = F2(0.0f, 0.0f);
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
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
        __syncwarp();   // the other lanes' copies too
        uint32_t xk[kSub][2][WK];
        float ks[kSub][2], km[kSub][2], vs[kSub][2], vm[kSub][2];   // of the keys g, g + 8
#pragma unroll
        for (int u = 0; u < kSub; ++u) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int key = u * 16 + x * 8 + swap_g;
                if (D == 128) {
                    const uint4 w = lds128(at + key * (D / 2) + (c ^ (swap_g & 2)) * 16);
                    xk[u][x][0] = w.x, xk[u][x][1] = w.y, xk[u][x][WK - 2] = w.z, xk[u][x][WK - 1] = w.w;
                } else {
                    const uint2 w = lds64(at + key * (D / 2) + c * 8);
                    xk[u][x][0] = w.x, xk[u][x][1] = w.y;
                }
                const uint32_t pk = __float_as_uint(lds32(at + 2 * S::kCodes + key * 4));
                const uint32_t pv = __float_as_uint(lds32(at + 2 * S::kCodes + (kUnit + key) * 4));
                ks[u][x] = __uint_as_float(pk << 16), km[u][x] = __uint_as_float(pk & 0xFFFF0000u);
                vs[u][x] = __uint_as_float(pv << 16), vm[u][x] = __uint_as_float(pv & 0xFFFF0000u);
            }
        }
        if (live < kUnit) {   // what lies behind the last key may be no number
#pragma unroll
            for (int u = 0; u < kSub; ++u)
#pragma unroll
                for (int x = 0; x < 2; ++x)
                    if (u * 16 + x * 8 + swap_g >= live)
                        ks[u][x] = km[u][x] = vs[u][x] = vm[u][x] = 0.0f;
        }

        // ---- S^T = K Q^T: s[u][t][2 x + y] is key g + 8 x, row 8 t + 2c + y
        float s[kSub][NT][4];
#pragma unroll
        for (int u = 0; u < kSub; ++u) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    s[u][t][k] = 0.0f;
#pragma unroll
            for (int w = 0; w < WK; ++w)
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const uint32_t w0 = half ? xk[u][0][w] >> 8 : xk[u][0][w], w1 = half ? xk[u][1][w] >> 8 : xk[u][1][w];
#pragma unroll
                    for (int t = 0; t < NT; ++t)
                        mma_f16(s[u][t], w0 & 0x000F000Fu, w1 & 0x000F000Fu, w0 & 0x00F000F0u, w1 & 0x00F000F0u,
                                qb[2 * w + half][t][0], qb[2 * w + half][t][1]);
                }
        }
        // ---- scores in log2 units (cap * tanh(y) = cap * (1 - 2 / (1 + e^{2y})), qs
        // and qm holding 2 log2(e) / cap); keys past the end are -inf. The product
        // is 2^-10 of q 2^-e . c.
#pragma unroll
        for (int u = 0; u < kSub; ++u)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int x = 0; x < 2; ++x) {   // (rows in pairs: one instruction for both)
                    const F2 qc = mul2(mul2(F2(s[u][t][2 * x], s[u][t][2 * x + 1]), F2(1024.0f, 1024.0f)),
                                       F2(qs[t][0], qs[t][1]));
                    const F2 y = fma2(qc, F2(ks[u][x], ks[u][x]), mul2(F2(km[u][x], km[u][x]), F2(qm[t][0], qm[t][1])));
                    s[u][t][2 * x] = y.lo(), s[u][t][2 * x + 1] = y.hi();
                }
        if (a.cap > 0.0f) {
#pragma unroll
            for (int u = 0; u < kSub; ++u)
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        s[u][t][k] = fmaf(-2.0f * kLog2e * a.cap, rcp(1.0f + ex2(s[u][t][k])), kLog2e * a.cap);
        }
        if (live_last & 512) {
            const int key0 = descs[i % kDescs].key0;
#pragma unroll
            for (int u = 0; u < kSub; ++u)
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        s[u][t][k] = u * 16 + (k >> 1) * 8 + swap_g < (MULTI ? sees[t][k & 1] - key0 : live) ? s[u][t][k]
                                                                                                         : -INFINITY;
        }
        // ---- weights under the reference as it stands; where one, times the size of
        // its value, would come near f16's end the reference is raised and they are
        // taken again. (The size: the larger of the step and the least value, so that
        // neither product of the weight leaves the range.)
        float p[kSub][NT][4];
        auto size = [&](int u, int x) { return fmaxf(fabsf(vs[u][x]), fabsf(vm[u][x])); };
        auto weigh = [&]() {
            float top = 0.0f;
#pragma unroll
            for (int u = 0; u < kSub; ++u)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const float z = fmaxf(size(u, x), kLeastScale);
                    float most = 0.0f;
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        const F2 y = add2(F2(s[u][t][2 * x], s[u][t][2 * x + 1]), F2(-m[t][0], -m[t][1]));
                        p[u][t][2 * x] = ex2(y.lo());
                        p[u][t][2 * x + 1] = ex2(y.hi());
                        most = fmaxf(most, fmaxf(p[u][t][2 * x], p[u][t][2 * x + 1]));
                    }
                    top = fmaxf(top, most * z);
                }
            return top;
        };
        if (__any_sync(0xFFFFFFFFu, weigh() > kMostWeight)) {
            float lift[kSub][2];   // log2 of the values' sizes
#pragma unroll
            for (int u = 0; u < kSub; ++u)
#pragma unroll
                for (int x = 0; x < 2; ++x)
                    lift[u][x] = fmaxf(log2f(size(u, x)), kLeastScaleLog2);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                float f[2];
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    float top = -INFINITY;
#pragma unroll
                    for (int u = 0; u < kSub; ++u)
                        top = fmaxf(top, fmaxf(s[u][t][y] + lift[u][0], s[u][t][2 + y] + lift[u][1]));
#pragma unroll
                    for (int x = 4; x < 32; x <<= 1)
                        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, x));
                    const float to = fmaxf(m[t][y], reference(top));
                    f[y] = ex2(m[t][y] - to);
                    m[t][y] = to;
#pragma unroll
                    for (int j = 0; j < KS; ++j) {
                        o[j][t][y] *= f[y];
                        o[j][t][2 + y] *= f[y];
                    }
                }
                l2[t] = mul2(l2[t], F2(f[0], f[1]));
                ln2[t] = mul2(ln2[t], F2(f[0], f[1]));
            }
            weigh();
        }
        // ---- the values' codes, only now: registers that hold them while the scores
        // are made are missing there (180 us with them before, 166 us so, 64 sequences
        // of 8192-16384 keys); and the slot to the next copy
        uint32_t xv[kSub][4][WV];
#pragma unroll
        for (int u = 0; u < kSub; ++u) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int key = u * 16 + (k >> 1) * 8 + c * 2 + ((k & 1) ^ swap_c);
                if (D == 128) {
                    const uint2 w = lds64(at + S::kCodes + key * (D / 2) + (g * 8 ^ (c & 1) * 32));
                    xv[u][k][0] = w.x, xv[u][k][WV - 1] = w.y;
                } else {
                    xv[u][k][0] = __float_as_uint(lds32(at + S::kCodes + key * (D / 2) + g * 4));
                }
            }
        }
        __syncwarp();
        issue(i + kStages);

        // ---- P^T and O^T += V^T P^T. A weight times its value's step is rounded to f16
        // (2^-11; a second operand for the rest would double these matrix products, and the
        // outputs' error against 64 bits, most of it bf16's own rounding, is 5-11 % larger
        // for it); the sum of the weights and their products with least values stay in fp32.
#pragma unroll
        for (int u = 0; u < kSub; ++u) {
            uint32_t pb[NT][2];
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const F2 weight(p[u][t][2 * x], p[u][t][2 * x + 1]);
                    F2 scaled = mul2(weight, F2(vs[u][x], vs[u][x]));
                    F2 least = fma2(weight, F2(vm[u][x], vm[u][x]), ln2[t]);
                    if (MULTI && (live_last & 512)) {   // what a row does not see may be no number
                        const bool y0 = s[u][t][2 * x] != -INFINITY, y1 = s[u][t][2 * x + 1] != -INFINITY;
                        scaled = F2(y0 ? scaled.lo() : 0.0f, y1 ? scaled.hi() : 0.0f);
                        least = F2(y0 ? least.lo() : ln2[t].lo(), y1 ? least.hi() : ln2[t].hi());
                    }
                    l2[t] = add2(l2[t], weight);
                    ln2[t] = least;
                    pb[t][x] = transpose8(pack_f16(scaled.lo(), scaled.hi()));
                }
#pragma unroll
            for (int w = 0; w < WV; ++w)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const uint32_t sel = q < 2 ? 0x5410u : 0x7632u;
                    uint32_t x0 = prmt(xv[u][0][w], xv[u][1][w], sel), x1 = prmt(xv[u][2][w], xv[u][3][w], sel);
                    if (q & 1)
                        x0 >>= 8, x1 >>= 8;
#pragma unroll
                    for (int t = 0; t < NT; ++t)
                        mma_f16(o[4 * w + q][t], x0 & 0x000F000Fu, x0 & 0x00F000F0u, x1 & 0x000F000Fu, x1 & 0x00F000F0u,
                                pb[t][0], pb[t][1]);
                }
        }

        // ---- the piece ends with its pair or with the warp's units
        if ((live_last & 256) || i + 1 == units) {
            const int64_t slot = static_cast<int64_t>(pair) + me;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                float l[2] = {l2[t].lo(), l2[t].hi()}, ln[2] = {ln2[t].lo(), ln2[t].hi()};
#pragma unroll
                for (int y = 0; y < 2; ++y) {
#pragma unroll
                    for (int x = 4; x < 32; x <<= 1) {
                        l[y] += __shfl_xor_sync(0xFFFFFFFFu, l[y], x);
                        ln[y] += __shfl_xor_sync(0xFFFFFFFFu, ln[y], x);
                    }
                    if (g == 0 && t * 8 + c * 2 + y < rows)
                        a.part_ml[slot * R + t * 8 + c * 2 + y] = make_float2(m[t][y], l[y]);
                }
                float* dst = a.part_o + (slot * R + t * 8 + c * 2) * D + g * (D / 8);
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    if (t * 8 + c * 2 + e < rows) {
#pragma unroll
                        for (int j = 0; j < KS; j += 2)   // values 2j and 2j + 1 of the chunk: rows g and g + 8
                            *reinterpret_cast<float4*>(dst + e * D + 2 * j) =
                                make_float4(fmaf(o[j][t][e], 0x1p24f, ln[e]), fmaf(o[j][t][2 + e], 0x1p20f, ln[e]),
                                            fmaf(o[j + 1][t][e], 0x1p24f, ln[e]),
                                            fmaf(o[j + 1][t][2 + e], 0x1p20f, ln[e]));
                    }
            }
            fresh = true;
        }
    }
}

static int ring_smem(int D, int B) { return kWarps * (D == 128 ? Ring<128>::total : Ring<64>::total) + (B + 1) * 4; }

template <int D, int NT, bool MULTI, int PER_SM>
static cudaError_t launch_pieces(const Kv4Attn& a, cudaStream_t s)
{
    const int smem = ring_smem(D, a.B);
    auto kern = kv4_attn_kernel<D, NT, MULTI, PER_SM>;
    // More than 48 KB, with what the kernel holds besides, have to be asked for: always
    // the most that a call can need, as another thread's call may be between here and its launch.
    if (smem > 47 * 1024) {
        const cudaError_t e =
            cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, ring_smem(D, kKv8MaxBatch));
        if (e != cudaSuccess)
            return e;
    }
    return launch_dependent(kern, dim3(a.warps / kWarps), dim3(kWarps * 32), smem, s, a);
}
// Tokens of a sequence that share a tile: as many as 8 rows hold, where the sequences
// are given apart (`seqs`); the codes of a unit are taken apart once for all of them.
// (16 sequences of 2000-4000 keys, 5 tokens each, us with a tile for each token / so:
// 32 query and 8 kv heads 60 / 48, 8 and 8 56 / 27. Two tokens of a larger group in 16
// rows would not pay: 16 rows cost 1.74 times what 8 do, as they leave room for half
// the warps; 48 query and 8 kv heads 58.9 / 57.5 with that, and it would be slower for
// an odd number of tokens.)
cudaError_t launch_kv4_attn(const Kv4Attn& in, int D, int num_sms, cudaStream_t s)
{
    Kv4Attn a = in;
    const int R = kv8_attn_row_tile(a.group);
    a.tiles = (a.group + R - 1) / R;
    a.per_tile = a.seqs && a.max_pages ? max(8 / a.group, 1) : 1;
    if (a.per_tile == 1)
        a.lead = nullptr;
    a.unit_shift = kUnitShift;
    const int64_t pairs = static_cast<int64_t>(a.Hkv) * a.B * a.tiles;
    // CTAs an SM holds: by registers, by shared memory (128 bytes of static arrays, 1 KB of
    // the system's, steps of 128)
    const int fit = 228 * 1024 / ((ring_smem(D, a.B) + 127) / 128 * 128 + 128 + 1024);
    // 16 rows of D 64 by two blocks until the tables allow 105 units an SM (16000 here). 16
    // query and 1 kv heads, us at two / three: 24 sequences of up to 5001 keys with 4 drafts
    // each, 15000 units, 21.6 / 23.6; 96 of 1000-3000, 9000, 17.6 / 18.3; 8 of 16000, 4000,
    // 13.8 / 15.1; 64 of 8000, 16000, 24.1 / 23.5; 128 of 4000, 16000, 24.7 / 23.6; 256 of
    // 4000, 32000, 37.5 / 35.2. Only the device knows the lengths: where all are as long as
    // the table three would win from 12000 on (48 of 8000 21.2 / 19.8), where the tables are
    // much wider than the lengths two would longer (128 of 0-5000, 20000 units, 21.6 / 21.9).
    const int64_t units = pairs * ((static_cast<int64_t>(a.max_pages) << a.page_shift) >> kUnitShift);
    const int blocks = min(R == 8 ? 4 : D == 64 && units >= 105 * static_cast<int64_t>(num_sms) ? 3 : 2, fit);
    a.warps = min(num_sms * blocks * kWarps, kKv8MaxWarps / kWarps * kWarps);
    a.free_warps = a.warps;
    // Shares by place where four blocks fit an SM (two or three, of 16 rows, gain nothing).
    // us with equal shares / proportions of 170:140:118:100 / 200:160:130:100 /
    // 250:190:140:100: 64 sequences of 8192-16384 keys of D 128 153 / 146 / 143 / 148, 256
    // of 500-1000 55.9 / 54.4 / 54.1 / 55.7, 32 of 4096-8192 of D 64 35.9 / 34.7 / 35.5 / 36.8.
    const int weights[2][4] = {{170, 140, 118, 100}, {200, 160, 130, 100}};
    a.places = blocks == 4 && a.warps == num_sms * blocks * kWarps ? blocks : 1;
    for (int i = 0; i < 4; ++i)
        a.place_weight[i] = weights[D == 128][i];
    // By twos up to 128 pieces a pair (8 sequences of 16000 keys, 16 query and 1 kv heads, 18.9
    // us without that bound / 17.1) and 1536 warps (32 of 500-1000, 48 and 8 heads, 1536 /
    // 2048 / all: 16.9 / 18.0 / 18.6; 128 of 30-90, 1024 / 1536: 15.9 / 13.8).
    a.spread = static_cast<int>(min(int64_t{1536}, 128 * pairs));
    cudaError_t e = cudaSuccess;
    if (a.max_pages)
        e = R == 16            ? (D == 128 ? launch_pieces<128, 2, false, 2>(a, s) : launch_pieces<64, 2, false, 3>(a, s))
            : a.per_tile == 1 ? (D == 128 ? launch_pieces<128, 1, false, 4>(a, s) : launch_pieces<64, 1, false, 4>(a, s))
                              : (D == 128 ? launch_pieces<128, 1, true, 4>(a, s) : launch_pieces<64, 1, true, 4>(a, s));
    if (e != cudaSuccess)
        return e;
    return launch_kv_join(a, Kv8Prefix{}, R, D, num_sms, s);
}

}  // namespace w4a8
