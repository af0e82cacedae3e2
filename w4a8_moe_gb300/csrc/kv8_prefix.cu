// Attention of a whole batch over its shared prefix: one pass of tensor-core
// matrix products over the prefix's pages for all sequences at once.
//
// "ROCm: enable trillion-parameter MoE models with INT4-FP8 single node",
// config.json (kv_cache_scheme FP8; 48 query and 8 key/value heads).
//
// For kv head h the rows are all (sequence, query head of h's group), R of
// them, and S = Q K^T, O = P V are [R, keys] and [R, D] matrix products. A CTA
// takes 256 rows (two 128-row tiles) and a range of 128-key tiles and runs,
// with S, P and O in tensor memory:
//   loader    warp 12: pages -> raw codes in shared memory (bulk copies)
//   converter warps 8-11, 14, 15: E4M3 -> f16 (exact), into the layouts the MMA reads
//   issuer    warp 13: S_t = Q_t K^T, O_t += P_t V, alternating the row tiles
//   softmax   warps 0-3 (tile 0), 4-7 (tile 1): one thread per row
// While one tile's softmax runs, the tensor core works for the other tile.
// Bound by a row tile's chain (maximum, exponentials, the second half of P V, the
// next Q K^T: some 2700 cycles a key tile against the two row tiles' 2048 of MMA).
// 256 sequences of 48 heads over 65536 tokens: 248 us on 144 SMs, 1.66 PFLOP/s;
// one key tile a CTA: 5.5 us with start and end.
//
// Numbers: q is normalized per row by a power of two and held in f16 (at most
// 2^-25 of the row's largest element is lost, one fp32 rounding), codes are
// exact in f16, S and O are fp32, P is rounded to f16 (2^-11 of each weight and
// 2^-33 of the largest, see kWeightTop), its sum is taken in fp32 before that
// rounding.
#include <math.h>

#include "internal.h"
#include "kv8.cuh"
#include "ptx.cuh"

namespace w4a8 {

namespace {

constexpr int kThreads = 512;
constexpr int kTile = 128;        // keys per tile, rows per row tile
constexpr int kHalf = 64;         // keys per raw slot
constexpr int kStages = 3;        // f16 operand tiles, K and V in turn
constexpr int kPairs = 3;         // pairs of converter warps
constexpr int kRaw = 6;           // raw slots
// A parity wait cannot tell a phase from the one two before it, and copies land
// out of order: whoever waits on a slot has to have seen each of its rounds, so
// a slot belongs to one pair. (Seven slots, visited by the pairs in turn, let a
// pair that was ahead take a slot's last round for its next: wrong values in one
// call of some hundred.)
static_assert(kRaw % kPairs == 0, "a raw slot has one pair of readers");
constexpr int kScaleRing = 4;     // tiles whose per-token scales are held
// A tile whose value scales lie within this factor takes its largest score and its
// largest scale for its largest product: at most this factor too much. Others look
// at every key (careful_tile).
constexpr float kNear = 64.0f;
// References (log2) up to which a tile goes the short way: there a weight's exponent
// is a fused product and difference, off from the rounded score that the reference
// was taken from by 2^-4 at most, and stays far inside f16. (A product and a
// difference of pairs, each with its own rounding, are fused by the compiler too:
// the other way takes single ones.)
constexpr float kFused = 0x1p20f;

template <int D>
struct Smem {
    static constexpr int kOperand = kTile * D * 2;          // one f16 operand tile
    static constexpr int kPanel = kTile * 128;              // 64 f16 columns of it
    static constexpr int q = 0;                             // [2] row tiles
    static constexpr int stage = q + 2 * kOperand;          // [kStages]: K_0, V_0, K_1, ...
    static constexpr int raw = stage + kStages * kOperand;  // [kRaw] of 64 x D codes
    static constexpr int scales = raw + kRaw * kHalf * D;   // [kScaleRing][2][128] fp32
    static constexpr int bars = scales + kScaleRing * 2 * kTile * 4;
    static constexpr int total = bars + 320;
};
// mbarriers, 8 bytes each
enum Bar {
    kRawFull = 0,                    // [kRaw]
    kRawEmpty = kRawFull + kRaw,     // [kRaw]
    kFull = kRawEmpty + kRaw,        // [kStages]
    kEmpty = kFull + kStages,        // [kStages]
    kSFull = kEmpty + kStages,       // [2] row tiles
    kPFull = kSFull + 2,             // [2]
    kPHalf = kPFull + 2,             // [2]
    kOFull = kPHalf + 2,             // [2]
    kScFull = kOFull + 2,            // [kScaleRing]
    kQFull = kScFull + kScaleRing,   // [2]
    kBars = kQFull + 2
};
static_assert(kBars * 8 + 8 <= 320, "barrier area");

// MMA, f16 operands, fp32 accumulators; B K-major or MN-major.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool b_mn)
{
    return (1u << 4) | (b_mn ? 1u << 16 : 0u) | (static_cast<uint32_t>(N >> 3) << 17) |
           (static_cast<uint32_t>(M >> 4) << 24);
}
// One thread issues an MMA of 64 cycles at a time, so what it does in between
// has to be short: descriptors are a constant high word and a low word that
// advances by constants, and whether D is added to is a constant.
__device__ __forceinline__ uint32_t elect_one()
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r;
}
template <bool kAcc>
__device__ __forceinline__ void mma_ss(uint32_t leader, uint32_t d, uint32_t alo, uint32_t ahi, uint32_t blo, uint32_t bhi,
                                       uint32_t idesc)
{
    if (leader)
        asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tmov.b64 a, {%1, %2};\n\tmov.b64 b, {%3, %4};\n\t"
                     "setp.ne.b32 p, %6, 0;\n\t"
                     "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, p;\n\t}" ::"r"(d), "r"(alo), "r"(ahi), "r"(blo),
                     "r"(bhi), "r"(idesc), "n"(kAcc ? 1 : 0)
                     : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t leader, uint32_t d, uint32_t a, uint32_t blo, uint32_t bhi,
                                       uint32_t idesc, uint32_t acc)
{
    if (leader)
        asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tmov.b64 b, {%2, %3};\n\tsetp.ne.b32 p, %5, 0;\n\t"
                     "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d), "r"(a), "r"(blo), "r"(bhi),
                     "r"(idesc), "r"(acc)
                     : "memory");
}
__device__ __forceinline__ void commit(uint32_t leader, uint32_t bar)
{
    if (leader)
        umma_commit(bar);
}
// Operands in the 128-byte swizzle: panels of 64 values (128 bytes) by all
// rows, 8-row groups 1024 bytes apart. Contracted axis contiguous (Q, K): the
// start advances 32 bytes per MMA inside a panel. Other axis contiguous (V):
// panels are kPanel apart, the start advances by 16 keys, 2048 bytes.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);   // group stride, version, swizzle
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t panel) { return (saddr >> 4) | ((panel >> 4) << 16); }
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(taddr));
}
__device__ __forceinline__ void ld_wait16(uint32_t (&r)[16])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :
                 : "memory");
}
// Wait for this warp's tensor-memory loads; the registers they fill pass
// through, so that no use of them can be moved ahead of the wait.
__device__ __forceinline__ void ld_wait32(uint32_t (&r)[32])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                   "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]),
                   "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                   "+r"(r[30]), "+r"(r[31])
                 :
                 : "memory");
}
__device__ __forceinline__ void sts128(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, uint32_t bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.wait_all;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void regs_inc()
{
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec()
{
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
__device__ __forceinline__ float max3(float a, float b, float c)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
template <bool B>
struct Const {
    static constexpr bool value = B;
};

}  // namespace

template <int D, bool TOK, bool CAP>
__global__ void __launch_bounds__(kThreads, 1) kv8_prefix_kernel(const __grid_constant__ Kv8Attn a,
                                                                 const __grid_constant__ Kv8Prefix pl)
{
    using L = Smem<D>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t bars = base + L::bars;
    auto bar = [&](int i) { return bars + 8u * i; };
    __shared__ int abort_flag;
    __shared__ uint32_t tmem_base;
    const volatile int* abort = &abort_flag;

    // the shuffles make warp-uniform what the issuer's instructions take from uniform registers
    const int tid = threadIdx.x, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0), lane = tid & 31;
    // CTA -> (split, row pair, head); neighbours share the head's keys
    const int rp = blockIdx.x % pl.row_pairs;
    const int h = (blockIdx.x / pl.row_pairs) % a.Hkv;
    const int split = blockIdx.x / (pl.row_pairs * a.Hkv);
    const int tile0 = split * pl.tiles_per_split;
    const int n = min(pl.tiles - tile0, pl.tiles_per_split);
    const int rows_all = a.B * a.group;
    const int row0 = rp * 2 * kTile;
    const int nt = rows_all - row0 > kTile ? 2 : 1;

    if (tid < kBars) {
        uint32_t count = 1;
        if (tid >= kRawEmpty && tid < kFull)
            count = 2;          // a pair of converter warps
        else if (tid >= kFull && tid < kEmpty)
            count = 4;          // two pairs, a half each
        else if ((tid >= kPFull && tid < kOFull) || tid >= kQFull)
            count = 4;          // a tile's softmax warps
        mbar_init(bar(tid), count);
        fence_mbar_init();
    }
    if (tid == 0)
        abort_flag = 0;
    if (warp == 13)
        tmem_alloc(smem_u32(&tmem_base), 512);
    __syncthreads();
    grid_dep_wait();
    grid_dep_launch();   // the kernel after this one needs nothing of it before its own end
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, tmem_base, 0);
    auto fail = [&]() {
        set_error(a.err, kErrBitTimeout);
        *const_cast<volatile int*>(&abort_flag) = 1;
    };
    auto wait = [&](int i, uint32_t parity) {
        if ((warp < 8 || warp == 13) ? mbar_wait_or_abort<0>(bar(i), parity, abort) : mbar_wait_or_abort<1000>(bar(i), parity, abort))
            return true;
        fail();
        return false;
    };
    auto wait_warp = [&](int i, uint32_t parity) { return __all_sync(0xFFFFFFFFu, wait(i, parity)) != 0; };

    // 512 threads start with 128 registers each; a softmax thread holds a row of 128 scores
    if (warp < 8)
        regs_inc<192>();
    else
        regs_dec<64>();

    if (warp < 8) {
        const int t = warp >> 2;       // row tile
        const int my_row = row0 + t * kTile + (tid & 127);
        const uint32_t staged = base + L::stage + L::kOperand + (tid & 255) * D * 2;
        float ks_head = 1.0f, vs_head = 1.0f;
        if (t < nt) {
            // -------------------------------------------------------- queries
            // A warp copies its 32 rows, whole rows at a time, to where V_0 and K_1
            // will stand.
            {
                constexpr int kLanes = D / 8, kPer = 32 / kLanes;
                const int sub = lane / kLanes, chunk = lane % kLanes;
                int row = my_row - lane + sub;
                int b = row / a.group, g = row - b * a.group;
#pragma unroll 4
                for (int i = 0; i < 32; i += kPer) {
                    const uint16_t* src = a.q + b * a.q_stride + static_cast<int64_t>(h * a.group + g) * D + chunk * 8;
                    const bool there = row < rows_all;   // else zeros
                    copy16(staged + (i + sub - lane) * D * 2 + chunk * 16, there ? src : a.q, there ? 16 : 0);
                    row += kPer;
                    for (g += kPer; g >= a.group; g -= a.group)
                        ++b;
                }
                if (!TOK) {
                    ks_head = __ldg(a.k_scale + h);
                    vs_head = __ldg(a.v_scale + h);
                }
            }
            // A thread finds its row's exponent and writes the row as an operand.
            // Row r takes its 16-byte chunks in the order i ^ x r, with x r a
            // product in GF(8): both x r and x r + r then pass through all of
            // 0..7, so neither the reads (rows a whole number of banks apart)
            // nor the writes (at chunk ^ r) of eight rows collide.
            copies_done();
            __syncwarp();
            const int r = tid & 127;
            const int turn = ((r << 1) & 4) | (((r ^ (r >> 2)) & 1) << 1) | ((r >> 2) & 1);
            bool ok = true;
            uint4 w[D / 8];
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
                w[i] = lds128(staged + (i ^ turn) * 16);
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {   // the larger magnitude of each half, side by side
                constexpr uint32_t mags = 0x7FFF7FFFu;
                top = __vmaxu2(top, __vmaxu2(__vmaxu2(w[i].x & mags, w[i].y & mags), __vmaxu2(w[i].z & mags, w[i].w & mags)));
            }
            top = max(top >> 16, top & 0xFFFFu);
            const int ex = static_cast<int>(top >> 7);
            const int e = top == 0 || ex == 255 ? 0 : min(max(ex, 1), 253) - 127;
            // a negative factor goes into q, so that the largest product is the largest score
            const float down = ((a.sm_scale < 0.0f) != (ks_head < 0.0f) ? -1.0f : 1.0f) * __int_as_float((127 - e) << 23);
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                const int chunk = i ^ turn;
                const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
                uint32_t f[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    f[j] = pack_f16(__uint_as_float(u[j] << 16) * down, __uint_as_float(u[j] & 0xFFFF0000u) * down);
                sts128(base + L::q + t * L::kOperand + (chunk >> 3) * L::kPanel + r * 128 +
                           (((chunk & 7) ^ (r & 7)) << 4),
                       f[0], f[1], f[2], f[3]);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(bar(kQFull + t));
            const float capl = a.cap * kLog2e;
            float c = fabsf(a.sm_scale * __int_as_float((127 + e) << 23) * ks_head);   // score = c * product
            c = CAP ? c / a.cap * (2.0f * kLog2e) : c * kLog2e;

            // -------------------------------------------------------- softmax
            const uint32_t ts = tmem + (static_cast<uint32_t>(warp & 3) << 21) + t * kTile;         // S, then P
            const uint32_t to = tmem + (static_cast<uint32_t>(warp & 3) << 21) + 2 * kTile + t * D;  // O
            float m = -INFINITY;
            bool enormous = false;   // whether a row of the warp has such a reference
            F2 l0(0.0f, 0.0f), l1(0.0f, 0.0f);
            const float* scales = reinterpret_cast<const float*>(smem_raw + (base - smem_u32(smem_raw)) + L::scales);
            // What a tile does to the row, scores in units of c:
            // the reference raised where the largest weight asks for it (kWeightMost;
            // the whole warp goes through its accumulators together),
            auto raise = [&](int i, float best) {
                const float next = fmaxf(m, reference(best));
                const float f = next == -INFINITY ? 1.0f : ex2(m - next);
                m = next;
                enormous = __any_sync(0xFFFFFFFFu, m > -INFINITY && fabsf(m) > kFused);
                l0 = mul2(l0, F2(f, f));
                l1 = mul2(l1, F2(f, f));
                if (i > 0) {
#pragma unroll 1
                    for (int ch = 0; ch < D / 16; ++ch) {
                        uint32_t x[16];
                        tmem_ld16(to + ch * 16, x);
                        ld_wait16(x);
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            x[j] = __float_as_uint(__uint_as_float(x[j]) * f);
                        tmem_st16(to + ch * 16, x);
                    }
                }
            };
            // the largest score in log2 units: cap * tanh(y) = cap * (1 - 2 / (1 + e^{2y})),
            // c holding 2 log2(e) / cap
            auto in_log2 = [&](float top) {
                const float x = __fmul_rn(top, c);   // what weigh() takes, where it does not fuse
                return CAP ? fmaf(-2.0f * capl, rcp(1.0f + ex2(x)), capl) : x;
            };
            // 32 keys' scores times their key scales,
            auto times_scales = [&](uint32_t (&r)[32], const float* f) {
#pragma unroll
                for (int j = 0; j < 32; j += 4) {
                    const float4 k4 = *reinterpret_cast<const float4*>(f + j);
                    const F2 x = mul2(F2(__uint_as_float(r[j]), __uint_as_float(r[j + 1])), F2(k4.x, k4.y));
                    const F2 y = mul2(F2(__uint_as_float(r[j + 2]), __uint_as_float(r[j + 3])), F2(k4.z, k4.w));
                    r[j] = __float_as_uint(x.lo()), r[j + 1] = __float_as_uint(x.hi());
                    r[j + 2] = __float_as_uint(y.lo()), r[j + 3] = __float_as_uint(y.hi());
                }
            };
            // their maximum,
            auto largest = [&](const uint32_t (&r)[32]) {
                float top = fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
#pragma unroll
                for (int j = 2; j < 32; j += 2)
                    top = max3(top, __uint_as_float(r[j]), __uint_as_float(r[j + 1]));
                return top;
            };
            // and their weights as f16, added up on the way. kCareful: of the first
            // `live` keys, the score rounded like the reference's before their
            // difference is taken. value_scales(j): of keys j to j + 3.
            auto weigh = [&](const uint32_t (&r)[32], auto value_scales, int ch, int live, auto careful) {
                constexpr bool kCareful = decltype(careful)::value;
                const float ref = m == -INFINITY ? 0.0f : m;
                const F2 c2(c, c), add(CAP ? capl - ref : -ref, CAP ? capl - ref : -ref);
                const F2 one(1.0f, 1.0f), two(-2.0f * capl, -2.0f * capl), zero(-0.0f, -0.0f);
                uint32_t p[16];
#pragma unroll
                for (int j = 0; j < 32; j += 4) {
                    float4 v4;
                    if (TOK)
                        v4 = value_scales(j);
#pragma unroll
                    for (int e = 0; e < 4; e += 2) {
                        const F2 s(__uint_as_float(r[j + e]), __uint_as_float(r[j + e + 1]));
                        F2 x = fma2(s, c2, CAP ? zero : add);
                        if (kCareful) {
                            x = F2(__fadd_rn(in_log2(s.lo()), -ref), __fadd_rn(in_log2(s.hi()), -ref));
                        } else if (CAP) {
                            x = add2(F2(ex2(x.lo()), ex2(x.hi())), one);
                            x = fma2(F2(rcp(x.lo()), rcp(x.hi())), two, add);
                        }
                        float w0 = ex2(x.lo()), w1 = ex2(x.hi());
                        if (kCareful) {
                            w0 = j + e < live ? w0 : 0.0f;
                            w1 = j + e + 1 < live ? w1 : 0.0f;
                        }
                        F2 w(w0, w1);
                        if (e == 0)
                            l0 = add2(l0, w);
                        else
                            l1 = add2(l1, w);
                        if (TOK)
                            w = mul2(w, e == 0 ? F2(v4.x, v4.y) : F2(v4.z, v4.w));
                        p[(j + e) >> 1] = pack_f16(w.lo(), w.hi());
                    }
                }
                tmem_st16(ts + ch * 16, p);
                if (ch & 1) {   // O can take half of the keys
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(bar((ch == 1 ? kPHalf : kPFull) + t));
                }
            };
            // A key tile: the whole row of scores in registers, `lift` the log2 of
            // the largest value scale. Nothing but the raised reference where that is
            // enormous.
            auto tile = [&](int i, float lift) {
                const float* ks = scales + (i % kScaleRing) * 2 * kTile;
                const float* vs = ks + kTile;
                if (!wait_warp(kSFull + t, i & 1))
                    return false;
                tc_fence_after();
                uint32_t r[4][32];
#pragma unroll
                for (int ch = 0; ch < 4; ++ch)
                    tmem_ld32(ts + ch * 32, r[ch]);
                float top[4];
#pragma unroll
                for (int ch = 0; ch < 4; ++ch) {
                    ld_wait32(r[ch]);
                    if (TOK)
                        times_scales(r[ch], ks + ch * 32);
                    top[ch] = largest(r[ch]);
                }
                const float best = in_log2(fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]))) + lift;
                if (__any_sync(0xFFFFFFFFu, best > m + kWeightMost)) {
                    raise(i, best);
                    if (enormous)
                        return true;
                }
#pragma unroll
                for (int ch = 0; ch < 4; ++ch) {
                    auto value_scales = [&](int j) { return *reinterpret_cast<const float4*>(vs + ch * 32 + j); };
                    weigh(r[ch], value_scales, ch, kTile, Const<false>());
                }
                return true;
            };
            // The other way, for the prefix's last tile, where keys past its end are
            // masked, for tiles whose value scales lie far apart and for those under an
            // enormous reference: it reads S twice but is a quarter of the code. A
            // lane holds the value scales v[j] of the keys lane + 32 j (0 past the end).
            auto careful_tile = [&](int i, float (&v)[4]) {
                const float* ks = scales + (i % kScaleRing) * 2 * kTile;
                if (!wait_warp(kSFull + t, i & 1))
                    return false;
                tc_fence_after();
                const int live = a.prefix_len - (tile0 + i) * kTile;
                if (TOK) {
                    // Values of a key that are all zero add nothing, whatever their
                    // scale (kv8_write gives them 1): 0 then, so that they lead no
                    // reference. V stands in its stage until this tile's weights are
                    // given; its barrier's phase before this one was K's of the tile
                    // before, which S is behind.
                    const int jv = 2 * i + 1;
                    if (!wait_warp(kFull + jv % kStages, (jv / kStages) & 1))
                        return false;
                    const uint32_t at = base + L::stage + (jv % kStages) * L::kOperand + lane * 128;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint32_t any = 0;
#pragma unroll 4
                        for (int x = 0; x < D / 8; ++x) {   // 16 bytes each, another bank group a lane
                            const uint4 w = lds128(at + j * 32 * 128 + (x >> 3) * L::kPanel + (((x + lane) & 7) << 4));
                            any |= w.x | w.y | w.z | w.w;
                        }
                        v[j] = (any & 0x7FFF7FFFu) ? v[j] : 0.0f;
                    }
                }
                auto of_chunk = [&](const float (&x)[4], int ch) { return ch < 2 ? (ch ? x[1] : x[0]) : (ch == 2 ? x[2] : x[3]); };
                float top = -INFINITY;
#pragma unroll 1
                for (int ch = 0; ch < 4; ++ch) {
                    uint32_t r[32];
                    tmem_ld32(ts + ch * 32, r);
                    ld_wait32(r);
                    if (TOK) {
                        times_scales(r, ks + ch * 32);
                        const float mine = fmaxf(log2f(fabsf(of_chunk(v, ch))), kLeastScaleLog2);
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            const float y = in_log2(__uint_as_float(r[j])) + __shfl_sync(0xFFFFFFFFu, mine, j);
                            top = fmaxf(top, ch * 32 + j < live ? y : -INFINITY);
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            r[j] = ch * 32 + j < live ? r[j] : 0xFF800000u;
                        top = fmaxf(top, largest(r));
                    }
                }
                top = TOK ? top : in_log2(top);
                if (__any_sync(0xFFFFFFFFu, top > m + kWeightMost))
                    raise(i, top);
#pragma unroll 1
                for (int ch = 0; ch < 4; ++ch) {
                    uint32_t r[32];
                    tmem_ld32(ts + ch * 32, r);
                    ld_wait32(r);
                    if (TOK)
                        times_scales(r, ks + ch * 32);
                    const float mine = of_chunk(v, ch);
                    auto value_scales = [&](int j) {
                        return make_float4(__shfl_sync(0xFFFFFFFFu, mine, j), __shfl_sync(0xFFFFFFFFu, mine, j + 1),
                                           __shfl_sync(0xFFFFFFFFu, mine, j + 2), __shfl_sync(0xFFFFFFFFu, mine, j + 3));
                    };
                    weigh(r, value_scales, ch, live - ch * 32, Const<true>());
                }
                return true;
            };
            for (int i = 0; i < n && ok; ++i) {
                bool whole = (tile0 + i + 1) * kTile <= a.prefix_len;
                float lift = 0.0f, v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                if (TOK) {
                    const int live = a.prefix_len - (tile0 + i) * kTile;
                    ok = wait_warp(kScFull + i % kScaleRing, (i / kScaleRing) & 1);
                    if (!ok)
                        break;
                    // magnitudes compare like their bits; a NaN counts as the largest
                    const float* vs = scales + ((i % kScaleRing) * 2 + 1) * kTile;
                    uint32_t most = 0, least = 0xFFFFFFFFu;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        v[j] = lane + 32 * j < live ? vs[lane + 32 * j] : 0.0f;
                        most = max(most, __float_as_uint(fabsf(v[j])));
                        least = min(least, __float_as_uint(fabsf(v[j])));
                    }
                    const float hi = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, most));
                    whole = whole && __uint_as_float(__reduce_min_sync(0xFFFFFFFFu, least)) * kNear >= hi;
                    lift = fmaxf(log2f(hi), kLeastScaleLog2);
                }
                if (whole && !enormous)
                    ok = tile(i, lift);
                if (ok && (!whole || enormous))
                    ok = careful_tile(i, v);
            }
            // -------------------------------------------------------- results
            // Each thread lays its row of O in shared memory (the operands are
            // done with once both row tiles are), from where its warp writes whole
            // rows. (A bulk copy of each row instead: 3300 cycles for 256 of them,
            // against 2950.)
            for (int x = 0; x < nt && ok; ++x)
                ok = wait_warp(kOFull + x, 0);
            if (ok) {
                tc_fence_after();
                constexpr int kRow = D * 4 + 16;   // 16 bytes past whole banks
                const uint32_t mine = base + L::stage + (tid & 255) * kRow;
#pragma unroll 1
                for (int ch = 0; ch < D / 32; ++ch) {
                    uint32_t r[32];
                    tmem_ld32(to + ch * 32, r);
                    ld_wait32(r);
#pragma unroll
                    for (int j = 0; j < 32; j += 4)
                        sts128(mine + ch * 128 + j * 4, r[j], r[j + 1], r[j + 2], r[j + 3]);
                }
                const int64_t at = (static_cast<int64_t>(split) * a.Hkv + h) * rows_all + my_row;
                if (my_row < rows_all)
                    pl.part_ml[at] = make_float2(m, (l0.lo() + l0.hi()) + (l1.lo() + l1.hi()));
                __syncwarp();
                constexpr int kRowLanes = D / 4, kRows = 32 / kRowLanes;   // lanes of a row, rows of a store
                const int sub = lane / kRowLanes, part = lane % kRowLanes;
                float4* dst = reinterpret_cast<float4*>(pl.part_o + (at - lane + sub) * D) + part;
                const uint32_t from = base + L::stage + ((tid & 224) + sub) * kRow + part * 16;
                const int rows = min(32, rows_all - (my_row - lane)) - sub;
#pragma unroll 8
                for (int x = 0; x < 32; x += kRows) {
                    const uint4 v = lds128(from + x * kRow);
                    if (x < rows)
                        dst[x * (D / 4)] = make_float4(__uint_as_float(v.x) * vs_head, __uint_as_float(v.y) * vs_head,
                                                       __uint_as_float(v.z) * vs_head, __uint_as_float(v.w) * vs_head);
                }
                tc_fence_before();
            }
        }
    } else if (warp < 12 || warp >= 14) {
        // ---------------------------------------------------------- converter
        // Three pairs of warps take half tiles in turn, so that one
        // pair's latencies pass under the others' work. A thread turns 16 codes
        // into 32 bytes of f16; eight threads cover 64 bytes of an even row and
        // the other 64 of the odd row below, so that neither the loads nor the
        // swizzled stores collide in a bank.
        const int cw = warp < 12 ? warp - 8 : warp - 10;
        const int ct = (cw & 1) * 32 + lane;
        const int q4 = ct & 3, odd = (ct >> 2) & 1, pr = ct >> 3;   // 8 row pairs at a time
        bool ok = true;
        for (int s = cw >> 1; s < 4 * n && ok; s += kPairs) {
            const int j = s >> 1, half = s & 1, slot = s % kRaw, stage = j % kStages;   // j: K_0, V_0, K_1, ...
            ok = wait_warp(kRawFull + slot, (s / kRaw) & 1);
            if (s >= 2 && s < 2 + kPairs)   // until then the queries stand in the later stages
                for (int x = 0; x < nt && ok; ++x)
                    ok = wait_warp(kQFull + x, 0);
            if (ok && j >= kStages)
                ok = wait_warp(kEmpty + stage, (j / kStages - 1) & 1);
            if (!ok)
                break;
            const uint32_t src = base + L::raw + slot * kHalf * D;
            const uint32_t dst = base + L::stage + stage * L::kOperand;
            const int live = a.prefix_len - (tile0 + (s >> 2)) * kTile - half * kHalf;
            constexpr int kPasses = D / 64;      // 64-byte parts of a row
            constexpr int kWork = 4 * kPasses;   // 16-code chunks of a thread
#pragma unroll
            for (int x0 = 0; x0 < kWork; x0 += 4) {
                uint4 w[4];
                auto place = [&](int x, int& row, int& c16) {
                    row = (x / kPasses) * 16 + pr * 2 + odd;
                    c16 = D == 128 ? q4 + 4 * (odd ^ (x & 1)) : q4;
                };
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    int row, c16;
                    place(x0 + x, row, c16);
                    w[x] = lds128(src + row * D + c16 * 16);
                    if (row >= live)
                        w[x] = make_uint4(0, 0, 0, 0);
                }
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    int row, c16;
                    place(x0 + x, row, c16);
                    const int key = half * kHalf + row;
                    const uint32_t u[4] = {w[x].x, w[x].y, w[x].z, w[x].w};
                    uint32_t f[8];
#pragma unroll
                    for (int y = 0; y < 4; ++y)
                        e4m3x4_to_f16x4(u[y], f[2 * y], f[2 * y + 1]);
                    const uint32_t at = dst + (c16 >> 2) * L::kPanel + key * 128;
                    const int ch = (c16 & 3) * 2;
                    sts128(at + ((ch ^ (key & 7)) << 4), f[0], f[1], f[2], f[3]);
                    sts128(at + (((ch + 1) ^ (key & 7)) << 4), f[4], f[5], f[6], f[7]);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(bar(kRawEmpty + slot));
                mbar_arrive(bar(kFull + stage));
            }
        }
    } else if (warp == 12) {
        // ------------------------------------------------------------- loader
        // Lane 4 x + y holds the page of copy y of half tile x of the next eight
        // (four tiles), loaded while the eight before are on their way.
        const int ck_shift = min(a.page_shift, 6);           // keys per copy
        const int ck = 1 << ck_shift;
        const int chunks = kHalf >> ck_shift;
        const int n_pages = (a.prefix_len + (1 << a.page_shift) - 1) >> a.page_shift;
        auto my_key = [&](int batch) { return tile0 * kTile + (batch * 8 + (lane >> 2)) * kHalf + (lane & 3) * ck; };
        auto my_page = [&](int batch) {
            const int key = my_key(batch), idx = key >> a.page_shift;
            if ((lane & 3) >= chunks || batch * 4 >= n || batch * 4 + (lane >> 3) >= n || key >= a.prefix_len)
                return 0;
            const int page = idx < n_pages ? __ldg(a.prefix_pages + idx) : -1;
            if (static_cast<unsigned>(page) < static_cast<unsigned>(a.num_pages))
                return page;
            set_error(a.err, kErrBitIndex);
            return 0;
        };
        int issued = 0, page = 0, next = my_page(0);
        bool ok = true;
        for (int s = 0; s < 4 * n && ok; ++s) {
            const int i = s >> 2, half = s & 1, slot = s % kRaw;
            const bool is_v = (s >> 1) & 1;
            if (s % 16 == 0) {
                page = next;
                next = my_page(s / 16 + 1);
            }
            const int key = my_key(s / 16);
            const bool mine = (lane >> 2) == (i & 3) * 2 + half && (lane & 3) < chunks && key < a.prefix_len;
            const int copies = __popc(__ballot_sync(0xFFFFFFFFu, mine));
            if (s >= kRaw)
                ok = wait_warp(kRawEmpty + slot, (s / kRaw - 1) & 1);
            if (!ok)
                break;
            const bool with_scales = TOK && !is_v;
            if (lane == 0) {
                mbar_arrive_expect_tx(bar(kRawFull + slot), copies * ck * D);
                if (with_scales && half == 0) {
                    const int live = min(a.prefix_len - (tile0 + i) * kTile, kTile);
                    mbar_arrive_expect_tx(bar(kScFull + i % kScaleRing), ((live + ck - 1) & ~(ck - 1)) * 8);
                }
            }
            __syncwarp();
            if (mine) {
                const int64_t row = ((static_cast<int64_t>(page) * a.Hkv + h) << a.page_shift) +
                                    (key & ((1 << a.page_shift) - 1));
                bulk_load(base + L::raw + slot * kHalf * D + (lane & 3) * ck * D,
                          (is_v ? a.v_cache : a.k_cache) + row * D, ck * D, bar(kRawFull + slot));
                if (with_scales) {
                    const uint32_t at = base + L::scales + (i % kScaleRing) * 2 * kTile * 4 +
                                        (half * kHalf + (lane & 3) * ck) * 4;
                    bulk_load(at, a.k_scale + row, ck * 4, bar(kScFull + i % kScaleRing));
                    bulk_load(at + kTile * 4, a.v_scale + row, ck * 4, bar(kScFull + i % kScaleRing));
                }
            }
            issued = s + 1;
        }
        // whatever happened to the other roles, the copies in flight end before
        // the CTA does (a raw slot's copies end before its successor's begin)
        if (lane == 0) {
            for (int s = max(issued - kRaw, 0); s < issued; ++s) {
                mbar_wait(bar(kRawFull + s % kRaw), (s / kRaw) & 1);
                if (TOK)
                    mbar_wait(bar(kScFull + (s >> 2) % kScaleRing), ((s >> 2) / kScaleRing) & 1);
            }
        }
    } else if (warp == 13) {
        // ------------------------------------------------------------- issuer
        // The whole warp walks the loop and one elected lane issues.
        // S_{i+1} overwrites P_i: one thread's MMAs run in order.
        const uint32_t leader = elect_one();
        constexpr uint32_t kIdS = idesc_f16(128, 128, false), kIdO = idesc_f16(128, D, true);
        const uint32_t k_lo = desc_lo(base + L::stage, 16), v_lo = desc_lo(base + L::stage, L::kPanel);
        constexpr uint32_t kStep = L::kOperand >> 4;
        auto scores = [&](int t, int i) {
            const uint32_t ts = tmem + t * kTile;
            const uint32_t q = desc_lo(base + L::q + t * L::kOperand, 16);
            const uint32_t k = k_lo + (2 * i % kStages) * kStep;
            mma_ss<false>(leader, ts, q, kDescHi, k, kDescHi, kIdS);
#pragma unroll
            for (int s = 1; s < D / 16; ++s) {
                const uint32_t off = ((s >> 2) * L::kPanel + (s & 3) * 32) >> 4;
                mma_ss<true>(leader, ts, q + off, kDescHi, k + off, kDescHi, kIdS);
            }
            commit(leader, bar(kSFull + t));
            if (t == nt - 1)
                commit(leader, bar(kEmpty + 2 * i % kStages));
        };
        bool ok = wait_warp(kFull, 0);
        for (int t = 0; t < nt && ok; ++t) {
            ok = wait_warp(kQFull + t, 0);
            if (ok) {
                tc_fence_after();
                scores(t, 0);
            }
        }
        for (int i = 0; i < n && ok; ++i) {
            const int jv = 2 * i + 1, jk = 2 * i + 2;
            const uint32_t v = v_lo + (jv % kStages) * kStep;
            ok = wait_warp(kFull + jv % kStages, (jv / kStages) & 1);
            for (int t = 0; t < nt && ok; ++t) {
                const uint32_t to = tmem + 2 * kTile + t * D, tp = tmem + t * kTile;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    ok = ok && wait_warp((half ? kPFull : kPHalf) + t, i & 1);
                    if (!ok)
                        break;
                    tc_fence_after();
#pragma unroll
                    for (int s = half * 4; s < half * 4 + 4; ++s)
                        mma_ts(leader, to, tp + s * 8, v + s * (2048 >> 4), kDescHi, kIdO, s > 0 || i > 0);
                }
                if (!ok)
                    break;
                if (t == nt - 1)
                    commit(leader, bar(kEmpty + jv % kStages));
                if (i + 1 == n) {
                    commit(leader, bar(kOFull + t));
                } else if (t > 0 || (ok = wait_warp(kFull + jk % kStages, (jk / kStages) & 1))) {
                    tc_fence_after();
                    scores(t, i + 1);
                }
            }
        }
        if (!ok && leader) {   // what was issued ends before tensor memory is freed
            mbar_init(bar(kBars), 1);
            fence_mbar_init();
            umma_commit(bar(kBars));
            mbar_wait(bar(kBars), 0);
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 13) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
        tmem_relinquish();
    }
}

// Splits that a plan may have, whatever the sequences' own keys: two waves.
int kv8_prefix_most_splits(int Hkv, int rows, int prefix_len)
{
    const int64_t base = static_cast<int64_t>(Hkv) * ((rows + 2 * kTile - 1) / (2 * kTile));
    const int64_t fill = 2 * ((kKv8PrefixCtas + base - 1) / base);
    const int64_t tiles = (prefix_len + kTile - 1) / kTile;
    return static_cast<int>(fill < tiles ? (fill < kKv8MaxSplits ? fill : kKv8MaxSplits)
                                         : (tiles < kKv8MaxSplits ? tiles : kKv8MaxSplits));
}

// Rows of partial results of a kv head (splits times `rows`) that a plan may have,
// as a bound that grows with `rows` and `prefix_len`: the splits go down where
// another pair of row tiles begins, but a workspace for the largest batch has to
// serve the smaller ones. With c = ceil(kKv8PrefixCtas / Hkv), r pairs have at
// most 2 ceil(c / r) splits of 2 kTile r rows, 4 kTile (c - 1 + r) in all.
int64_t kv8_prefix_most_rows(int Hkv, int rows, int prefix_len)
{
    const int64_t c = (kKv8PrefixCtas + Hkv - 1) / Hkv, r = (rows + 2 * kTile - 1) / (2 * kTile);
    const int64_t few = static_cast<int64_t>(kv8_prefix_most_splits(Hkv, 1, prefix_len)) * rows;
    const int64_t many = 4 * kTile * (c - 1 + r);
    return few < many ? few : many;
}

Kv8Prefix kv8_prefix_plan(int Hkv, int rows, int prefix_len, int D, float tile_us, int64_t own_max,
                          int num_sms)
{
    Kv8Prefix p = {};
    p.tiles = (prefix_len + kTile - 1) / kTile;
    p.row_pairs = (rows + 2 * kTile - 1) / (2 * kTile);
    // The time of a split, in us. A CTA takes tile_us for a key tile (one row tile
    // or two: a tile's chain of products and softmax bounds both) and some 5 for its
    // start and end. The sequences' own keys take 4 and their bytes, either on the
    // SMs that the prefix leaves or on all, the others joining after the prefix; a
    // part f of the SMs reads at some f (2 - f) of the full rate (beside a prefix on
    // 72 and 48 SMs: 0.80 and 0.87). Every split is written and read once more.
    struct Split {
        int splits, per;
        float us, rate, slow, join;   // slow: 1 / rate
        float with(float own_us) const
        {
            float own = 0.0f;
            if (own_us > 0.0f) {
                const float early = rate * (us > 4.0f ? us - 4.0f : 0.0f);
                own = us + 4.0f + (own_us > early ? own_us - early : 0.0f);
                if (rate > 0.0f && 4.0f + own_us * slow < own)
                    own = 4.0f + own_us * slow;
            }
            return (own > us ? own : us) + join;
        }
    };
    const int base = Hkv * p.row_pairs;   // below 2^21, and 2^27 times the splits
    const float join_us = static_cast<float>(Hkv) * rows * D * (8 / 8e6f);
    const int most = kv8_prefix_most_splits(Hkv, rows, prefix_len);
    Split all[kKv8MaxSplits];
    int n = 0;
    float alone = 0.0f;
    for (int s = 1; s <= most; ++s) {
        const int per = (p.tiles + s - 1) / s;
        const int splits = (p.tiles + per - 1) / per;
        if (s > 1 && splits < s)
            continue;   // the same as one before
        const int taken = base * splits, waves = (taken + num_sms - 1) / num_sms;
        Split& x = all[n++];
        x.splits = splits;
        x.per = per;
        x.us = waves * (per * tile_us + 5.0f);
        const float free = waves > 1 ? 0.0f : static_cast<float>(num_sms - taken) / num_sms;
        x.rate = free * (2.0f - free);
        x.slow = 1.0f / x.rate;
        x.join = splits * join_us;
        const float us = x.us + x.join;
        alone = n == 1 || us < alone ? us : alone;
    }
    // The lengths stand on the device, and a page table's width only bounds them. So
    // the split is taken that is the least behind the best one for any own keys
    // between a quarter of the prefix's work and as much again (more of them, and
    // the split hardly matters), as far as the tables hold so many. Of 38 batches of
    // 8-256 sequences over 1024-65536 tokens with up to 40000 own tokens each, tables
    // tight and 32768 wide, the time is 1.05 times the best split's in the mean and
    // 1.20 times at most. By half of what the tables hold, with the wide ones, us: 64
    // sequences over 8192 131 (now 29.6), 128 over 32768 365 (103), 256 over 65536 707
    // (266), 32 over 1024, capped, 34.9 (14.8).
    const float bytes_us = static_cast<float>(own_max) * Hkv * (2 * D / 5.5e6f);
    constexpr int kLoads = 3;
    constexpr float kLoad[kLoads] = {0.25f, 0.5f, 1.0f};
    float worst[kKv8MaxSplits];
    for (int j = 0; j < kLoads; ++j) {
        const float own_us = kLoad[j] * alone < bytes_us ? kLoad[j] * alone : bytes_us;
        float us[kKv8MaxSplits], best = 0.0f;
        for (int i = 0; i < n; ++i) {
            us[i] = all[i].with(own_us);
            best = i == 0 || us[i] < best ? us[i] : best;
        }
        const float scale = 1.0f / best;
        for (int i = 0; i < n; ++i)
            worst[i] = j == 0 || us[i] * scale > worst[i] ? us[i] * scale : worst[i];
        if (own_us >= bytes_us)
            break;
    }
    int at = 0;
    for (int i = 1; i < n; ++i)
        at = worst[i] < worst[at] ? i : at;
    p.splits = all[at].splits;
    p.tiles_per_split = all[at].per;
    p.us = all[at].us;
    return p;
}

template <int D, bool TOK, bool CAP>
static cudaError_t launch(const Kv8Attn& a, const Kv8Prefix& p, cudaStream_t s)
{
    auto kern = kv8_prefix_kernel<D, TOK, CAP>;
    const int smem = Smem<D>::total + 1024;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess)
        return e;
    return launch_dependent(kern, dim3(p.splits * a.Hkv * p.row_pairs), dim3(kThreads), smem, s, a, p);
}

template <int D>
static cudaError_t launch(const Kv8Attn& a, const Kv8Prefix& p, int per_token, cudaStream_t s)
{
    if (a.cap > 0.0f)
        return per_token ? launch<D, true, true>(a, p, s) : launch<D, false, true>(a, p, s);
    return per_token ? launch<D, true, false>(a, p, s) : launch<D, false, false>(a, p, s);
}

cudaError_t launch_kv8_prefix(const Kv8Attn& a, const Kv8Prefix& p, int D, int per_token, cudaStream_t s)
{
    return D == 128 ? launch<128>(a, p, per_token, s) : launch<64>(a, p, per_token, s);
}

}  // namespace w4a8
