// attn_tiles.cu -- q8_tree_attention for more than 16 packed rows a unit:
// 128 rows x 128 keys a tile on the 5th-generation tensor cores.
//
//     S = Q K^T,  P = 2^(S * scale - m),  O += P V,  l += rowsum(P)
//
// f32 precision on f16 MMAs: q and the weights are sums of two f16 parts
// (22 bits), both parts are multiplied with the same key or value tile into
// the same f32 accumulator, so a tile costs 2 * (D/16 + 8) MMAs of K = 16.
//
// Tensor memory (512 columns): S, P (64 columns of high parts, 64 of low
// parts: the second product's A operand), O and the sum of earlier Os
// (kChain, below), one each.  S is free as soon as the softmax warps have read
// it, so the next tile's scores are computed while this tile's weights are,
// and P is written when the last tile's products are done, while they were
// being computed: neither product waits for the other's operands.  (With P
// over S, in two or three buffers, a tile's scores had to wait for the
// products two or three tiles back.)  V is used as it lies in the cache
// ([key][dim], N-major).
//
// Eight softmax warps work on every tile, 16 rows each (two warps per lane
// quarter of tensor memory): a tile's weights take half the time that four
// warps would need, and a row has one owner for the whole unit, so there is
// one (m, l), one O and nothing to join at the end.  Scores are read in the
// 16x256b shape: a thread has two rows at 32 columns each, f16 holds them in 64
// registers between the maximum and the weights, and a key's scale is read
// once for two rows.
//
// Roles: warps 0 and 2 copy K and V tiles (one TMA box per run of keys that
// share a page); warp 1 issues the scores' MMAs and warp 3 the products' (one warp for
// both left the tensor core idle a third of the time: it queues only a few
// MMAs ahead, and every wait of the issuing warp is a gap); warps 4-11 are the
// softmax warps; for int8, warps 12-15 widen the codes to f16 tiles (exact), a
// key's scale multiplies its score column and a value's scale its weight
// column.  At a unit's end the next unit's queries go to shared memory before
// the rows go out, so its first scores are computed meanwhile.
//
// Measured (head_dim 128, 28 heads on 4): a causal prompt of 3325 tokens, f16,
// 145 us (79.3 GFLOP, 547 TFLOP/s of the attention's products; the MMAs do
// them twice, in two parts: 1094 TFLOP/s); 8 trees of up to 16 nodes over up
// to 16001 keys, f16, 50 us (198 MB, 3.9 TB/s); 4 trees of up to 64 nodes over
// up to 30011 keys, int8, 158 us.  A tile's two products take 2048 cycles of
// the tensor core; f16 tiles follow each other every 2750 cycles, int8 tiles
// every 5000.  What bounds them is the softmax warps' chain of dependent steps
// (scores, maximum, vote, weights, store), which all eight walk in step, two a
// scheduler: 43 % (f16) and 51 % (int8) of the issue slots are used, and most
// waits are for tensor memory.  int8 scores are read twice, and free the next
// scores' place only then.  A unit's start and end cost 12000 more, some 5000
// of them for q's two parts.
//
// Every mbarrier wait is bounded; one that runs out raises the CTA's abort
// flag and the error word, and all roles drain and exit.
#include <cuda.h>

#include <type_traits>

#include "attn_common.cuh"

namespace {

using q8::AttnArgs;
using q8::Unit;

__device__ unsigned int g_tiles_err;

constexpr int kRows = 128, kTile = 128;
// What a unit costs beside its tiles, in tiles (12000 cycles of 2750; the prompt of 3325 tokens with 3: 162 us, 4: 145, 5: 141).
constexpr int kHead = 5;
constexpr int kWholeTiles = 16;  // of a unit that one CTA does, however many there are: lengths may be ragged
constexpr float kWeightBits = 6.0f;  // weights are 2^(s - m + 6): below 2^14 while m may lag by 2^8
constexpr float kRaise = 8.0f;
constexpr int kScaleSlots = 4;
// The tensor core's f32 accumulation truncates: O loses about 1e-7 of itself
// per MMA, always towards zero (measured: 2.8e-5 after 31 tiles of 16 MMAs
// with values of one sign).  After kChain tiles O is therefore added to a sum
// of its own, rounded to nearest, and starts again.
constexpr int kChain = 4;

template <int D, bool kInt8>
struct Lay {
    static constexpr int kThreads = kInt8 ? 512 : 384;
    // registers per thread after setmaxnreg; their sum is the launch's
    static constexpr int kRegsLaunch = kInt8 ? 128 : 168;
    static constexpr int kRegsSoft = kInt8 ? 160 : 184, kRegsCtl = kInt8 ? 96 : 136, kRegsConv = 96;
    static_assert(256 * kRegsSoft + 128 * kRegsCtl + (kInt8 ? 128 * kRegsConv : 0) <= kThreads * kRegsLaunch, "registers");

    static constexpr int kMat = 128 * D * 2;            // a 128-row f16 tile
    static constexpr int kBufs = kInt8 ? 1 : 2;         // f16 tiles of K, and of V
    static constexpr int offQ = 0;                      // high parts, low parts
    static constexpr int offK = offQ + 2 * kMat;
    static constexpr int offV = offK + kBufs * kMat;
    static constexpr int offRaw = offV + kBufs * kMat;  // int8: two stages of K codes, two of V codes
    static constexpr int kRaw = 128 * D;
    static constexpr int offScale = offRaw + (kInt8 ? 4 * kRaw : 0);   // slots of 128 k scales, 128 v scales
    static constexpr int offOnes = offScale + (kInt8 ? kScaleSlots * 1024 : 0);  // int8: 128 scales of 1
    static constexpr int offRow = offOnes + (kInt8 ? 512 : 0);
    static constexpr int offBar = offRow + 2 * 128 * 4;  // before it: q scales of this unit and the next
    // barriers, by index
    // f16 tiles: full, empty, by the tile's parity (for int8 one buffer, still two barriers)
    static constexpr int bKf = 0, bKe = 2, bVf = 4, bVe = 6;
    static constexpr int bRKf = 8, bRKe = 10, bRVf = 12, bRVe = 14;  // int8 codes
    static constexpr int bCf = 16, bCe = 20;                         // int8 scales
    // scores written, scores read, weights written, products done; queries written
    static constexpr int bSf = 24, bSr = 25, bPf = 26, bPd = 27, bQf = 28, bDrain = 29, kBars = 31;
    static constexpr int offMisc = offBar + kBars * 8 + 8;
    static constexpr int offPre = offMisc + 32;
    static int smem(int batch) { return offPre + (batch + 1) * 4 + 1024; }
    static_assert(offPre + (Q8_KV_MAX_BATCH + 1) * 4 + 1024 <= 227 * 1024, "shared memory");
    static constexpr int kColP = 128, kColO = 256, kColSum = 384;  // S lies at 0
};

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tc_commit(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// The MMAs' operands are computed by the whole warp (they are uniform, and the
// instruction wants them in uniform registers); `one` is set in the one lane
// that issues.

// D (tensor memory) (+)= A (shared memory) B (shared memory)
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc, uint32_t one)
{
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(one)
        : "memory");
}

// D (tensor memory) (+)= A (tensor memory) B (shared memory)
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc, uint32_t one)
{
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(acc), "r"(one)
        : "memory");
}

// 16 lanes x 64 columns (16x256b, 8 repetitions): registers 4*rep + {0, 1} are
// lane i/4, columns 8*rep + 2*(i%4) + {0, 1}; 4*rep + {2, 3} the same of lane
// i/4 + 8.  Valid after tc_wait_ld and tc_regs32.
__device__ __forceinline__ void tc_ld16x64(uint32_t taddr, uint32_t *r)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
        "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}

// The same with 32 columns (16x256b, 4 repetitions).
__device__ __forceinline__ void tc_ld16x32(uint32_t taddr, uint32_t *r)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

__device__ __forceinline__ void tc_st16x32w(uint32_t taddr, const uint32_t *r)
{
    asm volatile(
        "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// 16 lanes x 32 columns (16x128b, 8 repetitions): registers 2*rep are lane
// i/4, column 4*rep + i%4; 2*rep + 1 the same of lane i/4 + 8.  What pairs of
// values read by tc_ld16x64 become when they are packed into a word each.
__device__ __forceinline__ void tc_st16x32(uint32_t taddr, const uint32_t *r)
{
    asm volatile(
        "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

__device__ __forceinline__ void tc_ld16x32p(uint32_t taddr, uint32_t *r)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.16x128b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

// No use of the registers is scheduled before the wait that precedes this.
__device__ __forceinline__ void tc_regs16(uint32_t *r)
{
    asm volatile(""
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                   "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]));
}
__device__ __forceinline__ void tc_regs32(uint32_t *r)
{
    tc_regs16(r);
    tc_regs16(r + 16);
}

// Shared-memory matrix descriptor, 128-byte swizzle: rows of 128 bytes in
// 1024-byte atoms of 8 rows.  K-major (Q, K: a row's 64 values of the
// contraction): sbo steps over 8 rows, lbo is unused.  N-major (V: a key's 64
// values of the output): sbo steps over 8 keys, lbo over 64 output columns.
__device__ __forceinline__ uint64_t desc128(uint32_t addr, uint32_t lbo, uint32_t sbo)
{
    return static_cast<uint64_t>((addr >> 4) & 0x3fffu) | static_cast<uint64_t>((lbo >> 4) & 0x3fffu) << 16 |
           static_cast<uint64_t>((sbo >> 4) & 0x3fffu) << 32 | static_cast<uint64_t>(1) << 46 |
           static_cast<uint64_t>(2) << 61;
}

// Instruction descriptor: D f32, A and B f16, M = 128; bit 16: B is N-major.
constexpr uint32_t idesc_f16(int n, bool b_n_major)
{
    return (1u << 4) | (b_n_major ? 1u << 16 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) | (8u << 24);
}

__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

// Bounded wait; gives up on the CTA's abort flag or after the limit, and
// then raises the flag and the error word.
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int *abort_flag)
{
    if (Q8_WAIT_LIMIT_NS == 0) {  // a build that gives up at once: one non-blocking test
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(bar), "r"(parity)
            : "memory");
        if (ok) return true;
        *abort_flag = 1;
        atomicOr(&g_tiles_err, q8::kErrTimeout);
        return false;
    }
    if (try_wait(bar, parity)) return true;
    const uint64_t t0 = q8::globaltimer_ns();
    for (;;) {
#pragma unroll 1
        for (int i = 0; i < 16; ++i)
            if (try_wait(bar, parity)) return true;
        if (*abort_flag) return false;
        if (q8::globaltimer_ns() - t0 > Q8_WAIT_LIMIT_NS) {
            *abort_flag = 1;
            atomicOr(&g_tiles_err, q8::kErrTimeout);
            return false;
        }
    }
}

__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int *abort_flag)
{
    return __all_sync(Q8_FULL_MASK, wait_bar(bar, parity, abort_flag));
}

// Lets asynchronous work land before the CTA exits, whatever the abort flag says.
__device__ __forceinline__ void drain_bar(uint32_t bar, uint32_t parity)
{
    const uint64_t t0 = q8::globaltimer_ns();
    while (!try_wait(bar, parity))
        if (q8::globaltimer_ns() - t0 > Q8_DRAIN_LIMIT_NS) {
            atomicOr(&g_tiles_err, q8::kErrTimeout);
            return;
        }
}

__device__ __forceinline__ void arrive(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void soft_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

template <uint32_t N>
__device__ __forceinline__ void setmaxnreg_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
template <uint32_t N>
__device__ __forceinline__ void setmaxnreg_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }

// One CTA's stretch of the line, piece by piece; every role walks it alike.  kWhole: units gridDim.x apart, whole.
template <bool kWhole>
struct Walk {
    int pos, begin, end;  // next place; the stretch
    Unit u;               // before the first piece: the unit at `begin`
    int t0, n, kend;      // first tile, tiles, keys end
    bool first;           // the stretch begins in this unit

    __device__ __forceinline__ bool next(const AttnArgs &a, const int *pre)
    {
        if constexpr (kWhole) {
            const int rts = (a.max_fresh * a.group + kRows - 1) / kRows;
            while (pos < end) {
                const int x = pos / rts;
                u.rt = pos - x * rts, u.b = x / a.kv_heads, u.kvh = x - u.b * a.kv_heads;
                pos += gridDim.x;
                q8::attn_sequence(a, u.b, u.cached, u.fresh, u.first);
                if (u.rt * kRows >= u.fresh * a.group) continue;
                u.tiles = q8::attn_tiles_of<kRows, kTile>(a, u.cached, u.fresh, u.rt);
                first = true;
                t0 = 0, n = u.tiles;
                kend = q8::attn_visible(a, u.cached, u.fresh, min((u.rt + 1) * kRows, u.fresh * a.group));
                return true;
            }
            return false;
        }
        while (pos < end) {
            first = pos == begin;
            if (!first) q8::attn_next_unit<kRows, kTile, kHead>(a, pre, u);
            t0 = max(0, pos - u.start - kHead);
            n = min(u.tiles, end - u.start - kHead) - t0;
            pos = u.start + kHead + u.tiles;
            kend = min((t0 + n) * kTile,
                       q8::attn_visible(a, u.cached, u.fresh, min((u.rt + 1) * kRows, u.fresh * a.group)));
            if (n > 0) return true;  // else only the unit's head: the next CTA has its tiles
        }
        return false;
    }
};

// One block of the plane, held by the four lanes of a quad: v[2 * i] are
// columns 8 * i + c2 + {0, 1} of the 32.  The steps of q8_encode8.
__device__ __forceinline__ void encode_quad(const AttnArgs &a, long long at, const float2 *v, int c2, bool valid)
{
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = fmaxf(m, fmaxf(fabsf(v[2 * i].x), fabsf(v[2 * i].y)));
    m = fmaxf(m, __shfl_xor_sync(Q8_FULL_MASK, m, 1));
    m = fmaxf(m, __shfl_xor_sync(Q8_FULL_MASK, m, 2));
    const float d = q8::q8_block_d(m), di = q8::q8_block_di(d);
    int sum = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int q0 = q8::q8_code(v[2 * i].x, di), q1 = q8::q8_code(v[2 * i].y, di);
        sum += q0 + q1;
        if (valid)
            *reinterpret_cast<uint16_t *>(a.qs + at + 8 * i + c2) =
                static_cast<uint16_t>((q0 & 0xff) | ((q1 & 0xff) << 8));
    }
    sum += __shfl_xor_sync(Q8_FULL_MASK, sum, 1);
    sum += __shfl_xor_sync(Q8_FULL_MASK, sum, 2);
    if (valid && c2 == 0) a.ds[at / 32] = q8::q8_dsword(d, sum);
}

template <int D, bool kInt8, bool kWhole>
__global__ void __launch_bounds__(Lay<D, kInt8>::kThreads, 1)
attn_tiles_kernel(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                  const __grid_constant__ AttnArgs a, const int box)
{
    using L = Lay<D, kInt8>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = q8::smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *sm = smem_raw + (base - raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + L::offBar);
    const uint32_t bar0 = base + L::offBar;
    auto bar = [&](int i) { return bar0 + 8u * i; };
    float *s_row = reinterpret_cast<float *>(sm + L::offRow);  // the rows' q scales, of this unit and the next
    volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + L::offMisc);
    volatile int *s_stop = abort_flag + 1, *s_poison = abort_flag + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + L::offMisc + 16);
    int *pre = reinterpret_cast<int *>(sm + L::offPre);

    if (tid == 0) {
        *abort_flag = 0;
        *s_stop = 0;
        *s_poison = 0;
        for (int i = 0; i < L::kBars; ++i) {
            int count = 1;  // TMA bytes or a commit
            if (i >= L::bCe && i < L::bCe + kScaleSlots) count = 8;  // softmax warps
            if (i >= L::bCf && i < L::bCf + kScaleSlots) count = 2;  // the keys' scales and the values'
            if (i == L::bSr || i == L::bPf || i == L::bQf) count = 8;
            if (kInt8 && ((i >= L::bKf && i < L::bKf + 2) || (i >= L::bVf && i < L::bVf + 2))) count = 128;  // widening warps
            if ((i >= L::bRKe && i < L::bRKe + 2) || (i >= L::bRVe && i < L::bRVe + 2)) count = 128;
            q8::mbar_init(bars + i, count);
        }
        q8::fence_mbar_init();
    }
    if (kInt8 && tid < 128) reinterpret_cast<float *>(sm + L::offOnes)[tid] = 1.0f;
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(q8::smem_u32(tmem_slot)),
                     "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    q8::griddep_launch_dependents();
    q8::griddep_wait();
    const int cta = blockIdx.x;
    bool bad_data = false;
    int per = 1;
    Walk<kWhole> w;
    if constexpr (kWhole) {
        w.pos = w.begin = cta;
        w.end = a.batch * a.kv_heads * ((a.max_fresh * a.group + kRows - 1) / kRows);
        w.u.start = 0;
        if (cta == 0)
            for (int b = tid; b < a.batch; b += L::kThreads) {
                int x, y, z;
                bad_data |= !q8::attn_sequence(a, b, x, y, z);
            }
    } else {
        bad_data = !q8::attn_line<kRows, kTile, kHead, L::kThreads>(a, pre);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    if constexpr (!kWhole) {
        const int total = pre[a.batch];
        per = max(1, (total + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x));
        const int s0 = min(total, cta * per);
        w.pos = w.begin = s0;
        w.end = min(total, s0 + per);
        if (w.pos < w.end) w.u = q8::attn_unit<kRows, kTile, kHead>(a, pre, w.pos);
    }

    if (warp < 4) {
        setmaxnreg_dec<L::kRegsCtl>();
        if (!(warp & 1)) {
            // -------------------------------------------------------- copies: warp 0 K tiles, warp 2 V tiles; a scale with
            // its values
            const bool is_v = warp == 2;
            const CUtensorMap *map = is_v ? &mv : &mk;
            const float *scales = is_v ? a.vs : a.ks;
            const int full = kInt8 ? (is_v ? L::bRVf : L::bRKf) : (is_v ? L::bVf : L::bKf);
            const int empty = kInt8 ? (is_v ? L::bRVe : L::bRKe) : (is_v ? L::bVe : L::bKe);
            const uint32_t ring = base + (kInt8 ? L::offRaw + (is_v ? 2 * L::kRaw : 0) : is_v ? L::offV : L::offK);
            constexpr int kStage = kInt8 ? L::kRaw : L::kMat;
            constexpr int kRowBytes = kInt8 ? D : 128;  // of a box row
            constexpr int kHalves = kInt8 ? 1 : D / 64;
            const int boxes = kTile / box;
            int T = 0, n_tiles = 0, n_scales = 0;  // tiles so far; copies issued of each kind
            bool ok = true;
            while (ok && w.next(a, pre)) {
                auto fetch = [&](int i) {  // cache row of this lane's box of tile i
                    const int key = (w.t0 + i) * kTile + lane * box;
                    if (i >= w.n || lane >= boxes || key >= w.kend) return 0;
                    const int pi = key / a.page;
                    int pg = a.table[static_cast<long long>(w.u.b) * a.max_pages + pi];
                    if (pg < 0 || pg >= a.n_pages) {
                        bad_data = true;
                        pg = 0;
                    }
                    return (pg * a.kv_heads + w.u.kvh) * a.page + (key - pi * a.page);
                };
                int row = fetch(0);
                for (int i = 0; i < w.n; ++i, ++T) {
                    const int next = fetch(i + 1);
                    const int key0 = (w.t0 + i) * kTile;
                    const int nb = min(boxes, (w.kend - key0 + box - 1) / box);
                    const int st = T & 1;
                    if (kInt8) {
                        const int cs = T % kScaleSlots;
                        ok = warp_wait(bar(L::bCe + cs), (static_cast<uint32_t>(T / kScaleSlots) & 1u) ^ 1u, abort_flag);
                        if (!ok) break;
                        if (lane == 0) q8::mbar_arrive_expect_tx(bars + L::bCf + cs, nb * box * 4);
                        __syncwarp();
                        if (lane < nb)
                            q8::bulk_g2s(sm + L::offScale + cs * 1024 + (is_v ? 512 : 0) + lane * box * 4, scales + row, box * 4,
                                         bars + L::bCf + cs);
                        n_scales = T + 1;
                    }
                    ok = warp_wait(bar(empty + st), (static_cast<uint32_t>(T >> 1) & 1u) ^ 1u, abort_flag);
                    if (!ok) break;
                    if (lane == 0) q8::mbar_arrive_expect_tx(bars + full + st, nb * box * kRowBytes * kHalves);
                    __syncwarp();
                    if (lane < nb) {
#pragma unroll
                        for (int h = 0; h < kHalves; ++h)
                            q8::tma_load_2d(ring + st * kStage + h * 16384 + lane * box * kRowBytes, map, h * 64, row,
                                            bar(full + st));
                    }
                    n_tiles = T + 1;
                    row = next;
                }
            }
            // the last copies must have landed before the CTA exits
            for (int t = max(0, n_tiles - 2); t < n_tiles; ++t)
                drain_bar(bar(full + (t & 1)), static_cast<uint32_t>(t >> 1) & 1u);
            for (int t = max(0, n_scales - kScaleSlots); t < n_scales; ++t)
                drain_bar(bar(L::bCf + t % kScaleSlots), static_cast<uint32_t>(t / kScaleSlots) & 1u);
        } else if (warp == 1) {
            // -------------------------------------------------------- scores
            constexpr uint32_t iS = idesc_f16(kTile, false);
            const uint32_t one = lane == 0;
            const uint32_t tm = __shfl_sync(Q8_FULL_MASK, tmem, 0);
            int T = 0;
            uint32_t piece = 0;
            bool ok = true;
            while (ok && w.next(a, pre)) {
                ok = warp_wait(bar(L::bQf), piece & 1u, abort_flag);
                ++piece;
                for (int i = 0; ok && i < w.n; ++i, ++T) {
                    ok = warp_wait(bar(L::bKf + (T & 1)), static_cast<uint32_t>(T >> 1) & 1u, abort_flag) &&
                         warp_wait(bar(L::bSr), (static_cast<uint32_t>(T) & 1u) ^ 1u, abort_flag);  // the tile before
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t k = desc128(base + L::offK + (T % L::kBufs) * L::kMat, 16, 1024);
#pragma unroll
                    for (int part = 1; part >= 0; --part) {  // low parts first: the accumulator is small meanwhile
                        const uint64_t q = desc128(base + L::offQ + part * L::kMat, 16, 1024);
#pragma unroll
                        for (int s = 0; s < D / 16; ++s) {
                            const uint32_t o = ((s >> 2) * 16384 + (s & 3) * 32) >> 4;
                            mma_ss(tm, q + o, k + o, iS, part == 0 || s > 0, one);
                        }
                    }
                    if (one) {
                        tc_commit(bar(L::bSf));
                        tc_commit(bar(L::bKe + (T & 1)));
                    }
                    __syncwarp();
                }
            }
            // every MMA issued must be complete before tensor memory is freed
            if (one) {
                tc_commit(bar(L::bDrain));
                drain_bar(bar(L::bDrain), 0);
            }
        } else if (warp == 3) {
            // -------------------------------------------------------- products
            constexpr uint32_t iO = idesc_f16(D, true);
            const uint32_t one = lane == 0;
            const uint32_t tm = __shfl_sync(Q8_FULL_MASK, tmem, 0);
            int T = 0;
            bool ok = true;
            while (ok && w.next(a, pre)) {
                for (int i = 0; i < w.n; ++i, ++T) {
                    ok = warp_wait(bar(L::bVf + (T & 1)), static_cast<uint32_t>(T >> 1) & 1u, abort_flag) &&
                         warp_wait(bar(L::bPf), static_cast<uint32_t>(T) & 1u, abort_flag);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t v = desc128(base + L::offV + (T % L::kBufs) * L::kMat, 16384, 1024);
#pragma unroll
                    for (int part = 1; part >= 0; --part)
#pragma unroll
                        for (int s = 0; s < kTile / 16; ++s)
                            mma_ts(tm + L::kColO, tm + L::kColP + 64u * part + 8u * s, v + ((2048u * s) >> 4), iO,
                                   part == 0 || s > 0 || i % kChain > 0, one);
                    if (one) {
                        tc_commit(bar(L::bPd));
                        tc_commit(bar(L::bVe + (T & 1)));
                    }
                    __syncwarp();
                }
            }
            if (one) {
                tc_commit(bar(L::bDrain + 1));
                drain_bar(bar(L::bDrain + 1), 0);
            }
        }
        __syncwarp();
    } else if (warp < 12) {
        setmaxnreg_inc<L::kRegsSoft>();
        // ------------------------------------------------------------ softmax
        const int sw = warp - 4, g = lane >> 2, c2 = 2 * (lane & 3);
        const int r0 = (warp & 3) * 32 + 16 * (sw >> 2) + g;  // this thread's rows of the tile: r0 and r0 + 8
        const uint32_t tl = tmem + (static_cast<uint32_t>((warp & 3) * 32 + 16 * (sw >> 2)) << 16);
        int T = 0;
        uint32_t piece = 0;
        if (!kWhole && tid == 128) a.desc[2 * cta + 1].w = 0;  // no first piece yet
        // Q: a warp per row (D = 128) or two rows (D = 64), eight warps, four loads at a time in a loop (straight-line
        // code that runs once costs more than its loads' latency); the rows are brought to L2 beforehand.
        constexpr int kPer = D == 128 ? 1 : 2, kLanes = 32 / kPer, kLoads = 16 / kPer;
        const int sub = lane % kLanes;
        auto prefetch_q = [&](const Unit &u) {
            const q8::RowMap map(a, u.rt * kRows);
            const int rr = (tid - 128) >> 1;
            if (rr < u.fresh * a.group - u.rt * kRows) {
                const float *row = a.q + map.at(a, u, rr, D) + (tid & 1) * (D / 2);
#pragma unroll
                for (int c = 0; c < D / 2; c += 32) asm volatile("prefetch.global.L2 [%0];" ::"l"(row + c));
            }
        };
        auto write_q = [&](const Unit &u, float *scales) {
            const q8::RowMap map(a, u.rt * kRows);
            const int rows = u.fresh * a.group - u.rt * kRows;
            // the row's largest value goes to [1, 2), the sign of the scale (or a scale of 0) into q: hidden scores
            // become -inf before they are scaled, so the scale of a row is never 0
            const float sign = a.scale < 0.0f ? -1.0f : a.scale == 0.0f ? 0.0f : 1.0f;
#pragma unroll 1
            for (int j0 = 0; j0 < kLoads; j0 += 4) {
                float4 x[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int rr = (sw + 8 * (j0 + j)) * kPer + lane / kLanes;
                    x[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    if (rr < rows) x[j] = __ldg(reinterpret_cast<const float4 *>(a.q + map.at(a, u, rr, D)) + sub);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int rr = (sw + 8 * (j0 + j)) * kPer + lane / kLanes;
                    // magnitudes order as their bits do; a NaN's exponent is clamped like an infinity's
                    uint32_t top =
                        __float_as_uint(fmaxf(fmaxf(fabsf(x[j].x), fabsf(x[j].y)), fmaxf(fabsf(x[j].z), fabsf(x[j].w))));
                    if (D == 128) {
                        top = __reduce_max_sync(Q8_FULL_MASK, top);
                    } else {
#pragma unroll
                        for (int o = 1; o < kLanes; o <<= 1) top = max(top, __shfl_xor_sync(Q8_FULL_MASK, top, o));
                    }
                    const int e = min(126, max(-126, static_cast<int>(top >> 23) - 127));
                    const float down = q8::pow2(-e) * sign;
                    uint2 hi, lo;
                    q8::split_f16(x[j].x * down, x[j].y * down, hi.x, lo.x);
                    q8::split_f16(x[j].z * down, x[j].w * down, hi.y, lo.y);
                    const int off = (sub >> 4) * 16384 + rr * 128 + ((((sub & 15) >> 1) ^ (rr & 7)) << 4) + (sub & 1) * 8;
                    *reinterpret_cast<uint2 *>(sm + L::offQ + off) = hi;
                    *reinterpret_cast<uint2 *>(sm + L::offQ + L::kMat + off) = lo;
                    if (sub == 0) scales[rr] = fmaxf(q8::pow2(e) * fabsf(a.scale), 1.17549435e-38f);
                }
            }
            q8::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) arrive(bar(L::bQf));
        };
        // Products of tiles up to t complete; asked for every tile in turn, before the next tile's weights are written.
        auto products_done = [&](int t) { return warp_wait(bar(L::bPd), static_cast<uint32_t>(t) & 1u, abort_flag); };
        bool more = w.next(a, pre);
        if (more) {
            prefetch_q(w.u);
            write_q(w.u, s_row);
            soft_sync();  // the scales
        }
        while (more) {
            const Unit &u = w.u;
            const int rows = u.fresh * a.group, row0 = u.rt * kRows, pslot = 2 * cta + (w.first ? 0 : 1);
            const int all_see = u.cached + (a.masks ? 0 : q8::attn_token(a, row0) + 1);  // keys below are seen by every row
            const q8::RowSight sight0 = q8::attn_sight(a, u, row0 + r0), sight1 = q8::attn_sight(a, u, row0 + r0 + 8);
            const bool partial = !kWhole && (w.t0 > 0 || w.n < u.tiles);
            float qq[2], m[2], l[2], ii[2], msum[2];
            int e[2];
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                qq[y] = s_row[128 * (piece & 1) + r0 + 8 * y];
                m[y] = msum[y] = -INFINITY, l[y] = 0.0f, ii[y] = q8::pow2(126), e[y] = -126;
            }
            bool ok = true;
            {  // (the walk's next state is not kept: the tiles need the registers)
                Walk<kWhole> ahead = w;
                if (ahead.next(a, pre)) prefetch_q(ahead.u);
            }
            for (int i = 0; ok && i < w.n; ++i) {
                const int t = T + i, key0 = (w.t0 + i) * kTile;
                const bool masked = key0 + kTile > min(all_see, w.kend);
                const float *sc = reinterpret_cast<const float *>(sm + L::offScale + (t % kScaleSlots) * 1024);
                ok = warp_wait(bar(L::bSf), static_cast<uint32_t>(t) & 1u, abort_flag) &&
                     (!kInt8 ||
                      warp_wait(bar(L::bCf + t % kScaleSlots), static_cast<uint32_t>(t / kScaleSlots) & 1u, abort_flag));
                if (!ok) break;
                tc_fence_after();
                float all_big = 0.0f;  // int8: the tile's largest value scale
                bool odd = masked;     // some row sees not every key, or a value scale is not finite
                if (kInt8) {
                    const float4 v4 = *reinterpret_cast<const float4 *>(sc + 128 + 4 * lane);
                    all_big = __uint_as_float(__reduce_max_sync(
                        Q8_FULL_MASK, __float_as_uint(fmaxf(fmaxf(fabsf(v4.x), fabsf(v4.y)), fmaxf(fabsf(v4.z), fabsf(v4.w))))));
                    const float sum = (v4.x + v4.y) + (v4.z + v4.w);
                    odd |= __any_sync(Q8_FULL_MASK, !(fabsf(sum) <= 3.4028235e38f));
                }
                // of keys k .. k + 31, those that a row sees, from this thread's first column on
                auto seen_of = [&](const q8::RowSight &sight, int k) {
                    const int below = max(0, min(32, sight.all - k)), sh = u.cached - k;  // bit b of the mask is key k + sh + b
                    uint32_t see = below == 32 ? ~0u : (1u << below) - 1u;
                    if (sh >= 0 && sh < 32) see |= static_cast<uint32_t>(sight.mask << sh);
                    else if (sh < 0 && sh > -64) see |= static_cast<uint32_t>(sight.mask >> -sh);
                    return see >> c2;
                };
                float top[2] = {-INFINITY, -INFINITY}, big[2] = {all_big, all_big};
                if (odd) big[0] = big[1] = 0.0f;
                if (odd) {
                    // Where a row sees not every key: scores go back with -inf for what it does not see.  int8: multiplied
                    // with their keys' scales already; the largest value scale is taken over what the row sees, and a scale
                    // that is not finite makes the scores that see it NaN.
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        uint32_t z[16];
                        tc_ld16x32(tl + 32 * c, z);
                        tc_wait_ld();
                        tc_regs16(z);
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            const uint32_t see = seen_of(y ? sight1 : sight0, key0 + 32 * c);
#pragma unroll
                            for (int j = 0; j < 8; ++j) {  // column 8 * (j / 2) + c2 + j % 2 of the 32
                                uint32_t &x = z[4 * (j >> 1) + 2 * y + (j & 1)];
                                const bool seen = (see >> (8 * (j >> 1) + (j & 1))) & 1u;
                                if (kInt8) {
                                    const int key = 32 * c + 8 * (j >> 1) + c2 + (j & 1);
                                    const float v = sc[128 + key];
                                    x = __float_as_uint(__uint_as_float(x) * sc[key]);
                                    if (!(fabsf(v) <= 3.4028235e38f)) x = 0x7fffffffu;
                                    else if (seen) big[y] = fmaxf(big[y], fabsf(v));
                                }
                                if (!seen) x = 0xff800000u;
                            }
                        }
                        tc_st16x32w(tl + 32 * c, z);
                    }
                    if (kInt8) {
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            big[y] = fmaxf(big[y], __shfl_xor_sync(Q8_FULL_MASK, big[y], 1));
                            big[y] = fmaxf(big[y], __shfl_xor_sync(Q8_FULL_MASK, big[y], 2));
                        }
                    }
                    tc_wait_st();
                }
                // The maximum, 64 columns at a time (f16: at once, read once).
                uint32_t s[kInt8 ? 32 : 64];
                const float *kk = odd ? reinterpret_cast<const float *>(sm + L::offOnes) : sc;
                auto read_scores = [&](int h) {  // int8: 64 columns from 64 * h on, multiplied with their keys' scales
                    tc_ld16x64(tl + 64 * h, s);
                    tc_wait_ld();
                    tc_regs32(s);
#pragma unroll
                    for (int rep = 0; rep < 8; ++rep) {
                        const float2 k2 = *reinterpret_cast<const float2 *>(kk + 64 * h + 8 * rep + c2);
#pragma unroll
                        for (int y = 0; y < 4; y += 2) {
                            const float2 z = __fmul2_rn(
                                make_float2(__uint_as_float(s[4 * rep + y]), __uint_as_float(s[4 * rep + y + 1])), k2);
                            s[4 * rep + y] = __float_as_uint(z.x);
                            s[4 * rep + y + 1] = __float_as_uint(z.y);
                        }
                    }
                };
                auto scores_read = [&]() {  // the next tile's may come
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) arrive(bar(L::bSr));
                };
                if constexpr (!kInt8) {
                    tc_ld16x64(tl, s);
                    tc_ld16x64(tl + 64, s + 32);
                    tc_wait_ld();
                    tc_regs32(s);
                    tc_regs32(s + 32);
                    scores_read();
                }
#pragma unroll 1
                for (int h = 0; h < (kInt8 ? 2 : 1); ++h) {
                    if (kInt8) read_scores(h);
#pragma unroll
                    for (int j = 0; j < (kInt8 ? 32 : 64); j += 4) {
                        top[0] = fmaxf(fmaxf(top[0], __uint_as_float(s[j])), __uint_as_float(s[j + 1]));
                        top[1] = fmaxf(fmaxf(top[1], __uint_as_float(s[j + 2])), __uint_as_float(s[j + 3]));
                    }
                }
                const float mo[2] = {m[0], m[1]};  // the references of O as it stands
                const int eo[2] = {e[0], e[1]};
                float f[2] = {1.0f, 1.0f};
                bool raise = i == 0;  // the first tile sets the references
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    top[y] = fmaxf(top[y], __shfl_xor_sync(Q8_FULL_MASK, top[y], 1));
                    top[y] = fmaxf(top[y], __shfl_xor_sync(Q8_FULL_MASK, top[y], 2));
                    top[y] *= qq[y];
                    raise |= top[y] > m[y] + kRaise;
                    if (kInt8) raise |= big[y] * ii[y] > 1.0f;
                }
                raise = __any_sync(Q8_FULL_MASK, raise);
                if (raise) {
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const float mn = fmaxf(m[y], top[y]);
                        f[y] = mn == m[y] ? 1.0f : q8::exp2_approx(m[y] - mn);
                        l[y] *= f[y];
                        m[y] = mn;
                        if (kInt8) {
                            const int en = min(126, max(e[y], static_cast<int>(__float_as_uint(big[y]) >> 23) - 126));
                            f[y] = e[y] - en < -126 ? 0.0f : f[y] * q8::pow2(e[y] - en);
                            e[y] = en;
                            ii[y] = q8::pow2(-en);
                        }
                    }
                }
                float2 ref[2], sum[2];
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const float z = m[y] == -INFINITY ? 0.0f : kWeightBits - m[y];
                    ref[y] = make_float2(z, z);
                    sum[y] = make_float2(0.0f, 0.0f);
                }
                // the weights, as pairs of f16 parts over the scores' registers
#pragma unroll 1
                for (int h = 0; h < (kInt8 ? 2 : 1); ++h) {
                    if (kInt8) read_scores(h);
                    if (kInt8 && h) scores_read();
#pragma unroll
                    for (int rep = 0; rep < (kInt8 ? 8 : 16); ++rep) {
                        float2 v2 = make_float2(1.0f, 1.0f);
                        if (kInt8) v2 = *reinterpret_cast<const float2 *>(sc + 128 + 64 * h + 8 * rep + c2);
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            uint32_t *z = s + 4 * rep + 2 * y;
                            float2 p = __ffma2_rn(make_float2(__uint_as_float(z[0]), __uint_as_float(z[1])),
                                                  make_float2(qq[y], qq[y]), ref[y]);
                            p.x = q8::exp2_approx(p.x);
                            p.y = q8::exp2_approx(p.y);
                            sum[y] = __fadd2_rn(sum[y], p);
                            if (kInt8) p = __fmul2_rn(p, __fmul2_rn(v2, make_float2(ii[y], ii[y])));  // |v2 * ii| <= 1 if seen
                            q8::split_f16(p.x, p.y, z[0], z[1]);
                        }
                    }
                    // P and O are free once the products of the tile before are done
                    if (h == 0 && t > 0) {
                        ok = products_done(t - 1);
                        tc_fence_after();
                    }
#pragma unroll
                    for (int c = 0; c < (kInt8 ? 1 : 2); ++c) {
                        uint32_t hi[16], lo[16];
#pragma unroll
                        for (int j = 0; j < 16; ++j) hi[j] = s[32 * c + 2 * j], lo[j] = s[32 * c + 2 * j + 1];
                        tc_st16x32(tl + L::kColP + 32 * (h + c), hi);
                        tc_st16x32(tl + L::kColP + 64 + 32 * (h + c), lo);
                    }
                }
                if (kInt8 && odd) {  // a hidden key's scale may be anything: 0 * it is not the weight
                    tc_wait_st();
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {  // high parts of 64 keys, and of the next 64; low parts
                        uint32_t z[16];
                        tc_ld16x32p(tl + L::kColP + 32 * c, z);
                        tc_wait_ld();
                        tc_regs16(z);
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            const uint32_t see = seen_of(j & 1 ? sight1 : sight0, key0 + 64 * (c & 1) + 32 * (j >> 3)) >> (8 * ((j >> 1) & 3));
                            z[j] &= (see & 1u ? 0xffffu : 0u) | (see & 2u ? 0xffff0000u : 0u);
                        }
                        tc_st16x32(tl + L::kColP + 32 * c, z);
                    }
                }
                if (!ok) break;
#pragma unroll
                for (int y = 0; y < 2; ++y) l[y] += sum[y].x + sum[y].y;
                if (raise && i % kChain > 0) {
#pragma unroll 1
                    for (int c = 0; c < D; c += 32) {
                        uint32_t o[16];
                        tc_ld16x32(tl + L::kColO + c, o);
                        tc_wait_ld();
                        tc_regs16(o);
#pragma unroll
                        for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f[(j >> 1) & 1]);
                        tc_st16x32w(tl + L::kColO + c, o);
                    }
                }
                if (!kInt8 && masked) {
                    // values that no row sees must not reach the MMA as 0 * NaN: non-finite ones in a tile with hidden
                    // keys become zero, and are added back at the end for the rows that see them
                    ok = warp_wait(bar(L::bVf + (t & 1)), static_cast<uint32_t>(t >> 1) & 1u, abort_flag);
                    if (!ok) break;
                    uint8_t *v = sm + L::offV + (t & 1) * L::kMat;
                    __half2 nan = __float2half2_rn(0.0f);  // stays 0 over finite values
#pragma unroll
                    for (int c = 0; c < L::kMat / 16; c += 256) {
                        const uint4 z = *reinterpret_cast<const uint4 *>(v + 16 * (c + tid - 128));
                        const __half2 *h = reinterpret_cast<const __half2 *>(&z);
#pragma unroll
                        for (int j = 0; j < 4; ++j) nan = __hfma2(h[j], __float2half2_rn(0.0f), nan);
                    }
                    if (__any_sync(Q8_FULL_MASK, __hisnan(__low2half(nan)) || __hisnan(__high2half(nan)))) {
                        for (int c = tid - 128; c < L::kMat / 16; c += 256) {
                            uint4 z = *reinterpret_cast<const uint4 *>(v + 16 * c);
                            uint32_t *zz = reinterpret_cast<uint32_t *>(&z);
                            bool hit = false;
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                if ((zz[j] & 0x7c00u) == 0x7c00u) zz[j] &= 0xffff0000u, hit = true;
                                if ((zz[j] & 0x7c000000u) == 0x7c000000u) zz[j] &= 0x0000ffffu, hit = true;
                            }
                            if (hit) {
                                *reinterpret_cast<uint4 *>(v + 16 * c) = z;
                                if (key0 + ((c >> 3) & 127) < w.kend) *s_poison = 1;
                            }
                        }
                    }
                    q8::fence_proxy_async_smem();
                    __syncwarp();
                }
                if (i > 0 && i % kChain == 0) {
                    // this tile's products start O anew: what it holds goes to the sum
                    float two[2], keep[2];
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        two[y] = kInt8 ? q8::pow2(eo[y]) : 1.0f;
                        keep[y] = msum[y] == -INFINITY ? 0.0f : q8::exp2_approx(msum[y] - mo[y]);
                        msum[y] = mo[y];
                    }
#pragma unroll 1
                    for (int c = 0; c < D; c += 32) {
                        uint32_t o[16], z[16];
                        tc_ld16x32(tl + L::kColO + c, o);
                        if (i > kChain) tc_ld16x32(tl + L::kColSum + c, z);
                        tc_wait_ld();
                        tc_regs16(o);
                        if (i > kChain) tc_regs16(z);
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            const int y = (j >> 1) & 1;
                            float v = two[y] * __uint_as_float(o[j]);
                            if (i > kChain) v += keep[y] * __uint_as_float(z[j]);
                            o[j] = __float_as_uint(v);
                        }
                        tc_st16x32w(tl + L::kColSum + c, o);
                    }
                }
                tc_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    arrive(bar(L::bPf));
                    if (kInt8) arrive(bar(L::bCe + t % kScaleSlots));
                }
            }
            Walk<kWhole> nx = w;
            more = nx.next(a, pre);
            if (more && ok) write_q(nx.u, s_row + 128 * ((piece & 1) ^ 1));  // every score of this unit is computed
            ok = ok && products_done(T + w.n - 1);
            tc_fence_after();
            soft_sync();  // s_poison is complete, the next unit's scales are written
            if (tid == 128) *s_stop = *abort_flag;
            const int poison = *s_poison;
            const q8::RowMap map(a, row0);
            float inv[2], keep[2];
            long long at[2];
            bool valid[2];
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                l[y] += __shfl_xor_sync(Q8_FULL_MASK, l[y], 1);
                l[y] += __shfl_xor_sync(Q8_FULL_MASK, l[y], 2);
                // the quotient; a row that saw nothing is 0
                inv[y] = partial ? 1.0f : l[y] == 0.0f ? 0.0f : __frcp_rn(l[y]);
                keep[y] = msum[y] == -INFINITY ? 0.0f : q8::exp2_approx(msum[y] - m[y]) * inv[y];
                valid[y] = row0 + r0 + 8 * y < rows;
                at[y] = map.at(a, u, r0 + 8 * y, D);
            }
            // rows out, 64 columns at a time: a store of the warp writes whole 32-byte sectors of eight rows
#pragma unroll 1
            for (int c = 0; ok && c < D; c += 64) {
                uint32_t o[32];
                tc_ld16x64(tl + L::kColO + c, o);
                tc_wait_ld();
                tc_regs32(o);
                float2 v[16];  // 2 * rep + y: row r0 + 8 y, columns c + 8 rep + c2 + {0, 1}
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const float two = kInt8 ? q8::pow2(e[j & 1]) : 1.0f;
                    v[j] = make_float2(two * __uint_as_float(o[2 * j]) * inv[j & 1], two * __uint_as_float(o[2 * j + 1]) * inv[j & 1]);
                }
                if (w.n > kChain) {  // and the sum of the chains before
                    tc_ld16x64(tl + L::kColSum + c, o);
                    tc_wait_ld();
                    tc_regs32(o);
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        v[j].x += keep[j & 1] * __uint_as_float(o[2 * j]);
                        v[j].y += keep[j & 1] * __uint_as_float(o[2 * j + 1]);
                    }
                }
                if (!kInt8 && poison) {  // the non-finite values that were left out, for the rows that see them
                    for (int key = max(w.t0 * kTile, (u.cached & ~(kTile - 1)) - kTile); key < w.kend; ++key) {
                        const int pi = key / a.page;
                        const int pg = a.table[static_cast<long long>(u.b) * a.max_pages + pi];
                        if (pg < 0 || pg >= a.n_pages) continue;
                        const __half *val = reinterpret_cast<const __half *>(a.v16) +
                                            (static_cast<long long>(pg * a.kv_heads + u.kvh) * a.page + (key - pi * a.page)) * D + c + c2;
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            if (!q8::attn_sees(y ? sight1 : sight0, u.cached, key)) continue;
#pragma unroll
                            for (int rep = 0; rep < 8; ++rep) {
                                const float2 z = __half22float2(*reinterpret_cast<const __half2 *>(val + 8 * rep));
                                if (!(fabsf(z.x) <= 65504.0f)) v[2 * rep + y].x += z.x;
                                if (!(fabsf(z.y) <= 65504.0f)) v[2 * rep + y].y += z.y;
                            }
                        }
                    }
                    __syncwarp();
                }
                if (partial) {
                    float *dst = a.part + (static_cast<long long>(pslot) * kRows + r0) * D + c + c2;
#pragma unroll
                    for (int j = 0; j < 16; ++j) *reinterpret_cast<float2 *>(dst + (j & 1) * 8 * D + 8 * (j >> 1)) = v[j];
                } else {
                    if (a.y) {
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            if (valid[j & 1]) *reinterpret_cast<float2 *>(a.y + at[j & 1] + c + 8 * (j >> 1) + c2) = v[j];
                    }
                    if (a.qs) {
#pragma unroll
                        for (int blk = 0; blk < 2; ++blk)
#pragma unroll
                            for (int y = 0; y < 2; ++y)
                                encode_quad(a, at[y] + c + 32 * blk, v + 8 * blk + y, c2, valid[y]);
                    }
                }
            }
            tc_fence_before();  // O is read: the next unit's products come after its first weights
            if (partial && c2 == 0) {
                a.ml[pslot * kRows + r0] = make_float2(m[0], l[0]);
                a.ml[pslot * kRows + r0 + 8] = make_float2(m[1], l[1]);
            }
            if (partial && w.first && tid == 128) {
                a.desc[2 * cta] = make_int4(u.start, u.start + kHead + u.tiles, per, u.start + kHead);
                a.desc[2 * cta + 1] = make_int4(u.b, u.kvh, u.rt, 1);
            }
            soft_sync();  // s_stop is written, s_poison is read
            if (*s_stop) break;
            if (tid == 128) *s_poison = 0;
            soft_sync();  // before a tile of the next unit sets it
            T += w.n;
            ++piece;
            w = nx;
        }
    } else if (kInt8) {
        setmaxnreg_dec<L::kRegsConv>();
        // ------------------------------------------------------------ int8 codes -> f16 tiles in the MMA's layout
        // Eight lanes take half a row each of two neighbouring rows: with the 128-byte swizzle their 16-byte
        // stores then fall into distinct banks.
        const int c0 = tid - 384;
        auto widen = [&](uint32_t src_off, uint32_t dst_off) {
            constexpr int kChunks = D / 16;  // 16 codes each
#pragma unroll 4
            for (int j = 0; j < kChunks; ++j) {
                const int idx = c0 + 128 * j;
                int rr, c;
                if (D == 128) {
                    // groups of 8 lanes: rows 2p, 2p + 1; lanes 0-3 take one half of the first, 4-7 the other half of
                    // the second, and the next group the remaining halves
                    const int g = idx >> 3, x = idx & 7, pair = g >> 1, flip = g & 1;
                    rr = 2 * pair + (x >> 2);
                    c = (x & 3) + 4 * ((x >> 2) ^ flip);
                } else {
                    rr = idx >> 2;
                    c = idx & 3;
                }
                const uint4 q = *reinterpret_cast<const uint4 *>(sm + src_off + rr * D + c * 16);
                uint4 lo, hi;
                q8::i8x4_to_f16x4(q.x, lo.x, lo.y);
                q8::i8x4_to_f16x4(q.y, lo.z, lo.w);
                q8::i8x4_to_f16x4(q.z, hi.x, hi.y);
                q8::i8x4_to_f16x4(q.w, hi.z, hi.w);
                const uint32_t dst = dst_off + (c >> 2) * 16384 + rr * 128;
                *reinterpret_cast<uint4 *>(sm + dst + (((2 * (c & 3)) ^ (rr & 7)) << 4)) = lo;
                *reinterpret_cast<uint4 *>(sm + dst + (((2 * (c & 3) + 1) ^ (rr & 7)) << 4)) = hi;
            }
            q8::fence_proxy_async_smem();
        };
        // the codes of the CTA's tile t, once the tile before has been used
        auto widen_k = [&](int t) {
            const int st = t & 1;
            if (!warp_wait(bar(L::bRKf + st), static_cast<uint32_t>(t >> 1) & 1u, abort_flag) ||
                (t > 0 && !warp_wait(bar(L::bKe + (st ^ 1)), static_cast<uint32_t>((t - 1) >> 1) & 1u, abort_flag)))
                return false;
            widen(L::offRaw + st * L::kRaw, L::offK);
            arrive(bar(L::bKf + st));
            arrive(bar(L::bRKe + st));
            return true;
        };
        auto widen_v = [&](int t) {
            const int st = t & 1;
            if (!warp_wait(bar(L::bRVf + st), static_cast<uint32_t>(t >> 1) & 1u, abort_flag) ||
                (t > 0 && !warp_wait(bar(L::bVe + (st ^ 1)), static_cast<uint32_t>((t - 1) >> 1) & 1u, abort_flag)))
                return false;
            widen(L::offRaw + (2 + st) * L::kRaw, L::offV);
            arrive(bar(L::bVf + st));
            arrive(bar(L::bRVe + st));
            return true;
        };
        int tiles = 0;
        while (w.next(a, pre)) tiles += w.n;
        // a tile's K before the last tile's V: the scores run ahead of the products
        bool ok = tiles == 0 || widen_k(0);
        for (int t = 0; ok && t < tiles; ++t) ok = (t + 1 == tiles || widen_k(t + 1)) && widen_v(t);
    }
    if (bad_data) atomicOr(&g_tiles_err, q8::kErrData);

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
    }
}

template <int D, bool kInt8>
int launch_tiles(const CUtensorMap &mk, const CUtensorMap &mv, const AttnArgs &a, int box, int slot, cudaStream_t s)
{
    using L = Lay<D, kInt8>;
    const void *fn = a.cluster ? reinterpret_cast<const void *>(attn_tiles_kernel<D, kInt8, true>)
                               : reinterpret_cast<const void *>(attn_tiles_kernel<D, kInt8, false>);
    if (!q8::set_max_dynamic_smem(fn, 227 * 1024, slot + (a.cluster ? 12 : 0))) return Q8_ERR_LAUNCH;
    if (a.cluster) {
        const int units = a.batch * a.kv_heads * ((a.max_fresh * a.group + kRows - 1) / kRows);
        return q8::launch_pdl(attn_tiles_kernel<D, kInt8, true>, dim3(min(units, q8::kAttnCtas)), dim3(L::kThreads), L::smem(0), s,
                              mk, mv, a, box);
    }
    const int st = q8::launch_pdl(attn_tiles_kernel<D, kInt8, false>, dim3(q8::kAttnCtas), dim3(L::kThreads), L::smem(a.batch), s, mk,
                                  mv, a, box);
    if (st != Q8_OK) return st;
    return q8::launch_pdl(q8::attn_combine_kernel<D, kRows>, dim3(q8::kAttnCtas - 1, 8), dim3(256), 0, s, a);
}

} // namespace

namespace q8 {

// 1: units are dealt out to CTAs, which do them whole, without line, workspace and second launch; 0: the line.  In tiles: a CTA's own,
// against its stretch of the line and the join, some six tiles more.  Measured in a graph, 28 heads on 4 of 128 f16 values,
// trees of up to 16 nodes, line / whole: 1 sequence of 380 keys 15.6 / 13.6 us, 1000 15.1 / 17.9; 9 of 1000 18.6 / 18.3; 38 of
// 380 23.4 / 14.7, of 1000 31.9 / 21.8; 61 (244 units) of 380 32.2 / 25.4; a prompt of 520 tokens 21.2 / 14.4.
int attn_tiles_cluster(int64_t units, int64_t max_len)
{
    const int64_t tiles = (max_len + kTile - 1) / kTile;
    const int64_t turns = (units + kAttnCtas - 1) / kAttnCtas;
    return tiles <= kWholeTiles && turns * (tiles + kHead) <= units * (tiles + kHead) / kAttnCtas + kHead + 6 ? 1 : 0;
}

int attn_tiles_launch(const AttnCall &c, cudaStream_t s)
{
    const int D = c.dim;
    int box = 16;  // keys of a copy: the largest power of two in the page, up to a tile
    while (box < kTile && c.a.page % (2 * box) == 0) box *= 2;
    const CUtensorMapDataType dt = c.int8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    const CUtensorMapSwizzle sw = c.int8 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B;
    const uint32_t inner = c.int8 ? D : 64;
    const uint64_t pitch = D * (c.int8 ? 1 : 2);
    CUtensorMap mk, mv;
    if (!make_map_2d(&mk, dt, c.k, D, c.layer_rows, pitch, inner, box, sw) ||
        !make_map_2d(&mv, dt, c.v, D, c.layer_rows, pitch, inner, box, sw))
        return Q8_ERR_CUDA;
    if (D == 128)
        return c.int8 ? launch_tiles<128, true>(mk, mv, c.a, box, 28, s) : launch_tiles<128, false>(mk, mv, c.a, box, 29, s);
    return c.int8 ? launch_tiles<64, true>(mk, mv, c.a, box, 30, s) : launch_tiles<64, false>(mk, mv, c.a, box, 31, s);
}

unsigned int *attn_tiles_error_word()
{
    void *p = nullptr;
    return cudaGetSymbolAddress(&p, g_tiles_err) == cudaSuccess ? static_cast<unsigned int *>(p) : nullptr;
}

} // namespace q8
