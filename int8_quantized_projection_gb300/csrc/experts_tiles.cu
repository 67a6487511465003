// experts_tiles.cu -- products of many sorted rows with their experts' Q8_0
// matrices on the 5th-generation tensor cores.
//
// Y[r][i] = sum_b d_w(e,i,b) * d_a(s,b) * isum(r,i,b), as gemm_tc.cu: the int8
// codes as f16 (exact), two K = 16 MMAs per 32-wide block into tensor memory
// (an exact integer below 2^24), which the epilogue scales and adds in f32.
// What differs: the rows of an expert are ragged and scattered over the plane,
// and each matrix meets only a few tiles of rows, so a pass that widens all
// weights first would cost as much as the products.
//
//   Tiles.  128 weight rows x 64 or 128 sorted rows of one expert.  An expert's
//   rows are dealt to ceil(rows / 128) tiles in groups of 64.  All
//   tiles lie on one line (expert, weight tile, row tile), which the offsets
//   on the device make, and CTA c takes tiles c, c + grid, ...: those that run
//   together share their weights in L2.  A CTA's pipelines run on from tile to
//   tile; only the epilogue's stores lie between the last block of one and the
//   first of the next.
//   Weights go to shared memory as they are (34-byte blocks, TMA boxes of 16
//   rows x 8 blocks, or 4-byte copies where rows of blocks are not 16-byte
//   aligned), and four warps widen them there, a row a thread.
//   Activations: a pre-pass widens the plane's codes to f16 once per plane row;
//   the rows of a tile are gathered from there four a copy (tile::gather4), so
//   no sorted copy of them is written.
//   Gate and up: the 128 rows of a tile are 64 rows of each, 16 by 16, so that
//   the two products of a channel meet in one thread, and the epilogue writes
//   the plane of silu(gate) * up.
//
// Warp roles (512 threads):
//   warp 0      gathers activation tiles, 2 blocks a stage
//   warp 1      MMA issuer (one thread), tensor memory
//   warp 2      weight copies, 8 blocks a slot
//   warp 3      activation scales, 4 blocks a slot, and which rows are in range
//   warps 4-7   widen weights
//   warps 8-15  epilogue: two warps per TMEM lane quarter, 32-column groups in turn
// Every mbarrier wait is bounded; a wait that runs out sets the CTA abort flag
// and the error word, and all roles drain and exit.
#include "experts_common.cuh"

namespace {

__device__ unsigned int g_tiles_err;

constexpr int BM = 128, kGroup = 64, kMaxGroups = 2, BN = kGroup * kMaxGroups;
constexpr int kStages = 3, kRawSlots = 2, kDwSlots = 2, kDaSlots = 3, kAcc = 4;
constexpr int kTmemBuf = BN, kTmemCols = kAcc * kTmemBuf;
constexpr int kThreads = 512, kWidenThreads = 128, kEpiWarps = 8, kEpiThreads = 256;
constexpr int kRegsCtl = 72, kRegsWiden = 72, kRegsEpi = 184;
static_assert(128 * kRegsCtl + kWidenThreads * kRegsWiden + kEpiThreads * kRegsEpi <= 128 * kThreads, "register split");

constexpr int kPiece = 8;                      // blocks of a weight slot
constexpr int kPitchTma = 34 * kPiece;         // 272: a row's piece
constexpr int kPitchAny = kPitchTma + 4;       // 276: with the two bytes that a row may start late; 69 words, odd
constexpr int kRawBytes = BM * kPitchAny;      // 35328
constexpr int kABytes = BM * 128, kBBytes = BN * 128;
constexpr int kDwBytes = kPiece * BM * 4, kDaBlocks = 4, kDaBytes = kDaBlocks * BN * 4 + 32;

constexpr int OFF_A = 0;
constexpr int OFF_B = OFF_A + kStages * kABytes;
constexpr int OFF_RAW = OFF_B + kStages * kBBytes;
constexpr int OFF_DW = OFF_RAW + kRawSlots * kRawBytes;
constexpr int OFF_DA = OFF_DW + kDwSlots * kDwBytes;
constexpr int OFF_AMAX = OFF_DA + kDaSlots * kDaBytes;  // [4][BN] f32
constexpr int OFF_CODES = OFF_AMAX + 4 * BN * 4;        // [BN][64] int8
constexpr int OFF_MASK = OFF_CODES + BN * 64;           // rows of the tile that are in range: 6 words
constexpr int OFF_CUM = OFF_MASK + 32;                  // row tiles before each expert
constexpr int kBars = 2 * kRawSlots + 3 * kStages + 2 * kDwSlots + 2 * kDaSlots + 2 * kAcc + 1;
constexpr int OFF_BAR = OFF_CUM + (Q8_MAX_EXPERTS + 2) * 4;
constexpr int OFF_MISC = OFF_BAR + kBars * 8;           // abort flag, TMEM address, sums of the scan
constexpr int kSmemBytes = OFF_MISC + 16 + 64 + 1024;   // + alignment slack
static_assert(OFF_BAR % 8 == 0 && OFF_DA % 16 == 0 && OFF_CODES % 16 == 0 && kSmemBytes <= 227 * 1024, "shared memory");

struct Bars {
    uint32_t b0;
    __device__ uint32_t at(int i) const { return b0 + 8u * i; }
    __device__ uint32_t raw_full(int s) const { return at(s); }
    __device__ uint32_t raw_empty(int s) const { return at(kRawSlots + s); }
    __device__ uint32_t a_full(int s) const { return at(2 * kRawSlots + s); }
    __device__ uint32_t b_full(int s) const { return at(2 * kRawSlots + kStages + s); }
    __device__ uint32_t ab_empty(int s) const { return at(2 * kRawSlots + 2 * kStages + s); }
    __device__ uint32_t dw_full(int s) const { return at(2 * kRawSlots + 3 * kStages + s); }
    __device__ uint32_t dw_empty(int s) const { return dw_full(kDwSlots + s); }
    __device__ uint32_t da_full(int s) const { return dw_full(2 * kDwSlots + s); }
    __device__ uint32_t da_empty(int s) const { return da_full(kDaSlots + s); }
    __device__ uint32_t acc_full(int s) const { return da_full(2 * kDaSlots + s); }
    __device__ uint32_t acc_empty(int s) const { return acc_full(kAcc + s); }
    __device__ uint32_t drain() const { return acc_full(2 * kAcc); }
};

// ---------------------------------------------------------------------------
// PTX
// ---------------------------------------------------------------------------
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tc_mma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void tc_commit(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// 16 lanes x 32 columns: thread 4g + m gets lanes g and g + 8 at columns 8 rep + 2 m + {0, 1} in registers 4 rep + {0, 1} and
// 4 rep + {2, 3}.  Valid after tc_wait_ld; tc_regs16 keeps their uses behind it.
__device__ __forceinline__ void tc_ld16x32(uint32_t taddr, uint32_t *r)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

__device__ __forceinline__ void tc_regs16(uint32_t *r)
{
    asm volatile(""
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]));
}

// K-major operand, 128-byte swizzle: rows of 128 bytes in 1024-byte atoms of 8 rows.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr)
{
    return static_cast<uint64_t>((addr >> 4) & 0x3fffu) | (1ull << 16) | (static_cast<uint64_t>(1024 >> 4) << 32) |
           (1ull << 46) | (2ull << 61);
}

// D f32, A and B f16, K-major, M = 128, N = columns.
__device__ __forceinline__ uint32_t mma_desc(int columns)
{
    return (1u << 4) | (static_cast<uint32_t>(columns >> 3) << 17) | (static_cast<uint32_t>(BM >> 4) << 24);
}

// Four rows of the f16 plane, 128 bytes of each from element x on, to 512 bytes at dst.
__device__ __forceinline__ void tma_gather4(uint32_t dst, const CUtensorMap *map, int x, int4 rows, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, "
        "%6}], [%7];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(rows.x), "r"(rows.y), "r"(rows.z), "r"(rows.w), "r"(bar)
        : "memory");
}

// 4 bytes to shared memory, of which the first `bytes` come from src and the rest are zeros.
__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src, int bytes)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

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

__device__ __forceinline__ bool wait_slow(uint32_t bar, uint32_t parity, volatile int *abort_flag)
{
    const uint64_t t0 = q8::globaltimer_ns();
    do {
        if (try_wait(bar, parity)) return true;
        if (*abort_flag) return false;
    } while (Q8_WAIT_LIMIT_NS != 0 && q8::globaltimer_ns() - t0 <= Q8_WAIT_LIMIT_NS);
    *abort_flag = 1;
    atomicOr(&g_tiles_err, q8::kErrTimeout);
    return false;
}

// Bounded wait: false on the CTA's abort flag or past the limit (which raises it and the error word).
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int *abort_flag)
{
    if (Q8_WAIT_LIMIT_NS != 0 && try_wait(bar, parity)) return true;
    return wait_slow(bar, parity, abort_flag);
}

// The same for a whole warp that goes on together.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int *abort_flag)
{
    return __all_sync(Q8_FULL_MASK, wait_bar(bar, parity, abort_flag));
}

// Wait for copies or MMAs in flight before the CTA exits, whatever the abort flag says; bounded.
__device__ __forceinline__ void drain_bar(uint32_t bar, uint32_t parity)
{
    const uint64_t t0 = q8::globaltimer_ns();
    while (!try_wait(bar, parity)) {
        if (q8::globaltimer_ns() - t0 > Q8_DRAIN_LIMIT_NS) {
            atomicOr(&g_tiles_err, q8::kErrTimeout);
            return;
        }
    }
}

__device__ __forceinline__ void arrive(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void expect_tx(uint32_t bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

__device__ __forceinline__ void epi_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kEpiThreads) : "memory"); }

// Barrier of the epilogue warps; true when `bad` is true in any of them.
__device__ __forceinline__ bool epi_any(bool bad)
{
    uint32_t out;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, 1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(out)
        : "r"(static_cast<uint32_t>(bad)), "n"(kEpiThreads)
        : "memory");
    return out != 0;
}

template <uint32_t N>
__device__ __forceinline__ void setmaxnreg_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
template <uint32_t N>
__device__ __forceinline__ void setmaxnreg_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }

// ---------------------------------------------------------------------------
// tiles
// ---------------------------------------------------------------------------
struct Tile {
    int e, nt;          // expert, weight tile
    int row0, rows;     // sorted rows
    int groups;         // of 64 columns
};

__device__ __forceinline__ int groups_of(int rows) { return (rows + kGroup - 1) / kGroup; }
__device__ __forceinline__ int row_tiles_of(int rows) { return (groups_of(rows) + kMaxGroups - 1) / kMaxGroups; }

// cum[e]: row tiles of the experts before e.
__device__ __forceinline__ Tile tile_at(const q8::ExpertsArgs &a, const int *cum, int weight_tiles, int64_t at)
{
    const int q = static_cast<int>(at / weight_tiles);
    int lo = 0, hi = a.experts;  // cum[lo] <= q < cum[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cum[mid] <= q)
            lo = mid;
        else
            hi = mid;
    }
    const int mine = cum[lo + 1] - cum[lo];
    const int rest = static_cast<int>(at - static_cast<int64_t>(cum[lo]) * weight_tiles);
    Tile t;
    t.e = lo;
    t.nt = rest / mine;
    const int j = rest - t.nt * mine;
    const q8::ExpertRows x = q8::expert_rows_of(a, lo);
    const int g = groups_of(x.count);
    const int g0 = static_cast<int>(static_cast<int64_t>(j) * g / mine), g1 = static_cast<int>(static_cast<int64_t>(j + 1) * g / mine);
    t.row0 = x.first + g0 * kGroup;
    t.rows = min(x.count, g1 * kGroup) - g0 * kGroup;
    t.groups = g1 - g0;
    return t;
}

// Weight row (of all experts' rows) at position r of a tile; in a pair of matrices positions 16 .. 31 of each 32 are w2's.
template <bool kPair>
__device__ __forceinline__ int tile_row(int nt, int r)
{
    return kPair ? 64 * nt + 16 * (r >> 5) + (r & 15) : BM * nt + r;
}

__device__ __forceinline__ int dw_slot(int r) { return (r >> 5) * 32 + (r & 7) * 4 + ((r >> 4) & 1) * 2 + ((r >> 3) & 1); }
// column -> place of its scale: the eight columns of a thread in a group of 32 are neighbours
__device__ __forceinline__ int da_slot(int c) { return (c & ~31) + ((c >> 1) & 3) * 8 + ((c >> 3) & 3) * 2 + (c & 1); }

// acc += (d_w * d_a) * P for one 16-lane x 32-column load
__device__ __forceinline__ void epi_math(float2 *acc, const uint32_t *p, const float *da, float dw_lo, float dw_hi)
{
    const float2 w0 = make_float2(dw_lo, dw_lo), w1 = make_float2(dw_hi, dw_hi);
#pragma unroll
    for (int rep = 0; rep < 4; ++rep) {
        const float2 d2 = make_float2(da[2 * rep], da[2 * rep + 1]);
        acc[2 * rep] = __ffma2_rn(__fmul2_rn(w0, d2), make_float2(__uint_as_float(p[4 * rep]), __uint_as_float(p[4 * rep + 1])),
                                  acc[2 * rep]);
        acc[2 * rep + 1] = __ffma2_rn(__fmul2_rn(w1, d2),
                                      make_float2(__uint_as_float(p[4 * rep + 2]), __uint_as_float(p[4 * rep + 3])),
                                      acc[2 * rep + 1]);
    }
}

// What an epilogue warp carries from block to block.
struct EpiState {
    uint8_t *sm;
    Bars B;
    volatile int *abort_flag;
    uint32_t taddr;      // this warp's lanes and first column group
    int q, h, g, m;      // TMEM lane quarter, half of the groups, lane = 4 g + m
    uint32_t blocks;     // blocks done before this tile
    uint32_t dw, da;     // slots used before this tile
};

// The blocks of one tile: NG 32-column groups of this warp.  The loads of the next group are in flight while one is scaled, across
// blocks too, and a block's buffer is free when its last group has landed.
template <int NG>
__device__ __forceinline__ bool epi_blocks(const EpiState &s, int nb, float2 *acc, uint32_t *mask)
{
    uint32_t p[2][32];
    auto buffer = [&](int j) { return s.taddr + ((s.blocks + j) % kAcc) * kTmemBuf; };
    auto full = [&](int j) {
        const uint32_t n = s.blocks + j;
        const bool ok = warp_wait(s.B.acc_full(n % kAcc), (n / kAcc) & 1u, s.abort_flag);
        tc_fence_after();
        return ok;
    };
    auto load = [&](uint32_t *r, int j, int c) {
        const uint32_t t = buffer(j) + 64u * c;
        tc_ld16x32(t, r);
        tc_ld16x32(t + (16u << 16), r + 16);
    };
    const float *sw = nullptr, *sa = nullptr;
    if (!full(0)) return false;
    load(p[0], 0, 0);
    for (int j0 = 0; j0 < nb; j0 += 2) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int j = j0 + u;
            if (u == 1 && j >= nb) break;
            if ((j & 3) == 0) {  // the next four blocks' scales
                const uint32_t d = s.da + (j >> 2);
                if (!warp_wait(s.B.da_full(d % kDaSlots), (d / kDaSlots) & 1u, s.abort_flag)) return false;
                sa = reinterpret_cast<const float *>(s.sm + OFF_DA + (d % kDaSlots) * kDaBytes) + 32 * s.h + 8 * s.m;
                if ((j & 7) == 0) {
                    const uint32_t w = s.dw + (j >> 3);
                    if (!warp_wait(s.B.dw_full(w % kDwSlots), (w / kDwSlots) & 1u, s.abort_flag)) return false;
                    sw = reinterpret_cast<const float *>(s.sm + OFF_DW + (w % kDwSlots) * kDwBytes) + 32 * s.q + 4 * s.g;
                }
                if (j + 4 >= nb) {
                    const uint32_t *bits =
                        reinterpret_cast<const uint32_t *>(s.sm + OFF_DA + (d % kDaSlots) * kDaBytes + kDaBlocks * BN * 4);
#pragma unroll
                    for (int c = 0; c < NG; ++c) mask[c] = bits[2 * c + s.h];
                }
            }
            const float4 w4 = *reinterpret_cast<const float4 *>(sw + (j & 7) * BM);
#pragma unroll
            for (int c = 0; c < NG; ++c) {
                const int step = u * NG + c;
                uint32_t *now = p[step & 1], *next = p[(step + 1) & 1];
                tc_wait_ld();
                tc_regs16(now);
                tc_regs16(now + 16);
                if (c + 1 < NG) {
                    load(next, j, c + 1);
                } else {
                    tc_fence_before();
                    if ((s.g | s.m) == 0) arrive(s.B.acc_empty((s.blocks + j) % kAcc));
                    if (j + 1 < nb) {
                        if (!full(j + 1)) return false;
                        load(next, j + 1, 0);
                    }
                }
                const float4 a0 = *reinterpret_cast<const float4 *>(sa + (j & 3) * BN + 64 * c);
                const float4 a1 = *reinterpret_cast<const float4 *>(sa + (j & 3) * BN + 64 * c + 4);
                const float da[8] = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w};
                epi_math(acc + 16 * c, now, da, w4.x, w4.y);
                epi_math(acc + 16 * c + 8, now + 16, da, w4.z, w4.w);
            }
            if ((j & 3) == 3 || j == nb - 1) {
                __syncwarp();
                const uint32_t d = s.da + (j >> 2), w = s.dw + (j >> 3);
                if ((s.g | s.m) == 0) {
                    arrive(s.B.da_empty(d % kDaSlots));
                    if ((j & 7) == 7 || j == nb - 1) arrive(s.B.dw_empty(w % kDwSlots));
                }
            }
        }  // two blocks are an even number of groups: the next pair starts in p[0] again
    }
    return true;
}

// kPair: w and w2, the plane of silu(w x) * (w2 x); else w and f32 rows.  kTma: nb % 8 == 0.
template <bool kPair, bool kTma>
__global__ void __launch_bounds__(kThreads, 1)
experts_tiles_kernel(const __grid_constant__ q8::ExpertsArgs a, const __grid_constant__ CUtensorMap tmW,
                     const __grid_constant__ CUtensorMap tmW2, const __grid_constant__ CUtensorMap tmB, int8_t *qs_out,
                     uint32_t *ds_out)
{
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_base = q8::smem_u32(smem_raw);
    const uint32_t base = (raw_base + 1023u) & ~1023u;
    uint8_t *sm = smem_raw + (base - raw_base);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const Bars B{base + OFF_BAR};
    volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + OFF_MISC);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + OFF_MISC + 4);
    int *scan = reinterpret_cast<int *>(sm + OFF_MISC + 16);
    int *cum = reinterpret_cast<int *>(sm + OFF_CUM);

    if (tid == 0) {
        *abort_flag = (*reinterpret_cast<volatile unsigned int *>(&g_tiles_err) & q8::kErrTimeout) ? 1 : 0;
        uint64_t *b = reinterpret_cast<uint64_t *>(sm + OFF_BAR);
        int i = 0;
        auto init = [&](int n, uint32_t count) {
            for (int k = 0; k < n; ++k) q8::mbar_init(b + i++, count);
        };
        init(kRawSlots, 1);                  // raw_full: copied bytes
        init(kRawSlots, kWidenThreads);      // raw_empty
        init(kStages, kWidenThreads);        // a_full
        init(kStages, 1);                    // b_full: copied bytes
        init(kStages, 1);                    // ab_empty: tcgen05.commit
        init(kDwSlots, kWidenThreads);       // dw_full
        init(kDwSlots, kEpiWarps);           // dw_empty
        init(kDaSlots, 1);                   // da_full
        init(kDaSlots, kEpiWarps);           // da_empty
        init(kAcc, 1);                       // acc_full: tcgen05.commit
        init(kAcc, kEpiWarps);               // acc_empty
        init(1, 1);                          // drain
        q8::fence_mbar_init();
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(q8::smem_u32(tmem_slot)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    q8::griddep_launch_dependents();
    q8::griddep_wait();  // the offsets and the widened plane come from earlier kernels
    {                    // row tiles before each expert: two experts a thread
        int n[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            n[k] = 0;
            if (2 * tid + k < a.experts) {
                const q8::ExpertRows x = q8::expert_rows_of(a, 2 * tid + k);
                if (x.bad && blockIdx.x == 0) atomicOr(&g_tiles_err, q8::kErrData);
                n[k] = row_tiles_of(x.count);
            }
        }
        int v = n[0] + n[1];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(Q8_FULL_MASK, v, o);
            if (lane >= o) v += u;
        }
        if (lane == 31) scan[warp] = v;
        __syncthreads();
        int before = 0;
        for (int w = 0; w < warp; ++w) before += scan[w];
        v += before;
        if (2 * tid < a.experts) cum[2 * tid + 1] = v - n[1];
        if (2 * tid + 1 < a.experts) cum[2 * tid + 2] = v;
        if (tid == 0) cum[0] = 0;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    const int nb = a.nb, stages = (nb + 1) / 2, pieces = (nb + kPiece - 1) / kPiece, scales = (nb + kDaBlocks - 1) / kDaBlocks;
    const int weight_tiles = kPair ? (a.n + 63) / 64 : (a.n + BM - 1) / BM;
    const int64_t total = static_cast<int64_t>(cum[a.experts]) * weight_tiles;

    if (warp < 4) {
        setmaxnreg_dec<kRegsCtl>();
        if (warp == 0) {
            // ------------------------------------------------------------ activations
            uint32_t n = 0;  // stages issued
            bool ok = true;
            for (int64_t at = blockIdx.x; at < total && ok; at += gridDim.x) {
                const Tile t = tile_at(a, cum, weight_tiles, at);
                int4 src[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    int r[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int c = 4 * (lane + 32 * k) + i;
                        const int64_t s = q8::source_row(a, t.row0 + min(c, t.rows - 1));
                        r[i] = s < 0 ? 0 : static_cast<int>(s);  // a row out of range: any, it is not stored
                    }
                    src[k] = make_int4(r[0], r[1], r[2], r[3]);
                }
                for (int s = 0; s < stages; ++s, ++n) {
                    const int slot = n % kStages;
                    ok = warp_wait(B.ab_empty(slot), ((n / kStages) & 1u) ^ 1u, abort_flag);
                    if (!ok) break;
                    if (lane == 0) expect_tx(B.b_full(slot), t.groups * kGroup * 128);
                    __syncwarp();
                    const uint32_t dst = base + OFF_B + slot * kBBytes;
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        if (lane + 32 * k < t.groups * (kGroup / 4))
                            tma_gather4(dst + 512 * (lane + 32 * k), &tmB, 64 * s, src[k], B.b_full(slot));
                }
            }
            if (lane == 0)  // the last stages issued must have landed before the CTA exits
                for (uint32_t s = n < kStages ? 0 : n - kStages; s < n; ++s) drain_bar(B.b_full(s % kStages), (s / kStages) & 1u);
        } else if (warp == 1) {
            // ------------------------------------------------------------ MMA issuer
            if (lane == 0) {
                uint32_t n = 0, blk = 0;
                bool ok = true;
                for (int64_t at = blockIdx.x; at < total && ok; at += gridDim.x) {
                    const Tile t = tile_at(a, cum, weight_tiles, at);
                    const uint32_t idesc = mma_desc(t.groups * kGroup);
                    for (int j = 0; j < nb; ++j, ++blk) {
                        const int slot = n % kStages;
                        if ((j & 1) == 0) {
                            ok = wait_bar(B.b_full(slot), (n / kStages) & 1u, abort_flag) &&
                                 wait_bar(B.a_full(slot), (n / kStages) & 1u, abort_flag);
                            if (!ok) break;
                        }
                        ok = wait_bar(B.acc_empty(blk % kAcc), ((blk / kAcc) & 1u) ^ 1u, abort_flag);
                        if (!ok) break;
                        tc_fence_after();
                        const uint32_t d = tmem + (blk % kAcc) * kTmemBuf;
                        const uint32_t pa = base + OFF_A + slot * kABytes + 64 * (j & 1);
                        const uint32_t pb = base + OFF_B + slot * kBBytes + 64 * (j & 1);
                        tc_mma_f16(d, smem_desc(pa), smem_desc(pb), idesc, 0);
                        tc_mma_f16(d, smem_desc(pa + 32), smem_desc(pb + 32), idesc, 1);
                        tc_commit(B.acc_full(blk % kAcc));
                        if ((j & 1) || j == nb - 1) {
                            tc_commit(B.ab_empty(slot));
                            ++n;
                        }
                    }
                }
                // every MMA must have completed before its operands and TMEM go
                tc_commit(B.drain());
                drain_bar(B.drain(), 0);
            }
        } else if (warp == 2) {
            // ------------------------------------------------------------ weights
            if (kTma) {
                uint32_t n = 0;
                bool ok = true;
                for (int64_t at = blockIdx.x; at < total && ok; at += gridDim.x) {
                    const Tile t = tile_at(a, cum, weight_tiles, at);
                    const int row = t.e * a.n + tile_row<kPair>(t.nt, 16 * lane);
                    for (int s = 0; s < pieces; ++s, ++n) {
                        const int slot = n % kRawSlots;
                        ok = warp_wait(B.raw_empty(slot), ((n / kRawSlots) & 1u) ^ 1u, abort_flag);
                        if (!ok) break;
                        if (lane == 0) expect_tx(B.raw_full(slot), BM * kPitchTma);
                        __syncwarp();
                        if (lane < 8)  // 16 rows each
                            q8::tma_load_2d(base + OFF_RAW + slot * kRawBytes + lane * 16 * kPitchTma,
                                            kPair && (lane & 1) ? &tmW2 : &tmW, kPitchTma / 2 * s, row, B.raw_full(slot));
                    }
                }
                if (lane == 0)
                    for (uint32_t s = n < kRawSlots ? 0 : n - kRawSlots; s < n; ++s)
                        drain_bar(B.raw_full(s % kRawSlots), (s / kRawSlots) & 1u);
            }
        } else {
            // ------------------------------------------------------------ activation scales
            uint32_t n = 0;
            bool ok = true, bad = false;
            for (int64_t at = blockIdx.x; at < total && ok; at += gridDim.x) {
                const Tile t = tile_at(a, cum, weight_tiles, at);
                const uint32_t *src[2 * kMaxGroups];
                uint32_t valid[2 * kMaxGroups];
#pragma unroll
                for (int i = 0; i < 2 * kMaxGroups; ++i) {
                    const int c = lane + 32 * i;
                    const int64_t s = c < t.rows ? q8::source_row(a, t.row0 + c) : -1;
                    bad |= c < t.rows && s < 0;
                    valid[i] = __ballot_sync(Q8_FULL_MASK, s >= 0);
                    src[i] = a.ds + (s < 0 ? 0 : s) * nb;
                }
                for (int s = 0; s < scales; ++s, ++n) {
                    const int slot = n % kDaSlots;
                    ok = warp_wait(B.da_empty(slot), ((n / kDaSlots) & 1u) ^ 1u, abort_flag);
                    if (!ok) break;
                    float *dst = reinterpret_cast<float *>(sm + OFF_DA + slot * kDaBytes);
#pragma unroll
                    for (int i = 0; i < 2 * kMaxGroups; ++i)
                        if (i < 2 * t.groups) {
                            const int c = da_slot(lane + 32 * i);
                            uint32_t w[kDaBlocks];
                            if (nb % kDaBlocks == 0) {
                                const uint4 v = *reinterpret_cast<const uint4 *>(src[i] + kDaBlocks * s);
                                w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
                            } else {
#pragma unroll
                                for (int k = 0; k < kDaBlocks; ++k) w[k] = kDaBlocks * s + k < nb ? src[i][kDaBlocks * s + k] : 0u;
                            }
#pragma unroll
                            for (int k = 0; k < kDaBlocks; ++k)
                                dst[k * BN + c] = __half2float(__ushort_as_half(static_cast<unsigned short>(w[k] & 0xffffu)));
                        }
                    if (lane < 2 * kMaxGroups) {
                        uint32_t v = valid[0];
#pragma unroll
                        for (int i = 1; i < 2 * kMaxGroups; ++i) v = lane == i ? valid[i] : v;
                        reinterpret_cast<uint32_t *>(dst + kDaBlocks * BN)[lane] = v;
                    }
                    __syncwarp();
                    if (lane == 0) arrive(B.da_full(slot));
                }
            }
            if (bad) atomicOr(&g_tiles_err, q8::kErrData);
        }
    } else if (warp < 8) {
        setmaxnreg_dec<kRegsWiden>();
        // ---------------------------------------------------------------- widen weights: a row a thread
        const int r = tid - 128;
        const int sw = r & 7, dslot = dw_slot(r);
        uint32_t n = 0, p = 0;  // stages and pieces done
        bool ok = true;
        // the part of piece s of a tile's rows that this warp widens, 4 bytes a copy (rows of blocks that are not 16-byte aligned)
        auto copy = [&](const Tile &t, int s, uint32_t to) {
            if (kTma) return;
            const int cb = min(kPiece, nb - s * kPiece);
            for (int k = 0; k < 32; ++k) {
                const int pos = 32 * (warp - 4) + k;
                const int64_t row = static_cast<int64_t>(t.e) * a.n + min(tile_row<kPair>(t.nt, pos), a.n - 1);
                const uint8_t *w = kPair && (pos & 16) ? a.w2 : a.w;
                const int64_t from = (row * nb + s * kPiece) * 34, end = from + cb * 34;
                const int64_t most = static_cast<int64_t>(a.experts) * a.n * nb * 34;
                for (int64_t o = (from & ~int64_t(3)) + 4 * lane; o < end; o += 128)
                    cp_async4(base + OFF_RAW + (to % kRawSlots) * kRawBytes + pos * kPitchAny +
                                  static_cast<uint32_t>(o - (from & ~int64_t(3))),
                              w + o, static_cast<int>(min(int64_t(4), most - o)));
            }
            cp_async_commit();
        };
        int64_t at = blockIdx.x;
        Tile t = {}, tn = {};
        if (at < total) {
            tn = tile_at(a, cum, weight_tiles, at);
            copy(tn, 0, 0);
        }
        for (; at < total && ok; at += gridDim.x) {
            t = tn;
            if (at + gridDim.x < total) tn = tile_at(a, cum, weight_tiles, at + gridDim.x);
            const int64_t row = static_cast<int64_t>(t.e) * a.n + min(tile_row<kPair>(t.nt, r), a.n - 1);
            for (int s = 0; s < pieces && ok; ++s, ++p) {
                const int slot = p % kRawSlots, dws = p % kDwSlots;
                const uint8_t *raw = sm + OFF_RAW + slot * kRawBytes;
                if (kTma) {
                    ok = wait_bar(B.raw_full(slot), (p / kRawSlots) & 1u, abort_flag);
                } else {
                    // the next piece's copies in flight while this one is widened
                    if (s + 1 < pieces)
                        copy(t, s + 1, p + 1);
                    else if (at + gridDim.x < total)
                        copy(tn, 0, p + 1);
                    else
                        cp_async_commit();
                    cp_async_wait<1>();
                    __syncwarp();
                }
                ok = ok && wait_bar(B.dw_empty(dws), ((p / kDwSlots) & 1u) ^ 1u, abort_flag);
                if (!ok) break;
                float *dw = reinterpret_cast<float *>(sm + OFF_DW + dws * kDwBytes) + dslot;
                const int cb = min(kPiece, nb - s * kPiece);
#pragma unroll
                for (int k = 0; k < kPiece / 2; ++k) {
                    if (!kTma && 2 * k >= cb) break;
                    const int st = n % kStages;
                    ok = wait_bar(B.ab_empty(st), ((n / kStages) & 1u) ^ 1u, abort_flag);
                    if (!ok) break;
                    uint8_t *out = sm + OFF_A + st * kABytes + r * 128;
                    if (kTma) {
                        uint32_t W[20];  // 68 bytes from word 17 k on
#pragma unroll
                        for (int i = 0; i < 5; ++i) {
                            const uint4 v = *reinterpret_cast<const uint4 *>(raw + r * kPitchTma + 64 * k + 16 * i);
                            W[4 * i] = v.x, W[4 * i + 1] = v.y, W[4 * i + 2] = v.z, W[4 * i + 3] = v.w;
                        }
                        dw[(2 * k) * BM] = __half2float(__ushort_as_half(static_cast<unsigned short>(W[k] & 0xffffu)));
                        dw[(2 * k + 1) * BM] = __half2float(__ushort_as_half(static_cast<unsigned short>(W[k + 8] >> 16)));
#pragma unroll
                        for (int c = 0; c < 8; ++c) {
                            uint4 o;
                            uint32_t q0, q1;
                            if (c < 4) {
                                q0 = __byte_perm(W[k + 2 * c], W[k + 2 * c + 1], 0x5432);
                                q1 = __byte_perm(W[k + 2 * c + 1], W[k + 2 * c + 2], 0x5432);
                            } else {
                                q0 = W[k + 2 * c + 1], q1 = W[k + 2 * c + 2];
                            }
                            q8::i8x4_to_f16x4(q0, o.x, o.y);
                            q8::i8x4_to_f16x4(q1, o.z, o.w);
                            *reinterpret_cast<uint4 *>(out + 16 * (c ^ sw)) = o;
                        }
                    } else {
#pragma unroll
                        for (int b = 0; b < 2; ++b) {
                            const int64_t from = (row * nb + s * kPiece) * 34;
                            const int at_byte = static_cast<int>(from & 2) + 34 * (2 * k + b);
                            const uint32_t *src = reinterpret_cast<const uint32_t *>(raw + r * kPitchAny) + (at_byte >> 2);
                            const bool odd = at_byte & 2, there = 2 * k + b < cb;  // an odd last block: the other half is not used
                            const uint32_t sel = odd ? 0x7654u : 0x5432u;
                            uint32_t W[9];
#pragma unroll
                            for (int i = 0; i < 9; ++i) W[i] = there ? src[i] : 0u;
                            dw[(2 * k + b) * BM] =
                                __half2float(__ushort_as_half(static_cast<unsigned short>(odd ? W[0] >> 16 : W[0] & 0xffffu)));
#pragma unroll
                            for (int c = 0; c < 4; ++c) {
                                uint4 o;
                                q8::i8x4_to_f16x4(__byte_perm(W[2 * c], W[2 * c + 1], sel), o.x, o.y);
                                q8::i8x4_to_f16x4(__byte_perm(W[2 * c + 1], W[2 * c + 2], sel), o.z, o.w);
                                *reinterpret_cast<uint4 *>(out + 16 * ((4 * b + c) ^ sw)) = o;
                            }
                        }
                    }
                    q8::fence_proxy_async_smem();
                    arrive(B.a_full(st));
                    ++n;
                }
                if (!ok) break;
                arrive(B.dw_full(dws));
                if (kTma)
                    arrive(B.raw_empty(slot));
                else
                    __syncwarp();  // the warp's next copies overwrite what its lanes have read
            }
        }
        if (!kTma) cp_async_wait<0>();
    } else {
        setmaxnreg_inc<kRegsEpi>();
        // ---------------------------------------------------------------- epilogue
        EpiState s;
        s.sm = sm, s.B = B, s.abort_flag = abort_flag;
        s.q = warp & 3, s.h = (warp - 8) >> 2, s.g = lane >> 2, s.m = lane & 3;
        s.taddr = tmem + (static_cast<uint32_t>(32 * s.q) << 16) + 32u * s.h;
        s.blocks = s.dw = s.da = 0;
        bool ok = true;
        for (int64_t at = blockIdx.x; at < total; at += gridDim.x) {
            const Tile t = tile_at(a, cum, weight_tiles, at);
            // values of this thread: rows 32 q + 16 sub + g + 8 e, columns 32 (2c + h) + 8 rep + 2 m + {0, 1}, in
            // acc[16 c + 8 sub + 2 rep + e]
            float2 acc[16 * kMaxGroups];
            uint32_t mask[kMaxGroups];
#pragma unroll
            for (int i = 0; i < 16 * kMaxGroups; ++i) acc[i] = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int i = 0; i < kMaxGroups; ++i) mask[i] = 0u;
            if (t.groups == 2)
                ok = epi_blocks<2>(s, nb, acc, mask);
            else
                ok = epi_blocks<1>(s, nb, acc, mask);
            tc_wait_ld();  // none left, unless a wait ran out
            s.blocks += nb, s.dw += pieces, s.da += scales;
            ok = __all_sync(Q8_FULL_MASK, ok && !*abort_flag);
            if (!kPair) {
                if (!ok) break;
#pragma unroll
                for (int c = 0; c < kMaxGroups; ++c) {
                    if (c >= t.groups) break;
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int sub = i >> 3, rep = (i >> 1) & 3, e = i & 1;
                        const int row = BM * t.nt + 32 * s.q + 16 * sub + s.g + 8 * e;
                        if (row >= a.n) continue;
                        const int bit = 8 * rep + 2 * s.m, col = 32 * (2 * c + s.h) + bit;
                        float *out = a.out + static_cast<int64_t>(t.row0 + col) * a.ld + row;
                        const float2 v = acc[16 * c + i];
                        if ((mask[c] >> bit) & 1u) out[0] = v.x;
                        if ((mask[c] >> (bit + 1)) & 1u) out[a.ld] = v.y;
                    }
                }
            } else {
                float *amax = reinterpret_cast<float *>(sm + OFF_AMAX);
                uint8_t *codes = sm + OFF_CODES;
                uint32_t *smask = reinterpret_cast<uint32_t *>(sm + OFF_MASK);
                if (epi_any(!ok)) break;  // all of them, so that none waits for another below
                // silu(gate) * up into acc[16 c + 2 rep + e]; the block's largest value: over e, g, and the warp of the other 16
                // channels through shared memory
#pragma unroll
                for (int c = 0; c < kMaxGroups; ++c) {
                    if (c >= t.groups) break;
#pragma unroll
                    for (int rep = 0; rep < 4; ++rep) {
                        float2 most = make_float2(0.0f, 0.0f);
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float2 &g = acc[16 * c + 2 * rep + e];
                            const float2 u = acc[16 * c + 8 + 2 * rep + e];
                            g.x = q8::silu_mul(g.x, u.x), g.y = q8::silu_mul(g.y, u.y);
                            most.x = fmaxf(most.x, fabsf(g.x)), most.y = fmaxf(most.y, fabsf(g.y));
                        }
#pragma unroll
                        for (int o = 4; o < 32; o <<= 1) {
                            most.x = fmaxf(most.x, __shfl_xor_sync(Q8_FULL_MASK, most.x, o));
                            most.y = fmaxf(most.y, __shfl_xor_sync(Q8_FULL_MASK, most.y, o));
                        }
                        if (s.g == 0)
                            *reinterpret_cast<float2 *>(amax + s.q * BN + 32 * (2 * c + s.h) + 8 * rep + 2 * s.m) = most;
                    }
                    if (s.q == 0 && lane == 0) smask[2 * c + s.h] = mask[c];
                }
                epi_sync();
#pragma unroll
                for (int c = 0; c < kMaxGroups; ++c) {
                    if (c >= t.groups) break;
#pragma unroll
                    for (int rep = 0; rep < 4; ++rep) {
                        const int col = 32 * (2 * c + s.h) + 8 * rep + 2 * s.m;
                        const float *other = amax + (s.q & ~1) * BN + col;
                        const float2 m0 = *reinterpret_cast<const float2 *>(other), m1 = *reinterpret_cast<const float2 *>(other + BN);
                        const float ix = q8::q8_block_di(q8::q8_block_d(fmaxf(m0.x, m1.x)));
                        const float iy = q8::q8_block_di(q8::q8_block_d(fmaxf(m0.y, m1.y)));
                        // channel 16 q + g + 8 e of column col: 16-byte chunks swizzled by (col / 2) % 4 = m
                        uint8_t *o = codes + col * 64 + 16 * (s.q ^ s.m) + s.g;
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float2 v = acc[16 * c + 2 * rep + e];
                            o[8 * e] = static_cast<uint8_t>(q8::q8_code(v.x, ix));
                            o[64 + 8 * e] = static_cast<uint8_t>(q8::q8_code(v.y, iy));
                        }
                    }
                }
                epi_sync();
                // a thread per (row, block of 32 channels)
                for (int i = tid - 256; i < 2 * t.rows; i += kEpiThreads) {
                    const int col = i >> 1, blk = i & 1, ch = 64 * t.nt + 32 * blk;
                    if (ch >= a.n || !((smask[col >> 5] >> (col & 31)) & 1u)) continue;
                    const int sz = (col >> 1) & 3;
                    const uint4 v0 = *reinterpret_cast<const uint4 *>(codes + col * 64 + 16 * ((2 * blk) ^ sz));
                    const uint4 v1 = *reinterpret_cast<const uint4 *>(codes + col * 64 + 16 * ((2 * blk + 1) ^ sz));
                    int sum = q8::dp4a(v0.x, 0x01010101u, 0);
                    sum = q8::dp4a(v0.y, 0x01010101u, sum), sum = q8::dp4a(v0.z, 0x01010101u, sum);
                    sum = q8::dp4a(v0.w, 0x01010101u, sum), sum = q8::dp4a(v1.x, 0x01010101u, sum);
                    sum = q8::dp4a(v1.y, 0x01010101u, sum), sum = q8::dp4a(v1.z, 0x01010101u, sum);
                    sum = q8::dp4a(v1.w, 0x01010101u, sum);
                    const float d = q8::q8_block_d(fmaxf(amax[(2 * blk) * BN + col], amax[(2 * blk + 1) * BN + col]));
                    const int64_t row = t.row0 + col;
                    uint4 *o = reinterpret_cast<uint4 *>(qs_out + row * a.n + ch);
                    o[0] = v0, o[1] = v1;
                    ds_out[row * (a.n >> 5) + (ch >> 5)] = q8::q8_dsword(d, sum);
                }
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
    }
}

// The plane's codes as f16, 16 a thread and round.
__global__ void __launch_bounds__(256)
experts_widen_plane_kernel(const uint4 *__restrict__ qs, int64_t chunks, uint4 *__restrict__ out)
{
    q8::griddep_launch_dependents();
    q8::griddep_wait();
    const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.x;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < chunks; i += stride) {
        const uint4 v = __ldg(qs + i);
        uint4 o0, o1;
        q8::i8x4_to_f16x4(v.x, o0.x, o0.y);
        q8::i8x4_to_f16x4(v.y, o0.z, o0.w);
        q8::i8x4_to_f16x4(v.z, o1.x, o1.y);
        q8::i8x4_to_f16x4(v.w, o1.z, o1.w);
        out[2 * i] = o0;
        out[2 * i + 1] = o1;
    }
}

template <bool kPair, bool kTma>
int launch(const q8::ExpertsArgs &a, const CUtensorMap &mw, const CUtensorMap &mw2, const CUtensorMap &mb, unsigned grid,
           int8_t *qs_out, uint32_t *ds_out, int slot, cudaStream_t s)
{
    if (!q8::set_max_dynamic_smem(reinterpret_cast<const void *>(experts_tiles_kernel<kPair, kTma>), kSmemBytes, slot))
        return Q8_ERR_LAUNCH;
    return q8::launch_pdl(experts_tiles_kernel<kPair, kTma>, dim3(grid), dim3(kThreads), kSmemBytes, s, a, mw, mw2, mb, qs_out,
                          ds_out);
}

} // namespace

namespace q8 {

int64_t experts_tiles_rows(int64_t plane_rows, bool gather, int64_t pairs)
{
    return gather || plane_rows < pairs ? plane_rows : pairs;
}

size_t experts_tiles_workspace(int64_t k, int64_t plane_rows, bool gather, int64_t pairs)
{
    return static_cast<size_t>(experts_tiles_rows(plane_rows, gather, pairs)) * k * 2;
}

int experts_tiles_launch(const ExpertsArgs &a, int8_t *qs_out, uint32_t *ds_out, void *workspace, cudaStream_t s)
{
    const int64_t k = 32 * static_cast<int64_t>(a.nb), rows = experts_tiles_rows(a.plane_rows, a.rows != nullptr, a.pairs);
    const bool pair = a.w2 != nullptr, tma = a.nb % kPiece == 0;
    CUtensorMap mw = {}, mw2 = {}, mb = {};
    const uint64_t wrows = static_cast<uint64_t>(a.experts) * a.n, pitch = static_cast<uint64_t>(a.nb) * 34;
    if (tma && (!make_map_2d(&mw, CU_TENSOR_MAP_DATA_TYPE_UINT16, a.w, pitch / 2, wrows, pitch, kPitchTma / 2, 16,
                             CU_TENSOR_MAP_SWIZZLE_NONE) ||
                (pair && !make_map_2d(&mw2, CU_TENSOR_MAP_DATA_TYPE_UINT16, a.w2, pitch / 2, wrows, pitch, kPitchTma / 2, 16,
                                      CU_TENSOR_MAP_SWIZZLE_NONE))))
        return Q8_ERR_LAUNCH;
    if (!make_map_2d(&mb, CU_TENSOR_MAP_DATA_TYPE_UINT16, workspace, static_cast<uint64_t>(k), static_cast<uint64_t>(rows),
                     static_cast<uint64_t>(k) * 2, 64, 1, CU_TENSOR_MAP_SWIZZLE_128B))
        return Q8_ERR_LAUNCH;
    const int64_t chunks = rows * (k / 16), ctas = (chunks + 255) / 256;
    const int sms = device_sm_count();
    const int64_t cap = static_cast<int64_t>(sms) * 8;
    int st = launch_pdl(experts_widen_plane_kernel, dim3(static_cast<unsigned>(ctas < cap ? ctas : cap)), dim3(256), 0, s,
                        reinterpret_cast<const uint4 *>(a.qs), chunks, static_cast<uint4 *>(workspace));
    if (st != Q8_OK) return st;
    const int64_t weight_tiles = pair ? (a.n + 63) / 64 : (a.n + BM - 1) / BM;
    const int64_t most = (a.pairs / BN + (a.experts < a.pairs ? a.experts : a.pairs)) * weight_tiles;
    const unsigned grid = static_cast<unsigned>(most < sms ? most : sms);
    if (pair) return tma ? launch<true, true>(a, mw, mw2, mb, grid, qs_out, ds_out, 48, s)
                         : launch<true, false>(a, mw, mw2, mb, grid, qs_out, ds_out, 49, s);
    return tma ? launch<false, true>(a, mw, mw2, mb, grid, qs_out, ds_out, 50, s)
               : launch<false, false>(a, mw, mw2, mb, grid, qs_out, ds_out, 51, s);
}

unsigned int *experts_tiles_error_word()
{
    void *p = nullptr;
    return cudaGetSymbolAddress(&p, g_tiles_err) == cudaSuccess ? static_cast<unsigned int *>(p) : nullptr;
}

} // namespace q8
