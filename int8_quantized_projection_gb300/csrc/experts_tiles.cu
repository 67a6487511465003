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
//   Tiles.  128 weight rows x 16 .. 128 sorted rows of one expert.  An expert's
//   rows are dealt to ceil(rows / 128) tiles in steps of 16.  All tiles lie on
//   one line (expert, weight tile, row tile), which the offsets on the device
//   make, and CTA c takes tiles c, c + grid, ...: those that run together share
//   their weights in L2.  A CTA's pipelines run on from tile to tile; only the
//   epilogue's stores lie between the last block of one and the first of the
//   next.
//   Weights go to shared memory as they are (34-byte blocks, TMA boxes of 32
//   rows x 8 blocks, or a bulk copy a row where rows of blocks are not 16-byte
//   aligned), and four warps widen them there, a row a thread.  The activations
//   are widened once, by a pass that also puts the rows and their scales in order,
//   since each meets all weight tiles of its expert.
//   Scales.  d_w(i) * d_a(t) of a block is a product of two vectors: a third MMA
//   computes it beside the integers, d_w and d_a in the first of its 16 columns
//   and zeros in the others (a product of two f16 is exact in f32).  So the
//   epilogue reads two numbers a value from tensor memory and does one fma,
//   without scales from shared memory (16 bytes a lane and four values) and
//   without products of them.
//   Gate and up: the 128 rows of a tile are 64 rows of each, 32 by 32.  Two
//   warps swap halves of their columns, then a warp has a block of 32 channels of
//   16 rows, and writes the plane of silu(gate) * up.
//   What bounds it: the round trip of a block between MMAs and epilogue, with two buffers of accumulators (256 columns each,
//   all of tensor memory).  So each buffer has an issuer of its own, and 16 epilogue warps hold 32 columns each: four a scheduler
//   hide one another's loads.  3325 tokens of 8 of 64 experts, 2 x 1280 x 3584: 1039 us, 470 TFLOP/s; with one issuer and eight
//   warps 1430, with two halves of 64 columns that have buffers, issuers and four warps each 1370.
//
// Warp roles (768 threads):
//   warps 0, 1   MMA issuers, a buffer each (warp 0: tensor memory)
//   warp 2       weight copies, 8 blocks a slot     warp 3   activation copies and scales, 2 blocks a stage
//   warps 4-7    widen weights                      warps 8-23   epilogue: a TMEM lane quarter and 32 columns each
// Every mbarrier wait is bounded; a wait that runs out sets the CTA abort flag
// and the error word, and all roles drain and exit.
#include "experts_common.cuh"

namespace {

__device__ unsigned int g_tiles_err;

constexpr int BM = 128, kGroup = 16, kMaxGroups = 8, BN = kGroup * kMaxGroups, kBox = 64;  // kBox: sorted rows of a copy
constexpr int kStages = 3, kRawSlots = 2, kAcc = 2;
constexpr int kTmemBuf = 2 * BN, kTmemCols = kAcc * kTmemBuf;  // integers, then scales
constexpr int kThreads = 768, kWidenThreads = 128, kEpiWarps = 16, kEpiThreads = 512;
constexpr int kWidenWarp = 4, kEpiWarp = 8;  // the first of them
constexpr int kRegsLaunch = 80, kRegsCtl = 40, kRegsWiden = 56, kRegsEpi = 96;
static_assert(128 * kRegsCtl + kWidenThreads * kRegsWiden + kEpiThreads * kRegsEpi <= kRegsLaunch * kThreads, "register split");
static_assert(kRegsLaunch * kThreads <= 65536 && (kRegsLaunch + 8) * kThreads > 65536, "registers at launch");

constexpr int kPiece = 8;                      // blocks of a weight slot
constexpr int kPitchTma = 34 * kPiece;         // 272: a row's piece
constexpr int kPitchAny = kPitchTma + 32;      // 304: a row may start up to 14 bytes late
constexpr int kRawBytes = BM * kPitchAny;      // 38912
constexpr int kABytes = BM * 128, kBBytes = BN * 128;
constexpr int kScBytes = 128 * 16;             // one block's scales: 128 rows of 8 f16, of which the first is used

constexpr int kStageBytes = kABytes + kBBytes + 4 * kScBytes;  // two blocks: codes of both sides, d_w twice, d_a twice
constexpr int OFF_B = kABytes, OFF_DW = OFF_B + kBBytes, OFF_DA = OFF_DW + 2 * kScBytes;  // in a stage
constexpr int OFF_ZERO = kStages * kStageBytes;         // columns 8 .. 15 of every scale operand
constexpr int OFF_RAW = OFF_ZERO + kScBytes;
constexpr int OFF_SWAP = OFF_RAW + kRawSlots * kRawBytes;  // [16 warps][8 columns][32] f32
constexpr int OFF_CUM = OFF_SWAP + kEpiWarps * 8 * 32 * 4;  // row tiles before each expert
constexpr int kTable = 96;                              // tiles of this CTA that are looked up once
constexpr int OFF_TABLE = (OFF_CUM + (Q8_MAX_EXPERTS + 2) * 4 + 15) / 16 * 16;
constexpr int kBars = 2 * kRawSlots + 2 * kStages + 2 * kAcc;
constexpr int OFF_BAR = OFF_TABLE + kTable * 16;
constexpr int OFF_MISC = OFF_BAR + kBars * 8;           // abort flag, TMEM address, sums of the scan
constexpr int kSmemBytes = OFF_MISC + 16 + kThreads / 8 + 1024;   // + alignment slack
static_assert(OFF_BAR % 8 == 0 && kStageBytes % 1024 == 0 && OFF_RAW % 128 == 0 && kSmemBytes <= 227 * 1024, "shared memory");

struct Bars {
    uint32_t b0;
    __device__ uint32_t at(int i) const { return b0 + 8u * i; }
    __device__ uint32_t raw_full(int s) const { return at(s); }
    __device__ uint32_t raw_empty(int s) const { return at(kRawSlots + s); }
    __device__ uint32_t ab_full(int s) const { return at(2 * kRawSlots + s); }
    __device__ uint32_t ab_empty(int s) const { return at(2 * kRawSlots + kStages + s); }
    __device__ uint32_t acc_full(int s) const { return at(2 * kRawSlots + 2 * kStages + s); }
    __device__ uint32_t drain(int s) const { return acc_full(kAcc + s); }
};

// ---------------------------------------------------------------------------
// PTX
// ---------------------------------------------------------------------------
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tc_commit(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// One block's MMAs and commits, by one lane of a warp that goes on together, in a row without branches: next to other roles' code a
// branch costs some 100 cycles.  a, b: codes (the second MMA's are 32 bytes on); sa, sb: scales; `live` false: the commit to
// `full` alone.
__device__ __forceinline__ void tc_block(uint32_t d, uint64_t a, uint64_t b, uint64_t sa, uint64_t sb, uint32_t idesc, bool live,
                                         uint32_t empty, uint32_t full)
{
    asm volatile(
        "{\n\t.reg .pred one, go, no, yes;\n\t"
        "elect.sync _|one, 0xffffffff;\n\t"
        "setp.ne.and.b32 go, %9, 0, one;\n\t"
        "setp.ne.b32 no, 0, 0;\n\tsetp.eq.b32 yes, 0, 0;\n\t"
        "@go tcgen05.mma.cta_group::1.kind::f16 [%0], %2, %3, %8, no;\n\t"
        "@go tcgen05.mma.cta_group::1.kind::f16 [%0], %4, %5, %8, yes;\n\t"
        "@go tcgen05.mma.cta_group::1.kind::f16 [%1], %6, %7, %8, no;\n\t"
        "@go tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%10];\n\t"
        "@one tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%11];\n\t}" ::"r"(d),
        "r"(d + BN), "l"(a), "l"(b), "l"(a + 2), "l"(b + 2), "l"(sa), "l"(sb), "r"(idesc), "r"(static_cast<uint32_t>(live)),
        "r"(empty), "r"(full)
        : "memory");
}

// 16 columns of the thread's own lane (warp w has lanes 32 (w % 4) and on).  Valid after tc_wait_ld; tc_regs16 keeps their uses
// behind it.  This shape gives 3.3 registers a cycle and scheduler; 16x256b, which spreads a row over eight lanes, one.
__device__ __forceinline__ void tc_ld16(uint32_t taddr, uint32_t *r)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

__device__ __forceinline__ void tc_regs16(uint32_t *r)
{
    asm volatile(""
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                   "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]));
}

// The arithmetic behind 8 pairs is done before any later volatile statement: their operands' registers are free for the next load.
__device__ __forceinline__ void order8(float2 *a)
{
    asm volatile(""
                 : "+f"(a[0].x), "+f"(a[0].y), "+f"(a[1].x), "+f"(a[1].y), "+f"(a[2].x), "+f"(a[2].y), "+f"(a[3].x), "+f"(a[3].y),
                   "+f"(a[4].x), "+f"(a[4].y), "+f"(a[5].x), "+f"(a[5].y), "+f"(a[6].x), "+f"(a[6].y), "+f"(a[7].x), "+f"(a[7].y));
}

// K-major operand, 128-byte swizzle: rows of 128 bytes in 1024-byte atoms of 8 rows.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr)
{
    return static_cast<uint64_t>((addr >> 4) & 0x3fffu) | (1ull << 16) | (static_cast<uint64_t>(1024 >> 4) << 32) |
           (1ull << 46) | (2ull << 61);
}

// K-major operand of 16 columns without swizzle: rows of 16 bytes for columns 0 .. 7 at addr, the zeros for columns 8 .. 15.
__device__ __forceinline__ uint64_t scale_desc(uint32_t addr, uint32_t zeros)
{
    return static_cast<uint64_t>((addr >> 4) & 0x3fffu) | (static_cast<uint64_t>(((zeros - addr) >> 4) & 0x3fffu) << 16) |
           (static_cast<uint64_t>(128 >> 4) << 32) | (1ull << 46);
}

// D f32, A and B f16, K-major, M = 128, N = columns.
__device__ __forceinline__ constexpr uint32_t mma_desc(int columns)
{
    return (1u << 4) | (static_cast<uint32_t>(columns >> 3) << 17) | (static_cast<uint32_t>(BM >> 4) << 24);
}

// One lane of a warp that goes on together.  What only one thread may do is done inside: with operands that are the same in all lanes
// an MMA takes some 40 cycles to issue; from a thread that has left its warp, 110.
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
    return p != 0;
}

// (A build without a limit, whose waits give up at once, asks without waiting.)
__device__ __forceinline__ bool test_wait(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
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

// Bounded wait: false on the CTA's abort flag or past the limit (which raises it and the error word).
__device__ __forceinline__ bool wait_slow(uint32_t bar, uint32_t parity, volatile int *abort_flag)
{
    const uint64_t t0 = q8::globaltimer_ns();
    do {
        if (Q8_WAIT_LIMIT_NS == 0 ? test_wait(bar, parity) : try_wait(bar, parity)) return true;
        if (*abort_flag) return false;
    } while (Q8_WAIT_LIMIT_NS != 0 && q8::globaltimer_ns() - t0 <= Q8_WAIT_LIMIT_NS);
    *abort_flag = 1;
    atomicOr(&g_tiles_err, q8::kErrTimeout);
    return false;
}

// For a whole warp that goes on together.  The producers wait like this: their waits have slack.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int *abort_flag)
{
    const bool ok = (Q8_WAIT_LIMIT_NS != 0 && try_wait(bar, parity)) || wait_slow(bar, parity, abort_flag);
    return __all_sync(Q8_FULL_MASK, ok);
}

// The hand-over between MMAs and epilogue is a chain of waits, so each is as short as it can be (60 cycles when the phase is over
// already; 100 with a vote).  The issuers' for a stage: a lane whose wait ran out is not live from then on.  It issues no MMA and
// frees no stage, so that nobody fills one that is still being copied into, but goes through all its blocks.
__device__ __forceinline__ void wait_live(bool &live, uint32_t bar, uint32_t parity, volatile int *abort_flag)
{
    if (!live) return;
    if (Q8_WAIT_LIMIT_NS != 0)
        for (int i = 0; i < 64; ++i)
            if (try_wait(bar, parity)) return;
    live = wait_slow(bar, parity, abort_flag);
}

// The epilogue's for a block's accumulators, whatever the abort flag says: the issuer commits every block, if need be without
// MMAs, after waits that are bounded.  The limit is behind all of those, in time and in tries.
__device__ __forceinline__ void wait_acc(uint32_t bar, uint32_t parity, volatile int *abort_flag)
{
    if (__builtin_expect(try_wait(bar, parity), 1)) return;
    const uint64_t t0 = q8::globaltimer_ns();
    for (uint32_t i = 0; i < (1u << 20) || q8::globaltimer_ns() - t0 <= 2 * (Q8_WAIT_LIMIT_NS + Q8_DRAIN_LIMIT_NS); ++i)
        if (try_wait(bar, parity)) return;
    *abort_flag = 1;
    atomicOr(&g_tiles_err, q8::kErrTimeout);
}

// A buffer of tensor memory is handed back by a named barrier: the epilogue warps arrive, the MMA warp waits, some 25 cycles
// for a wait where an mbarrier takes 100 and its arrival as long again (3325 tokens, with tiles in two halves of 64 columns: 1370
// us, by mbarriers 1650).  Both sides pass each barrier once per block, in step: a warp arrives for block b + kAcc only behind
// its commit, which the issuer makes behind the barrier of block b.
constexpr int kHandOver = 2;  // barriers 2 and 3
__device__ __forceinline__ void acc_release(int buf)
{
    asm volatile("bar.arrive %0, %1;" ::"r"(kHandOver + buf), "n"(kEpiThreads + 32) : "memory");
}
__device__ __forceinline__ void acc_acquire(int buf)
{
    asm volatile("bar.sync %0, %1;" ::"r"(kHandOver + buf), "n"(kEpiThreads + 32) : "memory");
}

// Wait for copies or MMAs in flight before the CTA exits, whatever the abort flag says; bounded, counted from t0.
__device__ __forceinline__ void drain_bar(uint32_t bar, uint32_t parity, uint64_t t0)
{
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
    int groups;         // of 16 columns
};

__device__ __forceinline__ int groups_of(int rows) { return (rows + kGroup - 1) / kGroup; }
__device__ __forceinline__ int row_tiles_of(int rows) { return (groups_of(rows) + kMaxGroups - 1) / kMaxGroups; }

// cum[e]: row tiles of the experts before e.
__device__ __forceinline__ Tile tile_at(const q8::ExpertsArgs &a, const int *cum, int weight_tiles, int at)
{
    const int q = at / weight_tiles;
    int lo = 0, hi = a.experts;  // cum[lo] <= q < cum[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cum[mid] <= q)
            lo = mid;
        else
            hi = mid;
    }
    const int mine = cum[lo + 1] - cum[lo];
    const int rest = at - cum[lo] * weight_tiles;
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

// Tile i of this CTA, from the table where it is there.
__device__ __forceinline__ Tile tile_of(const q8::ExpertsArgs &a, const int *cum, const int4 *table, int weight_tiles, int i)
{
    if (i >= kTable) return tile_at(a, cum, weight_tiles, blockIdx.x + i * gridDim.x);
    const int4 v = table[i];
    return {v.x & 0xffff, v.y, v.z, v.w, v.x >> 16};
}

// Weight row (of an expert's) at position r of a tile; in a pair of matrices positions 32 .. 63 and 96 .. 127 are w2's.
template <bool kPair>
__device__ __forceinline__ int tile_row(int nt, int r)
{
    return kPair ? 64 * nt + 32 * (r >> 6) + (r & 31) : BM * nt + r;
}

// An MMA issuer: the blocks that go to one buffer of accumulators.  An MMA takes its operands from uniform registers; where the
// compiler sees that all lanes have the same (constants, the loops' bounds by a reduction), it computes them there.
template <int kBuf>
__device__ __forceinline__ void issue(const q8::ExpertsArgs &a, const int *cum, const int4 *table, int weight_tiles, int tiles,
                                      const Bars &B, uint32_t base, volatile int *abort_flag)
{
    const int lane = threadIdx.x & 31, nb = a.nb;
    constexpr uint32_t d = kBuf * kTmemBuf;           // all of tensor memory is this CTA's: from 0 on
    uint32_t blk = 0, done = 0, slot = 0, phase = 0;  // blocks, and this buffer's; stage and its phase
    bool live = true;
    const int n = __reduce_max_sync(Q8_FULL_MASK, tiles);
    for (int i = 0; i < n; ++i) {
        const uint32_t idesc = mma_desc(kGroup * __reduce_max_sync(Q8_FULL_MASK, tile_of(a, cum, table, weight_tiles, i).groups));
        const int u = (kBuf ^ blk) & 1;  // blocks take the buffers in turn: of a stage this one's
        for (int j = 0; j < nb; j += 2) {
            const uint32_t stage = base + slot * kStageBytes;
            const uint64_t pa = smem_desc(stage) + 4 * u, pb = smem_desc(stage + OFF_B) + 4 * u;
            // the next block's columns 8 .. 15 lie that much nearer
            constexpr uint64_t next = (kScBytes >> 4) - (static_cast<uint64_t>(kScBytes >> 4) << 16);
            const uint64_t sa = scale_desc(stage + OFF_DW, base + OFF_ZERO) + u * next;
            const uint64_t sb = scale_desc(stage + OFF_DA, base + OFF_ZERO) + u * next;
            wait_live(live, B.ab_full(slot), phase, abort_flag);
            __syncwarp();  // lanes may leave the wait one by one; the barrier below wants the whole warp (1035 -> 1041 us; only there 1046)
            if (j + u < nb) {
                if (done) acc_acquire(kBuf);
                tc_fence_after();
                tc_block(d, pa, pb, sa, sb, idesc, live, B.ab_empty(slot), B.acc_full(kBuf));
                ++done;
            } else if (lane == 0 && live) {
                arrive(B.ab_empty(slot));
            }
            __syncwarp();
            if (++slot == kStages) slot = 0, phase ^= 1u;
        }
        blk += nb;
    }
    // every MMA must have completed before its operands and TMEM go
    if (elect_one()) tc_commit(B.drain(kBuf));
    __syncwarp();
    if (done) acc_acquire(kBuf);  // the last block's
    drain_bar(B.drain(kBuf), 0, q8::globaltimer_ns());
}

// kPair: w and w2, the plane of silu(w x) * (w2 x); else w and f32 rows.  kTma: nb % 8 == 0.
template <bool kPair, bool kTma>
__global__ void __launch_bounds__(kThreads, 1)
experts_tiles_kernel(const __grid_constant__ q8::ExpertsArgs a, const __grid_constant__ CUtensorMap tmW,
                     const __grid_constant__ CUtensorMap tmW2, const __grid_constant__ CUtensorMap tmB,
                     const uint32_t *__restrict__ scales, int8_t *qs_out, uint32_t *ds_out)
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
        init(kRawSlots, kTma ? 1 : 4);  // raw_full: copied bytes, of each warp where the widening warps copy
        init(kRawSlots, 4);             // raw_empty: a warp each
        init(kStages, 6);             // ab_full: four widening warps, the copied bytes, their scales
        init(kStages, kAcc);          // ab_empty: tcgen05.commit of the issuers
        init(kAcc, 1);                // acc_full: tcgen05.commit
        init(kAcc, 1);                // drain
        q8::fence_mbar_init();
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(q8::smem_u32(tmem_slot)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    // of a scale operand's eight columns only the first is ever written
    for (int i = tid; i < kScBytes / 16; i += kThreads) {
        const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
        *reinterpret_cast<uint4 *>(sm + OFF_ZERO + 16 * i) = zero;
        for (int k = 0; k < 4 * kStages; ++k)
            *reinterpret_cast<uint4 *>(sm + (k >> 2) * kStageBytes + OFF_DW + (k & 3) * kScBytes + 16 * i) = zero;
    }
    q8::fence_proxy_async_smem();
    q8::griddep_launch_dependents();
    q8::griddep_wait();  // the offsets and the plane come from earlier kernels
    bool many = false;  // more tiles than 31 bits number: possible only where offsets fall, so that experts overlap
    {  // row tiles before each expert: two experts a thread
        int n[2], falls = 0;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            n[k] = 0;
            if (2 * tid + k < a.experts) {
                const q8::ExpertRows x = q8::expert_rows_of(a, 2 * tid + k);
                if (x.bad && blockIdx.x == 0) atomicOr(&g_tiles_err, q8::kErrData);
                falls |= x.bad;
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
        many = __syncthreads_or(falls) && a.many;
        for (int w = 0; w < warp; ++w) v += scan[w];
        if (2 * tid < a.experts) cum[2 * tid + 1] = v - n[1];
        if (2 * tid + 1 < a.experts) cum[2 * tid + 2] = v;
        if (tid == 0) cum[0] = 0;
    }
    __syncthreads();
    const int weight_tiles = kPair ? (a.n + 63) / 64 : (a.n + BM - 1) / BM;
    const int total = many ? 0 : cum[a.experts] * weight_tiles;  // else below 2^31: y would not fit otherwise
    const int tiles = (total - static_cast<int>(blockIdx.x) + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x);
    int4 *table = reinterpret_cast<int4 *>(sm + OFF_TABLE);
    if (tid < kTable && tid < tiles) {
        const Tile t = tile_at(a, cum, weight_tiles, blockIdx.x + tid * gridDim.x);
        table[tid] = make_int4(t.e | t.groups << 16, t.nt, t.row0, t.rows);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    const int nb = a.nb, stages = (nb + 1) / 2, pieces = (nb + kPiece - 1) / kPiece;

    if (warp < kWidenWarp) {
        setmaxnreg_dec<kRegsCtl>();
        if (warp == 0) {
            issue<0>(a, cum, table, weight_tiles, tiles, B, base, abort_flag);
        } else if (warp == 1) {
            issue<1>(a, cum, table, weight_tiles, tiles, B, base, abort_flag);
        } else if (warp == 2 && kTma) {
            // ------------------------------------------------------------ weights
            uint32_t n = 0;
            bool ok = true;
            for (int i = 0; i < tiles && ok; ++i) {
                const Tile t = tile_of(a, cum, table, weight_tiles, i);
                const int row = t.e * a.n + tile_row<kPair>(t.nt, 0);
                for (int s = 0; s < pieces; ++s, ++n) {
                    const int slot = n % kRawSlots;
                    ok = warp_wait(B.raw_empty(slot), ((n / kRawSlots) & 1u) ^ 1u, abort_flag);
                    if (!ok) break;
                    const uint32_t dst = base + OFF_RAW + slot * kRawBytes;
                    if (elect_one()) {
                        expect_tx(B.raw_full(slot), BM * kPitchTma);
#pragma unroll
                        for (int k = 0; k < 4; ++k)  // 32 rows each
                            q8::tma_load_2d(dst + k * 32 * kPitchTma, kPair && (k & 1) ? &tmW2 : &tmW, kPitchTma / 2 * s,
                                            row + (kPair ? 32 * (k >> 1) : 32 * k), B.raw_full(slot));
                    }
                    __syncwarp();
                }
            }
            // the last copies must have landed before the CTA exits
            const uint64_t t0 = q8::globaltimer_ns();
            for (uint32_t s = n < kRawSlots ? 0 : n - kRawSlots; s < n; ++s)
                drain_bar(B.raw_full(s % kRawSlots), (s / kRawSlots) & 1u, t0);
        } else if (warp == 3) {
            // ------------------------------------------------------------ activations and their scales: columns lane, lane + 32, ...
            uint32_t n = 0;
            bool ok = true;
            for (int at = 0; at < tiles && ok; ++at) {
                const Tile t = tile_of(a, cum, table, weight_tiles, at);
                const uint32_t *from = scales + static_cast<int64_t>(t.row0 + lane) * stages;
                uint32_t ahead[BN / 32];  // the next stage's: a load takes half as long as a stage
                auto load = [&]() {
#pragma unroll
                    for (int i = 0; i < BN / 32; ++i) ahead[i] = lane + 32 * i < t.rows ? __ldg(from + 32 * i * stages) : 0u;
                    ++from;
                };
                load();
                for (int s = 0; s < stages; ++s, ++n) {
                    const int slot = n % kStages;
                    ok = warp_wait(B.ab_empty(slot), ((n / kStages) & 1u) ^ 1u, abort_flag);
                    if (!ok) break;
                    const uint32_t dst = base + slot * kStageBytes + OFF_B;
                    if (elect_one()) {  // rows behind the expert's are the next one's, or stale: their columns are not stored
                        expect_tx(B.ab_full(slot), (t.rows > kBox ? 2 : 1) * kBox * 128);
                        q8::tma_load_2d(dst, &tmB, 64 * s, t.row0, B.ab_full(slot));
                        if (t.rows > kBox) q8::tma_load_2d(dst + kBox * 128, &tmB, 64 * s, t.row0 + kBox, B.ab_full(slot));
                    }
                    __syncwarp();
                    uint16_t *da = reinterpret_cast<uint16_t *>(sm + slot * kStageBytes + OFF_DA + lane * 16);
#pragma unroll
                    for (int i = 0; i < BN / 32; ++i) {
                        da[256 * i] = static_cast<uint16_t>(ahead[i]);
                        da[256 * i + kScBytes / 2] = static_cast<uint16_t>(ahead[i] >> 16);
                    }
                    if (s + 1 < stages) load();
                    q8::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) arrive(B.ab_full(slot));
                }
            }
            const uint64_t t0 = q8::globaltimer_ns();
            for (uint32_t s = n < kStages ? 0 : n - kStages; s < n; ++s) drain_bar(B.ab_full(s % kStages), (s / kStages) & 1u, t0);
        }
    } else if (warp < kEpiWarp) {
        setmaxnreg_dec<kRegsWiden>();
        // ---------------------------------------------------------------- widen weights: a row a thread
        const int r = tid - 32 * kWidenWarp;
        const int sw = r & 7;
        uint32_t n = 0, p = 0;  // stages and pieces done
        bool ok = true;
        // piece s of this thread's row, as many 16-byte units as hold it, where no TMA box can have it
        uint32_t copied = 0;
        auto copy = [&](const Tile &t, int s) {
            if (kTma) return;
            const int slot = copied % kRawSlots, cb = min(kPiece, nb - s * kPiece);
            const uint8_t *w = kPair && (warp & 1) ? a.w2 : a.w;
            const int64_t most = static_cast<int64_t>(a.experts) * a.n * nb * 34, whole = most & ~int64_t(15);
            const int64_t from = ((static_cast<int64_t>(t.e) * a.n + min(tile_row<kPair>(t.nt, r), a.n - 1)) * nb + s * kPiece) * 34;
            const int64_t start = from & ~int64_t(15), stop = (from + cb * 34 + 15) & ~int64_t(15);
            const int bytes = static_cast<int>(max(min(stop, whole) - start, int64_t(0)));
            uint8_t *dst = sm + OFF_RAW + slot * kRawBytes + r * kPitchAny;
            const int all = __reduce_add_sync(Q8_FULL_MASK, bytes);
            q8::fence_proxy_async_smem();  // this warp has read what lies there
            if (lane == 0) expect_tx(B.raw_full(slot), all);
            __syncwarp();
            if (bytes) q8::bulk_g2s(dst, w + start, bytes, reinterpret_cast<uint64_t *>(sm + OFF_BAR) + slot);
            if (stop > whole)  // the last bytes of the last matrix, where they do not fill 16
                for (int64_t o = max(whole, start); o < most; o += 2)
                    *reinterpret_cast<uint16_t *>(dst + (o - start)) = *reinterpret_cast<const uint16_t *>(w + o);
            ++copied;
        };
        Tile t = {}, tn = {};
        if (!kTma && tiles > 0) {
            tn = tile_of(a, cum, table, weight_tiles, 0);
            copy(tn, 0);
        }
        for (int at = 0; at < tiles && ok; ++at) {
            if (!kTma) {
                t = tn;
                if (at + 1 < tiles) tn = tile_of(a, cum, table, weight_tiles, at + 1);
            }
            const int64_t row = static_cast<int64_t>(t.e) * a.n + min(tile_row<kPair>(t.nt, r), a.n - 1);
            for (int s = 0; s < pieces && ok; ++s, ++p) {
                const int slot = p % kRawSlots;
                const uint8_t *raw = sm + OFF_RAW + slot * kRawBytes;
                if (s + 1 < pieces)  // the next piece's copies are in flight while this one is widened
                    copy(t, s + 1);
                else if (at + 1 < tiles)
                    copy(tn, 0);
                ok = warp_wait(B.raw_full(slot), (p / kRawSlots) & 1u, abort_flag);
                if (!ok) break;
                const int cb = min(kPiece, nb - s * kPiece);
#pragma unroll (kTma ? kPiece / 2 : 1)  // unrolled only where words of the piece are named at compile time
                for (int k = 0; k < kPiece / 2; ++k) {
                    if (!kTma && 2 * k >= cb) break;
                    const int st = n % kStages;
                    ok = warp_wait(B.ab_empty(st), ((n / kStages) & 1u) ^ 1u, abort_flag);
                    if (!ok) break;
                    uint8_t *out = sm + st * kStageBytes + r * 128;
                    uint16_t *dw = reinterpret_cast<uint16_t *>(sm + st * kStageBytes + OFF_DW + r * 16);
                    if (kTma) {
                        uint32_t W[20];  // 68 bytes from word 17 k on
#pragma unroll
                        for (int i = 0; i < 5; ++i) {
                            const uint4 v = *reinterpret_cast<const uint4 *>(raw + r * kPitchTma + 64 * k + 16 * i);
                            W[4 * i] = v.x, W[4 * i + 1] = v.y, W[4 * i + 2] = v.z, W[4 * i + 3] = v.w;
                        }
                        dw[0] = static_cast<uint16_t>(W[k]);
                        dw[kScBytes / 2] = static_cast<uint16_t>(W[k + 8] >> 16);
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
                            const int at_byte = static_cast<int>(from & 15) + 34 * (2 * k + b);
                            const uint32_t *src = reinterpret_cast<const uint32_t *>(raw + r * kPitchAny) + (at_byte >> 2);
                            const bool odd = at_byte & 2, there = 2 * k + b < cb;  // an odd last block: the other half is not used
                            const uint32_t sel = odd ? 0x7654u : 0x5432u;
                            uint32_t W[9];
#pragma unroll
                            for (int i = 0; i < 9; ++i) W[i] = there ? src[i] : 0u;
                            dw[b * (kScBytes / 2)] = static_cast<uint16_t>(odd ? W[0] >> 16 : W[0]);
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
                    __syncwarp();
                    if (lane == 0) arrive(B.ab_full(st));
                    ++n;
                }
                if (!ok) break;
                __syncwarp();  // the slot may be written again: by the copies of this warp, or once all four are done
                if (kTma && lane == 0) arrive(B.raw_empty(slot));
            }
        }
        // the last copies must have landed before the CTA exits
        const uint64_t t0 = q8::globaltimer_ns();
        for (uint32_t i = copied < kRawSlots ? 0 : copied - kRawSlots; i < copied; ++i)
            drain_bar(B.raw_full(i % kRawSlots), (i / kRawSlots) & 1u, t0);
    } else {
        setmaxnreg_inc<kRegsEpi>();
        // ---------------------------------------------------------------- epilogue
        const int q = warp & 3, col = 32 * ((warp - kEpiWarp) >> 2);  // lanes 32 q .., columns col ..
        const uint32_t taddr = tmem + (static_cast<uint32_t>(32 * q) << 16) + col;
        uint32_t blk = 0;
        for (int at = 0; at < tiles; ++at) {
            const Tile t = tile_of(a, cum, table, weight_tiles, at);
            const bool mine = col < t.rows;
            float2 acc[16];  // columns col + 2 i, + 1 of position 32 q + lane
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[i] = make_float2(0.0f, 0.0f);
            if (!mine) {  // in step with the others
                for (int j = 0; j < nb; ++j, ++blk) {
                    wait_acc(B.acc_full(blk % kAcc), (blk / kAcc) & 1u, abort_flag);
                    __syncwarp();
                    acc_release(blk % kAcc);
                }
            } else {
// a jump back costs some 130 cycles beside the other roles' code: 3325 tokens 1200 us with one block a round, 1070 with four,
// 1110 with eight
#pragma unroll 4
                for (int j = 0; j < nb; ++j) {
                    if (!kPair) asm volatile("" : "+r"(blk));  // else the buffers' addresses of all four blocks stay in registers
                    const uint32_t buf = taddr + (blk % kAcc) * kTmemBuf;
                    wait_acc(B.acc_full(blk % kAcc), (blk / kAcc) & 1u, abort_flag);
                    __syncwarp();
                    tc_fence_after();
#pragma unroll
                    for (int x = 0; x < 2; ++x) {  // 16 columns at a time: four warps a scheduler hide each other's loads
                        uint32_t p[16], c[16];
                        tc_ld16(buf + 16 * x, p);
                        tc_ld16(buf + BN + 16 * x, c);
                        tc_wait_ld();
                        tc_regs16(p), tc_regs16(c);
                        if (x == 1) {
                            tc_fence_before();
                            acc_release(blk % kAcc);
                        }
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            acc[8 * x + i] =
                                __ffma2_rn(make_float2(__uint_as_float(c[2 * i]), __uint_as_float(c[2 * i + 1])),
                                           make_float2(__uint_as_float(p[2 * i]), __uint_as_float(p[2 * i + 1])), acc[8 * x + i]);
                        order8(acc + 8 * x);
                    }
                    ++blk;
                }
            }
            const bool ok = __all_sync(Q8_FULL_MASK, !*abort_flag);
            // of the 32 columns from c0 on
            auto valid = [&](int c0) {
                return __ballot_sync(Q8_FULL_MASK, c0 + lane < t.rows && q8::source_row(a, t.row0 + c0 + lane) >= 0);
            };
            if (!kPair) {
                if (!ok || !mine) continue;  // after an abort the tiles are walked, not stored
                const int row = BM * t.nt + 32 * q + lane;
                const uint32_t m = valid(col);
                float *out = a.out + static_cast<int64_t>(t.row0 + col) * a.ld + row;
                if (row < a.n) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        if ((m >> (2 * i)) & 1u) *out = acc[i].x;
                        out += a.ld;
                        if ((m >> (2 * i + 1)) & 1u) *out = acc[i].y;
                        out += a.ld;
                        asm volatile("" : "+l"(out));  // one address after the other: all at once would not fit beside acc
                    }
                }
            } else {
                if (epi_any(!ok)) continue;  // all of them, so that none waits for another below
                // warp q even has 32 gate channels, q odd the same up channels, of 32 columns: even keeps the first 16 columns
                const int up = q & 1;
                float *box = reinterpret_cast<float *>(sm + OFF_SWAP) + (warp - kEpiWarp) * 256 + lane;
                const float *from = reinterpret_cast<float *>(sm + OFF_SWAP) + ((warp - kEpiWarp) ^ 1) * 256 + lane;
                float v[16];
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    if (mine) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float2 g = acc[4 * x + i], u = acc[8 + 4 * x + i];  // this and the other half's columns
                            box[32 * (2 * i)] = up ? g.x : u.x;
                            box[32 * (2 * i + 1)] = up ? g.y : u.y;
                        }
                    }
                    epi_sync();
                    if (mine) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float2 g = acc[4 * x + (i >> 1)], u = acc[8 + 4 * x + (i >> 1)];
                            const float own = up ? (i & 1 ? u.y : u.x) : (i & 1 ? g.y : g.x), other = from[32 * i];
                            v[8 * x + i] = up ? q8::silu_mul(other, own) : q8::silu_mul(own, other);
                        }
                    }
                    if (x == 0) epi_sync();
                }
                if (!mine) continue;
                const int c0 = col + 16 * up, ch = 64 * t.nt + 32 * (q >> 1);
                const uint32_t m = valid(c0);
                if (ch >= a.n) continue;
                // lanes i and i + 16 get column c0 + i's largest value (NaN counts where all are) and encode its block's scale
                float top = 0.0f;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    float x;
                    asm("redux.sync.max.abs.f32 %0, %1, 0xffffffff;" : "=f"(x) : "f"(v[i]));
                    if ((lane & 15) == i) top = x;
                }
                const float d = q8::q8_block_d(top);
                const float di = q8::q8_block_di(d);
                // columns with rows whose scale is subnormal, infinite or NaN
                const uint32_t odd = __ballot_sync(Q8_FULL_MASK, !q8::block_rounds_by_add(d)) & m & 0xffffu;
                int sum = 0;
                int8_t *out = qs_out + static_cast<int64_t>(t.row0 + c0) * a.n + ch + lane;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int code = q8::q8_code_bits(v[i], __shfl_sync(Q8_FULL_MASK, di, i)), all = __reduce_add_sync(Q8_FULL_MASK, code);
                    if ((lane & 15) == i) sum = all;
                    if ((m >> i) & 1u) *out = static_cast<int8_t>(code);
                    out += a.n;
                    asm volatile("" : "+l"(out));
                }
                if (odd) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int code = q8::q8_code(v[i], __shfl_sync(Q8_FULL_MASK, di, i)), all = __reduce_add_sync(Q8_FULL_MASK, code);
                        if (!((odd >> i) & 1u)) continue;
                        if ((lane & 15) == i) sum = all;
                        out[static_cast<int64_t>(i - 16) * a.n] = static_cast<int8_t>(code);
                    }
                }
                if (lane < 16 && ((m >> lane) & 1u))
                    ds_out[static_cast<int64_t>(t.row0 + c0 + lane) * (a.n >> 5) + (ch >> 5)] = q8::q8_dsword(d, sum);
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
    }
}

// The experts' rows' codes as f16, out [pairs][16 chunks], 16 codes a thread and round; and their scales, two blocks a word.
__global__ void __launch_bounds__(256)
experts_sort_plane_kernel(const __grid_constant__ q8::ExpertsArgs a, uint4 *__restrict__ out, uint32_t *__restrict__ scales)
{
    q8::griddep_launch_dependents();
    q8::griddep_wait();
    const int chunks = 2 * a.nb, words = (a.nb + 1) / 2, lane = threadIdx.x & 31;  // of a row
    const int first = min(max(a.offsets[0], 0), a.pairs), rows = min(max(a.offsets[a.experts], 0), a.pairs);
    const int warps = gridDim.x * (blockDim.x / 32);
    // in 64 bits: a step behind the last row may pass 31
    for (int64_t at = static_cast<int64_t>(first) + blockIdx.x * (blockDim.x / 32) + (threadIdx.x >> 5); at < rows; at += warps) {
        const int r = static_cast<int>(at);
        int64_t src = q8::source_row(a, r);
        if (src < 0) {  // out of range: any, it is not stored
            src = 0;
            if (lane == 0) atomicOr(&g_tiles_err, q8::kErrData);
        }
        const uint32_t *ds = a.ds + src * a.nb;
        for (int i = lane; i < words; i += 32) {
            const uint32_t d0 = __ldg(ds + 2 * i), d1 = 2 * i + 1 < a.nb ? __ldg(ds + 2 * i + 1) : 0u;
            scales[static_cast<int64_t>(r) * words + i] = __byte_perm(d0, d1, 0x5410);
        }
        const uint4 *from = reinterpret_cast<const uint4 *>(a.qs) + src * chunks;
        uint4 *to = out + static_cast<int64_t>(r) * 2 * chunks;
#pragma unroll 4
        for (int i = lane; i < chunks; i += 32) {
            const uint4 v = __ldg(from + i);
            uint4 o0, o1;
            q8::i8x4_to_f16x4(v.x, o0.x, o0.y);
            q8::i8x4_to_f16x4(v.y, o0.z, o0.w);
            q8::i8x4_to_f16x4(v.z, o1.x, o1.y);
            q8::i8x4_to_f16x4(v.w, o1.z, o1.w);
            to[2 * i] = o0;
            to[2 * i + 1] = o1;
        }
    }
}

template <bool kPair, bool kTma>
int launch(const q8::ExpertsArgs &a, const CUtensorMap &mw, const CUtensorMap &mw2, const CUtensorMap &mb, const uint32_t *scales, unsigned grid,
           int8_t *qs_out, uint32_t *ds_out, int slot, cudaStream_t s)
{
    // the epilogue's registers come from those that the CTA is launched with: built with fewer, it would wait for them for ever
    static const bool registers = [] {
        cudaFuncAttributes f = {};
        return cudaFuncGetAttributes(&f, experts_tiles_kernel<kPair, kTma>) == cudaSuccess && f.numRegs >= kRegsLaunch;
    }();
    if (!registers || !q8::set_max_dynamic_smem(reinterpret_cast<const void *>(experts_tiles_kernel<kPair, kTma>), kSmemBytes, slot))
        return Q8_ERR_LAUNCH;
    return q8::launch_pdl(experts_tiles_kernel<kPair, kTma>, dim3(grid), dim3(kThreads), kSmemBytes, s, a, mw, mw2, mb, scales,
                          qs_out, ds_out);
}

} // namespace

namespace q8 {

size_t experts_tiles_workspace(int64_t k, int64_t pairs)
{
    return static_cast<size_t>(pairs) * k * 2 + static_cast<size_t>(pairs) * ((k / 32 + 1) / 2) * 4;  // codes, scales
}

int experts_tiles_launch(const ExpertsArgs &args, int8_t *qs_out, uint32_t *ds_out, void *workspace, cudaStream_t s)
{
    ExpertsArgs a = args;
    const bool pair = a.w2 != nullptr, tma = a.nb % kPiece == 0;
    CUtensorMap mw = {}, mw2 = {}, mb = {};
    const uint64_t wrows = static_cast<uint64_t>(a.experts) * a.n, pitch = static_cast<uint64_t>(a.nb) * 34;
    if (tma && (!make_map_2d(&mw, CU_TENSOR_MAP_DATA_TYPE_UINT16, a.w, pitch / 2, wrows, pitch, kPitchTma / 2, 32,
                             CU_TENSOR_MAP_SWIZZLE_NONE) ||
                (pair && !make_map_2d(&mw2, CU_TENSOR_MAP_DATA_TYPE_UINT16, a.w2, pitch / 2, wrows, pitch, kPitchTma / 2, 32,
                                      CU_TENSOR_MAP_SWIZZLE_NONE))))
        return Q8_ERR_LAUNCH;
    const uint64_t row = static_cast<uint64_t>(a.nb) * 64;  // bytes of f16
    if (!make_map_2d(&mb, CU_TENSOR_MAP_DATA_TYPE_UINT16, workspace, row / 2, static_cast<uint64_t>(a.pairs), row, 64, kBox,
                     CU_TENSOR_MAP_SWIZZLE_128B))
        return Q8_ERR_LAUNCH;
    uint32_t *scales = reinterpret_cast<uint32_t *>(static_cast<char *>(workspace) + static_cast<int64_t>(a.pairs) * row);
    const int sms = device_sm_count();
    const int64_t ctas = (a.pairs + 7) / 8, cap = static_cast<int64_t>(sms) * 8;
    const int st = launch_pdl(experts_sort_plane_kernel, dim3(static_cast<unsigned>(ctas < cap ? ctas : cap)), dim3(256), 0, s, a,
                              static_cast<uint4 *>(workspace), scales);
    if (st != Q8_OK) return st;
    const int64_t weight_tiles = pair ? (a.n + 63) / 64 : (a.n + BM - 1) / BM;
    a.many = (a.experts / 2 + 1) * (static_cast<int64_t>(a.pairs) / BN + 1) * weight_tiles > INT32_MAX;
    const int64_t most = (a.pairs / BN + (a.experts < a.pairs ? a.experts : a.pairs)) * weight_tiles;
    const unsigned grid = static_cast<unsigned>(most < sms ? most : sms);
    if (pair) return tma ? launch<true, true>(a, mw, mw2, mb, scales, grid, qs_out, ds_out, 48, s)
                         : launch<true, false>(a, mw, mw2, mb, scales, grid, qs_out, ds_out, 49, s);
    return tma ? launch<false, true>(a, mw, mw2, mb, scales, grid, qs_out, ds_out, 50, s)
               : launch<false, false>(a, mw, mw2, mb, scales, grid, qs_out, ds_out, 51, s);
}

unsigned int *experts_tiles_error_word()
{
    void *p = nullptr;
    return cudaGetSymbolAddress(&p, g_tiles_err) == cudaSuccess ? static_cast<unsigned int *>(p) : nullptr;
}

} // namespace q8
