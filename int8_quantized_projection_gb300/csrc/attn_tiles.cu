// attn_tiles.cu -- q8_tree_attention for more than 16 packed rows a unit:
// 128 rows x 128 keys a tile on the 5th-generation tensor cores.
//
//     S = Q K^T,  P = 2^(S * scale - m),  O += P V,  l += rowsum(P)
//
// f32 precision on f16 MMAs: q and the weights are sums of two f16 parts
// (22 bits), both parts are multiplied with the same key or value tile into
// the same f32 accumulator, so a tile costs 2 * (D/16 + 8) MMAs of K = 16.
//
// Two softmax warpgroups take the tiles in turn, each with a score buffer and
// an accumulator of its own in tensor memory (S0, S1, O0, O1: 512 columns for
// D = 128) and its own (m, l), joined once per piece: they never wait for each
// other, and while one computes weights the tensor core works on the other's
// scores or product.  A thread owns a row, so maxima and sums need no
// shuffles; P overwrites S in place (per 32 keys 16 columns of high parts
// and 16 of low parts) and is the second product's A operand from tensor memory.  V is used
// as it lies in the cache ([key][dim], N-major).
//
// Roles: warp 0 copies K and V tiles (one TMA box per run of keys that share
// a page), warp 1 issues the MMAs, warps 4-11 are the softmax warpgroups; for
// int8, warps 12-15 widen the codes to f16 tiles (exact), a key's scale
// multiplies its score column and a value's scale its weight column.
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
constexpr int kHead = 3;             // what a unit costs beside its tiles, in tiles
constexpr float kWeightBits = 6.0f;  // weights are 2^(s - m + 6): below 2^14 while m may lag by 2^8
constexpr float kRaise = 8.0f;
constexpr int kScaleSlots = 4;

template <int D, bool kInt8>
struct Lay {
    static constexpr int kThreads = kInt8 ? 512 : 384;
    // registers per thread after setmaxnreg; their sum is the launch's
    static constexpr int kRegsLaunch = kInt8 ? 128 : 168;
    static constexpr int kRegsSoft = kInt8 ? 176 : 208, kRegsCtl = kInt8 ? 56 : 88, kRegsConv = 104;
    static_assert(256 * kRegsSoft + 128 * kRegsCtl + (kInt8 ? 128 * kRegsConv : 0) <= kThreads * kRegsLaunch, "registers");

    static constexpr int kMat = 128 * D * 2;            // a 128-row f16 tile
    static constexpr int kBufs = kInt8 ? 1 : 2;         // f16 tiles of K, and of V
    static constexpr int offQ = 0;                      // high parts, low parts
    // at a piece's end the finished rows pass through here: D/2 values and 16 bytes of padding per row and warpgroup
    static constexpr int kOutRow = D / 2 * 4 + 16;
    static constexpr int offK = offQ + 2 * kMat + 4096;
    static_assert(2 * 128 * kOutRow <= 2 * kMat + 4096, "rows out");
    static constexpr int offV = offK + kBufs * kMat;
    static constexpr int offRaw = offV + kBufs * kMat;  // int8: two stages of K codes, two of V codes
    static constexpr int kRaw = 128 * D;
    static constexpr int offScale = offRaw + (kInt8 ? 4 * kRaw : 0);   // slots of 128 k scales, 128 v scales
    static constexpr int offRow = offScale + (kInt8 ? kScaleSlots * 1024 : 0);
    // per row: q scale; m, l and 2^e of each warpgroup
    static constexpr int offBar = offRow + 128 * 4 * 7;
    // barriers, by index
    static constexpr int bKf = 0, bKe = 2, bVf = 4, bVe = 6;      // f16 tiles: full, empty
    static constexpr int bRKf = 8, bRKe = 10, bRVf = 12, bRVe = 14;  // int8 codes
    static constexpr int bCf = 16, bCe = 20;                      // int8 scales
    static constexpr int bSf = 24, bPf = 26, bQf = 28, bOf = 29, bDrain = 30, kBars = 31;
    static constexpr int offMisc = offBar + kBars * 8 + 8;
    static constexpr int offPre = offMisc + 32;
    static int smem(int batch) { return offPre + (batch + 1) * 4 + 1024; }
    static_assert(offPre + (Q8_KV_MAX_BATCH + 1) * 4 + 1024 <= 227 * 1024, "shared memory");
    static constexpr int kColO = 256;                   // S0, S1 at 0, 128; O0, O1 from here
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

// 32 columns of this thread's lane; valid after tc_wait_ld and tc_regs32.
__device__ __forceinline__ void tc_ld32(uint32_t taddr, uint32_t *r)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
        "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}

__device__ __forceinline__ void tc_regs32(uint32_t *r)
{
#pragma unroll
    for (int i = 0; i < 32; i += 16)
        asm volatile(""
                     : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), "+r"(r[i + 5]),
                       "+r"(r[i + 6]), "+r"(r[i + 7]), "+r"(r[i + 8]), "+r"(r[i + 9]), "+r"(r[i + 10]), "+r"(r[i + 11]),
                       "+r"(r[i + 12]), "+r"(r[i + 13]), "+r"(r[i + 14]), "+r"(r[i + 15]));
}

__device__ __forceinline__ void tc_st16(uint32_t taddr, const uint32_t *r)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
            taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
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
        atomicOr(&g_tiles_err, q8::kKvErrTimeout);
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
            atomicOr(&g_tiles_err, q8::kKvErrTimeout);
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
            atomicOr(&g_tiles_err, q8::kKvErrTimeout);
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

// One CTA's stretch of the line, piece by piece; every role walks it alike.
struct Walk {
    int pos, begin, end;  // next place; the stretch
    Unit u;               // before the first piece: the unit at `begin`
    int t0, n, kend;      // first tile, tiles, keys end
    bool first;           // the stretch begins in this unit

    __device__ __forceinline__ bool next(const AttnArgs &a, const int *pre)
    {
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

// One block of the plane: 32 consecutive values of a finished row in one
// thread, encoded by the steps of q8_encode8 without its shuffles.
__device__ __forceinline__ void encode32(const AttnArgs &a, long long at, const float (&o)[32])
{
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) m = fmaxf(m, fabsf(o[i]));
    const float d = q8::q8_block_d(m), di = q8::q8_block_di(d);
    int sum = 0;
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int c0 = q8::q8_code(o[4 * i], di), c1 = q8::q8_code(o[4 * i + 1], di);
        const int c2 = q8::q8_code(o[4 * i + 2], di), c3 = q8::q8_code(o[4 * i + 3], di);
        sum += c0 + c1 + c2 + c3;
        w[i] = q8::pack4(c0, c1, c2, c3);
    }
    uint4 *dst = reinterpret_cast<uint4 *>(a.qs + at);
    dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
    dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
    a.ds[at / 32] = q8::q8_dsword(d, sum);
}

template <int D, bool kInt8>
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
    float *s_row = reinterpret_cast<float *>(sm + L::offRow);  // [0]: q scale, [1 + 3g ..]: m, l, 2^e of warpgroup g
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
            if (i == L::bCe || (i > L::bCe && i < L::bCe + kScaleSlots)) count = 128;  // the tile's warpgroup
            if (i >= L::bPf && i < L::bPf + 2) count = 128;
            if (i == L::bQf) count = 256;
            if (kInt8 && (i == L::bKf || i == L::bVf)) count = 128;  // written by the widening warps
            if ((i >= L::bRKe && i < L::bRKe + 2) || (i >= L::bRVe && i < L::bRVe + 2)) count = 128;
            q8::mbar_init(bars + i, count);
        }
        q8::fence_mbar_init();
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(q8::smem_u32(tmem_slot)),
                     "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    q8::griddep_launch_dependents();
    q8::griddep_wait();
    bool bad_data = !q8::attn_line<kRows, kTile, kHead, L::kThreads>(a, pre);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int total = pre[a.batch];
    const int per = max(1, (total + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x));
    const int cta = blockIdx.x;
    const int s0 = min(total, cta * per);
    Walk w;
    w.pos = w.begin = s0;
    w.end = min(total, s0 + per);
    if (w.pos < w.end) w.u = q8::attn_unit<kRows, kTile, kHead>(a, pre, w.pos);

    if (warp < 4) {
        setmaxnreg_dec<L::kRegsCtl>();
        if (warp == 0) {
            // -------------------------------------------------------- copies: K and V tiles, key scales
            int T = 0, nk = 0, nv = 0, nc = 0;  // tiles so far; copies issued of each kind
            bool ok = true;
            while (ok && w.next(a, pre)) {
                const int boxes = kTile / box;
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
                    const int ahead = fetch(i + 1);
                    const int key0 = (w.t0 + i) * kTile;
                    const int nb = min(boxes, (w.kend - key0 + box - 1) / box);
                    const int st = T & 1;
                    const uint32_t par = static_cast<uint32_t>(T >> 1) & 1u;
                    constexpr int kRowBytes = kInt8 ? D : 128;  // of a box row
                    constexpr int kHalves = kInt8 ? 1 : D / 64;
                    auto copy = [&](int full, int empty, const CUtensorMap *map, int off) {
                        if (!warp_wait(bar(empty + st), par ^ 1u, abort_flag)) return false;
                        if (lane == 0) q8::mbar_arrive_expect_tx(bars + full + st, nb * box * kRowBytes * kHalves);
                        __syncwarp();
                        if (lane < nb) {
#pragma unroll
                            for (int h = 0; h < kHalves; ++h)
                                q8::tma_load_2d(base + off + h * 16384 + lane * box * kRowBytes, map, h * 64, row,
                                                bar(full + st));
                        }
                        return true;
                    };
                    if (kInt8) {
                        const int cs = T % kScaleSlots;
                        ok = warp_wait(bar(L::bCe + cs), (static_cast<uint32_t>(T / kScaleSlots) & 1u) ^ 1u, abort_flag);
                        if (!ok) break;
                        if (lane == 0) q8::mbar_arrive_expect_tx(bars + L::bCf + cs, nb * box * 8);
                        __syncwarp();
                        if (lane < nb) {
                            uint8_t *dst = sm + L::offScale + cs * 1024 + lane * box * 4;
                            q8::bulk_g2s(dst, a.ks + row, box * 4, bars + L::bCf + cs);
                            q8::bulk_g2s(dst + 512, a.vs + row, box * 4, bars + L::bCf + cs);
                        }
                        nc = T + 1;
                        ok = copy(L::bRKf, L::bRKe, &mk, L::offRaw + st * L::kRaw);
                        if (!ok) break;
                        nk = T + 1;
                        ok = copy(L::bRVf, L::bRVe, &mv, L::offRaw + (2 + st) * L::kRaw);
                        if (!ok) break;
                        nv = T + 1;
                    } else {
                        ok = copy(L::bKf, L::bKe, &mk, L::offK + st * L::kMat);
                        if (!ok) break;
                        nk = T + 1;
                        ok = copy(L::bVf, L::bVe, &mv, L::offV + st * L::kMat);
                        if (!ok) break;
                        nv = T + 1;
                    }
                    row = ahead;
                }
            }
            // the last copies must have landed before the CTA exits
            for (int t = max(0, nk - 2); t < nk; ++t)
                drain_bar(bar((kInt8 ? L::bRKf : L::bKf) + (t & 1)), static_cast<uint32_t>(t >> 1) & 1u);
            for (int t = max(0, nv - 2); t < nv; ++t)
                drain_bar(bar((kInt8 ? L::bRVf : L::bVf) + (t & 1)), static_cast<uint32_t>(t >> 1) & 1u);
            for (int t = max(0, nc - kScaleSlots); t < nc; ++t)
                drain_bar(bar(L::bCf + t % kScaleSlots), static_cast<uint32_t>(t / kScaleSlots) & 1u);
        } else if (warp == 1) {
            // -------------------------------------------------------- MMAs
            constexpr uint32_t iS = idesc_f16(kTile, false), iO = idesc_f16(D, true);
            const uint32_t one = lane == 0;
            const uint32_t tm = __shfl_sync(Q8_FULL_MASK, tmem, 0);
            int T = 0;
            uint32_t piece = 0, pph[2] = {0, 0};
            bool ok = true;
            auto scores = [&](int t, int b) {  // tile t of the CTA into score buffer b
                const int st = t % L::kBufs;
                if (!warp_wait(bar(L::bKf + st), static_cast<uint32_t>(t / L::kBufs) & 1u, abort_flag)) return false;
                tc_fence_after();
                const uint64_t k = desc128(base + L::offK + st * L::kMat, 16, 1024);
#pragma unroll
                for (int part = 1; part >= 0; --part) {  // low parts first: the accumulator is small while they are added
                    const uint64_t q = desc128(base + L::offQ + part * L::kMat, 16, 1024);
#pragma unroll
                    for (int s = 0; s < D / 16; ++s) {
                        const uint32_t o = ((s >> 2) * 16384 + (s & 3) * 32) >> 4;
                        mma_ss(tm + 128u * b, q + o, k + o, iS, part == 0 || s > 0, one);
                    }
                }
                if (one) {
                    tc_commit(bar(L::bKe + st));
                    tc_commit(bar(L::bSf + b));
                }
                __syncwarp();
                return true;
            };
            while (ok && w.next(a, pre)) {
                ok = warp_wait(bar(L::bQf), piece & 1u, abort_flag);
                if (!ok) break;
                tc_fence_after();
                for (int i = 0; ok && i < min(2, w.n); ++i) ok = scores(T + i, i);
                for (int i = 0; ok && i < w.n; ++i) {
                    const int t = T + i, b = i & 1, st = t % L::kBufs;
                    ok = warp_wait(bar(L::bVf + st), static_cast<uint32_t>(t / L::kBufs) & 1u, abort_flag) &&
                         warp_wait(bar(L::bPf + b), b ? pph[1] : pph[0], abort_flag);
                    if (!ok) break;
                    if (b) pph[1] ^= 1u; else pph[0] ^= 1u;
                    tc_fence_after();
                    const uint64_t v = desc128(base + L::offV + st * L::kMat, 16384, 1024);
                    const uint32_t d = tm + L::kColO + D * b, p = tm + 128u * b;
#pragma unroll
                    for (int part = 1; part >= 0; --part)
#pragma unroll
                        for (int s = 0; s < kTile / 16; ++s)
                            mma_ts(d, p + 32u * (s >> 1) + 8u * (s & 1) + 16u * part, v + ((2048u * s) >> 4), iO,
                                   part == 0 || s > 0 || i >= 2, one);
                    if (one) tc_commit(bar(L::bVe + st));
                    __syncwarp();
                    if (i + 2 < w.n) ok = scores(t + 2, b);
                }
                if (!ok) break;
                if (one) tc_commit(bar(L::bOf));
                __syncwarp();
                T += w.n;
                ++piece;
            }
            // every MMA issued must be complete before tensor memory is freed
            if (one) {
                tc_commit(bar(L::bDrain));
                drain_bar(bar(L::bDrain), 0);
            }
        }
        __syncwarp();
    } else if (warp < 12) {
        setmaxnreg_inc<L::kRegsSoft>();
        // ------------------------------------------------------------ softmax: a thread owns row r of the unit's tile
        const int wg = (warp - 4) >> 2, r = (warp & 3) * 32 + lane;
        const uint32_t tl = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
        const uint32_t ts = tl + 128u * wg, to = tl + L::kColO + D * wg;
        int T = 0;
        uint32_t piece = 0, sph = 0;
        if (tid == 128) a.desc[2 * cta + 1].w = 0;  // no first piece yet
        // Q: a warp per row (D = 128) or two rows (D = 64), eight warps.  A unit's rows are in registers before the unit
        // before it is finished.
        constexpr int kPer = D == 128 ? 1 : 2, kLanes = 32 / kPer, kLoads = 16 / kPer;
        const int sub = lane % kLanes;
        auto q_row = [&](int j) { return ((warp - 4) + 8 * j) * kPer + lane / kLanes; };
        float4 x[kLoads];
        auto load_q = [&](const Unit &u) {
            const q8::RowMap map(a, u.rt * kRows);
            const int rows = u.fresh * a.group - u.rt * kRows;
#pragma unroll
            for (int j = 0; j < kLoads; ++j) {
                const int rr = q_row(j);
                x[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (rr < rows) x[j] = __ldg(reinterpret_cast<const float4 *>(a.q + map.at(a, u, rr, D)) + sub);
            }
        };
        bool more = w.next(a, pre);
        if (more) load_q(w.u);
        while (more) {
            const Unit &u = w.u;
            const int rows = u.fresh * a.group, row0 = u.rt * kRows;
            {
                // the row's largest value goes to [1, 2), the sign of the scale into q
                const float sign = a.scale < 0.0f ? -1.0f : 1.0f;
#pragma unroll
                for (int j = 0; j < kLoads; ++j) {
                    const int rr = q_row(j);
                    float m = fmaxf(fmaxf(fabsf(x[j].x), fabsf(x[j].y)), fmaxf(fabsf(x[j].z), fabsf(x[j].w)));
#pragma unroll
                    for (int o = 1; o < kLanes; o <<= 1) m = fmaxf(m, __shfl_xor_sync(Q8_FULL_MASK, m, o));
                    const int e = min(126, max(-126, static_cast<int>(__float_as_uint(m) >> 23) - 127));
                    const float down = q8::pow2(-e) * sign;
                    uint2 hi, lo;
                    q8::split_f16(x[j].x * down, x[j].y * down, hi.x, lo.x);
                    q8::split_f16(x[j].z * down, x[j].w * down, hi.y, lo.y);
                    const int off = (sub >> 4) * 16384 + rr * 128 + ((((sub & 15) >> 1) ^ (rr & 7)) << 4) + (sub & 1) * 8;
                    *reinterpret_cast<uint2 *>(sm + L::offQ + off) = hi;
                    *reinterpret_cast<uint2 *>(sm + L::offQ + L::kMat + off) = lo;
                    if (sub == 0) s_row[rr] = q8::pow2(e) * fabsf(a.scale);
                }
                q8::fence_proxy_async_smem();
                tc_fence_before();  // the last piece's tensor-memory loads are done
                arrive(bar(L::bQf));
                soft_sync();
            }
            const float qs = s_row[r];
            const q8::RowSight sight = q8::attn_sight(a, u, row0 + r);
            const int all_see = u.cached + (a.masks ? 0 : row0 / a.group + 1);  // keys below are seen by every row
            float m = -INFINITY, l = 0.0f, ie = 1.0f;
            int e = 0;
            bool ok = true;
            for (int i = wg; i < w.n; i += 2) {
                if (!warp_wait(bar(L::bSf + wg), sph, abort_flag)) {
                    ok = false;
                    break;
                }
                sph ^= 1u;
                const int t = T + i, key0 = (w.t0 + i) * kTile;
                const bool masked = key0 + kTile > min(all_see, w.kend);
                const float *sc = reinterpret_cast<const float *>(sm + L::offScale + (t % kScaleSlots) * 1024);
                if (kInt8 && !warp_wait(bar(L::bCf + t % kScaleSlots), static_cast<uint32_t>(t / kScaleSlots) & 1u, abort_flag)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                // Two passes over the scores, 32 columns at a time: the maximum, then the weights, which go back to
                // the columns their scores came from (16 of high parts, 16 of low parts).  Holding all 128 scores
                // between the passes would take 128 registers; reading tensor memory twice is cheaper.
                auto weigh = [&](auto hidden) {
                    constexpr bool kMasked = decltype(hidden)::value;
                    uint32_t see[4];  // the keys this row sees, a bit each
                    if constexpr (kMasked) {
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const int k = key0 + 32 * c, below = max(0, min(32, sight.all - k));
                            see[c] = below == 32 ? ~0u : (1u << below) - 1u;
                            const int sh = u.cached - k;  // bit b of the mask is key k + sh + b
                            if (sh >= 0 && sh < 32) see[c] |= static_cast<uint32_t>(sight.mask << sh);
                            else if (sh < 0 && sh > -64) see[c] |= static_cast<uint32_t>(sight.mask >> -sh);
                        }
                    }
                    uint32_t s[2][32];
                    // int8: 32 scores times their keys' scales
                    auto key_scales = [&](uint32_t *x, int c) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const float4 k4 = *reinterpret_cast<const float4 *>(sc + 32 * c + 4 * j);
                            const float2 y = __fmul2_rn(
                                make_float2(__uint_as_float(x[4 * j]), __uint_as_float(x[4 * j + 1])), make_float2(k4.x, k4.y));
                            const float2 z = __fmul2_rn(
                                make_float2(__uint_as_float(x[4 * j + 2]), __uint_as_float(x[4 * j + 3])), make_float2(k4.z, k4.w));
                            x[4 * j] = __float_as_uint(y.x), x[4 * j + 1] = __float_as_uint(y.y);
                            x[4 * j + 2] = __float_as_uint(z.x), x[4 * j + 3] = __float_as_uint(z.y);
                        }
                    };
                    float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
                    for (int c = 0; c < 4; c += 2) {
                        tc_ld32(ts + 32 * c, s[0]);
                        tc_ld32(ts + 32 * c + 32, s[1]);
                        tc_wait_ld();
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            tc_regs32(s[h]);
                            if (kInt8) key_scales(s[h], c + h);
                            if constexpr (kMasked) {
#pragma unroll
                                for (int j = 0; j < 32; ++j)
                                    if ((see[c + h] >> j) & 1u) mx[h] = fmaxf(mx[h], __uint_as_float(s[h][j]));
                            } else {
#pragma unroll
                                for (int j = 0; j < 32; j += 2)
                                    mx[h] = fmaxf(fmaxf(mx[h], __uint_as_float(s[h][j])), __uint_as_float(s[h][j + 1]));
                            }
                        }
                    }
                    float big = 0.0f;  // int8: the largest value scale that the row sees
                    if (kInt8) {
                        if constexpr (!kMasked) {  // the same keys for every row: four a lane
                            const float4 v4 = *reinterpret_cast<const float4 *>(sc + 128 + 4 * lane);
                            const float vv[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                if (vv[j] <= 3.4028235e38f) big = fmaxf(big, vv[j]);
#pragma unroll
                            for (int o = 1; o < 32; o <<= 1) big = fmaxf(big, __shfl_xor_sync(Q8_FULL_MASK, big, o));
                        } else {
#pragma unroll
                            for (int c = 0; c < 4; ++c)
#pragma unroll 8
                                for (int j = 0; j < 32; ++j) {
                                    const float x = sc[128 + 32 * c + j];
                                    if (((see[c] >> j) & 1u) && x <= 3.4028235e38f) big = fmaxf(big, x);
                                }
                        }
                    }
                    float top = fmaxf(mx[0], mx[1]);
                    if (top != -INFINITY) top *= qs;
                    bool raise = top > m + kRaise;
                    if (kInt8) raise |= big * ie > 1.0f;
                    if (i == wg) {  // the first tile: nothing accumulated yet
                        m = top;
                        if (kInt8) {
                            e = min(126, max(-126, static_cast<int>(__float_as_uint(big) >> 23) - 126));
                            ie = q8::pow2(-e);
                        }
                    } else if (__any_sync(Q8_FULL_MASK, raise)) {
                        const float mn = fmaxf(m, top);
                        float f = mn == m ? 1.0f : q8::exp2_approx(m - mn);
                        l *= f;
                        m = mn;
                        if (kInt8) {
                            const int en = min(126, max(e, static_cast<int>(__float_as_uint(big) >> 23) - 126));
                            f = e - en < -126 ? 0.0f : f * q8::pow2(e - en);
                            e = en;
                            ie = q8::pow2(-e);
                        }
                        // the products so far are complete: their MMAs came before this tile's scores
#pragma unroll 1
                        for (int c = 0; c < D; c += 32) {
                            tc_ld32(to + c, s[0]);
                            tc_wait_ld();
                            tc_regs32(s[0]);
#pragma unroll
                            for (int j = 0; j < 32; ++j) s[0][j] = __float_as_uint(__uint_as_float(s[0][j]) * f);
                            tc_st16(to + c, s[0]);
                            tc_st16(to + c + 16, s[0] + 16);
                        }
                    }
                    const float ref = m == -INFINITY ? 0.0f : m - kWeightBits;
                    const float2 q2 = make_float2(qs, qs), r2 = make_float2(-ref, -ref);
                    float2 sum = make_float2(0.0f, 0.0f);
                    tc_ld32(ts, s[0]);
                    tc_wait_ld();
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint32_t *x = s[c & 1];
                        tc_regs32(x);
                        if (c < 3) tc_ld32(ts + 32 * (c + 1), s[(c + 1) & 1]);  // lands while this one is worked on
                        if (kInt8) key_scales(x, c);
                        uint32_t hi[16], lo[16];
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            float2 p = __ffma2_rn(make_float2(__uint_as_float(x[2 * j]), __uint_as_float(x[2 * j + 1])), q2, r2);
                            p.x = q8::exp2_approx(p.x);
                            p.y = q8::exp2_approx(p.y);
                            if constexpr (kMasked) {
                                if (!((see[c] >> (2 * j)) & 1u)) p.x = 0.0f;
                                if (!((see[c] >> (2 * j + 1)) & 1u)) p.y = 0.0f;
                            }
                            sum = __fadd2_rn(sum, p);
                            if (kInt8) {
                                float2 v = *reinterpret_cast<const float2 *>(sc + 128 + 32 * c + 2 * j);
                                if constexpr (kMasked) {
                                    if (!((see[c] >> (2 * j)) & 1u)) v.x = 0.0f;
                                    if (!((see[c] >> (2 * j + 1)) & 1u)) v.y = 0.0f;
                                }
                                p = __fmul2_rn(p, __fmul2_rn(v, make_float2(ie, ie)));
                            }
                            q8::split_f16(p.x, p.y, hi[j], lo[j]);
                        }
                        tc_st16(ts + 32 * c, hi);
                        tc_st16(ts + 32 * c + 16, lo);
                        if (c < 3) tc_wait_ld();
                    }
                    l += sum.x + sum.y;
                };
                if (masked) weigh(std::true_type{}); else weigh(std::false_type{});
                if (!kInt8 && masked) {
                    // values that no row sees must not reach the MMA as 0 * NaN: non-finite ones in a tile with hidden
                    // keys become zero, and are added back at the end for the rows that see them
                    const int st = t & 1;
                    if (!warp_wait(bar(L::bVf + st), static_cast<uint32_t>(t >> 1) & 1u, abort_flag)) {
                        ok = false;
                        break;
                    }
                    uint8_t *v = sm + L::offV + st * L::kMat;
                    for (int c = r; c < L::kMat / 16; c += 128) {
                        uint4 x = *reinterpret_cast<const uint4 *>(v + 16 * c);
                        uint32_t *xx = reinterpret_cast<uint32_t *>(&x);
                        bool hit = false;
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            if ((xx[j] & 0x7c00u) == 0x7c00u) xx[j] &= 0xffff0000u, hit = true;
                            if ((xx[j] & 0x7c000000u) == 0x7c000000u) xx[j] &= 0x0000ffffu, hit = true;
                        }
                        if (hit) {
                            *reinterpret_cast<uint4 *>(v + 16 * c) = x;
                            if (key0 + ((c >> 3) & 127) < w.kend) *s_poison = 1;
                        }
                    }
                    q8::fence_proxy_async_smem();
                    __syncwarp();
                }
                tc_wait_st();
                tc_fence_before();
                arrive(bar(L::bPf + wg));
                if (kInt8) arrive(bar(L::bCe + t % kScaleSlots));
            }
            Walk nx = w;
            more = nx.next(a, pre);
            if (more) load_q(nx.u);
            ok = ok && warp_wait(bar(L::bOf), piece & 1u, abort_flag);
            tc_fence_after();
            s_row[128 * (1 + 3 * wg) + r] = m;
            s_row[128 * (2 + 3 * wg) + r] = l;
            s_row[128 * (3 + 3 * wg) + r] = kInt8 ? q8::pow2(e) : 1.0f;
            soft_sync();
            if (tid == 128) *s_stop = *abort_flag;
            const int poison = *s_poison;
            const float m0 = s_row[128 + r], m1 = s_row[128 * 4 + r];
            const float mm = fmaxf(m0, m1);
            float f0 = m0 == -INFINITY ? 0.0f : m0 == mm ? 1.0f : q8::exp2_approx(m0 - mm);
            float f1 = m1 == -INFINITY ? 0.0f : m1 == mm ? 1.0f : q8::exp2_approx(m1 - mm);
            const float ll = f0 * s_row[128 * 2 + r] + f1 * s_row[128 * 5 + r];
            const float g0 = s_row[128 * 3 + r], g1 = s_row[128 * 6 + r];
            const bool partial = w.t0 > 0 || w.n < u.tiles;
            const int pslot = 2 * cta + (w.first ? 0 : 1);
            const bool valid = row0 + r < rows;
            const long long at = q8::RowMap(a, row0).at(a, u, r, D);
            float *out = partial ? a.part + (static_cast<long long>(pslot) * kRows + r) * D : a.y ? a.y + at : nullptr;
            if (!partial) {  // the quotient; a row that saw nothing is 0
                const float inv = ll == 0.0f ? 0.0f : __frcp_rn(ll);
                f0 *= inv, f1 *= inv;
            }
            // Warpgroup g finishes columns [g * D/2, (g + 1) * D/2) of every row.  A thread puts its half row into
            // shared memory (all scores are computed, so Q's place is free) and hands it to one bulk copy: stores
            // from the registers would touch 32 rows each.
            uint8_t *stage = sm + L::offQ + (wg * 128 + r) * L::kOutRow;
#pragma unroll 1
            for (int c = wg * (D / 2); ok && c < (wg + 1) * (D / 2); c += 32) {
                uint32_t x0[32], x1[32];
                tc_ld32(tl + L::kColO + c, x0);
                if (w.n > 1) tc_ld32(tl + L::kColO + D + c, x1);
                tc_wait_ld();
                tc_regs32(x0);
                float o[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) o[j] = f0 * (g0 * __uint_as_float(x0[j]));
                if (w.n > 1) {
                    tc_regs32(x1);
#pragma unroll
                    for (int j = 0; j < 32; ++j) o[j] += f1 * (g1 * __uint_as_float(x1[j]));
                }
                if (valid && !kInt8 && poison) {  // the non-finite values that were left out, if this row sees them
                    for (int key = max(w.t0 * kTile, (u.cached & ~(kTile - 1)) - kTile); key < w.kend; ++key) {
                        if (!q8::attn_sees(sight, u.cached, key)) continue;
                        const int pi = key / a.page;
                        const int pg = a.table[static_cast<long long>(u.b) * a.max_pages + pi];
                        if (pg < 0 || pg >= a.n_pages) continue;
                        const __half *v = reinterpret_cast<const __half *>(a.v16) +
                                          (static_cast<long long>(pg * a.kv_heads + u.kvh) * a.page + (key - pi * a.page)) * D + c;
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            const float y = __half2float(v[j]);
                            if (!(fabsf(y) <= 65504.0f)) o[j] += y;
                        }
                    }
                }
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    *reinterpret_cast<float4 *>(stage + (c - wg * (D / 2)) * 4 + 16 * j) =
                        make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
                if (valid && !partial && a.qs) encode32(a, at + c, o);
                __syncwarp();
            }
            if (ok && valid && out) {
                q8::fence_proxy_async_smem();
                asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(out + wg * (D / 2)),
                             "r"(q8::smem_u32(stage)), "r"(D / 2 * 4)
                             : "memory");
            }
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
            if (partial && wg == 0) a.ml[pslot * kRows + r] = make_float2(mm, ll);
            if (partial && w.first && tid == 128) {
                a.desc[2 * cta] = make_int4(u.start, u.start + kHead + u.tiles, per, u.start + kHead);
                a.desc[2 * cta + 1] = make_int4(u.b, u.kvh, u.rt, 1);
            }
            asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");  // Q's place is free again
            soft_sync();  // s_stop is written, s_poison and the row words are read
            if (*s_stop) break;
            if (tid == 128) *s_poison = 0;  // set again after the next piece's first barrier at the earliest
            T += w.n;
            ++piece;
            w = nx;
        }
        asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");  // the rows have left before the CTA does
    } else if (kInt8) {
        setmaxnreg_dec<L::kRegsConv>();
        // ------------------------------------------------------------ int8 codes -> f16 tiles in the MMA's layout
        // Eight lanes take half a row each of two neighbouring rows: with the 128-byte swizzle their 16-byte
        // stores then fall into distinct banks.
        const int c0 = tid - 384;
        int T = 0;
        bool ok = true;
        auto widen = [&](uint32_t src_off, uint32_t dst_off) {
            constexpr int kChunks = D / 16;  // 16 codes each
#pragma unroll
            for (int j = 0; j < 128 * kChunks / 128; ++j) {
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
        while (ok && w.next(a, pre)) {
            for (int i = 0; i < w.n; ++i, ++T) {
                const int st = T & 1;
                const uint32_t rpar = static_cast<uint32_t>(T >> 1) & 1u, par = static_cast<uint32_t>(T) & 1u;
                ok = warp_wait(bar(L::bRKf + st), rpar, abort_flag) && warp_wait(bar(L::bKe), par ^ 1u, abort_flag);
                if (!ok) break;
                widen(L::offRaw + st * L::kRaw, L::offK);
                arrive(bar(L::bKf));
                arrive(bar(L::bRKe + st));
                ok = warp_wait(bar(L::bRVf + st), rpar, abort_flag) && warp_wait(bar(L::bVe), par ^ 1u, abort_flag);
                if (!ok) break;
                widen(L::offRaw + (2 + st) * L::kRaw, L::offV);
                arrive(bar(L::bVf));
                arrive(bar(L::bRVe + st));
            }
        }
    }
    if (bad_data) atomicOr(&g_tiles_err, q8::kKvErrData);

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
    if (!q8::set_max_dynamic_smem(reinterpret_cast<const void *>(attn_tiles_kernel<D, kInt8>), 227 * 1024, slot))
        return Q8_ERR_LAUNCH;
    const int st = q8::launch_pdl(attn_tiles_kernel<D, kInt8>, dim3(q8::kAttnCtas), dim3(L::kThreads), L::smem(a.batch), s, mk,
                                  mv, a, box);
    if (st != Q8_OK) return st;
    return q8::launch_pdl(q8::attn_combine_kernel<D, kRows>, dim3(q8::kAttnCtas - 1, kRows * D / 4 / 256), dim3(256), 0, s, a);
}

} // namespace

namespace q8 {

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

int attn_tiles_take_error(cudaStream_t s)
{
    unsigned int v = 0, zero = 0;
    if (cudaMemcpyFromSymbolAsync(&v, g_tiles_err, sizeof(v), 0, cudaMemcpyDeviceToHost, s) != cudaSuccess ||
        cudaMemcpyToSymbolAsync(g_tiles_err, &zero, sizeof(zero), 0, cudaMemcpyHostToDevice, s) != cudaSuccess ||
        cudaStreamSynchronize(s) != cudaSuccess)
        return Q8_ERR_CUDA;
    return (v & kKvErrTimeout) ? Q8_ERR_DEVICE_TIMEOUT : v ? Q8_ERR_DATA : Q8_OK;
}

} // namespace q8
