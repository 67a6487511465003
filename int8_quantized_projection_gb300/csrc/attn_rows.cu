// attn_rows.cu -- q8_tree_attention for up to 16 packed rows a unit
// (single-token decode, small trees), and the join of partial results.
//
//     s_j = scale * q.k_j,  p_j = 2^(s_j - m),  O = sum p_j v_j,  l = sum p_j
//
// with the running maximum m per row.  Bound by the cache's bytes: a key and a
// value are read once for all the rows of a unit, so at 8 rows 32 operations
// fall on a byte of f16, far below what even the warp-level MMA does per byte
// of HBM.  So the design is a stream: 12 or 8 warps a CTA, each with a ring of
// its own into which one lane copies 16 keys and 16 values by TMA, with no
// barrier between the warps until a piece ends.  192 KB of copies are in
// flight per SM.
//
// f32 precision on f16 MMAs: a row's q (scaled by a power of two) is the sum
// of two f16 parts, and m16n8k16 has 16 rows where 8 are wanted, so rows 0-7
// of the A operand are the high parts and rows 8-15 the low parts of the same
// 8 rows.  A thread's accumulators c0, c1 (row g) and c2, c3 (row g + 8) are
// then the two halves of the same two scores, and the same holds for the
// softmax weights and O: the second half of the precision costs no extra MMA
// and no shuffle.  int8 codes are widened exactly to f16; a key's scale
// multiplies its score, a value's scale its weight (with a running power of
// two per row, so that weights stay within f16's range for any scales).
//
// The maximum is raised only when it grows by more than 2^8: weights are
// kept at 2^6 below the reference, so they stay under 2^14 in f16, and the 64
// or 128 multiplications of a rescale are rare.
//
// Measured (head_dim 128, 28 heads on 4): one decode over 262139 keys, f16,
// 86.5 us (537 MB, 6.2 TB/s, 0.92 of a copy's rate); 61 ragged ones of up to
// 8191 keys, int8, 73 us (326 MB, 4.5 TB/s).  Some 10 us of each call are the
// launches, the line, the first copies' latency, and the join.  int8 is bound
// by the warps' chains of dependent steps, some 520 instructions for 16 keys, of
// which the widening is a fifth (52 % of the issue slots are used): 16 warps
// instead of 12 with q in shared memory came to 78 us, the next unit's copies
// before the join to 75.6, two chains of score MMAs to 78.6; none was kept.
#include <cooperative_groups.h>
#include <cuda.h>

#include "attn_common.cuh"

namespace {

__device__ unsigned int g_rows_err;

using q8::AttnArgs;
using q8::Unit;
namespace cg = cooperative_groups;

// What a unit costs beside its tiles, in tiles (61 ragged int8 decodes of up to 8191 keys with 1: 86 us, 2: 79, 3: 74, 6: 76).
constexpr int kHead = 3;
constexpr int kClusterTiles = 8;     // of a CTA of a cluster, however many units there are: lengths may be ragged
static_assert(kClusterTiles <= 64, "a CTA of a cluster keeps one chain");
constexpr float kWeightBits = 6.0f;  // weights are 2^(s - m + 6)
constexpr float kRaise = 8.0f;       // m may lag the maximum by this
// The MMA's f32 accumulation truncates: with values of one sign O loses 1e-7 of
// itself per MMA (measured: 2.5e-5 after 257).  After this many tiles, one MMA
// per tile and value in each warp, a piece's result goes to the workspace,
// rounded to nearest, and the next tiles start anew: up to 6e-6 of a result whose
// values have one sign is lost, and half of that with chains of 32, for one more
// pass over the rows' O every 32 tiles.
constexpr int kChain = 64;

template <int D, bool kInt8, int RG>
struct Ring {
    // Twelve warps where 8 rows leave them the registers: a group of 16 keys is a chain of dependent steps (copy, MMAs,
    // maximum, exponentials, MMAs) of some 2000 cycles, so it takes three warps a scheduler to keep up with HBM.
    static constexpr int kWarps = RG == 1 ? 12 : 8, kThreads = 32 * kWarps;
    static constexpr int kTile = 16 * kWarps;              // keys of a tile: 16 per warp
    static constexpr int kMat = 16 * D * (kInt8 ? 1 : 2);  // 16 keys
    static constexpr int kStage = 2 * kMat;                // and 16 values
    static constexpr int kStages = 196608 / (kWarps * kStage) < 8 ? 196608 / (kWarps * kStage) : 8;
    static constexpr int kScales = kInt8 ? 128 : 0;        // 16 + 16 f32 a stage
    static constexpr int offScales = kWarps * kStages * kStage;
    static constexpr int offBars = offScales + kWarps * kStages * kScales;
    static constexpr int offPre = offBars + kWarps * kStages * 8;
    static int smem(int batch) { return offPre + (batch + 1) * 4 + 1024; }
};
// the largest ring leaves room for the prefix sums of the largest batch (and 3 KB of static arrays)
constexpr int kMaxDynamic = 224 * 1024;
template <int D, bool kInt8, int RG>
constexpr bool ring_fits() { return Ring<D, kInt8, RG>::offPre + (Q8_KV_MAX_BATCH + 1) * 4 + 1024 <= kMaxDynamic; }
static_assert(ring_fits<128, false, 1>() && ring_fits<128, true, 1>() && ring_fits<64, false, 1>() && ring_fits<64, true, 1>() &&
                  ring_fits<128, false, 2>() && ring_fits<128, true, 2>() && ring_fits<64, false, 2>() &&
                  ring_fits<64, true, 2>(),
              "shared memory");

__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// Byte offset of 16-byte chunk c of int8 row `key` (128-byte swizzle for
// rows of 128 bytes, 64-byte swizzle for rows of 64).
template <int D>
__device__ __forceinline__ int code_chunk(int key, int c)
{
    return D == 128 ? key * 128 + ((c ^ (key & 7)) << 4) : key * 64 + ((c ^ ((key >> 1) & 3)) << 4);
}

// State of 8 packed rows in one warp; a thread's share of row lane/4.
template <int D>
struct RowState {
    float o[D / 8][4];
    float m, l;  // reference (log2) and this thread's part of the sum
    int e;       // int8: weights are scaled by 2^-e
    float ie;
};

// S -> weights -> O for 16 keys of one row group.  s: this thread's scores,
// at keys 8*(i/2) + 2*(lane%4) + i%2, -inf where not seen.  v: the keys'
// value scales, 0 where not seen.  Returns the A operand of the second product.
template <int D, bool kInt8>
__device__ __forceinline__ void weights(RowState<D> &st, const float (&s)[4], const float (&v)[4], uint32_t (&a)[4])
{
    float mx = fmaxf(fmaxf(s[0], s[1]), fmaxf(s[2], s[3]));
    mx = fmaxf(mx, __shfl_xor_sync(Q8_FULL_MASK, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(Q8_FULL_MASK, mx, 2));
    float big = 0.0f;
    if (kInt8) {  // the largest scale among the keys this row sees
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (fabsf(v[i]) <= 3.4028235e38f) big = fmaxf(big, fabsf(v[i]));
        big = fmaxf(big, __shfl_xor_sync(Q8_FULL_MASK, big, 1));
        big = fmaxf(big, __shfl_xor_sync(Q8_FULL_MASK, big, 2));
    }
    bool raise = mx > st.m + kRaise;  // also from -inf to anything
    if (kInt8) raise |= big * st.ie > 1.0f;
    if (__any_sync(Q8_FULL_MASK, raise)) {
        const float m = fmaxf(st.m, mx);
        float f = st.m == m ? 1.0f : q8::exp2_approx(st.m - m);
        st.l *= f;
        st.m = m;
        if (kInt8) {
            const int e = min(127, max(st.e, static_cast<int>(__float_as_uint(big) >> 23) - 126));
            const int drop = st.e - e;  // <= 0
            f = drop < -126 ? 0.0f : f * q8::pow2(drop);
            st.e = e;
            st.ie = q8::pow2(max(-126, -e));
        }
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) st.o[n][i] *= f;
    }
    const float ref = st.m == -INFINITY ? 0.0f : st.m - kWeightBits;
    float p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        p[i] = q8::exp2_approx(s[i] - ref);
        st.l += p[i];
        if (kInt8) p[i] *= v[i] * st.ie;
    }
    q8::split_f16(p[0], p[1], a[0], a[1]);
    q8::split_f16(p[2], p[3], a[2], a[3]);
}

// kCluster: a unit is a cluster's, whose CTAs join in shared memory (clusters of one CTA take units in turn); else the CTAs
// share the line.
template <int D, bool kInt8, int RG, bool kCluster>
__global__ void __launch_bounds__(Ring<D, kInt8, RG>::kThreads, 1)
attn_rows_kernel(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                 const __grid_constant__ AttnArgs a)
{
    using R = Ring<D, kInt8, RG>;
    constexpr int kRows = 8 * RG, kWarps = R::kWarps, kThreads = R::kThreads, kTile = R::kTile;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = q8::smem_u32(smem_raw);
    uint8_t *sm = smem_raw + (((raw + 1023u) & ~1023u) - raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, gid = lane >> 2, tig = lane & 3;
    uint8_t *ring = sm + warp * R::kStages * R::kStage;
    uint8_t *ring_sc = sm + R::offScales + warp * R::kStages * R::kScales;
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + R::offBars) + warp * R::kStages;
    int *pre = reinterpret_cast<int *>(sm + R::offPre);
    __shared__ float s_m[kWarps][kRows], s_l[kWarps][kRows], s_f[kWarps][kRows];
    __shared__ float2 s_sum[kRows], s_next[kRows];  // (m, l) of the chains before
    __shared__ int s_poison;

    if (lane == 0)
        for (int i = 0; i < R::kStages; ++i) q8::mbar_init(bars + i, kInt8 ? 33 : 1);  // the codes' bytes; int8: each lane's scale
    if (tid == 0) s_poison = 0;
    q8::fence_mbar_init();
    q8::griddep_launch_dependents();
    q8::griddep_wait();
    const int cta = blockIdx.x;
    bool bad_data = false;
    int s0 = 0, s1 = 1, per = 1, rank = 0;
    Unit u;
    const int step = kCluster ? static_cast<int>(gridDim.x) / a.cluster : 0;  // clusters: units that far apart are one's
    if constexpr (kCluster) {
        s0 = cta / a.cluster, s1 = a.batch * a.kv_heads;
        rank = cta - s0 * a.cluster;
        u.fresh = 0;
        __syncthreads();  // the barriers and s_poison are set
    } else {
        bad_data = !q8::attn_line<kRows, kTile, kHead, kThreads>(a, pre);
        const int total = pre[a.batch];
        per = max(1, (total + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x));
        s0 = min(total, cta * per), s1 = min(total, s0 + per);
        if (tid == 0) a.desc[2 * cta + 1].w = 0;  // no first piece yet
    }

    int slot = 0, phase = 0, wslot = 0;  // the ring: next to read (and its parity), next to fill
    bool dead = false;
    float4 *const shared_o = reinterpret_cast<float4 *>(sm + kWarps * kRows * D * 4);  // a.cluster: this CTA's part of the unit
    for (int pos = s0; pos < s1;) {
        int ta, tb;
        const bool first = pos == s0;
        if constexpr (kCluster) {
            u.b = pos / a.kv_heads, u.kvh = pos - u.b * a.kv_heads, u.rt = u.start = 0;
            pos += step;
            bad_data |= !q8::attn_sequence(a, u.b, u.cached, u.fresh, u.first);
            if (u.fresh == 0) continue;
            u.tiles = q8::attn_tiles_of<kRows, kTile>(a, u.cached, u.fresh, 0);
            ta = rank * u.tiles / a.cluster, tb = (rank + 1) * u.tiles / a.cluster;
            if (ta == tb)  // no tile falls to this CTA
                for (int i = tid; i < kRows * D / 4; i += kThreads) {
                    shared_o[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    if (i < kRows) s_sum[i] = make_float2(-INFINITY, 0.0f);
                }
        } else {
            if (first) u = q8::attn_unit<kRows, kTile, kHead>(a, pre, pos);
            else q8::attn_next_unit<kRows, kTile, kHead>(a, pre, u);
            ta = max(0, pos - u.start - kHead), tb = max(0, min(u.tiles, s1 - u.start - kHead));
            pos = u.start + kHead + u.tiles;
        }
        // (no tiles: only the unit's head, the next CTA has them)
        for (int t0 = ta; t0 < tb; t0 += kChain) {
            const int t1 = min(tb, t0 + kChain);
            const int rows = u.fresh * a.group, row0 = u.rt * kRows;
            const int seen = q8::attn_visible(a, u.cached, u.fresh, min(row0 + kRows, rows));
            const int k0 = t0 * kTile + warp * 16, k1 = min(t1 * kTile, seen);
            const int n = dead || k0 >= k1 ? 0 : (k1 - k0 + kTile - 1) / kTile;  // this warp's 16-key groups

            float2 x[RG][D / 8];  // the rows' q: asked for before the copies, so as not to queue behind them
#pragma unroll
            for (int rg = 0; rg < RG; ++rg) {
                const int row = row0 + rg * 8 + gid, tok = q8::attn_token(a, row);
                const float *src =
                    a.q + (static_cast<long long>(u.first + tok) * a.heads + u.kvh * a.group + (row - tok * a.group)) * D;
#pragma unroll
                for (int s = 0; s < D / 8; ++s) {
                    // the contraction's order is free: for int8 a thread's keys come as 8 consecutive codes
                    const int c = kInt8 ? 32 * (s / 4) + 8 * tig + 2 * (s % 4) : 8 * s + 2 * tig;
                    x[rg][s] = make_float2(0.0f, 0.0f);
                    if (row < rows) x[rg][s] = __ldg(reinterpret_cast<const float2 *>(src + c));
                }
            }

            // cache rows of the groups, 32 at a time, a lane each
            auto fetch = [&](int i) {
                i += lane;
                if (i >= n) return 0;
                const int key = k0 + i * kTile, pi = key / a.page;
                int pg = a.table[static_cast<long long>(u.b) * a.max_pages + pi];
                if (pg < 0 || pg >= a.n_pages) {
                    bad_data = true;
                    pg = 0;
                }
                return (pg * a.kv_heads + u.kvh) * a.page + (key - pi * a.page);
            };
            int base = 0, rows_now = fetch(0), rows_next = fetch(32);
            auto issue = [&](int i) {
                if (i >= base + 32) {
                    base += 32;
                    rows_now = rows_next;
                    rows_next = fetch(base + 32);
                }
                const int row = __shfl_sync(Q8_FULL_MASK, rows_now, i - base);
                if (lane == 0) {
                    uint8_t *dst = ring + wslot * R::kStage;
                    uint64_t *bar = bars + wslot;
                    q8::mbar_arrive_expect_tx(bar, R::kStage);
                    const uint32_t d = q8::smem_u32(dst), bb = q8::smem_u32(bar);
                    constexpr int kBox = kInt8 ? D : 64;  // elements of a box row
                    constexpr int kBoxBytes = 16 * kBox * (kInt8 ? 1 : 2);
#pragma unroll
                    for (int h = 0; h < D / kBox; ++h) {
                        q8::tma_load_2d(d + h * kBoxBytes, &mk, h * kBox, row, bb);
                        q8::tma_load_2d(d + R::kMat + h * kBoxBytes, &mv, h * kBox, row, bb);
                    }
                }
                if (kInt8) {  // 16 scales of the keys, 16 of the values, a lane each: two bulk copies of 64 bytes took 4 % longer
                    const float *src = (lane < 16 ? a.ks : a.vs) + row + (lane & 15);
                    const uint32_t dst = q8::smem_u32(ring_sc + wslot * R::kScales + lane * 4), bb = q8::smem_u32(bars + wslot);
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
                    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bb) : "memory");
                }
                wslot = wslot + 1 == R::kStages ? 0 : wslot + 1;
            };
            for (int i = 0; i < min(n, R::kStages); ++i) issue(i);

            // q of this thread's rows, in two f16 parts
            uint32_t qa[RG][D / 16][4];
            float qs[RG];
            q8::RowSight sight[RG];
#pragma unroll
            for (int rg = 0; rg < RG; ++rg) {
                sight[rg] = q8::attn_sight(a, u, row0 + rg * 8 + gid);
                float amax = 0.0f;
#pragma unroll
                for (int s = 0; s < D / 8; ++s) amax = fmaxf(amax, fmaxf(fabsf(x[rg][s].x), fabsf(x[rg][s].y)));
                amax = fmaxf(amax, __shfl_xor_sync(Q8_FULL_MASK, amax, 1));
                amax = fmaxf(amax, __shfl_xor_sync(Q8_FULL_MASK, amax, 2));
                // the row's largest value to [1, 2): the low parts keep 22 bits of it
                const int e = min(126, max(-126, static_cast<int>(__float_as_uint(amax) >> 23) - 127));
                const float down = q8::pow2(-e);
                qs[rg] = q8::pow2(e) * a.scale;
#pragma unroll
                for (int s = 0; s < D / 16; ++s) {
                    q8::split_f16(x[rg][2 * s].x * down, x[rg][2 * s].y * down, qa[rg][s][0], qa[rg][s][1]);
                    q8::split_f16(x[rg][2 * s + 1].x * down, x[rg][2 * s + 1].y * down, qa[rg][s][2], qa[rg][s][3]);
                }
            }

            RowState<D> st[RG];
#pragma unroll
            for (int rg = 0; rg < RG; ++rg) {
                st[rg].m = -INFINITY;
                st[rg].l = 0.0f;
                st[rg].e = -126;
                st[rg].ie = q8::pow2(126);
#pragma unroll
                for (int i = 0; i < D / 8; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) st[rg].o[i][j] = 0.0f;
            }
            // keys that every row of the tile sees
            const int all_see = u.cached + (a.masks ? 0 : q8::attn_token(a, row0) + 1);

            for (int i = 0; i < n; ++i) {
                if (!__all_sync(Q8_FULL_MASK, q8::mbar_wait_bounded(bars + slot, phase))) {
                    // let the copies in flight land, then go on without them
                    int sl = slot, ph = phase;
                    for (int j = i; j < min(n, i + R::kStages); ++j) {
                        q8::mbar_wait_bounded(bars + sl, ph, Q8_DRAIN_LIMIT_NS);
                        if (++sl == R::kStages) sl = 0, ph ^= 1;
                    }
                    if (lane == 0) atomicOr(&g_rows_err, q8::kErrTimeout);
                    dead = true;
                    break;
                }
                const int key0 = k0 + i * kTile;
                const bool masked = key0 + 16 > all_see;
                uint8_t *stage = ring + slot * R::kStage;
                const uint32_t sk = q8::smem_u32(stage), sv = sk + R::kMat;
                const float *sc = reinterpret_cast<const float *>(ring_sc + slot * R::kScales);

                bool wrote = false;
                if (!kInt8 && masked) {
                    // values that no row sees must not reach the MMA as 0 * NaN: rows past the sequence become
                    // zero, and so do non-finite values of keys that some row may not see (added back at the end)
                    for (int c = lane; c < 16 * D / 8; c += 32) {
                        uint4 *p = reinterpret_cast<uint4 *>(stage + R::kMat) + c;
                        uint4 w = *p;
                        uint32_t *ww = reinterpret_cast<uint32_t *>(&w);
                        bool hit = false;
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            if ((ww[j] & 0x7c00u) == 0x7c00u) ww[j] &= 0xffff0000u, hit = true;
                            if ((ww[j] & 0x7c000000u) == 0x7c000000u) ww[j] &= 0x0000ffffu, hit = true;
                        }
                        if (hit) {
                            *p = w;
                            wrote = true;
                            if (key0 + ((c >> 3) & 15) < k1) s_poison = 1;
                        }
                    }
                    if (wrote) q8::fence_proxy_async_smem();  // before the ring's next copy into this stage
                    __syncwarp();
                }

                float acc[RG][2][4];
#pragma unroll
                for (int rg = 0; rg < RG; ++rg)
#pragma unroll
                    for (int t = 0; t < 2; ++t)
#pragma unroll
                        for (int j = 0; j < 4; ++j) acc[rg][t][j] = 0.0f;
                if (!kInt8) {
                    const int key = ((lane >> 4) << 3) + (lane & 7);
#pragma unroll
                    for (int s = 0; s < D / 16; ++s) {
                        const int c = (s & 3) * 2 + ((lane >> 3) & 1);
                        uint32_t b[4];
                        ldsm4(b, sk + (s >> 2) * 2048 + key * 128 + ((c ^ (key & 7)) << 4));
#pragma unroll
                        for (int rg = 0; rg < RG; ++rg) {
                            mma(acc[rg][0], qa[rg][s], b[0], b[1]);
                            mma(acc[rg][1], qa[rg][s], b[2], b[3]);
                        }
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < D / 32; ++c)
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            const int key = 8 * t + gid;
                            const uint2 w = *reinterpret_cast<const uint2 *>(
                                stage + code_chunk<D>(key, 2 * c + (tig >> 1)) + (tig & 1) * 8);
                            uint32_t b0, b1, b2, b3;
                            q8::i8x4_to_f16x4(w.x, b0, b1);
                            q8::i8x4_to_f16x4(w.y, b2, b3);
#pragma unroll
                            for (int rg = 0; rg < RG; ++rg) {
                                mma(acc[rg][t], qa[rg][2 * c], b0, b1);
                                mma(acc[rg][t], qa[rg][2 * c + 1], b2, b3);
                            }
                        }
                }
                float vs[4] = {1.0f, 1.0f, 1.0f, 1.0f};
                float2 k01, k89;
                if (kInt8) {
                    k01 = *reinterpret_cast<const float2 *>(sc + 2 * tig);
                    k89 = *reinterpret_cast<const float2 *>(sc + 8 + 2 * tig);
                    const float2 v01 = *reinterpret_cast<const float2 *>(sc + 16 + 2 * tig);
                    const float2 v89 = *reinterpret_cast<const float2 *>(sc + 24 + 2 * tig);
                    vs[0] = v01.x, vs[1] = v01.y, vs[2] = v89.x, vs[3] = v89.y;
                }
                uint32_t pa[RG][4];
#pragma unroll
                for (int rg = 0; rg < RG; ++rg) {
                    float s[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        s[j] = (acc[rg][j >> 1][j & 1] + acc[rg][j >> 1][2 + (j & 1)]) * qs[rg];
                    if (kInt8) s[0] *= k01.x, s[1] *= k01.y, s[2] *= k89.x, s[3] *= k89.y;
                    float v[4] = {vs[0], vs[1], vs[2], vs[3]};
                    if (masked) {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (!q8::attn_sees(sight[rg], u.cached, key0 + 8 * (j >> 1) + 2 * tig + (j & 1)))
                                s[j] = -INFINITY, v[j] = 0.0f;
                    }
                    weights<D, kInt8>(st[rg], s, v, pa[rg]);
                }
                if (!kInt8) {
                    const int key = (((lane >> 3) & 1) << 3) + (lane & 7);
#pragma unroll
                    for (int j = 0; j < D / 16; ++j) {
                        const int c = (j & 3) * 2 + (lane >> 4);
                        uint32_t b[4];
                        ldsm4t(b, sv + (j >> 2) * 2048 + key * 128 + ((c ^ (key & 7)) << 4));
#pragma unroll
                        for (int rg = 0; rg < RG; ++rg) {
                            mma(st[rg].o[2 * j], pa[rg], b[0], b[1]);
                            mma(st[rg].o[2 * j + 1], pa[rg], b[2], b[3]);
                        }
                    }
                } else {
                    // output column gid of tile 4*j + x is value dimension 4*(gid + 8*j) + x: a thread's four
                    // codes of a key are then one word, and pairs of keys interleave by byte permutes
                    const uint8_t *vb = stage + R::kMat;
#pragma unroll
                    for (int j = 0; j < D / 32; ++j) {
                        const int wi = gid + 8 * j;
                        uint32_t w[4];
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const int key = 2 * tig + (x & 1) + 8 * (x >> 1);
                            w[x] = *reinterpret_cast<const uint32_t *>(vb + code_chunk<D>(key, wi >> 2) + (wi & 3) * 4);
                        }
                        uint32_t b[4][2];
                        q8::i8x4_to_f16x4(__byte_perm(w[0], w[1], 0x5140), b[0][0], b[1][0]);
                        q8::i8x4_to_f16x4(__byte_perm(w[0], w[1], 0x7362), b[2][0], b[3][0]);
                        q8::i8x4_to_f16x4(__byte_perm(w[2], w[3], 0x5140), b[0][1], b[1][1]);
                        q8::i8x4_to_f16x4(__byte_perm(w[2], w[3], 0x7362), b[2][1], b[3][1]);
#pragma unroll
                        for (int x = 0; x < 4; ++x)
#pragma unroll
                            for (int rg = 0; rg < RG; ++rg) mma(st[rg].o[4 * j + x], pa[rg], b[x][0], b[x][1]);
                    }
                }
                if (++slot == R::kStages) slot = 0, phase ^= 1;
                __syncwarp();  // every lane has read the stage
                if (i + R::kStages < n) issue(i + R::kStages);
            }

            // join the warps: numerators to shared memory (the rings are empty now), scaled by 2^e at the read
            __syncthreads();
            float *om = reinterpret_cast<float *>(sm);
#pragma unroll
            for (int rg = 0; rg < RG; ++rg) {
                float l = st[rg].l;
                l += __shfl_xor_sync(Q8_FULL_MASK, l, 1);
                l += __shfl_xor_sync(Q8_FULL_MASK, l, 2);
                const int r = rg * 8 + gid;
                if (tig == 0) {
                    s_m[warp][r] = st[rg].m;
                    s_l[warp][r] = l;
                    s_f[warp][r] = kInt8 ? q8::pow2(st[rg].e) : 1.0f;
                }
                float *o = om + (warp * kRows + r) * D;
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    const float x = st[rg].o[i][0] + st[rg].o[i][2], y = st[rg].o[i][1] + st[rg].o[i][3];
                    if (!kInt8) {
                        *reinterpret_cast<float2 *>(o + 8 * i + 2 * tig) = make_float2(x, y);
                    } else {
                        const int c = 4 * (2 * tig + 8 * (i >> 2)) + (i & 3);
                        o[c] = x;
                        o[c + 4] = y;
                    }
                }
            }
            __syncthreads();
            const bool partial = ta > 0 || tb < u.tiles, rows_out = t1 == tb && !partial;
            const int pslot = 2 * cta + (first ? 0 : 1);
            const int poison = s_poison;
            for (int i = tid; i < kRows * D / 4; i += kThreads) {
                const int r = i / (D / 4), c = (i % (D / 4)) * 4;
                float m = -INFINITY;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) m = fmaxf(m, s_m[w][r]);
                float l = 0.0f;
                float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const float f = s_m[w][r] == -INFINITY ? 0.0f : s_m[w][r] == m ? 1.0f : q8::exp2_approx(s_m[w][r] - m);
                    l += f * s_l[w][r];
                    const float4 x = *reinterpret_cast<const float4 *>(om + (w * kRows + r) * D + c);
                    const float g = s_f[w][r];
                    o.x += f * (g * x.x), o.y += f * (g * x.y), o.z += f * (g * x.z), o.w += f * (g * x.w);
                }
                if (!kInt8 && poison) {  // the non-finite values that were left out, for the rows that see them
                    const q8::RowSight sg = q8::attn_sight(a, u, row0 + r);
                    for (int key = max(t0 * kTile, (u.cached & ~15) - 16); key < k1; ++key) {
                        if (!q8::attn_sees(sg, u.cached, key)) continue;
                        const int pi = key / a.page;
                        const int pg = a.table[static_cast<long long>(u.b) * a.max_pages + pi];
                        if (pg < 0 || pg >= a.n_pages) continue;
                        const long long row =
                            static_cast<long long>(pg * a.kv_heads + u.kvh) * a.page + (key - pi * a.page);
                        const __half *v = reinterpret_cast<const __half *>(a.v16) + row * D + c;
                        const float x[4] = {__half2float(v[0]), __half2float(v[1]), __half2float(v[2]), __half2float(v[3])};
                        if (!(fabsf(x[0]) <= 65504.0f)) o.x += x[0];
                        if (!(fabsf(x[1]) <= 65504.0f)) o.y += x[1];
                        if (!(fabsf(x[2]) <= 65504.0f)) o.z += x[2];
                        if (!(fabsf(x[3]) <= 65504.0f)) o.w += x[3];
                    }
                }
                float4 *sum = reinterpret_cast<float4 *>(a.part + (static_cast<long long>(pslot) * kRows + r) * D + c);
                if (t0 > ta) {  // the chains before, by the thread that wrote them
                    const float2 ml = s_sum[r];
                    const float4 x = *sum;
                    const float mn = fmaxf(m, ml.x);
                    const float f = m == -INFINITY ? 0.0f : m == mn ? 1.0f : q8::exp2_approx(m - mn);
                    const float g = ml.x == -INFINITY ? 0.0f : ml.x == mn ? 1.0f : q8::exp2_approx(ml.x - mn);
                    o = make_float4(f * o.x + g * x.x, f * o.y + g * x.y, f * o.z + g * x.z, f * o.w + g * x.w);
                    l = f * l + g * ml.y;
                    m = mn;
                }
                if (kCluster && a.cluster > 1) {
                    shared_o[i] = o;
                    if (c == 0) s_sum[r] = make_float2(m, l);
                } else if (!rows_out) {
                    *sum = o;
                    if (c == 0) {
                        s_next[r] = make_float2(m, l);
                        if (partial && t1 == tb) a.ml[pslot * kRows + r] = make_float2(m, l);
                    }
                } else {
                    q8::attn_store<D>(a, u, row0 + r, c, o, l, row0 + r < rows);
                }
            }
            if (!kCluster && partial && first && t1 == tb && tid == 0) {
                a.desc[2 * cta] = make_int4(u.start, u.start + kHead + u.tiles, per, u.start + kHead);
                a.desc[2 * cta + 1] = make_int4(u.b, u.kvh, u.rt, 1);
            }
            if (pos < s1 || t1 < tb) {  // the ring's next copies come after these reads and writes
                q8::fence_proxy_async_smem();
                __syncthreads();
                if (tid == 0) s_poison = 0;
                if (tid < kRows) s_sum[tid] = s_next[tid];
                __syncthreads();
            }
        }
    }
    if (bad_data) atomicOr(&g_rows_err, q8::kErrData);
    if (kCluster && a.cluster > 1 && u.fresh > 0) {
        // join the CTAs of the one unit, in the order of their tiles; a warp takes 32 times 4 columns, whole blocks of the
        // plane
        cg::cluster_group cluster = cg::this_cluster();
        cluster.sync();
        for (int g = warp * a.cluster + rank; g < kRows * D / 128; g += kWarps * a.cluster) {
            const int i = 32 * g + lane, r = i / (D / 4), c = (i % (D / 4)) * 4;
            float m = -INFINITY, l = 0.0f;
            float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            for (int k = 0; k < a.cluster; ++k) m = fmaxf(m, cluster.map_shared_rank(s_sum, k)[r].x);
            for (int k = 0; k < a.cluster; ++k) {
                const float2 ml = cluster.map_shared_rank(s_sum, k)[r];
                const float4 x = cluster.map_shared_rank(shared_o, k)[i];
                const float f = ml.x == -INFINITY ? 0.0f : ml.x == m ? 1.0f : q8::exp2_approx(ml.x - m);
                l += f * ml.y;
                o.x += f * x.x, o.y += f * x.y, o.z += f * x.z, o.w += f * x.w;
            }
            q8::attn_store<D>(a, u, r, c, o, l, r < u.fresh * a.group);
        }
        cluster.sync();  // every CTA keeps its shared memory until the others have read it
    }
}

template <int D, bool kInt8, int RG>
int launch_rows(const CUtensorMap &mk, const CUtensorMap &mv, const AttnArgs &a, int slot, cudaStream_t s)
{
    using R = Ring<D, kInt8, RG>;
    const int smem = R::smem(a.batch);
    const void *fn = a.cluster ? reinterpret_cast<const void *>(attn_rows_kernel<D, kInt8, RG, true>)
                               : reinterpret_cast<const void *>(attn_rows_kernel<D, kInt8, RG, false>);
    if (!q8::set_max_dynamic_smem(fn, kMaxDynamic, slot + (a.cluster ? 12 : 0))) return Q8_ERR_LAUNCH;
    const int units = a.batch * a.kv_heads;
    if (a.cluster)
        return q8::launch_pdl_cluster(attn_rows_kernel<D, kInt8, RG, true>,
                                      dim3(min(units, q8::kAttnCtas / a.cluster) * a.cluster), dim3(R::kThreads),
                                      R::smem(0), s, a.cluster, mk, mv, a);
    const int st = q8::launch_pdl(attn_rows_kernel<D, kInt8, RG, false>, dim3(q8::kAttnCtas), dim3(R::kThreads), smem, s, mk, mv, a);
    if (st != Q8_OK) return st;
    return q8::launch_pdl(q8::attn_combine_kernel<D, 8 * RG>, dim3(q8::kAttnCtas - 1, 4 * RG), dim3(256), 0, s,
                          a);
}

} // namespace

namespace q8 {

// The CTAs of a unit that join in shared memory, or 0 for the line.  A cluster has no line to add up, no workspace and no
// second launch, but a unit gets eight CTAs at most, and those of a short unit are idle.  In tiles: a CTA's own
// and its start, against a stretch of the line with its start and the join, some three tiles more.  Measured in a graph, 28
// heads on 4 of 128 f16 values, lengths ragged up to the one given, line / clusters of the size that the rule takes: 1
// sequence of 380 keys 9.9 / 7.9 us (2 CTAs), 4097 10.6 / 9.9 (8); 5 sequences of 1500 11.8 / 9.4 (4); 8 of 6000 17.6 / 15.7
// (4); 16 of 1500 15.2 / 12.2 (2); 38 of 380 17.7 / 9.4 (1), of 1500 23.6 / 17.7 (1); 61, whose 244 units are dealt out to 152
// CTAs, of 380 19.4 / 16.1, of 1500 30.8 / 28.9.  Left to the line: 1 of 12000, 13.1 us (14.4 in clusters of 8), and 9 of 6000,
// whose 36 clusters of 4 may not all fit, 18.7.
int attn_rows_cluster(int rows, int64_t units, int64_t max_len)
{
    const int64_t tile = rows == 8 ? Ring<128, false, 1>::kTile : Ring<128, false, 2>::kTile, tiles = (max_len + tile - 1) / tile;
    // The GPU has room for 15 clusters of 8, 36 of 4, 76 of 2 at once (units of 1500 keys: 15 of 8 8.2 us, 16 14.9; 36 of 4
    // 8.9, 37 14.4): a little less is used, since GPUs differ in which SMs they have.
    int c = units <= 14 ? 8 : units <= 34 ? 4 : units <= 74 ? 2 : 1;
    while (c > 1 && c >= 2 * tiles) c /= 2;
    // more units than CTAs: each CTA takes every kAttnCtas-th
    const int64_t mine = (tiles + c - 1) / c, turns = (units * c + kAttnCtas - 1) / kAttnCtas;
    return mine <= kClusterTiles && turns * (mine + kHead) <= units * (tiles + kHead) / kAttnCtas + kHead + 3 ? c : 0;
}

int attn_rows_launch(const AttnCall &c, int rows, cudaStream_t s)
{
    const int D = c.dim;
    const CUtensorMapDataType dt = c.int8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    const CUtensorMapSwizzle sw = c.int8 && D == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
    const uint32_t box = c.int8 ? D : 64;
    const uint64_t pitch = D * (c.int8 ? 1 : 2);
    CUtensorMap mk, mv;
    if (!make_map_2d(&mk, dt, c.k, D, c.layer_rows, pitch, box, 16, sw) ||
        !make_map_2d(&mv, dt, c.v, D, c.layer_rows, pitch, box, 16, sw))
        return Q8_ERR_CUDA;
    if (D == 128) {
        if (c.int8)
            return rows == 8 ? launch_rows<128, true, 1>(mk, mv, c.a, 20, s) : launch_rows<128, true, 2>(mk, mv, c.a, 21, s);
        return rows == 8 ? launch_rows<128, false, 1>(mk, mv, c.a, 22, s) : launch_rows<128, false, 2>(mk, mv, c.a, 23, s);
    }
    if (c.int8)
        return rows == 8 ? launch_rows<64, true, 1>(mk, mv, c.a, 24, s) : launch_rows<64, true, 2>(mk, mv, c.a, 25, s);
    return rows == 8 ? launch_rows<64, false, 1>(mk, mv, c.a, 26, s) : launch_rows<64, false, 2>(mk, mv, c.a, 27, s);
}

unsigned int *attn_rows_error_word()
{
    void *p = nullptr;
    return cudaGetSymbolAddress(&p, g_rows_err) == cudaSuccess ? static_cast<unsigned int *>(p) : nullptr;
}

} // namespace q8
