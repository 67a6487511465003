// attn_common.cuh -- what the kernels of q8_tree_attention share: the
// arguments, the split of the work over CTAs, visibility and the epilogue.
//
// Rows.  The `group` query heads that read one key/value head are packed with
// the fresh tokens of a sequence into one list of rows, row r = token r/group,
// head r%group, so a key that is loaded serves all of them.  A unit is a tile
// of kRows such rows of one (sequence, key/value head); its cost is the number
// of kTile-key tiles the last row of the tile can see.
//
// Split.  All units' tiles lie on one line, in the order (sequence, head, row
// tile), and each CTA takes an equal stretch of it: a long context is spread
// over many CTAs and short ones share one, whatever the mix of lengths, and
// no CTA has more than one tile above the mean.  Only the lengths on the device
// decide, so a captured graph stays balanced as the contexts grow.  A unit
// that crosses a boundary leaves one partial (m, l, O) per piece in the
// workspace (a CTA has two at most: its first and its last) and
// attn_combine_kernel joins them in the order of the line.
// Units over short contexts take another form: a cluster of 1 to 8 CTAs per
// unit, joined in shared memory (attn_rows_cluster), or a CTA
// (attn_tiles_cluster).
#pragma once

#include "kv_common.cuh"

namespace q8 {

struct AttnArgs {
    const float *q;
    const int32_t *table, *cached, *starts;
    const long long *masks;
    const float *ks, *vs;  // this layer's scales (int8)
    const uint16_t *v16;   // this layer's v as f16 bits (the rare path for non-finite values)
    float *y;
    int8_t *qs;
    uint32_t *ds;
    float *part;           // [2 * grid][rows][D] partial numerators
    float2 *ml;            // [2 * grid][rows] partial (m, l)
    int4 *desc;            // [2 * grid] the first piece of each CTA, if it is a part of a unit
    long long tokens;
    int batch, heads, kv_heads, group, max_pages, page, n_pages, max_fresh, max_len;
    unsigned group_inv;    // kv_inverse(group)
    int cluster;           // CTAs of a unit, which join in shared memory, or 0: the line
    float scale;           // softmax scale * log2(e)
};

struct Unit {
    int b, kvh, rt;      // sequence, key/value head, row tile
    int tiles;           // key tiles; it costs kHead more
    int start;           // its place on the line: kHead, then the tiles
    int cached, fresh, first;  // the sequence's lengths and first row of q
};

// Token of a packed row (a division costs some 150 cycles, and a unit's start
// is a chain of such steps).
__device__ __forceinline__ int attn_token(const AttnArgs &a, int row) { return kv_divide(row, a.group, a.group_inv); }

// Keys that rows [0, r_end) of a sequence's packed rows can see at most.
__device__ __forceinline__ int attn_visible(const AttnArgs &a, int cached, int fresh, int r_end)
{
    if (a.masks) return cached + fresh;
    return cached + min(fresh, attn_token(a, r_end - 1) + 1);
}

// Lengths of sequence b; fresh = 0 (no work) when a value is out of range.
__device__ __forceinline__ bool attn_sequence(const AttnArgs &a, int b, int &cached, int &fresh, int &first)
{
    cached = a.cached[b];
    first = a.starts[b];
    const long long f = static_cast<long long>(a.starts[b + 1]) - first;
    const long long len = f + cached;
    if (f < 0 || f > a.max_fresh || first < 0 || first + f > a.tokens || cached < 0 || len > a.max_len ||
        (len + a.page - 1) / a.page > a.max_pages) {
        fresh = 0;
        return false;
    }
    fresh = static_cast<int>(f);
    return true;
}

// Tiles of row tile rt of a sequence.
template <int kRows, int kTile>
__device__ __forceinline__ int attn_tiles_of(const AttnArgs &a, int cached, int fresh, int rt)
{
    return (attn_visible(a, cached, fresh, min((rt + 1) * kRows, fresh * a.group)) + kTile - 1) / kTile;
}

// Packed row -> token and head of the group, for rows of one unit: a product
// instead of a division (exact below 1024 for groups up to 64).
struct RowMap {
    int row0, tok0, rem0;
    unsigned magic;
    int group;

    __device__ __forceinline__ RowMap(const AttnArgs &a, int row0_)
        : row0(row0_), tok0(attn_token(a, row0_)), rem0(row0_ - tok0 * a.group), magic((65535u + a.group) / a.group), group(a.group)
    {
    }
    __device__ __forceinline__ int token(int r) const { return tok0 + static_cast<int>(((rem0 + r) * magic) >> 16); }
    // element offset of row row0 + r in q and y
    __device__ __forceinline__ long long at(const AttnArgs &a, const Unit &u, int r, int dim) const
    {
        const int t = token(r);
        return (static_cast<long long>(u.first + t) * a.heads + u.kvh * group + (row0 + r - t * group)) * dim;
    }
};

// The line: pre[b] = cost of the sequences before b (pre[batch] = all).  All
// threads of the CTA call it; ends with a barrier.  False when a sequence is
// out of range.
template <int kRows, int kTile, int kHead, int kThreads>
__device__ __forceinline__ bool attn_line(const AttnArgs &a, int *pre)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rts = (a.max_fresh * a.group + kRows - 1) / kRows;
    bool ok = true;
    if (rts <= 8) {  // a thread per sequence
        for (int b = tid; b < a.batch; b += kThreads) {
            int cached, fresh, first, sum = 0;
            ok &= attn_sequence(a, b, cached, fresh, first);
            for (int r = 0; r * kRows < fresh * a.group; ++r) sum += attn_tiles_of<kRows, kTile>(a, cached, fresh, r) + kHead;
            pre[b + 1] = sum * a.kv_heads;
        }
    } else {  // prompts: a warp per sequence
        for (int b = warp; b < a.batch; b += kThreads / 32) {
            int cached, fresh, first, sum = 0;
            ok &= attn_sequence(a, b, cached, fresh, first);
            for (int r = lane; r * kRows < fresh * a.group; r += 32)
                sum += attn_tiles_of<kRows, kTile>(a, cached, fresh, r) + kHead;
            sum = __reduce_add_sync(Q8_FULL_MASK, sum);
            if (lane == 0) pre[b + 1] = sum * a.kv_heads;
        }
    }
    __syncthreads();
    if (warp == 0) {
        int run = 0;
        for (int b0 = 0; b0 < a.batch; b0 += 32) {
            int v = b0 + lane < a.batch ? pre[b0 + lane + 1] : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(Q8_FULL_MASK, v, o);
                if (lane >= o) v += x;
            }
            if (b0 + lane < a.batch) pre[b0 + lane + 1] = run + v;
            run += __shfl_sync(Q8_FULL_MASK, v, 31);
        }
        if (lane == 0) pre[0] = 0;
    }
    __syncthreads();
    return ok;
}

// The unit at place `pos` of the line; all lanes of a warp call it and get it
// (causal row tiles differ in cost: the lanes add up 32 of them at a time).
template <int kRows, int kTile, int kHead>
__device__ __forceinline__ Unit attn_unit(const AttnArgs &a, const int *pre, int pos)
{
    int lo = 0, hi = a.batch;  // pre[lo] <= pos < pre[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (pre[mid] <= pos) lo = mid; else hi = mid;
    }
    Unit u;
    u.b = lo;
    attn_sequence(a, lo, u.cached, u.fresh, u.first);
    const int per_head = (pre[lo + 1] - pre[lo]) / a.kv_heads;
    u.kvh = (pos - pre[lo]) / per_head;
    u.start = pre[lo] + u.kvh * per_head;
    const int rts = (u.fresh * a.group + kRows - 1) / kRows, lane = threadIdx.x & 31;
    u.rt = 0;
    u.tiles = attn_tiles_of<kRows, kTile>(a, u.cached, u.fresh, 0);
    if (a.masks) {
        u.rt = (pos - u.start) / (u.tiles + kHead);
        u.start += u.rt * (u.tiles + kHead);
    } else if (rts > 1) {
        for (int r0 = 0; r0 < rts; r0 += 32) {
            const int mine = r0 + lane < rts ? attn_tiles_of<kRows, kTile>(a, u.cached, u.fresh, r0 + lane) + kHead : 0;
            int v = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(Q8_FULL_MASK, v, o);
                if (lane >= o) v += x;
            }
            const unsigned past = __ballot_sync(Q8_FULL_MASK, pos < u.start + v);
            const int at = past ? __ffs(past) - 1 : 31;
            u.tiles = __shfl_sync(Q8_FULL_MASK, mine, at) - kHead;
            u.rt = r0 + at;
            const int end = __shfl_sync(Q8_FULL_MASK, v, at);
            if (past || r0 + 32 >= rts) {
                u.start += end - u.tiles - kHead;
                break;
            }
            u.start += end;
        }
    }
    return u;
}

// The unit behind u on the line (u is not the last).
template <int kRows, int kTile, int kHead>
__device__ __forceinline__ void attn_next_unit(const AttnArgs &a, const int *pre, Unit &u)
{
    u.start += u.tiles + kHead;
    if ((u.rt + 1) * kRows < u.fresh * a.group) {
        ++u.rt;
    } else {
        u.rt = 0;
        if (++u.kvh == a.kv_heads) {
            u.kvh = 0;
            do ++u.b;
            while (u.b + 1 < a.batch && pre[u.b + 1] <= u.start);  // empty sequences take no place
            attn_sequence(a, u.b, u.cached, u.fresh, u.first);
        }
    }
    u.tiles = attn_tiles_of<kRows, kTile>(a, u.cached, u.fresh, u.rt);
}

// What one packed row can see: keys below `all`, and of the fresh ones those
// set in `mask`.
struct RowSight {
    int all;
    unsigned long long mask;
};

__device__ __forceinline__ RowSight attn_sight(const AttnArgs &a, const Unit &u, int row)
{
    RowSight s;
    const int tok = attn_token(a, row);
    if (tok >= u.fresh) {  // a row of the tile that does not exist
        s.all = 0;
        s.mask = 0;
    } else if (a.masks) {
        s.all = u.cached;
        s.mask = static_cast<unsigned long long>(a.masks[u.first + tok]);
        if (u.fresh < 64) s.mask &= (1ull << u.fresh) - 1;
    } else {
        s.all = u.cached + tok + 1;
        s.mask = 0;
    }
    return s;
}

__device__ __forceinline__ bool attn_sees(const RowSight &s, int cached, int key)
{
    const unsigned f = static_cast<unsigned>(key - cached);
    return key < s.all || (f < 64u && ((s.mask >> f) & 1));
}

// Four consecutive values of a finished row (the 8 lanes of an aligned group
// of 8 hold 32 consecutive ones): y and the plane.  All lanes of the warp
// call it; `valid` says whether this lane's row exists.
template <int D>
__device__ __forceinline__ void attn_store(const AttnArgs &a, const Unit &u, int row, int c, float4 o, float l,
                                           bool valid)
{
    // a row that saw nothing has l = 0 and O = 0
    const float inv = l == 0.0f ? 0.0f : __frcp_rn(l);
    const float4 r = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
    const int tok = attn_token(a, row);
    const long long at =
        (static_cast<long long>(u.first + tok) * a.heads + u.kvh * a.group + (row - tok * a.group)) * D + c;
    if (a.y && valid) *reinterpret_cast<float4 *>(a.y + at) = r;
    if (a.qs) {
        const Q8Enc e = q8_encode8(r);
        if (valid) {
            *reinterpret_cast<uint32_t *>(a.qs + at) = e.qword;
            if ((c & 31) == 0) a.ds[at / 32] = e.dsword;
        }
    }
}

// A query value in two f16 parts: hi + lo is v to 22 bits (|v| < 2^15).
__device__ __forceinline__ void split_f16(float a, float b, uint32_t &hi, uint32_t &lo)
{
    const __half2 h = __floats2half2_rn(a, b);
    const float2 f = __half22float2(h);
    const __half2 l = __floats2half2_rn(a - f.x, b - f.y);
    hi = *reinterpret_cast<const uint32_t *>(&h);
    lo = *reinterpret_cast<const uint32_t *>(&l);
}

__device__ __forceinline__ float exp2_approx(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// 2^e for e in [-126, 127]
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }

constexpr int kAttnCtas = 152;  // the split is over this many CTAs whatever the device's count: results do not depend on it

// One call's attention as the launchers take it.
struct AttnCall {
    AttnArgs a;
    const uint8_t *k, *v;  // this layer
    int64_t layer_rows;
    int dim;
    bool int8;
};

// rows of a unit: 8 or 16 (attn_rows.cu), 128 (attn_tiles.cu)
int attn_rows_launch(const AttnCall &c, int rows, cudaStream_t s);
int attn_rows_cluster(int rows, int64_t units, int64_t max_len);  // AttnArgs::cluster
int attn_tiles_cluster(int64_t units, int64_t max_len);
int attn_tiles_launch(const AttnCall &c, cudaStream_t s);

// Joins the pieces of every unit that crosses a boundary of the split: CTA
// (c - 1, y) takes every gridDim.y-th group of rows of the unit that lies
// across the start of c's stretch, unless an earlier boundary lies in the same
// unit.  Bound by latency: the descriptor, the pieces' (m, l), their numerators,
// each one round of loads; 256 threads are kGroup rows x D/4 columns x as many
// parts of the pieces, whose sums are added in a fixed order.  Units of few
// rows have many pieces (33 for one sequence of 4097 tokens), those of 128 rows
// few.
template <int D, int kRows>
static __global__ void __launch_bounds__(256) attn_combine_kernel(const __grid_constant__ AttnArgs a)
{
    constexpr int kCols = D / 4, kGroup = kRows == 128 ? 8 : 2, kParts = 256 / (kGroup * kCols);
    __shared__ float s_f[kGroup][kAttnCtas], s_l[kGroup];
    __shared__ float4 s_o[kParts][kGroup][kCols];
    griddep_launch_dependents();
    griddep_wait();
    const int c = blockIdx.x + 1, tid = threadIdx.x;
    const int4 d0 = a.desc[2 * c], d1 = a.desc[2 * c + 1];
    if (d1.w == 0) return;
    // the unit's place, its end, and the place of its first tile
    const int u0 = d0.x, u1 = d0.y, per = d0.z, f0 = d0.w;
    if (c * per <= f0 || (c - 1) * per > f0) return;
    const int head = 2 * (c - 1) + ((c - 1) * per >= u0 ? 0 : 1);
    const int pieces = 1 + (u1 - 1) / per - c + 1;  // CTAs c .. (u1 - 1) / per, and c - 1
    auto at = [&](int k) { return k == 0 ? head : 2 * (c + k - 1); };
    Unit u;
    u.b = d1.x, u.kvh = d1.y, u.rt = d1.z;
    attn_sequence(a, u.b, u.cached, u.fresh, u.first);
    const int rows = min(kRows, u.fresh * a.group - u.rt * kRows);
    const int part = tid / (kGroup * kCols), y = (tid / kCols) % kGroup, col = (tid % kCols) * 4;
    for (int r0 = kGroup * blockIdx.y; r0 < rows; r0 += kGroup * gridDim.y) {
        // warp y: the row's (m, l) and each piece's factor
        if (tid < 32 * kGroup) {
            const int w = tid >> 5, lane = tid & 31;
            float2 ml[(kAttnCtas + 31) / 32];
            float m = -INFINITY, l = 0.0f;
#pragma unroll
            for (int j = 0; j < (kAttnCtas + 31) / 32; ++j) {
                ml[j] = make_float2(-INFINITY, 0.0f);
                if (lane + 32 * j < pieces && r0 + w < kRows) ml[j] = a.ml[at(lane + 32 * j) * kRows + r0 + w];
                m = fmaxf(m, ml[j].x);
            }
#pragma unroll
            for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(Q8_FULL_MASK, m, o));
#pragma unroll
            for (int j = 0; j < (kAttnCtas + 31) / 32; ++j) {
                const float f = ml[j].x == -INFINITY ? 0.0f : ml[j].x == m ? 1.0f : exp2_approx(ml[j].x - m);
                if (lane + 32 * j < pieces) s_f[w][lane + 32 * j] = f;
                l += f * ml[j].y;
            }
#pragma unroll
            for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(Q8_FULL_MASK, l, o);
            if (lane == 0) s_l[w] = l;
        }
        // the numerators' loads do not wait for the factors
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        bool waited = false;
        for (int k0 = part; k0 < pieces || !waited; k0 += 8 * kParts) {
            float4 x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (k0 + j * kParts < pieces && r0 + y < kRows)
                    x[j] = *reinterpret_cast<const float4 *>(
                        a.part + (static_cast<long long>(at(k0 + j * kParts)) * kRows + r0 + y) * D + col);
            if (!waited) {
                __syncthreads();
                waited = true;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (k0 + j * kParts < pieces && r0 + y < kRows) {
                    const float f = s_f[y][k0 + j * kParts];
                    o.x += f * x[j].x, o.y += f * x[j].y, o.z += f * x[j].z, o.w += f * x[j].w;
                }
        }
        s_o[part][y][tid % kCols] = o;
        __syncthreads();
        if (tid < kGroup * kCols) {
#pragma unroll
            for (int p = 1; p < kParts; ++p) {
                const float4 z = s_o[p][y][tid % kCols];
                o.x += z.x, o.y += z.y, o.z += z.z, o.w += z.w;
            }
            attn_store<D>(a, u, u.rt * kRows + r0 + y, col, o, s_l[y], r0 + y < rows);
        }
        __syncthreads();
    }
}

} // namespace q8
