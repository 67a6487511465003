// experts_rows.cu -- products of a few sorted rows an expert with their experts'
// Q8_0 matrices: a stream over the weights of the experts that have rows.
//
// The block dot products run on mma.sync m16n8k16 (16 weight rows x 8 sorted
// rows), two MMAs a block, as in the small-batch kernel of gemv.cu: exact
// integers, scaled by d_w * d_a and added in f32.  The weight codes enter as
// 1152 + q (a byte permute makes that f16 from the code, a subtraction less per
// two codes), and the accumulator starts at -1152 times the sum of the row's
// codes in the block: |sum| < 2^24, so the integer is exact all the same.
//
//   The line.  A segment is up to 8 or 16 rows of one expert (and a slice of k where a
//   row's activations would not fit shared memory); it has an item for every 16
//   weight rows.  All segments' items lie on one line, from the offsets on the
//   device, and CTA c takes an equal stretch of it.  Within one segment of its
//   stretch the CTA's warps share the items' 8-block pieces equally: a warp
//   takes a stretch of pieces, stores the items that are all its own and leaves
//   the ends to be added up through shared memory, in warp order.
//   Weights come through a ring of a warp's own, a TMA box of 16 rows x 8 blocks
//   (272 bytes a row) a slot; its next pieces are asked for across items and
//   segments.  Where rows of blocks are not 16-byte aligned each row's piece is a
//   bulk copy of its own, from the 16-byte boundary before it to the one behind.
//   Activations of a segment lie in shared memory in the order of the MMA's B
//   fragments, widened to f16 once; rows that the segment does not have are not
//   written: what lies there enters columns that are not stored.
#include "experts_common.cuh"

namespace {

__device__ unsigned int g_rows_err;

constexpr int kWarps = 16, kThreads = 32 * kWarps;
constexpr int kPiece = 8;                    // blocks
constexpr int kPitchTma = 34 * kPiece;       // 272
constexpr int kPitchAny = kPitchTma + 32;    // 304: a row may start up to 14 bytes late; 76 words, so rows g and words m fall on 32 banks
constexpr int kSlots = 2;                    // of a warp's ring
__host__ __device__ constexpr int slot_bytes(bool tma) { return 16 * (tma ? kPitchTma : kPitchAny); }
static_assert(slot_bytes(true) % 128 == 0 && slot_bytes(false) % 128 == 0, "TMA destination");

struct RowsArgs {
    q8::ExpertsArgs x;
    int groups, slices, slice_blocks;  // items of a segment, slices of k, their blocks (the last may have fewer)
    int64_t part;                      // floats from one slice's output to the next's
};

// shared memory: ring [kWarps][kSlots] | B fragments [blocks][NT][32] uint4 | scales [blocks][NT][4] float4 | rows of each expert
// | cost before each | barriers; the partial items [kWarps][2][NT][32] float4 take the fragments' place.  nt: tiles of 8 rows a
// segment has.
struct Layout {
    int act, scale, rows, cum, bar, total;
    __host__ __device__ Layout(bool tma, int nt, int blocks)
    {
        act = kWarps * kSlots * slot_bytes(tma);
        scale = act + (blocks > 2 * kWarps ? blocks : 2 * kWarps) * 512 * nt;
        rows = scale + blocks * 64 * nt;
        cum = rows + Q8_MAX_EXPERTS * 8;
        bar = cum + (Q8_MAX_EXPERTS + 2) * 4;
        total = bar + kWarps * 8 * kSlots + 128;
    }
};

struct Segment {
    int e, first, rows, slice;  // expert, its sorted rows, slice of k
    int b0, blocks;             // blocks of the slice
    int i0, i1;                 // items of this CTA's stretch, from the segment's own start (none: i0 == i1)
    int next;                   // place on the line behind them
};

// What an item costs on the line: 16 rows take 1.28 times as long as 8 (241000 cycles for 143 items, 188000).
__host__ __device__ constexpr int item_cost(int rows) { return rows > 8 ? 5 : 4; }

// Segments of an expert with `count` rows and their cost, in items of one group and slice.
template <int NT>
__device__ __forceinline__ int expert_cost(int count)
{
    const int full = count / (8 * NT), rest = count - full * 8 * NT;
    return full * item_cost(8 * NT) + (rest ? item_cost(rest) : 0);
}

// The segment at place i of the line, cut to the stretch that ends at `end`: the items that start in it.  cum[e]: cost of the
// experts before e; rows[e]: its first and their number.
template <int NT>
__device__ __forceinline__ Segment segment_at(const RowsArgs &a, const int2 *rows, const int *cum, int i, int end)
{
    int lo = 0, hi = a.x.experts;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cum[mid] <= i)
            lo = mid;
        else
            hi = mid;
    }
    const int first = rows[lo].x, count = rows[lo].y;
    const int whole = item_cost(8 * NT) * a.groups * a.slices;
    const int chunk = min((i - cum[lo]) / whole, (count - 1) / (8 * NT));
    Segment s;
    s.e = lo;
    s.first = first + chunk * 8 * NT;
    s.rows = min(8 * NT, count - chunk * 8 * NT);
    const int cost = item_cost(s.rows);
    s.slice = (i - cum[lo] - chunk * whole) / (cost * a.groups);
    s.b0 = s.slice * a.slice_blocks;
    s.blocks = min(a.slice_blocks, a.x.nb - s.b0);
    const int start = cum[lo] + chunk * whole + s.slice * cost * a.groups, stop = start + cost * a.groups;
    s.i0 = (i - start + cost - 1) / cost;
    s.i1 = end >= stop ? a.groups : (end - start + cost - 1) / cost;
    s.next = min(stop, end);
    return s;
}

// The pieces that warp w takes of a segment's items: units u .. end - 1, unit = item * pieces + piece.
__device__ __forceinline__ int share(int units, int w) { return static_cast<int>(static_cast<int64_t>(units) * w / kWarps); }

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Four codes -> 1152 + q as two f16x2 words.
__device__ __forceinline__ void biased_f16(uint32_t q, uint32_t &lo, uint32_t &hi)
{
    const uint32_t x = q ^ 0x80808080u;
    lo = __byte_perm(x, 0x64646464u, 0x5140);
    hi = __byte_perm(x, 0x64646464u, 0x5342);
}

// A 16 x 8 tile's values: this lane's rows g and g + 8 of the weights, sorted rows 8t + 2m and 8t + 2m + 1.
__device__ __forceinline__ void store_item(const RowsArgs &a, const Segment &s, int item, int n16, int g, int m, int t, float4 v)
{
    const int i = s.i0 + item;
    const bool second = i >= n16;
    const int row = 16 * (second ? i - n16 : i) + g;
    float *out = a.x.out + s.slice * a.part + (second ? a.x.n : 0) + row;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int r = 8 * t + 2 * m + k;
        if (r < s.rows && q8::source_row(a.x, s.first + r) >= 0) {
            float *o = out + (s.first + r) * a.x.ld;
            if (row < a.x.n) o[0] = k ? v.y : v.x;
            if (row + 8 < a.x.n) o[8] = k ? v.w : v.z;
        }
    }
}

// One unit: 16 weight rows x up to 8 blocks against T tiles of 8 rows.  late: byte of the slot's rows where the pieces start.
template <bool kTma, int NT, int T>
__device__ __forceinline__ void unit(const uint8_t *slot, int late, int cb, const uint4 *bf, const float4 *sc, int g, int m,
                                     float2 (&acc)[NT][2])
{
    const int pitch = kTma ? kPitchTma / 4 : kPitchAny / 4;
    const uint32_t *w0 = reinterpret_cast<const uint32_t *>(slot) + g * pitch, *w1 = w0 + 8 * pitch;
#pragma unroll
    for (int j = 0; j < kPiece; ++j) {
        if (!kTma && j >= cb) break;
        uint32_t q[4];  // words m of rows g and g + 8, then words m + 4
        float dw0, dw1;
        if (kTma) {
            const int w = (34 * j) >> 2;
            const uint32_t h0 = w0[w], h1 = w1[w];
            if (j & 1) {  // the scale in the upper half, codes in whole words
                dw0 = __half2float(__ushort_as_half(static_cast<unsigned short>(h0 >> 16)));
                dw1 = __half2float(__ushort_as_half(static_cast<unsigned short>(h1 >> 16)));
                q[0] = w0[w + 1 + m], q[1] = w1[w + 1 + m], q[2] = w0[w + 5 + m], q[3] = w1[w + 5 + m];
            } else {
                dw0 = __half2float(__ushort_as_half(static_cast<unsigned short>(h0 & 0xffffu)));
                dw1 = __half2float(__ushort_as_half(static_cast<unsigned short>(h1 & 0xffffu)));
                q[0] = __byte_perm(w0[w + m], w0[w + m + 1], 0x5432), q[1] = __byte_perm(w1[w + m], w1[w + m + 1], 0x5432);
                q[2] = __byte_perm(w0[w + m + 4], w0[w + m + 5], 0x5432);
                q[3] = __byte_perm(w1[w + m + 4], w1[w + m + 5], 0x5432);
            }
        } else {
            const int byte = late + 34 * j, w = byte >> 2;
            const uint32_t sel = byte & 2 ? 0x7654u : 0x5432u;
            const int up = byte & 2 ? 16 : 0;
            dw0 = __half2float(__ushort_as_half(static_cast<unsigned short>(w0[w] >> up)));
            dw1 = __half2float(__ushort_as_half(static_cast<unsigned short>(w1[w] >> up)));
            q[0] = __byte_perm(w0[w + m], w0[w + m + 1], sel), q[1] = __byte_perm(w1[w + m], w1[w + m + 1], sel);
            q[2] = __byte_perm(w0[w + m + 4], w0[w + m + 5], sel), q[3] = __byte_perm(w1[w + m + 4], w1[w + m + 5], sel);
        }
        uint32_t f0[4], f1[4];
        biased_f16(q[0], f0[0], f0[2]);
        biased_f16(q[1], f0[1], f0[3]);
        biased_f16(q[2], f1[0], f1[2]);
        biased_f16(q[3], f1[1], f1[3]);
#pragma unroll
        for (int t = 0; t < T; ++t) {
            const uint4 b = bf[(j * NT + t) * 32];
            const float4 d = sc[(j * NT + t) * 4];
            float c[4] = {d.z, d.w, d.z, d.w};
            mma16816(c, f0, b.x, b.y);
            mma16816(c, f1, b.z, b.w);
            const float2 da = make_float2(d.x, d.y);
            acc[t][0] = __ffma2_rn(__fmul2_rn(make_float2(dw0, dw0), da), make_float2(c[0], c[1]), acc[t][0]);
            acc[t][1] = __ffma2_rn(__fmul2_rn(make_float2(dw1, dw1), da), make_float2(c[2], c[3]), acc[t][1]);
        }
    }
}

template <bool kTma, int NT>
__global__ void __launch_bounds__(kThreads, 1)
experts_rows_kernel(const __grid_constant__ RowsArgs a, const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmW2)
{
    extern __shared__ __align__(128) uint8_t sm[];
    __shared__ int scan[kWarps], source[8 * NT];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, m = lane & 3;
    const Layout L(kTma, NT, a.slice_blocks);
    int *cum = reinterpret_cast<int *>(sm + L.cum);
    int2 *rows = reinterpret_cast<int2 *>(sm + L.rows);  // first and number of each expert's
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + L.bar) + warp * kSlots;
    uint8_t *ring = sm + warp * kSlots * slot_bytes(kTma);
    if (lane == 0) {
        for (int i = 0; i < kSlots; ++i) q8::mbar_init(bars + i, 1);
        q8::fence_mbar_init();
    }
    q8::griddep_launch_dependents();
    q8::griddep_wait();
    bool many = false;  // a line that passes 31 bits: possible only where offsets fall, so that experts overlap; nothing is computed
    {                   // cost of the experts before each: two experts a thread
        int n[2], falls = 0;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            n[k] = 0;
            if (2 * tid + k < a.x.experts) {
                const q8::ExpertRows x = q8::expert_rows_of(a.x, 2 * tid + k);
                if (x.bad && blockIdx.x == 0) atomicOr(&g_rows_err, q8::kErrData);
                falls |= x.bad;
                rows[2 * tid + k] = make_int2(x.first, x.count);
                n[k] = expert_cost<NT>(x.count) * a.slices * a.groups;
            }
        }
        int v = n[0] + n[1];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(Q8_FULL_MASK, v, o);
            if (lane >= o) v += u;
        }
        if (lane == 31) scan[warp] = v;
        many = __syncthreads_or(falls) && a.x.many;
        for (int w = 0; w < warp; ++w) v += scan[w];
        if (2 * tid < a.x.experts) cum[2 * tid + 1] = v - n[1];
        if (2 * tid + 1 < a.x.experts) cum[2 * tid + 2] = v;
        if (tid == 0) cum[0] = 0;
        __syncthreads();
    }
    const int line = many ? 0 : cum[a.x.experts];
    const int end = static_cast<int>(static_cast<int64_t>(line) * (blockIdx.x + 1) / gridDim.x);
    int at = static_cast<int>(static_cast<int64_t>(line) * blockIdx.x / gridDim.x);
    const int n16 = (a.x.n + 15) / 16;

    // what this warp asks for: its units of this and later segments
    Segment fs = {};
    int fu = 0, fend = 0, fpieces = 1, fnext = at, fitem = 0, fpiece = 0;
    uint32_t asked = 0, used = 0;
    auto fetch = [&]() {  // the next unit into the next slot; every slot it goes to has been read
        while (fu == fend) {
            if (fnext >= end) return;
            fs = segment_at<NT>(a, rows, cum, fnext, end);
            fnext = fs.next;
            fpieces = (fs.blocks + kPiece - 1) / kPiece;
            const int units = (fs.i1 - fs.i0) * fpieces;
            fu = share(units, warp), fend = share(units, warp + 1);
            fitem = fu / fpieces, fpiece = fu - fitem * fpieces;
        }
        const int item = fs.i0 + fitem, piece = fpiece;
        if (++fpiece == fpieces) fpiece = 0, ++fitem;
        const bool second = item >= n16;
        const int row = 16 * (second ? item - n16 : item), b = fs.b0 + piece * kPiece;
        uint8_t *slot = ring + (asked % kSlots) * slot_bytes(kTma);
        uint64_t *bar = bars + asked % kSlots;
        if (kTma) {
            if (lane == 0) {
                q8::mbar_arrive_expect_tx(bar, 16 * kPitchTma);
                q8::tma_load_2d(q8::smem_u32(slot), second ? &tmW2 : &tmW, b * 17, fs.e * a.x.n + row, q8::smem_u32(bar));
            }
        } else {
            const uint8_t *w = second ? a.x.w2 : a.x.w;
            const int cb = min(kPiece, fs.b0 + fs.blocks - b);
            const int64_t most = static_cast<int64_t>(a.x.experts) * a.x.n * a.x.nb * 34, whole = most & ~int64_t(15);
            const int64_t from =
                ((static_cast<int64_t>(fs.e) * a.x.n + min(row + (lane & 15), a.x.n - 1)) * a.x.nb + b) * 34;
            const int64_t start = from & ~int64_t(15), stop = (from + cb * 34 + 15) & ~int64_t(15);
            const int bytes = lane < 16 ? static_cast<int>(max(min(stop, whole) - start, int64_t(0))) : 0;
            uint8_t *dst = slot + (lane & 15) * kPitchAny;
            const int all = __reduce_add_sync(Q8_FULL_MASK, bytes);
            if (lane == 0) q8::mbar_arrive_expect_tx(bar, all);
            __syncwarp();
            if (bytes) q8::bulk_g2s(dst, w + start, bytes, bar);
            if (lane < 16 && stop > whole)  // the last bytes of the last matrix, where they do not fill 16
                for (int64_t o = max(whole, start); o < most; o += 2)
                    *reinterpret_cast<uint16_t *>(dst + (o - start)) = *reinterpret_cast<const uint16_t *>(w + o);
        }
        ++asked;
        ++fu;
    };
    for (int i = 0; i < kSlots; ++i) fetch();

    bool dead = false;  // a wait ran out
    while (at < end) {
        const Segment s = segment_at<NT>(a, rows, cum, at, end);
        if (s.i0 == s.i1) {
            at = s.next;
            continue;
        }
        const int pieces = (s.blocks + kPiece - 1) / kPiece, units = (s.i1 - s.i0) * pieces;
        if (tid < s.rows) {
            const int64_t src = q8::source_row(a.x, s.first + tid);
            if (src < 0) atomicOr(&g_rows_err, q8::kErrData);
            source[tid] = src < 0 ? 0 : static_cast<int>(src);  // out of range: any, it is not stored
        }
        __syncthreads();  // and the segment before is done with the activations and the partial items
        // activations: lane (g, m) of a fragment has words m and m + 4 of row g's block.  A thread takes half a block (words 4 h ..
        // 4 h + 3), four of them in flight, since under the stream a load takes some 2 us
        const int tasks = s.blocks * s.rows * 2;
        for (int i0 = tid; i0 - lane < tasks; i0 += 4 * kThreads) {  // whole warps
            uint4 w[4] = {};
            uint32_t d[4] = {};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int i = i0 + k * kThreads, h = i & 1, rb = i >> 1, b = rb / s.rows, r = rb - b * s.rows;
                if (i < tasks) {
                    const int64_t at_block = static_cast<int64_t>(source[r]) * a.x.nb + s.b0 + b;
                    w[k] = __ldg(reinterpret_cast<const uint4 *>(a.x.qs) + at_block * 2 + h);
                    d[k] = __ldg(a.x.ds + at_block);
                }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int i = i0 + k * kThreads, h = i & 1, rb = i >> 1, b = rb / s.rows, r = rb - b * s.rows;
                const uint32_t q[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
                int sum = 0;
#pragma unroll
                for (int mm = 0; mm < 4; ++mm) sum = q8::dp4a(q[mm], 0x01010101u, sum);
                sum += __shfl_xor_sync(Q8_FULL_MASK, sum, 1);  // the block's other half
                if (i >= tasks) continue;
                uint2 *f = reinterpret_cast<uint2 *>(sm + L.act) + ((b * NT + (r >> 3)) * 32 + 4 * (r & 7)) * 2 + h;
#pragma unroll
                for (int mm = 0; mm < 4; ++mm) {
                    uint2 o;
                    q8::i8x4_to_f16x4(q[mm], o.x, o.y);
                    f[2 * mm] = o;
                }
                // row 2m + x of a tile: scale at 4m + x, start of the accumulator at 4m + 2 + x
                float *sc = reinterpret_cast<float *>(sm + L.scale) + (b * NT + (r >> 3)) * 16 + 4 * ((r & 7) >> 1) + (r & 1);
                sc[2 * h] = h ? -1152.0f * static_cast<float>(sum)
                              : __half2float(__ushort_as_half(static_cast<unsigned short>(d[k] & 0xffffu)));
            }
        }
        __syncthreads();
        const int u0 = share(units, warp), u1 = share(units, warp + 1);
        float2 acc[NT][2];               // rows g and g + 8 of the weights
        float4 head[NT], tail[NT];       // the parts of the first and the last item that other warps have pieces of
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            acc[t][0] = acc[t][1] = make_float2(0.f, 0.f);
            head[t] = tail[t] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        int item = u0 / pieces, piece = u0 - item * pieces;
        const int item0 = item;
        for (int u = u0; u < u1; ++u) {
            const int slot_i = used % kSlots;
            if (!__all_sync(Q8_FULL_MASK, q8::mbar_wait_bounded(bars + slot_i, (used / kSlots) & 1u))) {
                dead = true;
                if (lane == 0) atomicOr(&g_rows_err, q8::kErrTimeout);
                break;  // no slot is asked for again; the CTA leaves at the segment's end
            }
            const uint8_t *slot = ring + slot_i * slot_bytes(kTma);
            const int cb = min(kPiece, s.blocks - piece * kPiece);
            int late = 0;  // where the row's piece starts in its slot (rows g and g + 8 alike: 8 rows are a multiple of 16 bytes)
            if (!kTma) {
                const int second = s.i0 + item >= n16;
                // rows behind the matrix are copies of its last one, whose piece starts elsewhere: they are not stored
                const int row = 16 * (s.i0 + item - (second ? n16 : 0)) + g;
                late = static_cast<int>(((static_cast<int64_t>(s.e) * a.x.n + min(row, a.x.n - 1)) * a.x.nb + s.b0 + piece * kPiece) * 34) & 15;
            }
            const uint4 *bf = reinterpret_cast<const uint4 *>(sm + L.act) + piece * kPiece * NT * 32 + lane;
            const float4 *sc = reinterpret_cast<const float4 *>(sm + L.scale) + piece * kPiece * NT * 4 + m;
            if (NT == 1 || s.rows <= 8)
                unit<kTma, NT, 1>(slot, late, cb, bf, sc, g, m, acc);
            else
                unit<kTma, NT, NT>(slot, late, cb, bf, sc, g, m, acc);
            __syncwarp();  // all lanes have read the slot
            ++used;
            fetch();
            if (piece == pieces - 1 || u == u1 - 1) {
                const int first_u = max(u0, item * pieces);
                const bool whole = first_u == item * pieces && piece == pieces - 1;
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const float4 v = make_float4(acc[t][0].x, acc[t][0].y, acc[t][1].x, acc[t][1].y);
                    if (whole) {
                        if (8 * t < s.rows) store_item(a, s, item, n16, g, m, t, v);
                    } else if (item == item0) {
                        head[t] = v;
                    } else {
                        tail[t] = v;
                    }
                    acc[t][0] = acc[t][1] = make_float2(0.f, 0.f);
                }
            }
            if (++piece == pieces) piece = 0, ++item;
        }
        const bool failed = __syncthreads_or(dead);  // the fragments have been read: the partial items take their place
        float4 *parts = reinterpret_cast<float4 *>(sm + L.act) + lane;
#pragma unroll
        for (int t = 0; t < NT; ++t) parts[(2 * warp * NT + t) * 32] = head[t], parts[((2 * warp + 1) * NT + t) * 32] = tail[t];
        __syncthreads();
        // items that several warps share: warp w adds up the one that starts among its pieces and ends among later ones'
        if (u1 > u0 && piece != 0 && !failed && item * pieces >= u0) {
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                if (8 * t >= s.rows) break;
                float4 sum = item == item0 ? head[t] : tail[t];
                for (int w = warp + 1; w < kWarps; ++w) {  // every later warp with pieces of it: its first item
                    const int v0 = share(units, w), v1 = share(units, w + 1);
                    if (v0 >= (item + 1) * pieces) break;
                    if (v1 == v0) continue;
                    const float4 x = parts[(2 * w * NT + t) * 32];
                    sum.x += x.x, sum.y += x.y, sum.z += x.z, sum.w += x.w;
                }
                store_item(a, s, item, n16, g, m, t, sum);
            }
        }
        at = s.next;
        if (failed) break;
    }
    // copies in flight land before the CTA exits (after a wait ran out; else there are none)
    for (; used < asked; ++used)
        if (!q8::mbar_wait_bounded(bars + used % kSlots, (used / kSlots) & 1u, Q8_DRAIN_LIMIT_NS) && lane == 0)
            atomicOr(&g_rows_err, q8::kErrTimeout);
}

// y = sum of the slices' outputs, in order, of the rows that have products; kJoin columns of a row at a time.
constexpr int kJoin = 512;
__global__ void __launch_bounds__(256) experts_join_kernel(const __grid_constant__ q8::ExpertsArgs a, const float *__restrict__ part, int slices)
{
    q8::griddep_launch_dependents();
    q8::griddep_wait();
    const int64_t stride = a.pairs * a.ld;
    const int segs = static_cast<int>((a.ld + kJoin - 1) / kJoin), first = a.offsets[0], last = a.offsets[a.experts];
    const int seen = q8::bad_offsets(a);
    int at = blockIdx.x, total = a.pairs * segs;  // below 25 * 1024 rows of 2^22 / kJoin
    bool known = false, bad = false;
    do {  // the first round's loads go out with those of the offsets, whatever these say
        const int r = at / segs;
        const int64_t c0 = (at - r * segs) * kJoin + threadIdx.x, row = r * a.ld;
        const int pair = at < total && a.rows ? a.rows[r] : 0;
        float v[kJoin / 256];
        for (int k = 0; k < slices; ++k) {
            const float *p = part + k * stride + row + c0;
#pragma unroll
            for (int x = 0; x < kJoin / 256; ++x) {
                const float add = at < total && c0 + 256 * x < a.ld ? p[256 * x] : 0.0f;
                v[x] = k ? v[x] + add : add;
            }
        }
        if (!known) {
            bad = __syncthreads_or(seen);
            known = true;
            if (bad && a.many) return;  // nothing has been computed
            total = min(max(last, 0), a.pairs) * segs;
        }
        if (at >= total || r < first || !q8::source_ok(a, r, pair) || (bad && !q8::expert_has(a, r))) continue;
#pragma unroll
        for (int x = 0; x < kJoin / 256; ++x)
            if (c0 + 256 * x < a.ld) a.out[row + c0 + 256 * x] = v[x];
    } while ((at += gridDim.x) < total);
}

constexpr int kMaxSmem = 227 * 1024 - 1024;

// Tiles of 8 rows a segment has, and the slices of k: as few as fit its activations beside the ring, of whole pieces.
struct Plan {
    int nt, slices, slice_blocks, smem;
};

Plan plan_of(int64_t experts, int64_t pairs, int nb)
{
    const bool tma = nb % kPiece == 0;
    Plan p = {pairs > 4 * experts ? 2 : 1, 1, nb, 0};
    while (Layout(tma, p.nt, p.slice_blocks).total > kMaxSmem) {
        ++p.slices;
        p.slice_blocks = ((nb + p.slices - 1) / p.slices + kPiece - 1) / kPiece * kPiece;
    }
    p.slices = (nb + p.slice_blocks - 1) / p.slice_blocks;
    p.smem = Layout(tma, p.nt, p.slice_blocks).total;
    return p;
}

int groups_of(const q8::ExpertsArgs &x) { return (x.n + 15) / 16 * (x.w2 ? 2 : 1); }

template <bool kTma, int NT>
int launch(const RowsArgs &a, const CUtensorMap &mw, const CUtensorMap &mw2, int smem, unsigned grid, int slot, cudaStream_t s)
{
    if (!q8::set_max_dynamic_smem(reinterpret_cast<const void *>(experts_rows_kernel<kTma, NT>), kMaxSmem, slot))
        return Q8_ERR_LAUNCH;
    return q8::launch_pdl(experts_rows_kernel<kTma, NT>, dim3(grid), dim3(kThreads), smem, s, a, mw, mw2);
}

} // namespace

namespace q8 {

int experts_rows_slices(int64_t experts, int64_t pairs, int64_t nb)
{
    return plan_of(experts, pairs, static_cast<int>(nb)).slices;
}

bool experts_rows_many(const ExpertsArgs &x)
{
    const int64_t items = static_cast<int64_t>(experts_rows_slices(x.experts, x.pairs, x.nb)) * groups_of(x);
    return (x.experts / 2 + 1) * (static_cast<int64_t>(x.pairs) / 8 + 1) * item_cost(8) * items > INT32_MAX;
}

// out: slices x pairs x ld floats where there are several, else the rows themselves.
int experts_rows_launch(const ExpertsArgs &x, float *out, cudaStream_t s)
{
    const Plan p = plan_of(x.experts, x.pairs, x.nb);
    RowsArgs a = {};
    a.x = x;
    a.x.out = out;
    a.groups = groups_of(x);
    a.slices = p.slices, a.slice_blocks = p.slice_blocks;
    a.part = static_cast<int64_t>(x.pairs) * x.ld;
    const bool tma = x.nb % kPiece == 0;
    CUtensorMap mw = {}, mw2 = {};
    const uint64_t rows = static_cast<uint64_t>(x.experts) * x.n, pitch = static_cast<uint64_t>(x.nb) * 34;
    if (tma && (!make_map_2d(&mw, CU_TENSOR_MAP_DATA_TYPE_UINT16, x.w, pitch / 2, rows, pitch, kPitchTma / 2, 16,
                             CU_TENSOR_MAP_SWIZZLE_NONE) ||
                (x.w2 && !make_map_2d(&mw2, CU_TENSOR_MAP_DATA_TYPE_UINT16, x.w2, pitch / 2, rows, pitch, kPitchTma / 2, 16,
                                      CU_TENSOR_MAP_SWIZZLE_NONE))))
        return Q8_ERR_LAUNCH;
    const unsigned grid = static_cast<unsigned>(device_sm_count());
    if (p.nt == 1)
        return tma ? launch<true, 1>(a, mw, mw2, p.smem, grid, 52, s) : launch<false, 1>(a, mw, mw2, p.smem, grid, 53, s);
    return tma ? launch<true, 2>(a, mw, mw2, p.smem, grid, 54, s) : launch<false, 2>(a, mw, mw2, p.smem, grid, 55, s);
}

int experts_join_launch(const float *part, int slices, const ExpertsArgs &x, cudaStream_t s)
{
    const int64_t ctas = x.pairs * ((x.ld + kJoin - 1) / kJoin), cap = static_cast<int64_t>(device_sm_count()) * 8;
    return launch_pdl(experts_join_kernel, dim3(static_cast<unsigned>(ctas < cap ? ctas : cap)), dim3(256), 0, s, x, part, slices);
}

unsigned int *experts_rows_error_word()
{
    void *p = nullptr;
    return cudaGetSymbolAddress(&p, g_rows_err) == cudaSuccess ? static_cast<unsigned int *>(p) : nullptr;
}

} // namespace q8
