// kv_cache.cu -- the paged key/value cache's bookkeeping: the step plan, the
// append of new k/v rows and the move of an accepted path.
#include <type_traits>

#include "kv_common.cuh"

namespace {

__device__ unsigned int g_kv_err;

// ---------------------------------------------------------------------------
// q8_kv_plan.  Everything is a prefix sum over sequences followed by
// independent work per page, token and node:
//     starts[b] = sum_{b' < b} fresh[b'],  base[b] = sum_{b' < b} opened[b'].
// A CTA owns kPlanSeqs consecutive sequences.  It adds up the sequences before
// its own by itself (at most 4096 pairs of integers, from L2, two per thread
// and round) instead of waiting for a scan kernel or for its neighbours, so
// the plan is one launch of independent CTAs and its time is one launch's
// latency.  gridDim.y CTAs share a segment's tokens when a few sequences
// bring many; the ancestor sets are the work of the first of them, two trees a
// warp, which is what many trees wait for.  Measured on the device: 1 sequence
// 2.8 us, 509 trees of up to 64 nodes 6.4 us.
// ---------------------------------------------------------------------------
constexpr int kPlanSeqs = 32, kPlanThreads = 512;

struct PlanArgs {
    const int32_t *cached, *fresh, *held, *free_pages, *parents;
    int32_t *table, *starts, *slots, *positions, *needed, *held_out;
    long long *masks;
    long long n_free, max_pages, tokens;
    int batch, page, n_pages;
};

struct PlanSeq {  // one sequence's lengths in pages and tokens, after the checks
    int fresh, cached, held, want;
    bool bad;
};

__device__ __forceinline__ PlanSeq plan_seq(const PlanArgs &a, int b)
{
    PlanSeq s;
    s.fresh = a.fresh[b];
    s.cached = a.cached[b];
    s.bad = s.fresh < 0 || s.cached < 0 || static_cast<long long>(s.cached) + s.fresh > 0x7fffffffll;
    if (s.fresh < 0) s.fresh = 0;  // its rows still count, so that the others keep their places
    if (s.bad) s.cached = 0;
    s.held = a.held ? a.held[b] : (s.cached + a.page - 1ll) / a.page;
    const long long want = (static_cast<long long>(s.cached) + s.fresh + a.page - 1) / a.page;
    // rows that would not fit open no page: their tokens get no slot
    if (s.held < 0 || s.held > a.max_pages || static_cast<long long>(s.held) * a.page < s.cached || want > a.max_pages ||
        (a.parents && s.fresh > Q8_TREE_MAX_NODES))
        s.bad = true;
    s.want = s.bad ? 0 : static_cast<int>(want);
    if (s.held < 0) s.held = 0;
    return s;
}

__global__ void __launch_bounds__(kPlanThreads) kv_plan_kernel(const __grid_constant__ PlanArgs a)
{
    __shared__ long long s_sum[2][kPlanThreads / 32];
    __shared__ long long s_start[kPlanSeqs + 1], s_base[kPlanSeqs];
    __shared__ int s_cached[kPlanSeqs], s_fresh[kPlanSeqs], s_held[kPlanSeqs], s_want[kPlanSeqs], s_bad[kPlanSeqs];
    q8::griddep_launch_dependents();
    q8::griddep_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int seg = blockIdx.x * kPlanSeqs;
    bool err = false;

    long long nf = 0, np = 0;
    for (int b = tid; b < seg; b += kPlanThreads) {
        const PlanSeq s = plan_seq(a, b);
        nf += s.fresh;
        np += max(0, s.want - s.held);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        nf += __shfl_xor_sync(Q8_FULL_MASK, nf, o);
        np += __shfl_xor_sync(Q8_FULL_MASK, np, o);
    }
    if (lane == 0) s_sum[0][warp] = nf, s_sum[1][warp] = np;
    __syncthreads();
    if (warp == 0) {
        long long f0 = lane < kPlanThreads / 32 ? s_sum[0][lane] : 0, p0 = lane < kPlanThreads / 32 ? s_sum[1][lane] : 0;
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            f0 += __shfl_xor_sync(Q8_FULL_MASK, f0, o);
            p0 += __shfl_xor_sync(Q8_FULL_MASK, p0, o);
        }
        PlanSeq s = {0, 0, 0, 0, false};
        const bool in = seg + lane < a.batch;
        if (in) s = plan_seq(a, seg + lane);
        err |= s.bad;
        const long long mine = max(0, s.want - s.held);
        long long fi = s.fresh, pi = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long x = __shfl_up_sync(Q8_FULL_MASK, fi, o), y = __shfl_up_sync(Q8_FULL_MASK, pi, o);
            if (lane >= o) fi += x, pi += y;
        }
        s_start[lane] = f0 + fi - s.fresh;
        s_base[lane] = p0 + pi - mine;
        s_cached[lane] = s.cached;
        s_fresh[lane] = s.fresh;
        s_held[lane] = s.held;
        s_want[lane] = s.want;
        s_bad[lane] = s.bad;
        if (lane == 31) s_start[32] = f0 + fi;
        if (in && blockIdx.y == 0) {
            // sums past 32 bits are past `tokens` as well: capped, and reported below
            const long long end = f0 + fi;
            a.starts[seg + lane] = static_cast<int32_t>(min(end - s.fresh, 0x7fffffffll));
            if (a.held_out) a.held_out[seg + lane] = s.bad ? s.held : max(s.want, s.held);
            if (end > a.tokens) err = true;
            if (seg + lane == a.batch - 1) {
                a.starts[a.batch] = static_cast<int32_t>(min(end, 0x7fffffffll));
                *a.needed = static_cast<int32_t>(min(p0 + pi, 0x7fffffffll));
            }
        }
    }
    __syncthreads();

    const int nseq = min(kPlanSeqs, a.batch - seg);
    // page i of a sequence, opened now or held already; -1 when it has none
    auto page_of = [&](int q, int i) -> int {
        int p;
        if (i < s_held[q]) {
            p = a.table[static_cast<long long>(seg + q) * a.max_pages + i];
        } else {
            const long long at = s_base[q] + (i - s_held[q]);
            if (at >= a.n_free) return -1;  // ran out: `needed` says so
            p = a.free_pages[at];
        }
        if (p < 0 || p >= a.n_pages) {
            err = true;
            return -1;
        }
        return p;
    };

    if (blockIdx.y == 0)
        for (int q = warp; q < nseq; q += kPlanThreads / 32)
            // -1 where there is no page: a row used before holds ids in range that belong to other sequences by now
            for (int i = s_held[q] + lane; i < s_want[q]; i += 32)
                a.table[static_cast<long long>(seg + q) * a.max_pages + i] = page_of(q, i);

    const long long t1 = min(s_start[kPlanSeqs], a.tokens);
    for (long long t = s_start[0] + tid + static_cast<long long>(kPlanThreads) * blockIdx.y; t < t1;
         t += static_cast<long long>(kPlanThreads) * gridDim.y) {
        int q = 0;  // the last sequence of the segment that starts at or before t (empty ones are passed over)
#pragma unroll
        for (int o = 16; o; o >>= 1)
            if (s_start[q + o] <= t) q += o;
        const int pos = s_cached[q] + static_cast<int>(t - s_start[q]);
        int slot = -1;
        if (!s_bad[q]) {
            const int i = pos / a.page, p = page_of(q, i);
            if (p >= 0) slot = p * a.page + (pos - i * a.page);
        }
        a.slots[t] = slot;
        if (!a.parents) a.positions[t] = pos;
    }

    // Ancestor sets by pointer jumping: after round r a node knows the nodes
    // up to 2^r steps above it; six rounds cover 64 nodes.  A warp takes a
    // tree, lane l its nodes l and l + 32.
    if (a.parents && blockIdx.y == 0)
        for (int q = warp; q < nseq; q += kPlanThreads / 32) {
            const long long s0 = s_start[q];
            const int n = static_cast<int>(max(0ll, min(static_cast<long long>(s_fresh[q]), a.tokens - s0)));
            if (s_bad[q] && s_fresh[q] > Q8_TREE_MAX_NODES) {
                for (int i = lane; i < n; i += 32) a.masks[s0 + i] = 0, a.positions[s0 + i] = s_cached[q];
                continue;
            }
            unsigned long long anc[2];
            int up[2];
            bool wrong = false;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int i = lane + 32 * e;
                up[e] = i < n ? a.parents[s0 + i] : -1;
                if (up[e] < -1 || up[e] >= i) up[e] = -1, wrong = true;
                anc[e] = i < n ? 1ull << i : 0ull;
            }
            if (__any_sync(Q8_FULL_MASK, wrong)) {  // not a tree: no node sees another
                err = true;
#pragma unroll
                for (int e = 0; e < 2; ++e) up[e] = -1, anc[e] = 0;
            }
#pragma unroll
            for (int r = 0; r < 6; ++r) {
                unsigned long long got[2];
                int next[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int src = up[e] & 31;
                    const unsigned long long m0 = __shfl_sync(Q8_FULL_MASK, anc[0], src);
                    const unsigned long long m1 = __shfl_sync(Q8_FULL_MASK, anc[1], src);
                    const int u0 = __shfl_sync(Q8_FULL_MASK, up[0], src), u1 = __shfl_sync(Q8_FULL_MASK, up[1], src);
                    got[e] = up[e] < 0 ? 0ull : up[e] < 32 ? m0 : m1;
                    next[e] = up[e] < 0 ? -1 : up[e] < 32 ? u0 : u1;
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) anc[e] |= got[e], up[e] = next[e];
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int i = lane + 32 * e;
                if (i < n) {
                    a.masks[s0 + i] = s_bad[q] ? 0 : static_cast<long long>(anc[e]);  // refused: its tokens have no slots
                    a.positions[s0 + i] = s_cached[q] + max(0, __popcll(anc[e]) - 1);
                }
            }
        }

    if (seg + nseq == a.batch)  // rows behind the last sequence
        for (long long t = max(s_start[kPlanSeqs], 0ll) + tid + static_cast<long long>(kPlanThreads) * blockIdx.y;
             t < a.tokens; t += static_cast<long long>(kPlanThreads) * gridDim.y)
            a.slots[t] = -1;
    if (err) atomicOr(&g_kv_err, q8::kErrData);
}

// ---------------------------------------------------------------------------
// q8_kv_append.  A row (one head of one token) is D/4 lanes with a float4
// each, so a warp takes 1 (D = 128) or 2 (D = 64) rows at a time; the row's
// amax is a shuffle over those lanes.  4 bytes are read and 2 or 1 written per
// value.  Four rows per lane group are loaded before the first is encoded, so
// that a prompt's call keeps enough bytes in flight; the loads do not depend on
// the slot, which is looked up meanwhile.  Not bound by memory: a prompt of 3325
// tokens is one wave of CTAs that load, then encode (59 % of the issue slots
// while an SM has work, most waits for the loads), and the launch is half the
// time.
// ---------------------------------------------------------------------------
// Its places are found by products instead of divisions, of which a thread
// would do twelve.  Measured: 3325 tokens of 4 heads of 128 values into an int8
// cache (17.1 MB) 5.6 us on the device, 3.0 TB/s, 7.1 with divisions; 1 token
// 1.2 us, a launch.
constexpr int kAppendThreads = 256, kAppendRows = 4;

struct AppendArgs {
    const float *k, *v;
    const int32_t *slots;
    uint8_t *kc, *vc;  // this layer's k and v
    float *ks, *vs;
    int rows;          // tokens * kv_heads, of k and again of v
    int kv_heads, page, n_slots;
    unsigned heads_inv, page_inv;  // q8::kv_inverse
};

template <int D, bool kInt8>
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(const __grid_constant__ AppendArgs a)
{
    constexpr int L = D / 4;                     // lanes of a row
    constexpr int kGroups = kAppendThreads / L;  // rows of a CTA at a time
    q8::griddep_launch_dependents();
    q8::griddep_wait();
    const int sub = threadIdx.x % L, grp = threadIdx.x / L;
    const int r0 = blockIdx.x * (kGroups * kAppendRows) + grp;
    float4 x[kAppendRows];
    int slot[kAppendRows];
#pragma unroll
    for (int u = 0; u < kAppendRows; ++u) {
        const int r = r0 + u * kGroups;
        slot[u] = -1;
        if (r < 2 * a.rows) {
            const bool is_v = r >= a.rows;
            const int i = is_v ? r - a.rows : r;
            x[u] = __ldg(reinterpret_cast<const float4 *>((is_v ? a.v : a.k) + static_cast<long long>(i) * D) + sub);
            slot[u] = a.slots[q8::kv_divide(i, a.kv_heads, a.heads_inv)];
        }
    }
#pragma unroll
    for (int u = 0; u < kAppendRows; ++u) {
        const int r = r0 + u * kGroups;
        if (slot[u] >= a.n_slots) {
            if (sub == 0) atomicOr(&g_kv_err, q8::kErrData);
            slot[u] = -1;
        }
        const bool is_v = r >= a.rows;
        const int i = is_v ? r - a.rows : r, h = i - q8::kv_divide(i, a.kv_heads, a.heads_inv) * a.kv_heads;
        const int pg = q8::kv_divide(slot[u], a.page, a.page_inv), off = slot[u] - pg * a.page;
        const long long row = (static_cast<long long>(pg) * a.kv_heads + h) * a.page + off;
        uint8_t *dst = is_v ? a.vc : a.kc;
        if (!kInt8) {
            if (slot[u] < 0) continue;
            const __half2 lo = __floats2half2_rn(x[u].x, x[u].y), hi = __floats2half2_rn(x[u].z, x[u].w);
            reinterpret_cast<uint2 *>(dst + row * D * 2)[sub] =
                make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
        } else {
            float4 w = slot[u] < 0 ? make_float4(0.0f, 0.0f, 0.0f, 0.0f) : x[u];
            float m = q8::max_nan(q8::max_nan(fabsf(w.x), fabsf(w.y)), q8::max_nan(fabsf(w.z), fabsf(w.w)));
#pragma unroll
            for (int o = 1; o < L; o <<= 1) m = q8::max_nan(m, __shfl_xor_sync(Q8_FULL_MASK, m, o));
            const float d = q8::q8_block_d(m), di = q8::q8_block_di(d);
            if (slot[u] < 0) continue;
            reinterpret_cast<uint32_t *>(dst + row * D)[sub] =
                q8::pack4(q8::q8_code(w.x, di), q8::q8_code(w.y, di), q8::q8_code(w.z, di), q8::q8_code(w.w, di));
            if (sub == 0) (is_v ? a.vs : a.ks)[row] = d;
        }
    }
}

// ---------------------------------------------------------------------------
// q8_kv_accept.  A CTA takes one sequence of one layer.  Rows move within the
// sequence's own fresh tokens, forward only: token j receives token path[j] >=
// j.  A thread owns 16 bytes of a row (or one scale) and walks the path in
// order, eight reads before their eight writes: the write of j can only hit
// the source of a later entry if path is not increasing, which is checked.
// Bound by latency: count, path, table and rows follow one another, so nine
// CTAs an SM (56 registers) hide one another's; with 67 registers, seven, it
// takes 10.2 us.  Measured: paths of up to 32 nodes of 128 sequences in 28 layers
// of 4 heads of 128 int8 values (28.4 MB) 8.8 us on the device, 3.2 TB/s.
// ---------------------------------------------------------------------------
constexpr int kAcceptThreads = 128;

struct AcceptArgs {
    uint8_t *k, *v;
    float *ks, *vs;
    const int32_t *table, *cached, *fresh, *paths, *counts;
    int32_t *lens;
    long long max_pages, layer_rows;
    int width, kv_heads, page, n_pages, words;  // words: 16-byte words of a row
};

__global__ void __launch_bounds__(kAcceptThreads, 9) kv_accept_kernel(const __grid_constant__ AcceptArgs a)
{
    __shared__ int s_src[Q8_TREE_MAX_NODES], s_dst[Q8_TREE_MAX_NODES];  // page * kv_heads * page_size + offset
    q8::griddep_launch_dependents();
    q8::griddep_wait();
    const int b = blockIdx.x, tid = threadIdx.x;
    const long long layer = blockIdx.y;
    const int n = a.counts[b], c0 = a.cached[b], f = a.fresh[b];
    bool bad = n < 0 || n > a.width || n > f || c0 < 0 || static_cast<long long>(c0) + f > 0x7fffffffll ||
               (static_cast<long long>(c0) + f + a.page - 1) / a.page > a.max_pages;
    bool stay = false;
    if (!bad && tid < n) {
        const int32_t *path = a.paths + static_cast<long long>(b) * a.width;
        const int p = path[tid];
        if (p < tid || p >= f || (tid > 0 && path[tid - 1] >= p)) {
            bad = true;
        } else {
            auto place = [&](int pos) {
                const int i = pos / a.page;
                const int pg = a.table[static_cast<long long>(b) * a.max_pages + i];
                if (pg < 0 || pg >= a.n_pages) {
                    bad = true;
                    return 0;
                }
                return pg * a.kv_heads * a.page + (pos - i * a.page);  // < 2^31: rows of a layer
            };
            stay = p == tid;
            s_src[tid] = place(c0 + p);
            s_dst[tid] = place(c0 + tid);
        }
    }
    // path is increasing, so the tokens that lie where they belong come first: those stay
    const int first = __syncthreads_count(stay);
    bad = __syncthreads_or(bad);
    if (layer == 0 && tid == 0) {
        a.lens[b] = c0 + (bad ? 0 : n);
        if (bad) atomicOr(&g_kv_err, q8::kErrData);
    }
    if (bad) return;

    auto walk = [&](auto *base, long long stride, int head_off) {
        for (int j0 = first; j0 < n; j0 += 8) {
            std::remove_reference_t<decltype(*base)> x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j0 + j < n) x[j] = base[(static_cast<long long>(s_src[j0 + j]) + head_off) * stride];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j0 + j < n) base[(static_cast<long long>(s_dst[j0 + j]) + head_off) * stride] = x[j];
        }
    };
    const int per = a.kv_heads * a.words;
    for (int i = tid; i < 2 * per; i += kAcceptThreads) {
        const bool is_v = i >= per;
        const int e = is_v ? i - per : i, h = e / a.words, w = e - h * a.words;
        uint4 *base = reinterpret_cast<uint4 *>((is_v ? a.v : a.k) + layer * a.layer_rows * a.words * 16) + w;
        walk(base, a.words, h * a.page);
    }
    if (a.ks)
        for (int i = tid; i < 2 * a.kv_heads; i += kAcceptThreads) {
            const bool is_v = i >= a.kv_heads;
            const int h = is_v ? i - a.kv_heads : i;
            walk((is_v ? a.vs : a.ks) + layer * a.layer_rows, 1, h * a.page);
        }
}

} // namespace

namespace q8 {

unsigned int *kv_error_word()
{
    void *p = nullptr;
    return cudaGetSymbolAddress(&p, g_kv_err) == cudaSuccess ? static_cast<unsigned int *>(p) : nullptr;
}

} // namespace q8

extern "C" int q8_kv_plan(const int32_t *cached, const int32_t *fresh, int64_t batch, const int32_t *held,
                          const int32_t *free_pages, int64_t n_free, int32_t *table, int64_t max_pages,
                          int64_t page_size, int64_t n_pages, const int32_t *parents, int64_t tokens, int32_t *starts,
                          int32_t *slots, int32_t *positions, int64_t *masks, int32_t *needed, int32_t *held_out,
                          void *stream)
{
    if (!cached || !fresh || !table || !starts || !slots || !positions || !needed) return Q8_ERR_ARG;
    if ((parents == nullptr) != (masks == nullptr) || n_free < 0 || (n_free > 0 && !free_pages)) return Q8_ERR_ARG;
    if (batch < 1 || batch > Q8_KV_MAX_BATCH || tokens < 1 || tokens >= (int64_t(1) << 31) || max_pages < 1 ||
        max_pages >= (int64_t(1) << 31) || !q8::kv_pages_ok(page_size, n_pages))
        return Q8_ERR_ARG;
    const void *all[] = {cached, fresh, held, free_pages, table, parents, starts, slots, positions, masks, needed,
                         held_out};
    for (const void *p : all)
        if (!q8::aligned16(p)) return Q8_ERR_ALIGN;
    const q8::Span spans[] = {{table, batch * max_pages * 4}, {starts, (batch + 1) * 4}, {slots, tokens * 4},
                              {positions, tokens * 4}, {masks, tokens * 8}, {needed, 4}, {held_out, batch * 4},
                              {cached, batch * 4}, {fresh, batch * 4}, {held, batch * 4}, {free_pages, n_free * 4},
                              {parents, tokens * 4}};
    if (q8::outputs_overlap(spans, 7, 12)) return Q8_ERR_ARG;
    if (!q8::device_is_sm103()) return Q8_ERR_DEVICE;
    PlanArgs a = {cached, fresh, held, free_pages, parents, table, starts, slots, positions, needed, held_out,
                  reinterpret_cast<long long *>(masks), n_free, max_pages, tokens, static_cast<int>(batch),
                  static_cast<int>(page_size), static_cast<int>(n_pages)};
    const int segs = static_cast<int>((batch + kPlanSeqs - 1) / kPlanSeqs);
    // enough CTAs that each writes a few rounds of tokens at most, up to one per SM
    const int64_t rounds = (tokens + int64_t(segs) * kPlanThreads - 1) / (int64_t(segs) * kPlanThreads);
    const int most = q8::device_sm_count() / segs;
    const int gy = static_cast<int>(rounds < 1 ? 1 : rounds > most ? (most < 1 ? 1 : most) : rounds);
    return q8::launch_pdl(kv_plan_kernel, dim3(segs, gy), dim3(kPlanThreads), 0, static_cast<cudaStream_t>(stream), a);
}

extern "C" int q8_kv_append(const q8_kv_cache *cache, int64_t layer, const float *k, const float *v,
                            const int32_t *slots, int64_t tokens, void *stream)
{
    if (!cache || !k || !v || !slots || tokens < 1 || tokens >= (int64_t(1) << 31)) return Q8_ERR_ARG;
    const int st = q8::kv_cache_status(cache);
    if (st == Q8_ERR_ARG) return st;
    if (layer < 0 || layer >= cache->layers) return Q8_ERR_ARG;
    if (st != Q8_OK) return st;
    if (!q8::aligned16(k) || !q8::aligned16(v) || !q8::aligned16(slots)) return Q8_ERR_ALIGN;
    const int D = cache->head_dim;
    const int64_t rows = tokens * cache->kv_heads, per = int64_t(kAppendThreads / (D / 4)) * kAppendRows;
    if (rows >= int64_t(1) << 29) return Q8_ERR_ARG;  // rows are counted in 32 bits
    const int64_t grid = (2 * rows + per - 1) / per;
    if (!q8::device_is_sm103()) return Q8_ERR_DEVICE;
    const int64_t lr = q8::kv_layer_rows(*cache), eb = q8::kv_element_bytes(*cache);
    const bool i8 = cache->dtype == Q8_KV_INT8;
    AppendArgs a = {k, v, slots, static_cast<uint8_t *>(cache->k) + layer * lr * D * eb,
                    static_cast<uint8_t *>(cache->v) + layer * lr * D * eb, i8 ? cache->k_scale + layer * lr : nullptr,
                    i8 ? cache->v_scale + layer * lr : nullptr, static_cast<int>(rows), cache->kv_heads, cache->page_size,
                    static_cast<int>(cache->n_pages * cache->page_size), q8::kv_inverse(cache->kv_heads),
                    q8::kv_inverse(cache->page_size)};
    auto fn = D == 128 ? (i8 ? kv_append_kernel<128, true> : kv_append_kernel<128, false>)
                       : (i8 ? kv_append_kernel<64, true> : kv_append_kernel<64, false>);
    return q8::launch_pdl(fn, dim3(static_cast<unsigned>(grid)), dim3(kAppendThreads), 0,
                          static_cast<cudaStream_t>(stream), a);
}

extern "C" int q8_kv_accept(const q8_kv_cache *cache, const int32_t *table, int64_t max_pages, const int32_t *cached,
                            const int32_t *fresh, int64_t batch, const int32_t *paths, const int32_t *counts,
                            int64_t width, int32_t *lens, void *stream)
{
    if (!cache || !table || !cached || !fresh || !paths || !counts || !lens) return Q8_ERR_ARG;
    const int st = q8::kv_cache_status(cache);
    if (st == Q8_ERR_ARG) return st;
    if (batch < 1 || batch > Q8_KV_MAX_BATCH || width < 1 || width > Q8_TREE_MAX_NODES || max_pages < 1 ||
        max_pages >= (int64_t(1) << 31) || cache->layers > 65535)
        return Q8_ERR_ARG;
    if (st != Q8_OK) return st;
    const void *all[] = {table, cached, fresh, paths, counts, lens};
    for (const void *p : all)
        if (!q8::aligned16(p)) return Q8_ERR_ALIGN;
    const q8::Span spans[] = {{lens, batch * 4}, {table, batch * max_pages * 4}, {cached, batch * 4}, {fresh, batch * 4},
                              {paths, batch * width * 4}, {counts, batch * 4}};
    if (q8::outputs_overlap(spans, 1, 6)) return Q8_ERR_ARG;
    if (!q8::device_is_sm103()) return Q8_ERR_DEVICE;
    AcceptArgs a = {static_cast<uint8_t *>(cache->k), static_cast<uint8_t *>(cache->v), cache->k_scale, cache->v_scale,
                    table, cached, fresh, paths, counts, lens, max_pages, q8::kv_layer_rows(*cache),
                    static_cast<int>(width), cache->kv_heads, cache->page_size, static_cast<int>(cache->n_pages),
                    cache->head_dim * q8::kv_element_bytes(*cache) / 16};
    return q8::launch_pdl(kv_accept_kernel, dim3(static_cast<unsigned>(batch), static_cast<unsigned>(cache->layers)),
                          dim3(kAcceptThreads), 0, static_cast<cudaStream_t>(stream), a);
}
