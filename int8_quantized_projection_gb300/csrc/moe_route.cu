// moe_route.cu -- routing of tokens to experts: the top_k experts of each
// token, their weights, and the (token, expert) pairs sorted by expert.
//
// Per token t with logits l and chosen experts c_0 .. c_{K-1} (largest logits
// first, of equal ones the lower expert):
//     weight_j = scale * exp(l[c_j] - l[c_0]) / sum,
// the sum over the chosen experts or over all of them.  Pair p = t * K + j goes
// to sorted row
//     place[p] = offsets[e] + |{pairs of expert e with a smaller p}|.
// A token's experts are distinct, so the second term counts tokens: within a
// chunk of tokens it is the population count of a bit set per expert, and the
// chunks before it are added up from a table of counts.  Nothing depends on the
// order in which threads arrive: the bits and counts are sets and sums of
// integers.
#include "kv_common.cuh"

namespace {

__device__ unsigned int g_route_err;

constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kMaxChunk = 1024;            // tokens of a CTA at most
constexpr int kOneLaunch = 64;             // tokens that one CTA routes by itself (two rounds of its warps; 128 take 13 us, in two launches 7)
constexpr int kBitBytes = 35 * 1024;       // shared memory of the bit sets
constexpr int kPlaceBytes = 4 * (3 * Q8_MAX_EXPERTS + kWarps);  // of the placing kernel's sums
static_assert(kThreads == Q8_MAX_EXPERTS && kBitBytes >= 4 * Q8_MAX_EXPERTS, "a thread and a word of bits per expert");
static_assert(kBitBytes + kPlaceBytes <= 48 * 1024, "shared memory of a launch that asks for no more");

struct RouteArgs {
    const float *logits;
    const int32_t *valid;
    int32_t *ids, *offsets, *rows, *places;
    float *weights;
    int32_t *counts;  // [chunks][experts]
    int tokens, experts, top_k, mode, chunk, chunks;
    float scale;
};

// A logit as an integer of the same order; 0 for one that is never chosen.
__device__ __forceinline__ uint32_t order_key(float l)
{
    const uint32_t b = __float_as_uint(l + 0.0f);  // -0 becomes +0: they are equal
    if ((b & 0x7fffffffu) > 0x7f800000u || b == 0xff800000u) return 0u;
    return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}

__device__ __forceinline__ float key_value(uint32_t k) { return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu)); }

// exp(l - m) for l <= m; 1 where both are the same infinity.
__device__ __forceinline__ float share_of(float l, float m) { return l == m ? 1.0f : expf(l - m); }

// One warp, one token: lane j < top_k returns the j-th expert (-1: none) and
// its weight.  EPL logits a lane: expert i * 32 + lane.
template <int EPL>
__device__ __forceinline__ void choose(const RouteArgs &a, int t, int lane, int &id, float &weight)
{
    uint32_t key[EPL];
    const float *l = a.logits + static_cast<int64_t>(t) * a.experts;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        const int e = i * 32 + lane;
        key[i] = e < a.experts ? order_key(__ldg(l + e)) : 0u;
    }
    uint32_t mine = 0u, first = 0u;
    float all = 0.0f;
    id = -1;
    for (int j = 0; j < a.top_k; ++j) {
        uint32_t best = 0u;
        int at = 0;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (key[i] > best) best = key[i], at = i;
        const uint32_t top = __reduce_max_sync(Q8_FULL_MASK, best);
        if (j == 0) {
            first = top;
            if (a.mode == Q8_ROUTE_ALL) {
                const float m = key_value(top);
#pragma unroll
                for (int i = 0; i < EPL; ++i)
                    if (key[i]) all += share_of(key_value(key[i]), m);
#pragma unroll
                for (int o = 16; o; o >>= 1) all += __shfl_xor_sync(Q8_FULL_MASK, all, o);
            }
        }
        if (top == 0u) break;  // no expert is left
        const int e = static_cast<int>(__reduce_min_sync(Q8_FULL_MASK, best == top ? at * 32u + lane : ~0u));
        if (lane == j) id = e, mine = top;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (i * 32 + lane == e) key[i] = 0u;
    }
    const float ex = mine ? share_of(key_value(mine), key_value(first)) : 0.0f;
    if (a.mode != Q8_ROUTE_ALL) {
        all = ex;
#pragma unroll
        for (int o = 16; o; o >>= 1) all += __shfl_xor_sync(Q8_FULL_MASK, all, o);
    }
    weight = mine ? ex / all * a.scale : 0.0f;
}

// Sums over the experts, a thread each: returns the inclusive one, and in `total` all of them.
__device__ __forceinline__ int scan_experts(int v, int *s_scan, int &total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(Q8_FULL_MASK, v, o);
        if (lane >= o) v += u;
    }
    if (lane == 31) s_scan[warp] = v;
    __syncthreads();
    if (warp == 0) {
        int w = s_scan[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(Q8_FULL_MASK, w, o);
            if (lane >= o) w += u;
        }
        s_scan[lane] = w;
    }
    __syncthreads();
    total = s_scan[kWarps - 1];
    return v + (warp ? s_scan[warp - 1] : 0);
}

// The second half: offsets, and each pair of this CTA's `tokens` from t0 on to its place.  `all`: this thread's expert's pairs,
// `before`: those of them in earlier chunks.  bits: [experts][words], bit t - t0 of an expert set where token t chose it.
__device__ __forceinline__ void place_pairs(const RouteArgs &a, const uint32_t *bits, int words, int t0, int tokens,
                                            int all, int before, int *s_base, int *s_scan)
{
    const int e = threadIdx.x;
    int total;
    const int sum = scan_experts(all, s_scan, total);
    if (e < a.experts) {
        s_base[e] = sum - all + before;
        if (blockIdx.x == 0) {
            a.offsets[e] = sum - all;
            if (e == a.experts - 1) a.offsets[a.experts] = sum;
        }
    }
    __syncthreads();
    const int pairs = tokens * a.top_k;
    const int64_t p0 = static_cast<int64_t>(t0) * a.top_k;
    for (int i = threadIdx.x; i < pairs; i += kThreads) {
        const int id = a.ids[p0 + i], t = i / a.top_k;
        int place = -1;
        if (id >= 0) {
            const uint32_t *set = bits + id * words;
            place = s_base[id] + __popc(set[t >> 5] & ((1u << (t & 31)) - 1u));
            for (int w = 0; w < t >> 5; ++w) place += __popc(set[w]);
            a.rows[place] = static_cast<int32_t>(p0 + i);
        }
        a.places[p0 + i] = place;
    }
    // rows behind the last pair: -1
    const int64_t stride = static_cast<int64_t>(gridDim.x) * kThreads, end = static_cast<int64_t>(a.tokens) * a.top_k;
    for (int64_t r = total + blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x; r < end; r += stride) a.rows[r] = -1;
}

// The experts of a chunk's tokens and how many chose each.  With kOne the chunk is the whole call, and its pairs are
// placed as well: one launch.
template <int EPL, bool kOne>
__global__ void __launch_bounds__(kThreads) route_choose_kernel(const __grid_constant__ RouteArgs a)
{
    extern __shared__ uint32_t bits[];
    __shared__ int s_base[kOne ? Q8_MAX_EXPERTS : 1], s_scan[kWarps];
    q8::griddep_launch_dependents();
    q8::griddep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int words = (a.chunk + 31) >> 5;
    const int t0 = blockIdx.x * a.chunk, tokens = min(a.chunk, a.tokens - t0);  // t0 + chunk may pass 31 bits
    int real = a.tokens;
    if (a.valid) {
        real = *a.valid;
        if ((real < 0 || real > a.tokens) && threadIdx.x == 0) atomicOr(&g_route_err, q8::kErrData);
    }
    for (int i = threadIdx.x; i < a.experts * words; i += kThreads) bits[i] = 0u;
    __syncthreads();
    for (int i = warp; i < tokens; i += kWarps) {
        const int t = t0 + i;
        int id = -1;
        float weight = 0.0f;
        if (t < real) choose<EPL>(a, t, lane, id, weight);
        if (lane < a.top_k) {
            const int64_t p = static_cast<int64_t>(t) * a.top_k + lane;
            a.ids[p] = id;
            a.weights[p] = weight;
            if (id >= 0) atomicOr(&bits[id * words + (i >> 5)], 1u << (i & 31));
        }
    }
    __syncthreads();
    const int e = threadIdx.x;
    int n = 0;
    if (e < a.experts)
        for (int w = 0; w < words; ++w) n += __popc(bits[e * words + w]);
    if (kOne)
        place_pairs(a, bits, words, t0, tokens, n, 0, s_base, s_scan);
    else if (e < a.experts)
        a.counts[static_cast<int64_t>(blockIdx.x) * a.experts + e] = n;
}

// The places, from the counts of all chunks: every CTA adds them up for itself (chunks x experts integers from L2), all threads
// taking part (a thread per expert alone: 13 us for 3325 tokens and 128 experts, so 8).
__global__ void __launch_bounds__(kThreads) route_place_kernel(const __grid_constant__ RouteArgs a)
{
    extern __shared__ uint32_t bits[];
    __shared__ int s_base[Q8_MAX_EXPERTS], s_all[Q8_MAX_EXPERTS], s_before[Q8_MAX_EXPERTS], s_scan[kWarps];
    static_assert(sizeof s_base + sizeof s_all + sizeof s_before + sizeof s_scan == kPlaceBytes, "counted for kBitBytes");
    q8::griddep_launch_dependents();
    q8::griddep_wait();
    const int e = threadIdx.x, words = (a.chunk + 31) >> 5;
    const int t0 = blockIdx.x * a.chunk, tokens = min(a.chunk, a.tokens - t0);
    for (int i = threadIdx.x; i < a.experts * words; i += kThreads) bits[i] = 0u;
    s_all[e] = s_before[e] = 0;
    __syncthreads();
    const int parts = kThreads / a.experts, part = e / a.experts, mine = e - part * a.experts;
    if (part < parts) {
        int all = 0, before = 0;
#pragma unroll 8
        for (int c = part; c < a.chunks; c += parts) {
            const int n = a.counts[static_cast<int64_t>(c) * a.experts + mine];
            all += n;
            before += c < static_cast<int>(blockIdx.x) ? n : 0;
        }
        atomicAdd(&s_all[mine], all);
        atomicAdd(&s_before[mine], before);
    }
    const int64_t p0 = static_cast<int64_t>(t0) * a.top_k;
    for (int i = threadIdx.x; i < tokens * a.top_k; i += kThreads) {
        const int id = a.ids[p0 + i], t = i / a.top_k;
        if (id >= 0) atomicOr(&bits[id * words + (t >> 5)], 1u << (t & 31));
    }
    __syncthreads();
    place_pairs(a, bits, words, t0, tokens, s_all[e], s_before[e], s_base, s_scan);
}

// Tokens of a CTA: all of them up to kOneLaunch, else an SM's share in whole words of bits, which have to fit kBitBytes.
int chunk_of(int64_t tokens, int64_t experts)
{
    const int64_t most = kBitBytes / (4 * experts) * 32;
    if (tokens <= kOneLaunch && tokens <= most) return static_cast<int>(tokens);
    const int64_t c = ((tokens + 151) / 152 + 31) / 32 * 32, cap = most < kMaxChunk ? most : kMaxChunk;
    return static_cast<int>(c > cap ? cap : c);
}

bool sizes_ok(int64_t tokens, int64_t experts, int64_t top_k)
{
    return tokens >= 1 && experts >= 1 && experts <= Q8_MAX_EXPERTS && top_k >= 1 && top_k <= Q8_MAX_TOP_K &&
           top_k <= experts && tokens <= ((int64_t(1) << 31) - 1) / top_k;
}

size_t bit_bytes(const RouteArgs &a) { return static_cast<size_t>(a.experts) * ((a.chunk + 31) / 32) * 4; }

template <int EPL>
int launch_choose(const RouteArgs &a, cudaStream_t s)
{
    const dim3 grid(static_cast<unsigned>(a.chunks)), block(kThreads);
    return a.chunks == 1 ? q8::launch_pdl(route_choose_kernel<EPL, true>, grid, block, bit_bytes(a), s, a)
                         : q8::launch_pdl(route_choose_kernel<EPL, false>, grid, block, bit_bytes(a), s, a);
}

} // namespace

extern "C" size_t q8_moe_route_workspace_bytes(int64_t tokens, int64_t experts, int64_t top_k)
{
    if (!sizes_ok(tokens, experts, top_k)) return 0;
    const int64_t chunk = chunk_of(tokens, experts), chunks = (tokens + chunk - 1) / chunk;
    return chunks == 1 ? 0 : static_cast<size_t>(chunks * experts) * 4;
}

extern "C" int q8_moe_route(const float *logits, int64_t tokens, int64_t experts, int64_t top_k, int mode, float scale,
                            const int32_t *valid, int32_t *ids, float *weights, int32_t *offsets, int32_t *rows,
                            int32_t *places, void *workspace, size_t workspace_bytes, void *stream)
{
    if (!logits || !ids || !weights || !offsets || !rows || !places || !sizes_ok(tokens, experts, top_k)) return Q8_ERR_ARG;
    if ((mode != Q8_ROUTE_CHOSEN && mode != Q8_ROUTE_ALL) || !(scale - scale == 0.0f)) return Q8_ERR_ARG;
    const size_t need = q8_moe_route_workspace_bytes(tokens, experts, top_k);
    if (need && (!workspace || workspace_bytes < need)) return Q8_ERR_ARG;
    const int64_t pairs = tokens * top_k;
    const q8::Span spans[] = {{ids, 4 * pairs}, {weights, 4 * pairs}, {offsets, 4 * (experts + 1)}, {rows, 4 * pairs},
                              {places, 4 * pairs}, {workspace, static_cast<int64_t>(need)}, {logits, 4 * tokens * experts},
                              {valid, 4}};
    if (q8::outputs_overlap(spans, 6, 8)) return Q8_ERR_ARG;
    for (const q8::Span &p : spans)
        if (!q8::aligned16(p.p)) return Q8_ERR_ALIGN;
    if (!q8::device_is_sm103()) return Q8_ERR_DEVICE;
    RouteArgs a = {};
    a.logits = logits, a.valid = valid, a.ids = ids, a.offsets = offsets, a.rows = rows, a.places = places;
    a.weights = weights, a.counts = static_cast<int32_t *>(workspace);
    a.tokens = static_cast<int>(tokens), a.experts = static_cast<int>(experts), a.top_k = static_cast<int>(top_k);
    a.mode = mode, a.scale = scale, a.chunk = chunk_of(tokens, experts), a.chunks = static_cast<int>((tokens + a.chunk - 1) / a.chunk);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int st = experts <= 64    ? launch_choose<2>(a, s)
                   : experts <= 128 ? launch_choose<4>(a, s)
                   : experts <= 256 ? launch_choose<8>(a, s)
                                    : launch_choose<32>(a, s);
    if (st != Q8_OK || a.chunks == 1) return st;
    return q8::launch_pdl(route_place_kernel, dim3(static_cast<unsigned>(a.chunks)), dim3(kThreads), bit_bytes(a), s, a);
}

namespace q8 {

unsigned int *route_error_word()
{
    void *p = nullptr;
    return cudaGetSymbolAddress(&p, g_route_err) == cudaSuccess ? static_cast<unsigned int *>(p) : nullptr;
}

} // namespace q8
