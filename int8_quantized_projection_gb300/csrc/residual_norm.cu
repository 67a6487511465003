// residual_norm.cu -- what lies between two blocks of a layer stack, in one
// pass over the rows: the weighted sum of a token's expert rows, the norm
// behind the block, its gate, the scaled residual, and the norm before the next
// block with the q8_0 plane of its output.
//
//     b'   = b + sum_j weights[t][j] * expert_rows[places[t][j]]
//     p    = w_post ? (b' * rsqrt(mean(b'^2) + eps_post)) * w_post : b'
//     h    = residual_scale * x + gate * p
//     y    = (h * rsqrt(mean(h^2) + eps)) * w, and its plane.
#include "kv_common.cuh"

namespace {

__device__ unsigned int g_resnorm_err;

struct NormArgs {
    const float4 *x, *b, *expert_rows, *w_post, *gate, *w;
    const int32_t *places;
    const float *weights;
    float4 *h, *y;
    uint32_t *qs, *ds;
    int64_t rows, rows_pad, expert_row_count, gate_stride;  // gate_stride: float4 from a row's gate to the next's
    int F, top_k;                                          // F = d / 4
    float residual_scale, eps_post, eps;
};

__device__ __forceinline__ float4 fma4(float s, float4 a, float4 c)
{
    return make_float4(fmaf(s, a.x, c.x), fmaf(s, a.y, c.y), fmaf(s, a.z, c.z), fmaf(s, a.w, c.w));
}

// Sum over the CTA, the same in every thread; red: one float per warp, used once between two barriers of the caller's.
__device__ __forceinline__ float cta_sum(float v, float *red)
{
    v = q8::rms_warp_sum(v);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    float tot = 0.0f;
    for (int i = 0; i < static_cast<int>(blockDim.x >> 5); ++i) tot += red[i];
    return tot;
}

// Streaming 16-byte load that does not allocate in L1, which is left to the vectors that all rows share.
__device__ __forceinline__ float4 ld_stream(const float4 *p)
{
    float4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.f32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "l"(p));
    return v;
}

// Few rows, or very wide ones: a CTA per row and round, J float4 a thread, which stay in registers from the first load to the last store: each input is read
// once and each output written once, so the rows' bytes bound it.  What hides the latencies: x is asked for before the block's
// output, U expert rows at a time, the places and weights of the CTA's next row while this one is computed, and several CTAs an
// SM.  x may be h, so it is not read through the non-coherent path.
template <int J, int U>
__global__ void __launch_bounds__(512) residual_rmsnorm_kernel(const __grid_constant__ NormArgs a)
{
    __shared__ float red[2][2][16];
    __shared__ int s_place[2][Q8_MAX_TOP_K];
    __shared__ float s_weight[2][Q8_MAX_TOP_K];
    const int tid = threadIdx.x, P = blockDim.x, F = a.F, d = 4 * F;
    q8::griddep_launch_dependents();
    q8::griddep_wait();
    const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
    auto places = [&](int64_t t, int buf) {
        if (tid < a.top_k && t < a.rows) {
            const int place = a.places[t * a.top_k + tid];
            const bool ok = place >= 0 && place < a.expert_row_count;
            if (!ok && place != -1) atomicOr(&g_resnorm_err, q8::kErrData);
            s_place[buf][tid] = ok ? place : -1;
            s_weight[buf][tid] = a.weights[t * a.top_k + tid];
        }
    };
    if (a.top_k) {
        places(blockIdx.x, 0);
        __syncthreads();
    }
    int it = 0;
    for (int64_t t = blockIdx.x; t < (a.qs ? a.rows_pad : a.rows); t += gridDim.x, it ^= 1) {
        if (t >= a.rows) {
            for (int f = tid; f < F; f += P) {
                a.qs[t * F + f] = 0u;
                if ((f & 7) == 0) a.ds[(t * F + f) >> 3] = 0u;
            }
            continue;
        }
        float4 v[J], x[J];
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int f = tid + j * P;
            if (U > 1) x[j] = f < F ? a.x[t * F + f] : zero;
            v[j] = a.b && f < F ? ld_stream(a.b + t * F + f) : zero;
        }
        for (int k0 = 0; k0 < a.top_k; k0 += U) {
            float4 e[U][J];
#pragma unroll
            for (int k = 0; k < U; ++k) {
                const int place = k0 + k < a.top_k ? s_place[it][k0 + k] : -1;
                const float4 *row = a.expert_rows + static_cast<int64_t>(place) * F;
#pragma unroll
                for (int j = 0; j < J; ++j)
                    if (place >= 0 && tid + j * P < F) e[k][j] = ld_stream(row + tid + j * P);
            }
#pragma unroll
            for (int k = 0; k < U; ++k) {
                if (k0 + k >= a.top_k || s_place[it][k0 + k] < 0) continue;
                const float weight = s_weight[it][k0 + k];
#pragma unroll
                for (int j = 0; j < J; ++j)
                    if (tid + j * P < F) v[j] = fma4(weight, e[k][j], v[j]);
            }
        }
        if (a.top_k) places(t + gridDim.x, it ^ 1);  // a barrier of this row's, or the one below, comes before their use
        if (a.w_post) {
            float ss = 0.0f;
#pragma unroll
            for (int j = 0; j < J; ++j) ss = q8::rms_sumsq4(ss, v[j]);
            const float scale = q8::rms_scale(cta_sum(ss, red[it][0]), d, a.eps_post);
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const int f = tid + j * P;
                if (f < F) v[j] = q8::rms_apply4(v[j], scale, __ldg(a.w_post + f));
            }
        }
        float ss = 0.0f;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int f = tid + j * P;
            if (f < F) {
                if (a.gate) {
                    const float4 *gate = a.gate + t * a.gate_stride + f;
                    const float4 g = a.gate_stride ? ld_stream(gate) : __ldg(gate);
                    v[j] = make_float4(v[j].x * g.x, v[j].y * g.y, v[j].z * g.z, v[j].w * g.w);
                }
                v[j] = fma4(a.residual_scale, U > 1 ? x[j] : a.x[t * F + f], v[j]);
                if (a.h) a.h[t * F + f] = v[j];
            }
            ss = q8::rms_sumsq4(ss, v[j]);
        }
        if (!a.w) {  // h alone
            if (a.top_k && !a.w_post) __syncthreads();
            continue;
        }
        const float scale = q8::rms_scale(cta_sum(ss, red[it][1]), d, a.eps);
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int f = tid + j * P;
            float4 o = zero;
            if (f < F) {
                o = q8::rms_apply4(v[j], scale, __ldg(a.w + f));
                if (a.y) a.y[t * F + f] = o;
            }
            if (a.qs) {
                const q8::Q8Enc e = q8::q8_encode8(o);
                if (f < F) {
                    a.qs[t * F + f] = e.qword;
                    if ((f & 7) == 0) a.ds[(t * F + f) >> 3] = e.dsword;
                }
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Many rows.  A row's inputs (b, top_k expert rows, a gate of its own, x) come one after the other through a ring of shared-memory
// slots, a bulk copy of d floats each, which a warp of its own keeps full across rows: the rings of the CTAs that an SM holds are in
// flight whatever the other warps wait for, where loads into registers leave the memory idle while a row is reduced (3325 rows of
// 3584 joined from eight: 97 us with four CTAs an SM).  The vectors that all rows share stay in registers.
// ---------------------------------------------------------------------------
constexpr int kNarrow = 512, kStreamMaxD = 8192;  // at the widest six slots for joined rows, two for others
constexpr int kStreamSmem = 200 * 1024;
constexpr int kMaxSlots = 64;

__device__ __forceinline__ void rows_sync(int threads) { asm volatile("bar.sync 1, %0;" ::"r"(threads) : "memory"); }

// Sum over the P threads of a row, the same in each.
__device__ __forceinline__ float row_sum(float v, float *red, int P)
{
    v = q8::rms_warp_sum(v);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncwarp();  // the barrier wants whole warps
    rows_sync(P);
    float tot = 0.0f;
    for (int i = 0; i < P >> 5; ++i) tot += red[i];
    return tot;
}

template <int J>
__global__ void __launch_bounds__(544, J <= 2 ? 2 : 1) residual_rmsnorm_stream_kernel(const __grid_constant__ NormArgs a, int slots)
{
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ __align__(8) uint64_t full[kMaxSlots], empty[kMaxSlots];
    __shared__ float weight[kMaxSlots];  // of the slot's expert row
    __shared__ int there[kMaxSlots];     // 0: no such row
    __shared__ float red[2][2][16];
    __shared__ volatile int stop;        // a wait for a row ran out: no slot is filled again
    const int tid = threadIdx.x, P = blockDim.x - 32, F = a.F, d = 4 * F, lane = tid & 31;
    const bool own_gate = a.gate && a.gate_stride;
    const int vectors = (a.b ? 1 : 0) + a.top_k + (own_gate ? 1 : 0) + 1;
    const int64_t bytes = static_cast<int64_t>(d) * 4;
    if (tid == 0) {
        for (int i = 0; i < slots; ++i) q8::mbar_init(full + i, 1), q8::mbar_init(empty + i, P / 32);
        stop = 0;
        q8::fence_mbar_init();
    }
    __syncthreads();
    q8::griddep_launch_dependents();
    q8::griddep_wait();
    if (tid >= P) {
        // ---------------------------------------------------------------- the copies: lane j has vector j of a row
        const int j0 = a.b ? 1 : 0;
        int slot = 0;
        uint32_t phase = 0, issued = 0;
        bool ok = true;
        int place = -1, next_place = -1;
        float w = 0.0f, next_w = 0.0f;
        auto ask = [&](int64_t t) {  // an expert row's place, a row ahead
            if (t < a.rows && lane >= j0 && lane < j0 + a.top_k) {
                next_place = a.places[t * a.top_k + lane - j0];
                next_w = a.weights[t * a.top_k + lane - j0];
            }
        };
        ask(blockIdx.x);
        for (int64_t t = blockIdx.x; t < a.rows && ok; t += gridDim.x) {
            place = next_place, w = next_w;
            ask(t + gridDim.x);
            const float4 *src = nullptr;
            if (lane < j0)
                src = a.b + t * F;
            else if (lane < j0 + a.top_k) {
                if (place >= 0 && place < a.expert_row_count)
                    src = a.expert_rows + static_cast<int64_t>(place) * F;
                else if (place != -1)
                    atomicOr(&g_resnorm_err, q8::kErrData);
            } else if (lane < vectors - 1)
                src = a.gate + t * F;
            else
                src = a.x + t * F;
            for (int k = 0; k < vectors; ++k) {
                ok = __all_sync(Q8_FULL_MASK, q8::mbar_wait_bounded(empty + slot, phase ^ 1u));
                if (!ok && lane == 0) atomicOr(&g_resnorm_err, q8::kErrTimeout);
                ok = __all_sync(Q8_FULL_MASK, ok && !stop);  // who gave a slot back unread set it before
                if (!ok) break;
                if (lane == k) {
                    weight[slot] = w;
                    there[slot] = src != nullptr;
                    if (src) {
                        q8::mbar_arrive_expect_tx(full + slot, static_cast<uint32_t>(bytes));
                        q8::bulk_g2s(ring + slot * bytes, src, static_cast<uint32_t>(bytes), full + slot);
                    } else {
                        q8::mbar_arrive(full + slot);
                    }
                }
                __syncwarp();
                ++issued;
                if (++slot == slots) slot = 0, phase ^= 1u;
            }
        }
        // the last copies must have landed before the CTA exits
        for (uint32_t i = issued < static_cast<uint32_t>(slots) ? 0 : issued - slots; i < issued; ++i)
            q8::mbar_wait_bounded(full + i % slots, (i / slots) & 1u, Q8_DRAIN_LIMIT_NS);
        return;
    }
    // -------------------------------------------------------------------- the rows
    const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
    float4 wp[J], wn[J], gc[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const int f = tid + j * P;
        wp[j] = a.w_post && f < F ? __ldg(a.w_post + f) : zero;
        wn[j] = a.w && f < F ? __ldg(a.w + f) : zero;
        gc[j] = a.gate && !own_gate && f < F ? __ldg(a.gate + f) : make_float4(1.f, 1.f, 1.f, 1.f);
    }
    int slot = 0;
    uint32_t phase = 0;
    bool dead = false;  // a wait ran out: the rows are walked without waiting, so that all threads pass the same barriers
    auto take = [&]() {
        if (!dead && !q8::mbar_wait_bounded(full + slot, phase)) {
            dead = true;
            stop = 1;
            atomicOr(&g_resnorm_err, q8::kErrTimeout);
        }
        return reinterpret_cast<const float4 *>(ring + slot * bytes) + tid;
    };
    auto give = [&]() {
        __syncwarp();
        if (lane == 0) q8::mbar_arrive(empty + slot);
        if (++slot == slots) slot = 0, phase ^= 1u;
    };
    int it = 0;
    for (int64_t t = blockIdx.x; t < (a.qs ? a.rows_pad : a.rows); t += gridDim.x, it ^= 1) {
        if (t >= a.rows) {
            for (int f = tid; f < F; f += P) {
                a.qs[t * F + f] = 0u;
                if ((f & 7) == 0) a.ds[(t * F + f) >> 3] = 0u;
            }
            continue;
        }
        float4 v[J];
#pragma unroll
        for (int j = 0; j < J; ++j) v[j] = zero;
        if (a.b) {
            const float4 *p = take();
#pragma unroll
            for (int j = 0; j < J; ++j)
                if (tid + j * P < F) v[j] = p[j * P];
            give();
        }
        for (int k = 0; k < a.top_k; ++k) {
            const float4 *p = take();
            const float w = weight[slot];
            if (there[slot]) {
#pragma unroll
                for (int j = 0; j < J; ++j)
                    if (tid + j * P < F) v[j] = fma4(w, p[j * P], v[j]);
            }
            give();
        }
        if (a.w_post) {
            float ss = 0.0f;
#pragma unroll
            for (int j = 0; j < J; ++j) ss = q8::rms_sumsq4(ss, v[j]);
            const float scale = q8::rms_scale(row_sum(ss, red[it][0], P), d, a.eps_post);
#pragma unroll
            for (int j = 0; j < J; ++j) v[j] = q8::rms_apply4(v[j], scale, wp[j]);
        }
        if (own_gate) {
            const float4 *p = take();
#pragma unroll
            for (int j = 0; j < J; ++j)
                if (tid + j * P < F) {
                    const float4 g = p[j * P];
                    v[j] = make_float4(v[j].x * g.x, v[j].y * g.y, v[j].z * g.z, v[j].w * g.w);
                }
            give();
        } else if (a.gate) {
#pragma unroll
            for (int j = 0; j < J; ++j)
                v[j] = make_float4(v[j].x * gc[j].x, v[j].y * gc[j].y, v[j].z * gc[j].z, v[j].w * gc[j].w);
        }
        float ss = 0.0f;
        {
            const float4 *p = take();
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const int f = tid + j * P;
                if (f < F) {
                    v[j] = fma4(a.residual_scale, p[j * P], v[j]);
                    if (a.h) a.h[t * F + f] = v[j];
                }
                ss = q8::rms_sumsq4(ss, v[j]);
            }
            give();
        }
        if (!a.w) continue;  // h alone
        const float scale = q8::rms_scale(row_sum(ss, red[it][1], P), d, a.eps);
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int f = tid + j * P;
            const float4 o = q8::rms_apply4(v[j], scale, wn[j]);  // zeros behind the row
            if (a.y && f < F) a.y[t * F + f] = o;
            if (a.qs) {
                const q8::Q8Enc e = q8::q8_encode8(o);
                if (f < F) {
                    a.qs[t * F + f] = e.qword;
                    if ((f & 7) == 0) a.ds[(t * F + f) >> 3] = e.dsword;
                }
            }
        }
    }
}

template <int J>
int launch_stream(const NormArgs &a, int64_t rows, int P, int slot, cudaStream_t s)
{
    // several CTAs share an SM, so that one works while another is at its barriers: fewer where a row has many vectors and a deep
    // ring tells (3325 rows of 3584: eight joined 88 us with rings for two CTAs, 92 for four; none 34.8 and 33.8).  How many an SM
    // holds goes by their registers (52, 56 and 96 a thread) too: two of 3584, one above d = 4608, whatever `threads` would
    // let it have, so that for top_k < 2 half of the shared memory or more stays unused there and at d = 7168 a ring has one slot
    const int threads = a.top_k >= 2 ? 1024 : 2048;
    const int bytes = 16 * a.F, want = threads / (P + 32) < 8 ? threads / (P + 32) : 8;
    const int ctas = want < 1 ? 1 : want, fit = kStreamSmem / ctas / bytes, slots = fit < kMaxSlots ? fit : kMaxSlots;
    if (!q8::set_max_dynamic_smem(reinterpret_cast<const void *>(residual_rmsnorm_stream_kernel<J>), kStreamSmem, slot))
        return Q8_ERR_LAUNCH;
    const int64_t cap = static_cast<int64_t>(q8::device_sm_count()) * ctas;
    return q8::launch_pdl(residual_rmsnorm_stream_kernel<J>, dim3(static_cast<unsigned>(rows < cap ? rows : cap)), dim3(P + 32),
                          static_cast<size_t>(slots) * bytes, s, a, slots);
}

// The grid is what fits the GPU at once, each CTA walking its rows.
template <int J, int U>
int launch(const NormArgs &a, int64_t rows, int P, cudaStream_t s)
{
    int per_sm = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, residual_rmsnorm_kernel<J, U>, P, 0) != cudaSuccess) return Q8_ERR_LAUNCH;
    const int64_t cap = static_cast<int64_t>(q8::device_sm_count()) * per_sm;
    return q8::launch_pdl(residual_rmsnorm_kernel<J, U>, dim3(static_cast<unsigned>(rows < cap ? rows : cap)), dim3(P), 0, s, a);
}

bool eps_ok(float eps) { return eps >= 0.0f && eps <= 3.4e38f; }

} // namespace

extern "C" int rmsnorm_residual_quant(const float *x, float residual_scale, const float *b, const float *expert_rows,
                                      int64_t expert_row_count, const int32_t *places, const float *weights,
                                      int64_t top_k, const float *w_post, float eps_post, const float *gate,
                                      int64_t gate_rows, const float *w, float eps, float *h, float *y, int64_t rows,
                                      int64_t d, int8_t *qs, uint32_t *ds, int64_t rows_pad, void *stream)
{
    if (rows < 0 || d <= 0 || d % 32 != 0 || d > 32768 || (!qs != !ds)) return Q8_ERR_ARG;
    if (qs && (rows_pad < rows || rows_pad < 1)) return Q8_ERR_ARG;
    const int64_t limit = (int64_t(1) << 61) / d;
    if (rows > limit || (qs && rows_pad > limit) || expert_row_count > limit) return Q8_ERR_ARG;
    if (rows > 0 && ((y || qs) != (w != nullptr) || !(h || y || qs))) return Q8_ERR_ARG;
    if (top_k < 0 || top_k > Q8_MAX_TOP_K || (top_k > 0) != (expert_rows != nullptr) || (top_k > 0) != (places != nullptr) ||
        (top_k > 0) != (weights != nullptr) || (top_k > 0 && (expert_row_count < 1 || expert_row_count >= int64_t(1) << 31)))
        return Q8_ERR_ARG;
    if (rows > 0 && (!x || (!b && top_k == 0))) return Q8_ERR_ARG;
    if (gate && gate_rows != 1 && gate_rows != rows) return Q8_ERR_ARG;
    if (!(residual_scale - residual_scale == 0.0f) || (w_post && !eps_ok(eps_post)) || (w && !eps_ok(eps))) return Q8_ERR_ARG;
    const int64_t row = 4 * d;
    const q8::Span spans[] = {{h, rows * row}, {y, rows * row}, {qs, rows_pad * d}, {ds, rows_pad * (d / 8)},
                              {h == x ? nullptr : x, rows * row}, {b, rows * row}, {expert_rows, expert_row_count * row},
                              {places, rows * top_k * 4}, {weights, rows * top_k * 4}, {w_post, row},
                              {gate, gate_rows * row}, {w, row}};
    if (q8::outputs_overlap(spans, 4, 12)) return Q8_ERR_ARG;
    if (!q8::aligned16(x)) return Q8_ERR_ALIGN;
    for (const q8::Span &p : spans)
        if (!q8::aligned16(p.p)) return Q8_ERR_ALIGN;
    if (!q8::device_is_sm103()) return Q8_ERR_DEVICE;
    const int64_t all = qs ? rows_pad : rows;
    if (all == 0) return Q8_OK;
    NormArgs a = {};
    auto f4 = [](const float *p) { return reinterpret_cast<const float4 *>(p); };
    a.x = f4(x), a.b = f4(b), a.expert_rows = f4(expert_rows), a.w_post = f4(w_post), a.gate = f4(gate), a.w = f4(w);
    a.places = places, a.weights = weights;
    a.h = reinterpret_cast<float4 *>(h), a.y = reinterpret_cast<float4 *>(y);
    a.qs = reinterpret_cast<uint32_t *>(qs), a.ds = ds;
    a.rows = rows, a.rows_pad = rows_pad, a.expert_row_count = expert_row_count;
    a.F = static_cast<int>(d / 4), a.gate_stride = gate_rows == 1 ? 0 : a.F, a.top_k = static_cast<int>(top_k);
    a.residual_scale = residual_scale, a.eps_post = eps_post, a.eps = eps;
    int J, P;
    q8::rms_row_mapping(a.F, q8::kRmsMaxThreadsOneRow, J, P);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    // narrow rows are done before a ring pays: 3325 of 512 take 6.2 us a CTA per row and 8.2 through the ring; 3000 of 8192 with
    // their own registers 46, through the ring 35
    if (all > q8::device_sm_count() && d > kNarrow && d <= kStreamMaxD) {
        if (J == 1) return launch_stream<1>(a, all, P, 56, s);
        if (J == 2) return launch_stream<2>(a, all, P, 57, s);
        return launch_stream<4>(a, all, P, 58, s);
    }
    switch (J) {
    case 1: return all > q8::device_sm_count() ? launch<1, 1>(a, all, P, s) : launch<1, 4>(a, all, P, s);
    case 2: return launch<2, 4>(a, all, P, s);
    case 4: return launch<4, 2>(a, all, P, s);
    case 8: return launch<8, 1>(a, all, P, s);
    default: return launch<16, 1>(a, all, P, s);
    }
}

namespace q8 {

unsigned int *resnorm_error_word()
{
    void *p = nullptr;
    return cudaGetSymbolAddress(&p, g_resnorm_err) == cudaSuccess ? static_cast<unsigned int *>(p) : nullptr;
}

} // namespace q8
