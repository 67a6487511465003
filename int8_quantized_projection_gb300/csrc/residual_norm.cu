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

// A CTA per row, J float4 a thread.
template <int J>
__global__ void __launch_bounds__(512) residual_rmsnorm_kernel(const __grid_constant__ NormArgs a)
{
    __shared__ float red[2][2][16];
    const int tid = threadIdx.x, P = blockDim.x, F = a.F, d = 4 * F;
    q8::griddep_launch_dependents();
    q8::griddep_wait();
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
        for (int j = 0; j < J; ++j) {
            const int f = tid + j * P;
            v[j] = a.b && f < F ? a.b[t * F + f] : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        for (int k = 0; k < a.top_k; ++k) {
            const int place = a.places[t * a.top_k + k];
            if (place < 0 || place >= a.expert_row_count) {
                if (place != -1 && tid == 0) atomicOr(&g_resnorm_err, q8::kErrData);
                continue;
            }
            const float weight = a.weights[t * a.top_k + k];
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const int f = tid + j * P;
                if (f < F) v[j] = fma4(weight, a.expert_rows[static_cast<int64_t>(place) * F + f], v[j]);
            }
        }
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
                    const float4 g = a.gate[t * a.gate_stride + f];
                    v[j] = make_float4(v[j].x * g.x, v[j].y * g.y, v[j].z * g.z, v[j].w * g.w);
                }
                v[j] = fma4(a.residual_scale, a.x[t * F + f], v[j]);
                if (a.h) a.h[t * F + f] = v[j];
            }
            ss = q8::rms_sumsq4(ss, v[j]);
        }
        if (!a.w) continue;  // h alone
        const float scale = q8::rms_scale(cta_sum(ss, red[it][1]), d, a.eps);
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int f = tid + j * P;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
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
    const int64_t cap = 152 * 8;
    const dim3 grid(static_cast<unsigned>(all < cap ? all : cap)), block(P);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    switch (J) {
    case 1: return q8::launch_pdl(residual_rmsnorm_kernel<1>, grid, block, 0, s, a);
    case 2: return q8::launch_pdl(residual_rmsnorm_kernel<2>, grid, block, 0, s, a);
    case 4: return q8::launch_pdl(residual_rmsnorm_kernel<4>, grid, block, 0, s, a);
    case 8: return q8::launch_pdl(residual_rmsnorm_kernel<8>, grid, block, 0, s, a);
    default: return q8::launch_pdl(residual_rmsnorm_kernel<16>, grid, block, 0, s, a);
    }
}

namespace q8 {

unsigned int *resnorm_error_word()
{
    void *p = nullptr;
    return cudaGetSymbolAddress(&p, g_resnorm_err) == cudaSuccess ? static_cast<unsigned int *>(p) : nullptr;
}

} // namespace q8
