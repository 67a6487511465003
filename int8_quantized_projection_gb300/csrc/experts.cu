// experts.cu -- products of sorted rows with their experts' Q8_0 matrices: the
// entry points, and SwiGLU of a gate and an up product into a q8_0 plane.
#include "experts_common.cuh"

namespace {

__device__ unsigned int g_experts_err;

// One warp, one weight row, the expert's rows one after another: lane l takes the blocks l, l + 32, ...
__global__ void __launch_bounds__(256) experts_plain_kernel(const __grid_constant__ q8::ExpertsArgs a)
{
    q8::griddep_launch_dependents();
    q8::griddep_wait();
    const int lane = threadIdx.x & 31, i = blockIdx.x * 8 + (threadIdx.x >> 5), e = blockIdx.y;
    const q8::ExpertRows x = q8::expert_rows_of(a, e);
    if (x.bad && threadIdx.x == 0) atomicOr(&g_experts_err, q8::kErrData);
    const int all = a.w2 ? 2 * a.n : a.n;
    if (i >= all) return;
    const uint8_t *w = i < a.n ? a.w + (static_cast<int64_t>(e) * a.n + i) * a.nb * 34
                               : a.w2 + (static_cast<int64_t>(e) * a.n + i - a.n) * a.nb * 34;
    for (int r = x.first; r < x.first + x.count; ++r) {
        const int64_t src = q8::source_row(a, r);
        if (src < 0) {
            if (lane == 0) atomicOr(&g_experts_err, q8::kErrData);
            continue;
        }
        float acc = 0.0f;
        for (int b = lane; b < a.nb; b += 32) {
            const uint16_t *p = reinterpret_cast<const uint16_t *>(w + static_cast<int64_t>(b) * 34);
            const uint32_t *q = reinterpret_cast<const uint32_t *>(a.qs + (src * a.nb + b) * 32);
            int sum = 0;
#pragma unroll
            for (int u = 0; u < 8; ++u) sum = q8::dp4a(p[1 + 2 * u] | (static_cast<uint32_t>(p[2 + 2 * u]) << 16), q[u], sum);
            const float dw = __half2float(__ushort_as_half(p[0]));
            const float da = __half2float(__ushort_as_half(static_cast<unsigned short>(a.ds[src * a.nb + b] & 0xffffu)));
            acc = fmaf(dw * da, static_cast<float>(sum), acc);
        }
        acc = q8::rms_warp_sum(acc);
        if (lane == 0) a.out[r * a.ld + i] = acc;
    }
}

int experts_launch(const q8::ExpertsArgs &a, cudaStream_t s)
{
    const int all = a.w2 ? 2 * a.n : a.n;
    return q8::launch_pdl(experts_plain_kernel, dim3((all + 7) / 8, a.experts), dim3(256), 0, s, a);
}

// gu [pairs][2 nf] (gate, then up) -> the plane of silu(gate) * up, rows up to the last expert's end.
__global__ void __launch_bounds__(256)
experts_swiglu_kernel(const float4 *__restrict__ gu, int F, const int32_t *__restrict__ offsets, int experts, int pairs,
                      uint32_t *__restrict__ qs, uint32_t *__restrict__ ds)
{
    q8::griddep_launch_dependents();
    q8::griddep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t warp = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
    const int64_t warps = (static_cast<int64_t>(gridDim.x) * blockDim.x) >> 5;
    const int64_t total = static_cast<int64_t>(min(max(offsets[experts], 0), pairs)) * F;
    for (int64_t base = warp * 32; base < total; base += warps * 32) {
        const int64_t i = base + lane, r = i / F;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i < total) o = q8::silu_mul4(gu[r * F + i], gu[r * F + i + F]);
        const q8::Q8Enc e = q8::q8_encode8(o);
        if (i < total) {
            qs[i] = e.qword;
            if ((lane & 7) == 0) ds[i >> 3] = e.dsword;
        }
    }
}

bool sizes_ok(int64_t experts, int64_t n, int64_t k, int64_t plane_rows, int64_t top_k, int64_t pairs)
{
    const int64_t most = int64_t(1) << 31;
    return experts >= 1 && experts <= Q8_MAX_EXPERTS && n >= 1 && n <= Q8_EXPERTS_MAX_N && k >= 32 && k <= Q8_EXPERTS_MAX_K &&
           k % 32 == 0 && experts * n < most && plane_rows >= 1 && plane_rows < most && top_k >= 1 && top_k <= Q8_MAX_TOP_K &&
           pairs >= 1 && pairs < most - 256;
}

bool many_rows(int64_t experts, int64_t pairs) { return pairs >= 32 * experts; }

int64_t weight_bytes(int64_t experts, int64_t n, int64_t k) { return experts * n * (k / 32) * 34; }

q8::ExpertsArgs args_of(const void *w, const void *w2, int64_t experts, int64_t n, int64_t k, const int8_t *qs,
                        const uint32_t *ds, int64_t plane_rows, const int32_t *offsets, const int32_t *rows, int64_t top_k,
                        int64_t pairs, float *out)
{
    q8::ExpertsArgs a = {};
    a.w = static_cast<const uint8_t *>(w), a.w2 = static_cast<const uint8_t *>(w2);
    a.qs = qs, a.ds = ds, a.offsets = offsets, a.rows = rows, a.out = out;
    a.plane_rows = plane_rows, a.ld = w2 ? 2 * n : n;
    a.experts = static_cast<int>(experts), a.n = static_cast<int>(n), a.nb = static_cast<int>(k / 32);
    a.top_k = static_cast<int>(top_k), a.pairs = static_cast<int>(pairs);
    return a;
}

} // namespace

extern "C" size_t q8_0_experts_gemm_workspace_bytes(int64_t experts, int64_t n, int64_t k, int64_t plane_rows,
                                                    int64_t top_k, int64_t pairs)
{
    if (!sizes_ok(experts, n, k, plane_rows, top_k, pairs) || !many_rows(experts, pairs)) return 0;
    return q8::experts_tiles_workspace(k, pairs);
}

extern "C" int q8_0_experts_gemm(const void *w, int64_t experts, int64_t n, int64_t k, const int8_t *qs, const uint32_t *ds,
                                 int64_t plane_rows, const int32_t *offsets, const int32_t *rows, int64_t top_k,
                                 int64_t pairs, float *y, void *workspace, size_t workspace_bytes, void *stream)
{
    if (!w || !qs || !ds || !offsets || !y || !sizes_ok(experts, n, k, plane_rows, top_k, pairs)) return Q8_ERR_ARG;
    const size_t need = q8_0_experts_gemm_workspace_bytes(experts, n, k, plane_rows, top_k, pairs);
    if (need && (!workspace || workspace_bytes < need)) return Q8_ERR_ARG;
    const q8::Span spans[] = {{y, pairs * n * 4}, {need ? workspace : nullptr, static_cast<int64_t>(need)},
                              {w, weight_bytes(experts, n, k)}, {qs, plane_rows * k}, {ds, plane_rows * (k / 8)},
                              {offsets, 4 * (experts + 1)}, {rows, 4 * pairs}};
    if (q8::outputs_overlap(spans, 2, 7)) return Q8_ERR_ARG;
    for (const q8::Span &p : spans)
        if (!q8::aligned16(p.p)) return Q8_ERR_ALIGN;
    if (!q8::device_is_sm103()) return Q8_ERR_DEVICE;
    const q8::ExpertsArgs a = args_of(w, nullptr, experts, n, k, qs, ds, plane_rows, offsets, rows, top_k, pairs, y);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return many_rows(experts, pairs) ? q8::experts_tiles_launch(a, nullptr, nullptr, workspace, s) : experts_launch(a, s);
}

extern "C" size_t q8_0_experts_gate_up_workspace_bytes(int64_t experts, int64_t nf, int64_t k, int64_t plane_rows,
                                                       int64_t top_k, int64_t pairs)
{
    if (!sizes_ok(experts, nf, k, plane_rows, top_k, pairs) || nf % 32 != 0) return 0;
    if (many_rows(experts, pairs)) return q8::experts_tiles_workspace(k, pairs);
    return static_cast<size_t>(pairs) * nf * 8;
}

extern "C" int q8_0_experts_gate_up(const void *w_gate, const void *w_up, int64_t experts, int64_t nf, int64_t k,
                                    const int8_t *qs, const uint32_t *ds, int64_t plane_rows, const int32_t *offsets,
                                    const int32_t *rows, int64_t top_k, int64_t pairs, int8_t *qs_out, uint32_t *ds_out,
                                    void *workspace, size_t workspace_bytes, void *stream)
{
    if (!w_gate || !w_up || !qs || !ds || !offsets || !qs_out || !ds_out || nf % 32 != 0 ||
        !sizes_ok(experts, nf, k, plane_rows, top_k, pairs))
        return Q8_ERR_ARG;
    const size_t need = q8_0_experts_gate_up_workspace_bytes(experts, nf, k, plane_rows, top_k, pairs);
    if (need && (!workspace || workspace_bytes < need)) return Q8_ERR_ARG;
    const q8::Span spans[] = {{qs_out, pairs * nf}, {ds_out, pairs * (nf / 8)}, {need ? workspace : nullptr, static_cast<int64_t>(need)},
                              {w_gate, weight_bytes(experts, nf, k)}, {w_up, weight_bytes(experts, nf, k)},
                              {qs, plane_rows * k}, {ds, plane_rows * (k / 8)}, {offsets, 4 * (experts + 1)},
                              {rows, 4 * pairs}};
    if (q8::outputs_overlap(spans, 3, 9)) return Q8_ERR_ARG;
    for (const q8::Span &p : spans)
        if (!q8::aligned16(p.p)) return Q8_ERR_ALIGN;
    if (!q8::device_is_sm103()) return Q8_ERR_DEVICE;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    float *gu = static_cast<float *>(workspace);
    const q8::ExpertsArgs a = args_of(w_gate, w_up, experts, nf, k, qs, ds, plane_rows, offsets, rows, top_k, pairs, gu);
    if (many_rows(experts, pairs)) return q8::experts_tiles_launch(a, qs_out, ds_out, workspace, s);
    const int st = experts_launch(a, s);
    if (st != Q8_OK) return st;
    const int64_t ctas = (pairs * nf / 4 + 255) / 256;
    return q8::launch_pdl(experts_swiglu_kernel, dim3(static_cast<unsigned>(ctas < 152 * 8 ? ctas : 152 * 8)), dim3(256), 0, s,
                          reinterpret_cast<const float4 *>(gu), static_cast<int>(nf / 4), offsets, static_cast<int>(experts),
                          static_cast<int>(pairs), reinterpret_cast<uint32_t *>(qs_out), ds_out);
}

namespace q8 {

unsigned int *experts_error_word()
{
    void *p = nullptr;
    return cudaGetSymbolAddress(&p, g_experts_err) == cudaSuccess ? static_cast<unsigned int *>(p) : nullptr;
}

} // namespace q8
