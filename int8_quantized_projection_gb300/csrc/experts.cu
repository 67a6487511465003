// experts.cu -- products of sorted rows with their experts' Q8_0 matrices: the
// entry points, and SwiGLU of a gate and an up product into a q8_0 plane.
#include "experts_common.cuh"

namespace {

__device__ __forceinline__ float4 add4(float4 a, float4 b) { return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w); }

// gu [slices][pairs][2 nf] (gate, then up; the slices of k are added up in order) -> the plane of silu(gate) * up, of the rows
// that have products.
__global__ void __launch_bounds__(256)
experts_swiglu_kernel(const __grid_constant__ q8::ExpertsArgs a, const float4 *__restrict__ gu, int slices,
                      uint32_t *__restrict__ qs, uint32_t *__restrict__ ds)
{
    q8::griddep_launch_dependents();
    q8::griddep_wait();
    const int lane = threadIdx.x & 31, F = a.n / 4, first = a.offsets[0], last = a.offsets[a.experts];
    const int seen = q8::bad_offsets(a);
    const int64_t room = static_cast<int64_t>(a.pairs) * F, step = (static_cast<int64_t>(gridDim.x) * blockDim.x) / 32 * 32;
    int64_t base = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) / 32 * 32, total = room;
    bool known = false, bad = false;
    do {  // the first round's loads go out with those of the offsets, whatever these say
        const int64_t i = base + lane;
        const int r = static_cast<unsigned>(i >> 3) / static_cast<unsigned>(F >> 3);  // below 25 * 1024 rows of 2^17 blocks
        float4 g = make_float4(0.f, 0.f, 0.f, 0.f), u = g;
        int pair = 0;
        if (i < total) {
            const float4 *p = gu + static_cast<int64_t>(r) * F + i;
            g = p[0], u = p[F];
            if (a.rows) pair = a.rows[r];
            for (int k = 1; k < slices; ++k) {
                p += 2 * room;
                g = add4(g, p[0]), u = add4(u, p[F]);
            }
        }
        if (!known) {
            bad = __syncthreads_or(seen);
            known = true;
            if (bad && a.many) return;  // nothing has been computed
            total = static_cast<int64_t>(min(max(last, 0), a.pairs)) * F;
        }
        const q8::Q8Enc e = q8::q8_encode8(q8::silu_mul4(g, u));
        if (i < total && r >= first && q8::source_ok(a, r, pair) && (!bad || q8::expert_has(a, r))) {
            qs[i] = e.qword;
            if ((lane & 7) == 0) ds[i >> 3] = e.dsword;
        }
    } while ((base += step) < total);
}

bool sizes_ok(int64_t experts, int64_t n, int64_t k, int64_t plane_rows, int64_t top_k, int64_t pairs)
{
    const int64_t most = int64_t(1) << 31;
    return experts >= 1 && experts <= Q8_MAX_EXPERTS && n >= 1 && n <= Q8_EXPERTS_MAX_N && k >= 32 && k <= Q8_EXPERTS_MAX_K &&
           k % 32 == 0 && experts * n < most && plane_rows >= 1 && plane_rows < most && top_k >= 1 && top_k <= Q8_MAX_TOP_K &&
           pairs >= 1 && pairs < most - 256;
}

// Whether the tensor cores' tiles or the stream over the weights take a call: by the rows an expert has on average, all that the
// host knows.  64 experts of 2 x 1280 x 3584: 20 rows each 217 us streamed, 250 in tiles; 30 rows 288 and 256.  Eight of
// 18944 x 3584: 16 rows 169 and 212, 32 rows 278 and 224.  128 of 3584 x 1440, whose rows are copied one by one: 22 rows 391
// and 500, 31 rows 510 and 510, so that such widths would like the stream a little longer.  The average is that of the capacity:
// a call whose pairs are mostly padding takes the tiles all the same.
bool many_rows(int64_t experts, int64_t pairs) { return pairs >= 25 * experts; }

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
    if (!sizes_ok(experts, n, k, plane_rows, top_k, pairs)) return 0;
    if (many_rows(experts, pairs)) return q8::experts_tiles_workspace(k, pairs);
    const int slices = q8::experts_rows_slices(experts, pairs, k / 32);
    return slices > 1 ? static_cast<size_t>(slices) * pairs * n * 4 : 0;
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
    q8::ExpertsArgs a = args_of(w, nullptr, experts, n, k, qs, ds, plane_rows, offsets, rows, top_k, pairs, y);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (many_rows(experts, pairs)) return q8::experts_tiles_launch(a, nullptr, nullptr, workspace, s);
    a.many = q8::experts_rows_many(a);
    if (!need) return q8::experts_rows_launch(a, y, s);
    float *part = static_cast<float *>(workspace);
    const int st = q8::experts_rows_launch(a, part, s);
    return st != Q8_OK ? st : q8::experts_join_launch(part, q8::experts_rows_slices(experts, pairs, k / 32), a, s);
}

extern "C" size_t q8_0_experts_gate_up_workspace_bytes(int64_t experts, int64_t nf, int64_t k, int64_t plane_rows,
                                                       int64_t top_k, int64_t pairs)
{
    if (!sizes_ok(experts, nf, k, plane_rows, top_k, pairs) || nf % 32 != 0) return 0;
    if (many_rows(experts, pairs)) return q8::experts_tiles_workspace(k, pairs);
    return static_cast<size_t>(q8::experts_rows_slices(experts, pairs, k / 32)) * pairs * nf * 8;
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
    q8::ExpertsArgs a = args_of(w_gate, w_up, experts, nf, k, qs, ds, plane_rows, offsets, rows, top_k, pairs, gu);
    if (many_rows(experts, pairs)) return q8::experts_tiles_launch(a, qs_out, ds_out, workspace, s);
    a.many = q8::experts_rows_many(a);
    const int st = q8::experts_rows_launch(a, gu, s);
    if (st != Q8_OK) return st;
    const int64_t ctas = (pairs * nf / 4 + 255) / 256;
    return q8::launch_pdl(experts_swiglu_kernel, dim3(static_cast<unsigned>(ctas < 152 * 8 ? ctas : 152 * 8)), dim3(256), 0, s,
                          a, reinterpret_cast<const float4 *>(gu), q8::experts_rows_slices(experts, pairs, k / 32),
                          reinterpret_cast<uint32_t *>(qs_out), ds_out);
}
