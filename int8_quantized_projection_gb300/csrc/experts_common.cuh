// experts_common.cuh -- what the kernels of the experts' products share: the
// arguments of a launch and the lookup of a sorted row's source.
#pragma once

#include "kv_common.cuh"

namespace q8 {

// One product over grouped rows: for the rows r of expert e, offsets[e] <= r < offsets[e + 1],
//     out[r * ld + i] = w[e][i] . plane[source(r)],   i < n,
// and with w2 the same for a second matrix into out[r * ld + n + i].
struct ExpertsArgs {
    const uint8_t *w, *w2;    // [experts][n] rows of nb Q8_0 blocks; w2 may be nullptr
    const int8_t *qs;         // plane [plane_rows][32 nb]
    const uint32_t *ds;       // [plane_rows][nb]
    const int32_t *offsets;   // [experts + 1]
    const int32_t *rows;      // pair of each sorted row, or nullptr: row r reads plane row r
    float *out;
    int64_t plane_rows, ld;
    int experts, n, nb, top_k, pairs;
    bool many;                // the work's numbers would pass 31 bits if every second expert had all rows
};

// Many rows an expert, on the tensor cores (experts_tiles.cu): the f32 rows, or with qs_out and w2 the plane of silu(w x) * (w2 x).
size_t experts_tiles_workspace(int64_t k, int64_t pairs);
int experts_tiles_launch(const ExpertsArgs &a, int8_t *qs_out, uint32_t *ds_out, void *workspace, cudaStream_t s);

// A few rows an expert (experts_rows.cu): the f32 rows into out, or, where k is cut into several slices, their parts [slices][pairs][ld],
// which the join adds up into a.out.  experts_rows_many: a.many, for all three.
int experts_rows_slices(int64_t experts, int64_t pairs, int64_t nb);
bool experts_rows_many(const ExpertsArgs &a);
int experts_rows_launch(const ExpertsArgs &a, float *out, cudaStream_t s);
int experts_join_launch(const float *part, int slices, const ExpertsArgs &a, cudaStream_t s);

// The rows of expert e, checked: an expert whose offsets are out of range has none.
struct ExpertRows {
    int first, count;
    bool bad;
};

__device__ __forceinline__ ExpertRows expert_rows_of(const ExpertsArgs &a, int e)
{
    const int lo = a.offsets[e], hi = a.offsets[e + 1];
    const bool bad = lo < 0 || hi < lo || hi > a.pairs;
    return {lo, bad ? 0 : hi - lo, bad};
}

// Plane row of sorted row r, or -1 where it is out of range.
__device__ __forceinline__ int64_t source_row(const ExpertsArgs &a, int r)
{
    int64_t s = r;
    if (a.rows) {
        const int p = a.rows[r];
        s = p < 0 ? -1 : p / a.top_k;
    }
    return s < a.plane_rows ? s : -1;
}

// The same question of sorted row r whose pair is p = rows[r]: whether it is in range.
__device__ __forceinline__ bool source_ok(const ExpertsArgs &a, int r, int p)
{
    return a.rows ? p >= 0 && p < a.plane_rows * a.top_k : r < a.plane_rows;
}

// The passes behind the stream read its products from a workspace, where rows that it stored nothing for hold anything: those that
// no expert with right offsets has, and those whose pair is out of range.  While all offsets are right, an expert has every row
// from offsets[0] to offsets[experts]; the CTA's threads look at all of them once, beside its first loads: this thread's share.
__device__ __forceinline__ int bad_offsets(const ExpertsArgs &a)
{
    int bad = 0;
    for (int e = threadIdx.x; e < a.experts; e += blockDim.x) bad |= expert_rows_of(a, e).bad;
    return bad;
}

// Where some are not: whether an expert has sorted row r, offsets[0] <= r < offsets[experts].
__device__ __forceinline__ bool expert_has(const ExpertsArgs &a, int r)
{
    int lo = 0, hi = a.experts;  // the last expert that starts at r or before
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.offsets[mid] <= r)
            lo = mid;
        else
            hi = mid;
    }
    const ExpertRows x = expert_rows_of(a, lo);
    return !x.bad && r - x.first < x.count;
}

} // namespace q8
