// Sums of columns over parts: out[c] = sum over p of partial[p, c] (fp32, each
// run of parts in order, then the runs).
#pragma once

#include "common.hpp"

namespace moe {

// partial [parts, 2 or 1 sets of `ld` columns]; the first n columns of a set go
// to out0 (and of the second to out1). ld is a multiple of 4.
struct ColumnJoin {
    const float* partial;
    void* out0;  // either may be null
    void* out1;
    int parts, n, ld, sets;
    int f32;     // outputs: fp32, else bf16
};

constexpr int kJoinColumns = 32;  // of a workgroup

inline int column_join_groups(const ColumnJoin& j) { return j.sets * ((j.n + kJoinColumns - 1) / kJoinColumns); }
constexpr int column_join_lds(int runs) { return runs * kJoinColumns * 4; }

// Workgroup `group` of column_join_groups, of 8 RUNS threads or more (those
// beyond wait): eight threads a part take four columns each, eight parts at once;
// RUNS runs of parts meet in LDS (column_join_lds bytes). The order of a sum
// goes by RUNS alone.
template <int RUNS>
__device__ __forceinline__ void column_join(const ColumnJoin& j, int group, float* lds) {
    constexpr int kAtOnce = 8;
    const int per = (j.n + kJoinColumns - 1) / kJoinColumns;
    const int set = group / per, c0 = group % per * kJoinColumns;
    void* out = set ? j.out1 : j.out0;
    if (!out) return;
    const int tid = (int)threadIdx.x, q = tid & 7, run = tid >> 3;
    const float* p = j.partial + (int64_t)set * j.ld + c0 + 4 * q;
    const int64_t step = (int64_t)j.sets * j.ld;
    const bool ok = c0 + 4 * q < j.ld && run < RUNS;
    f32x4 sum = {0, 0, 0, 0};
    for (int k0 = run; k0 < j.parts; k0 += kAtOnce * RUNS) {
        f32x4 v[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            const int k = k0 + i * RUNS;
            v[i] = ok && k < j.parts ? *(const f32x4*)(p + k * step) : f32x4{0, 0, 0, 0};
        }
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) sum += v[i];
    }
    if (run < RUNS) *(f32x4*)(lds + run * kJoinColumns + 4 * q) = sum;
    // Halves, down to the eight runs that one thread a column sums.
#pragma unroll
    for (int half = RUNS / 2; half >= 8; half /= 2) {
        __syncthreads();
        if (run < half) {
            sum += *(const f32x4*)(lds + (run + half) * kJoinColumns + 4 * q);
            *(f32x4*)(lds + run * kJoinColumns + 4 * q) = sum;
        }
    }
    __syncthreads();
    const int c = c0 + tid;
    if (tid >= kJoinColumns || c >= j.n) return;
    float v = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) v += lds[k * kJoinColumns + tid];
    if (j.f32) ((float*)out)[c] = v;
    else ((uint16_t*)out)[c] = f32_to_bf16_bits(v);
}

// few: kFewRuns runs, as beside tiles; else 128.
constexpr int kFewRuns = 32;
hipError_t launch_column_join(const ColumnJoin& j, bool few, hipStream_t s);

}  // namespace moe
