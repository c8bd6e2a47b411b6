// Residual addition and layer norm of token rows, and its backward pass:
//   s = x + residual;  n = (s - mean(s)) / sqrt(var(s) + eps);
//   y = n weight + bias;
//   g = dy weight;  ds = (g - mean(g) - n mean(g n)) / sqrt(var + eps) + dres;
//   dweight = sum over rows of dy n;  dbias = sum over rows of dy.
// Forward sums are fp64, s and s^2 in one pass: the variance is their
// difference, which fp64 holds to 2^-52 (mean / deviation)^2, and squares of an
// fp32 stream's largest numbers do not overflow. Backward sums are fp32, and n is of
// the saved mean, one fp32 number: off by up to 2^-24 |mean| r. (What it lost could be
// found again only from the whole row, which the workgroups that sum columns do not see.)
//
// Both are bound by memory: a row is read once and stays in registers between
// its sums and its outputs. Forward, 16384 rows of 3584 with a bf16 residual: 81 us,
// 5.8 TB/s (a plain copy of 1 GiB: 5.1); backward with the stream's gradient 83 us,
// 5.8 TB/s, and 5 for the join of the column sums. Rows that are not 16-byte
// aligned: 106 and 107 (3583 columns). Rows of 16 waves, forward: 4000 of 20000 135
// us, 4.7 TB/s, 1000 of 65536 109, 4.8 (4000 of 16384, in four waves: 97, 5.4).
#include "common.hpp"
#include "layer_norm_plan.hpp"
#include "row_io.hpp"
#include "train.hpp"

namespace moe {

using namespace rows;

// WAVES waves hold a row of at most WAVES * 512 * NC elements. WAVES == 1:
// four rows a workgroup.
template <int WAVES, int NC, int MODE>
__global__ __launch_bounds__(WAVES == 1 ? 256 : WAVES * 64) void layer_norm_kernel(LayerNormArgs a) {
    constexpr int kLanes = WAVES * 64;
    const int tid = WAVES == 1 ? (int)threadIdx.x & 63 : (int)threadIdx.x;
    const int t = WAVES == 1 ? (int)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6)
                             : (int)blockIdx.x;
    if (WAVES == 1 && t >= a.T) return;  // whole waves; no barrier below when WAVES == 1
    const uint16_t* xr = a.x + t * a.ldx;
    const char* rr = (const char*)a.residual + t * a.ldr * (a.res_f32 ? 4 : 2);
    char* ro = (char*)a.residual_out + t * a.ldro * (a.res_f32 ? 4 : 2);
    const int H = a.H;
    auto first = [&](int c) { return (c * kLanes + tid) * 8; };
    // (A lane past the row's end fetches its first eight, not used.)
    auto inside = [&](int c) { return first(c) < H ? first(c) : 0; };
    f32x8 s[NC];
    double sum = 0.0, sq = 0.0;
    Raw8 fx[NC], fr[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) fx[c] = fetch8<MODE>(xr, false, inside(c), H);
    if (a.residual) {
#pragma unroll
        for (int c = 0; c < NC; ++c) fr[c] = fetch8<MODE>(rr, a.res_f32, inside(c), H);
    }
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int i = first(c);
        s[c] = widen8<MODE>(fx[c], false, i, H);
        if (a.residual) s[c] += widen8<MODE>(fr[c], a.res_f32, i, H);
        if (a.residual_out && i < H) put8<MODE>(ro, a.res_f32, i, H, s[c]);
        const int skip = i < H ? skip8<MODE>(i, H) : 8;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const double v = (double)(e >= skip ? s[c][e] : 0.0f);
            sum += v;
            sq = fma(v, v, sq);
        }
    }
    sum = wave_sum(sum);
    sq = wave_sum(sq);
    if constexpr (WAVES > 1) {
        __shared__ double part[WAVES][2];
        if ((tid & 63) == 0) {
            part[tid >> 6][0] = sum;
            part[tid >> 6][1] = sq;
        }
        __syncthreads();
        sum = sq = 0.0;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            sum += part[w][0];
            sq += part[w][1];
        }
    }
    const double mean = sum / (double)H;
    double var = sq / (double)H - mean * mean;
    var = var < 0.0 ? 0.0 : var;  // (a NaN stays one)
    const float rstd = (float)(1.0 / sqrt(var + (double)a.eps));
    // The mean as two fp32 numbers: next to a mean that is large against the
    // deviations, fp32 alone would lose them.
    const float mh = (float)mean, ml = fabsf(mh) < __builtin_inff() ? (float)(mean - (double)mh) : 0.0f;
    if (a.mean && tid == 0) {
        a.mean[t] = mh;
        a.rstd[t] = rstd;
    }
    if (!a.y) return;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int i = first(c);
        if (i >= H) continue;
        const Raw8 fw = fetch8<MODE>(a.weight, a.weight_f32, i, H);
        Raw8 fb;
        if (a.bias) fb = fetch8<MODE>(a.bias, a.weight_f32, i, H);
        const f32x8 w = widen8<MODE>(fw, a.weight_f32, i, H);
        f32x8 v = {0, 0, 0, 0, 0, 0, 0, 0};
        if (a.bias) v = widen8<MODE>(fb, a.weight_f32, i, H);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = fmaf(((s[c][e] - mh) - ml) * rstd, w[e], v[e]);
        put8<MODE>(a.y + t * a.ldy, false, i, H, v);
    }
}

template <int WAVES, int NC>
static void launch(const LayerNormArgs& a, bool vec, hipStream_t s) {
    const dim3 grid(WAVES == 1 ? (unsigned)((a.T + 3) / 4) : (unsigned)a.T), block(WAVES == 1 ? 256 : WAVES * 64);
    if (vec) hipLaunchKernelGGL((layer_norm_kernel<WAVES, NC, kAligned>), grid, block, 0, s, a);
    else if (a.H >= 8) hipLaunchKernelGGL((layer_norm_kernel<WAVES, NC, kAnywhere>), grid, block, 0, s, a);
    else if constexpr (WAVES == 1) hipLaunchKernelGGL((layer_norm_kernel<WAVES, NC, kTiny>), grid, block, 0, s, a);
}

static bool wide(const void* p, int64_t ld, int bytes) {
    return p == nullptr || ((uintptr_t)p % 16 == 0 && (ld * bytes) % 16 == 0);
}

hipError_t launch_layer_norm(const LayerNormArgs& a, hipStream_t s) {
    // A launch holds fewer than 2^32 threads (1024 a row at most).
    constexpr int kMostRows = 1 << 21;
    const int64_t rb = a.res_f32 ? 4 : 2;
    for (int t = 0; t < a.T; t += kMostRows) {
        LayerNormArgs b = a;
        b.T = a.T - t < kMostRows ? a.T - t : kMostRows;
        b.x = a.x + t * a.ldx;
        if (a.residual) b.residual = (const char*)a.residual + t * a.ldr * rb;
        if (a.residual_out) b.residual_out = (char*)a.residual_out + t * a.ldro * rb;
        if (a.y) b.y = a.y + t * a.ldy;
        if (a.mean) {
            b.mean = a.mean + t;
            b.rstd = a.rstd + t;
        }
        const bool vec = b.H % 8 == 0 && wide(b.x, b.ldx, 2) && wide(b.residual, b.ldr, (int)rb) &&
                         wide(b.residual_out, b.ldro, (int)rb) && wide(b.y, b.ldy, 2) && wide(b.weight, 0, 4) &&
                         wide(b.bias, 0, 4);
        // Waves a row that its columns keep busy (1024 columns, 32768 rows: 46 us in
        // two waves, 61 in four).
        if (b.H <= 512) launch<1, 1>(b, vec, s);
        else if (b.H <= 1024) launch<2, 1>(b, vec, s);
        else if (b.H <= 2048) launch<4, 1>(b, vec, s);
        else if (b.H <= 4096) launch<4, 2>(b, vec, s);
        else if (b.H <= 8192) launch<4, 4>(b, vec, s);
        else if (b.H <= 16384) launch<4, 8>(b, vec, s);
        else if (b.H <= 32768) launch<16, 4>(b, vec, s);
        else launch<16, 8>(b, vec, s);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

// ------------------------------------------------------------- backward
// A workgroup goes through rows blockIdx.x, + gridDim.x, ... and keeps its
// columns' sums of dy n and dy in registers, so the rows are read once.
template <int WAVES, int NC, int MODE, bool S32>
__device__ __forceinline__ void layer_norm_bwd_rows(const LayerNormBwdArgs& a, int groups) {
    constexpr int kLanes = WAVES * 64, kRows = WAVES == 1 ? 4 : 1;
    const int tid = WAVES == 1 ? (int)threadIdx.x & 63 : (int)threadIdx.x;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int H = a.H;
    const float inv = 1.0f / (float)H;
    __shared__ float part[WAVES > 1 ? 2 : 1][WAVES][2];
    auto first = [&](int c) { return (c * kLanes + tid) * 8; };
    const f32x8 zero = {0, 0, 0, 0, 0, 0, 0, 0};
    // (A lane past the row's end fetches its first eight, not used.)
    auto inside = [&](int c) { return first(c) < H ? first(c) : 0; };
    f32x8 aw[NC], ab[NC];
    Raw8 fw[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        aw[c] = ab[c] = zero;
        fw[c] = fetch8<MODE>(a.weight, a.weight_f32, inside(c), H);
    }
    int flip = 0;
    const int64_t step = (int64_t)groups * kRows;
    for (int64_t t = (int64_t)blockIdx.x * kRows + (WAVES == 1 ? wave : 0); t < a.T; t += step) {
        const float mean = a.mean[t], rstd = a.rstd[t];
        Raw8 fd[NC], fs[NC], fr[NC];
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            fd[c] = fetch8<MODE>(a.dy + t * a.lddy, false, inside(c), H);
            fs[c] = fetch8<MODE>((const char*)a.s + t * a.lds * (S32 ? 4 : 2), S32, inside(c), H);
        }
        if (a.dres) {
#pragma unroll
            for (int c = 0; c < NC; ++c) fr[c] = fetch8<MODE>((const char*)a.dres + t * a.lddr * (S32 ? 4 : 2), S32, inside(c), H);
        }
        f32x8 d[NC], n[NC];
        float sg = 0.0f, sgn = 0.0f;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int i = first(c), skip = i < H ? skip8<MODE>(i, H) : 8;
            const f32x8 w = widen8<MODE>(fw[c], a.weight_f32, i, H);
            d[c] = widen8<MODE>(fd[c], false, i, H);
            n[c] = widen8<MODE>(fs[c], S32, i, H);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float own = e >= skip ? d[c][e] : 0.0f;
                // (Of a lane past the row, which could be infinite.)
                n[c][e] = MODE == kAligned && i >= H ? 0.0f : (n[c][e] - mean) * rstd;
                aw[c][e] = fmaf(own, n[c][e], aw[c][e]);
                ab[c][e] += own;
                d[c][e] *= w[e];
                const float g = own * w[e];
                sg += g;
                sgn = fmaf(g, n[c][e], sgn);
            }
        }
        sg = wave_sum(sg);
        sgn = wave_sum(sgn);
        if constexpr (WAVES > 1) {
            // Two sets in turn: a wave that is a row ahead writes the other.
            if ((tid & 63) == 0) {
                part[flip][wave][0] = sg;
                part[flip][wave][1] = sgn;
            }
            __syncthreads();
            sg = sgn = 0.0f;
#pragma unroll
            for (int k = 0; k < WAVES; ++k) {
                sg += part[flip][k][0];
                sgn += part[flip][k][1];
            }
            flip ^= 1;
        }
        const float mg = sg * inv, mgn = sgn * inv;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int i = first(c);
            if (i >= H) continue;
            f32x8 v;
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = rstd * ((d[c][e] - mg) - n[c][e] * mgn);
            if (a.dres) v += widen8<MODE>(fr[c], S32, i, H);
            if (a.dx) put8<MODE>(a.dx + t * a.lddx, false, i, H, v);
            if (a.dresidual) put8<MODE>((char*)a.dresidual + t * a.lddro * (S32 ? 4 : 2), S32, i, H, v);
        }
    }
    if (!a.partial) return;
    const int ld = (H + 7) & ~7;
    float* p = a.partial + (int64_t)blockIdx.x * 2 * ld;
    // (What lies behind the row's last column is not read as numbers.)
    if constexpr (WAVES == 1) {
        __shared__ float sum[4][512];
        const int i = first(0), skip = i < H ? skip8<MODE>(i, H) : 8, at = i - skip;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            __syncthreads();
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e >= skip) sum[wave][at + e] = k ? ab[0][e] : aw[0][e];
            __syncthreads();
            for (int c = (int)threadIdx.x; c < H; c += 256) p[k * ld + c] = (sum[0][c] + sum[1][c]) + (sum[2][c] + sum[3][c]);
        }
    } else {
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int i = first(c), skip = skip8<MODE>(i, H);
            if (i >= H) continue;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const f32x8 v = k ? ab[c] : aw[c];
                if (skip == 0) {
                    *(f32x4*)(p + k * ld + i) = __builtin_shufflevector(v, v, 0, 1, 2, 3);
                    *(f32x4*)(p + k * ld + i + 4) = __builtin_shufflevector(v, v, 4, 5, 6, 7);
                } else {
#pragma unroll
                    for (int e = 1; e < 8; ++e)
                        if (e >= skip) p[k * ld + i - skip + e] = v[e];
                }
            }
        }
    }
}

template <int WAVES, int NC, int MODE, bool S32>
__global__ __launch_bounds__(WAVES == 1 ? 256 : WAVES * 64) void layer_norm_bwd_kernel(LayerNormBwdArgs a) {
    layer_norm_bwd_rows<WAVES, NC, MODE, S32>(a, (int)gridDim.x);
}

// Few rows: workgroups of a row (four rows for one wave a row) and, in the same
// launch, workgroups of 32 columns that go through all rows again for the sums,
// which makes no partial sums and no second launch. Those take as many rows
// a turn as they have threads, and a turn is a latency of memory: 777 rows of 1001, in
// two waves, are seven turns, 11.8 us.
template <int WAVES, int NC, int MODE, bool S32>
__global__ __launch_bounds__(WAVES == 1 ? 256 : WAVES * 64) void layer_norm_bwd_few_kernel(LayerNormBwdArgs a, int row_groups) {
    constexpr int kThreads = WAVES == 1 ? 256 : WAVES * 64, kRuns = kThreads / 4, kAtOnce = 4;
    if ((int)blockIdx.x < row_groups) {
        a.partial = nullptr;
        layer_norm_bwd_rows<WAVES, NC, MODE, S32>(a, row_groups);
        return;
    }
    // Four lanes a row, eight columns each; the runs of rows meet in LDS.
    __shared__ float lds[2][kRuns][32 + 1];
    const int tid = (int)threadIdx.x, q = tid & 3, run = tid >> 2, H = a.H;
    const int c0 = ((int)blockIdx.x - row_groups) * 32, i = c0 + q * 8, at = i < H ? i : 0;
    f32x8 aw = {0, 0, 0, 0, 0, 0, 0, 0}, ab = aw;
    for (int t0 = run; t0 < a.T; t0 += kRuns * kAtOnce) {
        Raw8 fd[kAtOnce], fs[kAtOnce];
        float mean[kAtOnce], rstd[kAtOnce];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            // (A row past the end: the first one, not used.)
            const int64_t t = t0 + k * kRuns < a.T ? t0 + k * kRuns : t0;
            mean[k] = a.mean[t];
            rstd[k] = a.rstd[t];
            fd[k] = fetch8<MODE>(a.dy + t * a.lddy, false, at, H);
            fs[k] = fetch8<MODE>((const char*)a.s + t * a.lds * (S32 ? 4 : 2), S32, at, H);
        }
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            if (t0 + k * kRuns >= a.T) continue;
            const f32x8 d = widen8<MODE>(fd[k], false, at, H), n = widen8<MODE>(fs[k], S32, at, H);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                aw[e] = fmaf(d[e], (n[e] - mean[k]) * rstd[k], aw[e]);
                ab[e] += d[e];
            }
        }
    }
    const int skip = i < H ? skip8<MODE>(i, H) : 8;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        if (e < skip) continue;
        lds[0][run][q * 8 - skip + e] = aw[e];
        lds[1][run][q * 8 - skip + e] = ab[e];
    }
    // 64 sums (32 columns, two sets) of kRuns runs, two threads each.
    __syncthreads();
    const int sum = (tid >> 1) & 63, set = sum >> 5, c = c0 + (sum & 31);
    float v = 0.0f;
    if (tid < 128) {
        for (int k = tid & 1; k < kRuns; k += 2) v += lds[set][k][sum & 31];
        v += dpp<0xB1>(v);  // (the neighbour's)
    }
    void* out = set ? a.dbias : a.dweight;
    if (tid >= 128 || (tid & 1) || !out || c >= H) return;
    if (a.weight_f32) ((float*)out)[c] = v;
    else ((uint16_t*)out)[c] = f32_to_bf16_bits(v);
}

// Rows that registers do not hold: a workgroup a row, which is read twice (the
// second time from L2). With the columns' sums below, 4000 rows of 12288 with a bf16
// stream 119 us (393 MB read or written once: 3.3 TB/s); of 10001: 138.
template <int MODE, bool S32>
__global__ __launch_bounds__(1024) void layer_norm_bwd_long_kernel(LayerNormBwdArgs a) {
    __shared__ float part[16][2];
    const int tid = (int)threadIdx.x, H = a.H;
    const int64_t t = (int64_t)blockIdx.x;
    const float mean = a.mean[t], rstd = a.rstd[t], inv = 1.0f / (float)H;
    const uint16_t* dr = a.dy + t * a.lddy;
    const char* sr = (const char*)a.s + t * a.lds * (S32 ? 4 : 2);
    float sg = 0.0f, sgn = 0.0f;
    for (int i = tid * 8; i < H; i += 8192) {
        const Raw8 fd = fetch8<MODE>(dr, false, i, H), fs = fetch8<MODE>(sr, S32, i, H), fw = fetch8<MODE>(a.weight, a.weight_f32, i, H);
        const f32x8 d = widen8<MODE>(fd, false, i, H), n = widen8<MODE>(fs, S32, i, H), w = widen8<MODE>(fw, a.weight_f32, i, H);
        const int skip = skip8<MODE>(i, H);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (e < skip) continue;
            const float g = d[e] * w[e];
            sg += g;
            sgn = fmaf(g, (n[e] - mean) * rstd, sgn);
        }
    }
    sg = wave_sum(sg);
    sgn = wave_sum(sgn);
    if ((tid & 63) == 0) {
        part[tid >> 6][0] = sg;
        part[tid >> 6][1] = sgn;
    }
    __syncthreads();
    sg = sgn = 0.0f;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
        sg += part[k][0];
        sgn += part[k][1];
    }
    const float mg = sg * inv, mgn = sgn * inv;
    for (int i = tid * 8; i < H; i += 8192) {
        const Raw8 fd = fetch8<MODE>(dr, false, i, H), fs = fetch8<MODE>(sr, S32, i, H), fw = fetch8<MODE>(a.weight, a.weight_f32, i, H);
        Raw8 fr;
        if (a.dres) fr = fetch8<MODE>((const char*)a.dres + t * a.lddr * (S32 ? 4 : 2), S32, i, H);
        const f32x8 d = widen8<MODE>(fd, false, i, H), n = widen8<MODE>(fs, S32, i, H), w = widen8<MODE>(fw, a.weight_f32, i, H);
        f32x8 v;
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = rstd * ((d[e] * w[e] - mg) - (n[e] - mean) * rstd * mgn);
        if (a.dres) v += widen8<MODE>(fr, S32, i, H);
        if (a.dx) put8<MODE>(a.dx + t * a.lddx, false, i, H, v);
        if (a.dresidual) put8<MODE>((char*)a.dresidual + t * a.lddro * (S32 ? 4 : 2), S32, i, H, v);
    }
}

// The sums over the rows alone: a thread eight columns, rows blockIdx.y, +
// gridDim.y, ..., four in flight (16000 rows of 10001 without the stream's gradient,
// with the rows' launch: 481 us, one at a time 890).
template <int MODE, bool S32>
__global__ __launch_bounds__(256) void layer_norm_columns_kernel(LayerNormBwdArgs a) {
    constexpr int kAtOnce = 4;
    const int i = ((int)blockIdx.x * 256 + (int)threadIdx.x) * 8, H = a.H;
    if (i >= H) return;
    f32x8 aw = {0, 0, 0, 0, 0, 0, 0, 0}, ab = aw;
    const int64_t step = (int64_t)gridDim.y;
    for (int64_t t0 = (int64_t)blockIdx.y; t0 < a.T; t0 += step * kAtOnce) {
        Raw8 fd[kAtOnce], fs[kAtOnce];
        float mean[kAtOnce], rstd[kAtOnce];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            // (A row past the end: the first one, not used.)
            const int64_t t = t0 + k * step < a.T ? t0 + k * step : t0;
            mean[k] = a.mean[t];
            rstd[k] = a.rstd[t];
            fd[k] = fetch8<MODE>(a.dy + t * a.lddy, false, i, H);
            fs[k] = fetch8<MODE>((const char*)a.s + t * a.lds * (S32 ? 4 : 2), S32, i, H);
        }
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            if (t0 + k * step >= a.T) continue;
            const f32x8 d = widen8<MODE>(fd[k], false, i, H), n = widen8<MODE>(fs[k], S32, i, H);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                aw[e] = fmaf(d[e], (n[e] - mean[k]) * rstd[k], aw[e]);
                ab[e] += d[e];
            }
        }
    }
    const int ld = (H + 7) & ~7, skip = skip8<MODE>(i, H);
    float* p = a.partial + (int64_t)blockIdx.y * 2 * ld + i - skip;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        if (e < skip) continue;
        p[e] = aw[e];
        p[ld + e] = ab[e];
    }
}

template <int RUNS>
__global__ __launch_bounds__(RUNS * 8) void column_join_kernel(ColumnJoin j) {
    __shared__ float lds[column_join_lds(RUNS) / 4];
    column_join<RUNS>(j, (int)blockIdx.x, lds);
}

hipError_t launch_column_join(const ColumnJoin& j, bool few, hipStream_t s) {
    const dim3 grid((unsigned)column_join_groups(j));
    if (few) hipLaunchKernelGGL(column_join_kernel<kFewRuns>, grid, dim3(kFewRuns * 8), 0, s, j);
    else hipLaunchKernelGGL(column_join_kernel<128>, grid, dim3(1024), 0, s, j);
    return hipGetLastError();
}

template <int WAVES, int NC, int MODE, bool S32>
static void launch_bwd_as(const LayerNormBwdArgs& a, hipStream_t s) {
    const bool sums = a.dweight || a.dbias;
    const int groups = layer_norm_row_groups(a.T, a.H, sums), threads = WAVES == 1 ? 256 : WAVES * 64;
    if (layer_norm_few_rows(a.T, a.H)) {
        const int rows = a.dx || a.dresidual ? groups : 0, cols = sums ? (a.H + 31) / 32 : 0;
        hipLaunchKernelGGL((layer_norm_bwd_few_kernel<WAVES, NC, MODE, S32>), dim3((unsigned)(rows + cols)), dim3(threads), 0, s, a, rows);
    } else if constexpr (WAVES < 16) {
        hipLaunchKernelGGL((layer_norm_bwd_kernel<WAVES, NC, MODE, S32>), dim3((unsigned)groups), dim3(threads), 0, s, a);
    }
}

template <int WAVES, int NC, bool S32>
static void launch_bwd_mode(const LayerNormBwdArgs& a, bool vec, hipStream_t s) {
    if (vec) launch_bwd_as<WAVES, NC, kAligned, S32>(a, s);
    else if (a.H >= 8) launch_bwd_as<WAVES, NC, kAnywhere, S32>(a, s);
    else if constexpr (WAVES == 1) launch_bwd_as<WAVES, NC, kTiny, S32>(a, s);
}

template <int WAVES, int NC>
static void launch_bwd(const LayerNormBwdArgs& a, bool vec, hipStream_t s) {
    if (a.s_f32) launch_bwd_mode<WAVES, NC, true>(a, vec, s);
    else launch_bwd_mode<WAVES, NC, false>(a, vec, s);
}

template <int MODE, bool S32>
static hipError_t launch_long(const LayerNormBwdArgs& a, hipStream_t s) {
    if (a.dx || a.dresidual) {
        constexpr int kMostRows = 1 << 21;  // of 1024 threads: a launch holds fewer than 2^32
        for (int t = 0; t < a.T; t += kMostRows) {
            LayerNormBwdArgs b = a;
            const int64_t sb = S32 ? 4 : 2;
            b.T = a.T - t < kMostRows ? a.T - t : kMostRows;
            b.dy = a.dy + t * a.lddy;
            b.s = (const char*)a.s + t * a.lds * sb;
            b.mean = a.mean + t;
            b.rstd = a.rstd + t;
            if (a.dres) b.dres = (const char*)a.dres + t * a.lddr * sb;
            if (a.dx) b.dx = a.dx + t * a.lddx;
            if (a.dresidual) b.dresidual = (char*)a.dresidual + t * a.lddro * sb;
            hipLaunchKernelGGL((layer_norm_bwd_long_kernel<MODE, S32>), dim3((unsigned)b.T), dim3(1024), 0, s, b);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
    }
    if (a.partial) {
        const dim3 grid((unsigned)((a.H + 2047) / 2048), (unsigned)layer_norm_parts(a.T, a.H));
        hipLaunchKernelGGL((layer_norm_columns_kernel<MODE, S32>), grid, dim3(256), 0, s, a);
    }
    return hipGetLastError();
}

hipError_t launch_layer_norm_bwd(const LayerNormBwdArgs& a, hipStream_t s) {
    const bool sums = a.dweight || a.dbias;
    if (a.T > 0) {
        const int sb = a.s_f32 ? 4 : 2;
        const bool vec = a.H % 8 == 0 && wide(a.dy, a.lddy, 2) && wide(a.s, a.lds, sb) && wide(a.dres, a.lddr, sb) &&
                         wide(a.dx, a.lddx, 2) && wide(a.dresidual, a.lddro, sb) && wide(a.weight, 0, 4);
        hipError_t e = hipSuccess;
        if (a.H <= 512) launch_bwd<1, 1>(a, vec, s);
        else if (a.H <= 1024) launch_bwd<2, 1>(a, vec, s);
        else if (a.H <= 2048) launch_bwd<4, 1>(a, vec, s);
        else if (a.H <= 4096) launch_bwd<4, 2>(a, vec, s);
        else if (a.H <= 8192) launch_bwd<8, 2>(a, vec, s);
        else if (layer_norm_few_rows(a.T, a.H)) launch_bwd<16, 2>(a, vec, s);
        else if (a.s_f32) e = vec ? launch_long<kAligned, true>(a, s) : launch_long<kAnywhere, true>(a, s);
        else e = vec ? launch_long<kAligned, false>(a, s) : launch_long<kAnywhere, false>(a, s);
        if (e == hipSuccess) e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (!sums || (a.T > 0 && layer_norm_few_rows(a.T, a.H))) return hipSuccess;
    return launch_column_join({a.partial, a.dweight, a.dbias, layer_norm_parts(a.T, a.H), a.H, (a.H + 7) & ~7, 2, a.weight_f32},
                              false, s);
}

}  // namespace moe
