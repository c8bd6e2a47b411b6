// Residual addition and layer norm of token rows, and its backward pass:
//   s = x + residual;  n = (s - mean(s)) / sqrt(var(s) + eps);
//   y = n weight + bias;
//   g = dy weight;  ds = (g - mean(g) - n mean(g n)) / sqrt(var + eps) + dres;
//   dweight = sum over rows of dy n;  dbias = sum over rows of dy.
// Forward sums are fp64, s and s^2 in one pass: the variance is their
// difference, which fp64 holds to 2^-52 (mean / deviation)^2, and squares of an
// fp32 stream's largest numbers do not overflow. Backward sums are fp32.
#include "common.hpp"
#include "row_io.hpp"
#include "train.hpp"

namespace moe {

using namespace rows;

// WAVES waves hold a row of at most WAVES * 512 * NC elements. WAVES == 1:
// four rows a workgroup.
template <int WAVES, int NC, bool VEC>
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
    f32x8 s[NC];
    double sum = 0.0, sq = 0.0;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int i = first(c);
        s[c] = f32x8{0, 0, 0, 0, 0, 0, 0, 0};
        if (i < H) {
            s[c] = load8<VEC>(xr, false, i, H);
            if (a.residual) s[c] += load8<VEC>(rr, a.res_f32, i, H);
        }
    }
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int i = first(c);
        if (a.residual_out && i < H) store8<VEC>(ro, a.res_f32, i, H, s[c]);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const double v = (double)s[c][e];
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
        const f32x8 w = load8<VEC>(a.weight, a.weight_f32, i, H);
        f32x8 v = {0, 0, 0, 0, 0, 0, 0, 0};
        if (a.bias) v = load8<VEC>(a.bias, a.weight_f32, i, H);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = fmaf(((s[c][e] - mh) - ml) * rstd, w[e], v[e]);
        store8<VEC>(a.y + t * a.ldy, false, i, H, v);
    }
}

template <int WAVES, int NC>
static void launch(const LayerNormArgs& a, bool vec, hipStream_t s) {
    const dim3 grid(WAVES == 1 ? (unsigned)((a.T + 3) / 4) : (unsigned)a.T), block(WAVES == 1 ? 256 : WAVES * 64);
    if (vec) hipLaunchKernelGGL((layer_norm_kernel<WAVES, NC, true>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((layer_norm_kernel<WAVES, NC, false>), grid, block, 0, s, a);
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
        if (b.H <= 512) launch<1, 1>(b, vec, s);
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
template <int WAVES, int NC, bool VEC, bool S32>
__global__ __launch_bounds__(WAVES == 1 ? 256 : WAVES * 64) void layer_norm_bwd_kernel(LayerNormBwdArgs a) {
    constexpr int kLanes = WAVES * 64, kRows = WAVES == 1 ? 4 : 1;
    const int tid = WAVES == 1 ? (int)threadIdx.x & 63 : (int)threadIdx.x;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int H = a.H;
    const float inv = 1.0f / (float)H;
    __shared__ float part[WAVES > 1 ? 2 : 1][WAVES][2];
    auto first = [&](int c) { return (c * kLanes + tid) * 8; };
    const f32x8 zero = {0, 0, 0, 0, 0, 0, 0, 0};
    f32x8 w[NC], aw[NC], ab[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        aw[c] = ab[c] = w[c] = zero;
        if (first(c) < H) w[c] = load8<VEC>(a.weight, a.weight_f32, first(c), H);
    }
    int flip = 0;
    for (int64_t t = (int64_t)blockIdx.x * kRows + (WAVES == 1 ? wave : 0); t < a.T; t += (int64_t)gridDim.x * kRows) {
        const float mean = a.mean[t], rstd = a.rstd[t];
        const char* sr = (const char*)a.s + t * a.lds * (S32 ? 4 : 2);
        f32x8 d[NC], n[NC];
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int i = first(c);
            d[c] = n[c] = zero;
            if (i < H) {
                d[c] = load8<VEC>(a.dy + t * a.lddy, false, i, H);
                n[c] = load8<VEC>(sr, S32, i, H);
            }
        }
        float sg = 0.0f, sgn = 0.0f;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int i = first(c);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                // (Columns past the row have dy and weight 0.)
                n[c][e] = (VEC ? i < H : i + e < H) ? (n[c][e] - mean) * rstd : 0.0f;
                aw[c][e] = fmaf(d[c][e], n[c][e], aw[c][e]);
                ab[c][e] += d[c][e];
                d[c][e] *= w[c][e];
                sg += d[c][e];
                sgn = fmaf(d[c][e], n[c][e], sgn);
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
            if (a.dres) v += load8<VEC>((const char*)a.dres + t * a.lddr * (S32 ? 4 : 2), S32, i, H);
            if (a.dx) store8<VEC>(a.dx + t * a.lddx, false, i, H, v);
            if (a.dresidual) store8<VEC>((char*)a.dresidual + t * a.lddro * (S32 ? 4 : 2), S32, i, H, v);
        }
    }
    if (!a.partial) return;
    float* p = a.partial + (int64_t)blockIdx.x * 2 * H;
    if constexpr (WAVES == 1) {
        __shared__ float sum[4][512];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            __syncthreads();
#pragma unroll
            for (int e = 0; e < 8; ++e) sum[wave][tid * 8 + e] = k ? ab[0][e] : aw[0][e];
            __syncthreads();
            for (int i = (int)threadIdx.x; i < H; i += 256) p[k * H + i] = (sum[0][i] + sum[1][i]) + (sum[2][i] + sum[3][i]);
        }
    } else {
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int i = first(c);
            if (i >= H) continue;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const f32x8 v = k ? ab[c] : aw[c];
                if constexpr (VEC) {
                    *(f32x4*)(p + k * H + i) = __builtin_shufflevector(v, v, 0, 1, 2, 3);
                    *(f32x4*)(p + k * H + i + 4) = __builtin_shufflevector(v, v, 4, 5, 6, 7);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (i + e < H) p[k * H + i + e] = v[e];
                }
            }
        }
    }
}

// Rows that registers do not hold: a workgroup a row, which is read twice (the
// second time from L2).
template <bool VEC, bool S32>
__global__ __launch_bounds__(1024) void layer_norm_bwd_long_kernel(LayerNormBwdArgs a) {
    __shared__ float part[16][2];
    const int tid = (int)threadIdx.x, H = a.H;
    const int64_t t = (int64_t)blockIdx.x;
    const float mean = a.mean[t], rstd = a.rstd[t], inv = 1.0f / (float)H;
    const uint16_t* dr = a.dy + t * a.lddy;
    const char* sr = (const char*)a.s + t * a.lds * (S32 ? 4 : 2);
    float sg = 0.0f, sgn = 0.0f;
    for (int i = tid * 8; i < H; i += 8192) {
        const f32x8 d = load8<VEC>(dr, false, i, H), n = load8<VEC>(sr, S32, i, H), w = load8<VEC>(a.weight, a.weight_f32, i, H);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (!VEC && i + e >= H) continue;
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
        const f32x8 d = load8<VEC>(dr, false, i, H), n = load8<VEC>(sr, S32, i, H), w = load8<VEC>(a.weight, a.weight_f32, i, H);
        f32x8 v;
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = rstd * ((d[e] * w[e] - mg) - (n[e] - mean) * rstd * mgn);
        if (a.dres) v += load8<VEC>((const char*)a.dres + t * a.lddr * (S32 ? 4 : 2), S32, i, H);
        if (a.dx) store8<VEC>(a.dx + t * a.lddx, false, i, H, v);
        if (a.dresidual) store8<VEC>((char*)a.dresidual + t * a.lddro * (S32 ? 4 : 2), S32, i, H, v);
    }
}

// The sums over the rows alone: a thread eight columns, rows blockIdx.y, +
// gridDim.y, ...
template <bool VEC, bool S32>
__global__ __launch_bounds__(256) void layer_norm_columns_kernel(LayerNormBwdArgs a) {
    const int i = ((int)blockIdx.x * 256 + (int)threadIdx.x) * 8, H = a.H;
    if (i >= H) return;
    f32x8 aw = {0, 0, 0, 0, 0, 0, 0, 0}, ab = aw;
    for (int64_t t = (int64_t)blockIdx.y; t < a.T; t += gridDim.y) {
        const float mean = a.mean[t], rstd = a.rstd[t];
        const f32x8 d = load8<VEC>(a.dy + t * a.lddy, false, i, H);
        const f32x8 n = load8<VEC>((const char*)a.s + t * a.lds * (S32 ? 4 : 2), S32, i, H);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            aw[e] = fmaf(d[e], (n[e] - mean) * rstd, aw[e]);
            ab[e] += d[e];
        }
    }
    float* p = a.partial + (int64_t)blockIdx.y * 2 * H;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        if (!VEC && i + e >= H) continue;
        p[i + e] = aw[e];
        p[H + i + e] = ab[e];
    }
}

// 32 columns of 32 runs of parts; the runs' sums meet in LDS.
__global__ __launch_bounds__(1024) void join_columns_kernel(const float* __restrict__ partial, int parts, int cols, int first,
                                                            void* __restrict__ out0, void* __restrict__ out1, int f32) {
    __shared__ float sum[32][33];
    const int x = (int)threadIdx.x & 31, y = (int)threadIdx.x >> 5;
    const int c = (int)blockIdx.x * 32 + x;
    float v = 0.0f;
    if (c < cols)
        for (int p = y; p < parts; p += 32) v += partial[(int64_t)p * cols + c];
    sum[y][x] = v;
    __syncthreads();
    if (y != 0 || c >= cols) return;
    v = 0.0f;
#pragma unroll
    for (int k = 0; k < 32; ++k) v += sum[k][x];
    void* out = c < first ? out0 : out1;
    const int at = c < first ? c : c - first;
    if (!out) return;
    if (f32) ((float*)out)[at] = v;
    else ((uint16_t*)out)[at] = f32_to_bf16_bits(v);
}

hipError_t launch_join_columns(const float* partial, int parts, int cols, int first, void* out0, void* out1, bool f32,
                               hipStream_t s) {
    hipLaunchKernelGGL(join_columns_kernel, dim3((unsigned)((cols + 31) / 32)), dim3(1024), 0, s, partial, parts, cols, first,
                       out0, out1, f32 ? 1 : 0);
    return hipGetLastError();
}

constexpr int kHeldColumns = 16384;  // of a row in registers, with the sums of its columns

int layer_norm_parts(int T, int H) {
    const int rows = H <= 512 ? 4 : 1;
    const int64_t groups = ((int64_t)T + rows - 1) / rows;
    const int most = H <= kHeldColumns ? 1024 : 64;
    return (int)(groups < most ? groups : most);
}

template <int WAVES, int NC>
static void launch_bwd(const LayerNormBwdArgs& a, bool vec, hipStream_t s) {
    const dim3 grid((unsigned)layer_norm_parts(a.T, a.H)), block(WAVES == 1 ? 256 : WAVES * 64);
    if (a.s_f32) {
        if (vec) hipLaunchKernelGGL((layer_norm_bwd_kernel<WAVES, NC, true, true>), grid, block, 0, s, a);
        else hipLaunchKernelGGL((layer_norm_bwd_kernel<WAVES, NC, false, true>), grid, block, 0, s, a);
    } else {
        if (vec) hipLaunchKernelGGL((layer_norm_bwd_kernel<WAVES, NC, true, false>), grid, block, 0, s, a);
        else hipLaunchKernelGGL((layer_norm_bwd_kernel<WAVES, NC, false, false>), grid, block, 0, s, a);
    }
}

template <bool VEC, bool S32>
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
            hipLaunchKernelGGL((layer_norm_bwd_long_kernel<VEC, S32>), dim3((unsigned)b.T), dim3(1024), 0, s, b);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
    }
    if (a.partial) {
        const dim3 grid((unsigned)((a.H + 2047) / 2048), (unsigned)layer_norm_parts(a.T, a.H));
        hipLaunchKernelGGL((layer_norm_columns_kernel<VEC, S32>), grid, dim3(256), 0, s, a);
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
        else if (a.H <= 2048) launch_bwd<4, 1>(a, vec, s);
        else if (a.H <= 4096) launch_bwd<4, 2>(a, vec, s);
        else if (a.H <= 8192) launch_bwd<8, 2>(a, vec, s);
        else if (a.H <= kHeldColumns) launch_bwd<16, 2>(a, vec, s);
        else if (a.s_f32) e = vec ? launch_long<true, true>(a, s) : launch_long<false, true>(a, s);
        else e = vec ? launch_long<true, false>(a, s) : launch_long<false, false>(a, s);
        if (e == hipSuccess) e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (!sums) return hipSuccess;
    return launch_join_columns(a.partial, a.T > 0 ? layer_norm_parts(a.T, a.H) : 0, 2 * a.H, a.H, a.dweight, a.dbias,
                               a.weight_f32, s);
}

}  // namespace moe
