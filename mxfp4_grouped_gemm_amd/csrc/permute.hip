// Token rows sorted by expert, and back to tokens:
//   permute:   pairs p = t topk + j sorted by (expert, p); out[row(p)] = x[t];
//   unpermute: out[t] = residual[t] + sum over j of weight[t, j] y[row(t, j)];
//   its gradients: dy[row(t, j)] = weight[t, j] dout[t],
//                  dweight[t, j] = <dout[t], y[row(t, j)]>.
// Pairs whose expert is outside [0, E) come last, as rows of zeros; their
// entry of `rows` is -1 - row, and they add nothing.
//
// All of them are bound by the rows' bytes. A row is moved by whole waves in
// 16-byte pieces at any element address.
#include "common.hpp"
#include "row_io.hpp"
#include "train.hpp"

namespace moe {

using namespace rows;

namespace {

typedef u32x4 __attribute__((aligned(1))) u32x4_byte;
typedef u32x2 __attribute__((aligned(1))) u32x2_byte;
typedef uint32_t __attribute__((aligned(1))) u32_byte;
typedef uint16_t __attribute__((aligned(1))) u16_byte;

constexpr int kMaxTopk = 64;
// Up to this many pairs each workgroup counts the pairs before its own.
constexpr int kFewPairs = 2048;
constexpr int kSlice = 1024;      // pairs ranked at once
constexpr int kMostChunks = 256;  // of slices; the scan takes them in one workgroup
constexpr int kKeys = 1025;       // experts, and none

__host__ __device__ __forceinline__ int64_t slices_a_chunk(int64_t pairs) {
    const int64_t slices = (pairs + kSlice - 1) / kSlice;
    return (slices + kMostChunks - 1) / kMostChunks;
}
__host__ __device__ __forceinline__ int chunks_of(int64_t pairs) {
    const int64_t per = slices_a_chunk(pairs) * kSlice;
    return (int)((pairs + per - 1) / per);
}

__device__ __forceinline__ int key_of(int id, int E) { return (unsigned)id < (unsigned)E ? id : E; }

// Bytes [16 i, 16 i + 16) of a row of n bytes, at any address.
__device__ __forceinline__ u32x4 load_piece(const char* row, int64_t at, int64_t n) {
    u32x4 v = {0, 0, 0, 0};
    if (at + 16 <= n) return *(const u32x4_byte*)(row + at);
    const int left = (int)(n - at);
    int o = 0;
    if (left & 8) {
        const u32x2 d = *(const u32x2_byte*)(row + at);
        v[0] = d[0];
        v[1] = d[1];
        o = 8;
    }
    if (left & 4) {
        const uint32_t d = *(const u32_byte*)(row + at + o);
        if (o) v[2] = d;
        else v[0] = d;
        o += 4;
    }
    uint32_t tail = 0;
    const int word = o / 4;
    if (left & 2) {
        tail = *(const u16_byte*)(row + at + o);
        o += 2;
    }
    if (left & 1) tail |= (uint32_t) * (const uint8_t*)(row + at + o) << (left & 2 ? 16 : 0);
    if (left & 3) {
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = k == word ? tail : v[k];
    }
    return v;
}

__device__ __forceinline__ void store_piece(char* row, int64_t at, int64_t n, u32x4 v) {
    if (at + 16 <= n) {
        *(u32x4_byte*)(row + at) = v;
        return;
    }
    const int left = (int)(n - at);
    int o = 0;
    if (left & 8) {
        *(u32x2_byte*)(row + at) = u32x2{v[0], v[1]};
        o = 8;
    }
    if (left & 4) {
        *(u32_byte*)(row + at + o) = o ? v[2] : v[0];
        o += 4;
    }
    uint32_t tail = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) tail = k == o / 4 ? v[k] : tail;
    if (left & 2) {
        *(u16_byte*)(row + at + o) = (uint16_t)tail;
        tail >>= 16;
        o += 2;
    }
    if (left & 1) *(uint8_t*)(row + at + o) = (uint8_t)tail;
}

// Copies one token's row to the rows of its pairs (place < 0: zeros to -1 -
// place), with all threads of the workgroup.
__device__ __forceinline__ void copy_rows(const PermuteArgs& a, int64_t t, const int* place) {
    const char* xr = (const char*)a.x + t * a.ldx;
    for (int64_t at = (int64_t)threadIdx.x * 16; at < a.row_bytes; at += (int64_t)blockDim.x * 16) {
        const u32x4 v = load_piece(xr, at, a.row_bytes);
        for (int j = 0; j < a.topk; ++j) {
            const int r = place[j];
            const int64_t row = r < 0 ? -1 - (int64_t)r : r;
            store_piece((char*)a.out + row * a.ldo, at, a.row_bytes, r < 0 ? u32x4{0, 0, 0, 0} : v);
        }
    }
}

// Few pairs: a workgroup a token counts the pairs before each of its own (a
// wave a pair); the last workgroup counts the experts' rows.
__global__ __launch_bounds__(256) void permute_few_kernel(PermuteArgs a) {
    __shared__ int place[kMaxTopk];
    const int tid = (int)threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int P = a.T * a.topk, E = a.E;
    if ((int)blockIdx.x == a.T) {
        __shared__ int count[kKeys];
        __shared__ int total[4];
        for (int k = tid; k <= E; k += 256) count[k] = 0;
        __syncthreads();
        for (int p = tid; p < P; p += 256) atomicAdd(&count[key_of(a.ids[p], E)], 1);
        __syncthreads();
        // Four keys a thread.
        int c[4], sum = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            c[i] = tid * 4 + i < E ? count[tid * 4 + i] : 0;
            sum += c[i];
        }
        int upto = sum;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const int o = __shfl_up(upto, d);
            if (lane >= d) upto += o;
        }
        if (lane == 63) total[w] = upto;
        __syncthreads();
        int base = upto - sum;
        for (int k = 0; k < w; ++k) base += total[k];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (tid * 4 + i < E) a.offsets[tid * 4 + i] = base;
            base += c[i];
        }
        if (tid == 255) a.offsets[E] = base;
        return;
    }
    const int t = (int)blockIdx.x;
    for (int j = w; j < a.topk; j += 4) {
        const int p = t * a.topk + j, key = key_of(a.ids[p], E);
        int before = 0;
        for (int q = lane; q < P + lane; q += 64) {  // (whole waves)
            const int k = q < P ? key_of(a.ids[q], E) : E + 1;
            before += __popcll(__ballot(k < key || (k == key && q < p)));
        }
        if (lane == 0) place[j] = key < E ? before : -1 - before;
    }
    __syncthreads();
    if (tid < a.topk) a.rows[(int64_t)t * a.topk + tid] = place[tid];
    copy_rows(a, t, place);
}

// The rank of each pair among those of its expert in its chunk (into `rows`),
// and the chunk's counts. A wave ranks 64 pairs by comparing the bits of their
// keys; the waves of a slice and the slices meet in LDS, in order.
__global__ __launch_bounds__(1024) void permute_rank_kernel(PermuteArgs a) {
    __shared__ uint16_t count[16][kKeys + 1];
    __shared__ int base[kKeys];
    const int tid = (int)threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t P = (int64_t)a.T * a.topk;
    const int E = a.E, bits = 32 - __builtin_clz(E);
    const int64_t per = slices_a_chunk(P) * kSlice, beg = (int64_t)blockIdx.x * per, end = beg + per < P ? beg + per : P;
    for (int k = tid; k <= E; k += 1024) base[k] = 0;
    for (int64_t p0 = beg; p0 < end; p0 += kSlice) {
        for (int k = lane; k <= E; k += 64) count[w][k] = 0;
        const int64_t p = p0 + tid;
        const bool ok = p < end;
        const int key = ok ? key_of(a.ids[p], E) : 0;
        uint64_t same = __ballot(ok);
        for (int b = 0; b < bits; ++b) {
            const uint64_t one = __ballot(key >> b & 1);
            same &= key >> b & 1 ? one : ~one;
        }
        const int rank = __popcll(same & ((1ull << lane) - 1));
        wave_lds_sync();
        if (ok && rank == 0) count[w][key] = (uint16_t)__popcll(same);
        __syncthreads();
        for (int k = tid; k <= E; k += 1024) {
            int sum = 0;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int c = count[i][k];
                count[i][k] = (uint16_t)sum;
                sum += c;
            }
            // Read below by others before the next slice's addition.
            count[0][k] = (uint16_t)sum;
        }
        __syncthreads();
        if (ok) a.rows[p] = base[key] + (w ? count[w][key] : 0) + rank;
        __syncthreads();
        for (int k = tid; k <= E; k += 1024) base[k] += count[0][k];
        __syncthreads();
    }
    int32_t* out = a.counts + (int64_t)blockIdx.x * (E + 1);
    for (int k = tid; k <= E; k += 1024) out[k] = base[k];
}

// counts [chunks, E + 1] -> the first row of each chunk's pairs of a key; the
// experts' offsets. One workgroup: `parts` runs of chunks for each key.
__global__ __launch_bounds__(1024) void permute_scan_kernel(PermuteArgs a, int chunks) {
    __shared__ int sum[1024 + 64];
    __shared__ int start[kKeys];
    __shared__ int total[16];
    const int tid = (int)threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int n = a.E + 1;
    int width = 64;
    while (width < n && width < 1024) width *= 2;  // keys at a time
    const int parts = 1024 / width, part = tid / width, per = (chunks + parts - 1) / parts;
    const int beg = part * per < chunks ? part * per : chunks, end = beg + per < chunks ? beg + per : chunks;
    for (int k0 = 0; k0 < n; k0 += width) {
        const int k = k0 + tid % width;
        int s = 0;
        if (k < n)
            for (int c = beg; c < end; ++c) s += a.counts[(int64_t)c * n + k];
        sum[tid] = s;
        __syncthreads();
        if (tid < width && k < n) {
            int v = 0;
            for (int i = 0; i < parts; ++i) {
                const int c = sum[i * width + tid];
                sum[i * width + tid] = v;
                v += c;
            }
            start[k] = v;
        }
        __syncthreads();
        if (k < n) {
            int v = sum[tid];
            for (int c = beg; c < end; ++c) {
                int32_t* p = a.counts + (int64_t)c * n + k;
                const int d = *p;
                *p = v;
                v += d;
            }
        }
        __syncthreads();
    }
    // start: the keys' totals -> their offsets (key E: after the 1024 at most
    // before it).
    const int mine = tid < a.E ? start[tid] : 0;
    int upto = mine;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int o = __shfl_up(upto, d);
        if (lane >= d) upto += o;
    }
    if (lane == 63) total[w] = upto;
    __syncthreads();
    for (int i = 0; i < w; ++i) upto += total[i];
    if (tid < a.E) a.offsets[tid] = upto - mine;
    if (tid == 1023) a.offsets[a.E] = upto;
}

// A workgroup a token.
__global__ __launch_bounds__(256) void permute_rows_kernel(PermuteArgs a) {
    __shared__ int place[kMaxTopk];
    const int64_t t = (int64_t)blockIdx.x, P = (int64_t)a.T * a.topk;
    const int tid = (int)threadIdx.x;
    if (tid < a.topk) {
        const int64_t p = t * a.topk + tid;
        const int key = key_of(a.ids[p], a.E);
        const int chunk = (int)(p / (slices_a_chunk(P) * kSlice));
        const int row = a.rows[p] + a.counts[(int64_t)chunk * (a.E + 1) + key] + a.offsets[key];
        place[tid] = key < a.E ? row : -1 - row;
        a.rows[p] = place[tid];
    }
    __syncthreads();
    copy_rows(a, t, place);
}

__global__ __launch_bounds__(256) void clear_kernel(int32_t* p, int n) {
    const int i = (int)(blockIdx.x * 256 + threadIdx.x);
    if (i < n) p[i] = 0;
}

}  // namespace

int64_t permute_workspace_bytes(int64_t pairs, int E) {
    return pairs <= kFewPairs ? 0 : ((int64_t)chunks_of(pairs) * (E + 1) * 4 + 255) / 256 * 256;
}

hipError_t launch_permute(const PermuteArgs& a, hipStream_t s) {
    const int64_t P = (int64_t)a.T * a.topk;
    if (P == 0) {
        hipLaunchKernelGGL(clear_kernel, dim3((unsigned)((a.E + 256) / 256)), dim3(256), 0, s, a.offsets, a.E + 1);
        return hipGetLastError();
    }
    if (P <= kFewPairs) {
        hipLaunchKernelGGL(permute_few_kernel, dim3((unsigned)a.T + 1), dim3(256), 0, s, a);
        return hipGetLastError();
    }
    const int chunks = chunks_of(P);
    hipLaunchKernelGGL(permute_rank_kernel, dim3((unsigned)chunks), dim3(1024), 0, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(permute_scan_kernel, dim3(1), dim3(1024), 0, s, a, chunks);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(permute_rows_kernel, dim3((unsigned)a.T), dim3(256), 0, s, a);
    return hipGetLastError();
}

// ------------------------------------------------------------- unpermute
// A lane eight columns of a token; its rows are fetched KB at a time.
template <int KB, bool VEC>
__global__ __launch_bounds__(256) void unpermute_kernel(UnpermuteArgs a, int pieces) {
    const int64_t idx = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t t = idx / pieces;
    if (t >= a.T) return;
    const int i = (int)(idx % pieces) * 8, H = a.H;
    const int64_t P = a.pairs;
    const int32_t* rw = a.rows + t * a.topk;
    const float* wt = a.weights + t * a.topk;
    f32x8 acc = {0, 0, 0, 0, 0, 0, 0, 0};
    for (int j0 = 0; j0 < a.topk; j0 += KB) {
        int r[KB];
        float w[KB];
        f32x8 v[KB];
#pragma unroll
        for (int j = 0; j < KB; ++j) {
            r[j] = j0 + j < a.topk ? rw[j0 + j] : -1;
            w[j] = a.weights && j0 + j < a.topk ? wt[j0 + j] : 1.0f;
        }
#pragma unroll
        for (int j = 0; j < KB; ++j) {
            v[j] = f32x8{0, 0, 0, 0, 0, 0, 0, 0};
            if (r[j] >= 0 && r[j] < P) v[j] = load8<VEC>((const char*)a.y + r[j] * a.ldy * (a.y_f32 ? 4 : 2), a.y_f32, i, H);
            else w[j] = 0.0f;  // (nothing, whatever its weight)
        }
#pragma unroll
        for (int j = 0; j < KB; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] = fmaf(w[j], v[j][e], acc[e]);
    }
    if (a.residual) acc += load8<VEC>((const char*)a.residual + t * a.ldr * (a.out_f32 ? 4 : 2), a.out_f32, i, H);
    store8<VEC>((char*)a.out + t * a.ldo * (a.out_f32 ? 4 : 2), a.out_f32, i, H, acc);
}

static bool wide(const void* p, int64_t ld, int bytes) {
    return p == nullptr || ((uintptr_t)p % 16 == 0 && (ld * bytes) % 16 == 0);
}

template <bool VEC>
static void launch_unpermute_kb(const UnpermuteArgs& a, hipStream_t s) {
    const int pieces = (a.H + 7) / 8;
    const dim3 grid((unsigned)(((int64_t)a.T * pieces + 255) / 256)), block(256);
    if (a.topk <= 2) hipLaunchKernelGGL((unpermute_kernel<2, VEC>), grid, block, 0, s, a, pieces);
    else if (a.topk <= 4) hipLaunchKernelGGL((unpermute_kernel<4, VEC>), grid, block, 0, s, a, pieces);
    else hipLaunchKernelGGL((unpermute_kernel<8, VEC>), grid, block, 0, s, a, pieces);
}

hipError_t launch_unpermute(const UnpermuteArgs& a, hipStream_t s) {
    const int yb = a.y_f32 ? 4 : 2, ob = a.out_f32 ? 4 : 2;
    const bool vec = a.H % 8 == 0 && wide(a.y, a.ldy, yb) && wide(a.residual, a.ldr, ob) && wide(a.out, a.ldo, ob);
    // A launch holds fewer than 2^32 threads.
    const int64_t most = ((int64_t)1 << 31) / ((a.H + 7) / 8);
    for (int64_t t = 0; t < a.T; t += most) {
        UnpermuteArgs b = a;
        b.T = (int)(a.T - t < most ? a.T - t : most);
        b.rows = a.rows + t * a.topk;
        if (a.weights) b.weights = a.weights + t * a.topk;
        if (a.residual) b.residual = (const char*)a.residual + t * a.ldr * ob;
        b.out = (char*)a.out + t * a.ldo * ob;
        if (vec) launch_unpermute_kb<true>(b, s);
        else launch_unpermute_kb<false>(b, s);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

// A workgroup a token: eight pairs at a time, their rows of y and dy by the
// token's row of dout; the dot products meet in LDS.
template <bool VEC>
__global__ __launch_bounds__(256) void unpermute_bwd_kernel(UnpermuteBwdArgs a) {
    constexpr int KB = 8;
    __shared__ float part[4][KB];
    const int tid = (int)threadIdx.x, H = a.H, w = tid >> 6;
    const int64_t t = (int64_t)blockIdx.x, P = (int64_t)a.T * a.topk;
    const char* dr = (const char*)a.dout + t * a.lddo * (a.out_f32 ? 4 : 2);
    for (int j0 = 0; j0 < a.topk; j0 += KB) {
        int r[KB];
        float wt[KB], dot[KB];
#pragma unroll
        for (int j = 0; j < KB; ++j) {
            r[j] = j0 + j < a.topk ? a.rows[t * a.topk + j0 + j] : 0;
            wt[j] = a.weights && j0 + j < a.topk ? a.weights[t * a.topk + j0 + j] : 1.0f;
            dot[j] = 0.0f;
        }
        for (int i = tid * 8; i < H; i += 2048) {
            const f32x8 d = load8<VEC>(dr, a.out_f32, i, H);
#pragma unroll
            for (int j = 0; j < KB; ++j) {
                if (j0 + j >= a.topk) continue;
                const int64_t row = r[j] < 0 ? -1 - (int64_t)r[j] : r[j];
                if (row >= P) continue;
                if (a.dweights && r[j] >= 0) {
                    const f32x8 y = load8<VEC>((const char*)a.y + row * a.ldy * (a.y_f32 ? 4 : 2), a.y_f32, i, H);
#pragma unroll
                    for (int e = 0; e < 8; ++e) dot[j] = fmaf(d[e], y[e], dot[j]);
                }
                if (a.dy) {
                    f32x8 v;
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] = r[j] < 0 ? 0.0f : wt[j] * d[e];
                    store8<VEC>((char*)a.dy + row * a.lddy * (a.y_f32 ? 4 : 2), a.y_f32, i, H, v);
                }
            }
        }
        if (a.dweights) {
#pragma unroll
            for (int j = 0; j < KB; ++j) {
                const float v = wave_sum(dot[j]);
                if ((tid & 63) == 0) part[w][j] = v;
            }
            __syncthreads();
            if (tid < KB && j0 + tid < a.topk)
                a.dweights[t * a.topk + j0 + tid] = (part[0][tid] + part[1][tid]) + (part[2][tid] + part[3][tid]);
            __syncthreads();
        }
    }
}

hipError_t launch_unpermute_bwd(const UnpermuteBwdArgs& a, hipStream_t s) {
    const int yb = a.y_f32 ? 4 : 2, ob = a.out_f32 ? 4 : 2;
    const bool vec = a.H % 8 == 0 && wide(a.dout, a.lddo, ob) && wide(a.y, a.ldy, yb) && wide(a.dy, a.lddy, yb);
    const dim3 grid((unsigned)a.T), block(256);
    if (vec) hipLaunchKernelGGL((unpermute_bwd_kernel<true>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((unpermute_bwd_kernel<false>), grid, block, 0, s, a);
    return hipGetLastError();
}

}  // namespace moe
