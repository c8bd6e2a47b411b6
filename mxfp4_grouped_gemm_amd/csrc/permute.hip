// Token rows sorted by expert, and back to tokens:
//   permute:   pairs p = t topk + j sorted by (expert, p); out[row(p)] = x[t];
//   unpermute: out[t] = residual[t] + sum over j of weight[t, j] y[row(t, j)];
//   its gradients: dy[row(t, j)] = weight[t, j] dout[t],
//                  dweight[t, j] = <dout[t], y[row(t, j)]>.
// Pairs whose expert is outside [0, E) come last, as rows of zeros; their
// entry of `rows` is -1 - row, and they add nothing.
//
// All of them are bound by the rows' bytes. A row is moved by whole waves in
// 16-byte pieces at any element address. Rows of 3584: 8192 x 8 pairs of 896 experts
// 96 us (5.5 TB/s) after 10 us of sort; back from 8192 x 15 with an fp32 residual
// 203 us (5.5 TB/s); gradients of 4099 x 4 rows of 2784 42 us (5.0 TB/s).
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
// Up to so many pairs each wave counts the pairs before its own: one launch, but
// the counting grows with their square, and the three launches copy wide rows
// faster (8 choices of 112 experts, one launch and three: rows of 3584, 2400 pairs
// 13.4 us and 18.8, 4096 pairs 26.4 and 18.6; rows of 1024, 4000 pairs 14.3 and
// 18.4, 6400 pairs 24.5 and 18.3).
constexpr int kFewPairs = 2560, kFewNarrowPairs = 4096;
constexpr int64_t kNarrowRow = 2048;  // bytes
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

// Few pairs: a wave a pair counts the pairs before it, and copies the row; the
// last workgroup counts the experts' rows. One launch, the latency of one
// memory round trip after the other.
__global__ __launch_bounds__(256) void permute_few_kernel(PermuteArgs a) {
    const int tid = (int)threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int P = a.T * a.topk, E = a.E;
    if ((int)blockIdx.x == (P + 3) / 4) {
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
    const int p = (int)blockIdx.x * 4 + w;
    if (p >= P) return;  // (no barrier follows)
    const char* xr = (const char*)a.x + p / a.topk * a.ldx;
    constexpr int kBatch = 8;  // pieces of the row, and slices of the ids, in flight
    const int64_t at0 = lane * 16;
    u32x4 v[kBatch];
    auto load = [&](int64_t at) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
            if (at + i * 1024 < a.row_bytes) v[i] = load_piece(xr, at + i * 1024, a.row_bytes);
    };
    load(at0);
    const int key = __builtin_amdgcn_readfirstlane(key_of(a.ids[p], E));
    int before = 0;
    for (int q0 = 0; q0 < P; q0 += 64 * kBatch) {
        int k[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int q = q0 + 64 * i + lane;
            k[i] = q < P ? key_of(a.ids[q], E) : E + 1;
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
            before += __popcll(__ballot(k[i] < key || (k[i] == key && q0 + 64 * i + lane < p)));
    }
    if (lane == 0) a.rows[p] = key < E ? before : -1 - before;
    char* out = (char*)a.out + before * a.ldo;
    for (int64_t at = at0;;) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
            if (at + i * 1024 < a.row_bytes) store_piece(out, at + i * 1024, a.row_bytes, key < E ? v[i] : u32x4{0, 0, 0, 0});
        at += kBatch * 1024;
        if (at >= a.row_bytes) break;  // (whole waves or the row's end)
        load(at);
    }
}

// The rank of each pair among those of its expert in its chunk (into `rows`),
// and the chunk's counts. 65536 pairs of 897 keys: 5.2 us. A wave ranks 64 pairs by comparing the bits of their
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
    // Sums of 64 keys each (key 1024 is in none).
    int sum = tid <= E ? base[tid] : 0;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) sum += __shfl_xor(sum, d);
    if (lane == 0) a.counts[(int64_t)gridDim.x * 2 * (E + 1) + (int64_t)blockIdx.x * 16 + w] = sum;
}

// counts [chunks, E + 1] -> the first row of each chunk's pairs of a key (behind
// counts), and the experts' offsets. A workgroup 64 keys: a wave takes a run of
// chunks; the keys below the workgroup's are summed by each workgroup itself,
// from the chunks' sums of 64 keys, so that one launch needs no order among
// workgroups (64 chunks of 897 keys: 5.0 us; without those sums 10.5; all keys
// in one workgroup, chunk after chunk, 27).
__global__ __launch_bounds__(1024) void permute_scan_kernel(PermuteArgs a, int chunks) {
    constexpr int kRun = kMostChunks / 16;
    __shared__ int sums[16][64];
    __shared__ int below[16];
    const int tid = (int)threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n = a.E + 1, k0 = (int)blockIdx.x * 64, k = k0 + lane;
    const int per = (chunks + 15) / 16, c0 = w * per;
    int v[kRun], sum = 0;
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
        v[i] = i < per && c0 + i < chunks && k < n ? a.counts[(int64_t)(c0 + i) * n + k] : 0;
        sum += v[i];
    }
    // (Four chunks of 16 sums a wave.)
    const int32_t* groups = a.counts + (int64_t)chunks * 2 * n;
    int low = 0;
#pragma unroll
    for (int i = 0; i < kMostChunks / 64; ++i) {
        const int c = 64 * i + 4 * w + lane / 16;
        low += c < chunks && lane % 16 < (int)blockIdx.x ? groups[c * 16 + lane % 16] : 0;
    }
#pragma unroll
    for (int d = 1; d < 64; d *= 2) low += __shfl_xor(low, d);
    sums[w][lane] = sum;
    if (lane == 0) below[w] = low;
    __syncthreads();
    int base = 0, mine = 0, total = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int s = sums[i][lane];
        mine += i < w ? s : 0;
        total += s;
        base += below[i];
    }
    int upto = total;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int o = __shfl_up(upto, d);
        if (lane >= d) upto += o;
    }
    base += upto - total;
    if (k >= n) return;
    if (w == 0) a.offsets[k] = base;  // (of key E: the end of the experts' rows)
    base += mine;
    int32_t* out = a.counts + (int64_t)chunks * n;
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
        if (i < per && c0 + i < chunks) out[(int64_t)(c0 + i) * n + k] = base;
        base += v[i];
    }
}

// The rows themselves: a workgroup takes `group` tokens, finds the places of
// their pairs and then copies, a thread a piece of a row. ONE: a token a
// workgroup, whose places are the same in all lanes.
constexpr int kGroupPairs = 1024;  // places a workgroup holds

template <bool ONE>
__global__ __launch_bounds__(256) void permute_rows_kernel(PermuteArgs a, int group, int pieces, int chunks) {
    __shared__ int place[ONE ? kMaxTopk : kGroupPairs];
    const int64_t t0 = (int64_t)blockIdx.x * group, P = (int64_t)a.T * a.topk;
    const int tid = (int)threadIdx.x;
    const int tokens = a.T - t0 < group ? (int)(a.T - t0) : group, pairs = tokens * a.topk, all = tokens * pieces;
    auto at_of = [&](int q) { return (int64_t)(ONE ? q : q % pieces) * 16; };
    auto load = [&](int q) {
        return load_piece((const char*)a.x + (t0 + (ONE ? 0 : q / pieces)) * a.ldx, at_of(q), a.row_bytes);
    };
    u32x4 v = {0, 0, 0, 0};
    if (tid < all) v = load(tid);  // on its way meanwhile
    const int64_t chunk_pairs = slices_a_chunk(P) * kSlice;
    const int32_t* first = a.counts + (int64_t)chunks * (a.E + 1);
    for (int i = tid; i < pairs; i += 256) {
        const int64_t p = t0 * a.topk + i;
        const int key = key_of(a.ids[p], a.E);
        const int row = a.rows[p] + first[p / chunk_pairs * (a.E + 1) + key];
        place[i] = key < a.E ? row : -1 - row;
        a.rows[p] = place[i];
    }
    __syncthreads();
    for (int q = tid; q < all;) {
        const int64_t at = at_of(q);
        const int* pl = place + (ONE ? 0 : q / pieces * a.topk);
        for (int j = 0; j < a.topk; ++j) {
            const int r = ONE ? __builtin_amdgcn_readfirstlane(pl[j]) : pl[j];
            const int64_t row = r < 0 ? -1 - (int64_t)r : r;
            store_piece((char*)a.out + row * a.ldo, at, a.row_bytes, r < 0 ? u32x4{0, 0, 0, 0} : v);
        }
        q += 256;
        if (q < all) v = load(q);
    }
}

__global__ __launch_bounds__(256) void clear_kernel(int32_t* p, int n) {
    const int i = (int)(blockIdx.x * 256 + threadIdx.x);
    if (i < n) p[i] = 0;
}

}  // namespace

static int64_t chunk_bytes(int64_t chunks, int E) { return (chunks * ((E + 1) * 2 + 16) * 4 + 255) / 256 * 256; }

int64_t permute_workspace_bytes(int64_t pairs, int E) {
    return pairs <= kFewPairs ? 0 : chunk_bytes(chunks_of(pairs), E);
}

// (Chunks of one slice up to the most there are, then fewer of several.)
int64_t permute_most_workspace_bytes(int64_t pairs, int E) {
    const int64_t slices = (pairs + kSlice - 1) / kSlice;
    return pairs <= kFewPairs ? 0 : chunk_bytes(slices < kMostChunks ? slices : kMostChunks, E);
}

hipError_t launch_permute(const PermuteArgs& a, hipStream_t s) {
    const int64_t P = (int64_t)a.T * a.topk;
    if (P == 0) {
        hipLaunchKernelGGL(clear_kernel, dim3((unsigned)((a.E + 256) / 256)), dim3(256), 0, s, a.offsets, a.E + 1);
        return hipGetLastError();
    }
    if (P <= kFewPairs || (P <= kFewNarrowPairs && a.row_bytes <= kNarrowRow)) {
        hipLaunchKernelGGL(permute_few_kernel, dim3((unsigned)(P + 3) / 4 + 1), dim3(256), 0, s, a);
        return hipGetLastError();
    }
    const int chunks = chunks_of(P);
    hipLaunchKernelGGL(permute_rank_kernel, dim3((unsigned)chunks), dim3(1024), 0, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(permute_scan_kernel, dim3((unsigned)(a.E + 64) / 64), dim3(1024), 0, s, a, chunks);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    // Rows of 128 pieces and more keep half of a workgroup's threads busy.
    const int pieces = (int)((a.row_bytes + 15) / 16);
    if (pieces >= 128) {
        hipLaunchKernelGGL(permute_rows_kernel<true>, dim3((unsigned)a.T), dim3(256), 0, s, a, 1, pieces, chunks);
    } else {
        int group = 512 / pieces;
        if (group > kGroupPairs / a.topk) group = kGroupPairs / a.topk;
        hipLaunchKernelGGL(permute_rows_kernel<false>, dim3((unsigned)((a.T + group - 1) / group)), dim3(256), 0, s, a, group,
                           pieces, chunks);
    }
    return hipGetLastError();
}

// ------------------------------------------------------------- unpermute
static bool wide(const void* p, int64_t ld, int bytes) {
    return p == nullptr || ((uintptr_t)p % 16 == 0 && (ld * bytes) % 16 == 0);
}

// A pair's row, or row 0 (loaded and not used) for one that adds nothing: no
// branch stands between the loads of a token's rows.
__device__ __forceinline__ int64_t safe_row(int r, int64_t P) { return r >= 0 && r < P ? r : 0; }

// A lane eight columns of a token, whose rows are fetched KB at a time. ONE: a
// workgroup a token, so rows and weights are scalars. (8192 x 15 rows of 3584: 203
// us; with a branch around each load and rows in vector registers 230.)
template <int KB, int MODE, bool ONE, bool Y32>
__global__ __launch_bounds__(512) void unpermute_kernel(UnpermuteArgs a, int pieces) {
    const int64_t idx = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int64_t t = ONE ? (int64_t)blockIdx.x : idx / pieces;
    if (t >= a.T) return;
    const int H = a.H;
    const int64_t P = a.pairs;
    const int32_t* rw = a.rows + t * a.topk;
    const float* wt = a.weights + t * a.topk;
    for (int q = ONE ? (int)threadIdx.x : (int)(idx % pieces); q < pieces; q += ONE ? (int)blockDim.x : pieces) {
        const int i = q * 8;
        f32x8 acc = {0, 0, 0, 0, 0, 0, 0, 0};
        Raw8 res;
        if (a.residual) res = fetch8<MODE>((const char*)a.residual + t * a.ldr * (a.out_f32 ? 4 : 2), a.out_f32, i, H);
        for (int j0 = 0; j0 < a.topk; j0 += KB) {
            int r[KB];
            float w[KB];
            Raw8 f[KB];
#pragma unroll
            for (int j = 0; j < KB; ++j) {
                const int k = j0 + j < a.topk ? j0 + j : a.topk - 1;
                r[j] = ONE ? __builtin_amdgcn_readfirstlane(rw[k]) : rw[k];
                w[j] = a.weights ? wt[k] : 1.0f;
                r[j] = j0 + j < a.topk ? r[j] : -1;
            }
#pragma unroll
            for (int j = 0; j < KB; ++j)
                f[j] = fetch8<MODE>((const char*)a.y + safe_row(r[j], P) * a.ldy * (Y32 ? 4 : 2), Y32, i, H);
#pragma unroll
            for (int j = 0; j < KB; ++j) {
                // (Nothing, whatever its weight and row 0 hold.)
                const bool ok = r[j] >= 0 && r[j] < P;
                const f32x8 v = widen8<MODE>(f[j], Y32, i, H);
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[e] = ok ? fmaf(w[j], v[e], acc[e]) : acc[e];
            }
        }
        if (a.residual) acc += widen8<MODE>(res, a.out_f32, i, H);
        put8<MODE>((char*)a.out + t * a.ldo * (a.out_f32 ? 4 : 2), a.out_f32, i, H, acc);
    }
}

// Threads of a workgroup that takes a row of so many pieces: whole waves, 512 at
// most, in even rounds.
static int row_threads(int pieces) {
    const int rounds = (pieces + 511) / 512;
    return ((pieces + rounds - 1) / rounds + 63) / 64 * 64;
}

template <int KB, int MODE, bool Y32>
static void launch_unpermute_as(const UnpermuteArgs& a, hipStream_t s) {
    const int pieces = (a.H + 7) / 8;
    if (pieces >= 64)
        hipLaunchKernelGGL((unpermute_kernel<KB, MODE, true, Y32>), dim3((unsigned)a.T), dim3(row_threads(pieces)), 0, s, a, pieces);
    else
        hipLaunchKernelGGL((unpermute_kernel<KB, MODE, false, Y32>), dim3((unsigned)(((int64_t)a.T * pieces + 255) / 256)), dim3(256),
                           0, s, a, pieces);
}

template <int MODE, bool Y32>
static void launch_unpermute_kb(const UnpermuteArgs& a, hipStream_t s) {
    if (a.topk <= 2) launch_unpermute_as<2, MODE, Y32>(a, s);
    else if (a.topk <= 4) launch_unpermute_as<4, MODE, Y32>(a, s);
    else launch_unpermute_as<8, MODE, Y32>(a, s);
}

template <int MODE>
static void launch_unpermute_type(const UnpermuteArgs& a, hipStream_t s) {
    if (a.y_f32) launch_unpermute_kb<MODE, true>(a, s);
    else launch_unpermute_kb<MODE, false>(a, s);
}

hipError_t launch_unpermute(const UnpermuteArgs& a, hipStream_t s) {
    const int yb = a.y_f32 ? 4 : 2, ob = a.out_f32 ? 4 : 2;
    const bool vec = a.H % 8 == 0 && wide(a.y, a.ldy, yb) && wide(a.residual, a.ldr, ob) && wide(a.out, a.ldo, ob);
    // A launch holds fewer than 2^32 threads.
    const int64_t most = ((int64_t)1 << 31) / (a.H / 8 + 64);
    for (int64_t t = 0; t < a.T; t += most) {
        UnpermuteArgs b = a;
        b.T = (int)(a.T - t < most ? a.T - t : most);
        b.rows = a.rows + t * a.topk;
        if (a.weights) b.weights = a.weights + t * a.topk;
        if (a.residual) b.residual = (const char*)a.residual + t * a.ldr * ob;
        b.out = (char*)a.out + t * a.ldo * ob;
        if (vec) launch_unpermute_type<kAligned>(b, s);
        else if (a.H >= 8) launch_unpermute_type<kAnywhere>(b, s);
        else launch_unpermute_type<kTiny>(b, s);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

// The gradients: KB pairs of a token at a time, their rows of y and dy by the
// token's row of dout. ONE: a workgroup a token, the dot products' parts meet
// in LDS; else `lanes` lanes a token (a power of two, eight columns each).
template <int KB, int MODE, bool ONE, bool Y32>
__global__ __launch_bounds__(512) void unpermute_bwd_kernel(UnpermuteBwdArgs a, int pieces, int lanes) {
    __shared__ float part[8][KB];
    const int tid = (int)threadIdx.x, H = a.H, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t P = (int64_t)a.T * a.topk;
    int64_t t = ONE ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * (256 / lanes) + tid / lanes;
    const bool here = t < a.T;
    if (!here) t = a.T - 1;  // (stays for the lanes' sums)
    const char* dr = (const char*)a.dout + t * a.lddo * (a.out_f32 ? 4 : 2);
    for (int j0 = 0; j0 < a.topk; j0 += KB) {
        int r[KB];
        float wt[KB], dot[KB];
        bool ok[KB];  // a row to write
#pragma unroll
        for (int j = 0; j < KB; ++j) {
            const int k = j0 + j < a.topk ? j0 + j : a.topk - 1;
            r[j] = a.rows[t * a.topk + k];
            if (ONE) r[j] = __builtin_amdgcn_readfirstlane(r[j]);
            wt[j] = a.weights ? a.weights[t * a.topk + k] : 1.0f;
            ok[j] = here && j0 + j < a.topk && (r[j] < 0 ? -1 - (int64_t)r[j] : r[j]) < P;
            dot[j] = 0.0f;
        }
        for (int q = ONE ? tid : tid % lanes; q < pieces; q += ONE ? (int)blockDim.x : pieces) {
            const int i = q * 8;
            const Raw8 fd = fetch8<MODE>(dr, a.out_f32, i, H);
            Raw8 y[KB];
            if (a.dweights) {
#pragma unroll
                for (int j = 0; j < KB; ++j)
                    y[j] = fetch8<MODE>((const char*)a.y + safe_row(r[j], P) * a.ldy * (Y32 ? 4 : 2), Y32, i, H);
            }
            const f32x8 d = widen8<MODE>(fd, a.out_f32, i, H);
            if (a.dweights) {
                const int skip = skip8<MODE>(i, H);
#pragma unroll
                for (int j = 0; j < KB; ++j) {
                    const f32x8 v = widen8<MODE>(y[j], Y32, i, H);
#pragma unroll
                    for (int e = 0; e < 8; ++e) dot[j] = e >= skip ? fmaf(d[e], v[e], dot[j]) : dot[j];
                }
            }
            if (a.dy) {
#pragma unroll
                for (int j = 0; j < KB; ++j) {
                    if (!ok[j]) continue;
                    const int64_t row = r[j] < 0 ? -1 - (int64_t)r[j] : r[j];
                    f32x8 v;
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] = r[j] < 0 ? 0.0f : wt[j] * d[e];
                    put8<MODE>((char*)a.dy + row * a.lddy * (Y32 ? 4 : 2), Y32, i, H, v);
                }
            }
        }
        if (!a.dweights) continue;
        if constexpr (ONE) {
#pragma unroll
            for (int j = 0; j < KB; ++j) {
                const float v = wave_sum(dot[j]);
                if ((tid & 63) == 0) part[w][j] = v;
            }
            __syncthreads();
            if (tid < KB && j0 + tid < a.topk) {
                float v = 0.0f;
                for (int k = 0; k < (int)blockDim.x / 64; ++k) v += part[k][tid];
                const int e = a.rows[t * a.topk + j0 + tid];
                a.dweights[t * a.topk + j0 + tid] = e >= 0 && e < P ? v : 0.0f;  // (of row 0 for the others)
            }
            __syncthreads();
        } else {
#pragma unroll
            for (int j = 0; j < KB; ++j) {
                float v = dot[j];
                for (int d = 1; d < lanes; d *= 2) v += __shfl_xor(v, d);
                if (here && j0 + j < a.topk && tid % lanes == 0)
                    a.dweights[t * a.topk + j0 + j] = r[j] >= 0 && r[j] < P ? v : 0.0f;
            }
        }
    }
}

template <int KB, int MODE, bool Y32>
static void launch_unpermute_bwd_as(const UnpermuteBwdArgs& a, hipStream_t s) {
    const int pieces = (a.H + 7) / 8;
    if (pieces > 32) {
        hipLaunchKernelGGL((unpermute_bwd_kernel<KB, MODE, true, Y32>), dim3((unsigned)a.T), dim3(row_threads(pieces)), 0, s, a, pieces, 0);
    } else {
        int lanes = 1;
        while (lanes < pieces) lanes *= 2;
        const int tokens = 256 / lanes;
        hipLaunchKernelGGL((unpermute_bwd_kernel<KB, MODE, false, Y32>), dim3((unsigned)((a.T + tokens - 1) / tokens)), dim3(256), 0, s, a,
                           pieces, lanes);
    }
}

template <int MODE, bool Y32>
static void launch_unpermute_bwd_kb(const UnpermuteBwdArgs& a, hipStream_t s) {
    if (a.topk <= 2) launch_unpermute_bwd_as<2, MODE, Y32>(a, s);
    else if (a.topk <= 4) launch_unpermute_bwd_as<4, MODE, Y32>(a, s);
    else launch_unpermute_bwd_as<8, MODE, Y32>(a, s);
}

template <int MODE>
static void launch_unpermute_bwd_type(const UnpermuteBwdArgs& a, hipStream_t s) {
    if (a.y_f32) launch_unpermute_bwd_kb<MODE, true>(a, s);
    else launch_unpermute_bwd_kb<MODE, false>(a, s);
}

hipError_t launch_unpermute_bwd(const UnpermuteBwdArgs& a, hipStream_t s) {
    const int yb = a.y_f32 ? 4 : 2, ob = a.out_f32 ? 4 : 2;
    const bool vec = a.H % 8 == 0 && wide(a.dout, a.lddo, ob) && wide(a.y, a.ldy, yb) && wide(a.dy, a.lddy, yb);
    if (vec) launch_unpermute_bwd_type<kAligned>(a, s);
    else if (a.H >= 8) launch_unpermute_bwd_type<kAnywhere>(a, s);
    else launch_unpermute_bwd_type<kTiny>(a, s);
    return hipGetLastError();
}

}  // namespace moe
