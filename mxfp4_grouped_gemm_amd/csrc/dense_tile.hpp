// LDS-tiled dense product C[m, n] = sum_k X[m, k] W[n, k] with the epilogues
// of the dense operators, on v_mfma_f32_16x16x32_bf16 or, for MXFP8 operands,
// v_mfma_scale_f32_16x16x128_f8f6f4.
//
// A workgroup owns a BM x BN tile of C and its waves a WM x WN grid of it.
// Both operands go to LDS in steps of 128 bytes of K (64 bf16 or 128 e4m3
// elements) with loads straight into LDS, one buffer ahead of the one that is
// multiplied (two buffers, one barrier a step; the buffers are separate
// __shared__ objects, so that the compiler sees that reads of one need not
// wait for loads into the other). Tiles that leave compute units idle have no
// second workgroup to hide a load behind: they run with four buffers (64 x 64
// tiles with eight), three (seven) steps of loads in flight.
//
// Tiles of 256 x 256 have the matrix cores busy for 60 and 55% of the time in the
// two products of the forward, 53 and 41% in MXFP8, 49% in dh and 78% in the
// gradients, at the clock that their power leaves (1.9 GHz in a long run); what
// the rest waits for has not been parted. 8192 tokens: gated, 4096 pairs
// over K = 3584, 336 us in a long run of this call alone (1.43 PFLOP/s of
// bf16); 3584 columns over K = 4096, 178 us (1.35); the library's plain
// products of these sizes take 321 and 169 there. One after the other, over
// three sets of inputs, both take 607 to 620 us with their epilogues, the library's two
// products alone 483. MFMAs of 32 x 32 were slower:
// the same LDS bytes, and fewer, longer instructions to place reads between.
//
// W is the MFMA's first operand, so a lane's four results are four
// consecutive n of one m. The rows of W are dealt to the fragments such that
// a lane's fragments are consecutive too (`n = 4 F q + 4 f + p` for fragment f
// of F, MFMA row i = 4 q + p): a lane owns 4 F consecutive outputs of a token.
//
// LDS layouts, in 16-byte pieces (the granule of a load into LDS, whose
// destination is fixed, so the piece that a lane fetches is permuted):
//  * K-major operand: 128-byte rows; piece c of row r sits at c ^ key(r),
//    key chosen such that the 16 rows of an operand read, two of which share
//    the 64 banks, touch every bank once.
//  * K as the row index (the other operand order of a backward product): rows
//    of BM or BN elements; the operand is read through the transposing LDS
//    read (four rows of 16 elements -> each lane four elements of one column).
//    Piece c of row k sits at c ^ key(k), such that the four rows of 16 lanes'
//    read, whose columns are consecutive (X) or 16 apart (W), share no bank.
#pragma once

#include <type_traits>

#include "common.hpp"
#include "dense.hpp"
#include "dense_epilogue.hpp"
#include "mx8.hpp"

namespace moe {
namespace dense {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int kEltBf16 = 0, kEltMx8 = 1;
constexpr int kGroupM = 4;      // tiles of M that share a column of W tiles
// Every load's record: masked lanes carry kOob, the others stay inside the
// tensor by construction (the tile's base is a 64-bit address).
constexpr uint32_t kRecord = 0x7fff0000u;

typedef __attribute__((address_space(3))) void* lds_ptr;

__device__ __forceinline__ void load_lds16(rsrc_t r, uint8_t* dst, uint32_t voff, uint32_t soff) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr)dst, 16, voff, soff, 0, 0);
}

// f(0), f(1), ... f(N - 1), each with its number as a constant.
template <int I, int N, class F>
__device__ __forceinline__ void each(F f) {
    if constexpr (I < N) {
        f(std::integral_constant<int, I>());
        each<I + 1, N>(f);
    }
}

// Asks the scheduler to spread READS LDS reads and LOADS loads evenly over
// MFMAS matrix instructions.
template <int READS, int LOADS, int MFMAS, int I = 0>
__device__ __forceinline__ void spread() {
    if constexpr (I < READS) {
        constexpr int loads = LOADS * (I + 1) / READS - LOADS * I / READS;
        constexpr int mfmas = MFMAS * (I + 1) / READS - MFMAS * I / READS;
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        if constexpr (loads > 0) __builtin_amdgcn_sched_group_barrier(0x20, loads, 0);
        if constexpr (mfmas > 0) __builtin_amdgcn_sched_group_barrier(0x8, mfmas, 0);
        spread<READS, LOADS, MFMAS, I + 1>();
    }
}

template <int W>
__device__ __forceinline__ void load_words(uint32_t (&d)[W], const void* p) {
    if constexpr (W == 4) {
        const u32x4 u = *(const u32x4*)p;
        d[0] = u[0], d[1] = u[1], d[2] = u[2], d[3] = u[3];
    } else {
        const u32x2 u = *(const u32x2*)p;
        d[0] = u[0], d[1] = u[1];
    }
}

// The same with two matrix instructions a read and the rest behind the last
// one, for the phase before a barrier, which waits for the reads.
template <int READS, int MFMAS, int I = 0>
__device__ __forceinline__ void spread_front() {
    if constexpr (I < READS) {
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        constexpr int mfmas = 2 * READS <= MFMAS ? (I + 1 < READS ? 2 : MFMAS - 2 * (READS - 1)) : I + 1 < MFMAS ? 1 : 0;
        if constexpr (mfmas > 0) __builtin_amdgcn_sched_group_barrier(0x8, mfmas, 0);
        spread_front<READS, MFMAS, I + 1>();
    }
}

// Four or eight consecutive outputs, rounded.
template <int V>
__device__ __forceinline__ void store_bf16(uint16_t* p, const float* v) {
    if constexpr (V == 8)
        *(u32x4*)p = u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
    else
        *(u32x2*)p = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
}

// Waits until at most LOADS of this wave's loads are in flight and its LDS
// reads are done, then for the workgroup. Loads complete in order, so what is
// left in flight are the latest steps'.
template <int LOADS>
__device__ __forceinline__ void sync_step() {
    if constexpr (LOADS == 0) {
        __syncthreads();
    } else {
        static_assert(LOADS < 64, "six bits");
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(LOADS) : "memory");
    }
}

template <int BM_, int BN_, int WM_, int WN_, bool XT_, bool WT_, int ELT_, int EPI_, bool SPLIT_, bool LORA_, int NB_ = 2,
          int KB_ = 128>
struct Tile {
    static constexpr int KB = KB_;  // bytes of K a step
    static constexpr int NB = NB_;  // LDS buffers
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, ELT = ELT_, EPI = EPI_;
    static constexpr bool XT = XT_, WT = WT_, SPLIT = SPLIT_, LORA = LORA_;
    static constexpr bool GATED = EPI == kEpiGated || EPI == kEpiGatedMx;
    static constexpr int NW = WM * WN, THREADS = NW * 64;
    static constexpr int FM = BM / WM / 16, FN = BN / WN / 16;
    static constexpr int F = GATED ? FN / 2 : FN;      // fragments of one column set
    static constexpr int BNC = GATED ? BN / 2 : BN;    // output columns (pairs) of a tile
    static constexpr int ESZ = ELT == kEltBf16 ? 2 : 1;
    static constexpr int BK = KB / ESZ;
    static constexpr int XBYTES = BM * KB, WBYTES = BN * KB;
    static constexpr int SBYTES = ELT == kEltMx8 ? (BM + BN) * 4 : 0;  // scales of a step
    static constexpr int BUF = XBYTES + WBYTES + SBYTES;
    static constexpr int XL = XBYTES / 1024 / NW, WL = WBYTES / 1024 / NW;  // loads a wave issues per step
    static_assert(XBYTES % (1024 * NW) == 0 && WBYTES % (1024 * NW) == 0, "whole loads");
    static_assert(ELT == kEltBf16 || (!XT && !WT), "MXFP8 operands are K-major");
};

// Swizzle keys (see the top).
template <int KB>
__device__ __forceinline__ int key_x(int r) {
    return KB == 128 ? (r >> 1) & 7 : (r >> 2) & 3;
}
template <int KB, int F>
__device__ __forceinline__ int key_w(int r) {
    constexpr int s = F == 4 ? 4 : F == 2 ? 3 : 2;
    return KB == 128 ? ((r >> 1) & 1) | (((r >> s) & 3) << 1) : (r >> s) & 3;
}
template <int PIECES>
__device__ __forceinline__ int key_t(int k) {
    return (2 * ((k & 3) | (((k >> 3) & 1) << 2))) & (PIECES - 1);
}

// For W, whose 16 columns of a read are groups of four at a stride of 16 (rows
// of 128 columns or more) or 8.
template <int PIECES>
__device__ __forceinline__ int key_tw(int k) {
    return PIECES >= 16 ? (k & 1) | ((k >> 3) & 1) << 1 | (k & 2) << 2 : key_t<PIECES>(k);
}

// Tokens without an adapter, in the searches over a tile's adapters.
constexpr int kNoAdapter = 0x7fffffff;

// Minimum over the 16 lanes of a row (rotations by 8, 4, 2 and 1).
__device__ __forceinline__ int min16(int v) {
#define MOE_MIN_ROR(N)                                                          \
    {                                                                           \
        const int o = __builtin_amdgcn_mov_dpp(v, 0x120 + N, 0xf, 0xf, true);   \
        v = o < v ? o : v;                                                      \
    }
    MOE_MIN_ROR(8)
    MOE_MIN_ROR(4)
    MOE_MIN_ROR(2)
    MOE_MIN_ROR(1)
#undef MOE_MIN_ROR
    return v;
}

// The adapters of a lane's tokens (one a fragment of X) and their ranks, loaded
// ahead of a tile's product.
template <class C>
struct LoraRows {
    int idx[C::FM], rank[C::FM], token[C::FM];  // token: M for rows past the end
};

// The tile's rows are rows m0.. of l.order or, without it, tokens m0...
template <class C>
__device__ __forceinline__ void lora_rows(const LoraArgs& l, int m0, int M, LoraRows<C>& o) {
    const int lane = (int)threadIdx.x & 63;
    const int r0 = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6) / C::WN * C::FM * 16 + (lane & 15);
    const rsrc_t ri = make_rsrc((l.order ? l.sorted : l.index) + m0, kRecord);
    uint32_t i[C::FM];
#pragma unroll
    for (int fm = 0; fm < C::FM; ++fm) {
        const int r = r0 + fm * 16;
        i[fm] = __builtin_amdgcn_raw_buffer_load_b32(ri, m0 + r < M ? (uint32_t)r * 4u : kOob, 0, 0);
        o.token[fm] = m0 + r < M ? m0 + r : M;
        o.rank[fm] = l.rank;
    }
    if (l.order) {
        const rsrc_t ro = make_rsrc(l.order + m0, kRecord);
#pragma unroll
        for (int fm = 0; fm < C::FM; ++fm) {
            const int r = r0 + fm * 16;
            const int t = __builtin_amdgcn_raw_buffer_load_b32(ro, m0 + r < M ? (uint32_t)r * 4u : kOob, 0, 0);
            o.token[fm] = m0 + r < M ? t : M;
        }
    }
#pragma unroll
    for (int fm = 0; fm < C::FM; ++fm)
        o.idx[fm] = m0 + r0 + fm * 16 < M && i[fm] < (uint32_t)l.n ? (int)i[fm] : kNoAdapter;
    if (!l.ranks) return;
    const rsrc_t rr = make_rsrc(l.ranks, kRecord);
#pragma unroll
    for (int fm = 0; fm < C::FM; ++fm) {
        const int r = __builtin_amdgcn_raw_buffer_load_b32(rr, o.idx[fm] != kNoAdapter ? (uint32_t)o.idx[fm] * 4u : kOob, 0, 0);
        o.rank[fm] = r < 0 ? 0 : r < l.rank ? r : l.rank;  // (negated and subtracted from below)
    }
}

// The low-rank term of a tile's accumulators: for each adapter that one of a
// wave's rows uses, acc += B[a] v over its rank, with v (fp32) split into two
// bf16 (hi + lo: 16 bits of it). The tile's rows of v, 64 ranks at a time, are
// summed over the parts and split once for all waves, into the first two LDS
// buffers (32 ranks each: 128-byte rows, hi in pieces 0..3, lo in 4..7,
// permuted as rows of X are). An adapter's part is a memory latency and a few
// matrix instructions, so the rows of B of the next three halves (of 32 ranks) are
// on their way while those of one are multiplied. n_of(f) gives the W row (of
// the stack's `brows` rows) of fragment f's MFMA row lane % 16, or -1.
template <class C, class NOF>
__device__ __forceinline__ void lora_accumulate(const LoraArgs& l, int64_t brows, int m0, int M, const LoraRows<C>& rows,
                                                f32x4 (&acc)[C::FN][C::FM], NOF n_of, uint8_t* s0, uint8_t* s1) {
    const int tid = (int)threadIdx.x, lane = tid & 63;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g = lane >> 4, l16 = lane & 15, r0 = w / C::WN * C::FM * 16;
    struct Step {
        int ad, h, rank;  // an adapter, the half of the 64 ranks, the adapter's rank
    };
    // The smallest adapter above `last` among the wave's rows.
    auto above = [&](int last) -> Step {
        int next = kNoAdapter, rank = 0;
#pragma unroll
        for (int fm = 0; fm < C::FM; ++fm) next = rows.idx[fm] > last && rows.idx[fm] < next ? rows.idx[fm] : next;
        next = __builtin_amdgcn_readfirstlane(min16(next));
#pragma unroll
        for (int fm = 0; fm < C::FM; ++fm) rank = rows.idx[fm] == next ? -rows.rank[fm] : rank;
        return {next, 0, -__builtin_amdgcn_readfirstlane(min16(rank))};
    };
    static_assert(C::BUF >= C::BM * 128 && C::NB >= 2, "a buffer holds 32 ranks of the tile's rows");
    constexpr int kAll = C::BM * 8 / C::THREADS;  // eights of ranks a thread stages
    constexpr int P = C::FM > 4 ? 1 : 2;          // at a time, as the registers allow
    for (int k0 = 0; k0 < l.rank; k0 += 64) {
        auto load_b = [&](u32x4 (&d)[C::FN], const Step& p) {
            const bool some = p.ad != kNoAdapter;
            const rsrc_t rb = make_rsrc(l.b + (int64_t)(some ? p.ad : 0) * brows * l.rank, kRecord);
            const int k = k0 + 32 * p.h + 8 * g;
#pragma unroll
            for (int f = 0; f < C::FN; ++f) {
                const int n = n_of(f);
                const uint32_t at = (uint32_t)(n * l.rank + k) * 2u;
                d[f] = bld16(rb, some & (n >= 0) & (k < l.rank) ? at : kOob);
            }
        };
        // The second half of an adapter whose rank reaches into it, else the
        // next adapter.
        auto after = [&](const Step& p) -> Step {
            return p.h == 0 && k0 + 32 < p.rank ? Step{p.ad, 1, p.rank} : above(p.ad);
        };
        u32x4 bu[4][C::FN];
        Step st[4];
        st[0] = above(-1);
        load_b(bu[0], st[0]);
        // The last loads into the buffers and the reads of them are done.
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
#pragma unroll
        for (int i0 = 0; i0 < kAll; i0 += P) {
            f32x4 v[P][2], part[kMaxLoraParts - 1][P][2];
            auto load_v = [&](f32x4 (&d)[P][2], int p) {
                const rsrc_t rv = make_rsrc(l.v + p * l.part_stride + (int64_t)m0 * l.vld, kRecord);
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    const int q = tid + (i0 + i) * C::THREADS, k = k0 + q % 8 * 8, t = q / 8;
                    const uint32_t at = (uint32_t)(t * l.vld + k) * 4u;
                    const uint32_t o = (m0 + t < M) & (k < l.rank) & (p < l.parts) ? at : kOob;
                    d[i][0] = __builtin_bit_cast(f32x4, bld16(rv, o));
                    d[i][1] = __builtin_bit_cast(f32x4, bld16(rv, o == kOob ? o : o + 16));
                }
            };
            load_v(v, 0);
            if (l.parts > 1) {
#pragma unroll
                for (int p = 1; p < kMaxLoraParts; ++p) load_v(part[p - 1], p);
#pragma unroll
                for (int p = 1; p < kMaxLoraParts; ++p)
#pragma unroll
                    for (int i = 0; i < P; ++i)
#pragma unroll
                        for (int h = 0; h < 2; ++h) v[i][h] += part[p - 1][i][h];
                if (l.scale) {
                    const rsrc_t ri = make_rsrc((l.order ? l.sorted : l.index) + m0, kRecord), rs = make_rsrc(l.scale, kRecord);
                    const rsrc_t rr = make_rsrc(l.ranks, kRecord);
#pragma unroll
                    for (int i = 0; i < P; ++i) {
                        const int q = tid + (i0 + i) * C::THREADS, t = q / 8;
                        const uint32_t ad = __builtin_amdgcn_raw_buffer_load_b32(ri, m0 + t < M ? (uint32_t)t * 4u : kOob, 0, 0);
                        const uint32_t at = m0 + t < M && ad < (uint32_t)l.n ? ad * 4u : kOob;
                        const float scale = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, at, 0, 0));
                        int rank = l.ranks ? (int)__builtin_amdgcn_raw_buffer_load_b32(rr, at, 0, 0) : l.rank;
                        rank = (rank < 0 ? 0 : rank < l.rank ? rank : l.rank) - (k0 + q % 8 * 8);
                        // Beyond the rank zeros stay zeros for any scale.
#pragma unroll
                        for (int e = 0; e < 8; ++e) v[i][e / 4][e % 4] = e < rank ? v[i][e / 4][e % 4] * scale : 0.0f;
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const int q = tid + (i0 + i) * C::THREADS, r = q / 8, c = q % 4;
                u32x4 hi, lo;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float x0 = v[i][e / 2][2 * (e & 1)], x1 = v[i][e / 2][2 * (e & 1) + 1];
                    hi[e] = pack_bf16x2(x0, x1);
                    // An infinite half has no rest.
                    const float h0 = __uint_as_float(hi[e] << 16), h1 = __uint_as_float(hi[e] & 0xffff0000u);
                    lo[e] = pack_bf16x2(fabsf(h0) < __builtin_inff() ? x0 - h0 : 0.0f, fabsf(h1) < __builtin_inff() ? x1 - h1 : 0.0f);
                }
                uint8_t* dst = (q % 8 < 4 ? s0 : s1) + r * 128;
                *(u32x4*)(dst + ((c ^ key_x<128>(r)) << 4)) = hi;
                *(u32x4*)(dst + (((4 + c) ^ key_x<128>(r)) << 4)) = lo;
            }
        }
        __syncthreads();
        auto multiply = [&](u32x4 (&d)[C::FN], const Step& p) {
            // Columns beyond the adapter's rank are not read as numbers.
            const int left = p.rank - (k0 + 32 * p.h + 8 * g);
            u32x4 keep;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int bits = (left - 2 * e) * 16;
                keep[e] = (uint32_t)((1ull << (bits < 0 ? 0 : bits > 32 ? 32 : bits)) - 1);
            }
#pragma unroll
            for (int f = 0; f < C::FN; ++f) d[f] &= keep;
            const uint8_t* buf = p.h ? s1 : s0;
#pragma unroll
            for (int fm = 0; fm < C::FM; ++fm) {
                // A lane's results are one token's: only those of this adapter
                // are kept (a NaN in its factors stays with its own tokens).
                const bool mine = rows.idx[fm] == p.ad;
                if (!__any(mine)) continue;
                const int r = r0 + fm * 16 + l16;
                const u32x4 hi = *(const u32x4*)(buf + r * 128 + ((g ^ key_x<128>(r)) << 4));
                const u32x4 lo = *(const u32x4*)(buf + r * 128 + (((4 + g) ^ key_x<128>(r)) << 4));
#pragma unroll
                for (int f = 0; f < C::FN; ++f) {
                    f32x4 o = mfma16x16x32(__builtin_bit_cast(bf16x8, d[f]), __builtin_bit_cast(bf16x8, hi), acc[f][fm]);
                    o = mfma16x16x32(__builtin_bit_cast(bf16x8, d[f]), __builtin_bit_cast(bf16x8, lo), o);
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[f][fm][e] = mine ? o[e] : acc[f][fm][e];
                }
            }
        };
        each<1, 4>([&](auto i) {
            st[i.value] = after(st[i.value - 1]);
            load_b(bu[i.value], st[i.value]);
        });
        auto use = [&](auto i) {
            if (st[i.value].ad == kNoAdapter) return false;
            multiply(bu[i.value], st[i.value]);
            st[i.value] = after(st[(i.value + 3) % 4]);
            load_b(bu[i.value], st[i.value]);
            return true;
        };
        while (use(std::integral_constant<int, 0>()) && use(std::integral_constant<int, 1>()) &&
               use(std::integral_constant<int, 2>()) && use(std::integral_constant<int, 3>())) {
        }
    }
}

// The LDS buffers of a kernel whose tiles need NB of BUF bytes: separate
// objects (see the top), of which the unused ones vanish.
#define MOE_TILE_BUFFERS(s, NB, BUF)                                      \
    __shared__ __align__(1024) uint8_t s##0_[BUF];                        \
    __shared__ __align__(1024) uint8_t s##1_[BUF];                        \
    __shared__ __align__(1024) uint8_t s##2_[(NB) > 2 ? (BUF) : 16];      \
    __shared__ __align__(1024) uint8_t s##3_[(NB) > 2 ? (BUF) : 16];      \
    __shared__ __align__(1024) uint8_t s##4_[(NB) > 4 ? (BUF) : 16];      \
    __shared__ __align__(1024) uint8_t s##5_[(NB) > 4 ? (BUF) : 16];      \
    __shared__ __align__(1024) uint8_t s##6_[(NB) > 4 ? (BUF) : 16];      \
    __shared__ __align__(1024) uint8_t s##7_[(NB) > 4 ? (BUF) : 16];      \
    uint8_t* const s[8] = {s##0_, s##1_, s##2_, s##3_, s##4_, s##5_, s##6_, s##7_}

// One tile: number `id` of the product's tiles, part `part` of a split K.
template <class C>
__device__ __forceinline__ void dense_tile(const DenseArgs& a, int id, int part, uint8_t* const (&s)[8]) {
    const int tid = (int)threadIdx.x, lane = tid & 63;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = w / C::WN, wn = w % C::WN;
    const int g = lane >> 4, l16 = lane & 15;

    // Tile of this workgroup. Consecutive workgroups go round-robin over the 8
    // XCDs; giving an XCD a contiguous run of tiles, in columns of kGroupM
    // tiles of M, keeps its W tiles in its own L2.
    const int tm = (a.M + C::BM - 1) / C::BM, tn = (a.N + C::BNC - 1) / C::BNC;
    const int total = tm * tn;
    {
        const int q = total / 8, r = total % 8, xcd = id % 8, i = id / 8;
        id = xcd * q + (xcd < r ? xcd : r) + i;
    }
    const int per = kGroupM * tn, grp = id / per, rest = id % per;
    const int gm = tm - grp * kGroupM < kGroupM ? tm - grp * kGroupM : kGroupM;
    const int m0 = (grp * kGroupM + rest % gm) * C::BM, n0 = rest / gm * C::BNC;

    const int steps = (a.K + C::BK - 1) / C::BK;
    int kt0 = 0, kt1 = steps;
    if constexpr (C::SPLIT) {
        const int z = part;
        kt0 = (int)((int64_t)steps * z / a.splits);
        kt1 = (int)((int64_t)steps * (z + 1) / a.splits);
    }

    // With an order of the tokens the tile's rows are gathered: their offsets
    // are from the first token.
    const bool gather = C::LORA && a.lora.order != nullptr;
    LoraRows<C> lrows;
    if constexpr (C::LORA) lora_rows<C>(a.lora, m0, a.M, lrows);

    // Loads: offsets of this lane's pieces from the tile's first element.
    const char* xb = (const char*)a.x + (C::XT ? (int64_t)m0 : gather ? 0 : (int64_t)m0 * a.ldx) * C::ESZ;
    const char* wb = (const char*)a.w + (C::WT ? (int64_t)n0 : (int64_t)n0 * a.ldw) * C::ESZ;
    uint32_t xo[C::XL], wo[C::WL];
    constexpr int kPieces = C::KB / 16;  // of a K-major row
    // K of a piece in its step (elements).
    auto xk = [&](int i) {
        const int p = (w * C::XL + i) * 64 + lane;
        if constexpr (C::XT) return (w * C::XL * 64 + lane) / (C::BM / 8) + i * 64 / (C::BM / 8);
        else return ((p % kPieces) ^ key_x<C::KB>(p / kPieces)) * (16 / C::ESZ);
    };
    auto wk = [&](int i) {
        const int p = (w * C::WL + i) * 64 + lane;
        if constexpr (C::WT) return (w * C::WL * 64 + lane) / (C::BN / 8) + i * 64 / (C::BN / 8);
        else return ((p % kPieces) ^ key_w<C::KB, C::F>(p / kPieces)) * (16 / C::ESZ);
    };
#pragma unroll
    for (int i = 0; i < C::XL; ++i) {
        const int p = (w * C::XL + i) * 64 + lane;  // piece of the tile
        if constexpr (C::XT) {
            constexpr int PR = C::BM / 8;  // pieces a row
            const int k = p / PR, c = (p % PR) ^ key_t<PR>(k);
            xo[i] = m0 + c * 8 < a.M ? (uint32_t)(k * a.ldx * 2 + c * 16) : kOob;
        } else {
            const int r = p / kPieces, c = (p % kPieces) ^ key_x<C::KB>(r);
            const int t = gather ? a.lora.order[m0 + r < a.M ? m0 + r : 0] : r;
            xo[i] = m0 + r < a.M ? (uint32_t)(t * a.ldx * C::ESZ + c * 16) : kOob;
        }
    }
#pragma unroll
    for (int i = 0; i < C::WL; ++i) {
        const int p = (w * C::WL + i) * 64 + lane;
        if constexpr (C::WT) {
            constexpr int PR = C::BN / 8;
            static_assert(C::FN == (PR >= 16 ? 4 : 2), "the keys are for this stride of a read's columns");
            const int k = p / PR, c = (p % PR) ^ key_tw<PR>(k);
            wo[i] = n0 + c * 8 < a.N ? (uint32_t)(k * a.ldw * 2 + c * 16) : kOob;
        } else {
            const int r = p / kPieces, c = (p % kPieces) ^ key_w<C::KB, C::F>(r);
            if constexpr (C::GATED) {
                // Rows [0, BNC) of the tile are gate rows, the others the up
                // rows, N rows further on: their own base (wo is 32 bits).
                const int col = r % C::BNC;
                wo[i] = n0 + col < a.N ? (uint32_t)(col * a.ldw * C::ESZ + c * 16) : kOob;
            } else {
                wo[i] = n0 + r < a.N ? (uint32_t)(r * a.ldw * C::ESZ + c * 16) : kOob;
            }
        }
    }
    const int64_t up = C::GATED ? (int64_t)a.N * a.ldw * C::ESZ : 0;

    const int kend = C::SPLIT && kt1 < steps ? kt1 * C::BK : a.K;
    // Loads of step kt into a buffer. Pieces past the end of K (all of them
    // for a step past the end) get out-of-range offsets: zeros, no traffic.
    auto issue = [&](uint8_t* buf, int kt) {
        const rsrc_t rx = make_rsrc(xb + (C::XT ? (int64_t)kt * C::BK * a.ldx * 2 : (int64_t)kt * C::KB), kRecord);
        const int64_t wadv = C::WT ? (int64_t)kt * C::BK * a.ldw * 2 : (int64_t)kt * C::KB;
        const rsrc_t rw = make_rsrc(wb + wadv, kRecord);
        const rsrc_t ru = make_rsrc(wb + wadv + up, kRecord);
        const int left = kend - kt * C::BK;
#pragma unroll
        for (int i = 0; i < C::XL; ++i)
            load_lds16(rx, buf + (w * C::XL + i) * 1024, xk(i) < left ? xo[i] : kOob, 0);
#pragma unroll
        for (int i = 0; i < C::WL; ++i) {
            const bool second = C::GATED && (w * C::WL + i) * (64 / kPieces) >= C::BNC;  // whole loads: uniform
            load_lds16(second ? ru : rw, buf + C::XBYTES + (w * C::WL + i) * 1024, wk(i) < left ? wo[i] : kOob, 0);
        }
    };

    // MXFP8 scales: a thread carries the four bytes of one row's step, rows of
    // X and then of W, through a register (a wave's rows share their base).
    static_assert(C::ELT != kEltMx8 || C::BM + C::BN == C::THREADS, "one row of scales a thread");
    // Rows of K / 32 bytes need not be aligned: the bytes of a step come from
    // the one or two aligned words that hold them.
    uint32_t slo = 0, shi = 0, so = 0;
    bool srow = false;
    const int kb = a.K / 32;
    const uint8_t* sbase = nullptr;
    if constexpr (C::ELT == kEltMx8) {
        const int r = w * 64;
        int64_t first;
        if (r < C::BM) {
            first = (int64_t)(m0 + r) * kb;
            sbase = a.xs;
            srow = m0 + r + lane < a.M;
        } else {
            const int rw = r - C::BM, col = n0 + (C::GATED ? rw % C::BNC : rw);
            first = (int64_t)(col + (C::GATED && rw >= C::BNC ? a.N : 0)) * kb;
            sbase = a.ws;
            srow = col + lane < a.N;
        }
        sbase += first & ~(int64_t)3;
        so = (uint32_t)(first & 3) + (uint32_t)(lane * kb);
    }
    auto load_scales = [&](int kt) {
        if constexpr (C::ELT == kEltMx8) {
            const rsrc_t rs = make_rsrc(sbase + (int64_t)kt * 4, kRecord);
            const int left = kb - kt * 4;  // bytes of the row from this step on
            const int in_word = (int)(so & 3);
            slo = __builtin_amdgcn_raw_buffer_load_b32(rs, srow && left > 0 ? so & ~3u : kOob, 0, 0);
            shi = __builtin_amdgcn_raw_buffer_load_b32(rs, srow && in_word > 0 && left + in_word > 4 ? (so & ~3u) + 4 : kOob, 0, 0);
        }
    };
    // Bytes past K get scale 2^-127 (their codes are zeros; a byte of the next
    // row could be the NaN scale).
    auto store_scales = [&](uint8_t* buf, int kt) {
        if constexpr (C::ELT == kEltMx8) {
            const int left = kb - kt * 4;
            const uint32_t keep = left >= 4 ? 0xffffffffu : left <= 0 ? 0u : (1u << (8 * left)) - 1u;
            *(uint32_t*)(buf + C::XBYTES + C::WBYTES + tid * 4) = __builtin_amdgcn_alignbyte(shi, slo, so & 3) & keep;
        }
    };

    f32x4 acc[C::FN][C::FM];
#pragma unroll
    for (int i = 0; i < C::FN; ++i)
#pragma unroll
        for (int j = 0; j < C::FM; ++j) acc[i][j] = f32x4{0, 0, 0, 0};

    // LDS row of W for fragment f, MFMA row i (K-major).
    auto wrow = [&](int f, int i) {
        const int half = C::GATED ? f / C::F : 0, ff = f % C::F;
        return half * C::BNC + wn * 16 * C::F + (i >> 2) * 4 * C::F + ff * 4 + (i & 3);
    };
    const int xr0 = wm * C::FM * 16;
    auto read_x = [&](const uint8_t* buf, int fm, int piece) -> u32x4 {
        const int r = xr0 + fm * 16 + l16;
        return *(const u32x4*)(buf + r * C::KB + ((piece ^ key_x<C::KB>(r)) << 4));
    };
    auto read_w = [&](const uint8_t* buf, int f, int piece) -> u32x4 {
        const int r = wrow(f, l16);
        return *(const u32x4*)(buf + C::XBYTES + r * C::KB + ((piece ^ key_w<C::KB, C::F>(r)) << 4));
    };
    // Transposed operand: four groups of four columns, c0 + q * stride, of K
    // rows 32 s + 8 g + 0..7.
    auto read_t = [&](const uint8_t* base, auto pieces, int c0, int stride, int s) -> bf16x8 {
        constexpr int PR = decltype(pieces)::value, pitch = PR * 16;
        bf16x4 v[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int k = 32 * s + 8 * g + 4 * h + (l16 >> 2);
            const int col = c0 + (l16 & 3) * stride;
            const uint8_t* p = base + k * pitch + ((((col >> 3) ^ (stride > 4 ? key_tw<PR>(k) : key_t<PR>(k))) << 4) | ((col & 4) << 1));
            typedef __attribute__((address_space(3))) bf16x4* tp;
            v[h] = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((tp)p);
        }
        return __builtin_shufflevector(v[0], v[1], 0, 1, 2, 3, 4, 5, 6, 7);
    };

    if constexpr (C::ELT == kEltBf16) {
        // A step is four phases, (K half s, half h of the wave's rows of X),
        // and while the MFMAs of one run, the operands of the next are read.
        // The step's one barrier sits before its last phase: there the reads
        // of this step's buffer are done and the next step's loads have
        // landed, so the buffer takes the loads of the step after the next.
        constexpr int FH = C::FM / 2;
        bf16x8 xf[2][FH], wf[2][C::FN];
        auto read_ws = [&](const uint8_t* buf, int s, int set) {
#pragma unroll
            for (int f = 0; f < C::FN; ++f) {
                if constexpr (C::WT) wf[set][f] = read_t(buf + C::XBYTES, std::integral_constant<int, C::BN / 8>(), wn * 16 * C::FN + f * 4, 4 * C::FN, s);
                else wf[set][f] = __builtin_bit_cast(bf16x8, read_w(buf, f, 4 * s + g));
            }
        };
        auto read_xs = [&](const uint8_t* buf, int s, int h) {
#pragma unroll
            for (int f = 0; f < FH; ++f) {
                if constexpr (C::XT) xf[h][f] = read_t(buf, std::integral_constant<int, C::BM / 8>(), xr0 + (h * FH + f) * 16, 4, s);
                else xf[h][f] = __builtin_bit_cast(bf16x8, read_x(buf, h * FH + f, 4 * s + g));
            }
        };
        auto multiply = [&](int s, int h) {
#pragma unroll
            for (int j = 0; j < FH; ++j)
#pragma unroll
                for (int i = 0; i < C::FN; ++i)
                    acc[i][h * FH + j] = mfma16x16x32(wf[s][i], xf[h][j], acc[i][h * FH + j]);
        };
        constexpr int kXR = FH * (C::XT ? 2 : 1), kWR = C::FN * (C::WT ? 2 : 1), kMfma = C::FN * FH;
        auto step = [&](uint8_t* cur, uint8_t* nxt, int ws, int kt) {
            read_xs(cur, 0, 1);
            multiply(ws, 0);
            spread<kXR, 0, kMfma>();
            if constexpr (C::KB == 128) {
                __builtin_amdgcn_sched_barrier(0);
                read_ws(cur, 1, 1);
                read_xs(cur, 1, 0);
                multiply(0, 1);
                spread<kXR + kWR, 0, kMfma>();
                __builtin_amdgcn_sched_barrier(0);
                read_xs(cur, 1, 1);
                multiply(1, 0);
                spread_front<kXR, kMfma>();
            }
            sync_step<(C::NB - 2) * (C::XL + C::WL)>();
            issue(cur, kt + C::NB);
            if constexpr (C::KB == 128) read_ws(nxt, 0, 0);
            else read_ws(nxt, 0, ws ^ 1);
            read_xs(nxt, 0, 0);
            multiply(C::KB == 128 ? 1 : ws, 1);
            spread<kXR + kWR, C::XL + C::WL, kMfma>();
            __builtin_amdgcn_sched_barrier(0);
        };
        static_assert(C::NB == 2 || C::NB == 4 || C::NB == 8, "the step's operand sets alternate");
        if (kt0 < kt1) {
            each<0, C::NB>([&](auto i) { issue(s[i.value], kt0 + i.value); });
            sync_step<(C::NB - 1) * (C::XL + C::WL)>();
            read_ws(s[0], 0, 0);
            read_xs(s[0], 0, 0);
            // A step for each buffer a turn; a step past the end multiplies
            // zeros.
            for (int kt = kt0; kt < kt1; kt += C::NB)
                each<0, C::NB>([&](auto i) {
                    constexpr int b = i.value;
                    step(s[b], s[(b + 1) % C::NB], C::KB == 128 ? 0 : b & 1, kt + b);
                });
        }
    } else {
        // A lane's 32 elements are pieces g and 4 + g; its scale operand is
        // that of block g of the step. A step is one phase a fragment of X,
        // with the next fragment read meanwhile; the barrier sits before the
        // last phase, which reads the next step's operands of W.
        i32x8 xf[2], wf[2][C::FN];
        int xsc[2], wsc[2][C::FN];
        auto join8 = [](u32x4 lo, u32x4 hi) {
            return __builtin_bit_cast(i32x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        };
        auto read_ws = [&](const uint8_t* buf, int s) {
            const uint8_t* sc = buf + C::XBYTES + C::WBYTES + C::BM * 4 + g;
#pragma unroll
            for (int f = 0; f < C::FN; ++f) {
                wf[s][f] = join8(read_w(buf, f, g), read_w(buf, f, 4 + g));
                wsc[s][f] = sc[wrow(f, l16) * 4];
            }
        };
        auto read_x1 = [&](const uint8_t* buf, int j) {
            xf[j & 1] = join8(read_x(buf, j, g), read_x(buf, j, 4 + g));
            xsc[j & 1] = buf[C::XBYTES + C::WBYTES + (xr0 + j * 16 + l16) * 4 + g];
        };
        auto multiply = [&](int s, int j) {
#pragma unroll
            for (int i = 0; i < C::FN; ++i)
                acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wf[s][i], xf[j & 1], acc[i][j], 0, 0, 0,
                                                                             wsc[s][i], 0, xsc[j & 1]);
        };
        static_assert(C::FM % 2 == 0, "the next step's first fragment goes to the free operand");
        auto step = [&](uint8_t* cur, uint8_t* nxt, int s, int kt) {
#pragma unroll
            for (int j = 0; j < C::FM - 1; ++j) {
                read_x1(cur, j + 1);
                multiply(s, j);
                __builtin_amdgcn_sched_barrier(0);
            }
            store_scales(nxt, kt + 1);
            __syncthreads();
            issue(cur, kt + 2);
            load_scales(kt + 2);
            read_ws(nxt, s ^ 1);
            read_x1(nxt, 0);
            multiply(s, C::FM - 1);
            __builtin_amdgcn_sched_barrier(0);
        };
        if (kt0 < kt1) {
            issue(s[0], kt0);
            load_scales(kt0);
            store_scales(s[0], kt0);
            __syncthreads();
            issue(s[1], kt0 + 1);
            load_scales(kt0 + 1);
            read_ws(s[0], 0);
            read_x1(s[0], 0);
            for (int kt = kt0; kt < kt1; kt += 2) {
                step(s[0], s[1], 0, kt);
                step(s[1], s[0], 1, kt + 1);
            }
        }
    }

    // Column of fragment f's lane results (the first of four), and the token.
    auto m_of = [&](int fm) {
        if constexpr (C::LORA) return lrows.token[fm];
        else return m0 + xr0 + fm * 16 + l16;
    };
    auto n_of = [&](int f) { return n0 + wn * 16 * C::F + g * 4 * C::F + (f % C::F) * 4; };
    if constexpr (C::LORA) {
        static_assert(!C::SPLIT, "the kernel that joins the parts adds the term");
        // As MFMA rows: row i = l16 of fragment f.
        auto nrow = [&](int f) {
            const int n = n0 + wn * 16 * C::F + (l16 >> 2) * 4 * C::F + (f % C::F) * 4 + (l16 & 3);
            return n < a.N ? n + (C::GATED && f >= C::F ? a.N : 0) : -1;
        };
        lora_accumulate<C>(a.lora, C::GATED ? 2 * (int64_t)a.N : a.N, m0, a.M, lrows, acc, nrow, s[0], s[1]);
    }

    if constexpr (C::SPLIT) {
        const int64_t cols = C::GATED ? 2 * (int64_t)a.N : a.N;
        float* pz = a.partial + (int64_t)part * a.M * cols;
#pragma unroll
        for (int j = 0; j < C::FM; ++j) {
            const int m = m_of(j);
            if (m >= a.M) continue;
#pragma unroll
            for (int f = 0; f < C::FN; ++f) {
                const int n = n_of(f);
                if (n < a.N) *(f32x4*)(pz + m * cols + n + (C::GATED && f >= C::F ? a.N : 0)) = acc[f][j];
            }
        }
        return;
    }

    // What the epilogue reads from memory is loaded for several tokens before
    // the first of them is stored (the compiler keeps loads behind stores that
    // could be to the same place).
    constexpr int V = C::F % 2 ? 4 : 8;          // consecutive outputs of a lane
    constexpr int VN = C::F * 4 / V;             // groups of them
    constexpr bool kBwd = C::EPI == kEpiGatedBwd, kReads = C::EPI == kEpiOut || kBwd;
    constexpr int JB = kBwd && C::FM > 4 ? C::FM / 2 : C::FM;  // tokens a batch
    uint32_t ra[kReads ? JB : 1][VN][V / 2], rb[kBwd ? JB : 1][VN][V / 2];
#pragma unroll
    for (int j = 0; j < C::FM; ++j) {
        const int m = m_of(j);
        const bool mok = m < a.M;
        if constexpr (kReads) {
            if (j % JB == 0 && (kBwd || a.addend)) {
#pragma unroll
                for (int jj = 0; jj < JB; ++jj)
#pragma unroll
                    for (int v = 0; v < VN; ++v) {
                        const int mm = m_of(j + jj), n = n_of(v * (V / 4));
                        if (mm >= a.M || n >= a.N) continue;
                        if constexpr (kBwd) {
                            const uint16_t* gu = a.gate_up + mm * 2 * (int64_t)a.N + n;
                            load_words<V / 2>(ra[jj][v], gu);
                            load_words<V / 2>(rb[jj][v], gu + a.N);
                        } else {
                            load_words<V / 2>(ra[jj][v], a.addend + mm * a.ldadd + n);
                        }
                    }
            }
        }
        if constexpr (C::EPI == kEpiOut) {
            if (!mok) continue;
#pragma unroll
            for (int f = 0; f < C::FN; f += V / 4) {
                const int n = n_of(f);
                if (n >= a.N) continue;
                float v[V];
#pragma unroll
                for (int e = 0; e < V; ++e) v[e] = acc[f + e / 4][j][e % 4];
                if (a.addend) {
                    const auto& d = ra[j % JB][f / (V / 4)];
#pragma unroll
                    for (int e = 0; e < V; ++e) v[e] += __uint_as_float(e & 1 ? d[e / 2] & 0xffff0000u : d[e / 2] << 16);
                }
                if (a.out_f32) {
#pragma unroll
                    for (int e = 0; e < V; e += 4)
                        *(f32x4*)((float*)a.out + m * a.ldo + n + e) = f32x4{v[e], v[e + 1], v[e + 2], v[e + 3]};
                } else {
                    store_bf16<V>((uint16_t*)a.out + m * a.ldo + n, v);
                }
            }
        } else if constexpr (C::GATED) {
            float h[C::F][4], big = 0.0f;
#pragma unroll
            for (int f = 0; f < C::F; ++f)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    h[f][r] = acc[f][j][r] * sigmoid(acc[f][j][r]) * acc[f + C::F][j][r];
                    big = fmaxf(big, mx8_finite_abs(h[f][r]));
                }
            if constexpr (C::EPI == kEpiGatedMx) {
                // F == 2: the 32 columns of a block are the 8 of each of the
                // four lanes l16, l16 + 16, ...; N % 32 == 0, so a block is
                // inside the row as a whole.
                static_assert(C::F == 2, "a wave's columns are one block");
                big = fmaxf(big, __shfl_xor(big, 16));
                big = fmaxf(big, __shfl_xor(big, 32));
                const uint32_t sb = mx8_scale_byte(big);
                const float inv = mx8_inv_scale(sb);
                const int n = n_of(0);
                if (mok && n < a.N) {
                    u32x2 o;
                    o[0] = mx8_pack4(h[0][0], h[0][1], h[0][2], h[0][3], inv);
                    o[1] = mx8_pack4(h[1][0], h[1][1], h[1][2], h[1][3], inv);
                    *(u32x2*)((uint8_t*)a.out + m * a.ldo + n) = o;
                    if (g == 0) a.hs[m * (int64_t)(a.N / 32) + (n >> 5)] = (uint8_t)sb;
                }
            } else {
                if (!mok) continue;
#pragma unroll
                for (int f = 0; f < C::F; f += V / 4) {
                    const int n = n_of(f);
                    if (n >= a.N) continue;
                    store_bf16<V>((uint16_t*)a.out + m * a.ldo + n, &h[f][0]);
                    if (a.gate_up) {
                        uint16_t* gu = a.gate_up + m * 2 * (int64_t)a.N + n;
                        float gv[V], uv[V];
#pragma unroll
                        for (int e = 0; e < V; ++e) {
                            gv[e] = acc[f + e / 4][j][e % 4];
                            uv[e] = acc[f + C::F + e / 4][j][e % 4];
                        }
                        store_bf16<V>(gu, gv);
                        store_bf16<V>(gu + a.N, uv);
                    }
                }
            }
        } else {  // kEpiGatedBwd
            if (!mok) continue;
#pragma unroll
            for (int f = 0; f < C::FN; f += V / 4) {
                const int n = n_of(f);
                if (n >= a.N) continue;
                const auto& gb = ra[j % JB][f / (V / 4)];
                const auto& ub = rb[j % JB][f / (V / 4)];
                float dg[V], du[V], h[V];
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float gv = __uint_as_float(e & 1 ? gb[e / 2] & 0xffff0000u : gb[e / 2] << 16);
                    const float uv = __uint_as_float(e & 1 ? ub[e / 2] & 0xffff0000u : ub[e / 2] << 16);
                    const float dh = acc[f + e / 4][j][e % 4], sg = sigmoid(gv), silu = gv * sg;
                    dg[e] = dh * uv * sg * (1.0f + gv * (1.0f - sg));
                    du[e] = dh * silu;
                    h[e] = silu * uv;
                }
                uint16_t* o = (uint16_t*)a.out + m * a.ldo + n;
                store_bf16<V>(o, dg);
                store_bf16<V>(o + a.N, du);
                if (a.h) store_bf16<V>(a.h + m * (int64_t)a.N + n, h);
            }
        }
    }
}

template <class C>
__global__ __launch_bounds__(C::THREADS, 2) void dense_kernel(DenseArgs a) {
    MOE_TILE_BUFFERS(s, C::NB, C::BUF);
    dense_tile<C>(a, (int)blockIdx.x, (int)blockIdx.y, s);
}

template <class C>
inline int64_t tiles_of(const DenseArgs& a) {
    return (int64_t)((a.M + C::BM - 1) / C::BM) * ((a.N + C::BNC - 1) / C::BNC);
}

template <class C>
inline hipError_t launch_tile(const DenseArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)tiles_of<C>(a), C::SPLIT ? (unsigned)a.splits : 1u), block(C::THREADS);
    hipLaunchKernelGGL((dense_kernel<C>), grid, block, 0, s, a);
    return hipGetLastError();
}

}  // namespace dense
}  // namespace moe
