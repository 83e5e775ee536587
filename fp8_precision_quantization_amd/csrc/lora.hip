// lora.hip -- low-rank adapters of many requests beside a shared projection on
// gfx950: every row of a batch adds its own adapter's product to its output.
//
// Mathematics, for row m with adapter l = ids[m]:
//   t = A_l x[m]              (A_l [slices * rank, inner], bf16; t in fp32)
//   out[m, n] = y[m, n] + gain[l] * sum_r B_l[n, r] t[slice of n, r]
// t is held in 32 bits and enters the second product as a sum of bf16 terms,
// two of them (16 significant bits) for a bf16 output, three (all 24) for an
// fp32 one; B's values are bf16, so every product is exact in fp32.
//
// Rows are sorted by adapter first: a tile is up to 16 or 128 rows of one
// adapter, wherever they are in the batch, so that A and B are read once a tile
// whatever the order of the ids.  The sort counts ids in 1024 buckets; a tile of
// a bucket that several adapters share takes them one after the other.
//
// Up to kFew rows (a decode step) there is one launch, k_lora_few, where the sizes
// let it gain.  Up to kSmall rows there are otherwise two.  k_shrink_small: a block
// (up to kFew rows each of its waves) sorts for itself, takes a tile of 16 rows and
// a part of the inner dimension, whose steps go round its four waves, so that it
// reads neither x nor A twice; the parts' sums and the tile's rows go to the
// workspace.
// k_expand_small: a block takes a tile and 256 columns of one slice, adds up the
// parts of t in their order and adds B t to y.  Products are 16x16x32 with ranks
// (columns of the output) as the matrix rows and batch rows as its columns.
//
// Larger batches (prompts) are sorted by a launch of their own and take tiles of
// 128 rows.  k_shrink_large: x and A go through LDS in three stages of 64 inner
// elements, loaded past the registers; read as matrix operands directly, four
// neighbouring lanes touch four rows, which the caches serve at a quarter of the
// rate (8192 rows, 192 ranks, inner 4096: 105 us).  k_expand_large: a wave takes
// 32 rows with the batch rows as the matrix rows and columns numbered so that a
// lane has 16 bytes of a row and 16 lanes 256 neighbouring ones; B goes through
// LDS, shared by the four waves.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "attention.hpp"
#include "launch.hpp"

namespace fp8mi {
namespace {

using namespace attn;

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kSmall = 1024;         // rows up to which blocks sort for themselves
constexpr int kFew = 64;             // rows up to which a wave sorts for itself
constexpr int kFewRank = 64;         // ranks up to which these take one launch
constexpr int kSmallTile = 16, kLargeTile = 128;
constexpr int kBuckets = 1024;
constexpr int kStepK = 64;           // inner elements of a step
constexpr int kChunk = 64;           // small: output columns of a wave

struct LoraParams {
    const uint16_t* x;
    int64_t ldx;
    const uint16_t *a, *b;
    const int32_t* ids;
    const float* gain;
    const void* y;
    void* out;
    int64_t ldy, ldo;
    int rows, inner, rank, adapters, columns;
    int slices, width;               // width: slices * rank
    int ends[4];                     // first column behind each slice
    int block_ends[4];               // expand: first column block behind each slice
    int slots;                       // tiles that the sort may make
    int splits, split_steps;         // parts of the inner dimension, their steps
    int groups;                      // shrink: blocks that share the ranks
    int chunks;                      // expand, large: of a block
    int2* tiles;                     // [slots][tile]: row and adapter (-1: none); small: row -1 where there is none
    int* counts;                     // [slots], large: rows of a tile
    float* part;                     // [splits, rows, width]
};

__device__ __forceinline__ int id_of(const LoraParams& p, int m) {
    const int l = p.ids[m];
    return l >= 0 && l < p.adapters ? l : -1;
}
__device__ __forceinline__ int bucket_of(int id) { return (id + 1) & (kBuckets - 1); }

__device__ __forceinline__ int wave_scan(int v, int lane) {
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const int t = __shfl_up(v, off, 64);
        if (lane >= off) v += t;
    }
    return v;
}

// The slice of column block cb, its columns [first, end) and the block's place in it.
struct Slice {
    int index, first, end, block;
    __device__ __forceinline__ Slice(const LoraParams& p, int cb) : first(0), end(p.ends[0]), block(cb) {
        index = (cb >= p.block_ends[0] ? 1 : 0) + (cb >= p.block_ends[1] ? 1 : 0) + (cb >= p.block_ends[2] ? 1 : 0);
#pragma unroll
        for (int i = 1; i < 4; ++i)
            if (index == i) {
                first = p.ends[i - 1];
                end = p.ends[i];
                block = cb - p.block_ends[i - 1];
            }
    }
};

// How t's bf16 terms lie along the matrix steps over the ranks.  With a multiple
// of 32 ranks the terms follow each other against one piece of B; else terms and
// ranks are one axis, filled up with zeros.
struct Ranks {
    int groups, steps, terms, pitch;     // groups of 8 ranks; bytes of a row of t in LDS
    bool whole;
    __host__ __device__ __forceinline__ Ranks(int rank, int terms_) {
        groups = rank >> 3;
        whole = rank % 32 == 0;
        steps = whole ? rank / 32 : (terms_ * groups + 3) / 4;
        terms = whole ? terms_ : 1;
        pitch = (whole ? terms_ * rank : steps * 32) * 2 + 16;
    }
};

// Infinities.  A term of t is what rounding to bf16 gives, the next one what that
// leaves.  A finite value that would round to infinity takes the largest bf16 instead;
// an infinite one leaves nothing, not inf - inf.
constexpr float kFar = 0x1.FFp127f;                 // rounds to infinity from here on

// The terms of N values: put(k, words of term k).
template <int kTerms, int N, class Put>
__device__ __forceinline__ void split_terms(float (&t)[N], Put&& put) {
    float far = 0.0f;
#pragma unroll
    for (int e = 0; e < N; ++e) far = fmaxf(far, __builtin_fabsf(t[e]));
    uint32_t w[N / 2];
    if (__any(far >= kFar)) [[unlikely]] {
#pragma unroll
        for (int k = 0; k < kTerms; ++k) {
#pragma unroll
            for (int e = 0; e < N; e += 2) {
                const bool a = __builtin_isinf(t[e]), b = __builtin_isinf(t[e + 1]);
                uint32_t v = pack2(t[e], t[e + 1]);
                v -= !a && (v & 0x7FFFu) == 0x7F80u ? 1u : 0u;
                v -= !b && (v & 0x7FFF0000u) == 0x7F800000u ? 0x10000u : 0u;
                t[e] = a ? 0.0f : t[e] - as_f32(v << 16);
                t[e + 1] = b ? 0.0f : t[e + 1] - as_f32(v & 0xFFFF0000u);
                w[e / 2] = v;
            }
            put(k, w);
        }
        return;
    }
#pragma unroll
    for (int k = 0; k < kTerms; ++k) {
#pragma unroll
        for (int e = 0; e < N; e += 2) {
            w[e / 2] = pack2(t[e], t[e + 1]);
            t[e] -= as_f32(w[e / 2] << 16);
            t[e + 1] -= as_f32(w[e / 2] & 0xFFFF0000u);
        }
        put(k, w);
    }
}

// B without what is not finite.  Only t's first terms may meet the whole of B: the
// others, and the zeros behind them, would turn an infinite element into NaN (0 * inf,
// or the opposite infinity).  The products take all of B, and are formed once more,
// carefully, where they hold NaN, which such a meeting always leaves (looking for it:
// 0.1 us of 6 for one row, 1.6 of 114 for 4096 rows of 128 ranks, elsewhere less).
__device__ __forceinline__ b8 finite_of(b8 v) {
    u4 w = __builtin_bit_cast(u4, v);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = cleared<kBf16>(w[i], not_finite<kBf16>(w[i]));
    return __builtin_bit_cast(b8, w);
}

// Whether some lane of the wave holds NaN (or infinities of both signs).
template <int N>
__device__ __forceinline__ bool any_nan(const f4 (&v)[N]) {
    f4 sum = v[0];
#pragma unroll
    for (int i = 1; i < N; ++i) sum += v[i];
    const float one = (sum[0] + sum[1]) + (sum[2] + sum[3]);
    return __any(one != one);
}

// t of a tile's rows (their numbers: row_of(i)) for one adapter, as bf16 terms in LDS.
template <int kTerms, class RowOf>
__device__ __forceinline__ void put_t(const LoraParams& p, uint8_t* s_t, const Ranks& ranks, int rows, int slice,
                                      float gain, RowOf&& row_of) {
    const int groups = ranks.groups;
    for (int i = threadIdx.x; i < rows * groups; i += kThreads) {
        const int r = i / groups, q = i - r * groups, row = row_of(r);
        f4 lo = {0, 0, 0, 0}, hi = {0, 0, 0, 0};
        if (row >= 0) {
            const float* from = p.part + (int64_t)row * p.width + slice * p.rank + q * 8;
            const int64_t next = (int64_t)p.rows * p.width;
#pragma unroll 4
            for (int s = 0; s < p.splits; ++s) {
                lo += *reinterpret_cast<const f4*>(from + s * next);
                hi += *reinterpret_cast<const f4*>(from + s * next + 4);
            }
        }
        float t[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            t[e] = lo[e] * gain;
            t[4 + e] = hi[e] * gain;
        }
        split_terms<kTerms>(t, [&](int k, const uint32_t (&w)[4]) {
            *reinterpret_cast<uint4*>(s_t + r * ranks.pitch + (k * groups + q) * 16) = make_uint4(w[0], w[1], w[2], w[3]);
        });
    }
    const int fill = ranks.whole ? 0 : ranks.steps * 4 - kTerms * groups;
    for (int i = threadIdx.x; i < rows * fill; i += kThreads) {
        const int r = i / fill;
        *reinterpret_cast<uint4*>(s_t + r * ranks.pitch + (kTerms * groups + i - r * fill) * 16) =
            make_uint4(0, 0, 0, 0);
    }
}

// Eight neighbouring values of an output row, to which fp32 ones are added.
template <typename OutT>
struct Eight {
    uint4 w[sizeof(OutT) / 2];
    __device__ __forceinline__ void load(const OutT* p) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(OutT) / 2; ++i) w[i] = reinterpret_cast<const uint4*>(p)[i];
    }
    __device__ __forceinline__ void store(OutT* p) const {
#pragma unroll
        for (int i = 0; i < (int)sizeof(OutT) / 2; ++i) reinterpret_cast<uint4*>(p)[i] = w[i];
    }
    __device__ __forceinline__ void add(f4 lo, f4 hi) {
        if constexpr (sizeof(OutT) == 2) {
            auto two = [&](uint32_t v, float a, float b) {
                return pack2(as_f32(v << 16) + a, as_f32(v & 0xFFFF0000u) + b);
            };
            w[0] = make_uint4(two(w[0].x, lo[0], lo[1]), two(w[0].y, lo[2], lo[3]), two(w[0].z, hi[0], hi[1]),
                              two(w[0].w, hi[2], hi[3]));
        } else {
            auto one = [](uint32_t v, float a) { return __builtin_bit_cast(uint32_t, as_f32(v) + a); };
            w[0] = make_uint4(one(w[0].x, lo[0]), one(w[0].y, lo[1]), one(w[0].z, lo[2]), one(w[0].w, lo[3]));
            w[1] = make_uint4(one(w[1].x, hi[0]), one(w[1].y, hi[1]), one(w[1].z, hi[2]), one(w[1].w, hi[3]));
        }
    }
};

// ------------------------------------------------------------ small batches --
// The rows of tile `slot` where a wave holds all ids: the tile of row `slot`, if
// that is the first, 17th, .. of its adapter.  As pick_tile, every wave by itself.
__device__ __forceinline__ bool pick_few(const LoraParams& p, int slot, int* row, int* id) {
    const int lane = threadIdx.x & 63, mine = lane < p.rows ? id_of(p, lane) : -2;
    const uint64_t same = __ballot(mine == __builtin_amdgcn_readlane(mine, slot));
    const int rank = __popcll(same & ((1ull << slot) - 1)), n = __popcll(same) - rank;
    if (rank % kSmallTile != 0) return false;
    // lane i of the tile's takes the i-th of these rows from row `slot` on
    const int at = __popcll(same & ((1ull << lane) - 1)) - rank;
    const bool in = (same >> lane & 1) && at >= 0;
    const int from = __builtin_amdgcn_ds_permute((in ? at : 63) * 4, lane);
    *id = __builtin_amdgcn_readlane(mine, slot);
    *row = __shfl(from, lane & (kSmallTile - 1), 64);
    if ((lane & (kSmallTile - 1)) >= n) {
        *row = -1;
        *id = -2;
    }
    return true;
}

// The rows of tile `slot`, sorted by this block for itself: lane i (and i + 16,
// i + 32, i + 48) gets row i and its adapter, row -1 where there is none.
// Returns false where there is no such tile (for the whole block).
__device__ __forceinline__ bool pick_tile(const LoraParams& p, int slot, int* row, int* id) {
    if (p.rows <= kFew) return pick_few(p, slot, row, id);
    __shared__ int s_count[kBuckets];
    constexpr int kEach = kSmall / kThreads;
    __shared__ int s_sum[kWaves], s_found[2], s_in[kEach * kWaves];
    __shared__ int2 s_rows[kSmallTile];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    *reinterpret_cast<int4*>(&s_count[tid * 4]) = make_int4(0, 0, 0, 0);
    if (tid < kSmallTile) s_rows[tid] = make_int2(-1, -1);
    if (tid == 0) s_found[0] = -1;
    int ids[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) ids[i] = tid + i * kThreads < p.rows ? id_of(p, tid + i * kThreads) : -1;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kEach; ++i)
        if (tid + i * kThreads < p.rows) atomicAdd(&s_count[bucket_of(ids[i])], 1);
    __syncthreads();
    static_assert(kBuckets == 4 * kThreads, "four buckets a thread");
    const int4 n = *reinterpret_cast<const int4*>(&s_count[tid * 4]);
    const int t0 = (n.x + kSmallTile - 1) / kSmallTile, t1 = t0 + (n.y + kSmallTile - 1) / kSmallTile,
              t2 = t1 + (n.z + kSmallTile - 1) / kSmallTile, t3 = t2 + (n.w + kSmallTile - 1) / kSmallTile;
    const int sum = wave_scan(t3, lane);
    if (lane == 63) s_sum[wave] = sum;
    __syncthreads();
    int before = sum - t3;
#pragma unroll
    for (int w = 0; w < kWaves - 1; ++w) before += w < wave ? s_sum[w] : 0;
    const int at = slot - before;
    if (at >= 0 && at < t3) {
        const int k = (at >= t0 ? 1 : 0) + (at >= t1 ? 1 : 0) + (at >= t2 ? 1 : 0);
        s_found[0] = tid * 4 + k;
        s_found[1] = at - (k == 0 ? 0 : k == 1 ? t0 : k == 2 ? t1 : t2);
    }
    __syncthreads();
    const int bucket = s_found[0], first = s_found[1] * kSmallTile;
    if (bucket < 0) return false;
    // the bucket's rows in their order, the same in every block: 64 rows of every
    // wave after the other
    uint64_t in[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        in[i] = __ballot(tid + i * kThreads < p.rows && bucket_of(ids[i]) == bucket);
        if (lane == 0) s_in[i * kWaves + wave] = __popcll(in[i]);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        if (i * kThreads >= p.rows) break;
        int at = __popcll(in[i] & ((1ull << lane) - 1)) - first;
        for (int k = 0; k < i * kWaves + wave; ++k) at += s_in[k];
        if ((in[i] >> lane & 1) && at >= 0 && at < kSmallTile) s_rows[at] = make_int2(tid + i * kThreads, ids[i]);
    }
    __syncthreads();
    const int2 mine = s_rows[lane & (kSmallTile - 1)];
    *row = mine.x;
    *id = mine.x < 0 ? -2 : mine.y;
    return true;
}

__device__ __forceinline__ uint32_t lds_address(const void* p) {
    return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)p;
}

// 64 lanes x 16 bytes into LDS [lds, lds + 1024).  No register result: nothing in
// flight targets a register, and only the explicit waits below order it.
__device__ __forceinline__ void load_to_lds(uint32_t lds, const void* from) {
    asm volatile("s_mov_b32 m0, %0\n\tglobal_load_lds_dwordx4 %1, off"
                 :: "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(from) : "memory", "m0");
}

// acc[k] += rank tile k of A times a tile of x^T over this wave's steps of 64 inner
// elements (first, first + stride, ..).  The steps go through kStages stages of LDS
// of the wave's own, past the registers: a load takes 8 rows of 128 bytes (xp, ap:
// row lane / 8 of each), where read as matrix operands directly neighbouring lanes
// would touch different rows, which the caches serve at a quarter of the rate.  Of
// its row a lane loads the 16-byte piece that belongs at place lane % 8, pieces
// being turned by the row so that 16 rows' reads of one fall into different banks.
template <int RT, int kStages>
__device__ __forceinline__ void multiply_staged(uint8_t* mine, const uint16_t* const (&xp)[2],
                                                const uint16_t* const (&ap)[RT * 2], int first, int stride, int steps,
                                                int inner, f4 (&acc)[RT]) {
    constexpr int kStage = (RT + 1) * 2048, kUnits = (RT + 1) * 2;
    const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
    const int piece = ((lane & 7) ^ (lane >> 3)) * 8;
    auto stage = [&](int i) {
        const uint32_t to = lds_address(mine) + (uint32_t)(i % kStages) * kStage;
        const int e = (first + i * stride) * kStepK + piece, at = e < inner ? e : 0;
#pragma unroll
        for (int k = 0; k < 2; ++k) load_to_lds(to + k * 1024, xp[k] + at);
#pragma unroll
        for (int k = 0; k < RT * 2; ++k) load_to_lds(to + 2048 + k * 1024, ap[k] + at);
    };
    for (int i = 0; i < min(kStages, steps); ++i) stage(i);
    for (int i = 0; i < steps; ++i) {
        // stage i is here when no more than the loads of those after it are left
        if (i + kStages <= steps) asm volatile("s_waitcnt vmcnt(%0)" ::"n"((kStages - 1) * kUnits) : "memory");
        else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        const uint8_t* const from = mine + i % kStages * kStage;
        const int st = first + i * stride;
        uint4 xf[2], af[RT][2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int at = c * 128 + ((h * 4 + g) ^ (c & 7)) * 16;
            xf[h] = *reinterpret_cast<const uint4*>(from + at);
#pragma unroll
            for (int k = 0; k < RT; ++k) af[k][h] = *reinterpret_cast<const uint4*>(from + (k + 1) * 2048 + at);
        }
        if (i + kStages < steps) {                  // the stage is read: free for the next
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            stage(i + kStages);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if ((st + 1) * kStepK > inner) {        // nothing behind the end
                const uint32_t keep = st * kStepK + h * 32 + g * 8 < inner ? ~0u : 0u;
                auto cut = [&](uint4& w) { w = make_uint4(w.x & keep, w.y & keep, w.z & keep, w.w & keep); };
                cut(xf[h]);
#pragma unroll
                for (int k = 0; k < RT; ++k) cut(af[k][h]);
            }
#pragma unroll
            for (int k = 0; k < RT; ++k)
                acc[k] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(b8, af[k][h]),
                                                                 __builtin_bit_cast(b8, xf[h]), acc[k], 0, 0, 0);
        }
    }
}

constexpr int kSmallStages = 2;
constexpr int small_lds(int rt) { return kWaves * kSmallStages * (rt + 1) * 2048; }

template <int RT>
__global__ __launch_bounds__(kThreads, 2) void k_shrink_small(const LoraParams p) {
    extern __shared__ __align__(1024) uint8_t smem[];   // the waves' stages
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 15, g = lane >> 4;
    const int group = blockIdx.x % p.groups, split = blockIdx.x / p.groups % p.splits,
              slot = blockIdx.x / (p.groups * p.splits);
    int row, id;
    const bool any = pick_tile(p, slot, &row, &id);
    if (split == 0 && group == 0 && threadIdx.x < kSmallTile)
        p.tiles[slot * kSmallTile + threadIdx.x] = any ? make_int2(row, id) : make_int2(-1, -1);
    if (!any) return;
    const int rank0 = group * RT * 16;
    const int total = (p.inner + kStepK - 1) / kStepK;
    const int s_begin = split * p.split_steps, s_end = min(s_begin + p.split_steps, total);
    uint8_t* const mine = smem + wave * (small_lds(RT) / kWaves);
    const uint16_t* xp[2];                              // of row lane / 8 of a load of 1 KiB
#pragma unroll
    for (int i = 0; i < 2; ++i) xp[i] = p.x + (int64_t)max(__shfl(row, i * 8 + (lane >> 3), 64), 0) * p.ldx;
    uint64_t left = __ballot(id >= 0);
    while (left) {
        const int l = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
        const uint64_t same = __ballot(id == l);
        left &= ~same;
        const uint16_t* ap[RT * 2];
#pragma unroll
        for (int i = 0; i < RT * 2; ++i)
            ap[i] = p.a + ((int64_t)l * p.width + min(rank0 + i * 8 + (lane >> 3), p.width - 1)) * p.inner;
        f4 acc[RT];
#pragma unroll
        for (int i = 0; i < RT; ++i) acc[i] = f4{0, 0, 0, 0};
        // everything before is done, so the counts of the stages are of their loads alone
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        multiply_staged<RT, kSmallStages>(mine, xp, ap, s_begin + wave, kWaves,
                                          max(s_end - s_begin - wave + kWaves - 1, 0) / kWaves, p.inner, acc);
        // the waves' sums, each over its own stages
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
        for (int i = 0; i < RT; ++i) reinterpret_cast<f4*>(mine)[i * 64 + lane] = acc[i];
        __syncthreads();
        for (int i = wave; i < RT; i += kWaves) {
            const int rank = rank0 + i * 16 + g * 4;
            if (rank >= p.width || !(same >> c & 1)) continue;
            f4 sum = reinterpret_cast<const f4*>(smem)[i * 64 + lane];
#pragma unroll
            for (int w = 1; w < kWaves; ++w)
                sum += reinterpret_cast<const f4*>(smem + w * (small_lds(RT) / kWaves))[i * 64 + lane];
            *reinterpret_cast<f4*>(p.part + ((int64_t)split * p.rows + row) * p.width + rank) = sum;
        }
        if (left) __syncthreads();
    }
}

template <typename OutT>
__global__ __launch_bounds__(kThreads, 5) void k_expand_small(const LoraParams p) {
    constexpr int kTerms = sizeof(OutT) == 2 ? 2 : 3;
    extern __shared__ __align__(16) uint8_t s_t[];      // [16 rows][terms of t, padded] bf16
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 15, g = lane >> 4;
    const int column_blocks = p.block_ends[3], slot = blockIdx.x / column_blocks;
    const int2* const tile = p.tiles + slot * kSmallTile;
    const int row = tile[c].x, id = row < 0 ? -2 : tile[c].y;
    if (__ballot(row >= 0) == 0) return;
    const Slice slice(p, blockIdx.x % column_blocks);
    const int n0 = slice.first + (slice.block * kWaves + wave) * kChunk, end = slice.end;
    const int n = n0 + g * 16;                          // this lane's 16 columns
    const bool on[2] = {n < end && row >= 0, n + 8 < end && row >= 0};
    const Ranks ranks(p.rank, kTerms);
    const OutT* const y = static_cast<const OutT*>(p.y) + (int64_t)max(row, 0) * p.ldy;
    OutT* const out = static_cast<OutT*>(p.out) + (int64_t)max(row, 0) * p.ldo;
    Eight<OutT> v[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) v[h].load(y + (on[h] ? n + h * 8 : 0));
    uint64_t left = __ballot(id >= 0);
    bool again = false;
    while (left) {
        const int l = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
        const uint64_t same = __ballot(id == l);
        left &= ~same;
        // matrix row rho of piece j is column n0 + 16 (rho / 4) + 4 j + rho % 4
        const uint16_t* bp[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            bp[j] = p.b + ((int64_t)l * p.columns + min(n0 + (c >> 2) * 16 + j * 4 + (c & 3), end - 1)) * p.rank;
        if (again) __syncthreads();
        again = true;
        put_t<kTerms>(p, s_t, ranks, kSmallTile, slice.index, p.gain ? p.gain[l] : 1.0f,
                      [&](int r) { return tile[r].x; });
        __syncthreads();
        f4 acc[4];
        auto products = [&](auto careful) {
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[j] = f4{0, 0, 0, 0};
            for (int s = 0; s < ranks.steps; ++s) {
                const int q = ranks.whole ? s * 4 + g : (s * 4 + g) % ranks.groups;
                b8 bf[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) bf[j] = *reinterpret_cast<const b8*>(bp[j] + q * 8);
                for (int t = 0; t < ranks.terms; ++t) {
                    const int at = t * ranks.groups + s * 4 + g;
                    const b8 tf = *reinterpret_cast<const b8*>(s_t + c * ranks.pitch + at * 16);
                    if (careful && at >= ranks.groups) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) bf[j] = finite_of(bf[j]);
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bf[j], tf, acc[j], 0, 0, 0);
                }
            }
        };
        products(std::false_type());
        if (any_nan(acc)) [[unlikely]] products(std::true_type());
        if (id == l) {
#pragma unroll
            for (int h = 0; h < 2; ++h) v[h].add(acc[2 * h], acc[2 * h + 1]);
        }
    }
    // (rows without an adapter as they are)
    if (id >= 0 || (id == -1 && p.out != p.y)) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (on[h]) v[h].store(out + n + h * 8);
    }
}

// Up to kFew rows, ranks of RT tiles of 16: one launch.  A block takes a tile and
// 64 columns a wave of one slice (1024 with 16 waves up to 32 ranks, 512 with eight
// above) and forms the slice's t itself, its waves going through the inner dimension
// side by side: A is read by every column block again (from the caches), which costs
// less than a second launch and the partial sums' way through memory.  Each wave
// stages steps of x and A in LDS of its own, in the layout that multiply_staged
// explains: two steps up to 16 ranks, one above, where the other waves' loads stand
// beside a wave's wait.
constexpr int few_waves(int rt) { return rt <= 2 ? 16 : 8; }
constexpr int few_stages(int rt) { return rt == 1 ? 2 : 1; }
constexpr int few_lds(int rt) { return few_waves(rt) * few_stages(rt) * (rt + 1) * 2048; }

template <int RT, typename OutT>
__global__ __launch_bounds__(64 * few_waves(RT), 1) void k_lora_few(const LoraParams p) {
    constexpr int kTerms = sizeof(OutT) == 2 ? 2 : 3;
    constexpr int kFewWaves = few_waves(RT), kStages = few_stages(RT), kStage = (RT + 1) * 2048;
    extern __shared__ __align__(1024) uint8_t smem[];   // the waves' stages, then
    uint8_t* const s_t = smem + few_lds(RT);            // [16 rows][terms of t, padded] bf16
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int c = lane & 15, g = lane >> 4;
    const int column_blocks = p.block_ends[3], slot = blockIdx.x / column_blocks;
    int row, id;
    if (!pick_few(p, slot, &row, &id)) return;
    const Slice slice(p, blockIdx.x % column_blocks);
    const int n0 = slice.first + (slice.block * kFewWaves + wave) * kChunk, end = slice.end;
    const int n = n0 + g * 16;                          // this lane's 16 columns
    const bool on[2] = {n < end && row >= 0, n + 8 < end && row >= 0};
    const OutT* const y = static_cast<const OutT*>(p.y) + (int64_t)max(row, 0) * p.ldy;
    OutT* const out = static_cast<OutT*>(p.out) + (int64_t)max(row, 0) * p.ldo;
    Eight<OutT> v[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) v[h].load(y + (on[h] ? n + h * 8 : 0));
    const int l = __builtin_amdgcn_readfirstlane(id);   // (the tile's first row's, all rows')
    if (l < 0) {                                        // without an adapter: as they are
        if (p.out != p.y) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if (on[h]) v[h].store(out + n + h * 8);
        }
        return;
    }
    const Ranks ranks(p.rank, kTerms);
    // matrix row rho of piece j is column n0 + 16 (rho / 4) + 4 j + rho % 4
    const uint16_t* bp[4];
    b8 bf[4];
    auto load_b = [&](int s) {
        const int q = ranks.whole ? s * 4 + g : (s * 4 + g) % ranks.groups;
#pragma unroll
        for (int j = 0; j < 4; ++j) bf[j] = *reinterpret_cast<const b8*>(bp[j] + q * 8);
    };
#pragma unroll
    for (int j = 0; j < 4; ++j)
        bp[j] = p.b + ((int64_t)l * p.columns + min(n0 + (c >> 2) * 16 + j * 4 + (c & 3), end - 1)) * p.rank;
    load_b(0);
    const float gain = p.gain ? p.gain[l] : 1.0f;

    const uint16_t *xp[2], *ap[RT * 2];                 // of row lane / 8 of a load of 1 KiB
#pragma unroll
    for (int i = 0; i < 2; ++i) xp[i] = p.x + (int64_t)max(__shfl(row, i * 8 + (lane >> 3), 64), 0) * p.ldx;
#pragma unroll
    for (int i = 0; i < RT * 2; ++i)
        ap[i] = p.a + ((int64_t)l * p.width + slice.index * p.rank + min(i * 8 + (lane >> 3), p.rank - 1)) * p.inner;
    f4 acc[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) acc[i] = f4{0, 0, 0, 0};
    const int total = (p.inner + kStepK - 1) / kStepK;
    uint8_t* const mine = smem + wave * kStages * kStage;
    multiply_staged<RT, kStages>(mine, xp, ap, wave, kFewWaves, (total - wave + kFewWaves - 1) / kFewWaves, p.inner, acc);
    // this wave's sums, over its own stages
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
    for (int i = 0; i < RT; ++i) reinterpret_cast<f4*>(mine)[i * 64 + lane] = acc[i];
    // zeros behind t's last term
    const int fill = ranks.whole ? 0 : ranks.steps * 4 - kTerms * ranks.groups;
    if (tid < 16 * fill) {
        const int r = tid / fill;
        *reinterpret_cast<uint4*>(s_t + r * ranks.pitch + (kTerms * ranks.groups + tid - r * fill) * 16) =
            make_uint4(0, 0, 0, 0);
    }
    __syncthreads();
    // four ranks of a row a thread: the waves' sums, in bf16 terms
    if (tid < RT * 64) {
        f4 t = reinterpret_cast<const f4*>(smem)[tid];
#pragma unroll
        for (int w = 1; w < kFewWaves; ++w) t += reinterpret_cast<const f4*>(smem + w * kStages * kStage)[tid];
        t *= gain;
        const int rank = (tid >> 6) * 16 + g * 4;       // (of row c)
        if (rank < p.rank) {
            float e[4] = {t[0], t[1], t[2], t[3]};
            split_terms<kTerms>(e, [&](int k, const uint32_t (&w)[2]) {
                *reinterpret_cast<uint2*>(s_t + c * ranks.pitch + (k * p.rank + rank) * 2) = make_uint2(w[0], w[1]);
            });
        }
    }
    __syncthreads();
    if (n0 >= end) return;
    f4 sum[4];
    auto products = [&](auto careful) {
#pragma unroll
        for (int j = 0; j < 4; ++j) sum[j] = f4{0, 0, 0, 0};
        for (int s = 0; s < ranks.steps; ++s) {
            if (careful || s > 0) load_b(s);
            for (int t = 0; t < ranks.terms; ++t) {
                const int at = t * ranks.groups + s * 4 + g;
                const b8 tf = *reinterpret_cast<const b8*>(s_t + c * ranks.pitch + at * 16);
                if (careful && at >= ranks.groups) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) bf[j] = finite_of(bf[j]);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    sum[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bf[j], tf, sum[j], 0, 0, 0);
            }
        }
    };
    products(std::false_type());
    if (any_nan(sum)) [[unlikely]] products(std::true_type());
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        v[h].add(sum[2 * h], sum[2 * h + 1]);
        if (on[h]) v[h].store(out + n + h * 8);
    }
}

// ------------------------------------------------------------ large batches --
// Sorts the rows into tiles: one block.
constexpr int kSortThreads = 1024;

// Adds every lane's row to its bucket's counter and returns the row's place: one
// addition where all 64 agree, which in prompts is most often so (one for each
// lane, 8192 rows of 8 adapters: 19 us against 11).
__device__ __forceinline__ int count_in(int* s_count, int bucket, bool on) {
    const int lane = threadIdx.x & 63;
    const uint64_t all = __ballot(on);
    if (all == 0) return 0;
    const int b = __builtin_amdgcn_readlane(bucket, __builtin_ctzll(all));
    int place = 0;
    if (__ballot(on && bucket == b) == all) {
        if (lane == 0) place = atomicAdd(&s_count[b], __popcll(all));
        return __builtin_amdgcn_readfirstlane(place) + __popcll(all & ((1ull << lane) - 1));
    }
    if (on) place = atomicAdd(&s_count[bucket], 1);
    return place;
}

__global__ __launch_bounds__(kSortThreads) void k_sort_rows(const LoraParams p) {
    constexpr int kRound = 8;               // rows of a thread that are on their way together
    __shared__ int s_count[kBuckets], s_first[kBuckets + 1];
    __shared__ int s_sum[kSortThreads / 64];
    static_assert(kBuckets == kSortThreads, "a bucket a thread");
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    s_count[tid] = 0;
    __syncthreads();
    int ids[kRound], place[kRound];
    auto load = [&](int m0) {
#pragma unroll
        for (int i = 0; i < kRound; ++i) {
            const int m = m0 + i * kSortThreads + tid;
            ids[i] = m < p.rows ? id_of(p, m) : -1;
        }
    };
    for (int m0 = 0; m0 < p.rows; m0 += kRound * kSortThreads) {
        load(m0);
#pragma unroll
        for (int i = 0; i < kRound; ++i)
            place[i] = count_in(s_count, bucket_of(ids[i]), m0 + i * kSortThreads + tid < p.rows);
    }
    __syncthreads();
    const int n = s_count[tid], tiles = (n + kLargeTile - 1) / kLargeTile;
    const int sum = wave_scan(tiles, lane);
    if (lane == 63) s_sum[wave] = sum;
    __syncthreads();
    int first = sum - tiles;
    for (int w = 0; w < wave; ++w) first += s_sum[w];
    s_first[tid] = first;
    if (tid == kBuckets - 1) s_first[kBuckets] = first + tiles;
    __syncthreads();
    for (int slot = tid; slot < p.slots; slot += kSortThreads) {
        // the last bucket whose tiles begin at or before this one
        int b = 0;
#pragma unroll
        for (int step = kBuckets / 2; step > 0; step >>= 1)
            if (s_first[b + step] <= slot) b += step;
        p.counts[slot] =
            slot < s_first[kBuckets] ? min(s_count[b] - (slot - s_first[b]) * kLargeTile, kLargeTile) : 0;
    }
    // (a row's place in its bucket follows the order of the additions; no result does)
    const bool again = p.rows > kRound * kSortThreads;
    if (again) {
        __syncthreads();
        s_count[tid] = 0;
        __syncthreads();
    }
    for (int m0 = 0; m0 < p.rows; m0 += kRound * kSortThreads) {
        if (again) load(m0);
#pragma unroll
        for (int i = 0; i < kRound; ++i) {
            const int m = m0 + i * kSortThreads + tid, b = bucket_of(ids[i]);
            if (again) place[i] = count_in(s_count, b, m < p.rows);
            if (m < p.rows) p.tiles[s_first[b] * kLargeTile + place[i]] = make_int2(m, ids[i]);
        }
    }
}

// Two waves a SIMD, so that one's reads of LDS stand beside the other's products:
// two halves of the rows by four quarters of the ranks, RT rank tiles each.
constexpr int kShrinkWaves = 8;

template <int RT>
__global__ __launch_bounds__(64 * kShrinkWaves, 1) void k_shrink_large(const LoraParams p) {
    constexpr int kStages = 3, kRow = kStepK * 2;                   // bytes of a row of a stage
    constexpr int kX = kLargeTile * kRow, kStage = kX + 4 * RT * 16 * kRow;
    // 1 KiB loads of a wave: 8 rows each
    constexpr int kXUnits = kLargeTile / 8 / kShrinkWaves, kAUnits = RT;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 15, g = lane >> 4;
    // neighbouring tiles, which often share an adapter, on one XCD (blocks go
    // round the eight) for its L2 to hold A
    const int unit = blockIdx.x >> 3, each = p.groups * p.splits;
    const int group = unit % p.groups, split = unit / p.groups % p.splits;
    const int slot = (int)(blockIdx.x & 7) * ((p.slots + 7) / 8) + unit / each;
    if (slot >= p.slots || unit / each >= (p.slots + 7) / 8) return;
    const int2* const tile = p.tiles + (int64_t)slot * kLargeTile;
    const int count = p.counts[slot];
    if (count == 0) return;
    const int id_a = lane < count ? tile[lane].y : -2, id_b = 64 + lane < count ? tile[64 + lane].y : -2;
    const int rank0 = group * RT * 64;
    const int total = (p.inner + kStepK - 1) / kStepK;
    const int s_begin = split * p.split_steps, s_end = min(s_begin + p.split_steps, total);
    const int quarter = wave & 3, rows0 = (wave >> 2) * 64;         // this wave's ranks and rows

    // What a lane loads: of row lane / 8 of a unit the 16-byte piece that belongs
    // at place lane % 8, pieces being turned by the row so that 16 rows' reads of
    // one piece fall into different banks.
    const int piece = ((lane & 7) ^ (lane >> 3)) * 8;
    const uint16_t* xp[kXUnits];
#pragma unroll
    for (int i = 0; i < kXUnits; ++i) {
        const int row = tile[min((wave * kXUnits + i) * 8 + (lane >> 3), count - 1)].x;
        xp[i] = p.x + (int64_t)row * p.ldx;
    }
    uint64_t left_a = __ballot(id_a >= 0), left_b = __ballot(id_b >= 0);
    while (left_a | left_b) {
        const int l = left_a ? __builtin_amdgcn_readlane(id_a, __builtin_ctzll(left_a))
                             : __builtin_amdgcn_readlane(id_b, __builtin_ctzll(left_b));
        const uint64_t same_a = __ballot(id_a == l), same_b = __ballot(id_b == l);
        left_a &= ~same_a;
        left_b &= ~same_b;
        const uint16_t* ap[kAUnits];
#pragma unroll
        for (int i = 0; i < kAUnits; ++i) {
            const int rank = min(rank0 + (wave * kAUnits + i) * 8 + (lane >> 3), p.width - 1);
            ap[i] = p.a + ((int64_t)l * p.width + rank) * p.inner;
        }
        auto stage = [&](int st) {
            const uint32_t to = lds_address(smem) + (uint32_t)((st - s_begin) % kStages) * kStage;
            const int e = st * kStepK + piece, at = e < p.inner ? e : 0;
#pragma unroll
            for (int i = 0; i < kXUnits; ++i) load_to_lds(to + (wave * kXUnits + i) * 1024, xp[i] + at);
#pragma unroll
            for (int i = 0; i < kAUnits; ++i) load_to_lds(to + kX + (wave * kAUnits + i) * 1024, ap[i] + at);
        };
        f4 acc[RT][4];
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) acc[i][k] = f4{0, 0, 0, 0};
        // everything loaded before is here, so the counts below are of the stages alone
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
        if (s_begin < s_end) stage(s_begin);
        if (s_begin + 1 < s_end) stage(s_begin + 1);
        for (int st = s_begin; st < s_end; ++st) {
            // this stage has arrived, in all waves; the one read last is free for the next but one
            if (st + 1 < s_end)
                asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(kXUnits + kAUnits) : "memory");
            else
                asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
            if (st + 2 < s_end) stage(st + 2);
            const uint8_t* const from = smem + (st - s_begin) % kStages * kStage;
            const bool cut = (st + 1) * kStepK > p.inner;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int at = ((h * 4 + g) ^ (c & 7)) * 16;
                uint4 xf[4], af[RT];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    xf[k] = *reinterpret_cast<const uint4*>(from + (rows0 + k * 16 + c) * kRow + at);
#pragma unroll
                for (int i = 0; i < RT; ++i)
                    af[i] = *reinterpret_cast<const uint4*>(from + kX + ((quarter * RT + i) * 16 + c) * kRow + at);
                if (cut) {                                          // nothing behind the end
                    const uint32_t keep = st * kStepK + h * 32 + g * 8 < p.inner ? ~0u : 0u;
                    auto clear = [&](uint4& w) { w = make_uint4(w.x & keep, w.y & keep, w.z & keep, w.w & keep); };
#pragma unroll
                    for (int k = 0; k < 4; ++k) clear(xf[k]);
#pragma unroll
                    for (int i = 0; i < RT; ++i) clear(af[i]);
                }
#pragma unroll
                for (int i = 0; i < RT; ++i)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        acc[i][k] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            __builtin_bit_cast(b8, af[i]), __builtin_bit_cast(b8, xf[k]), acc[i][k], 0, 0, 0);
            }
        }
        const uint64_t same = rows0 ? same_b : same_a;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (!(same >> (k * 16 + c) & 1)) continue;
            float* const to = p.part + ((int64_t)split * p.rows + tile[rows0 + k * 16 + c].x) * p.width;
#pragma unroll
            for (int i = 0; i < RT; ++i) {
                const int rank = rank0 + (quarter * RT + i) * 16 + g * 4;
                if (rank < p.width) *reinterpret_cast<f4*>(to + rank) = acc[i][k];
            }
        }
    }
}

// Columns of a step: 8 neighbouring ones a lane in bf16, 4 in fp32.
template <typename OutT> constexpr int kEach = sizeof(OutT) == 2 ? 8 : 4;

template <typename OutT>
__global__ __launch_bounds__(kThreads, 2) void k_expand_large(const LoraParams p) {
    constexpr int kTerms = sizeof(OutT) == 2 ? 2 : 3, J = kEach<OutT>, kCols = 16 * J;
    extern __shared__ __align__(16) uint8_t smem[];     // t of 128 rows, then two steps' B
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int c = lane & 15, g = lane >> 4;
    const int column_blocks = p.block_ends[3], slot = blockIdx.x / column_blocks;
    const int2* const tile = p.tiles + (int64_t)slot * kLargeTile;
    const int count = p.counts[slot];
    if (count == 0) return;
    const Slice slice(p, blockIdx.x % column_blocks);
    const int n_begin = slice.first + slice.block * p.chunks * kCols, n_end = min(n_begin + p.chunks * kCols, slice.end);
    const Ranks ranks(p.rank, kTerms);
    uint8_t* const s_b = smem + kLargeTile * ranks.pitch;
    const int b_bytes = kCols * p.rank * 2, pieces = J * 16 * ranks.groups;
    const OutT* const y = static_cast<const OutT*>(p.y);
    OutT* const out = static_cast<OutT*>(p.out);

    // this lane's rows: 4 g + i of the wave's two matrix tiles
    int rows[2][4], ids[2][4];
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int at = wave * 32 + k * 16 + g * 4 + i;
            const int2 e = tile[min(at, count - 1)];
            rows[k][i] = e.x;
            ids[k][i] = at < count ? e.y : -2;
        }
    auto load_y = [&](uint4 (&v)[2][4], int n0) {
        const int n = n0 + c * J < n_end ? n0 + c * J : n_begin;
        int none = 0;
        asm volatile("" : "+v"(none));              // addresses anew each step, not kept in registers
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[k][i] = __builtin_bit_cast(
                    uint4, __builtin_nontemporal_load(reinterpret_cast<const u4*>(y + (rows[k][i] + none) * p.ldy + n)));
    };
    auto store = [&](const uint4& v, int k, int i, int n0) {
        int none = 0;
        asm volatile("" : "+v"(none));
        if (n0 + c * J < n_end)
            __builtin_nontemporal_store(__builtin_bit_cast(u4, v),
                                        reinterpret_cast<u4*>(out + (rows[k][i] + none) * p.ldo + n0 + c * J));
    };

    const int id_a = lane < count ? tile[lane].y : -2, id_b = 64 + lane < count ? tile[64 + lane].y : -2;
    // rows without an adapter stay as they are
    if (p.out != p.y && __any(id_a == -1 || id_b == -1))
        for (int n = n_begin + c * J; n < n_end; n += kCols)
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (ids[k][i] == -1)
                        *reinterpret_cast<uint4*>(out + rows[k][i] * p.ldo + n) =
                            *reinterpret_cast<const uint4*>(y + rows[k][i] * p.ldy + n);
    uint64_t left_a = __ballot(id_a >= 0), left_b = __ballot(id_b >= 0);
    bool again = false;
    while (left_a | left_b) {
        const int l = left_a ? __builtin_amdgcn_readlane(id_a, __builtin_ctzll(left_a))
                             : __builtin_amdgcn_readlane(id_b, __builtin_ctzll(left_b));
        left_a &= ~__ballot(id_a == l);
        left_b &= ~__ballot(id_b == l);
        const uint16_t* const b = p.b + (int64_t)l * p.columns * p.rank;
        // B of a step into LDS: piece (j, q, c) is ranks 8 q.. of column n0 + c J + j
        auto stage_b = [&](int n0, int buf) {
            for (int i = tid; i < pieces; i += kThreads) {          // (whole waves)
                const int jq = i >> 4, j = jq / ranks.groups, q = jq - j * ranks.groups;
                const int n = min(n0 + (i & 15) * J + j, slice.end - 1);
                load_to_lds(lds_address(s_b) + buf * b_bytes + (i & ~63) * 16, b + (int64_t)n * p.rank + q * 8);
            }
        };
        if (again) __syncthreads();
        again = true;
        uint4 v[2][4];                              // y, on its way during the step before
        stage_b(n_begin, 0);
        load_y(v, n_begin);
        put_t<kTerms>(p, smem, ranks, kLargeTile, slice.index, p.gain ? p.gain[l] : 1.0f,
                      [&](int r) { return r < count ? tile[r].x : -1; });
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
        int buf = 0;
        for (int n0 = n_begin; n0 < n_end; n0 += kCols, buf ^= 1) {
            const bool more = n0 + kCols < n_end;
            if (more) stage_b(n0 + kCols, buf ^ 1);
            f4 acc[2][J];
            auto products = [&](auto careful) {
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int j = 0; j < J; ++j) acc[k][j] = f4{0, 0, 0, 0};
                for (int s = 0; s < ranks.steps; ++s) {
                    const int q = ranks.whole ? s * 4 + g : (s * 4 + g) % ranks.groups;
                    b8 bf[J];
#pragma unroll
                    for (int j = 0; j < J; ++j)
                        bf[j] =
                            *reinterpret_cast<const b8*>(s_b + buf * b_bytes + ((j * ranks.groups + q) * 16 + c) * 16);
                    for (int t = 0; t < ranks.terms; ++t) {
                        const int at = t * ranks.groups + s * 4 + g;
                        if (careful && at >= ranks.groups) {
#pragma unroll
                            for (int j = 0; j < J; ++j) bf[j] = finite_of(bf[j]);
                        }
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const b8 tf = *reinterpret_cast<const b8*>(
                                smem + (wave * 32 + k * 16 + c) * ranks.pitch + at * 16);
#pragma unroll
                            for (int j = 0; j < J; ++j)
                                acc[k][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(tf, bf[j], acc[k][j], 0, 0, 0);
                        }
                    }
                }
            };
            products(std::false_type());
            if (any_nan(acc[0]) | any_nan(acc[1])) [[unlikely]] products(std::true_type());
            // y of this step and B of the next are here
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (ids[k][i] != l) continue;
                    uint4 w = v[k][i];
                    if constexpr (sizeof(OutT) == 2) {
                        auto two = [&](uint32_t v, float a, float d) {
                            return pack2(as_f32(v << 16) + a, as_f32(v & 0xFFFF0000u) + d);
                        };
                        w = make_uint4(two(w.x, acc[k][0][i], acc[k][1][i]), two(w.y, acc[k][2][i], acc[k][3][i]),
                                       two(w.z, acc[k][J - 4][i], acc[k][J - 3][i]),
                                       two(w.w, acc[k][J - 2][i], acc[k][J - 1][i]));
                    } else {
                        auto one = [](uint32_t v, float a) { return __builtin_bit_cast(uint32_t, as_f32(v) + a); };
                        w = make_uint4(one(w.x, acc[k][0][i]), one(w.y, acc[k][1][i]), one(w.z, acc[k][2][i]),
                                       one(w.w, acc[k][3][i]));
                    }
                    store(w, k, i, n0);
                }
            if (more) load_y(v, n0 + kCols);
            asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        }
    }
}

// How a call is shared out.
struct Plan {
    bool few, small;
    int slots, tile;                 // tiles that the sort may make, rows of one
    int rank_tiles, groups, splits, split_steps;
    int64_t shrink_blocks;
};

Plan plan_of(const LoraArgs& a) {
    Plan p;
    p.small = a.rows <= kSmall;
    // One launch where its blocks are resident together and a block's pass over the
    // inner dimension, which grows with the rows of A and x, is shorter than a
    // second launch (1 .. 64 rows, 6144 columns: 16 ranks of inner 4096 in 6.0 .. 6.8
    // us against 7.8 .. 9.1, of 8192 in 8.0 .. 11.7 against 8.1 .. 10.8; 32 ranks of
    // 4096 in 7.4 .. 11.9 against 8.5 .. 10.4, of 8192 in 10 .. 18 against 9 .. 16; 64
    // ranks of 2048 in 7.3 .. 8.6 against 8.4 .. 9.2, of 8192 in 14 .. 23 against 10
    // .. 13; in two rounds of blocks, 14336 columns, 13 against 11).  A second launch
    // costs the host 3 us more.  The grid has blocks for a tile of every row, most of
    // them empty: where an adapter's first row is among the last, its blocks wait for
    // empty ones of the first round (64 rows of 24 adapters 7.0 .. 8.0 us by the order
    // of the ids, 11.5 with one adapter in the last row alone).
    const int tiles_of_16 = (int)std::min<int64_t>(a.rows, (a.rows + 15) / 16 + a.adapters), rt = (a.rank + 15) / 16;
    p.few = a.rows <= kFew && a.rank <= kFewRank && a.inner * (rt == 3 ? 5 : rt + 1) <= 16384 &&
            tiles_of_16 * (a.columns / (few_waves(rt) * kChunk) + a.slices) <= 256;
    p.tile = p.small ? kSmallTile : kLargeTile;
    p.slots = a.rows <= kFew ? (int)a.rows
                             : (int)(a.rows / p.tile + std::min<int64_t>({a.rows, (int64_t)a.adapters + 1, kBuckets}));
    const int ranks = (a.slices * a.rank + 15) / 16, steps = (int)((a.inner + kStepK - 1) / kStepK);
    int splits;
    if (p.small) {
        p.groups = (ranks + 5) / 6;
        p.rank_tiles = (ranks + p.groups - 1) / p.groups;
        if (p.rank_tiles == 5) p.rank_tiles = 6;
        // Parts of the inner dimension: about a block a CU for the tiles that rows
        // spread evenly over the adapters make, every wave with a step or more, and
        // no more than 16 rows of t for the second launch to add.  A power of two:
        // blocks go round the eight XCDs, so that each one's L2 then holds the same
        // part of A for all tiles (700 rows of 8 adapters, 32 ranks, inner 14336:
        // four parts 16.8 us, five 20.7; 331 rows of 12: eight 12.2, six 14.9).
        const double each = (double)a.rows / a.adapters;            // rows of an adapter, spread evenly
        const int64_t expected = (int64_t)(a.adapters * std::max(1 - std::exp(-each), each / 16 + 0.5));
        const int tiles = (int)std::clamp<int64_t>(expected, 1, std::min(p.slots, tiles_of_16));
        splits = std::clamp(256 / (tiles * p.groups), 1, 16);
        while (splits & (splits - 1)) splits &= splits - 1;
    } else {
        p.groups = (ranks + 11) / 12;
        p.rank_tiles = ((ranks + p.groups - 1) / p.groups + 3) / 4;
        // Blocks take a CU each: whole rounds of 256, and one round where it can be.
        const int64_t blocks = (int64_t)p.slots * p.groups;
        splits = (int)std::clamp<int64_t>((blocks <= 128 ? 256 : 512) / blocks, 1, 8);
    }
    const int waves = p.small ? kWaves : 1, turn = splits * waves;     // whole turns of the waves
    p.split_steps = std::max((steps + turn - 1) / turn * waves, kWaves);
    p.splits = std::max(1, (steps + p.split_steps - 1) / p.split_steps);
    p.shrink_blocks = (int64_t)(p.small ? p.slots : (p.slots + 7) / 8 * 8) * p.splits * p.groups;
    return p;
}

int64_t tile_bytes(const Plan& p) { return (int64_t)p.slots * p.tile * 8; }
int64_t count_bytes(const Plan& p) { return p.small ? 0 : ((int64_t)p.slots * 4 + 15) / 16 * 16; }

// Column blocks of the second launch.
template <typename OutT>
int64_t column_blocks(const LoraArgs& a, const Plan& plan, int* chunks, int (&ends)[4]) {
    const int cols = plan.few ? few_waves((a.rank + 15) / 16) * kChunk : plan.small ? kWaves * kChunk : 16 * kEach<OutT>;
    auto count = [&](int run, int64_t tiles) {
        int blocks = 0;
        for (int i = 0; i < 4; ++i) {
            const int n = i < a.slices ? a.columns_of[i] : 0;
            blocks += (n + run - 1) / run;
            ends[i] = blocks;
        }
        return blocks * tiles;
    };
    *chunks = 1;
    if (!plan.small) {
        // One resident round of two blocks a CU where runs of up to 16 steps allow
        // (a block's rows of t are read once for its run): 8192 rows of 6144
        // columns in 438 blocks 51 us, in 657 63, in 876 63, in 365 61.
        // Of the slots about half of those that adapters' last tiles may need are
        // empty (3818 rows of 47 adapters, 6280 columns of fp32: 94 us with all of
        // them counted, 85 so).
        const int most = 16;
        const int64_t full = a.rows / plan.tile, tiles = full + (plan.slots - full + 1) / 2;
        while (*chunks < most && count(cols * *chunks, tiles) > 512) ++*chunks;
    }
    return count(cols * *chunks, plan.slots);
}

template <int RT>
hipError_t shrink_large(const LoraParams& p, const Plan& plan, hipStream_t stream) {
    constexpr int bytes = 3 * (kLargeTile + 64 * RT) * kStepK * 2;
    static_assert(bytes <= 160 * 1024, "LDS");
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&k_shrink_large<RT>),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((k_shrink_large<RT>), dim3((unsigned)plan.shrink_blocks), dim3(64 * kShrinkWaves), bytes, stream,
                       p);
    return hipGetLastError();
}

template <int RT>
hipError_t shrink_small(const LoraParams& p, const Plan& plan, hipStream_t stream) {
    constexpr int bytes = small_lds(RT);
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&k_shrink_small<RT>),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((k_shrink_small<RT>), dim3((unsigned)plan.shrink_blocks), dim3(kThreads), bytes, stream, p);
    return hipGetLastError();
}

hipError_t run_shrink(const LoraParams& p, const Plan& plan, hipStream_t stream) {
    if (!plan.small)
        return plan.rank_tiles == 1   ? shrink_large<1>(p, plan, stream)
               : plan.rank_tiles == 2 ? shrink_large<2>(p, plan, stream)
                                      : shrink_large<3>(p, plan, stream);
    switch (plan.rank_tiles) {
    case 1: return shrink_small<1>(p, plan, stream);
    case 2: return shrink_small<2>(p, plan, stream);
    case 3: return shrink_small<3>(p, plan, stream);
    case 4: return shrink_small<4>(p, plan, stream);
    default: return shrink_small<6>(p, plan, stream);
    }
}

template <typename OutT>
hipError_t run_few(const LoraArgs& a, LoraParams& p, const Plan& plan, hipStream_t stream) {
    const dim3 grid((unsigned)column_blocks<OutT>(a, plan, &p.chunks, p.block_ends));
    const auto launch = [&](auto rt) {
        constexpr int kRT = decltype(rt)::value;
        const int bytes = few_lds(kRT) + kSmallTile * Ranks(p.rank, sizeof(OutT) == 2 ? 2 : 3).pitch;
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&k_lora_few<kRT, OutT>),
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL((k_lora_few<kRT, OutT>), grid, dim3(64 * few_waves(kRT)), bytes, stream, p);
        return hipGetLastError();
    };
    if (p.rank <= 16) return launch(std::integral_constant<int, 1>());
    if (p.rank <= 32) return launch(std::integral_constant<int, 2>());
    return launch(std::integral_constant<int, 4>());
}

template <typename OutT>
hipError_t run_expand(const LoraArgs& a, LoraParams& p, const Plan& plan, hipStream_t stream) {
    const int64_t blocks = column_blocks<OutT>(a, plan, &p.chunks, p.block_ends);
    const Ranks ranks(p.rank, sizeof(OutT) == 2 ? 2 : 3);
    const dim3 grid((unsigned)blocks), block(kThreads);
    if (plan.small) {
        hipLaunchKernelGGL((k_expand_small<OutT>), grid, block, kSmallTile * ranks.pitch, stream, p);
        return hipGetLastError();
    }
    const int bytes = kLargeTile * ranks.pitch + 2 * 16 * kEach<OutT> * p.rank * 2;
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&k_expand_large<OutT>),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, 160 * 1024);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((k_expand_large<OutT>), grid, block, bytes, stream, p);
    return hipGetLastError();
}

}  // namespace

int64_t lora_workspace(const LoraArgs& a) {
    if (a.rows == 0) return 0;
    const Plan p = plan_of(a);
    if (p.few) return 0;
    return tile_bytes(p) + count_bytes(p) + (int64_t)p.splits * a.rows * a.slices * a.rank * 4;
}

// The largest launch in blocks of kThreads threads (2^32 threads and more are
// not launched): k_shrink_large has twice as many, k_lora_few's few blocks are far
// below their count here.
int64_t lora_blocks(const LoraArgs& a) {
    const Plan plan = plan_of(a);
    return std::max(plan.shrink_blocks * (plan.small ? 1 : kShrinkWaves / kWaves),
                    (int64_t)plan.slots * (a.columns / 64 + a.slices));
}

hipError_t launch_lora(const LoraArgs& a) {
    const Plan plan = plan_of(a);
    LoraParams p;
    p.x = a.x; p.ldx = a.ldx; p.a = a.a; p.b = a.b; p.ids = a.ids; p.gain = a.gain; p.y = a.y; p.out = a.out;
    p.ldy = a.ldy; p.ldo = a.ldo; p.rows = (int)a.rows; p.inner = (int)a.inner; p.rank = a.rank;
    p.adapters = a.adapters; p.columns = (int)a.columns; p.slices = a.slices; p.width = a.slices * a.rank;
    int end = 0;
    for (int i = 0; i < 4; ++i) {
        end += i < a.slices ? a.columns_of[i] : 0;
        p.ends[i] = end;
    }
    p.slots = plan.slots; p.splits = plan.splits; p.split_steps = plan.split_steps; p.groups = plan.groups;
    p.tiles = reinterpret_cast<int2*>(a.workspace);
    p.counts = reinterpret_cast<int*>(a.workspace + tile_bytes(plan));
    p.part = reinterpret_cast<float*>(a.workspace + tile_bytes(plan) + count_bytes(plan));
    if (plan.few)
        return a.out_bf16 ? run_few<uint16_t>(a, p, plan, a.stream) : run_few<float>(a, p, plan, a.stream);
    if (!plan.small) {
        hipLaunchKernelGGL(k_sort_rows, dim3(1), dim3(kSortThreads), 0, a.stream, p);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    const hipError_t e = run_shrink(p, plan, a.stream);
    if (e != hipSuccess) return e;
    return a.out_bf16 ? run_expand<uint16_t>(a, p, plan, a.stream) : run_expand<float>(a, p, plan, a.stream);
}

}  // namespace fp8mi
