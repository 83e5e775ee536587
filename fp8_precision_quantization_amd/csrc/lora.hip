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
// Two launches.  k_lora_shrink: a block takes a tile of rows that share an
// adapter and a part of the inner dimension, whose steps go round its four
// waves, so that neither x nor A is read twice by a block; the parts' sums go to
// the workspace.  k_lora_expand: a block takes a row tile and a run of columns
// of one slice, adds up the parts of t (in their order) and adds B t to y.
// Products are 16x16x32 with ranks (columns of the output) as the matrix rows
// and batch rows as its columns; a wave's 64 columns of the output are numbered
// so that a lane gets 16 neighbouring ones of a row.
//
// Row tiles.  Up to kGathered rows, a tile is up to 16 rows with one adapter,
// wherever they are in the batch: every wave looks through the ids by itself and
// block i goes on if its row i is the first, 17th, .. of its adapter.  (A decode
// step of many users.)  Larger batches hold prompts, whose rows lie together: a
// tile is 64 neighbouring rows, and the adapters among them are taken one after
// the other.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "attention.hpp"
#include "launch.hpp"

namespace fp8mi {
namespace {

using namespace attn;

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kGathered = 1024;      // rows up to which a tile's rows may lie anywhere
constexpr int kStepK = 64;           // inner elements of a wave's step
constexpr int kChunk = 64;           // output columns of a wave's step

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
    int splits, split_steps;         // parts of the inner dimension, their steps
    int groups, chunks;              // shrink: blocks that share the ranks; expand: chunks of a wave
    float* part;                     // [splits, rows, width]
};

__device__ __forceinline__ int id_of(const LoraParams& p, int m) {
    const int l = p.ids[m];
    return l >= 0 && l < p.adapters ? l : -1;
}

// The rows of a tile: lane i (of the first 16 CT) knows row i's number and its
// adapter, -1 for a row that is not there (-2) or has none.
template <int CT>
struct Tile {
    int row = 0, id = -2;
    bool any = false;
    __device__ __forceinline__ Tile(const LoraParams& p, int slot, int* s_rows) {
        const int lane = threadIdx.x & 63;
        if constexpr (CT == 1) {
            const int mine = id_of(p, slot);
            if (mine < 0) {                  // a row of its own, to copy
                row = slot;
                id = lane == 0 ? -1 : -2;
                any = true;
                return;
            }
            int ids[kGathered / 64];
#pragma unroll
            for (int i = 0; i < kGathered / 64; ++i) {
                if (i * 64 >= p.rows) break;
                ids[i] = id_of(p, min(i * 64 + lane, p.rows - 1));
            }
            int before = 0, rank = 0;        // of the rows looked at with this adapter, of row `slot`
            if (lane < 16) s_rows[lane] = -1;
            wave_sync();
            // the rank of row `slot` first: the rows below it
#pragma unroll
            for (int i = 0; i < kGathered / 64; ++i) {
                if (i * 64 >= slot) break;
                const int m = i * 64 + lane;
                rank += __popcll(__ballot(ids[i] == mine && m < slot));
            }
            if (rank % 16 != 0) return;
#pragma unroll
            for (int i = 0; i < kGathered / 64; ++i) {
                if (i * 64 >= p.rows) break;
                const int m = i * 64 + lane;
                const uint64_t same = __ballot(ids[i] == mine && m < p.rows);
                const int at = before + __popcll(same & ((1ull << lane) - 1)) - rank;
                if ((same >> lane & 1) && at >= 0 && at < 16) s_rows[at] = m;
                before += __popcll(same);
            }
            wave_sync();
            row = s_rows[lane & 15];
            id = row < 0 ? -2 : mine;
            row = max(row, 0);
            any = true;
        } else {
            row = slot * 16 * CT + lane;
            id = row < p.rows ? id_of(p, row) : -2;
            row = min(row, p.rows - 1);
            any = true;
        }
    }
};

template <int CT, int RT>
__global__ __launch_bounds__(kThreads, 2) void k_lora_shrink(const LoraParams p) {
    __shared__ int s_rows[kWaves][16];
    __shared__ f4 s_sum[2][RT * CT * 64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 15, g = lane >> 4;
    int block = blockIdx.x;
    const int group = block % p.groups;
    block /= p.groups;
    const int split = block % p.splits, slot = block / p.splits;
    const Tile<CT> tile(p, slot, s_rows[wave]);
    if (!tile.any) return;
    const int rank0 = group * RT * 16;
    const int total = (p.inner + kStepK - 1) / kStepK;
    const int s_begin = split * p.split_steps, s_end = min(s_begin + p.split_steps, total);

    int rows[CT];                    // this lane's row of each column tile
#pragma unroll
    for (int i = 0; i < CT; ++i) rows[i] = __shfl(tile.row, i * 16 + c, 64);
    uint64_t left = __ballot(tile.id >= 0);
    while (left) {
        const int l = __builtin_amdgcn_readlane(tile.id, __builtin_ctzll(left));
        const uint64_t same = __ballot(tile.id == l);
        left &= ~same;
        const uint16_t* const ap = p.a + (int64_t)l * p.width * p.inner;
        f4 acc[RT][CT];
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
            for (int k = 0; k < CT; ++k) acc[i][k] = f4{0, 0, 0, 0};
        struct StepA {
            uint4 a[RT][2];
        };
        struct StepX {
            uint4 x[CT][2];
        };
        // a lane's 16 elements of a step: both operands agree on the order
        auto piece = [&](const uint16_t* from, int st, int h) {
            const int e = st * kStepK + g * 16 + h * 8;
            const bool in = e < p.inner;
            const uint32_t keep = in ? ~0u : 0u;
            const uint4 w = *reinterpret_cast<const uint4*>(from + (in ? e : 0));
            return make_uint4(w.x & keep, w.y & keep, w.z & keep, w.w & keep);
        };
        auto load_x = [&](StepX& s, int st) {
#pragma unroll
            for (int k = 0; k < CT; ++k)
#pragma unroll
                for (int h = 0; h < 2; ++h) s.x[k][h] = piece(p.x + rows[k] * p.ldx, st, h);
        };
        auto load_a = [&](StepA& s, int st, int h) {
            int rank = rank0 + c;
            asm volatile("" : "+v"(rank));      // addresses anew each step: kept, they take the accumulators' registers
#pragma unroll
            for (int i = 0; i < RT; ++i)
                s.a[i][h] = piece(ap + (int64_t)min(rank + i * 16, p.width - 1) * p.inner, st, h);
        };
        auto multiply = [&](const StepA& sa, const StepX& sx, int h) {
#pragma unroll
            for (int i = 0; i < RT; ++i)
#pragma unroll
                for (int k = 0; k < CT; ++k)
                    acc[i][k] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                        __builtin_bit_cast(b8, sa.a[i][h]), __builtin_bit_cast(b8, sx.x[k][h]), acc[i][k], 0, 0, 0);
        };
        int st = s_begin + wave;
        if (st < s_end) {
            // x is a step ahead, A (from the caches, shared by the tiles) too
            // where registers allow
            constexpr bool kAheadA = RT * (CT + 4) <= 24;
            StepX x, next_x;
            StepA a, next_a;
            load_x(x, st);
            if (kAheadA) {
                load_a(a, st, 0);
                load_a(a, st, 1);
            }
            for (; st < s_end; st += kWaves) {
                if (!kAheadA) load_a(a, st, 0);
                if (st + kWaves < s_end) {
                    load_x(next_x, st + kWaves);
                    if (kAheadA) {
                        load_a(next_a, st + kWaves, 0);
                        load_a(next_a, st + kWaves, 1);
                    }
                }
                multiply(a, x, 0);
                if (!kAheadA) load_a(a, st, 1);
                multiply(a, x, 1);
                x = next_x;
                if (kAheadA) a = next_a;
            }
        }
        // the four waves' sums: 2 and 3 to 0 and 1, then 1 to 0
        if (wave >= 2)
#pragma unroll
            for (int i = 0; i < RT * CT; ++i) s_sum[wave - 2][i * 64 + lane] = acc[i / CT][i % CT];
        __syncthreads();
        if (wave < 2)
#pragma unroll
            for (int i = 0; i < RT * CT; ++i) acc[i / CT][i % CT] += s_sum[wave][i * 64 + lane];
        __syncthreads();
        if (wave == 1)
#pragma unroll
            for (int i = 0; i < RT * CT; ++i) s_sum[0][i * 64 + lane] = acc[i / CT][i % CT];
        __syncthreads();
        if (wave == 0) {
#pragma unroll
            for (int i = 0; i < RT; ++i) {
                const int rank = rank0 + i * 16 + g * 4;
#pragma unroll
                for (int k = 0; k < CT; ++k) {
                    const f4 sum = acc[i][k] + s_sum[0][(i * CT + k) * 64 + lane];
                    if (rank < p.width && (same >> (k * 16 + c) & 1))
                        *reinterpret_cast<f4*>(p.part + ((int64_t)split * p.rows + rows[k]) * p.width + rank) = sum;
                }
            }
        }
        if (left) __syncthreads();
    }
}

// Eight neighbouring values of an output row as fp32, and back.
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

template <int CT, typename OutT>
__global__ __launch_bounds__(kThreads, 2) void k_lora_expand(const LoraParams p) {
    constexpr int kTerms = sizeof(OutT) == 2 ? 2 : 3;
    __shared__ int s_rows[kWaves][16];
    extern __shared__ __align__(16) uint8_t s_t[];      // [16 CT rows][kTerms * rank, padded] bf16
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 15, g = lane >> 4;
    const int column_blocks = p.block_ends[3], slot = blockIdx.x / column_blocks;
    int cb = blockIdx.x % column_blocks;
    const Tile<CT> tile(p, slot, s_rows[wave]);
    if (!tile.any) return;
    const int slice = (cb >= p.block_ends[0] ? 1 : 0) + (cb >= p.block_ends[1] ? 1 : 0) + (cb >= p.block_ends[2] ? 1 : 0);
    int first = 0, end = p.ends[0];
#pragma unroll
    for (int i = 1; i < 4; ++i)
        if (slice >= i) {
            first = p.ends[i - 1];
            end = p.ends[i];
        }
#pragma unroll
    for (int i = 0; i < 3; ++i) cb -= slice == i + 1 ? p.block_ends[i] : 0;
    // this wave's chunks of columns
    const int n_begin = first + (cb * kWaves + wave) * p.chunks * kChunk, n_end = min(n_begin + p.chunks * kChunk, end);

    int rows[CT];
#pragma unroll
    for (int i = 0; i < CT; ++i) rows[i] = __shfl(tile.row, i * 16 + c, 64);
    const int groups = p.rank >> 3;                     // of 8 ranks
    // Matrix steps over the ranks.  With a multiple of 32 the terms of t follow
    // each other against one piece of B; else terms and ranks are one axis.
    const bool whole = p.rank % 32 == 0;
    const int steps = whole ? p.rank / 32 : (kTerms * groups + 3) / 4, terms = whole ? kTerms : 1;
    const int pitch = (whole ? kTerms * p.rank : steps * 32) * 2 + 16;
    const OutT* y = static_cast<const OutT*>(p.y);
    OutT* out = static_cast<OutT*>(p.out);

    // rows without an adapter stay as they are
    const uint64_t bare = __ballot(tile.id == -1);
    if (bare && out != y) {
        for (int n = n_begin + g * 16; n < n_end; n += kChunk)
#pragma unroll
            for (int k = 0; k < CT; ++k)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    if ((bare >> (k * 16 + c) & 1) && n + h * 8 < n_end) {
                        const uint4* from = reinterpret_cast<const uint4*>(y + rows[k] * p.ldy + n + h * 8);
                        uint4* to = reinterpret_cast<uint4*>(out + rows[k] * p.ldo + n + h * 8);
#pragma unroll
                        for (int i = 0; i < (int)sizeof(OutT) / 2; ++i) to[i] = from[i];
                    }
    }
    uint64_t left = __ballot(tile.id >= 0);
    bool again = false;
    while (left) {
        const int l = __builtin_amdgcn_readlane(tile.id, __builtin_ctzll(left));
        const uint64_t same = __ballot(tile.id == l);
        left &= ~same;
        if (again) __syncthreads();
        again = true;
        // t of the tile's rows in bf16 terms
        const float gain = p.gain ? p.gain[l] : 1.0f;
        for (int i = threadIdx.x; i < 16 * CT * groups; i += kThreads) {
            const int r = i / groups, q = i - r * groups;
            const int row = CT == 1 ? s_rows[wave][r] : min(slot * 16 * CT + r, p.rows - 1);
            f4 lo = {0, 0, 0, 0}, hi = {0, 0, 0, 0};
            if (row >= 0) {
                const float* from = p.part + (int64_t)row * p.width + slice * p.rank + q * 8;
#pragma unroll 4
                for (int s = 0; s < p.splits; ++s) {
                    lo += *reinterpret_cast<const f4*>(from + (int64_t)s * p.rows * p.width);
                    hi += *reinterpret_cast<const f4*>(from + (int64_t)s * p.rows * p.width + 4);
                }
            }
            float t[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                t[e] = lo[e] * gain;
                t[4 + e] = hi[e] * gain;
            }
#pragma unroll
            for (int k = 0; k < kTerms; ++k) {
                // one term of two values, which keep what it leaves
                auto term = [](float& a, float& b) {
                    const uint32_t w = pack2(a, b);
                    a -= as_f32(w << 16);
                    b -= as_f32(w & 0xFFFF0000u);
                    return w;
                };
                *reinterpret_cast<uint4*>(s_t + r * pitch + (k * groups + q) * 16) =
                    make_uint4(term(t[0], t[1]), term(t[2], t[3]), term(t[4], t[5]), term(t[6], t[7]));
            }
        }
        if (!whole)
            for (int i = threadIdx.x; i < 16 * CT * (steps * 4 - kTerms * groups); i += kThreads) {
                const int n = steps * 4 - kTerms * groups, r = i / n;
                *reinterpret_cast<uint4*>(s_t + r * pitch + (kTerms * groups + i - r * n) * 16) = make_uint4(0, 0, 0, 0);
            }
        __syncthreads();

        for (int n0 = n_begin; n0 < n_end; n0 += kChunk) {
            const int n = n0 + g * 16;              // this lane's 16 columns
            Eight<OutT> v[CT][2];
#pragma unroll
            for (int k = 0; k < CT; ++k)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    v[k][h].load(y + rows[k] * p.ldy + (n + h * 8 < n_end ? n + h * 8 : n0));
            // matrix row rho of piece j is column n0 + 16 (rho / 4) + 4 j + rho % 4
            const uint16_t* bp[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                bp[j] = p.b + ((int64_t)l * p.columns + min(n0 + (c >> 2) * 16 + j * 4 + (c & 3), end - 1)) * p.rank;
            f4 acc[4][CT];
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int k = 0; k < CT; ++k) acc[j][k] = f4{0, 0, 0, 0};
            for (int s = 0; s < steps; ++s) {
                const int q = whole ? s * 4 + g : (s * 4 + g) % groups;
                b8 bf[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) bf[j] = *reinterpret_cast<const b8*>(bp[j] + q * 8);
                for (int t = 0; t < terms; ++t) {
                    const uint8_t* tp = s_t + c * pitch + (t * groups + s * 4 + g) * 16;
#pragma unroll
                    for (int k = 0; k < CT; ++k) {
                        const b8 tf = *reinterpret_cast<const b8*>(tp + k * 16 * pitch);
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            acc[j][k] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bf[j], tf, acc[j][k], 0, 0, 0);
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < CT; ++k)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    if ((same >> (k * 16 + c) & 1) && n + h * 8 < n_end) {
                        v[k][h].add(acc[2 * h][k], acc[2 * h + 1][k]);
                        v[k][h].store(out + rows[k] * p.ldo + n + h * 8);
                    }
        }
    }
}

// How a call is shared out.
struct Plan {
    bool gathered;
    int slots, tiles;                // blocks of rows; about as many have work
    int rank_tiles, groups, splits, split_steps;
    int64_t shrink_blocks;
};

Plan plan_of(const LoraArgs& a) {
    Plan p;
    p.gathered = a.rows <= kGathered;
    const int width = a.slices * a.rank, all = (width + 15) / 16;
    p.slots = p.gathered ? (int)a.rows : (int)((a.rows + 63) / 64);
    p.tiles = p.gathered ? (int)std::min<int64_t>(a.rows, (a.rows + 15) / 16 + a.adapters) : p.slots;
    p.groups = (all + 5) / 6;
    const int each = (all + p.groups - 1) / p.groups;
    p.rank_tiles = each == 5 ? 6 : each;
    const int steps = (int)((a.inner + kStepK - 1) / kStepK);
    // Parts of the inner dimension: about two blocks a CU, every wave with a
    // step or more, and no more than 16 rows of t for the second launch to add.
    int splits = 512 / (p.tiles * p.groups);
    splits = std::clamp(splits, 1, 16);
    p.split_steps = std::max((steps + splits - 1) / splits, kWaves);
    p.splits = std::max(1, (steps + p.split_steps - 1) / p.split_steps);
    p.shrink_blocks = (int64_t)p.slots * p.splits * p.groups;
    return p;
}

template <int CT>
hipError_t run_shrink(const LoraParams& p, const Plan& plan, hipStream_t stream) {
    const dim3 grid((unsigned)plan.shrink_blocks), block(kThreads);
    switch (plan.rank_tiles) {
    case 1: hipLaunchKernelGGL((k_lora_shrink<CT, 1>), grid, block, 0, stream, p); break;
    case 2: hipLaunchKernelGGL((k_lora_shrink<CT, 2>), grid, block, 0, stream, p); break;
    case 3: hipLaunchKernelGGL((k_lora_shrink<CT, 3>), grid, block, 0, stream, p); break;
    case 4: hipLaunchKernelGGL((k_lora_shrink<CT, 4>), grid, block, 0, stream, p); break;
    default: hipLaunchKernelGGL((k_lora_shrink<CT, 6>), grid, block, 0, stream, p); break;
    }
    return hipGetLastError();
}

template <int CT, typename OutT>
hipError_t run_expand(LoraParams& p, const Plan& plan, hipStream_t stream) {
    constexpr int kTerms = sizeof(OutT) == 2 ? 2 : 3;
    int ends[4], from = 0, blocks = 0;
    p.chunks = CT == 1 ? 1 : 2;
    for (int i = 0; i < 4; ++i) {
        const int run = kWaves * p.chunks * kChunk;
        blocks += (p.ends[i] - from + run - 1) / run;
        from = p.ends[i];
        ends[i] = blocks;
    }
    for (int i = 0; i < 4; ++i) p.block_ends[i] = ends[i];
    const int kv = p.rank % 32 == 0 ? kTerms * p.rank : (kTerms * p.rank + 31) / 32 * 32;
    const int bytes = 16 * CT * (kv * 2 + 16);
    hipLaunchKernelGGL((k_lora_expand<CT, OutT>), dim3((unsigned)((int64_t)plan.slots * blocks)), dim3(kThreads), bytes,
                       stream, p);
    return hipGetLastError();
}

}  // namespace

int64_t lora_workspace(const LoraArgs& a) {
    return a.rows == 0 ? 0 : (int64_t)plan_of(a).splits * a.rows * a.slices * a.rank * 4;
}

// Blocks of the larger launch: 2^32 threads and more are not launched.
int64_t lora_blocks(const LoraArgs& a) {
    const Plan plan = plan_of(a);
    return std::max(plan.shrink_blocks, (int64_t)plan.slots * ((a.columns + kWaves * kChunk - 1) / (kWaves * kChunk) + 4));
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
    p.splits = plan.splits; p.split_steps = plan.split_steps; p.groups = plan.groups;
    p.part = reinterpret_cast<float*>(a.workspace);
    hipError_t e = plan.gathered ? run_shrink<1>(p, plan, a.stream) : run_shrink<4>(p, plan, a.stream);
    if (e != hipSuccess) return e;
    if (plan.gathered)
        return a.out_bf16 ? run_expand<1, uint16_t>(p, plan, a.stream) : run_expand<1, float>(p, plan, a.stream);
    return a.out_bf16 ? run_expand<4, uint16_t>(p, plan, a.stream) : run_expand<4, float>(p, plan, a.stream);
}

}  // namespace fp8mi
