// evict.hip -- eviction from the paged KV cache by accumulated attention
// weight on gfx950.  Of a sequence of n > budget tokens every KV head keeps
// the first `sinks`, the last `recent` and, of those between, the
// budget - sinks - recent with the largest weights (the lower position among
// equals), and its kept tokens move together in their order.
//
// k_evict_select: one block per (KV head, sequence).  A radix select finds
// the k-th largest weight in three histogram passes over 11, 11 and 10 bits
// of an order-preserving key (2048 bins: softmax weights crowd few exponents,
// so coarse bins would serialize the counters), then one pass counts and one
// writes the kept positions in order, each wave on a run of its own with
// ballots.  The weights are re-read from the L2 in every pass.
//
// k_evict_move: kept[r] >= r and increasing, so rows can move in place if a
// block takes them in order, reads a tile before it writes it, and no other
// block touches the same bytes: what a tile overwrites lies below everything
// that later tiles read.  A block owns one of K, V, their scales or the
// weights of a (head, sequence).  Into other pages the tiles are independent
// and spread over the grid.
#include <hip/hip_runtime.h>

#include "attention.hpp"

namespace fp8mi {
namespace {

using attn::row_of_entry;
using attn::seq_len;

constexpr int kSelThreads = 1024;
constexpr int kSelWaves = kSelThreads / 64;
constexpr int kBins = 2048;
constexpr int kMoveThreads = 512;
constexpr int kPieces = 8;              // pieces a thread moves per tile

// Order-preserving key: larger weight, larger key; -0 equals +0, NaN is largest.
__device__ __forceinline__ uint32_t key_of(float w) {
    const uint32_t u = __float_as_uint(w);
    if (w != w) return 0xFFFFFFFFu;
    if (w == 0.0f) return 0x80000000u;
    return (u >> 31) ? ~u : u | 0x80000000u;
}

__global__ __launch_bounds__(kSelThreads) void k_evict_select(const EvictArgs a) {
    __shared__ uint32_t hist[kBins];
    __shared__ uint32_t wave_tot[kSelWaves];
    __shared__ uint32_t found[2];           // bin, and how many above it
    __shared__ uint32_t n_gt[kSelWaves], n_eq[kSelWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int h = blockIdx.x, b = blockIdx.y;
    const int n = seq_len(a.kv, b);
    const int64_t bh = (int64_t)b * a.kv.heads + h;
    int32_t* kept = a.kept + bh * a.budget;
    if (h == 0 && tid == 0) a.new_lens[b] = min(n, a.budget);
    if (n <= a.budget) {
        for (int r = tid; r < a.budget; r += kSelThreads) kept[r] = r < n ? r : -1;
        return;
    }
    const int lo = a.sinks, hi = n - a.recent;          // the tokens chosen among
    const int k = a.budget - a.sinks - a.recent;
    for (int r = tid; r < a.sinks; r += kSelThreads) kept[r] = r;
    for (int r = tid; r < a.recent; r += kSelThreads) kept[a.sinks + k + r] = hi + r;
    if (k == 0) return;
    const float* w = a.weights + bh * a.ldw;

    uint32_t key = 0, need = (uint32_t)k;               // bits of the k-th largest found so far
    int low = 32;                                       // lowest bit of them
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        const int width = pass < 2 ? 11 : 10;
        const int next = low - width;
        for (int i = tid; i < kBins; i += kSelThreads) hist[i] = 0;
        __syncthreads();
#pragma unroll 4
        for (int j = lo + tid; j < hi; j += kSelThreads) {
            const uint32_t u = key_of(w[j]);
            if (pass == 0 || (u >> low) == (key >> low)) atomicAdd(&hist[(u >> next) & ((1u << width) - 1)], 1u);
        }
        __syncthreads();
        // keys above bin 2t + 1, by a scan from the top bin down
        const int b1 = kBins - 1 - 2 * tid, b0 = b1 - 1;
        const uint32_t h1 = hist[b1], h0 = hist[b0];
        uint32_t sum = h1 + h0;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const uint32_t t = __shfl_up(sum, off, 64);
            if (lane >= off) sum += t;
        }
        if (lane == 63) wave_tot[wave] = sum;
        __syncthreads();
        uint32_t above = sum - h1 - h0;
        for (int i = 0; i < wave; ++i) above += wave_tot[i];
        if (above < need && need <= above + h1) { found[0] = b1; found[1] = above; }
        if (above + h1 < need && need <= above + h1 + h0) { found[0] = b0; found[1] = above + h1; }
        __syncthreads();
        key |= found[0] << next;
        need -= found[1];
        low = next;
    }
    // keep every key above `key`, and the first `need` equal to it
    const int run = ((hi - lo + kSelThreads - 1) / kSelThreads) * 64;
    const int r0 = lo + wave * run, r1 = min(hi, r0 + run);
    uint32_t gt = 0, eq = 0;
#pragma unroll 4
    for (int j = r0 + lane; j < r0 + run; j += 64) {
        const uint32_t u = j < r1 ? key_of(w[j]) : 0;
        gt += __popcll(__ballot(j < r1 && u > key));
        eq += __popcll(__ballot(j < r1 && u == key));
    }
    if (lane == 0) { n_gt[wave] = gt; n_eq[wave] = eq; }
    __syncthreads();
    gt = 0; eq = 0;
    for (int i = 0; i < wave; ++i) { gt += n_gt[i]; eq += n_eq[i]; }
    const uint64_t below = (1ull << lane) - 1;
    for (int j = r0 + lane; j < r0 + run; j += 64) {
        const uint32_t u = j < r1 ? key_of(w[j]) : 0;
        const uint64_t mg = __ballot(j < r1 && u > key), me = __ballot(j < r1 && u == key);
        const uint32_t g = gt + __popcll(mg & below), e = eq + __popcll(me & below);
        if (j < r1 && (u > key || (u == key && e < need))) kept[a.sinks + g + min(e, need)] = j;
        gt += __popcll(mg);
        eq += __popcll(me);
    }
}

// Moves rows [0, m) of one array, `per` pieces of type T a row: piece q of
// row r from src(kept[r], q) to dst(r, q); a null address is left out.
template <typename T, typename Src, typename Dst>
__device__ __forceinline__ void move_rows(const int32_t* kept, int m, int per, bool in_place, int first, int step,
                                          Src src, Dst dst) {
    const int rows = kMoveThreads * kPieces / per;      // of a tile
    const int tiles = (m + rows - 1) / rows;
    for (int tile = first; tile < tiles; tile += step) {
        const int r0 = tile * rows, rn = min(m - r0, rows);
        if (in_place && kept[r0 + rn - 1] == r0 + rn - 1) continue;     // nothing before it was dropped
        T v[kPieces];
        T* to[kPieces];
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int p = threadIdx.x + i * kMoveThreads, r = p / per, q = p - r * per;
            to[i] = nullptr;
            if (r < rn) {
                const T* from = src(kept[r0 + r], q);
                if (from) {
                    to[i] = dst(r0 + r, q);
                    v[i] = *from;
                }
            }
        }
        // every read of the tile has arrived before any of it is written;
        // what is written is read by no later tile
        if (in_place) {
            __builtin_amdgcn_s_waitcnt(0);
            __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < kPieces; ++i)
            if (to[i]) *to[i] = v[i];
    }
}

__global__ __launch_bounds__(kMoveThreads) void k_evict_move(const EvictArgs a, int parts) {
    const KvView& kv = a.kv;
    const int part = blockIdx.x % parts, h = blockIdx.x / parts, b = blockIdx.y;
    const int first = blockIdx.z, step = gridDim.z;
    const int n = seq_len(kv, b), m = min(n, a.budget);
    const int64_t bh = (int64_t)b * kv.heads + h;
    const int32_t* kept = a.kept + bh * a.budget;
    const bool weights_in_place = a.weights == a.weights_out;
    const bool in_place = part == 4 ? weights_in_place : a.dst_table == nullptr;
    if (in_place && (n <= a.budget || first > 0)) return;

    auto src_row = [&](int j) { return row_of_entry(kv, kv.table[b * kv.table_ld + (j >> kv.page_shift)], j); };
    auto dst_row = [&](int r) {
        const int32_t* t = in_place ? kv.table + b * kv.table_ld : a.dst_table + b * a.dst_ld;
        return row_of_entry(kv, t[r >> kv.page_shift], r);
    };
    const int stp = in_place ? 1 : step;
    if (part < 2) {
        uint4* data = static_cast<uint4*>(part == 0 ? kv.k : kv.v);
        const int per = kv.head_dim * ((part == 0 ? kv.k_st : kv.v_st) == FP8_KV_BF16 ? 2 : 1) / 16;
        auto at = [&](int row, int q) -> uint4* {
            return row < 0 ? nullptr : data + ((int64_t)row * kv.heads + h) * per + q;
        };
        move_rows<uint4>(kept, m, per, in_place, first, stp, [&](int j, int q) { return at(src_row(j), q); },
                         [&](int r, int q) { return at(dst_row(r), q); });
    } else if (part < 4) {
        float* sc = part == 2 ? kv.k_scale : kv.v_scale;
        if (sc == nullptr || kv.per_head) return;
        auto at = [&](int row) -> float* { return row < 0 ? nullptr : sc + (int64_t)row * kv.heads + h; };
        move_rows<float>(kept, m, 1, in_place, first, stp, [&](int j, int) { return at(src_row(j)); },
                         [&](int r, int) { return at(dst_row(r)); });
    } else {
        const float* from = a.weights + bh * a.ldw;
        float* to = a.weights_out + bh * a.ldwo;
        move_rows<float>(kept, m, 1, in_place, first, stp, [&](int j, int) { return from + j; },
                         [&](int r, int) { return to + r; });
        // nothing has been received behind the kept tokens
        const int end = in_place ? n : a.budget;
        for (int r = m + first * kMoveThreads + threadIdx.x; r < end; r += stp * kMoveThreads) to[r] = 0.0f;
    }
}

}  // namespace

hipError_t launch_evict(const EvictArgs& a) {
    const dim3 grid((unsigned)a.kv.heads, (unsigned)a.kv.batch);
    hipLaunchKernelGGL(k_evict_select, grid, dim3(kSelThreads), 0, a.stream, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    constexpr int parts = 5;
    const int64_t widest = a.kv.head_dim / 8;           // 16-byte pieces of a bf16 row
    const int64_t tiles = (a.budget * widest + kMoveThreads * kPieces - 1) / (kMoveThreads * kPieces);
    const bool in_place = a.dst_table == nullptr && a.weights == a.weights_out;
    const dim3 move((unsigned)(parts * a.kv.heads), (unsigned)a.kv.batch,
                    in_place ? 1u : (unsigned)(tiles < 1 ? 1 : tiles > 64 ? 64 : tiles));
    hipLaunchKernelGGL(k_evict_move, move, dim3(kMoveThreads), 0, a.stream, a, parts);
    return hipGetLastError();
}

}  // namespace fp8mi
