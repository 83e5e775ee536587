// evict.hip -- eviction from the paged KV cache by accumulated attention
// weight on gfx950.  Of a sequence of n > budget tokens every KV head keeps
// the first `sinks`, the last `recent` and, of those between, the
// budget - sinks - recent with the largest weights (the lower position among
// equals), and its kept tokens move together in their order.
//
// Measured on one MI355X, 8 KV heads of 128 in E4M3, pages of 16: 16 sequences
// cut from 16384 to 4096 tokens into other pages 96-98 us (selection 21, move
// 70-76, which reads and writes 280 MB in rows of 128 bytes: 4 TB/s where a
// copy reaches 5.2), in place 107 us; one sequence from 1100 to 1024 15-20 us,
// two dependent launches of 7 and 5 us.
//
// Selection: one block per (KV head, sequence).  A radix select finds the
// k-th largest weight in three histogram passes over 11, 11 and 10 bits of an
// order-preserving key (2048 bins: softmax weights crowd few exponents, so
// coarse bins would serialize the counters); then ballots count, and place,
// the kept positions in order.  Up to 32768 tokens the keys stay in registers
// and each weight is read once (whole calls of 16 sequences: from 16384 tokens
// 98 us against 106 with the weights read again in every pass, from 8000 51
// against 56, and 53 with registers for 32768).
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

// What one block of a selection chooses from, and the outputs that need no
// choice: false if nothing is left to choose.
struct Choice {
    const float* w;
    int32_t* kept;
    int lo, hi;                 // positions chosen among
    int k;                      // how many of them stay
};

__device__ __forceinline__ bool begin_choice(const EvictArgs& a, int tid, Choice* c) {
    const int h = blockIdx.x, b = blockIdx.y;
    const int n = seq_len(a.kv, b);
    const int64_t bh = (int64_t)b * a.kv.heads + h;
    int32_t* kept = a.kept + bh * a.budget;
    if (h == 0 && tid == 0) a.new_lens[b] = min(n, a.budget);
    if (n <= a.budget) {
        for (int r = tid; r < a.budget; r += kSelThreads) kept[r] = r < n ? r : -1;
        return false;
    }
    *c = Choice{a.weights + bh * a.ldw, kept + a.sinks, a.sinks, n - a.recent, a.budget - a.sinks - a.recent};
    for (int r = tid; r < a.sinks; r += kSelThreads) kept[r] = r;
    for (int r = tid; r < a.recent; r += kSelThreads) kept[a.sinks + c->k + r] = c->hi + r;
    return c->k > 0;
}

struct SelLds {
    uint32_t hist[kBins];
    uint32_t wave_tot[kSelWaves];
    uint32_t found[2];          // bin, and how many keys lie above it
};

// One radix pass: with the histogram of the keys that match `key` above bit
// `low` in place, extends `key` by the bin that holds the need-th largest.
__device__ __forceinline__ void find_bin(SelLds& s, int tid, int next, uint32_t* key, uint32_t* need) {
    const int lane = tid & 63, wave = tid >> 6;
    // keys above bin 2t + 1, by a scan from the top bin down
    const int b1 = kBins - 1 - 2 * tid, b0 = b1 - 1;
    const uint32_t h1 = s.hist[b1], h0 = s.hist[b0];
    uint32_t sum = h1 + h0;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const uint32_t t = __shfl_up(sum, off, 64);
        if (lane >= off) sum += t;
    }
    if (lane == 63) s.wave_tot[wave] = sum;
    __syncthreads();
    uint32_t tot = lane < kSelWaves ? s.wave_tot[lane] : 0;
#pragma unroll
    for (int off = 1; off < kSelWaves; off <<= 1) {
        const uint32_t t = __shfl_up(tot, off, 64);
        if (lane >= off) tot += t;
    }
    const uint32_t above = sum - h1 - h0 + (wave ? __shfl(tot, wave - 1, 64) : 0);
    if (above < *need && *need <= above + h1) { s.found[0] = b1; s.found[1] = above; }
    if (above + h1 < *need && *need <= above + h1 + h0) { s.found[0] = b0; s.found[1] = above + h1; }
    __syncthreads();
    *key |= s.found[0] << next;
    *need -= s.found[1];
}

constexpr int kPasses = 3;
__device__ __forceinline__ int low_bit(int pass) { return pass == 0 ? 21 : pass == 1 ? 10 : 0; }

// The keys stay in registers, KPT a thread: key i of thread t is position
// lo + i * 1024 + t.  For up to KPT * 1024 tokens; each weight is read once.
template <int KPT>
__global__ __launch_bounds__(kSelThreads) void k_evict_select_regs(const EvictArgs a) {
    __shared__ SelLds s;
    __shared__ uint32_t n_gt[KPT * kSelWaves], n_eq[KPT * kSelWaves];   // per 64 positions; then their prefix sums
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    Choice c;
    if (!begin_choice(a, tid, &c)) return;
    uint32_t u[KPT];
    uint32_t live = 0;
    const int size = c.hi - c.lo;
#pragma unroll
    for (int i = 0; i < KPT; ++i) {                     // all loads before the first use
        if (i * kSelThreads >= size) break;
        u[i] = __float_as_uint(c.w[min(c.lo + i * kSelThreads + tid, c.hi - 1)]);
    }
#pragma unroll
    for (int i = 0; i < KPT; ++i) {
        if (i * kSelThreads >= size) break;
        u[i] = key_of(__uint_as_float(u[i]));
        live |= (i * kSelThreads + tid < size ? 1u : 0u) << i;
    }
    uint32_t key = 0, need = (uint32_t)c.k;
#pragma unroll
    for (int pass = 0; pass < kPasses; ++pass) {
        const int next = low_bit(pass), low = pass == 0 ? 32 : low_bit(pass - 1);
        for (int i = tid; i < kBins; i += kSelThreads) s.hist[i] = 0;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < KPT; ++i) {
            if (i * kSelThreads >= size) break;
            if ((live >> i & 1) && (pass == 0 || (u[i] >> (low & 31)) == (key >> (low & 31))))
                atomicAdd(&s.hist[(u[i] >> next) & ((1u << (low - next)) - 1)], 1u);
        }
        __syncthreads();
        find_bin(s, tid, next, &key, &need);
    }
    // keep every key above `key`, and the first `need` equal to it
#pragma unroll
    for (int i = 0; i < KPT; ++i) {
        if (i * kSelThreads >= size) break;
        const bool in = live >> i & 1;
        const uint64_t mg = __ballot(in && u[i] > key), me = __ballot(in && u[i] == key);
        if (lane == 0) {
            n_gt[i * kSelWaves + wave] = __popcll(mg);
            n_eq[i * kSelWaves + wave] = __popcll(me);
        }
    }
    __syncthreads();
    // exclusive prefix sums over the runs of 64, by wave 0 and wave 1, each
    // lane over consecutive ones
    if (wave < 2) {
        constexpr int E = KPT * kSelWaves / 64;
        uint32_t* v = (wave == 0 ? n_gt : n_eq) + lane * E;
        const int end = (size + 63) / 64 - lane * E;            // runs that were counted
        uint32_t own[E], sum = 0;
#pragma unroll
        for (int i = 0; i < E; ++i) {
            own[i] = i < end ? v[i] : 0;
            sum += own[i];
        }
        uint32_t at = sum;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const uint32_t t = __shfl_up(at, off, 64);
            if (lane >= off) at += t;
        }
        at -= sum;
#pragma unroll
        for (int i = 0; i < E; ++i) {
            v[i] = at;
            at += own[i];
        }
    }
    __syncthreads();
    const uint64_t below = (1ull << lane) - 1;
#pragma unroll
    for (int i = 0; i < KPT; ++i) {
        if (i * kSelThreads >= size) break;
        const bool in = live >> i & 1;
        const uint64_t mg = __ballot(in && u[i] > key), me = __ballot(in && u[i] == key);
        const uint32_t g = n_gt[i * kSelWaves + wave] + __popcll(mg & below);
        const uint32_t e = n_eq[i * kSelWaves + wave] + __popcll(me & below);
        if (in && (u[i] > key || (u[i] == key && e < need)))
            c.kept[g + min(e, need)] = c.lo + i * kSelThreads + tid;
    }
}

// Any number of tokens: the weights are read again (from the L2) in every
// pass, and each wave writes out a run of its own.
__global__ __launch_bounds__(kSelThreads) void k_evict_select(const EvictArgs a) {
    __shared__ SelLds s;
    __shared__ uint32_t n_gt[kSelWaves], n_eq[kSelWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    Choice c;
    if (!begin_choice(a, tid, &c)) return;
    uint32_t key = 0, need = (uint32_t)c.k;
#pragma unroll 1
    for (int pass = 0; pass < kPasses; ++pass) {
        const int next = low_bit(pass), low = pass == 0 ? 32 : low_bit(pass - 1);
        for (int i = tid; i < kBins; i += kSelThreads) s.hist[i] = 0;
        __syncthreads();
#pragma unroll 8
        for (int j = c.lo + tid; j < c.hi; j += kSelThreads) {
            const uint32_t u = key_of(c.w[j]);
            if (pass == 0 || (u >> (low & 31)) == (key >> (low & 31)))
                atomicAdd(&s.hist[(u >> next) & ((1u << (low - next)) - 1)], 1u);
        }
        __syncthreads();
        find_bin(s, tid, next, &key, &need);
    }
    const int run = ((c.hi - c.lo + kSelThreads - 1) / kSelThreads) * 64;
    const int r0 = c.lo + wave * run, r1 = min(c.hi, r0 + run);
    uint32_t gt = 0, eq = 0;
#pragma unroll 8
    for (int j = r0 + lane; j < r0 + run; j += 64) {
        const uint32_t u = j < r1 ? key_of(c.w[j]) : 0;
        gt += __popcll(__ballot(j < r1 && u > key));
        eq += __popcll(__ballot(j < r1 && u == key));
    }
    if (lane == 0) { n_gt[wave] = gt; n_eq[wave] = eq; }
    __syncthreads();
    gt = 0; eq = 0;
    for (int i = 0; i < wave; ++i) { gt += n_gt[i]; eq += n_eq[i]; }
    const uint64_t below = (1ull << lane) - 1;
#pragma unroll 8
    for (int j = r0 + lane; j < r0 + run; j += 64) {
        const uint32_t u = j < r1 ? key_of(c.w[j]) : 0;
        const uint64_t mg = __ballot(j < r1 && u > key), me = __ballot(j < r1 && u == key);
        const uint32_t g = gt + __popcll(mg & below), e = eq + __popcll(me & below);
        if (j < r1 && (u > key || (u == key && e < need))) c.kept[g + min(e, need)] = j;
        gt += __popcll(mg);
        eq += __popcll(me);
    }
}

// Where a block's rows come from and go to.
struct Route {
    const int32_t* kept;
    const int32_t* from;        // page tables of the sequence
    const int32_t* to;
    int shift, capacity;
    int m;                      // rows kept
    bool in_place;
    int first, step;            // tiles of this block
    // cache row of token j, whose page is `entry`; -1 where there is none
    __device__ __forceinline__ int row(int entry, int j) const {
        const int64_t r = ((int64_t)entry << shift) + (j & ((1 << shift) - 1));
        return r >= 0 && r < capacity ? (int)r : -1;
    }
    __device__ __forceinline__ int src(int j) const { return row(from[j >> shift], j); }
    __device__ __forceinline__ int dst(int r) const { return row(to[r >> shift], r); }
};

// Copies rows of one array of a head into other pages: `per` pieces of type T a row, rows
// `pitch` pieces apart.  A thread's pieces are the same part of rows a pass
// apart, kPieces of them in flight.
template <typename T>
__device__ __forceinline__ void copy_rows(const Route& w, T* data, int64_t pitch, int per) {
    const int pass = kMoveThreads / per, tile_rows = pass * kPieces;
    const int rr = threadIdx.x / per, q = threadIdx.x - rr * per;
    T* const base = data + q;
    for (int r0 = w.first * tile_rows; r0 < w.m; r0 += w.step * tile_rows) {
        // loads in three rounds, none of them conditional: positions, pages, rows
        int j[kPieces], to[kPieces];
        T v[kPieces];
#pragma unroll
        for (int i = 0; i < kPieces; ++i) j[i] = w.kept[min(r0 + i * pass + rr, w.m - 1)];
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int r = r0 + i * pass + rr;
            j[i] = w.src(j[i]);
            to[i] = w.dst(min(r, w.m - 1));
            if (j[i] < 0 || r >= w.m || rr >= pass) to[i] = -1;
        }
#pragma unroll
        for (int i = 0; i < kPieces; ++i) v[i] = base[max(j[i], 0) * pitch];
#pragma unroll
        for (int i = 0; i < kPieces; ++i)
            if (to[i] >= 0) base[to[i] * pitch] = v[i];
    }
}

// The same in place, by one block: tile after tile, each through four stages,
// one a round, so that every round issues the loads of three tiles at once:
// positions, page entries, pieces, and the stores.  2 sequences from 60000 to
// 30000 tokens 304 us against 361 with one tile at a time (4 from 16384 to
// 12000: 121 against 141); where a block has one tile, above, the registers of
// the stages cost more than they bring (99 against 112).
template <typename T>
__device__ __forceinline__ void move_in_place(const Route& w, T* data, int64_t pitch, int per) {
    const int pass = kMoveThreads / per, tile_rows = pass * kPieces;
    const int rr = threadIdx.x / per, q = threadIdx.x - rr * per;
    T* const base = data + q;
    int r0 = 0;
    for (; r0 < w.m; r0 += tile_rows) {         // nothing before these was dropped
        const int last = min(r0 + tile_rows, w.m) - 1;
        if (w.kept[last] != last) break;
    }
    if (r0 >= w.m) return;
    // No load is conditional: past the end they repeat the last row, and what
    // they bring is not stored.
    int kept[kPieces];
    int at[kPieces], entry[kPieces], to_entry[kPieces];
    T x[kPieces], y[kPieces];
    int x_to[kPieces], y_to[kPieces];
    auto row_of = [&](int i, int tile) { return tile + i * pass + rr; };
    auto positions = [&](int tile) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) kept[i] = w.kept[min(row_of(i, tile), w.m - 1)];
    };
    auto entries = [&](int tile) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            at[i] = kept[i];
            entry[i] = w.from[at[i] >> w.shift];
            to_entry[i] = w.to[min(row_of(i, tile), w.m - 1) >> w.shift];
        }
    };
    auto pieces = [&](int tile, T* v, int* to) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int r = row_of(i, tile), src = w.row(entry[i], at[i]);
            to[i] = src < 0 || r >= w.m || rr >= pass ? -1 : w.row(to_entry[i], r);
            v[i] = base[max(src, 0) * pitch];
        }
    };
    // Every read of the tile has arrived before any of it is written.  What is
    // written is read by no later tile, so their reads may be on the way.
    auto store = [&](T* v, const int* to) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) asm volatile("" : "+v"(v[i]));
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kPieces; ++i)
            if (to[i] >= 0) base[to[i] * pitch] = v[i];
    };
    positions(r0);
    entries(r0);
    positions(r0 + tile_rows);
    pieces(r0, x, x_to);
    entries(r0 + tile_rows);
    positions(r0 + 2 * tile_rows);
    for (;;) {
        pieces(r0 + tile_rows, y, y_to);
        entries(r0 + 2 * tile_rows);
        positions(r0 + 3 * tile_rows);
        store(x, x_to);
        r0 += tile_rows;
        if (r0 >= w.m) break;
        pieces(r0 + tile_rows, x, x_to);
        entries(r0 + 2 * tile_rows);
        positions(r0 + 3 * tile_rows);
        store(y, y_to);
        r0 += tile_rows;
        if (r0 >= w.m) break;
    }
}

template <bool IN_PLACE, typename T>
__device__ __forceinline__ void move_rows(const Route& w, T* data, int64_t pitch, int per) {
    if constexpr (IN_PLACE) move_in_place(w, data, pitch, per);
    else copy_rows(w, data, pitch, per);
}

template <bool IN_PLACE>
__global__ __launch_bounds__(kMoveThreads) void k_evict_move(const EvictArgs a, int parts) {
    const KvView& kv = a.kv;
    const int part = blockIdx.x % parts, h = blockIdx.x / parts, b = blockIdx.y;
    const int n = seq_len(kv, b), m = min(n, a.budget);
    const int64_t bh = (int64_t)b * kv.heads + h;
    const bool in_place = part == 4 ? a.weights == a.weights_out : IN_PLACE;
    if (in_place && (n <= a.budget || blockIdx.z > 0)) return;
    if (part < 4 && (kv.capacity == 0 || m == 0)) return;
    const int32_t* from = kv.table + b * kv.table_ld;
    const Route w = {a.kept + bh * a.budget, from, in_place || part == 4 ? from : a.dst_table + b * a.dst_ld,
                     kv.page_shift, (int)kv.capacity, m, in_place, (int)blockIdx.z, in_place ? 1 : (int)gridDim.z};
    const int kper = kv.head_dim * (kv.k_st == FP8_KV_BF16 ? 2 : 1) / 16;
    const int vper = kv.head_dim * (kv.v_st == FP8_KV_BF16 ? 2 : 1) / 16;
    // (K and V, or their scales, may be one array: it moves once)
    switch (part) {
    case 0:
        move_rows<IN_PLACE>(w, static_cast<attn::u4*>(kv.k) + (int64_t)h * kper, (int64_t)kv.heads * kper, kper);
        break;
    case 1:
        if (kv.v != kv.k)
            move_rows<IN_PLACE>(w, static_cast<attn::u4*>(kv.v) + (int64_t)h * vper, (int64_t)kv.heads * vper, vper);
        break;
    case 2:
        if (kv.k_scale && !kv.per_head) move_rows<IN_PLACE>(w, kv.k_scale + h, (int64_t)kv.heads, 1);
        break;
    case 3:
        if (kv.v_scale && kv.v_scale != kv.k_scale && !kv.per_head)
            move_rows<IN_PLACE>(w, kv.v_scale + h, (int64_t)kv.heads, 1);
        break;
    default: {
        const float* src = a.weights + bh * a.ldw;
        float* dst = a.weights_out + bh * a.ldwo;
        constexpr int rows = kMoveThreads * kPieces;
        for (int r0 = w.first * rows; r0 < m; r0 += w.step * rows) {
            float v[kPieces];
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                const int r = r0 + i * kMoveThreads + threadIdx.x;
                v[i] = r < m ? src[w.kept[r]] : 0.0f;
            }
            if (in_place) {
                __builtin_amdgcn_s_waitcnt(0);
                __syncthreads();
            }
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                const int r = r0 + i * kMoveThreads + threadIdx.x;
                if (r < m) dst[r] = v[i];
            }
        }
        // nothing has been received behind the kept tokens
        const int end = in_place ? n : a.budget;
        for (int r = m + w.first * kMoveThreads + threadIdx.x; r < end; r += w.step * kMoveThreads) dst[r] = 0.0f;
    }
    }
}

}  // namespace

hipError_t launch_evict(const EvictArgs& a) {
    const dim3 grid((unsigned)a.kv.heads, (unsigned)a.kv.batch), threads(kSelThreads);
    if (a.kv.max_len <= 8 * kSelThreads)
        hipLaunchKernelGGL(k_evict_select_regs<8>, grid, threads, 0, a.stream, a);
    else if (a.kv.max_len <= 32 * kSelThreads)
        hipLaunchKernelGGL(k_evict_select_regs<32>, grid, threads, 0, a.stream, a);
    else
        hipLaunchKernelGGL(k_evict_select, grid, threads, 0, a.stream, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    constexpr int parts = 5;
    const bool wide = a.kv.k_st == FP8_KV_BF16 || a.kv.v_st == FP8_KV_BF16;
    const int64_t widest = a.kv.head_dim * (wide ? 2 : 1) / 16;         // 16-byte pieces of a row
    const int64_t rows = kMoveThreads / widest * kPieces, tiles = (a.budget + rows - 1) / rows;
    const dim3 move((unsigned)(parts * a.kv.heads), (unsigned)a.kv.batch,
                    a.dst_table == nullptr ? 1u : (unsigned)(tiles < 1 ? 1 : tiles > 64 ? 64 : tiles));
    if (a.dst_table == nullptr)
        hipLaunchKernelGGL(k_evict_move<true>, move, dim3(kMoveThreads), 0, a.stream, a, parts);
    else
        hipLaunchKernelGGL(k_evict_move<false>, move, dim3(kMoveThreads), 0, a.stream, a, parts);
    return hipGetLastError();
}

}  // namespace fp8mi
