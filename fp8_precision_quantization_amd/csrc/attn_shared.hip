// attn_shared.hip -- attention of a batch whose sequences begin with the same
// tokens, in the same pages: the shared prefix is read once for all of them.
//
// Mathematics: that of attn_decode.hip and attn_extend.hip.  The tokens a row
// sees are cut at the prefix's end; both parts give (m, l, o), which join by
// m = max, l and o scaled by 2^(m_s - m) and added.
//
// k_shared.  One launch holds two kinds of blocks.  To the prefix, the batch is
// one sequence without an order: the rows are (query, head in the group) of all
// sequences, 128 a block, and a KV head's blocks share the prefix's steps in even
// parts (extend_rows: matrix products against LDS tiles; a row's own position
// masks only where a sequence ends inside the prefix).  Behind it every sequence
// has tokens of its own: with one new token each, waves share them evenly whatever
// their lengths (decode_share, memory bound); with several, as row tiles of
// their sequence (extend_rows).  The two kinds need different parts of a CU, so
// they are resident together rather than one after the other.
//
// k_shared_few.  Up to 32 rows of one new token each read the prefix as waves read
// the tails, 16 rows a wave against 32-token steps in registers: less parallel
// work in a row (4 sequences, 2000 + up to 130 tokens: 13.2 us), but an eighth of
// a block tile's products and none of its partial results' 64 KiB (4 sequences on
// 32768 tokens 28 us against 42, 8 sequences 33 against 42, 16 sequences 50
// against 44).
//
// k_shared_join reads a row's pieces of both parts in their order.
//
// Measured (8 KV heads of 128 and 32 query heads; in brackets every sequence by
// itself, kv_attention without a prefix): 64 sequences on 8192 shared tokens of
// E4M3 and up to 600 of their own 28 us and 7 for the join (138 together); 24 with
// six new tokens each on 32768 of E5M2 and up to 1000, 90 and 7 (481).  A block of
// the prefix takes 11 us (three dependent reads, then 64 KiB of partial results,
// 3 us of them) and 1.8 us a step of 64 tokens, bound by the decoding and softmax
// beside the products; the tails hide behind it (27.0 us without them, 28.2 with).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "attn_decode.hpp"
#include "attn_extend.hpp"

namespace fp8mi {
namespace {

using namespace attn;

struct SharedParams {
    extend::ExtendParams e;      // splits: pieces of a row, the prefix's first; least: fewest steps of a tail's piece
    decode::DecodeParams d;      // the tails where every sequence has one new token
    decode::DecodeParams few;    // the prefix where the queries are few
    int from;                    // tokens of the prefix, a multiple of extend::kStep
    int blocks;                  // of the prefix
    bool is_few;                 // the prefix is read by k_shared_few
    int splits, chunk;           // of the prefix: pieces, their steps
    int tail_splits;             // of a tail's row tile
    int tail_tiles;
};

// A query of the call: whether it is in a sequence, its place there, its position.
struct Place {
    bool in;
    int b, i, n, pos;
    __device__ __forceinline__ Place(const extend::ExtendParams& a, int token) : b(0) {
        if (a.q_offsets == nullptr) {
            b = min(token / a.each, a.kv.batch - 1);
        } else {
            for (int hi = a.kv.batch; hi - b > 1;) {
                const int mid = (b + hi) >> 1;
                if (a.q_offsets[mid] <= token) b = mid; else hi = mid;
            }
        }
        int first;
        extend::queries_of(a, b, &first, &n);
        i = token - first;
        in = i >= 0 && i < n;
        pos = seq_len(a.kv, b) - n + i;
    }
};

template <int KST, int VST, int DP, bool kOne>
__global__ __launch_bounds__(extend::kThreads, DP <= 128 ? 2 : 1) void k_shared(const SharedParams p) {
    extern __shared__ __align__(16) uint8_t smem[];
    const extend::ExtendParams& a = p.e;
    const KvView& kv = a.kv;
    const bool prefix = (int)blockIdx.x < p.blocks;
    if (kOne && !prefix) {
        decode::decode_share<KST, VST, DP, 1, decode::kTail>(p.d, (int)blockIdx.x - p.blocks, [](int) { return 0; });
        return;
    }
    int block = (int)blockIdx.x - (prefix ? 0 : p.blocks);
    const int h = block % kv.heads;
    block /= kv.heads;
    const int lane_row = (int)(threadIdx.x >> 6) * 32 + (int)(threadIdx.x & 31);
    extend::Rows at;
    Steps<extend::kStep> steps(-1, -1, 0, 0);
    at.partial = true;
    if (prefix) {
        const int split = block % p.splits, r = block / p.splits * extend::kRows + lane_row, token = r / a.group;
        const Place place(a, token);
        at.live = token < a.total_q && place.in;
        at.token = token;
        at.head = h * a.group + (r - token * a.group);
        at.pos = at.live ? place.pos : -1;
        at.p_first = -1;            // a sequence may end inside the prefix
        at.p_last = p.from - 1;
        at.table = kv.table;
        steps = Steps<extend::kStep>(p.from - 1, p.from - 1, 0, 0);
        at.s_begin = split * p.chunk;
        at.s_end = min(at.s_begin + p.chunk, steps.count);
        at.part = split;
    } else {
        const int split = block % p.tail_splits;
        const extend::Tile tile(a, p.tail_tiles - 1 - block / p.tail_splits);
        if (!tile.any()) return;
        steps = Steps<extend::kStep>(tile.p_last, tile.p_last, 0, 0, p.from);
        const int even = (steps.count + p.tail_splits - 1) / p.tail_splits, chunk = max(even, a.least);
        at.s_begin = split * chunk;
        at.s_end = min(at.s_begin + chunk, steps.count);
        if (at.s_begin >= steps.count) return;
        const int r = tile.row0 + lane_row, tok = r / a.group;
        at.live = r < tile.rows;
        at.token = tile.q_first + tok;
        at.head = h * a.group + (r - tok * a.group);
        at.pos = at.live ? tile.base + tok : -1;
        at.p_first = max(tile.p_first, 0);
        at.p_last = tile.p_last;
        at.table = kv.table + tile.b * kv.table_ld;
        at.part = p.splits + split;
    }
    extend::extend_rows<KST, VST, DP, true>(a, *reinterpret_cast<extend::Lds<DP>*>(smem), h, steps, at);
}

// Few queries, one new token a sequence: waves read the prefix as they read the
// tails, its columns being the query heads of all sequences, 16 a wave.
template <int KST, int VST, int DP>
__global__ __launch_bounds__(64 * decode::kWaves, DP <= 128 ? 2 : 1) void k_shared_few(const SharedParams p) {
    const int block = (int)blockIdx.x - p.blocks;
    if (block < 0)
        decode::decode_share<KST, VST, DP, 1, decode::kPrefix>(
            p.few, (int)blockIdx.x, [&](int token) { return seq_len(p.few.kv, token) - 1; });
    else
        decode::decode_share<KST, VST, DP, 1, decode::kTail>(p.d, block, [](int) { return 0; });
}

constexpr int kJoinThreads = 256;
constexpr int kJoinWaves = kJoinThreads / 64;

// Joins the pieces of a row, the prefix's first, in their order.  A row takes W
// waves of a block, a thread 4 channels, and what a wave has lanes for goes on to
// further pieces side by side.  The prefix's first pieces are on their way while
// the tail's are looked up.
template <bool kOne>
__global__ __launch_bounds__(kJoinThreads) void k_shared_join(const SharedParams p, int W) {
    constexpr int kFirst = 8;
    __shared__ f4 s_acc[kJoinThreads];
    const extend::ExtendParams& a = p.e;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int rows = a.total_q * a.q_heads, mine = (int)blockIdx.x * (kJoinWaves / W) + wave / W;
    const int row = min(mine, rows - 1);                // (token, query head)
    const int part_of = wave % W;
    const int D = a.kv.head_dim, quads = D >> 2, sides = 64 / quads, side = lane / quads, d = (lane - side * quads) * 4;
    const int token = row / a.q_heads, hq = row - token * a.q_heads, h = hq / a.group;
    const int at = part_of * sides + side, apart = W * sides;
    const float2* const pre_ml = a.part_ml + (int64_t)row * a.splits;
    const float* const pre_o = a.part_o + (int64_t)row * a.splits * D + d;
    const bool on = side < sides;
    f4 o[kFirst];
    float o_m[kFirst];
#pragma unroll
    for (int i = 0; i < kFirst; ++i) {
        const int piece = min(at + i * apart, p.splits - 1);
        o[i] = *reinterpret_cast<const f4*>(pre_o + (int64_t)piece * D);
        o_m[i] = pre_ml[piece].x;
    }
    const float2 ml = pre_ml[min(lane, p.splits - 1)];
    // (a wave's V scale of the head is in its weights already)
    const float by_head = p.is_few ? 1.0f : extend::v_scale_of(a.kv, h);

    // the tail's pieces: where they are, how far apart, how many
    bool there = mine < rows;
    int n = 0;
    const float2* tail_ml = nullptr;
    const float* tail_o = nullptr;
    int64_t next = 1;
    float tail_head = 1.0f;
    if constexpr (kOne) {
        const decode::Work w = decode::work_of<decode::kTail>(p.d, 0, token, lane);
        const int i0 = w.before / w.chunk;
        n = (w.before + decode::steps_of<decode::kTail>(p.d, w.len) - 1) / w.chunk - i0 + 1;
        const int64_t first = (int64_t)(i0 + token) * a.q_heads + hq;
        tail_ml = p.d.part_ml + first;
        tail_o = p.d.part_o + first * D + d;
        next = a.q_heads;
    } else {
        const Place place(a, token);
        there = there && place.in;
        if (place.in) {
            // the row tile that this row is in: its last position bounds the steps
            const int r0 = (place.i * a.group + hq - h * a.group) / extend::kRows * extend::kRows;
            const int last = place.pos - place.i + (min(r0 + extend::kRows, place.n * a.group) - 1) / a.group;
            const int steps = Steps<extend::kStep>(last, last, 0, 0, p.from).count;
            const int even = (steps + p.tail_splits - 1) / p.tail_splits, chunk = max(even, a.least);
            n = (steps + chunk - 1) / chunk;
        }
        tail_ml = pre_ml + p.splits;
        tail_o = pre_o + (int64_t)p.splits * D;
        tail_head = by_head;
    }
    float m = ml.x;
    for (int i = lane + 64; i < p.splits; i += 64) m = fmaxf(m, pre_ml[i].x);
    for (int i = lane; i < n; i += 64) m = fmaxf(m, tail_ml[i * next].x);
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) m = fmaxf(m, __shfl_xor(m, off, 64));
    float l = lane < p.splits ? ml.y * __builtin_amdgcn_exp2f(ml.x - m) : 0.0f;
    for (int i = lane + 64; i < p.splits; i += 64) l += pre_ml[i].y * __builtin_amdgcn_exp2f(pre_ml[i].x - m);
    for (int i = lane; i < n; i += 64) l += tail_ml[i * next].y * __builtin_amdgcn_exp2f(tail_ml[i * next].x - m);
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) l += __shfl_xor(l, off, 64);

    f4 acc = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < kFirst; ++i)
        if (at + i * apart < p.splits) acc += o[i] * __builtin_amdgcn_exp2f(o_m[i] - m);
#pragma unroll 4
    for (int i = at + kFirst * apart; i < p.splits; i += apart)
        acc += *reinterpret_cast<const f4*>(pre_o + (int64_t)i * D) * __builtin_amdgcn_exp2f(pre_ml[i].x - m);
    acc *= by_head;
#pragma unroll 2
    for (int i = at; i < n; i += apart)
        acc += *reinterpret_cast<const f4*>(tail_o + i * next * D) *
               (tail_head * __builtin_amdgcn_exp2f(tail_ml[i * next].x - m));
    s_acc[threadIdx.x] = acc;
    if (W == 1) wave_sync();
    else __syncthreads();
    if (!on || side != 0 || part_of != 0 || !there) return;
    const f4* const others = s_acc + (threadIdx.x - lane);
    for (int v = 0; v < W; ++v)
        for (int s = v == 0 ? 1 : 0; s < sides; ++s) acc += others[v * 64 + s * quads + lane];
    const float r = l == 0.0f ? 0.0f : 1.0f / l;
    *reinterpret_cast<uint2*>(a.out + (int64_t)token * a.ldo + (int64_t)hq * D + d) =
        make_uint2(pack2(acc[0] * r, acc[1] * r), pack2(acc[2] * r, acc[3] * r));
    if (d == 0 && a.lse) a.lse[row] = l == 0.0f ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * kLn2;
}

// How a call is shared out.
struct Plan {
    bool one, few;
    int64_t prefix_blocks, tail_blocks;
    int splits, chunk;               // of the prefix
    int tail_splits, least, tail_tiles;
    int shares;                      // one new token a sequence: as attn_decode.hip's
    int64_t ml, o, tail_ml, tail_o;  // bytes of the parts of the workspace
};

// Waves of the join that share a row: 128 rows 13.3 us a call with four, 15.0 with
// one; 512 rows 23.1 and 21.7, 2048 rows 38.3 and 36.7.
int join_waves(int64_t rows) { return rows < 512 ? kJoinWaves : 1; }

int64_t up16(int64_t n) { return (n + 15) / 16 * 16; }

// Numbers that the plan aims at, of 256 CUs, E4M3 with 32 query heads on 8 KV heads
// of 128 unless named otherwise, us a call:
// - blocks of the prefix: 64 sequences of one token on 8192 and up to 600 of their
//   own with 128, 256, 384, 512 of them 47, 36, 44, 51 (200 on 16384: 249, 139, 127,
//   104); of several tokens, 24 times 6 on 32768 of E5M2, 311, 172, 152, 132, but 8
//   times 4 on 4096 21, 28, 28, 28;
// - parts of a row: 16 to 128 at most differ nowhere but there (16: 22);
// - waves of few queries' prefix: 8 sequences on 32768 with 512, 1024, 2048 of them
//   47, 34, 38;
// - waves of tails of one token: 64 sequences up to 600 behind 8192 with 512, 1024,
//   2048 39, 36, 38, 32 up to 8000 behind 2048 156, 112, 118;
// - steps of such a wave, at least: 4 sequences up to 130 behind 2000 with 1, 2, 4
//   15, 15, 17;
// - blocks of tails of several tokens: 8 times 4 on 1024 and up to 12000 with 256,
//   512, 1024 98, 79, 82; parts of a row tile, 24 times 6 as above with 8, 16, 32 at
//   most 157, 151, 151; steps of a part, 8 times 4 on 4096 with 2, 4, 8 at least 24,
//   28, 28, elsewhere the same.
Plan plan_of(const AttnArgs& a, bool ragged) {
    Plan p = {};
    const int64_t group = a.q_heads / a.kv.heads, rows = a.total_q * group, heads = a.kv.heads;
    p.one = !ragged && a.total_q == a.kv.batch;
    const int64_t tiles = (rows + extend::kRows - 1) / extend::kRows;
    const int64_t steps = a.from / extend::kStep, tail = std::max<int64_t>(a.kv.max_len - a.from, 0);
    const int64_t want = p.one ? 256 : 384;
    int64_t s = std::clamp<int64_t>(want / (tiles * heads), 1, std::min<int64_t>(64, std::max<int64_t>(steps / 2, 1)));
    p.chunk = (int)((steps + s - 1) / s);
    p.splits = (int)((steps + p.chunk - 1) / p.chunk);
    p.prefix_blocks = tiles * heads * p.splits;
    p.few = p.one && rows <= 32;
    if (p.few) {
        const int64_t units = heads * ((rows + 15) / 16), all = a.from / decode::kStep;
        s = std::clamp<int64_t>(1024 / units, 1, std::max<int64_t>(all / 2, 1));
        p.chunk = (int)((all + s - 1) / s);
        p.splits = (int)((all + p.chunk - 1) / p.chunk);
        p.prefix_blocks = ((p.splits + 7) / 8 * units + decode::kWaves - 1) / decode::kWaves * 8;
    }
    if (p.one) {
        const int64_t units = heads * ((group + 15) / 16);
        const int64_t most = std::max<int64_t>((tail + decode::kStep - 1) / decode::kStep, 1) * a.kv.batch;
        p.shares = (int)std::max<int64_t>(std::min<int64_t>((1024 + units - 1) / units, most), 1);
        p.tail_blocks = ((p.shares + 7) / 8 * units + decode::kWaves - 1) / decode::kWaves * 8;
        const int64_t pieces = (int64_t)(p.shares + a.kv.batch) * a.q_heads;
        p.tail_ml = up16(pieces * 8);
        p.tail_o = pieces * a.kv.head_dim * 4;
    } else {
        const int64_t each = a.total_q / a.kv.batch;
        p.tail_tiles = (int)(ragged ? rows / extend::kRows + a.kv.batch
                                    : a.kv.batch * ((each * group + extend::kRows - 1) / extend::kRows));
        const int64_t tail_steps = (tail + extend::kStep - 1) / extend::kStep;
        p.least = 4;
        p.tail_splits = (int)std::clamp<int64_t>(std::min(512 / (p.tail_tiles * heads), tail_steps / 4), 1, 16);
        p.tail_blocks = (int64_t)p.tail_tiles * heads * p.tail_splits;
    }
    const int64_t pieces = a.total_q * a.q_heads * (p.splits + p.tail_splits);
    p.ml = up16(pieces * 8);
    p.o = pieces * a.kv.head_dim * 4;
    return p;
}

template <int KST, int VST, int DP, bool kOne>
hipError_t run(const SharedParams& p, const Plan& plan, hipStream_t stream) {
    constexpr int bytes = sizeof(extend::Lds<DP>);
    static_assert(bytes <= 158 * 1024, "LDS");
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&k_shared<KST, VST, DP, kOne>),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((k_shared<KST, VST, DP, kOne>), dim3((unsigned)(plan.prefix_blocks + plan.tail_blocks)),
                       dim3(extend::kThreads), bytes, stream, p);
    return hipGetLastError();
}

template <int KST, int VST, int DP>
hipError_t run_few(const SharedParams& p, const Plan& plan, hipStream_t stream) {
    hipLaunchKernelGGL((k_shared_few<KST, VST, DP>), dim3((unsigned)(plan.prefix_blocks + plan.tail_blocks)),
                       dim3(64 * decode::kWaves), 0, stream, p);
    return hipGetLastError();
}

template <int KST, int VST, bool kOne>
hipError_t run_dim(const SharedParams& p, const Plan& plan, hipStream_t stream) {
    const int D = p.e.kv.head_dim;
    if (kOne && plan.few)
        return D <= 64    ? run_few<KST, VST, 64>(p, plan, stream)
               : D <= 128 ? run_few<KST, VST, 128>(p, plan, stream)
                          : run_few<KST, VST, 256>(p, plan, stream);
    return D <= 64    ? run<KST, VST, 64, kOne>(p, plan, stream)
           : D <= 128 ? run<KST, VST, 128, kOne>(p, plan, stream)
                      : run<KST, VST, 256, kOne>(p, plan, stream);
}

template <int KST, bool kOne>
hipError_t run_v(const SharedParams& p, const Plan& plan, hipStream_t stream) {
    switch (p.e.kv.v_st) {
    case FP8_KV_E4M3: return run_dim<KST, kE4M3, kOne>(p, plan, stream);
    case FP8_KV_E5M2: return run_dim<KST, kE5M2, kOne>(p, plan, stream);
    default: return run_dim<KST, kBf16, kOne>(p, plan, stream);
    }
}

template <bool kOne>
hipError_t run_k(const SharedParams& p, const Plan& plan, hipStream_t stream) {
    hipError_t e;
    switch (p.e.kv.k_st) {
    case FP8_KV_E4M3: e = run_v<kE4M3, kOne>(p, plan, stream); break;
    case FP8_KV_E5M2: e = run_v<kE5M2, kOne>(p, plan, stream); break;
    default: e = run_v<kBf16, kOne>(p, plan, stream); break;
    }
    if (e != hipSuccess) return e;
    const int64_t rows = (int64_t)p.e.total_q * p.e.q_heads;
    const int W = join_waves(rows);
    hipLaunchKernelGGL((k_shared_join<kOne>), dim3((unsigned)((rows * W + kJoinWaves - 1) / kJoinWaves)),
                       dim3(kJoinThreads), 0, stream, p, W);
    return hipGetLastError();
}

}  // namespace

int64_t shared_workspace(const AttnArgs& a, bool ragged) {
    const Plan p = plan_of(a, ragged);
    return p.ml + up16(p.o) + p.tail_ml + p.tail_o;
}

int64_t shared_blocks(const AttnArgs& a, bool ragged) {
    const Plan p = plan_of(a, ragged);
    return std::max({p.prefix_blocks + p.tail_blocks, a.total_q * a.q_heads * join_waves(a.total_q * a.q_heads) / kJoinWaves + 1,
                     a.weighted ? extend_blocks(a, ragged) : 0});
}

hipError_t launch_shared(const AttnArgs& a) {
    const Plan plan = plan_of(a, a.q_offsets != nullptr);
    SharedParams p = {};
    const int group = a.q_heads / a.kv.heads;
    p.e.kv = a.kv; p.e.q = a.q; p.e.ldq = a.ldq; p.e.total_q = (int)a.total_q; p.e.each = (int)(a.total_q / a.kv.batch);
    p.e.q_heads = a.q_heads; p.e.group = group; p.e.q_offsets = a.q_offsets; p.e.scale_log2 = a.scale * kLog2e;
    p.e.out = a.out; p.e.ldo = a.ldo; p.e.lse = a.lse;
    p.e.splits = plan.splits + plan.tail_splits; p.e.least = plan.least;
    p.e.part_ml = reinterpret_cast<float2*>(a.workspace);
    p.e.part_o = reinterpret_cast<float*>(a.workspace + plan.ml);
    p.from = a.from; p.blocks = (int)plan.prefix_blocks; p.splits = plan.splits; p.chunk = plan.chunk;
    p.tail_splits = plan.tail_splits; p.tail_tiles = plan.tail_tiles;
    if (plan.one) {
        p.d.kv = a.kv; p.d.q = a.q; p.d.ldq = a.ldq; p.d.q_heads = a.q_heads; p.d.group = group;
        p.d.col_tiles = (group + 15) / 16; p.d.scale_log2 = a.scale * kLog2e; p.d.from = a.from;
        p.d.shares = plan.shares; p.d.least = 2;
        uint8_t* tail = a.workspace + plan.ml + up16(plan.o);
        p.d.part_ml = reinterpret_cast<float2*>(tail);
        p.d.part_o = reinterpret_cast<float*>(tail + plan.tail_ml);
    }
    if (plan.few) {
        p.is_few = true;
        p.few = p.d;
        p.few.columns = (int)a.total_q * group;
        p.few.col_tiles = (p.few.columns + 15) / 16;
        p.few.shares = p.few.pieces = plan.splits;
        p.few.part_ml = p.e.part_ml;
        p.few.part_o = p.e.part_o;
    }
    const hipError_t e = plan.one ? run_k<true>(p, plan, a.stream) : run_k<false>(p, plan, a.stream);
    return e != hipSuccess || !a.weighted ? e : launch_attention_weights(a);
}

}  // namespace fp8mi
