// attn_decode.hip -- attention of one new token per sequence over the paged
// KV cache on gfx950, read in place: split over the cache's length, joined by
// a second kernel.
//
// Mathematics, for a query head and the tokens j it sees, in powers of two:
//   x_j = (q . k_j) * scale_k_j * scale * log2(e)
//   m = max x_j,  l = sum 2^(x_j - m),  o = sum 2^(x_j - m) * scale_v_j * v_j
//   out = o / l,  lse = (m + log2 l) * ln 2
// with k_j, v_j the decoded codes (exact in bf16) and the FP8 scales applied
// to the fp32 score and to the fp32 weight, so neither loses bits to them.
// (m, l, o) of disjoint sets of tokens join by m = max, l and o scaled by
// 2^(m_s - m) and added.
//
// Layout.  A wave takes steps of 32 tokens of one (sequence, KV head) on its
// own; the query heads that share the KV head are the 16 columns of the
// matrix instruction (16x16x32 bf16), so a cached vector is read once for all
// of them.  Scores come as S^T = K Q^T: a lane gets, for its query column,
// the tokens 4g..4g+3 of each half step (g = lane / 16), which are exactly
// the 8 weights it has to hold as the B operand of O^T = V^T P^T when that
// product's 32 tokens are numbered the same way.  Weights therefore never
// leave their lane, and K and V go from memory to registers without LDS: K
// rows as 16-byte pieces in the A operand's order, V rows as VD consecutive
// channels a lane, transposed in registers by byte permutes between pairs of
// tokens before the codes become bf16.  LDS carries only the step's 32 row
// numbers and 64 scales.
//
// P is held as bf16 head plus bf16 remainder (two matrix products), so that
// the weights keep 16 significant bits; the kernel waits for memory, not for
// the matrix cores, and the second product costs nothing that shows.  An
// infinite value of V times a remainder would be the opposite infinity or
// NaN, so a step that holds one multiplies the remainders with its finite
// values alone (looking for them: bf16 K and V of 128 channels, 64 sequences up
// to 4096, 113 -> 116 us, other storages the same time).
//
// Bound by HBM: 2 * group operations a code byte.  Measured on one MI355X, 8
// KV heads of 128, group 4: 8 sequences of 65536 tokens (E5M2, scale per
// head) 197 us = 5.5 TB/s, where a read-only probe reaches 7.2; 64 ragged
// sequences up to 4096 (E4M3, scale per (token, head), pages of 16) 65 us =
// 4.3 TB/s, of which the join is 5.  One sequence of 517 tokens takes 15 us:
// lens -> page entry -> scales, K and V are dependent reads, then the join.
#include <hip/hip_runtime.h>

#include "attn_decode.hpp"

namespace fp8mi {
namespace {

using namespace attn;
using namespace decode;

constexpr int kMaxScored = 64;  // query heads of a KV head up to which scores are stored for the weights

template <int KST, int VST, int DP, int NT>
__global__ __launch_bounds__(64 * kWaves, DP <= 128 && NT == 1 ? 2 : 1) void k_decode(const DecodeParams a) {
    decode_share<KST, VST, DP, NT, kWhole>(a, (int)blockIdx.x, [](int) { return 0; });
}

constexpr int kJoinThreads = 256;
constexpr int kJoinWaves = kJoinThreads / 64;

// weights[b, h, j] += sum over the group of 2^(x_j - lse), one thread a token.
__global__ __launch_bounds__(kJoinThreads) void k_decode_weights(const DecodeParams a) {
    const int h = blockIdx.x % a.kv.heads, tile = blockIdx.x / a.kv.heads, b = blockIdx.y;
    const int at = tile * kJoinThreads + threadIdx.x, lane = threadIdx.x & 63;
    const int pos = seq_len(a.kv, b) - 1;
    const Steps<kStep> steps(pos, pos, a.window, a.sinks);
    if (tile * kJoinThreads >= steps.count * kStep) return;
    const int j = steps.token(at / kStep) + at % kStep;
    const bool seen = at < steps.count * kStep && sees(j, pos, a.window, a.sinks);
    const int64_t hq0 = (int64_t)b * a.q_heads + h * a.group;
    float w = 0.0f;
    const float z = lane < a.group ? a.lse[hq0 + lane] * kLog2e : 0.0f;     // at most kMaxScored heads
#pragma unroll 4
    for (int g = 0; g < a.group; ++g) {
        const float lse = as_f32(__builtin_amdgcn_readlane(__builtin_bit_cast(int, z), g));
        const float x = seen ? a.scores[(hq0 + g) * a.span + at] : -INFINITY;
        w += x == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(x - lse);
    }
    if (seen) a.weights[((int64_t)b * a.kv.heads + h) * a.ldw + j] += w;
}

// Joins the pieces of a sequence that several shares hold, in their order: a
// query head takes `a.join_waves` waves of a block, a thread 4 channels, and
// what a wave has lanes for goes on to further pieces side by side.
__global__ __launch_bounds__(kJoinThreads) void k_decode_join(const DecodeParams a) {
    __shared__ f4 s_acc[kJoinThreads];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), b = blockIdx.y;
    const int W = a.join_waves, part_of = wave % W;
    const int hq = blockIdx.x * (kJoinWaves / W) + wave / W;
    const Work w = work_of<kWhole>(a, 0, b, lane);
    const int i0 = w.before / w.chunk, n = (w.before + steps_of<kWhole>(a, w.len) - 1) / w.chunk - i0 + 1;
    if (n <= 1 || hq >= a.q_heads) return;              // the same for all W waves
    const int D = a.kv.head_dim, quads = D >> 2;
    const int64_t part = (int64_t)(i0 + b) * a.q_heads + hq, next = a.q_heads;
    const float2* ml = a.part_ml + part;
    const int sides = 64 / quads, side = lane / quads, d = (lane - side * quads) * 4;
    const int s0 = part_of * sides + side, apart = W * sides;
    const bool on = side < sides;
    // the first pieces are read beside the maxima and sums
    constexpr int kFirst = 4;
    f4 o[kFirst];
    float piece_m[kFirst];
#pragma unroll
    for (int i = 0; i < kFirst; ++i) {
        const int64_t s = min(s0 + i * apart, n - 1) * next;
        o[i] = *reinterpret_cast<const f4*>(a.part_o + (part + s) * D + d);
        piece_m[i] = ml[s].x;
    }
    const float2 all = join_ml(ml, next, n, lane);
    const float m = all.x, l = all.y;
    f4 acc = {0, 0, 0, 0};
    if (on) {
#pragma unroll
        for (int i = 0; i < kFirst; ++i)
            if (s0 + i * apart < n) acc += o[i] * __builtin_amdgcn_exp2f(piece_m[i] - m);
#pragma unroll 4
        for (int s = s0 + kFirst * apart; s < n; s += apart) {
            const float f = __builtin_amdgcn_exp2f(ml[s * next].x - m);
            acc += *reinterpret_cast<const f4*>(a.part_o + (part + s * next) * D + d) * f;
        }
    }
    s_acc[threadIdx.x] = acc;
    if (W == 1) wave_sync();
    else __syncthreads();
    if (side != 0 || part_of != 0) return;
    const f4* mine = s_acc + (threadIdx.x - lane);
    for (int v = 0; v < W; ++v)
        for (int s = v == 0 ? 1 : 0; s < sides; ++s) acc += mine[v * 64 + s * quads + lane];
    const float r = l == 0.0f ? 0.0f : 1.0f / l;
    *reinterpret_cast<uint2*>(a.out + b * a.ldo + (int64_t)hq * D + d) =
        make_uint2(pack2(acc[0] * r, acc[1] * r), pack2(acc[2] * r, acc[3] * r));
    if (d == 0 && a.lse)
        a.lse[(int64_t)b * a.q_heads + hq] = l == 0.0f ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * kLn2;
}

// How a launch is shared out: waves per KV head and column tile.
struct Plan {
    int col_tiles, wide, shares, least;
    bool joined;                 // a sequence may lie in several shares
    bool scores;                 // the weights come from stored scores
    int64_t blocks, span;        // span: tokens of the longest sequence's steps
};

Plan plan_of(const AttnArgs& a) {
    Plan p;
    const int group = a.q_heads / a.kv.heads;
    p.wide = group > 16 && a.kv.head_dim <= 128 ? 2 : 1;    // column tiles of a wave (256 channels: registers for one)
    p.col_tiles = (group + 16 * p.wide - 1) / (16 * p.wide);
    int64_t steps = (a.kv.max_len + kStep - 1) / kStep;     // of the longest sequence
    if (a.window > 0) {
        const int64_t seen = (a.window + kStep - 1) / kStep + 1 + (a.sinks + kStep - 1) / kStep;
        steps = seen < steps ? seen : steps;
    }
    if (steps < 1) steps = 1;
    const int64_t units = (int64_t)a.kv.heads * p.col_tiles, most = steps * a.kv.batch;
    // 2048 waves are two per SIMD, all resident at once, so equal shares end
    // together; 1.5 to 6 times as many (more loads in flight, but more partial
    // results and a second round) took 3-40 % longer over batches of 1 to 64.
    const int64_t target = 2048;
    p.least = 4;                 // steps worth a share's prologue and its row in the join
    int64_t shares = (target + units - 1) / units;
    shares = shares < most ? shares : most;
    p.shares = (int)(shares < 1 ? 1 : shares);
    p.joined = steps > 1;
    p.span = steps * kStep;
    // Weights from stored scores, or from the keys read again by k_weights,
    // which takes 32 rows of queries at a time however few there are.  16
    // sequences up to 8192, whole calls in us, stored / read again: 8 KV heads
    // of 128 in E4M3, group 4 56 / 142, group 32 110 / 180; 2 KV heads, group
    // 64 77 / 84 (bf16 79 / 82, 256 channels 102 / 130), group 128 117 / 105.
    p.scores = a.weighted && group <= kMaxScored;
    p.blocks = ((p.shares + 7) / 8 * units + kWaves - 1) / kWaves * 8;
    return p;
}

int64_t weights_tiles(const Plan& p) { return (p.span + kJoinThreads - 1) / kJoinThreads; }

template <int KST, int VST, int DP>
hipError_t launch_wide(const DecodeParams& p, const Plan& plan, hipStream_t stream) {
    const dim3 grid((unsigned)plan.blocks), block(64 * kWaves);
    if constexpr (DP <= 128) {
        if (plan.wide == 2) {
            hipLaunchKernelGGL((k_decode<KST, VST, DP, 2>), grid, block, 0, stream, p);
            return hipGetLastError();
        }
    }
    hipLaunchKernelGGL((k_decode<KST, VST, DP, 1>), grid, block, 0, stream, p);
    return hipGetLastError();
}

template <int KST, int VST>
hipError_t launch_dim(const DecodeParams& p, const Plan& plan, hipStream_t stream) {
    if (p.kv.head_dim <= 64) return launch_wide<KST, VST, 64>(p, plan, stream);
    if (p.kv.head_dim <= 128) return launch_wide<KST, VST, 128>(p, plan, stream);
    return launch_wide<KST, VST, 256>(p, plan, stream);
}

template <int KST>
hipError_t launch_v(const DecodeParams& p, const Plan& plan, hipStream_t stream) {
    switch (p.kv.v_st) {
    case FP8_KV_E4M3: return launch_dim<KST, kE4M3>(p, plan, stream);
    case FP8_KV_E5M2: return launch_dim<KST, kE5M2>(p, plan, stream);
    default: return launch_dim<KST, kBf16>(p, plan, stream);
    }
}

}  // namespace

// Bytes of the parts of the workspace: (m, l) and o of the pieces, scores.
struct Parts {
    int64_t ml = 0, o = 0, scores = 0;
    Parts(const AttnArgs& a, const Plan& p) {
        const int64_t pieces = p.joined ? (int64_t)(p.shares + a.kv.batch) * a.q_heads : 0;
        ml = (pieces * 8 + 15) / 16 * 16;
        o = pieces * a.kv.head_dim * 4;
        scores = p.scores ? (int64_t)a.kv.batch * a.q_heads * p.span * 4 : 0;
    }
};

int64_t decode_workspace(const AttnArgs& a) {
    const Parts parts(a, plan_of(a));
    return parts.ml + parts.o + parts.scores;
}

// Of the launch that computes the weights: the others have a few thousand blocks.
int64_t decode_blocks(const AttnArgs& a) {
    if (!a.weighted) return 0;
    const Plan plan = plan_of(a);
    return plan.scores ? weights_tiles(plan) * a.kv.heads : extend_blocks(a, false);
}

hipError_t launch_decode(const AttnArgs& a) {
    const Plan plan = plan_of(a);
    DecodeParams p;
    p.kv = a.kv; p.q = a.q; p.ldq = a.ldq; p.q_heads = a.q_heads; p.group = a.q_heads / a.kv.heads;
    p.col_tiles = plan.col_tiles; p.scale_log2 = a.scale * kLog2e; p.window = a.window; p.sinks = a.sinks; p.from = 0;
    p.shares = plan.shares; p.least = plan.least; p.out = a.out; p.ldo = a.ldo; p.lse = a.lse;
    const Parts parts(a, plan);
    p.part_ml = reinterpret_cast<float2*>(a.workspace);
    p.part_o = reinterpret_cast<float*>(a.workspace + parts.ml);
    p.scores = plan.scores ? reinterpret_cast<float*>(a.workspace + parts.ml + parts.o) : nullptr;
    p.span = plan.span; p.weights = a.weights; p.ldw = a.ldw;
    // Few pieces a sequence: a wave each is enough, in a quarter of the blocks
    // (64 sequences of 5 pieces 5.0 us against 8.2; 16 of 17 pieces 6.2 against 5.6).
    p.join_waves = plan.shares / a.kv.batch > 8 ? kJoinWaves : 1;
    hipError_t e;
    switch (a.kv.k_st) {
    case FP8_KV_E4M3: e = launch_v<kE4M3>(p, plan, a.stream); break;
    case FP8_KV_E5M2: e = launch_v<kE5M2>(p, plan, a.stream); break;
    default: e = launch_v<kBf16>(p, plan, a.stream); break;
    }
    if (e != hipSuccess) return e;
    if (plan.joined) {
        const unsigned heads = (unsigned)(kJoinWaves / p.join_waves);
        hipLaunchKernelGGL(k_decode_join, dim3(((unsigned)a.q_heads + heads - 1) / heads, (unsigned)a.kv.batch),
                           dim3(kJoinThreads), 0, a.stream, p);
        e = hipGetLastError();
    }
    if (e != hipSuccess || !a.weighted) return e;
    if (!plan.scores) return launch_attention_weights(a);
    const unsigned tiles = (unsigned)weights_tiles(plan);
    hipLaunchKernelGGL(k_decode_weights, dim3(tiles * (unsigned)a.kv.heads, (unsigned)a.kv.batch), dim3(kJoinThreads),
                       0, a.stream, p);
    return hipGetLastError();
}

}  // namespace fp8mi
