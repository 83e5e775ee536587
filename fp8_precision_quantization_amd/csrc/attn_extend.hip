// attn_extend.hip -- attention of several tokens per sequence (prompts,
// chunks, drafted tokens) over the paged KV cache on gfx950, and the weights
// every cached token receives from a call's queries.
//
// k_extend.  The query heads of one KV head share its keys, so a sequence's
// rows are (token, head in the group), token-major; a block takes 128
// consecutive rows (32 a wave) of one KV head and walks the cached tokens any
// of them sees in steps of 64, with a running maximum and sum per row.
// A step's K and V go through registers into LDS as bf16 (decoded once for
// all waves) while the step before is computed on, and a step is taken in two
// halves of 32 tokens, so that the matrix products of one stand beside the
// exponentials of the other (prefill below: 345 -> 340 us).  Scores are
// S^T = K Q^T (32x32x16 bf16 products, queries as columns): a lane holds one
// row's scores for half of the step's tokens, so maxima and sums need one
// exchange (lanes l and l + 32), and the weights are already the B operand of
// O^T = V^T P^T when that product numbers its 16 tokens as the accumulator
// rows lie.  V^T is read from the row-major LDS tile by transposing reads.
// FP8 scales per token multiply the fp32 score and the fp32 weight, V's scale
// per head the fp32 output; the weight is then rounded once to bf16, by 2^-8
// of itself at most, while the row's sum adds it unrounded: an output is off
// by up to 2^-8 of sum p |v|, as much as its own bf16 rounding, for rows in
// which few tokens weigh most, and by less where many do, whose errors are
// independent.  (A second product with the remainder, as for one new token,
// would double the products with V.)  A row that sees one token has the weight
// 1 exactly: with bf16 V, a scale per head, or scales per token that are powers
// of two, it returns that token's values bit for bit.
//
// LDS rows are padded (K by 16 bytes, V by 64) so that the 16-byte reads of
// 16 K rows, and the transposing reads of 4 V rows, fall into different banks.
//
// Values of V that are not finite (and tokens whose own V scale is not): a product
// with weight 0 would turn a token that one row does not see into NaN for that
// row.  Staging puts 0 in their place and marks the step; a block that met one
// goes over its marked steps once more at the end and adds these values, row
// by row, to the rows that see them.
//
// Bound by the vector units and the matrix cores together: per 64-token step
// and row 64 exponentials, scale products, maxima and roundings stand against
// 256 operations a channel; counters read 67 % vector and 47 % matrix busy.
// Measured on one MI355X, 8 KV heads of 128, group 4: 2 prompts of 4096 (K
// bf16, V E4M3) 326-340 us = 810-840 TFLOP/s of visible products, where a
// library 8192^3 bf16 product reaches 1373; one prompt of 8192 in a window of
// 1024 202-212 us = 620 (18 steps a tile, three of them masked: the tile's
// prologue and epilogue are 15 %).  128 rows a block leave two blocks on a CU,
// so one's loads and barriers stand beside the other's products; 256 rows (one
// block) were 4 % faster on the first and 18 % slower on ragged short chunks.
//
// k_weights.  weights[b, h, j] += sum over the rows of 2^(x_ij - lse_i): a
// block owns 128 tokens of a (sequence, KV head) with their K in registers
// and walks the rows that see them, so every weight has one writer and the
// sums have a fixed order.  Bound by the vector units (an fma, an exponential
// and an addition a score) and by uneven blocks: 3 sequences of up to 512 new
// tokens over up to 4096 cached take 77 us.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "attn_extend.hpp"

namespace fp8mi {
namespace {

using namespace attn;
using namespace extend;

template <int KST, int VST, int DP>
__global__ __launch_bounds__(kThreads, DP <= 128 ? 2 : 1) void k_extend(const ExtendParams a) {
    extern __shared__ __align__(16) uint8_t smem[];
    const KvView& kv = a.kv;
    const int h = blockIdx.x % kv.heads, split = blockIdx.x / kv.heads % a.splits;
    // later (longer) tiles first
    const Tile tile(a, (int)(gridDim.x / kv.heads / a.splits - 1 - blockIdx.x / kv.heads / a.splits));
    if (!tile.any()) return;
    const Steps<kStep> steps(tile.p_first, tile.p_last, a.window, a.sinks);
    const int chunk = chunk_of(a, steps.count);
    Rows at;
    at.s_begin = split * chunk;
    at.s_end = min(at.s_begin + chunk, steps.count);
    if (at.s_begin >= steps.count && split > 0) return;
    const int r = tile.row0 + (int)(threadIdx.x >> 6) * 32 + (int)(threadIdx.x & 31), tok = r / a.group;
    at.live = r < tile.rows;
    at.token = tile.q_first + tok;
    at.head = h * a.group + (r - tok * a.group);
    at.pos = at.live ? tile.base + tok : -1;
    at.p_first = tile.p_first;
    at.p_last = tile.p_last;
    at.table = kv.table + tile.b * kv.table_ld;
    at.partial = chunk < steps.count;
    at.part = split;
    extend_rows<KST, VST, DP, false>(a, *reinterpret_cast<Lds<DP>*>(smem), h, steps, at);
}

// Joins the blocks of a row tile in their order; threads take 4 channels of a
// row each.
constexpr int kJoinRows = 16;

__global__ __launch_bounds__(kThreads) void k_extend_join(const ExtendParams a) {
    const int h = blockIdx.x % a.kv.heads;
    const Tile tile(a, blockIdx.x / a.kv.heads);
    if (!tile.any()) return;
    const Steps<kStep> steps(tile.p_first, tile.p_last, a.window, a.sinks);
    const int chunk = chunk_of(a, steps.count);
    if (chunk >= steps.count) return;
    const int n = (steps.count + chunk - 1) / chunk;
    const int D = a.kv.head_dim, quads = D >> 2;
    const int r0 = tile.row0 + blockIdx.y * kJoinRows, rn = min(r0 + kJoinRows, tile.rows) - r0;
    for (int i = threadIdx.x; i < rn * quads; i += kThreads) {
        const int r = r0 + i / quads, d = i % quads * 4;
        const int tok = tile.q_first + r / a.group, hq = h * a.group + r % a.group;
        const int64_t row = (int64_t)tok * a.q_heads + hq;
        const float2* ml = a.part_ml + row * a.splits;
        float m = kLowest, l = 0.0f;
        for (int s = 0; s < n; ++s) m = fmaxf(m, ml[s].x);
        f4 acc = {0, 0, 0, 0};
#pragma unroll 4
        for (int s = 0; s < n; ++s) {
            const float f = __builtin_amdgcn_exp2f(ml[s].x - m);
            l += ml[s].y * f;
            acc += *reinterpret_cast<const f4*>(a.part_o + (row * a.splits + s) * D + d) * f;
        }
        const float inv = l == 0.0f ? 0.0f : v_scale_of(a.kv, h) / l;
        *reinterpret_cast<uint2*>(a.out + (int64_t)tok * a.ldo + (int64_t)hq * D + d) =
            make_uint2(pack2(acc[0] * inv, acc[1] * inv), pack2(acc[2] * inv, acc[3] * inv));
        if (d == 0 && a.lse) a.lse[row] = l == 0.0f ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * kLn2;
    }
}

// Weights: a wave holds 32 tokens' K as the A operand; a step's queries go
// through LDS (read from memory row by row, as columns of the product they
// would be 64 separate lines a load: 168 us where LDS took 102) and are shared
// by the block's four waves, 128 rows at a time so that 32 rows' products
// stand beside the exponentials of the 32 before (101 -> 95 us against 64 rows
// one after the other; rows that advance without divisions 95 -> 78).
template <int DP>
struct WeightsLds {
    static constexpr int kR = DP <= 128 ? 128 : 64;     // rows of a step
    static constexpr int kQ = DP * 2 + 16;              // bytes of a padded row
    alignas(16) uint8_t q[2][kR * kQ];
    float lse[2][kR];
    int pos[2][kR];
};

template <int KST, int DP>
__global__ __launch_bounds__(kThreads, DP <= 128 ? 2 : 1) void k_weights(const ExtendParams a) {
    constexpr int KM = DP / 16;
    constexpr int KC = DP * kElemBytes<KST> / 32;       // 16-byte pieces of K a lane holds
    constexpr int R = WeightsLds<DP>::kR, kQ = WeightsLds<DP>::kQ;
    constexpr int PR = DP / 8, PT = R * PR / kThreads;  // 16-byte pieces of a row, of a thread
    extern __shared__ __align__(16) uint8_t smem[];
    WeightsLds<DP>& lds = *reinterpret_cast<WeightsLds<DP>*>(smem);
    auto& s_q = lds.q;
    auto& s_lse = lds.lse;
    auto& s_pos = lds.pos;
    const KvView& kv = a.kv;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int c = lane & 31, g = lane >> 5;
    const int h = blockIdx.x % kv.heads, b = blockIdx.y;
    const int len = seq_len(kv, b);
    const int block0 = (int)(blockIdx.x / kv.heads) * kRows, j0 = block0 + wave * 32;
    if (block0 >= len) return;
    int q_first, n;
    queries_of(a, b, &q_first, &n);
    const int G = a.group, D = kv.head_dim, base = len - n;

    // rows (token of the call, head in the group) that see any of the block's tokens
    int i_lo = block0 - base, i_hi = n;
    if (a.window > 0 && block0 >= a.sinks)      // (a window and a position may add up to 2^31)
        i_hi = (int)std::min<int64_t>(i_hi, (int64_t)block0 + kRows - 1 + a.window - base);
    i_lo = i_lo < 0 ? 0 : i_lo;
    if (i_lo >= i_hi) return;
    const int r_first = i_lo * G, r_end = i_hi * G;

    // Q of a step into registers and from there into LDS; a row past the end
    // reads one of the last token's and has an infinite lse: it gives nothing.
    // (token, head) of a thread's rows advance without divisions: pieces u and
    // u + 1 are kThreads / PR rows apart, steps R rows.
    struct RowAt {
        int tok, head;
        __device__ __forceinline__ void advance(int tokens, int heads, int group) {
            tok += tokens;
            head += heads;
            const bool over = head >= group;
            tok += over ? 1 : 0;
            head -= over ? group : 0;
        }
    };
    constexpr int kApart = kThreads / PR;
    const int piece_tok = kApart / G, piece_head = kApart - piece_tok * G;
    const int step_tok = R / G, step_head = R - step_tok * G;
    const int first_of = tid / PR, e_of = tid % PR * 8;     // row in the step, first channel
    RowAt q_at = {i_lo + first_of / G, first_of % G}, lse_at = {i_lo + tid % R / G, tid % R % G};
    const bool in_dim = D == DP || e_of < D;
    const uint32_t keep = in_dim ? ~0u : 0u;
    const uint16_t* q_base = a.q + (int64_t)q_first * a.ldq + (int64_t)h * G * D + (in_dim ? e_of : 0);
    const float* lse_base = a.lse + (int64_t)q_first * a.q_heads + h * G;
    uint4 qu[PT];
    float lse;
    int pos;
    auto load = [&](int r0) {
        RowAt at = q_at;
#pragma unroll
        for (int u = 0; u < PT; ++u) {
            qu[u] = *reinterpret_cast<const uint4*>(q_base + min(at.tok, i_hi - 1) * a.ldq + at.head * D);
            at.advance(piece_tok, piece_head, G);
        }
        q_at.advance(step_tok, step_head, G);
        const int tok = min(lse_at.tok, i_hi - 1);
        lse = lse_base[(int64_t)tok * a.q_heads + lse_at.head];
        lse = r0 + tid % R >= r_end || lse == -INFINITY ? INFINITY : lse * kLog2e;
        pos = base + tok;
        lse_at.advance(step_tok, step_head, G);
    };
    auto put = [&](int i) {
#pragma unroll
        for (int u = 0; u < PT; ++u)
            *reinterpret_cast<uint4*>(&s_q[i & 1][(first_of + u * kApart) * kQ + e_of * 2]) =
                make_uint4(qu[u].x & keep, qu[u].y & keep, qu[u].z & keep, qu[u].w & keep);
        if (tid < R) {
            s_lse[i & 1][tid] = lse;
            s_pos[i & 1][tid] = pos;
        }
    };
    load(r_first);

    const int j = j0 + c;
    int row = -1;
    if (j < len) row = row_of_entry(kv, kv.table[(j < a.from ? 0 : b * kv.table_ld) + (j >> kv.page_shift)], j);
    uint4 kr[KC];
#pragma unroll
    for (int i = 0; i < KC; ++i) {
        const int e = (i * 32 + g * 16) / kElemBytes<KST>;
        kr[i] = make_uint4(0, 0, 0, 0);
        if (row >= 0 && e < D)
            kr[i] = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(kv.k) +
                                                    ((int64_t)row * kv.heads + h) * D * kElemBytes<KST> + i * 32 +
                                                    g * 16);
    }
    float sc = a.scale_log2;
    if (KST != kBf16) sc *= kv.per_head ? kv.k_scale[h] : row >= 0 ? kv.k_scale[(int64_t)row * kv.heads + h] : 0.0f;
    b8 kf[KM];
#pragma unroll
    for (int s = 0; s < KM; ++s) {
        uint4 w;
        if constexpr (KST == kBf16) {
            w = kr[s];
        } else {
            const uint4 t = kr[s >> 1];
            const uint32_t w0 = (s & 1) ? t.z : t.x, w1 = (s & 1) ? t.w : t.y;
            w = make_uint4(decode2<KST>(w0, false), decode2<KST>(w0, true), decode2<KST>(w1, false),
                           decode2<KST>(w1, true));
        }
        kf[s] = __builtin_bit_cast(b8, w);
    }
    // of the accumulator's token rows: the factor, and whether it is there
    float ks[16];
    uint32_t there = 0;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        const int t = (e >> 2) * 8 + g * 4 + (e & 3);
        ks[e] = __shfl(sc, t, 64);
        there |= (__shfl(row, t, 64) >= 0 ? 1u : 0u) << e;
    }
    float w[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) w[e] = 0.0f;
    put(0);
    __syncthreads();
    for (int i = 0, r0 = r_first; r0 < r_end; ++i, r0 += R) {
        if (r0 + R < r_end) load(r0 + R);
        // 32 rows at a time: the products of the next ones beside the
        // exponentials of the last
        f16v x[2];
        b8 qf[4];
        auto read_q = [&](int n) {              // operand n % KM of rows 32 (n / KM)..
            const int s = n % KM, e = KST == kBf16 ? s * 16 + g * 8 : (s >> 1) * 32 + g * 16 + (s & 1) * 8;
            qf[n & 3] = *reinterpret_cast<const b8*>(&s_q[i & 1][(n / KM * 32 + c) * kQ + e * 2]);
        };
        constexpr int H = R / 32;
        read_q(0);
        read_q(1);
        read_q(2);
        float z[2];
        int p[2];
#pragma unroll
        for (int half = 0; half <= H; ++half) {
            // exponentials of rows half - 1, products of rows half
            if (half < H) {
                z[half & 1] = s_lse[i & 1][half * 32 + c];
                p[half & 1] = s_pos[i & 1][half * 32 + c];
            }
            if (half > 0) {
                // what is not seen, and rows that give nothing (z infinite), weigh 0
                const int o = (half - 1) & 1;
                const int lo = a.window > 0 ? p[o] - a.window + 1 : 0;
#pragma unroll
                for (int e = 0; e < 16; ++e) x[o][e] = x[o][e] * ks[e] - z[o];
                if (!__all(j0 + 31 <= p[o] && (j0 >= lo || j0 + 31 < a.sinks))) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const int t = j0 + (e >> 2) * 8 + g * 4 + (e & 3);
                        const bool seen = (t <= p[o]) & ((t >= lo) | (t < a.sinks));
                        x[o][e] = seen ? x[o][e] : -INFINITY;
                    }
                }
            }
            if (half < H) x[half & 1] = f16v{0};
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int s = 0; s < KM; ++s) {
                const int n = half * KM + s;
                if (half < H) {
                    if (n + 3 < H * KM) read_q(n + 3);
                    x[half & 1] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf[s], qf[n & 3], x[half & 1], 0, 0, 0);
                }
                if (half > 0) {
#pragma unroll
                    for (int e = s * 16 / KM; e < (s + 1) * 16 / KM; ++e) {
                        w[e] += __builtin_amdgcn_exp2f(x[(half - 1) & 1][e]);
                        asm volatile("" : "+v"(w[e]));
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        if (r0 + R < r_end) put(i + 1);
        __syncthreads();
    }
    float* to = a.weights + ((int64_t)b * kv.heads + h) * a.ldw;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) w[e] += __shfl_xor(w[e], off, 64);
        const int t = j0 + (e >> 2) * 8 + g * 4 + (e & 3);
        if (c == 0 && t < len && (there >> e & 1)) to[t] += w[e];
    }
}

// Row tiles of a call, spare slots of a ragged one included.
int64_t tiles_of(const AttnArgs& a, bool ragged) {
    const int64_t group = a.q_heads / a.kv.heads, each = a.total_q / a.kv.batch;
    return ragged ? a.total_q * group / kRows + a.kv.batch : a.kv.batch * ((each * group + kRows - 1) / kRows);
}
int64_t weights_tiles(const AttnArgs& a) { return (a.kv.max_len + kRows - 1) / kRows; }

template <int KST, int VST, int DP>
hipError_t run_extend(const ExtendParams& p, unsigned tiles, hipStream_t stream) {
    static_assert(sizeof(Lds<DP>) <= 160 * 1024, "LDS");
    constexpr int bytes = sizeof(Lds<DP>);
    hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&k_extend<KST, VST, DP>),
                                       hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((k_extend<KST, VST, DP>), dim3(tiles * p.kv.heads * p.splits), dim3(kThreads), bytes, stream, p);
    e = hipGetLastError();
    if (e != hipSuccess || p.splits == 1) return e;
    hipLaunchKernelGGL(k_extend_join, dim3(tiles * p.kv.heads, kRows / kJoinRows), dim3(kThreads), 0, stream, p);
    return hipGetLastError();
}

template <int KST, int VST>
hipError_t extend_dim(const ExtendParams& p, unsigned tiles, hipStream_t stream) {
    if (p.kv.head_dim <= 64) return run_extend<KST, VST, 64>(p, tiles, stream);
    if (p.kv.head_dim <= 128) return run_extend<KST, VST, 128>(p, tiles, stream);
    return run_extend<KST, VST, 256>(p, tiles, stream);
}

template <int KST>
hipError_t extend_v(const ExtendParams& p, unsigned tiles, hipStream_t stream) {
    switch (p.kv.v_st) {
    case FP8_KV_E4M3: return extend_dim<KST, kE4M3>(p, tiles, stream);
    case FP8_KV_E5M2: return extend_dim<KST, kE5M2>(p, tiles, stream);
    default: return extend_dim<KST, kBf16>(p, tiles, stream);
    }
}

template <int KST, int DP>
hipError_t run_weights(const ExtendParams& p, dim3 grid, hipStream_t stream) {
    constexpr int bytes = sizeof(WeightsLds<DP>);
    static_assert(bytes <= 160 * 1024, "LDS");
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&k_weights<KST, DP>),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((k_weights<KST, DP>), grid, dim3(kThreads), bytes, stream, p);
    return hipGetLastError();
}

template <int KST>
hipError_t weights_dim(const ExtendParams& p, unsigned tiles, hipStream_t stream) {
    const dim3 grid(tiles * p.kv.heads, (unsigned)p.kv.batch);
    if (p.kv.head_dim <= 64) return run_weights<KST, 64>(p, grid, stream);
    if (p.kv.head_dim <= 128) return run_weights<KST, 128>(p, grid, stream);
    return run_weights<KST, 256>(p, grid, stream);
}

ExtendParams params_of(const AttnArgs& a) {
    ExtendParams p;
    p.kv = a.kv; p.q = a.q; p.ldq = a.ldq; p.total_q = (int)a.total_q; p.each = (int)(a.total_q / a.kv.batch);
    p.q_heads = a.q_heads; p.group = a.q_heads / a.kv.heads; p.q_offsets = a.q_offsets; p.scale_log2 = a.scale * kLog2e;
    p.window = a.window; p.sinks = a.sinks; p.from = a.from; p.out = a.out; p.ldo = a.ldo; p.lse = a.lse;
    p.weights = a.weights; p.ldw = a.ldw;
    p.splits = 1; p.least = 1; p.part_ml = nullptr; p.part_o = nullptr;
    return p;
}

// Blocks that share a row tile's steps.  As many as make up one resident round
// of 512, of 2 steps or more (one sequence, 32 queries, 8 KV heads: over 1024
// tokens 17 us against 26 with pieces of 8 steps); in a ragged batch two rounds
// where pieces keep 8 steps, since its tiles differ in length (12 sequences, up
// to 77 queries and 3001 tokens: 66 us, one round 73, unsplit 103; of equal
// lengths, 2 x 64 queries over 60000 tokens: 219 us, one round 190).  The join
// reads all pieces one after the other, which bounds their number (one
// sequence, 32 queries: over 4096 tokens 24 pieces 23 us and 32 29, over 100000
// 24 pieces 142 and 32 119).  Where max_len is no more than 8 steps every tile
// stays whole: the join costs what it saves.  (A short tile of a batch whose
// max_len is larger is cut all the same, into pieces of 2 to 4 steps.)
int splits_of(const AttnArgs& a, bool ragged, int* least) {
    const int64_t group = a.q_heads / a.kv.heads, blocks = tiles_of(a, ragged) * a.kv.heads;
    int64_t steps = (a.kv.max_len + kStep - 1) / kStep;
    if (a.window > 0) {
        // a tile's tokens, their window and the sinks
        const int64_t span = kRows / group + 1 + a.window;
        const int64_t seen = (span + kStep - 1) / kStep + 1 + (a.sinks + kStep - 1) / kStep;
        steps = seen < steps ? seen : steps;
    }
    *least = 4;
    if (steps <= 8 || blocks < 1) return 1;
    const int64_t one = std::min(512 / blocks, steps / 2), two = ragged ? std::min(1024 / blocks, steps / 8) : 0;
    const int64_t s = std::clamp<int64_t>(std::max(one, two), 1, steps <= 128 ? 24 : 32);
    // shorter tiles of a ragged batch take fewer blocks, not shorter pieces
    // (16 sequences up to 60 queries and 1500 tokens: 47 us, from 2 steps on 52)
    *least = (int)std::clamp<int64_t>(steps / s, 2, 4);
    return (int)s;
}

}  // namespace

int64_t extend_workspace(const AttnArgs& a, bool ragged) {
    int least;
    const int64_t s = splits_of(a, ragged, &least), rows = a.total_q * a.q_heads;
    return s == 1 ? 0 : (rows * s * 8 + 15) / 16 * 16 + rows * s * a.kv.head_dim * 4;
}

int64_t extend_blocks(const AttnArgs& a, bool ragged) {
    int least;
    const int64_t tiles = tiles_of(a, ragged) * splits_of(a, ragged, &least);
    return std::max(tiles, a.weighted ? weights_tiles(a) : 0) * a.kv.heads;
}

hipError_t launch_extend(const AttnArgs& a) {
    ExtendParams p = params_of(a);
    p.splits = splits_of(a, a.q_offsets != nullptr, &p.least);
    const unsigned tiles = (unsigned)tiles_of(a, a.q_offsets != nullptr);
    const int64_t rows = a.total_q * a.q_heads;
    p.part_ml = reinterpret_cast<float2*>(a.workspace);
    p.part_o = reinterpret_cast<float*>(a.workspace + (rows * p.splits * 8 + 15) / 16 * 16);
    hipError_t e;
    switch (a.kv.k_st) {
    case FP8_KV_E4M3: e = extend_v<kE4M3>(p, tiles, a.stream); break;
    case FP8_KV_E5M2: e = extend_v<kE5M2>(p, tiles, a.stream); break;
    default: e = extend_v<kBf16>(p, tiles, a.stream); break;
    }
    return e != hipSuccess || !a.weighted ? e : launch_attention_weights(a);
}

hipError_t launch_attention_weights(const AttnArgs& a) {
    if (a.kv.max_len == 0) return hipSuccess;
    const ExtendParams p = params_of(a);
    const unsigned tiles = (unsigned)weights_tiles(a);
    switch (a.kv.k_st) {
    case FP8_KV_E4M3: return weights_dim<kE4M3>(p, tiles, a.stream);
    case FP8_KV_E5M2: return weights_dim<kE5M2>(p, tiles, a.stream);
    default: return weights_dim<kBf16>(p, tiles, a.stream);
    }
}

}  // namespace fp8mi
