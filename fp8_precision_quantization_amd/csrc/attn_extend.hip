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

#include "attention.hpp"

namespace fp8mi {
namespace {

using namespace attn;

constexpr int kStep = 64;        // cached tokens of one step
constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kRows = 32 * kWaves;
constexpr int kMarks = 1024;

struct ExtendParams {
    KvView kv;
    const uint16_t* q;
    int64_t ldq;
    int total_q, each;           // each: queries of every sequence without q_offsets
    int q_heads, group;
    const int32_t* q_offsets;
    float scale_log2;
    int window, sinks;
    uint16_t* out;
    int64_t ldo;
    float* lse;
    float* weights;
    int64_t ldw;
    int splits, least;           // blocks that may share a row tile's steps, the fewest of one
    float2* part_ml;             // [total_q * q_heads, splits]
    float* part_o;               // [total_q * q_heads, splits, head_dim]
};

// Queries of sequence b: the first and their number, inside [0, total_q].
__device__ __forceinline__ void queries_of(const ExtendParams& a, int b, int* first, int* n) {
    if (a.q_offsets == nullptr) {
        *first = b * a.each;
        *n = a.each;
    } else {
        const int lo = min(max(a.q_offsets[b], 0), a.total_q), hi = min(max(a.q_offsets[b + 1], lo), a.total_q);
        *first = lo;
        *n = hi - lo;
    }
}

// V's scale of a KV head where it has one for all tokens, else 1.
__device__ __forceinline__ float v_scale_of(const KvView& kv, int h) {
    return kv.per_head && kv.v_scale ? kv.v_scale[h] : 1.0f;
}

// With q_offsets: slot of the first row tile of sequence b.  A sequence's
// tiles start at floor(first row / kRows) + b: increasing in b, and no two
// sequences share a slot, without a prefix sum over the sequences.
__device__ __forceinline__ int first_slot(const ExtendParams& a, int b) {
    return min(max(a.q_offsets[b], 0), a.total_q) * a.group / kRows + b;
}

// The row tile of a slot: its sequence, rows [row0, row0 + kRows) of that
// sequence's rows, the positions of its first and last token.
struct Tile {
    int b = 0, q_first, rows, row0, base, p_first, p_last;
    __device__ __forceinline__ Tile(const ExtendParams& a, int slot) {
        int n, len;
        if (a.q_offsets == nullptr) {
            // tile by tile over the sequences: taken from the last slot on, the
            // longest tiles of all of them come first
            b = slot % a.kv.batch;
            row0 = slot / a.kv.batch * kRows;
            queries_of(a, b, &q_first, &n);
            len = seq_len(a.kv, b);
        } else {
            // first_slot increases: halve down to 64 sequences, then one look,
            // at everything of them that is needed
            int hi = a.kv.batch;
            while (hi - b > 64) {
                const int mid = (b + hi) >> 1;
                if (first_slot(a, mid) <= slot) b = mid; else hi = mid;
            }
            const int mine = min(b + (int)(threadIdx.x & 63), hi - 1);
            int first, count;
            queries_of(a, mine, &first, &count);
            const int tokens = seq_len(a.kv, mine), start = first * a.group / kRows + mine;
            const uint64_t at = __ballot(start <= slot);
            const int l = min(at ? 63 - __builtin_clzll(at) : 0, hi - 1 - b);
            q_first = __builtin_amdgcn_readlane(first, l);
            n = __builtin_amdgcn_readlane(count, l);
            len = __builtin_amdgcn_readlane(tokens, l);
            row0 = (slot - __builtin_amdgcn_readlane(start, l)) * kRows;
            b += l;
        }
        rows = n * a.group;
        base = len - n;
        p_first = base + row0 / a.group;
        p_last = base + (min(row0 + kRows, rows) - 1) / a.group;
    }
    __device__ __forceinline__ bool any() const { return row0 >= 0 && row0 < rows; }
};

// Steps of one block of a row tile: an even part, and no fewer than a.least.
__device__ __forceinline__ int chunk_of(const ExtendParams& a, int steps) {
    const int even = (steps + a.splits - 1) / a.splits;
    return even < a.least ? a.least : even;
}

template <int DP>
struct Lds {
    static constexpr int kK = DP * 2 + 16, kV = DP * 2 + 64;     // bytes of a padded row
    struct Buf {
        alignas(16) uint8_t k[kStep * kK];
        alignas(16) uint8_t v[kStep * kV];
        alignas(16) float ks[kStep];
        alignas(16) float vs[kStep];
    };
    Buf buf[2];
    alignas(16) int row[4][kStep];
    uint32_t bad[kMarks / 32];      // step i marks bit i % kMarks
};

// One value of the cache as fp32.
template <int ST>
__device__ __forceinline__ float value_at(const uint8_t* p, int d) {
    if constexpr (ST == kBf16) return as_f32((uint32_t)reinterpret_cast<const uint16_t*>(p)[d] << 16);
    else return as_f32(decode2<ST>(p[d], false) << 16);
}

// 16 values of a cache row: 16 bytes of codes or 32 of bf16
template <int ST>
struct Unit {
    uint4 w[kElemBytes<ST>];
    __device__ __forceinline__ void load(const uint8_t* p) {
#pragma unroll
        for (int i = 0; i < kElemBytes<ST>; ++i) w[i] = reinterpret_cast<const uint4*>(p)[i];
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < kElemBytes<ST>; ++i) w[i] = make_uint4(0, 0, 0, 0);
    }
    // 1 if anything is not finite; clears these values
    __device__ __forceinline__ bool clean() {
        uint32_t any = 0;
#pragma unroll
        for (int i = 0; i < kElemBytes<ST>; ++i)
            any |= not_finite<ST>(w[i].x) | not_finite<ST>(w[i].y) | not_finite<ST>(w[i].z) | not_finite<ST>(w[i].w);
        if (any) {
#pragma unroll
            for (int i = 0; i < kElemBytes<ST>; ++i) {
                w[i].x = cleared<ST>(w[i].x, not_finite<ST>(w[i].x));
                w[i].y = cleared<ST>(w[i].y, not_finite<ST>(w[i].y));
                w[i].z = cleared<ST>(w[i].z, not_finite<ST>(w[i].z));
                w[i].w = cleared<ST>(w[i].w, not_finite<ST>(w[i].w));
            }
        }
        return any != 0;
    }
    // as bf16 into LDS: two pieces of 16 bytes, `apart` bytes from each other
    __device__ __forceinline__ void put(uint8_t* to, int apart) const {
        uint4 a, b;
        if constexpr (ST == kBf16) {
            a = w[0];
            b = w[1];
        } else {
            a = make_uint4(decode2<ST>(w[0].x, false), decode2<ST>(w[0].x, true), decode2<ST>(w[0].y, false),
                           decode2<ST>(w[0].y, true));
            b = make_uint4(decode2<ST>(w[0].z, false), decode2<ST>(w[0].z, true), decode2<ST>(w[0].w, false),
                           decode2<ST>(w[0].w, true));
        }
        *reinterpret_cast<uint4*>(to) = a;
        *reinterpret_cast<uint4*>(to + apart) = b;
    }
};

// First channel of piece p (8 channels) of an LDS row: the even pieces of the
// row come first, then the odd ones, so that the lanes that stage a row write
// 16 bytes next to each other.  Q and the output follow the same order.
template <int DP>
__device__ __forceinline__ constexpr int channel_of(int p) {
    return p < DP / 16 ? p * 16 : (p - DP / 16) * 16 + 8;
}

typedef short s4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ s4 read_tr(const uint8_t* p) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s4*)(uintptr_t)p);
}

template <int KST, int VST, int DP>
__global__ __launch_bounds__(kThreads, DP <= 128 ? 2 : 1) void k_extend(const ExtendParams a) {
    constexpr int KM = DP / 16;                     // matrix steps over the channels of K
    constexpr int DT = DP / 32;                     // 32-channel tiles of the output
    constexpr int UR = DP / 16;                     // units of a row
    constexpr int UT = kStep * UR / kThreads;       // units a thread stages
    using L = Lds<DP>;
    extern __shared__ __align__(16) uint8_t smem[];
    L& lds = *reinterpret_cast<L*>(smem);

    const KvView& kv = a.kv;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int c = lane & 31, g = lane >> 5;
    const int h = blockIdx.x % kv.heads, split = blockIdx.x / kv.heads % a.splits;
    // later (longer) tiles first
    const Tile tile(a, (int)(gridDim.x / kv.heads / a.splits - 1 - blockIdx.x / kv.heads / a.splits));
    if (!tile.any()) return;
    const int b = tile.b, q_first = tile.q_first, rows = tile.rows, row0 = tile.row0, base = tile.base;
    const int p_first = tile.p_first, p_last = tile.p_last;
    const int G = a.group, D = kv.head_dim;
    const Steps<kStep> steps(p_first, p_last, a.window, a.sinks);
    const int chunk = chunk_of(a, steps.count), s_begin = split * chunk, s_end = min(s_begin + chunk, steps.count);
    if (s_begin >= steps.count && split > 0) return;

    // this lane's row
    const int r = row0 + wave * 32 + c;
    const bool live = r < rows;
    const int tok = r / G, hq = h * G + (r - tok * G);
    const int pos = live ? base + tok : -1;
    b8 qf[KM];
    {
        const uint16_t* qr = a.q + (int64_t)(q_first + tok) * a.ldq + (int64_t)hq * D;
#pragma unroll
        for (int s = 0; s < KM; ++s) {
            uint4 t = make_uint4(0, 0, 0, 0);
            const int e = channel_of<DP>(2 * s) + g * (channel_of<DP>(2 * s + 1) - channel_of<DP>(2 * s));
            if (live && e < D) t = *reinterpret_cast<const uint4*>(qr + e);
            qf[s] = __builtin_bit_cast(b8, t);
        }
    }
    f16v o[DT];
#pragma unroll
    for (int i = 0; i < DT; ++i) o[i] = f16v{0};
    float m = 0.0f, l = 0.0f, limit = kLowest;      // limit: where the row's reference moves

    const int64_t k_row = (int64_t)kv.heads * D * kElemBytes<KST>, v_row = (int64_t)kv.heads * D * kElemBytes<VST>;
    const uint8_t* kb = static_cast<const uint8_t*>(kv.k) + (int64_t)h * D * kElemBytes<KST>;
    const uint8_t* vb = static_cast<const uint8_t*>(kv.v) + (int64_t)h * D * kElemBytes<VST>;
    const int32_t* table = kv.table + b * kv.table_ld;
    const bool k_tok = KST != kBf16 && !kv.per_head, v_tok = VST != kBf16 && !kv.per_head;
    float scale_log2 = a.scale_log2;
    asm volatile("" : "+s"(scale_log2));      // a register: selects below must not pick an argument's address
    const float k_head = (KST == kBf16 || k_tok ? 1.0f : kv.k_scale[h]) * scale_log2;

    // Staging.  No load is conditional, so that a wait for one counts the later
    // ones: tokens that are not there (their score is masked, their weight 0)
    // read row 0, steps past the end the last token.
    Unit<KST> ku[UT];
    Unit<VST> vu[UT];
    float sc = 0.0f;
    // the scale a thread stages: K's of token tid, or V's of token tid - kStep
    const bool key = (tid & kStep) == 0, per_token = key ? k_tok : v_tok;
    const float* const k_scales = k_tok ? kv.k_scale : reinterpret_cast<const float*>(table);
    const float* const v_scales = v_tok ? kv.v_scale : reinterpret_cast<const float*>(table);
    const float* const scales = key ? k_scales : v_scales;
    const float scale_of_head = key ? k_head : 1.0f, scale_by = key ? scale_log2 : 1.0f;
    auto entry_of = [&](int i) -> int {         // the page of token tid % kStep of a step
        const int j = steps.token(min(i, s_end - 1)) + (tid & (kStep - 1));
        return table[min(j, p_last) >> kv.page_shift];
    };
    auto put_row = [&](int i, int entry) {
        const int j = steps.token(i) + tid;
        if (tid < kStep) lds.row[i & 3][tid] = i < s_end && j <= p_last ? row_of_entry(kv, entry, j) : -1;
    };
    auto load = [&](int i) {                    // a step's K, V and scales into registers
        const int* rows_i = lds.row[i & 3];
        const int64_t srow = max(rows_i[tid & (kStep - 1)], 0);
        sc = scales[per_token ? srow * kv.heads + h : 0];
#pragma unroll
        for (int u = 0; u < UT; ++u) {
            const int t = (tid + u * kThreads) / UR, e = ((tid + u * kThreads) % UR) * 16;
            const int64_t row = max(rows_i[t], 0);
            const int d = D == DP || e < D ? e : 0;
            ku[u].load(kb + row * k_row + d * kElemBytes<KST>);
            vu[u].load(vb + row * v_row + d * kElemBytes<VST>);
        }
    };
    auto mark = [&](int i) { atomicOr(&lds.bad[i % kMarks / 32], 1u << (i % 32)); };
    // K or V of one unit into a step's LDS buffer, the scales with the first
    auto put = [&](int i, int part) {
        typename L::Buf& buf = lds.buf[i & 1];
        const int u = part >> 1, t = (tid + u * kThreads) / UR, e = (tid + u * kThreads) % UR;
        if (part & 1) {
            if (D < DP && e * 16 >= D) vu[u].clear();
            if (vu[u].clean() && lds.row[i & 3][t] >= 0) mark(i);
            vu[u].put(buf.v + t * L::kV + e * 16, UR * 16);
        } else {
            if (D < DP && e * 16 >= D) ku[u].clear();
            ku[u].put(buf.k + t * L::kK + e * 16, UR * 16);
        }
        if (part == 0 && tid < 2 * kStep) {
            const bool there = lds.row[i & 3][tid & (kStep - 1)] >= 0;
            float s = per_token ? sc * scale_by : scale_of_head;
            if (per_token && (!there || (!key && !__builtin_isfinite(s)))) {
                if (there) mark(i);
                s = 0.0f;
            }
            (key ? buf.ks : buf.vs)[tid & (kStep - 1)] = s;
        }
    };

    // Rows are known three steps ahead, K and V are in registers one step ahead
    // and in LDS the step before they are needed.
    int entry = 0;
    if (s_begin < s_end) {
        if (tid < kMarks / 32) lds.bad[tid] = 0;
        const int e0 = entry_of(s_begin), e1 = entry_of(s_begin + 1), e2 = entry_of(s_begin + 2);
        entry = entry_of(s_begin + 3);
        put_row(s_begin, e0);
        put_row(s_begin + 1, e1);
        put_row(s_begin + 2, e2);
        __syncthreads();
        load(s_begin);
#pragma unroll
        for (int n = 0; n < 2 * UT; ++n) put(s_begin, n);
        load(s_begin + 1);
        // Q has arrived before the loop, which then waits for no load of its own step
#pragma unroll
        for (int s = 0; s < KM; ++s) asm volatile("" : "+v"(qf[s]));
        __syncthreads();
    }
    for (int i = s_begin; i < s_end; ++i) {
        const typename L::Buf& buf = lds.buf[i & 1];
        const int* rows_i = lds.row[i & 3];
        const int j0 = steps.token(i);
        const bool there = rows_i[lane] >= 0;

        // The step in halves of 32 tokens, so that matrix products of one run
        // beside the exponentials of the other:
        //   S0 = K0 Q | S1 = K1 Q with P0 = 2^S0 | O += V0 P0 with P1 = 2^S1 |
        //   O += V1 P1 with the next step's K and V into LDS
        // LDS reads run a few products ahead; the scheduling barriers keep
        // this order.
        b8 kf[4];
        auto read_k = [&](int n) {
            kf[n & 3] = *reinterpret_cast<const b8*>(buf.k + (n / KM * 32 + c) * L::kK + n % KM * 32 + g * 16);
        };
        read_k(0);
        read_k(1);
        read_k(2);

        const bool edge = j0 + kStep - 1 > p_first ||
                          (a.window > 0 && j0 <= p_last - a.window && j0 + kStep - 1 >= a.sinks);
        const bool masked = edge || !__all(there);
        f16v x[2];
        uint32_t pw[16];            // the weights as bf16 pairs, 4 words a B operand
        float part[2] = {0, 0};
        f4 vs[4];
        // scores of half t against the row's reference m (0 until the row has
        // seen a token), masked; the reference moves if one passes the limit
        auto scores = [&](int t) {
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                f4 ks = f4{scale_log2, scale_log2, scale_log2, scale_log2};
                if (KST != kBf16) ks = *reinterpret_cast<const f4*>(&buf.ks[t * 32 + u * 8 + g * 4]);
                vs[u] = f4{1, 1, 1, 1};
                if (VST != kBf16) vs[u] = *reinterpret_cast<const f4*>(&buf.vs[t * 32 + u * 8 + g * 4]);
#pragma unroll
                for (int e = 0; e < 4; ++e) x[t][u * 4 + e] = __builtin_fmaf(x[t][u * 4 + e], ks[e], -m);
            }
            if (masked) {
                const int lo = a.window > 0 ? pos - a.window + 1 : 0;
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int at = t * 32 + u * 8 + g * 4;
                    const int4 rr = *reinterpret_cast<const int4*>(&rows_i[at]);
                    const int ra[4] = {rr.x, rr.y, rr.z, rr.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int j = j0 + at + e;
                        const bool seen = (ra[e] >= 0) & (j <= pos) & ((j >= lo) | (j < a.sinks));
                        x[t][u * 4 + e] = seen ? x[t][u * 4 + e] : -INFINITY;
                    }
                }
            }
            float mx = -INFINITY;
#pragma unroll
            for (int e = 0; e < 16; ++e) mx = fmaxf(mx, x[t][e]);
            if (__any(mx > limit)) {
                // The first reference is the largest score itself, so that
                // the weight of a row's only token is 1 and rounds to itself;
                // from then on m moves by whole powers of two, so everything
                // that depends on it, the first half's bf16 weights included,
                // scales exactly.
                mx = max_xor32(mx);
                const float to = limit == kLowest ? mx : __builtin_ceilf(mx), up = mx > limit ? to : 0.0f;
                const float f = limit == kLowest ? 1.0f : __builtin_amdgcn_exp2f(-up);  // before the first: o, l are 0
                limit = mx > limit ? kSlack : limit;
                m += up;
                l *= f;
#pragma unroll
                for (int e = 0; e < 16; ++e) x[t][e] -= up;
                if (t == 1) {
                    part[0] *= f;
                    part[1] *= f;
#pragma unroll
                    for (int e = 0; e < 8; ++e) pw[e] = pack2(as_f32(pw[e] << 16) * f, as_f32(pw[e] & 0xFFFF0000u) * f);
                }
#pragma unroll
                for (int d = 0; d < DT; ++d)
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[d][e] = o[d][e] * f;
            }
        };
        // part n of `parts` of half t's weights; the bf16 pairs as they fill
        auto weights = [&](int t, int n, int parts) {
#pragma unroll
            for (int e = n * 16 / parts; e < (n + 1) * 16 / parts; ++e) {
                const float w = __builtin_amdgcn_exp2f(x[t][e]);
                part[e & 1] += w;
                x[t][e] = VST == kBf16 ? w : w * vs[e >> 2][e & 3];
                if (e & 1) {
                    uint32_t& q = pw[t * 8 + (e >> 1)];
                    q = pack2(x[t][e - 1], x[t][e]);
                    // here, beside the products, and not where they are used
                    asm volatile("" : "+v"(q), "+v"(part[0]), "+v"(part[1]));
                }
            }
        };
        x[0] = f16v{0};
        x[1] = f16v{0};
#pragma unroll
        for (int n = 0; n < KM; ++n) {
            read_k(n + 3);
            x[0] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf[n & 3], qf[n], x[0], 0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);
        }
        scores(0);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int n = KM; n < 2 * KM; ++n) {
            if (n + 3 < 2 * KM) read_k(n + 3);
            x[1] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf[n & 3], qf[n - KM], x[1], 0, 0, 0);
            weights(0, n - KM, KM);
            __builtin_amdgcn_sched_barrier(0);
        }
        // V^T of product n: tokens of group n / DT, channels of tile n % DT.
        // Lane i of 16 points at row i / 4, channels 4 (i % 4).. of a 4 x 16
        // block and receives its column i.
        b8 vf[4];
        const uint8_t* vp =
            buf.v + (g * 4 + ((lane & 15) >> 2)) * L::kV + (((lane >> 4) & 1) * 16 + (lane & 3) * 4) * 2;
        auto read_v = [&](int n) {
            const uint8_t* p = vp + n / DT * 16 * L::kV + n % DT * 64;
            const s4 lo = read_tr(p), hi = read_tr(p + 8 * L::kV);
            vf[n & 3] = __builtin_bit_cast(b8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        };
        read_v(0);
        read_v(1);
        read_v(2);
        scores(1);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int n = 0; n < 4 * DT; ++n) {
            if (n + 3 < 4 * DT) read_v(n + 3);
            const u4 pf = u4{pw[n / DT * 4], pw[n / DT * 4 + 1], pw[n / DT * 4 + 2], pw[n / DT * 4 + 3]};
            o[n % DT] =
                __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf[n & 3], __builtin_bit_cast(b8, pf), o[n % DT], 0, 0, 0);
            if (n < 2 * DT) weights(1, n, 2 * DT);
            else if ((n - 2 * DT) % (DT / UT) == 0) put(i + 1, (n - 2 * DT) / (DT / UT));
            __builtin_amdgcn_sched_barrier(0);
        }
        put_row(i + 3, entry);
        entry = entry_of(i + 4);
        load(i + 2);
        l += part[0] + part[1];
        asm volatile("" : "+v"(l));
        __syncthreads();
    }

    l = sum_xor32(l);
    uint32_t met = 0;
    if (s_begin < s_end && lane < kMarks / 32) met = lds.bad[lane];
    if (__any(met != 0)) {
        for (int i = s_begin; i < s_end; ++i) {
            if (!(lds.bad[i % kMarks / 32] >> (i % 32) & 1)) continue;
            for (int j = steps.token(i); j < steps.token(i) + kStep && j <= p_last; ++j) {
                const int row = row_of_entry(kv, table[j >> kv.page_shift], j);
                if (row < 0) continue;
                const uint8_t* vr = vb + row * v_row;
                const float s = v_tok ? kv.v_scale[(int64_t)row * kv.heads + h] : 1.0f;
                bool odd = !__builtin_isfinite(s);
                for (int d = lane; d < D; d += 64) odd = odd || !__builtin_isfinite(value_at<VST>(vr, d));
                if (!__any(odd)) continue;
                // the token's score for this lane's row
                const uint8_t* kr = kb + row * k_row;
                const uint16_t* qr = a.q + (int64_t)(q_first + tok) * a.ldq + (int64_t)hq * D;
                float x = 0.0f;
                if (live)
                    for (int d = 0; d < D; ++d) x += value_at<KST>(kr, d) * as_f32((uint32_t)qr[d] << 16);
                x *= k_head * (k_tok ? kv.k_scale[(int64_t)row * kv.heads + h] : 1.0f);
                const float w = __builtin_amdgcn_exp2f(x - m);
                if (!sees(j, pos, a.window, a.sinks)) continue;
#pragma unroll
                for (int d = 0; d < DT; ++d)
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const int ch = channel_of<DP>(d * 4 + (e >> 2)) + g * 4 + (e & 3);
                        if (ch < D) {
                            const float v = value_at<VST>(vr, ch);
                            if (!__builtin_isfinite(v) || !__builtin_isfinite(s)) o[d][e] += w * (v * s);
                        }
                    }
            }
        }
    }
    if (!live) return;
    const int64_t row = (int64_t)(q_first + tok) * a.q_heads + hq;
    if (chunk < steps.count) {                  // one of several blocks of this tile
        if (g == 0) a.part_ml[row * a.splits + split] = make_float2(limit == kLowest ? kLowest : m, l);
        float* to = a.part_o + (row * a.splits + split) * D;
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int ch = channel_of<DP>(d * 4 + u) + g * 4;
                if (ch < D)
                    *reinterpret_cast<f4*>(to + ch) =
                        f4{o[d][u * 4], o[d][u * 4 + 1], o[d][u * 4 + 2], o[d][u * 4 + 3]};
            }
        return;
    }
    const float inv = l == 0.0f ? 0.0f : v_scale_of(kv, h) / l;
    uint16_t* to = a.out + (int64_t)(q_first + tok) * a.ldo + (int64_t)hq * D;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int ch = channel_of<DP>(d * 4 + u) + g * 4;
            if (ch < D)
                *reinterpret_cast<uint2*>(to + ch) =
                    make_uint2(pack2(o[d][u * 4] * inv, o[d][u * 4 + 1] * inv),
                               pack2(o[d][u * 4 + 2] * inv, o[d][u * 4 + 3] * inv));
        }
    if (g == 0 && a.lse) a.lse[row] = l == 0.0f ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * kLn2;
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
    if (j < len) row = row_of_entry(kv, kv.table[b * kv.table_ld + (j >> kv.page_shift)], j);
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
    p.window = a.window; p.sinks = a.sinks; p.out = a.out; p.ldo = a.ldo; p.lse = a.lse;
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
