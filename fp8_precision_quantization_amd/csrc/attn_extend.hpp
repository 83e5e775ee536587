// attn_extend.hpp -- a block of query rows over the paged KV cache in steps of
// 64 tokens: the work of attn_extend.hip's kernel, which also takes the shared
// prefix of attn_shared.hip.  Mathematics, layout and measurements stand in
// attn_extend.hip.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>

#include "attention.hpp"

namespace fp8mi {
namespace {

using namespace attn;

namespace extend {

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
    int from;                    // k_weights: the first tokens, read from the first row's pages by every sequence
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

// The rows of a block and the tokens it walks.  Of this lane's row: whether
// there is one, its query token, its query head and its position.
struct Rows {
    bool live;
    int token, head, pos;
    int p_first, p_last;            // of the block: lowest position (-1: to be found), last token that any row sees
    const int32_t* table;
    int s_begin, s_end;             // this block's steps
    bool partial;                   // one of several blocks of these rows: the results are joined
    int part;                       // which
};

// One block's rows of one KV head over its steps of the cached tokens.
template <int KST, int VST, int DP, bool kFind>
__device__ __forceinline__ void extend_rows(const ExtendParams& a, Lds<DP>& lds, int h, const Steps<kStep>& steps,
                                            const Rows& at) {
    constexpr int KM = DP / 16;                     // matrix steps over the channels of K
    constexpr int DT = DP / 32;                     // 32-channel tiles of the output
    constexpr int UR = DP / 16;                     // units of a row
    constexpr int UT = kStep * UR / kThreads;       // units a thread stages
    using L = Lds<DP>;

    const KvView& kv = a.kv;
    const int tid = threadIdx.x, lane = tid & 63;
    const int g = lane >> 5, c = lane & 31;
    int p_first = at.p_first;
    const int p_last = at.p_last, s_begin = at.s_begin, s_end = at.s_end;
    const int D = kv.head_dim, hq = at.head, pos = at.pos;
    const bool live = at.live;
    const int32_t* const table = at.table;
    b8 qf[KM];
    {
        const uint16_t* qr = a.q + (int64_t)at.token * a.ldq + (int64_t)hq * D;
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
    if (kFind && p_first < 0) {         // of the wave's rows, whose positions have been on their way until here
        p_first = live ? min(pos, p_last) : p_last;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) p_first = min(p_first, __shfl_xor(p_first, off, 64));
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
                const uint16_t* qr = a.q + (int64_t)at.token * a.ldq + (int64_t)hq * D;
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
    const int64_t row = (int64_t)at.token * a.q_heads + hq;
    if (at.partial) {
        if (g == 0) a.part_ml[row * a.splits + at.part] = make_float2(limit == kLowest ? kLowest : m, l);
        float* to = a.part_o + (row * a.splits + at.part) * D;
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
    uint16_t* to = a.out + (int64_t)at.token * a.ldo + (int64_t)hq * D;
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

}  // namespace extend
}  // namespace
}  // namespace fp8mi
