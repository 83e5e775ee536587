// attn_decode.hpp -- one new token per sequence over the paged KV cache, a
// wave's share of the batch's steps: the work of attn_decode.hip's kernel, which
// also takes the sequences' own tokens behind the shared prefix of
// attn_shared.hip.  Mathematics, layout and measurements stand in
// attn_decode.hip.
#pragma once

#include <hip/hip_runtime.h>

#include "attention.hpp"

namespace fp8mi {
namespace {

using namespace attn;

namespace decode {

constexpr int kStep = 32;       // tokens of one wave step
constexpr int kWaves = 4;

struct DecodeParams {
    KvView kv;
    const uint16_t* q;
    int64_t ldq;
    int q_heads, group, col_tiles;
    float scale_log2;
    int window, sinks;
    int from;                    // kTail: the first token, a multiple of 64; kPrefix: the prefix's length
    int columns, pieces;         // kPrefix: query heads of a KV head over the whole batch, pieces of a row
    int shares, least;           // waves that share the batch's steps, per KV head and column tile
    uint16_t* out;
    int64_t ldo;
    float* lse;
    float2* part_ml;             // [shares + batch, q_heads]
    float* part_o;               // [shares + batch, q_heads, head_dim]
    float* scores;               // null, or [batch, q_heads, span]: x_j of every token of every step
    int64_t span;
    float* weights;
    int64_t ldw;
    int join_waves;              // waves of the join that share a query head: 1 or kJoinWaves
};

// How a batch's steps are shared out.  The sequences' steps lie one after the
// other (a sequence without any counts as one, for its zeros); share i takes
// `chunk` of them from i * chunk, across sequence borders, so workers have
// equal work whatever the lengths.  The piece of sequence b in share i has
// slot i + b of the partial results: each next piece starts a new share or a
// new sequence, so slots are distinct.
struct Work {
    int total = 0, chunk = 0;
    int b = 0, len = 0, before = 0;      // a sequence, its tokens and the steps before it
};

// What a launch's waves read: every sequence (kWhole), of every sequence the
// tokens from a.from on (kTail), or the first a.from tokens of the first row's
// pages for the queries of all sequences at once (kPrefix).
enum Part { kWhole, kTail, kPrefix };

// The steps of a sequence's newest token.
template <Part kPart>
__device__ __forceinline__ Steps<kStep> steps_at(const DecodeParams& a, int pos) {
    constexpr bool all = kPart == kWhole;
    return Steps<kStep>(pos, pos, all ? a.window : 0, all ? a.sinks : 0, kPart == kTail ? a.from : 0);
}

template <Part kPart>
__device__ __forceinline__ int steps_of(const DecodeParams& a, int len) {
    const int n = steps_at<kPart>(a, len - 1).count;
    return n < 1 ? 1 : n;
}

__device__ __forceinline__ int wave_scan(int v, int lane) {
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const int t = __shfl_up(v, off, 64);
        if (lane >= off) v += t;
    }
    return v;
}

// The total and the chunk, then the sequence that step `at` of the whole (or,
// with seq >= 0, the sequence `seq`) lies in.  Every wave computes it for
// itself, 64 sequences at a time.
template <Part kPart>
__device__ __forceinline__ Work work_of(const DecodeParams& a, int share, int seq, int lane) {
    Work w;
    const int B = a.kv.batch;
    int sum = 0, mine = 0, len = 0;      // of the last 64 sequences looked at
    auto look = [&](int b0) {
        len = b0 + lane < B ? seq_len(a.kv, b0 + lane) : 0;
        mine = b0 + lane < B ? steps_of<kPart>(a, len) : 0;
        sum = wave_scan(mine, lane);
    };
    for (int b0 = 0; b0 < B; b0 += 64) {
        look(b0);
        w.total += __builtin_amdgcn_readlane(sum, 63);
    }
    const int even = (w.total + a.shares - 1) / a.shares, mean = (w.total + B - 1) / B;
    const int least = mean < a.least ? mean : a.least;     // a share's fewest steps, unless sequences are shorter
    w.chunk = even < least ? least : even;
    const int at = share * w.chunk;
    for (int b0 = 0; b0 < B; b0 += 64) {
        if (B > 64) look(b0);
        const uint64_t in = seq >= 0 ? (seq < b0 + 64 ? 1ull << (seq & 63) : 0)
                                     : __ballot(w.before + sum > at && mine > 0);
        if (in) {
            const int l = __builtin_ctzll(in);
            w.b = b0 + l;
            w.len = __builtin_amdgcn_readlane(len, l);
            w.before += __builtin_amdgcn_readlane(sum, l) - __builtin_amdgcn_readlane(mine, l);
            return w;
        }
        w.before += __builtin_amdgcn_readlane(sum, 63);
    }
    return w;
}

template <int N>
__device__ __forceinline__ int min_of(const int (&v)[N]) {
    int r = v[0];
#pragma unroll
    for (int i = 1; i < N; ++i) r = min(r, v[i]);
    return r;
}

// VD values of one token (one lane's channels) as raw words
template <int W>
struct Raw {
    uint32_t w[W];
};

template <int W>
__device__ __forceinline__ Raw<W> load_raw(const uint8_t* p) {
    Raw<W> r;
    if constexpr (W == 1) {
        r.w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else if constexpr (W == 2) {
        const uint2 t = *reinterpret_cast<const uint2*>(p);
        r.w[0] = t.x; r.w[1] = t.y;
    } else {
#pragma unroll
        for (int i = 0; i < W; i += 4) {
            const uint4 t = *reinterpret_cast<const uint4*>(p + 4 * i);
            r.w[i] = t.x; r.w[i + 1] = t.y; r.w[i + 2] = t.z; r.w[i + 3] = t.w;
        }
    }
    return r;
}

// One step's loads: K pieces, V words, the scale of this lane's token (K's in
// lanes 0-31, V's in 32-63), which of the lane's 8 tokens are not seen.
template <int KC, int VW>
struct Loads {
    uint4 k[2][KC];
    Raw<VW> v[8];
    float scale;
    uint32_t hide;
    uint64_t there;
};

// One worker's (a wave's) share of the steps, for its KV head and columns.
// kTail and kPrefix: every piece into the partial results.  pos_of(token), kPrefix:
// a query's position, which masks where its sequence ends inside the prefix.
template <int KST, int VST, int DP, int NT, Part kPart, class PosOf>
__device__ __forceinline__ void decode_share(const DecodeParams& a, int block, PosOf&& pos_of) {
    constexpr int VD = DP / 16;                         // channels of V a lane holds
    constexpr int KC = DP * kElemBytes<KST> / 64;       // 16-byte pieces of K a lane holds per token
    constexpr int KM = DP / 32;                         // matrix steps over the channels
    constexpr int VW = VD * kElemBytes<VST> / 4;        // words of V a lane holds per token
    // a step is loaded while the one before is computed on, where registers allow
    constexpr bool kAhead = NT * (8 * KC + 8 * VW) <= 64;
    __shared__ __align__(16) int s_row[kWaves][kStep];
    __shared__ __align__(16) float s_scale[kWaves][2 * kStep];

    const KvView& kv = a.kv;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 15, g = lane >> 4;
    // A worker is one wave.  The KV heads of a share are neighbours, in one
    // block and on one XCD: their scales and page entries share cache lines.
    const int units = kv.heads * a.col_tiles;
    const int worker = (block >> 3) * kWaves + wave;
    const int hc = worker % units, share = (worker / units) * 8 + (block & 7);
    if (share >= a.shares) return;
    const int h = hc % kv.heads, ct = hc / kv.heads;
    Work work;
    if constexpr (kPart == kPrefix) {
        work.total = a.from / kStep;
        work.chunk = (work.total + a.shares - 1) / a.shares;
        work.len = a.from;
    } else {
        work = work_of<kPart>(a, share, -1, lane);
    }
    const int share_end = min(work.total, (share + 1) * work.chunk);
    for (int at = share * work.chunk, b = work.b, len = work.len, before = work.before; at < share_end;) {
    const int pos = len - 1;
    const Steps<kStep> steps = steps_at<kPart>(a, pos);
    const int seq_steps = steps.count < 1 ? 1 : steps.count;
    const int s_begin = at - before, s_end = min(steps.count, share_end - before);

    const int D = kv.head_dim;
    const int head0 = ct * 16 * NT;                     // first query head of this block within the group
    // (kPrefix: the columns are (query, head in the group))
    const int columns = kPart == kPrefix ? a.columns : a.group;
    b8 qf[NT][KM];
    int ends[NT];                                       // kPrefix: the last token a column sees
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int hq = head0 + nt * 16 + c;
        const uint16_t* qr;
        if constexpr (kPart == kPrefix) {
            const int col = min(hq, columns - 1), token = col / a.group;
            qr = a.q + token * a.ldq + (int64_t)(h * a.group + col - token * a.group) * D;
            ends[nt] = pos_of(token);
        } else {
            qr = a.q + b * a.ldq + (int64_t)(h * a.group + hq) * D;
        }
#pragma unroll
        for (int s = 0; s < KM; ++s) {
            const int e = KST == kBf16 ? s * 32 + g * 8 : (s >> 1) * 64 + g * 16 + (s & 1) * 8;
            uint4 t = make_uint4(0, 0, 0, 0);
            if (hq < columns && e < D) t = *reinterpret_cast<const uint4*>(qr + e);
            qf[nt][s] = __builtin_bit_cast(b8, t);
        }
    }

    f4 o[NT][VD];
    float m[NT], l[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        m[nt] = kLowest; l[nt] = 0.0f;
#pragma unroll
        for (int i = 0; i < VD; ++i) o[nt][i] = f4{0, 0, 0, 0};
    }

    const int64_t k_row = (int64_t)kv.heads * D * kElemBytes<KST>, v_row = (int64_t)kv.heads * D * kElemBytes<VST>;
    const uint8_t* kb = static_cast<const uint8_t*>(kv.k) + (int64_t)h * D * kElemBytes<KST>;
    const uint8_t* vb = static_cast<const uint8_t*>(kv.v) + (int64_t)h * D * kElemBytes<VST> +
                        (VD * c < D ? VD * c : 0) * kElemBytes<VST>;
    const int32_t* table = kv.table + b * kv.table_ld;
    const float k_head = (KST == kBf16 ? 1.0f : kv.per_head ? kv.k_scale[h] : 0.0f) * a.scale_log2;
    const float v_head = VST == kBf16 ? 1.0f : kv.per_head ? kv.v_scale[h] : 0.0f;
    const bool k_per_token = KST != kBf16 && !kv.per_head, v_per_token = VST != kBf16 && !kv.per_head;

    const int half = lane & 31;
    // This lane's page entry of a step; a step or token past the end reads a
    // valid entry, which row_of drops.
    auto entry_of = [&](int st) -> int {
        const int j = min(steps.token(min(st, s_end - 1)) + half, pos);
        return table[j >> kv.page_shift];
    };
    auto row_of = [&](int st, int entry) -> int {
        const int j = steps.token(st) + half;
        return st < s_end && sees(j, pos, kPart == kWhole ? a.window : 0, kPart == kWhole ? a.sinks : 0) ? row_of_entry(kv, entry, j) : -1;
    };
    // A step's loads.  None of them is conditional, so a wait for one step's
    // does not wait for the next one's: a token that is not seen reads row 0.
    auto load = [&](Loads<KC, VW>& s, int row) {
        s.there = __ballot(row >= 0);
        wave_sync();
        s_row[wave][half] = row;
        wave_sync();
        const bool key = lane < 32, per_token = key ? k_per_token : v_per_token;
        const float* sp = per_token ? (key ? kv.k_scale : kv.v_scale) : reinterpret_cast<const float*>(table);
        s.scale = sp[per_token ? (int64_t)max(row, 0) * kv.heads + h : 0];
        s.scale = row < 0 ? 0.0f : !per_token ? (key ? k_head : v_head) : key ? s.scale * a.scale_log2 : s.scale;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const uint8_t* p = kb + max(s_row[wave][16 * t + c], 0) * k_row;
#pragma unroll
            for (int i = 0; i < KC; ++i) {
                const int e = (i * 64 + g * 16) / kElemBytes<KST>;
                s.k[t][i] = *reinterpret_cast<const uint4*>(p + (e < D ? i * 64 + g * 16 : 0));
            }
        }
        s.hide = 0;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int4 r = *reinterpret_cast<const int4*>(&s_row[wave][16 * t + 4 * g]);
            const int ra[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s.hide |= (ra[i] < 0 ? 1u : 0u) << (4 * t + i);
                s.v[4 * t + i] = load_raw<VW>(vb + max(ra[i], 0) * v_row);
            }
        }
    };
    if (s_begin < s_end) {
    Loads<KC, VW> cur, next;
    int entry = entry_of(s_begin);
    const int row = row_of(s_begin, entry);
    entry = entry_of(s_begin + 1);
    load(cur, row);
    for (int st = s_begin; st < s_end; ++st, cur = next) {
        const int row = row_of(st + 1, entry);
        entry = entry_of(st + 2);
        if (kAhead) load(next, row);
        if (cur.there == 0) {
            if (kPart == kWhole && a.scores && lane < kStep)
                for (int col = head0; col < min(head0 + 16 * NT, a.group); ++col)
                    a.scores[((int64_t)b * a.q_heads + h * a.group + col) * a.span + st * kStep + lane] = -INFINITY;
            if (!kAhead) load(next, row);
            continue;
        }
        const bool whole = cur.there == ~0ull;
        wave_sync();
        s_scale[wave][lane] = cur.scale;
        wave_sync();
        if (D < DP) {            // pieces past head_dim
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int i = 0; i < KC; ++i)
                    if ((i * 64 + g * 16) / kElemBytes<KST> >= D) cur.k[t][i] = make_uint4(0, 0, 0, 0);
        }

        // scores of the step: x[nt][4t + i] of token 16t + 4g + i
        float x[NT][8];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            f4 s[NT];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) s[nt] = f4{0, 0, 0, 0};
#pragma unroll
            for (int e = 0; e < KM; ++e) {
                uint4 w;
                if constexpr (KST == kBf16) {
                    w = cur.k[t][e];
                } else {
                    const uint4 r = cur.k[t][e >> 1];
                    const uint32_t w0 = (e & 1) ? r.z : r.x, w1 = (e & 1) ? r.w : r.y;
                    w = make_uint4(decode2<KST>(w0, false), decode2<KST>(w0, true), decode2<KST>(w1, false),
                                   decode2<KST>(w1, true));
                }
                const b8 kf = __builtin_bit_cast(b8, w);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    s[nt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, qf[nt][e], s[nt], 0, 0, 0);
            }
            const f4 ks = *reinterpret_cast<const f4*>(&s_scale[wave][16 * t + 4 * g]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) x[nt][4 * t + i] = s[nt][i] * ks[i];
        }
        if (!whole) {
            // a token the query does not see: no weight, and nothing of its
            // vector (which may hold anything, NaN included)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const bool hidden = cur.hide >> i & 1;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) x[nt][i] = hidden ? -INFINITY : x[nt][i];
#pragma unroll
                for (int w = 0; w < VW; ++w) cur.v[i].w[w] = hidden ? 0 : cur.v[i].w[w];
            }
        }
        // kPrefix: where a column's sequence ends before this step does, tokens that
        // it does not see and others do; what these hold that is not finite
        // must not meet its weights of 0, and is added apart.
        bool cut = false;
        uint32_t odd_tokens = 0;            // of this lane's 8
        if constexpr (kPart == kPrefix) {
            const int first = steps.token(st);
            cut = __any(min_of(ends) < first + kStep - 1);
            if (cut) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        x[nt][i] = first + (i >> 2) * 16 + 4 * g + (i & 3) <= ends[nt] ? x[nt][i] : -INFINITY;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    uint32_t any = 0;
#pragma unroll
                    for (int w = 0; w < VW; ++w) {
                        const uint32_t t = not_finite<VST>(cur.v[i].w[w]);
                        any |= t;
                        cur.v[i].w[w] = cleared<VST>(cur.v[i].w[w], t);
                    }
                    odd_tokens |= (any ? 1u : 0u) << i;
                }
            }
        }
        if (kPart == kWhole && a.scores) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int col = head0 + nt * 16 + c;
                if (col < a.group) {
                    float* to = a.scores + ((int64_t)b * a.q_heads + h * a.group + col) * a.span + st * kStep + 4 * g;
                    *reinterpret_cast<f4*>(to) = f4{x[nt][0], x[nt][1], x[nt][2], x[nt][3]};
                    *reinterpret_cast<f4*>(to + 16) = f4{x[nt][4], x[nt][5], x[nt][6], x[nt][7]};
                }
            }
        }
        // Infinite values of V (E4M3 has none), or scales that may make a
        // weight infinite: the remainders must not meet them, since a negative
        // one would bring the opposite infinity and a zero one NaN.
        uint32_t infinite = __builtin_fabsf(cur.scale) < 0x1p100f ? 0 : 1;
        if constexpr (VST != kE4M3) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int w = 0; w < VW; ++w) infinite |= not_finite<VST>(cur.v[i].w[w]);
        }
        const bool odd = __any(infinite != 0);
        // weights, as the B operand of the second product
        float vs[8];
        {
            const f4 v0 = *reinterpret_cast<const f4*>(&s_scale[wave][32 + 4 * g]);
            const f4 v1 = *reinterpret_cast<const f4*>(&s_scale[wave][48 + 4 * g]);
#pragma unroll
            for (int i = 0; i < 4; ++i) { vs[i] = v0[i]; vs[4 + i] = v1[i]; }
        }
        b8 ph[NT], pl[NT];
        float weight[NT][8];                // kPrefix
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float mx = x[nt][0];
#pragma unroll
            for (int i = 1; i < 8; ++i) mx = fmaxf(mx, x[nt][i]);
            if (__any(mx > m[nt] + kSlack)) {
                const float mn = fmaxf(m[nt], max_xor16(max_xor32(mx)));
                const float f = __builtin_amdgcn_exp2f(m[nt] - mn);
                m[nt] = mn;
                l[nt] *= f;
#pragma unroll
                for (int i = 0; i < VD; ++i) o[nt][i] *= f;
            }
            float p[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                p[i] = __builtin_amdgcn_exp2f(x[nt][i] - m[nt]);
                l[nt] += p[i];
                p[i] *= vs[i];      // a scale that is not seen is 0
                if constexpr (kPart == kPrefix) {
                    if (cut && x[nt][i] == -INFINITY) p[i] = 0.0f;
                    weight[nt][i] = p[i];
                }
            }
            u4 hi, lo;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                hi[i] = pack2(p[2 * i], p[2 * i + 1]);
                lo[i] = pack2(p[2 * i] - as_f32(hi[i] << 16), p[2 * i + 1] - as_f32(hi[i] & 0xFFFF0000u));
            }
            ph[nt] = __builtin_bit_cast(b8, hi);
            pl[nt] = __builtin_bit_cast(b8, lo);
        }
        // O^T += V^T P^T; matrix step d holds channel VD * (row of the tile) + d
        auto products = [&](auto word, auto add) {
#pragma unroll
            for (int w = 0; w < VW; ++w) {
                if constexpr (VST == kBf16) {
                    u4 f0, f1;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t x0 = word(2 * i, w), x1 = word(2 * i + 1, w);
                        f0[i] = __builtin_amdgcn_perm(x1, x0, 0x05040100u);
                        f1[i] = __builtin_amdgcn_perm(x1, x0, 0x07060302u);
                    }
                    add(2 * w, f0);
                    add(2 * w + 1, f1);
                } else {
                    u4 f[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t x0 = word(2 * i, w), x1 = word(2 * i + 1, w);
                        const uint32_t p0 = __builtin_amdgcn_perm(x1, x0, 0x05010400u);
                        const uint32_t p1 = __builtin_amdgcn_perm(x1, x0, 0x07030602u);
                        f[0][i] = decode2<VST>(p0, false);
                        f[1][i] = decode2<VST>(p0, true);
                        f[2][i] = decode2<VST>(p1, false);
                        f[3][i] = decode2<VST>(p1, true);
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) add(4 * w + e, f[e]);
                }
            }
        };
        if (odd) [[unlikely]] {
            // The remainders times the finite values alone, then in their place
            // 2^-24 of the heads, below the sum's last bit: an infinity meets
            // the head's sign twice.
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                u4 lo = __builtin_bit_cast(u4, pl[nt]);
#pragma unroll
                for (int i = 0; i < 4; ++i) lo[i] = cleared<kBf16>(lo[i], not_finite<kBf16>(lo[i]));
                pl[nt] = __builtin_bit_cast(b8, lo);
            }
            products([&](int i, int w) {
                uint32_t x = cur.v[i].w[w];
                asm volatile("" : "+v"(x));         // what is decoded from it is not kept for the products below
                return cleared<VST>(x, not_finite<VST>(x));
            }, [&](int d, u4 w) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    o[nt][d] =
                        __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(b8, w), pl[nt], o[nt][d], 0, 0, 0);
            });
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const u4 hi = __builtin_bit_cast(u4, ph[nt]);
                u4 lo;
                // (a head whose 2^-24 is no normal number: the head again)
                auto small = [](float x) { return __builtin_fabsf(x) < 0x1p-96f ? x : x * 0x1p-24f; };
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    lo[i] = pack2(small(as_f32(hi[i] << 16)), small(as_f32(hi[i] & 0xFFFF0000u)));
                pl[nt] = __builtin_bit_cast(b8, lo);
            }
        }
        products([&](int i, int w) { return cur.v[i].w[w]; }, [&](int d, u4 w) {
            const b8 vf = __builtin_bit_cast(b8, w);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                o[nt][d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf, ph[nt], o[nt][d], 0, 0, 0);
                o[nt][d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf, pl[nt], o[nt][d], 0, 0, 0);
            }
        });
        if constexpr (kPart == kPrefix) {
            if (cut && __any(odd_tokens != 0)) [[unlikely]] {
                for (int i = 0; i < 8; ++i) {
                    const uint64_t lanes = __ballot(odd_tokens >> i & 1);
                    for (int gt = 0; gt < 4; ++gt) {
                        if (!(lanes >> (16 * gt) & 0xFFFF)) continue;
                        const int j = steps.token(st) + (i >> 2) * 16 + 4 * gt + (i & 3);
                        const int row = row_of_entry(kv, table[j >> kv.page_shift], j);
                        const uint8_t* vr = static_cast<const uint8_t*>(kv.v) +
                                            (max(row, 0) * v_row + (int64_t)h * D * kElemBytes<VST>);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            float mine = 0.0f;
#pragma unroll
                            for (int k = 0; k < 8; ++k) mine = k == i ? weight[nt][k] : mine;
                            const float w = __shfl(mine, c + 16 * gt, 64);
                            if (row < 0 || j > ends[nt]) continue;
#pragma unroll
                            for (int k = 0; k < 4; ++k)
#pragma unroll
                                for (int d = 0; d < VD; ++d) {
                                    const int ch = VD * (4 * g + k) + d;
                                    const float v = ch < D ? value_at<VST>(vr, ch) : 0.0f;
                                    if (!__builtin_isfinite(v)) o[nt][d][k] += w * v;
                                }
                        }
                    }
                }
            }
        }
        if (!kAhead) load(next, row);
    }
    }

    const bool alone = kPart == kWhole && s_begin == 0 && share_end - before >= seq_steps;      // the sequence's only piece
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int col = head0 + nt * 16 + c, hq = h * a.group + col;
        const float sum = sum_xor16(sum_xor32(l[nt]));
        if (col >= columns) continue;
        const float f = !alone ? 1.0f : sum == 0.0f ? 0.0f : 1.0f / sum;
        int64_t part = (int64_t)(share + b) * a.q_heads + hq;
        if constexpr (kPart == kPrefix) {
            const int token = col / a.group;
            part = ((int64_t)token * a.q_heads + h * a.group + col - token * a.group) * a.pieces + share;
        }
        if (g == 0) {
            if (!alone) a.part_ml[part] = make_float2(m[nt], sum);
            else if (a.lse)
                a.lse[(int64_t)b * a.q_heads + hq] =
                    sum == 0.0f ? -INFINITY : (m[nt] + __builtin_amdgcn_logf(sum)) * kLn2;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int d0 = VD * (4 * g + i);
            if (d0 >= D) continue;
#pragma unroll
            for (int d = 0; d < VD; d += 4) {
                const f4 v = f4{o[nt][d][i], o[nt][d + 1][i], o[nt][d + 2][i], o[nt][d + 3][i]} * f;
                if (alone)
                    *reinterpret_cast<uint2*>(a.out + b * a.ldo + (int64_t)hq * D + d0 + d) =
                        make_uint2(pack2(v[0], v[1]), pack2(v[2], v[3]));
                else
                    *reinterpret_cast<f4*>(a.part_o + part * D + d0 + d) = v;
            }
        }
    }
    before += seq_steps;
    at = before;
    if (kPart != kPrefix && at < share_end) len = seq_len(kv, ++b);
    }
}

// The maximum and sum of a query head's row over its sequence's n pieces,
// 64 at a time; every lane returns them.
__device__ __forceinline__ float2 join_ml(const float2* ml, int64_t next, int n, int lane) {
    float m = kLowest, l = 0.0f;
    for (int s = lane; s < n; s += 64) m = fmaxf(m, ml[s * next].x);
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) m = fmaxf(m, __shfl_xor(m, off, 64));
    for (int s = lane; s < n; s += 64) l += ml[s * next].y * __builtin_amdgcn_exp2f(ml[s * next].x - m);
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) l += __shfl_xor(l, off, 64);
    return make_float2(m, l);
}

}  // namespace decode
}  // namespace
}  // namespace fp8mi
