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

#include "attention.hpp"

namespace fp8mi {
namespace {

using namespace attn;

constexpr int kStep = 32;       // tokens of one wave step
constexpr int kWaves = 4;
constexpr int kMaxScored = 64;  // query heads of a KV head up to which scores are stored for the weights

struct DecodeParams {
    KvView kv;
    const uint16_t* q;
    int64_t ldq;
    int q_heads, group, col_tiles;
    float scale_log2;
    int window, sinks;
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

__device__ __forceinline__ int steps_of(const DecodeParams& a, int len) {
    const int n = Steps<kStep>(len - 1, len - 1, a.window, a.sinks).count;
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
__device__ __forceinline__ Work work_of(const DecodeParams& a, int share, int seq, int lane) {
    Work w;
    const int B = a.kv.batch;
    int sum = 0, mine = 0, len = 0;      // of the last 64 sequences looked at
    auto look = [&](int b0) {
        len = b0 + lane < B ? seq_len(a.kv, b0 + lane) : 0;
        mine = b0 + lane < B ? steps_of(a, len) : 0;
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

template <int KST, int VST, int DP, int NT>
__global__ __launch_bounds__(64 * kWaves, DP <= 128 && NT == 1 ? 2 : 1) void k_decode(const DecodeParams a) {
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
    const int worker = (blockIdx.x >> 3) * kWaves + wave;
    const int hc = worker % units, share = (worker / units) * 8 + (blockIdx.x & 7);
    if (share >= a.shares) return;
    const int h = hc % kv.heads, ct = hc / kv.heads;
    const Work work = work_of(a, share, -1, lane);
    const int share_end = min(work.total, (share + 1) * work.chunk);
    for (int at = share * work.chunk, b = work.b, len = work.len, before = work.before; at < share_end;) {
    const int pos = len - 1;
    const Steps<kStep> steps(pos, pos, a.window, a.sinks);
    const int seq_steps = steps.count < 1 ? 1 : steps.count;
    const int s_begin = at - before, s_end = min(steps.count, share_end - before);

    const int D = kv.head_dim;
    const int head0 = ct * 16 * NT;                     // first query head of this block within the group
    b8 qf[NT][KM];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int hq = head0 + nt * 16 + c;
        const uint16_t* qr = a.q + b * a.ldq + (int64_t)(h * a.group + hq) * D;
#pragma unroll
        for (int s = 0; s < KM; ++s) {
            const int e = KST == kBf16 ? s * 32 + g * 8 : (s >> 1) * 64 + g * 16 + (s & 1) * 8;
            uint4 t = make_uint4(0, 0, 0, 0);
            if (hq < a.group && e < D) t = *reinterpret_cast<const uint4*>(qr + e);
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
        return st < s_end && sees(j, pos, a.window, a.sinks) ? row_of_entry(kv, entry, j) : -1;
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
            if (a.scores && lane < kStep)
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
        if (a.scores) {
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
        if (!kAhead) load(next, row);
    }
    }

    const bool alone = s_begin == 0 && share_end - before >= seq_steps;      // the sequence's only piece
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int col = head0 + nt * 16 + c, hq = h * a.group + col;
        const float sum = sum_xor16(sum_xor32(l[nt]));
        if (col >= a.group) continue;
        const float f = !alone ? 1.0f : sum == 0.0f ? 0.0f : 1.0f / sum;
        const int64_t part = (int64_t)(share + b) * a.q_heads + hq;
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
    if (at < share_end) len = seq_len(kv, ++b);
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
    const Work w = work_of(a, 0, b, lane);
    const int i0 = w.before / w.chunk, n = (w.before + steps_of(a, w.len) - 1) / w.chunk - i0 + 1;
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
    p.col_tiles = plan.col_tiles; p.scale_log2 = a.scale * kLog2e; p.window = a.window; p.sinks = a.sinks;
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
