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
// the matrix cores, and the second product costs nothing that shows.
#include <hip/hip_runtime.h>

#include "attention.hpp"

namespace fp8mi {
namespace {

using namespace attn;

constexpr int kStep = 32;       // tokens of one wave step
constexpr int kWaves = 4;

struct DecodeParams {
    KvView kv;
    const uint16_t* q;
    int64_t ldq;
    int q_heads, group, col_tiles;
    float scale_log2;
    int window, sinks;
    int chunk, splits;           // steps of a split, splits of the longest sequence
    uint16_t* out;
    int64_t ldo;
    float* lse;
    float2* part_ml;             // [batch, q_heads, splits]
    float* part_o;               // [batch, q_heads, splits, head_dim]
};

__device__ __forceinline__ int splits_of(const DecodeParams& a, int len) {
    const Steps<kStep> st(len - 1, len - 1, a.window, a.sinks);
    return (st.count + a.chunk - 1) / a.chunk;
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

template <int KST, int VST, int DP, int NT>
__global__ __launch_bounds__(64 * kWaves) void k_decode(const DecodeParams a) {
    constexpr int VD = DP / 16;                         // channels of V a lane holds
    constexpr int KC = DP * kElemBytes<KST> / 64;       // 16-byte pieces of K a lane holds per token
    constexpr int KM = DP / 32;                         // matrix steps over the channels
    constexpr int VW = VD * kElemBytes<VST> / 4;        // words of V a lane holds per token
    constexpr int kOPad = DP + 4;
    __shared__ int s_row[kWaves][kStep];
    __shared__ float s_scale[kWaves][2 * kStep];
    __shared__ float s_ml[kWaves][2][16 * NT];
    __shared__ float s_o[16 * NT][kOPad];

    const KvView& kv = a.kv;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int c = lane & 15, g = lane >> 4;
    // All KV heads of a run of tokens on one XCD (their scales share lines).
    const int units = kv.heads * a.col_tiles;
    const int xcd = blockIdx.x & 7, k = blockIdx.x >> 3;
    const int hc = k % units, run = (k / units) * 8 + xcd;
    if (run >= kv.batch * a.splits) return;
    const int h = hc % kv.heads, ct = hc / kv.heads;
    const int b = run / a.splits, split = run % a.splits;

    const int len = seq_len(kv, b);
    const int pos = len - 1;
    const Steps<kStep> steps(pos, pos, a.window, a.sinks);
    const int nsplit = (steps.count + a.chunk - 1) / a.chunk;
    if (split >= nsplit && split > 0) return;
    const int s_end = min(steps.count, (split + 1) * a.chunk);

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
    // the page of this lane's token of a step, -1 where the query does not see it
    auto entry_of = [&](int st) -> int {
        if (st >= s_end) return -1;
        const int j = steps.token(st) + half;
        return sees(j, pos, a.window, a.sinks) ? table[j >> kv.page_shift] : -1;
    };
    int entry = entry_of(split * a.chunk + wave);
    for (int st = split * a.chunk + wave; st < s_end; st += kWaves) {
        const int j = steps.token(st) + half;
        const int row = entry >= 0 ? row_of_entry(kv, entry, j) : -1;
        entry = entry_of(st + kWaves);
        const uint64_t there = __ballot(row >= 0);
        if (there == 0) continue;
        const bool whole = there == ~0ull;
        wave_sync();
        s_row[wave][half] = row;
        wave_sync();
        float sc = lane < 32 ? k_head : v_head;
        if (lane < 32 ? k_per_token : v_per_token) {
            sc = 0.0f;
            if (row >= 0) sc = (lane < 32 ? kv.k_scale : kv.v_scale)[(int64_t)row * kv.heads + h];
            if (lane < 32) sc *= a.scale_log2;
        }
        uint4 kr[2][KC];
        int vrow[8];
        Raw<VW> vr[8];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const uint8_t* p = kb + max(s_row[wave][16 * t + c], 0) * k_row;
#pragma unroll
            for (int i = 0; i < KC; ++i) {
                const int e = (i * 64 + g * 16) / kElemBytes<KST>;
                kr[t][i] = make_uint4(0, 0, 0, 0);
                if (e < D) kr[t][i] = *reinterpret_cast<const uint4*>(p + i * 64 + g * 16);
            }
        }
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int4 r = *reinterpret_cast<const int4*>(&s_row[wave][16 * t + 4 * g]);
            vrow[4 * t] = r.x; vrow[4 * t + 1] = r.y; vrow[4 * t + 2] = r.z; vrow[4 * t + 3] = r.w;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) vr[i] = load_raw<VW>(vb + max(vrow[i], 0) * v_row);
        s_scale[wave][lane] = sc;
        wave_sync();

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
                    w = kr[t][e];
                } else {
                    const uint4 r = kr[t][e >> 1];
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
                if (vrow[i] < 0) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) x[nt][i] = -INFINITY;
#pragma unroll
                    for (int w = 0; w < VW; ++w) vr[i].w[w] = 0;
                }
            }
        }
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
                p[i] = vrow[i] < 0 ? 0.0f : p[i] * vs[i];
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
        auto add = [&](int d, u4 w) {
            const b8 vf = __builtin_bit_cast(b8, w);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                o[nt][d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf, ph[nt], o[nt][d], 0, 0, 0);
                o[nt][d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf, pl[nt], o[nt][d], 0, 0, 0);
            }
        };
#pragma unroll
        for (int w = 0; w < VW; ++w) {
            if constexpr (VST == kBf16) {
                u4 f0, f1;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t x0 = vr[2 * i].w[w], x1 = vr[2 * i + 1].w[w];
                    f0[i] = __builtin_amdgcn_perm(x1, x0, 0x05040100u);
                    f1[i] = __builtin_amdgcn_perm(x1, x0, 0x07060302u);
                }
                add(2 * w, f0);
                add(2 * w + 1, f1);
            } else {
                u4 f[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t x0 = vr[2 * i].w[w], x1 = vr[2 * i + 1].w[w];
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
    }

    // the block's waves, joined in their order
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        l[nt] = sum_xor16(sum_xor32(l[nt]));
        if (g == 0) {
            s_ml[wave][0][nt * 16 + c] = m[nt];
            s_ml[wave][1][nt * 16 + c] = l[nt];
        }
    }
    __syncthreads();
    float mt[NT], lt[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        mt[nt] = kLowest; lt[nt] = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) mt[nt] = fmaxf(mt[nt], s_ml[w][0][nt * 16 + c]);
#pragma unroll
        for (int w = 0; w < kWaves; ++w)
            lt[nt] += s_ml[w][1][nt * 16 + c] * __builtin_amdgcn_exp2f(s_ml[w][0][nt * 16 + c] - mt[nt]);
    }
    for (int w = 0; w < kWaves; ++w) {
        if (wave == w) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const float f = __builtin_amdgcn_exp2f(m[nt] - mt[nt]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
#pragma unroll
                    for (int d = 0; d < VD; d += 4) {
                        f4* to = reinterpret_cast<f4*>(&s_o[nt * 16 + c][VD * (4 * g + i) + d]);
                        f4 v = f4{o[nt][d][i] * f, o[nt][d + 1][i] * f, o[nt][d + 2][i] * f, o[nt][d + 3][i] * f};
                        *to = w == 0 ? v : *to + v;
                    }
                }
            }
        }
        __syncthreads();
    }
    // every wave holds mt, lt of column c: publish them for the writers below
    if (wave == 0 && g == 0) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            s_ml[0][0][nt * 16 + c] = mt[nt];
            s_ml[0][1][nt * 16 + c] = lt[nt];
        }
    }
    __syncthreads();
    const int cols = min(16 * NT, a.group - head0);
    const int quads = D >> 2;
    for (int i = threadIdx.x; i < cols * quads; i += 64 * kWaves) {
        const int col = i / quads, d = (i - col * quads) * 4;
        const int hq = h * a.group + head0 + col;
        const float mm = s_ml[0][0][col], ll = s_ml[0][1][col];
        const f4 v = *reinterpret_cast<const f4*>(&s_o[col][d]);
        if (nsplit <= 1) {
            const float r = ll == 0.0f ? 0.0f : 1.0f / ll;
            *reinterpret_cast<uint2*>(a.out + b * a.ldo + (int64_t)hq * D + d) =
                make_uint2(pack2(v[0] * r, v[1] * r), pack2(v[2] * r, v[3] * r));
            if (d == 0 && a.lse)
                a.lse[(int64_t)b * a.q_heads + hq] = ll == 0.0f ? -INFINITY : (mm + __builtin_amdgcn_logf(ll)) * kLn2;
        } else {
            const int64_t part = ((int64_t)b * a.q_heads + hq) * a.splits + split;
            *reinterpret_cast<f4*>(a.part_o + part * D + d) = v;
            if (d == 0) a.part_ml[part] = make_float2(mm, ll);
        }
    }
}

// One block per (query head, sequence): joins the splits in their order.
// Threads take 4 channels each, several splits side by side.
constexpr int kJoinThreads = 256;

__global__ __launch_bounds__(kJoinThreads) void k_decode_join(const DecodeParams a) {
    __shared__ f4 s_acc[kJoinThreads];
    const int hq = blockIdx.x, b = blockIdx.y;
    const int n = splits_of(a, seq_len(a.kv, b));
    if (n <= 1) return;
    const int D = a.kv.head_dim, quads = D >> 2;
    const int64_t part = ((int64_t)b * a.q_heads + hq) * a.splits;
    const float2* ml = a.part_ml + part;
    float m = kLowest, l = 0.0f;
    for (int s = 0; s < n; ++s) m = fmaxf(m, ml[s].x);
    for (int s = 0; s < n; ++s) l += ml[s].y * __builtin_amdgcn_exp2f(ml[s].x - m);
    const int lanes = kJoinThreads / quads;             // splits side by side (4 or more)
    const int side = threadIdx.x / quads, d = (threadIdx.x - side * quads) * 4;
    f4 acc = {0, 0, 0, 0};
    if (side < lanes) {
        for (int s = side; s < n; s += lanes) {
            const float f = __builtin_amdgcn_exp2f(ml[s].x - m);
            acc += *reinterpret_cast<const f4*>(a.part_o + (part + s) * D + d) * f;
        }
    }
    s_acc[threadIdx.x] = acc;
    __syncthreads();
    if (side != 0) return;
    for (int s = 1; s < lanes; ++s) acc += s_acc[s * quads + threadIdx.x];
    const float r = l == 0.0f ? 0.0f : 1.0f / l;
    *reinterpret_cast<uint2*>(a.out + b * a.ldo + (int64_t)hq * D + d) =
        make_uint2(pack2(acc[0] * r, acc[1] * r), pack2(acc[2] * r, acc[3] * r));
    if (d == 0 && a.lse)
        a.lse[(int64_t)b * a.q_heads + hq] = l == 0.0f ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * kLn2;
}

// How a launch is split: steps of a split and splits of the longest sequence.
struct Plan {
    int col_tiles, wide, chunk, splits;
    int64_t blocks;
};

Plan plan_of(const AttnArgs& a) {
    Plan p;
    const int group = a.q_heads / a.kv.heads;
    p.wide = group > 16 ? 2 : 1;
    p.col_tiles = (group + 16 * p.wide - 1) / (16 * p.wide);
    int64_t steps = (a.kv.max_len + kStep - 1) / kStep;
    if (a.window > 0) {
        const int64_t seen = (a.window + kStep - 1) / kStep + 1 + (a.sinks + kStep - 1) / kStep;
        steps = seen < steps ? seen : steps;
    }
    if (steps < 1) steps = 1;
    const int64_t units = (int64_t)a.kv.batch * a.kv.heads * p.col_tiles;
    // enough blocks to fill the CUs several times over, and at least two
    // steps for each wave of a block
    int64_t chunk = (steps * units + 1023) / 1024;
    const int64_t least = 2 * kWaves;
    chunk = chunk < least ? least : chunk;
    chunk = chunk < steps ? chunk : steps;
    p.chunk = (int)chunk;
    p.splits = (int)((steps + chunk - 1) / chunk);
    p.blocks = (((int64_t)a.kv.batch * p.splits + 7) / 8) * 8 * a.kv.heads * p.col_tiles;
    return p;
}

template <int KST, int VST, int DP>
hipError_t launch_wide(const DecodeParams& p, const Plan& plan, hipStream_t stream) {
    const dim3 grid((unsigned)plan.blocks), block(64 * kWaves);
    if (plan.wide == 1)
        hipLaunchKernelGGL((k_decode<KST, VST, DP, 1>), grid, block, 0, stream, p);
    else
        hipLaunchKernelGGL((k_decode<KST, VST, DP, 2>), grid, block, 0, stream, p);
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

int64_t decode_workspace(const AttnArgs& a) {
    const Plan p = plan_of(a);
    if (p.splits <= 1) return 0;
    const int64_t parts = (int64_t)a.kv.batch * a.q_heads * p.splits;
    return ((parts * 8 + 15) / 16) * 16 + parts * a.kv.head_dim * 4;
}

hipError_t launch_decode(const AttnArgs& a) {
    const Plan plan = plan_of(a);
    DecodeParams p;
    p.kv = a.kv; p.q = a.q; p.ldq = a.ldq; p.q_heads = a.q_heads; p.group = a.q_heads / a.kv.heads;
    p.col_tiles = plan.col_tiles; p.scale_log2 = a.scale * kLog2e; p.window = a.window; p.sinks = a.sinks;
    p.chunk = plan.chunk; p.splits = plan.splits; p.out = a.out; p.ldo = a.ldo; p.lse = a.lse;
    const int64_t parts = (int64_t)a.kv.batch * a.q_heads * plan.splits;
    p.part_ml = reinterpret_cast<float2*>(a.workspace);
    p.part_o = reinterpret_cast<float*>(a.workspace + ((parts * 8 + 15) / 16) * 16);
    hipError_t e;
    switch (a.kv.k_st) {
    case FP8_KV_E4M3: e = launch_v<kE4M3>(p, plan, a.stream); break;
    case FP8_KV_E5M2: e = launch_v<kE5M2>(p, plan, a.stream); break;
    default: e = launch_v<kBf16>(p, plan, a.stream); break;
    }
    if (e != hipSuccess || plan.splits <= 1) return e;
    hipLaunchKernelGGL(k_decode_join, dim3((unsigned)a.q_heads, (unsigned)a.kv.batch), dim3(kJoinThreads), 0, a.stream,
                       p);
    return hipGetLastError();
}

}  // namespace fp8mi
