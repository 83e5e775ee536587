// kvappend.hip -- new tokens into the paged KV cache on gfx950, with the
// position rotation of q and k on the way: one launch rotates q (bf16 out),
// rotates and casts k, casts v and scatters both into their cache rows.
//
// Mathematics.  Pair i of the first rotary_dim channels of a head turns by
// angle = position * inv_freq[i], the position being that of the pair's axis:
//   (a, b) -> (a cos - b sin, b cos + a sin)
// in fp32, the pairs being (i, i + rotary_dim / 2) or (2i, 2i + 1).  The angle
// is formed in 64 bits and reduced to a part of a turn there: at position
// 10^6 an fp32 angle would be off by 0.03 rad, one in 64 bits by 10^-10.  k and
// v are then cast as the store alone casts them (kvcache.hip): a head's amax,
// s = fmax / amax, codes of x * s, 1 / s beside them; or the head's fixed scale.
//
// Layout.  The rows of a call are (token, head) with a token's q, k and v heads
// one after the other; a row gets LPR lanes of 16 channels, two units of 8: the
// units (u, u + rotary_dim / 16), so that both halves of a pair are in one
// lane, and two neighbours where nothing turns.  A block takes an even run of
// rows and computes the sines and cosines of its tokens once, in LDS, while its
// first rows are on their way.
//
// Measured (E4M3, bf16 in): 8192 tokens of 32 + 8 + 8 heads of 128 move 185 MB in 40
// us from cold caches (4.6 TB/s; a copy of 2 GiB reaches 5.1) and in 31 with what
// the caches hold; 1531 tokens of 48 heads of 96 on three axes 9.3 us; one token 3.5
// us, a launch and three dependent reads.  The blocks' tables of sines cost least
// in one round of eight blocks a CU (six passes of rows a block for 8192 tokens; in
// rounds of two blocks a CU 36 us); with pointers and pitches chosen by a row's kind
// from the arguments in memory, not in registers, 8192 tokens took 66 us.
#include <hip/hip_runtime.h>

#include "cast_unit.hpp"
#include "device_common.hpp"
#include "launch.hpp"

namespace fp8mi {
namespace {

using namespace cast;
constexpr int kThreads = 256;

typedef float f2 __attribute__((ext_vector_type(2)));
typedef __bf16 b2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const f2 v = {a, b};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, b2));
}

struct AppendParams {
    const void *q, *k, *v;
    int64_t ldq, ldk, ldv;
    uint16_t* q_out;
    int64_t ldqo;
    void *k_cache, *v_cache;
    float *k_scale, *v_scale;
    int k_st, v_st;
    bool per_head, pow2, interleaved;
    int q_heads, heads, head_dim, rotary;
    int64_t capacity;
    const int64_t* slots;
    const int64_t* positions;
    int64_t pos_ld;
    int ends[4];                 // first pair behind each axis
    const float* inv_freq;
    uint32_t rows, run;          // rows of the call, of a block
    fp8_diag* diag;
};

// Cosine and sine of a pair's angle.
__device__ __forceinline__ f2 turn_of(const AppendParams& a, int64_t t, int i) {
    const int axis = (i >= a.ends[0] ? 1 : 0) + (i >= a.ends[1] ? 1 : 0) + (i >= a.ends[2] ? 1 : 0);
    const double turns = (double)a.positions[axis * a.pos_ld + t] * ((double)a.inv_freq[i] * 0.15915494309189535);
    float s, c;
    sincospif(2.0f * (float)(turns - __builtin_rint(turns)), &s, &c);
    return f2{c, s};
}

// The codes (or bf16 values) of one unit.
template <bool DIAG>
__device__ __forceinline__ void put_unit(void* cache, int64_t at, int st, const Pack<float>& p, float s,
                                         Counters& cnt) {
    if (st == FP8_KV_BF16) {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(cache) + at) =
            make_uint4(pack_bf16(p.get(0), p.get(1)), pack_bf16(p.get(2), p.get(3)), pack_bf16(p.get(4), p.get(5)),
                       pack_bf16(p.get(6), p.get(7)));
    } else {
        const uint2 w = st == FP8_KV_E4M3 ? encode_unit<kE4M3, DIAG>(p, s, cnt) : encode_unit<kE5M2, DIAG>(p, s, cnt);
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(cache) + at) = w;
    }
}

// An argument as a register: a choice between two arguments must not become a
// choice of their addresses, which would put all of them into scratch memory.
template <typename T>
__device__ __forceinline__ T held(T x) {
    asm volatile("" : "+s"(x));
    return x;
}

// What differs between q, k and v rows (role 0, 1, 2).
template <typename T>
struct ByRole {
    T q, k, v;
    __device__ __forceinline__ ByRole(T q_, T k_, T v_) : q(held(q_)), k(held(k_)), v(held(v_)) {}
    __device__ __forceinline__ T of(int role) const { return role == 0 ? q : role == 1 ? k : v; }
};

template <typename InT, int LPR, bool DIAG>
__global__ __launch_bounds__(kThreads) void k_kv_append(const AppendParams a) {
    extern __shared__ __align__(16) f2 s_turn[];        // [tokens of the block][rotary / 2]
    __shared__ uint32_t lds[16];
    constexpr int kPass = kThreads / LPR;               // rows of a pass
    typedef const InT __attribute__((address_space(1))) * In;
    const ByRole<const InT*> in(static_cast<const InT*>(a.q), static_cast<const InT*>(a.k), static_cast<const InT*>(a.v));
    const ByRole<int64_t> ld(a.ldq, a.ldk, a.ldv);
    const ByRole<int> before(0, a.q_heads, a.q_heads + a.heads), units(a.rotary >> 4, a.rotary >> 4, 0);
    const ByRole<int> storage(FP8_KV_BF16, a.k_st, a.v_st);
    const ByRole<void*> out(nullptr, a.k_cache, a.v_cache);
    const ByRole<float*> scales(nullptr, a.k_scale, a.v_scale);

    const int j = threadIdx.x & (LPR - 1);
    const uint32_t width = (uint32_t)(a.q_heads + 2 * a.heads);
    const uint32_t first = blockIdx.x * a.run, end = min(first + a.run, a.rows), t0 = first / width;
    const uint32_t pass_t = kPass / width, pass_h = kPass - pass_t * width;
    // the row of this lane: token, place among the token's rows
    uint32_t r = first + threadIdx.x / LPR, t = r / width, place = r - t * width;

    // What a lane holds of a row that is on its way.
    struct Row {
        Pack<InT> raw[2];
        int64_t slot;
        uint32_t t;
        int head, role, u0, u1;
        bool on, turns;
    };
    auto load = [&](Row& row) {
        row.t = t;
        row.role = (int)place < before.k ? 0 : (int)place < before.v ? 1 : 2;
        row.head = (int)place - before.of(row.role);
        const int pair_units = units.of(row.role);
        row.turns = j < pair_units;
        row.u0 = row.turns ? j : 2 * j;
        row.u1 = row.turns ? j + pair_units : 2 * j + 1;
        row.on = r < end && j < a.head_dim >> 4;
        row.slot = -1;
        if (row.on) {
            const In x = (In)(in.of(row.role) + (int64_t)t * ld.of(row.role) + (int64_t)row.head * a.head_dim);
            row.raw[0] = load_unit<InT>((const InT*)(x + row.u0 * 8), 0, 8, true);
            row.raw[1] = load_unit<InT>((const InT*)(x + row.u1 * 8), 0, 8, true);
            if (row.role != 0) row.slot = a.slots ? a.slots[t] : (int64_t)t;
        }
        r += kPass;
        t += pass_t;
        place += pass_h;
        const bool over = place >= width;
        t += over ? 1 : 0;
        place -= over ? width : 0;
    };

    Row row;
    load(row);
    const int pairs = a.rotary >> 1;
    if (pairs > 0) {
        const int n = (int)((end - 1) / width - t0 + 1) * pairs;
        for (int i = threadIdx.x; i < n; i += kThreads) {
            const int token = i / pairs;
            s_turn[i] = turn_of(a, (int64_t)t0 + token, i - token * pairs);
        }
        __syncthreads();
    }
    Counters cnt;
    for (uint32_t at = first; at < end; at += kPass) {
        Row next;
        load(next);
        Pack<float> p[2];
        uint32_t m = 0;
        if (row.on) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) p[i].w[e] = __float_as_uint(row.raw[i].get(e));
            if (row.turns) {
                const f2* turn = s_turn + (row.t - t0) * pairs;
                if (a.interleaved) {
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const f2 cs = turn[(i ? row.u1 : row.u0) * 4 + e];
                            const float x = p[i].get(2 * e), y = p[i].get(2 * e + 1);
                            p[i].w[2 * e] = __float_as_uint(x * cs.x - y * cs.y);
                            p[i].w[2 * e + 1] = __float_as_uint(y * cs.x + x * cs.y);
                        }
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const f2 cs = turn[row.u0 * 8 + e];
                        const float x = p[0].get(e), y = p[1].get(e);
                        p[0].w[e] = __float_as_uint(x * cs.x - y * cs.y);
                        p[1].w[e] = __float_as_uint(y * cs.x + x * cs.y);
                    }
                }
            }
            m = max(p[0].abs_max(), p[1].abs_max());
        }
        m = group_max_u32<LPR>(m);      // every lane of the wave takes part
        if (row.on && row.role == 0) {
            uint16_t* to = a.q_out + (int64_t)row.t * a.ldqo + (int64_t)row.head * a.head_dim;
            put_unit<false>(to, row.u0 * 8, FP8_KV_BF16, p[0], 1.0f, cnt);
            put_unit<false>(to, row.u1 * 8, FP8_KV_BF16, p[1], 1.0f, cnt);
        } else if (row.on && row.slot >= 0 && row.slot < a.capacity) {
            const int st = storage.of(row.role);
            float* const sc = scales.of(row.role);
            const int64_t vec = row.slot * a.heads + row.head;
            float s = 1.0f;
            if (st != FP8_KV_BF16) {
                if (a.per_head) {
                    s = recip_rn(sc[row.head]);
                } else {
                    s = st == FP8_KV_E4M3 ? scale_from_amax_bits<kE4M3>(m, a.pow2)
                                          : scale_from_amax_bits<kE5M2>(m, a.pow2);
                    if (j == 0) sc[vec] = recip_rn(s);
                }
            }
            put_unit<DIAG>(out.of(row.role), vec * a.head_dim + row.u0 * 8, st, p[0], s, cnt);
            put_unit<DIAG>(out.of(row.role), vec * a.head_dim + row.u1 * 8, st, p[1], s, cnt);
        }
        row = next;
    }
    if constexpr (DIAG) block_add_diag(cnt, lds, a.diag);
}

template <typename InT, int LPR>
hipError_t launch_rows(AppendParams& p, bool diag, int num_cus, hipStream_t stream) {
    constexpr int kPass = kThreads / LPR;
    const uint32_t width = (uint32_t)(p.q_heads + 2 * p.heads);
    // As many rows a block as make up one round of 8 blocks a CU, so that a
    // token's sines serve many heads, up to 8 passes and 16 KiB of them (8192
    // tokens of 32 + 8 + 8 heads 31 us; rounds of 2 blocks a CU 36).
    const uint32_t round = kPass * 8u * (uint32_t)num_cus;
    uint32_t passes = (p.rows + round - 1) / round;
    passes = passes > 8 ? 8 : passes;
    auto turns = [&](uint32_t n) {
        return ((n * kPass - 1) / width + 2) * (uint32_t)(p.rotary >> 1) * (uint32_t)sizeof(f2);
    };
    while (passes > 1 && turns(passes) > 16384) --passes;
    p.run = passes * kPass;
    const unsigned bytes = turns(passes);
    const dim3 grid((p.rows + p.run - 1) / p.run), block(kThreads);
    if (diag) hipLaunchKernelGGL((k_kv_append<InT, LPR, true>), grid, block, bytes, stream, p);
    else hipLaunchKernelGGL((k_kv_append<InT, LPR, false>), grid, block, bytes, stream, p);
    return hipGetLastError();
}

template <typename InT>
hipError_t launch_in(AppendParams& p, bool diag, int num_cus, hipStream_t stream) {
    if (p.head_dim <= 64) return launch_rows<InT, 4>(p, diag, num_cus, stream);
    if (p.head_dim <= 128) return launch_rows<InT, 8>(p, diag, num_cus, stream);
    return launch_rows<InT, 16>(p, diag, num_cus, stream);
}

}  // namespace

hipError_t launch_kv_append(const KvAppendArgs& a) {
    AppendParams p;
    p.q = a.q; p.k = a.k; p.v = a.v; p.ldq = a.ldq; p.ldk = a.ldk; p.ldv = a.ldv;
    p.q_out = a.q_out; p.ldqo = a.ldqo;
    p.k_cache = a.kv.k; p.v_cache = a.kv.v; p.k_scale = a.kv.k_scale; p.v_scale = a.kv.v_scale;
    p.k_st = a.kv.k_st; p.v_st = a.kv.v_st; p.per_head = a.kv.per_head; p.pow2 = a.pow2;
    p.interleaved = a.interleaved; p.q_heads = a.q_heads; p.heads = a.kv.heads; p.head_dim = a.kv.head_dim;
    p.rotary = a.rotary; p.capacity = a.kv.capacity; p.slots = a.slots; p.positions = a.positions;
    p.pos_ld = a.pos_ld; p.inv_freq = a.inv_freq; p.diag = a.diag;
    int end = 0;
    for (int i = 0; i < 4; ++i) {
        end += i < a.axes ? a.sections[i] : 0;
        p.ends[i] = i < a.axes - 1 ? end : a.rotary;
    }
    p.rows = (uint32_t)(a.n_tokens * (a.q_heads + 2 * a.kv.heads));
    const bool diag = a.diag != nullptr;
    return a.in_bf16 ? launch_in<uint16_t>(p, diag, a.num_cus, a.stream) : launch_in<float>(p, diag, a.num_cus, a.stream);
}

}  // namespace fp8mi
