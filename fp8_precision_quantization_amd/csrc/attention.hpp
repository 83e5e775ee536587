// attention.hpp -- device helpers shared by the kernels that read the paged
// KV cache in place (attn_decode.hip, attn_extend.hip): where a token's row
// lies, decoding cache rows into bf16 matrix operands, and which tokens a
// query sees.
//
// Sequence b holds L = lens[b] cached tokens, token j in cache row
// page_table[b][j / page] * page + j % page.  A query at position p sees
// token j if j <= p and, with a window W > 0, if j > p - W or j < sinks.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.hpp"
#include "launch.hpp"

namespace fp8mi {
namespace attn {

typedef __bf16 b2 __attribute__((ext_vector_type(2)));
typedef __bf16 b8 __attribute__((ext_vector_type(8)));
typedef float f2 __attribute__((ext_vector_type(2)));
typedef float f4 __attribute__((ext_vector_type(4)));
typedef float f16v __attribute__((ext_vector_type(16)));
typedef uint32_t u2 __attribute__((ext_vector_type(2)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));

constexpr int kBf16 = 2;                    // storage code beside kE4M3 / kE5M2
constexpr float kLowest = -3.402823466e38f; // running maximum of a row that has seen nothing
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// A row's running maximum moves only when a score passes it by this much (in
// powers of two), so most steps rescale nothing; sums then hold terms of at
// most 2^8, far inside fp32.
constexpr float kSlack = 8.0f;

template <int ST> constexpr int kElemBytes = ST == kBf16 ? 2 : 1;

// Two codes (bytes 0,1 or 2,3 of w) as two bf16, exactly: every E4M3 and E5M2
// value, subnormals included, is a bf16 value; NaN stays NaN.
template <int ST>
__device__ __forceinline__ uint32_t decode2(uint32_t w, bool high) {
    b2 r;
    if constexpr (ST == kE4M3)
        r = high ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true)
                 : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false);
    else
        r = high ? __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(w, 1.0f, true)
                 : __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(w, 1.0f, false);
    return __builtin_bit_cast(uint32_t, r);
}

// Words of w that hold a value that is not finite, and the same words with
// these values cleared.
template <int ST>
__device__ __forceinline__ uint32_t not_finite(uint32_t w) {
    uint32_t t;     // the top bit of every element that is not finite
    if constexpr (ST == kE4M3) t = ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
    else if constexpr (ST == kE5M2) t = ((w & 0x7C7C7C7Cu) + 0x04040404u) & 0x80808080u;
    else t = ((w & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
    return t;
}
template <int ST>
__device__ __forceinline__ uint32_t cleared(uint32_t w, uint32_t t) {
    return ST == kBf16 ? w & ~((t >> 15) * 0xFFFFu) : w & ~((t >> 7) * 0xFFu);
}

// Two fp32 -> two bf16 (round to nearest even), low half first.
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const f2 v = {a, b};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, b2));
}

__device__ __forceinline__ float as_f32(uint32_t bits) { return __builtin_bit_cast(float, bits); }

// max / sum over lanes l and l ^ 32, and over l and l ^ 16 (register moves)
__device__ __forceinline__ float max_xor32(float v) {
    const uint32_t u = __builtin_bit_cast(uint32_t, v);
    const u2 r = __builtin_bit_cast(u2, __builtin_amdgcn_permlane32_swap(u, u, false, false));
    return fmaxf(as_f32(r.x), as_f32(r.y));
}
__device__ __forceinline__ float max_xor16(float v) {
    const uint32_t u = __builtin_bit_cast(uint32_t, v);
    const u2 r = __builtin_bit_cast(u2, __builtin_amdgcn_permlane16_swap(u, u, false, false));
    return fmaxf(as_f32(r.x), as_f32(r.y));
}
__device__ __forceinline__ float sum_xor32(float v) {
    const uint32_t u = __builtin_bit_cast(uint32_t, v);
    const u2 r = __builtin_bit_cast(u2, __builtin_amdgcn_permlane32_swap(u, u, false, false));
    return as_f32(r.x) + as_f32(r.y);
}
__device__ __forceinline__ float sum_xor16(float v) {
    const uint32_t u = __builtin_bit_cast(uint32_t, v);
    const u2 r = __builtin_bit_cast(u2, __builtin_amdgcn_permlane16_swap(u, u, false, false));
    return as_f32(r.x) + as_f32(r.y);
}

// LDS exchange inside one wave: its LDS operations complete in order, so
// only the compiler has to be kept from moving them.
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

__device__ __forceinline__ int seq_len(const KvView& kv, int b) {
    const int n = kv.lens[b];
    return n < 0 ? 0 : n > kv.max_len ? (int)kv.max_len : n;
}

// Cache row of token j of a sequence, or -1 where its page lies outside the
// cache (a page that is not there: its tokens are seen by no query).
__device__ __forceinline__ int row_of_entry(const KvView& kv, int entry, int j) {
    const int64_t row = ((int64_t)entry << kv.page_shift) + (j & ((1 << kv.page_shift) - 1));
    return row >= 0 && row < kv.capacity ? (int)row : -1;
}

// The tokens that queries at positions [first, last] may see, as steps of
// STEP tokens: first the steps that hold sinks and no window token, then all
// steps from the first window token to `last`.
template <int STEP>
struct Steps {
    int sink_steps, first_step, count;
    __device__ __forceinline__ Steps(int first, int last, int window, int sinks) {
        int lo = window > 0 ? first - window + 1 : 0;
        lo = lo < 0 ? 0 : lo;
        first_step = lo / STEP;
        const int s = window > 0 ? (sinks + STEP - 1) / STEP : 0;
        sink_steps = s < first_step ? s : first_step;
        count = last < 0 ? 0 : sink_steps + (last / STEP - first_step + 1);
    }
    // first token of step i
    __device__ __forceinline__ int token(int i) const {
        return (i < sink_steps ? i : i - sink_steps + first_step) * STEP;
    }
};

__device__ __forceinline__ bool sees(int j, int p, int window, int sinks) {
    return j <= p && (window <= 0 || j > p - window || j < sinks);
}

}  // namespace attn
}  // namespace fp8mi
