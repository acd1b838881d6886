// attend_device.hpp -- what the kernels over the paged cache share: operand
// types, conversions of cached values, exact parts of queries, divisions by the
// page size and the sharing of long sequences.  Internal to libmx.so.
#pragma once
#include "decode_kernels.hpp"

namespace mxk {
using namespace mxd;

namespace {

typedef __bf16 bf8v __attribute__((ext_vector_type(8)));
typedef __bf16 bf2v __attribute__((ext_vector_type(2)));
typedef float f2v __attribute__((ext_vector_type(2)));
typedef float f4v __attribute__((ext_vector_type(4)));
typedef short s2v __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ float e8m0(uint32_t c) {
    return c == 255u ? bitsf(0x7fc00000u) : bitsf(c ? c << 23 : 0x00400000u);
}
__device__ __forceinline__ uint32_t bits_of(bf2v v) {
    uint32_t u;
    __builtin_memcpy(&u, &v, 4);
    return u;
}
__device__ __forceinline__ bf8v frag(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    const uint32_t u[4] = {a, b, c, d};
    bf8v v;
    __builtin_memcpy(&v, u, 16);
    return v;
}

// t / d for t < 2^31 by a multiply: mul = ceil(2^shift / d), 2^shift >= 2^31 d
__device__ __forceinline__ uint32_t over(uint32_t t, Div d) { return (uint32_t)(((uint64_t)t * d.mul) >> d.shift); }
Div div_by(int d) {
    int lg = 0;
    while ((1 << lg) < d) lg++;
    Div o;
    o.shift = 31 + lg;
    o.mul = (uint32_t)((((uint64_t)1 << o.shift) + d - 1) / d);
    return o;
}

// Bits of one value
constexpr int kind_bits(int kind) { return kind == KV_BF16 ? 16 : kind == KV_FP8 ? 8 : 4; }

// `bytes` (4, 8 or 16; 1 or 2 for small V runs) from p into dwords of o
template <int BYTES>
__device__ __forceinline__ void load_bytes(uint32_t* o, const uint8_t* p) {
    if constexpr (BYTES == 16) {
        const u32x4 v = *reinterpret_cast<const u32x4*>(p);
        o[0] = v[0]; o[1] = v[1]; o[2] = v[2]; o[3] = v[3];
    } else if constexpr (BYTES == 8) {
        const u32x2 v = *reinterpret_cast<const u32x2*>(p);
        o[0] = v[0]; o[1] = v[1];
    } else if constexpr (BYTES == 4) {
        o[0] = *reinterpret_cast<const uint32_t*>(p);
    } else if constexpr (BYTES == 2) {
        o[0] = *reinterpret_cast<const uint16_t*>(p);
    } else {
        o[0] = *p;
    }
}

// values 2 i, 2 i + 1 of the run in w as a bf16 pair times 2^e
template <int KIND, int I>
__device__ __forceinline__ uint32_t pair_of(const uint32_t* w, float s) {
    if constexpr (KIND == KV_BF16) return w[I];
    else if constexpr (KIND == KV_FP8) return bits_of(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)w[I / 2], s, (I & 1) != 0));
    else return bits_of(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[I / 4], s, I & 3));
}

template <int... I>
struct seq {};
template <int N, int... I>
struct make_seq : make_seq<N - 1, N - 1, I...> {};
template <int... I>
struct make_seq<0, I...> { typedef seq<I...> type; };
// f(integral_constant 0), ... f(integral_constant N - 1)
template <int V>
struct ic { static constexpr int value = V; };
template <typename F, int... I>
__device__ __forceinline__ void each_(F&& f, seq<I...>) { (f(ic<I>{}), ...); }
template <int N, typename F>
__device__ __forceinline__ void each(F&& f) { each_(f, typename make_seq<N>::type{}); }

// a query value as its exact bf16 parts (bits in the upper halves)
struct Parts {
    uint32_t h, m, l;
};
__device__ __forceinline__ Parts parts_of(float x) {
    const uint32_t u = fbits(x);
    if ((u & 0x7f800000u) == 0x7f800000u) return Parts{(uint32_t)bf16_rne(x) << 16, 0u, 0u};
    const float r = x - bitsf(u & 0xffff0000u);
    return Parts{u & 0xffff0000u, fbits(r) & 0xffff0000u, fbits(r - bitsf(fbits(r) & 0xffff0000u)) & 0xffff0000u};
}
__device__ __forceinline__ uint32_t pack_hi(uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, 0x07060302u); }

constexpr int UNIT = 128;
__device__ __forceinline__ int64_t units_of(int len) { return (len + UNIT - 1) / UNIT; }

__device__ __forceinline__ int workers_used(int64_t units, int workers) { return (int)(units < workers ? units : workers); }

// sum over the workgroup of T threads, in every thread
template <int T>
__device__ __forceinline__ int64_t block_total(int64_t v, int64_t* sh) {
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) v += __shfl_xor(v, o, 64);
    if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
    __syncthreads();
    int64_t t = 0;
#pragma unroll
    for (int i = 0; i < T / 64; i++) t += sh[i];
    __syncthreads();
    return t;
}

}  // namespace
}  // namespace mxk
