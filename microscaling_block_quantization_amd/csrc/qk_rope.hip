// qk_rope.hip -- norm of each query and key head and rotation by the token's
// position, in one pass, and its gradient.
//
// Mathematics.  n = x rstd, rstd = (mean x^2 + eps)^-1/2, u = w n, and each
// pair (u_a, u_b) is turned by the angle of the position.  Backward: g is the
// output's gradient turned back, dw = sum g n, h = w g, and since rstd depends
// on every x, dx = rstd (h - n mean(h n)).  rstd is formed again from x (a
// read of it is needed for n anyway), so forward keeps nothing.
//
// Both are bound by memory: 2 (forward) or 3 (backward) passes over the heads
// and nothing else, so the layout serves the loads.  A lane holds 16 values of
// a head as two 16-byte chunks (bf16), and the chunks are chosen so that both
// halves of each of its eight pairs are its own: 8 u .. and rot/2 + 8 u .. of
// the rotated part, 16 u .. elsewhere or when pairs are adjacent.  A head is
// then 4 to 64 lanes (8 at 128 values), the norm's sum a few lane exchanges
// inside them, the rotation in registers, and a lane's eight cosines and sines
// are the same for every head of a token: it takes several heads of one token
// at once, which also keeps that many loads in flight.
// Measured (8192 tokens of 32 + 8 heads of 128, bf16, inputs from memory):
// forward 33.6 us, 5.1 TB/s; backward with its weight sums 58 us, 4.4 TB/s; a
// large copy reaches 5.1.
#include "decode_kernels.hpp"

// nothing here is held to bits: fused multiply-adds are as exact and half the work
#pragma clang fp contract(fast)

namespace mxk {
using namespace mxd;

namespace {

constexpr int RT = 256;               // threads per workgroup

typedef __bf16 bf2v __attribute__((ext_vector_type(2)));
typedef float f2v __attribute__((ext_vector_type(2)));
typedef float f4v __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float ld1(const void* p, int64_t i, bool bf) {
    return bf ? bf16f(static_cast<const uint16_t*>(p)[i]) : static_cast<const float*>(p)[i];
}

// sum over an aligned group of LP lanes, the same in each
template <int LP>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int o = 1; o < LP; o <<= 1) v += __shfl_xor(v, o, 64);
    return v;
}

template <bool BF>
__device__ __forceinline__ void load8(float* f, const void* base, int64_t at) {
    if constexpr (BF) {
        const u32x4 v = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(base) + at);
#pragma unroll
        for (int e = 0; e < 4; e++) { f[2 * e] = bf16lo(v[e]); f[2 * e + 1] = bf16hi(v[e]); }
    } else {
        const float4* s = reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
        const float4 a = s[0], b = s[1];
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w; f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    }
}
// A launch that writes more than the chip's L2 holds (eight times 4 MiB) writes
// past it, backward also reads past it: forward 8192 tokens of 40 heads of 128,
// inputs from memory, 42.9 -> 33.6 us (streamed loads as well: 36.7), backward
// 61 -> 58; a smaller launch leaves its output where the next kernel finds it.
constexpr int64_t STREAM_BYTES = 32 << 20;
template <bool NT>
__device__ __forceinline__ void put16(u32x4* p, u32x4 v) {
    if constexpr (NT) __builtin_nontemporal_store(v, p);
    else *p = v;
}
template <bool NT>
__device__ __forceinline__ u32x4 get16(const u32x4* p) {
    if constexpr (NT) return __builtin_nontemporal_load(p);
    else return *p;
}

template <bool BF, bool NT>
__device__ __forceinline__ void store8(const float* f, void* base, int64_t at) {
    if constexpr (BF) {
        u32x4 v;
#pragma unroll
        for (int e = 0; e < 4; e++) {
            const f2v p = {f[2 * e], f[2 * e + 1]};
            const bf2v b = __builtin_convertvector(p, bf2v);              // one instruction: to nearest even, NaN quiet
            uint32_t w;
            __builtin_memcpy(&w, &b, 4);
            v[e] = w;
        }
        put16<NT>(reinterpret_cast<u32x4*>(static_cast<uint16_t*>(base) + at), v);
    } else {
        u32x4* d = reinterpret_cast<u32x4*>(static_cast<float*>(base) + at);
        put16<NT>(d, u32x4{fbits(f[0]), fbits(f[1]), fbits(f[2]), fbits(f[3])});
        put16<NT>(d + 1, u32x4{fbits(f[4]), fbits(f[5]), fbits(f[6]), fbits(f[7])});
    }
}

// weight values of a lane's two chunks
__device__ __forceinline__ void load_w(float* w, const void* p, bool bf, int a, int b) {
    if (bf) { load8<true>(w, p, a); load8<true>(w + 8, p, b); }
    else { load8<false>(w, p, a); load8<false>(w + 8, p, b); }
}

// The pair arithmetic of a lane's 16 values: pairs are (v[i], v[8 + i]), or
// (v[2 i], v[2 i + 1]) when adjacent.  SIGN -1 turns back.
template <int SIGN>
__device__ __forceinline__ void turn(float* v, const float* c, const float* s, bool adjacent) {
    if (adjacent) {
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const float a = v[2 * i], b = v[2 * i + 1], sn = SIGN * s[i];
            v[2 * i] = a * c[i] - b * sn;
            v[2 * i + 1] = b * c[i] + a * sn;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const float a = v[i], b = v[8 + i], sn = SIGN * s[i];
            v[i] = a * c[i] - b * sn;
            v[8 + i] = b * c[i] + a * sn;
        }
    }
}

// cosines and sines of the position's row from pair i0 on; a position outside
// the table gives NaN
__device__ __forceinline__ void load_turn(const RopeParams& p, int64_t token, int i0, float* c, float* s) {
    const int pos = p.positions[token];
    const bool ok = pos >= 0 && (int64_t)pos < p.table_rows;
    const int64_t at = (int64_t)(ok ? pos : 0) * (p.rot / 2) + i0;
    load8<false>(c, p.cos, at);
    load8<false>(s, p.sin, at);
#pragma unroll
    for (int i = 0; i < 8; i++) {
        c[i] = ok ? c[i] : bitsf(0x7fc00000u);
        s[i] = ok ? s[i] : bitsf(0x7fc00000u);
    }
}

// The queries' set or the keys', field by field (indexing the arguments would
// put them in memory).
__device__ __forceinline__ RopeSet set_of(const RopeParams& p, bool k) {
    const RopeSet &a = p.set[0], &b = p.set[1];
    RopeSet S;
    S.x = k ? b.x : a.x;
    S.g = k ? b.g : a.g;
    S.y = k ? b.y : a.y;
    S.x_ts = k ? b.x_ts : a.x_ts;
    S.x_hs = k ? b.x_hs : a.x_hs;
    S.g_ts = k ? b.g_ts : a.g_ts;
    S.g_hs = k ? b.g_hs : a.g_hs;
    S.y_ts = k ? b.y_ts : a.y_ts;
    S.y_hs = k ? b.y_hs : a.y_hs;
    S.heads = k ? b.heads : a.heads;
    S.w = k ? b.w : a.w;
    S.dw = k ? b.dw : a.dw;
    S.parts = k ? b.parts : a.parts;
    S.b0 = k ? b.b0 : a.b0;
    S.nb = k ? b.nb : a.nb;
    return S;
}

// One set (queries or keys) of this launch: workgroups [b0, b0 + nb) take it.
// LP lanes a head, HB heads of one token a lane.  dim and rot multiples of 16.
template <bool BF, int LP, int HB, bool NT>
__global__ __launch_bounds__(RT) void k_rope(RopeParams p) {
    const RopeSet S = set_of(p, blockIdx.x >= p.set[0].nb);
    const uint32_t block = blockIdx.x - S.b0;
    const int u = threadIdx.x % LP;                      // this lane's 16 values
    const uint32_t slot = block * (RT / LP) + threadIdx.x / LP;
    const uint32_t groups = (S.heads + HB - 1) / HB;
    const uint32_t token = slot / groups, h0 = (slot - token * groups) * HB;
    if ((int64_t)token >= p.tokens) return;              // whole groups of LP lanes leave
    const bool live = u < p.dim / 16, turns = u < p.rot / 16;
    const int a = turns && !p.adjacent ? 8 * u : 16 * u;
    const int b = turns && !p.adjacent ? p.rot / 2 + 8 * u : 16 * u + 8;

    float v[HB][16];
    if (live) {
#pragma unroll
        for (int h = 0; h < HB; h++) {
            const uint32_t hh = h0 + h < S.heads ? h0 + h : S.heads - 1;
            const int64_t at = (int64_t)token * S.x_ts + (int64_t)hh * S.x_hs;
            load8<BF>(v[h], S.x, at + a);
            load8<BF>(v[h] + 8, S.x, at + b);
        }
    } else {
#pragma unroll
        for (int h = 0; h < HB; h++)
#pragma unroll
            for (int e = 0; e < 16; e++) v[h][e] = 0.f;
    }
    float c[8], s[8];
    if (turns) load_turn(p, token, 8 * u, c, s);
    if (S.w) {
        float w[16];
        if (live) load_w(w, S.w, p.w_bf16, a, b);
        else {
#pragma unroll
            for (int e = 0; e < 16; e++) w[e] = 0.f;
        }
#pragma unroll
        for (int h = 0; h < HB; h++) {
            float q = 0.f;
#pragma unroll
            for (int e = 0; e < 16; e++) q += v[h][e] * v[h][e];
            const float rstd = 1.0f / sqrtf(group_sum<LP>(q) / (float)p.dim + p.eps);
#pragma unroll
            for (int e = 0; e < 16; e++) v[h][e] = v[h][e] * rstd * w[e];
        }
    }
    if (turns) {
#pragma unroll
        for (int h = 0; h < HB; h++) turn<1>(v[h], c, s, p.adjacent);
    }
    if (live) {
#pragma unroll
        for (int h = 0; h < HB; h++) {
            if (h0 + h >= S.heads) break;
            const int64_t at = (int64_t)token * S.y_ts + (int64_t)(h0 + h) * S.y_hs;
            store8<BF, NT>(v[h], S.y, at + a);
            store8<BF, NT>(v[h] + 8, S.y, at + b);
        }
    }
}

// 16 values of a head as loaded
template <bool BF>
struct Raw {
    u32x4 v[BF ? 2 : 4];
};
template <bool BF, bool NT>
__device__ __forceinline__ void load_raw(Raw<BF>& o, const void* base, int64_t at, int a, int b) {
    if constexpr (BF) {
        const uint16_t* p = static_cast<const uint16_t*>(base) + at;
        o.v[0] = get16<NT>(reinterpret_cast<const u32x4*>(p + a));
        o.v[1] = get16<NT>(reinterpret_cast<const u32x4*>(p + b));
    } else {
        const float* p = static_cast<const float*>(base) + at;
        o.v[0] = get16<NT>(reinterpret_cast<const u32x4*>(p + a));
        o.v[1] = get16<NT>(reinterpret_cast<const u32x4*>(p + a + 4));
        o.v[2] = get16<NT>(reinterpret_cast<const u32x4*>(p + b));
        o.v[3] = get16<NT>(reinterpret_cast<const u32x4*>(p + b + 4));
    }
}
template <bool BF>
__device__ __forceinline__ void widen(float* f, const Raw<BF>& o) {
#pragma unroll
    for (int e = 0; e < 16; e++) {
        if constexpr (BF) f[e] = (e & 1) ? bf16hi(o.v[e / 8][e % 8 / 2]) : bf16lo(o.v[e / 8][e % 8 / 2]);
        else f[e] = bitsf(o.v[BF ? 0 : e / 4][e % 4]);
    }
}

// Backward: the same lanes and chunks; a workgroup walks over its share of the
// set's tokens and keeps the weight gradient of its lanes in registers, joins
// them over its lanes in a fixed order and writes one partial row.  The next
// heads are loaded, as they lie in memory, before the present ones are worked
// on, and the position of the ones after that, which the angles' loads wait for.
template <bool BF, int LP, int HB, bool NT>
__global__ __launch_bounds__(RT, 2) void k_rope_back(RopeParams p) {
    __shared__ float sh[RT / 64][16 * LP];
    const RopeSet S = set_of(p, blockIdx.x >= p.set[0].nb);
    const uint32_t block = blockIdx.x - S.b0;
    const int u = threadIdx.x % LP;
    const uint32_t groups = (S.heads + HB - 1) / HB;
    const uint32_t slots = (uint32_t)p.tokens * groups, stride = S.nb * (RT / LP);
    const bool live = u < p.dim / 16, turns = u < p.rot / 16;
    // lanes past the head's values load the last ones and drop what they get
    const int ul = live ? u : p.dim / 16 - 1;
    const bool halves = ul < p.rot / 16 && !p.adjacent;
    const int a = halves ? 8 * ul : 16 * ul, b = halves ? p.rot / 2 + 8 * ul : 16 * ul + 8;
    const bool norm = S.w != nullptr;

    float w[16], dw[16];
#pragma unroll
    for (int e = 0; e < 16; e++) { w[e] = 0.f; dw[e] = 0.f; }
    if (norm && live) load_w(w, S.w, p.w_bf16, a, b);

    struct Set {
        Raw<BF> x[HB], g[HB];
        u32x4 c[2], s[2];
        uint32_t token, h0;
        bool ok;                       // the position lies in the table
    };
    const int cu = turns ? 8 * u : 0;
    auto position = [&](uint32_t slot) { return p.rot ? p.positions[slot / groups] : 0; };
    auto load = [&](Set& o, uint32_t slot, int pos) {
        o.token = slot / groups;
        o.h0 = (slot - o.token * groups) * HB;
        o.ok = pos >= 0 && (int64_t)pos < p.table_rows;
#pragma unroll
        for (int h = 0; h < HB; h++) {
            const uint32_t hh = o.h0 + h < S.heads ? o.h0 + h : S.heads - 1;
            load_raw<BF, NT>(o.g[h], S.g, (int64_t)o.token * S.g_ts + (int64_t)hh * S.g_hs, a, b);
            if (norm) load_raw<BF, NT>(o.x[h], S.x, (int64_t)o.token * S.x_ts + (int64_t)hh * S.x_hs, a, b);
        }
        if (p.rot) {
            const int64_t at = (o.ok ? (int64_t)pos : 0) * (p.rot / 2) + cu;
            const u32x4 *c = reinterpret_cast<const u32x4*>(p.cos + at), *s = reinterpret_cast<const u32x4*>(p.sin + at);
            o.c[0] = c[0]; o.c[1] = c[1];
            o.s[0] = s[0]; o.s[1] = s[1];
        }
    };
    auto work = [&](const Set& o) {
        float c[8], s[8];
        if (turns) {
#pragma unroll
            for (int i = 0; i < 8; i++) {
                c[i] = o.ok ? bitsf(o.c[i / 4][i % 4]) : bitsf(0x7fc00000u);
                s[i] = o.ok ? bitsf(o.s[i / 4][i % 4]) : bitsf(0x7fc00000u);
            }
        }
#pragma unroll
        for (int h = 0; h < HB; h++) {
            const bool own = o.h0 + h < S.heads;              // not the repeated last head
            float g[16];
            widen(g, o.g[h]);
            if (turns) turn<-1>(g, c, s, p.adjacent);
            if (norm) {
                float x[16], q = 0.f, m = 0.f;
                widen(x, o.x[h]);
#pragma unroll
                for (int e = 0; e < 16; e++) {
                    if (!live) x[e] = g[e] = 0.f;
                    q += x[e] * x[e];
                    m += g[e] * w[e] * x[e];
                }
                const float rstd = 1.0f / sqrtf(group_sum<LP>(q) / (float)p.dim + p.eps);
                m = group_sum<LP>(m) / (float)p.dim * rstd;   // mean of h n
#pragma unroll
                for (int e = 0; e < 16; e++) {
                    const float n = x[e] * rstd;
                    if (own) dw[e] += g[e] * n;
                    g[e] = rstd * (g[e] * w[e] - n * m);
                }
            }
            if (live && own) {
                const int64_t at = (int64_t)o.token * S.y_ts + (int64_t)(o.h0 + h) * S.y_hs;
                store8<BF, NT>(g, S.y, at + a);
                store8<BF, NT>(g + 8, S.y, at + b);
            }
        }
    };
    // Writing onto the incoming gradient: every slot's heads are read by the
    // lanes that write them, and before they do.
    const uint32_t first = block * (RT / LP) + threadIdx.x / LP;
    if (first < slots) {
        auto at = [&](uint32_t slot) { return slot < slots ? slot : first; };
        Set one, two;
        load(one, first, position(first));
        int ahead = position(at(first + stride));
        for (uint32_t slot = first; slot < slots; slot += 2 * stride) {
            if (slot + stride < slots) load(two, slot + stride, ahead);
            ahead = position(at(slot + 2 * stride));
            __builtin_amdgcn_sched_barrier(0);
            work(one);
            if (slot + stride >= slots) break;
            if (slot + 2 * stride < slots) load(one, slot + 2 * stride, ahead);
            ahead = position(at(slot + 3 * stride));
            __builtin_amdgcn_sched_barrier(0);
            work(two);
        }
    }
    if (!S.w) return;                                    // uniform
    // lanes with the same values, then the waves
#pragma unroll
    for (int e = 0; e < 16; e++) {
#pragma unroll
        for (int o = LP; o < 64; o <<= 1) dw[e] += __shfl_xor(dw[e], o, 64);
    }
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    if (lane < LP) {
#pragma unroll
        for (int e = 0; e < 16; e++) sh[wave][16 * lane + e] = dw[e];
    }
    __syncthreads();
    // value 16 u + e of the lanes is element a + e (e < 8) or b + e - 8
    for (int i = threadIdx.x; i < p.dim; i += RT) {
        float t = 0.f;
#pragma unroll
        for (int k = 0; k < RT / 64; k++) t += sh[k][i];
        const int ui = i / 16, e = i % 16;
        const bool tu = ui < p.rot / 16 && !p.adjacent;
        const int at = e < 8 ? (tu ? 8 * ui : 16 * ui) + e : (tu ? p.rot / 2 + 8 * ui : 16 * ui + 8) + e - 8;
        S.parts[(int64_t)block * p.dim + at] = t;
    }
}

// Any other dim and rot: a wave per head, pairs of single values 64 apart.
// Pair i < rot/2 turns; the rest are neighbours past the rotated part.
constexpr int GP = 8;                 // pairs per lane: dim <= 1024
__device__ __forceinline__ void gen_pair(const RopeParams& p, int i, int& a, int& b) {
    if (i < p.rot / 2) {
        a = p.adjacent ? 2 * i : i;
        b = p.adjacent ? 2 * i + 1 : i + p.rot / 2;
    } else {
        a = 2 * i;
        b = 2 * i + 1;
    }
}
__device__ __forceinline__ float wsum(float v) { return group_sum<64>(v); }

template <bool BF>
__device__ __forceinline__ void st1(void* p, int64_t i, float v) {
    if constexpr (BF) static_cast<uint16_t*>(p)[i] = bf16_rne(v);
    else static_cast<float*>(p)[i] = v;
}

template <bool BF, bool BACK>
__global__ __launch_bounds__(RT) void k_rope_any(RopeParams p) {
    __shared__ float sh[BACK ? RT / 64 : 1][BACK ? 2 * GP * 64 : 1];
    const RopeSet S = set_of(p, blockIdx.x >= p.set[0].nb);
    const uint32_t block = blockIdx.x - S.b0;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint32_t slots = (uint32_t)p.tokens * S.heads, stride = S.nb * (RT / 64);
    float da[GP], db[GP];
#pragma unroll
    for (int k = 0; k < GP; k++) da[k] = db[k] = 0.f;
    for (uint32_t slot = block * (RT / 64) + wave; slot < slots; slot += stride) {
        const uint32_t token = slot / S.heads, h = slot - token * S.heads;
        const int64_t ax = (int64_t)token * S.x_ts + (int64_t)h * S.x_hs;
        const int64_t ag = (int64_t)token * S.g_ts + (int64_t)h * S.g_hs;
        const int64_t ay = (int64_t)token * S.y_ts + (int64_t)h * S.y_hs;
        const int pos = p.rot ? p.positions[token] : 0;
        const bool ok = pos >= 0 && (int64_t)pos < p.table_rows;
        float xa[GP], xb[GP], ga[GP], gb[GP], wa[GP], wb[GP];
        float q = 0.f, m = 0.f;
#pragma unroll
        for (int k = 0; k < GP; k++) {
            const int i = lane + 64 * k;
            xa[k] = xb[k] = ga[k] = gb[k] = wa[k] = wb[k] = 0.f;
            if (i >= p.dim / 2) continue;
            int a, b;
            gen_pair(p, i, a, b);
            if (!BACK || S.w) { xa[k] = ld1(S.x, ax + a, BF); xb[k] = ld1(S.x, ax + b, BF); }
            if (S.w) { wa[k] = ld1(S.w, a, p.w_bf16); wb[k] = ld1(S.w, b, p.w_bf16); }
            float c = 1.f, s = 0.f;
            if (i < p.rot / 2) {
                const int64_t t = (int64_t)pos * (p.rot / 2) + i;
                c = ok ? p.cos[t] : bitsf(0x7fc00000u);
                s = ok ? p.sin[t] : bitsf(0x7fc00000u);
            }
            if constexpr (BACK) {
                const float fa = ld1(S.g, ag + a, BF), fb = ld1(S.g, ag + b, BF);
                ga[k] = i < p.rot / 2 ? fa * c + fb * s : fa;
                gb[k] = i < p.rot / 2 ? fb * c - fa * s : fb;
                m += ga[k] * wa[k] * xa[k] + gb[k] * wb[k] * xb[k];
            } else {
                ga[k] = c;
                gb[k] = s;
            }
            q += xa[k] * xa[k] + xb[k] * xb[k];
        }
        const float rstd = S.w ? 1.0f / sqrtf(wsum(q) / (float)p.dim + p.eps) : 1.f;
        if constexpr (BACK) m = wsum(m) / (float)p.dim * rstd;
#pragma unroll
        for (int k = 0; k < GP; k++) {
            const int i = lane + 64 * k;
            if (i >= p.dim / 2) continue;
            int a, b;
            gen_pair(p, i, a, b);
            if constexpr (BACK) {
                if (S.w) {
                    const float na = xa[k] * rstd, nb = xb[k] * rstd;
                    da[k] += ga[k] * na;
                    db[k] += gb[k] * nb;
                    ga[k] = rstd * (ga[k] * wa[k] - na * m);
                    gb[k] = rstd * (gb[k] * wb[k] - nb * m);
                }
                st1<BF>(S.y, ay + a, ga[k]);
                st1<BF>(S.y, ay + b, gb[k]);
            } else {
                const float ua = S.w ? xa[k] * rstd * wa[k] : xa[k], ub = S.w ? xb[k] * rstd * wb[k] : xb[k];
                st1<BF>(S.y, ay + a, i < p.rot / 2 ? ua * ga[k] - ub * gb[k] : ua);
                st1<BF>(S.y, ay + b, i < p.rot / 2 ? ub * ga[k] + ua * gb[k] : ub);
            }
        }
    }
    if constexpr (BACK) {
        if (!S.w) return;
#pragma unroll
        for (int k = 0; k < GP; k++) {
            sh[wave][lane + 64 * k] = da[k];
            sh[wave][GP * 64 + lane + 64 * k] = db[k];
        }
        __syncthreads();
        for (int i = threadIdx.x; i < p.dim / 2; i += RT) {
            float ta = 0.f, tb = 0.f;
#pragma unroll
            for (int k = 0; k < RT / 64; k++) { ta += sh[k][i]; tb += sh[k][GP * 64 + i]; }
            int a, b;
            gen_pair(p, i, a, b);
            S.parts[(int64_t)block * p.dim + a] = ta;
            S.parts[(int64_t)block * p.dim + b] = tb;
        }
    }
}

// The partial rows of a set added up: four values a workgroup, each thread
// every 256th row, then the threads in order.
__global__ __launch_bounds__(RT) void k_rope_weights(RopeParams p) {
    __shared__ f4v sh[RT];
    const RopeSet S = set_of(p, blockIdx.y != 0);
    if (!S.w) return;
    const int i = blockIdx.x * 4, tid = threadIdx.x;
    f4v t = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < ROPE_PARTS / RT; k++) {
        const uint32_t b = k * RT + tid;
        if (b < S.nb) t += *reinterpret_cast<const f4v*>(S.parts + (int64_t)b * p.dim + i);
    }
    sh[tid] = t;
#pragma unroll
    for (int n = RT / 2; n; n /= 2) {
        __syncthreads();
        if (tid < n) sh[tid] += sh[tid + n];
    }
    if (tid == 0) *reinterpret_cast<f4v*>(S.dw + i) = sh[0];
}

constexpr int64_t BACK_BLOCKS = 512;   // most workgroups of a backward launch: two on each CU

// Workgroups of each set: one per RT / LP slots; where that is more than `cap`
// in all, as many rounds as it takes, the same for both sets.
uint32_t set_blocks(RopeParams& p, int lp, int hb, int64_t cap) {
    int64_t need[2], rounds = 1;
    for (int i = 0; i < 2; i++)
        need[i] = p.set[i].heads ? (p.tokens * ((p.set[i].heads + hb - 1) / hb) + RT / lp - 1) / (RT / lp) : 0;
    if (cap)                                              // a block more than the chip holds would be a round of its own
        while ((need[0] + rounds - 1) / rounds + (need[1] + rounds - 1) / rounds > cap) rounds++;
    uint32_t at = 0;
    for (int i = 0; i < 2; i++) {
        p.set[i].b0 = at;
        p.set[i].nb = (uint32_t)((need[i] + rounds - 1) / rounds);
        at += p.set[i].nb;
    }
    return at;
}

bool streams(const RopeParams& p, bool bf) {
    return p.tokens * (int64_t)(p.set[0].heads + p.set[1].heads) * p.dim * (bf ? 2 : 4) > STREAM_BYTES;
}

template <bool BF, int LP, int HB>
hipError_t forward(RopeParams& p, hipStream_t s) {
    const uint32_t n = set_blocks(p, LP, HB, 0);
    if (!n) return hipSuccess;
    if (!grid_ok(n, RT)) return TOO_LARGE;
    if (streams(p, BF)) k_rope<BF, LP, HB, true><<<n, RT, 0, s>>>(p);
    else k_rope<BF, LP, HB, false><<<n, RT, 0, s>>>(p);
    return hipGetLastError();
}
template <bool BF, int LP, int HB>
hipError_t backward(RopeParams& p, hipStream_t s) {
    const uint32_t n = set_blocks(p, LP, HB, BACK_BLOCKS);
    if (!n) return hipSuccess;
    if (streams(p, BF)) k_rope_back<BF, LP, HB, true><<<n, RT, 0, s>>>(p);
    else k_rope_back<BF, LP, HB, false><<<n, RT, 0, s>>>(p);
    return hipGetLastError();
}
// Heads per lane.  Forward: as many as leave four workgroups for each CU (bf16,
// 40 heads of 128, us with four, two and one: 8192 tokens 37, 40, 43; 2048
// tokens 12.9, 12.0, 13.5; 1 token 5.3, 4.2, 3.5); fp32 two at most (71 against
// 73 with four).  Backward, bf16: two where that still fills the chip (8192
// tokens 60 us against 66 with one; 64 tokens 8.1 against 7.2); fp32 one (two
// spill: 9.7 us against 8.7 for 333 tokens of 16 heads of 96).
template <bool BF, int LP>
hipError_t go(RopeParams& p, bool back, hipStream_t s) {
    auto blocks = [&](int hb) {
        int64_t t = 0;
        for (const RopeSet& S : p.set) t += p.tokens * ((S.heads + hb - 1) / hb);
        return t / (RT / LP);
    };
    if (back) {
        if constexpr (BF)
            if (blocks(2) >= BACK_BLOCKS) return backward<BF, LP, 2>(p, s);
        return backward<BF, LP, 1>(p, s);
    }
    if constexpr (BF)
        if (blocks(4) >= 1024) return forward<BF, LP, 4>(p, s);
    if (blocks(2) >= 1024) return forward<BF, LP, 2>(p, s);
    return forward<BF, LP, 1>(p, s);
}

template <bool BF>
hipError_t pick(RopeParams& p, bool back, hipStream_t s) {
    if (p.dim % 16 || p.rot % 16) {
        const uint32_t n = set_blocks(p, 64, 1, back ? ROPE_PARTS : 1 << 16);
        if (!n) return hipSuccess;
        if (back) k_rope_any<BF, true><<<n, RT, 0, s>>>(p);
        else k_rope_any<BF, false><<<n, RT, 0, s>>>(p);
        return hipGetLastError();
    }
    const int units = p.dim / 16;
    if (units <= 4) return go<BF, 4>(p, back, s);
    if (units <= 8) return go<BF, 8>(p, back, s);
    if (units <= 16) return go<BF, 16>(p, back, s);
    if (units <= 32) return go<BF, 32>(p, back, s);
    return go<BF, 64>(p, back, s);
}

}  // namespace

hipError_t launch_rope(RopeParams p, bool bf16, bool back, hipStream_t s) {
    // each set's weight partials lie after the other's
    p.set[1].parts = p.set[0].parts + (int64_t)ROPE_PARTS * p.dim;
    hipError_t e = bf16 ? pick<true>(p, back, s) : pick<false>(p, back, s);
    if (e != hipSuccess || !back || (!p.set[0].w && !p.set[1].w)) return e;
    k_rope_weights<<<dim3((unsigned)(p.dim / 4), 2), RT, 0, s>>>(p);
    return hipGetLastError();
}

}  // namespace mxk
