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
#include "mx_kernels.hpp"

namespace mxk {
using namespace mxd;

namespace {

constexpr int RT = 256;               // threads per workgroup

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
template <bool BF>
__device__ __forceinline__ void store8(const float* f, void* base, int64_t at) {
    if constexpr (BF) {
        u32x4 v;
#pragma unroll
        for (int e = 0; e < 4; e++) v[e] = (uint32_t)bf16_rne(f[2 * e]) | (uint32_t)bf16_rne(f[2 * e + 1]) << 16;
        *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(base) + at) = v;
    } else {
        float4* d = reinterpret_cast<float4*>(static_cast<float*>(base) + at);
        d[0] = make_float4(f[0], f[1], f[2], f[3]);
        d[1] = make_float4(f[4], f[5], f[6], f[7]);
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
    if (pos >= 0 && (int64_t)pos < p.table_rows) {
        const int64_t at = (int64_t)pos * (p.rot / 2) + i0;
        load8<false>(c, p.cos, at);
        load8<false>(s, p.sin, at);
    } else {
#pragma unroll
        for (int i = 0; i < 8; i++) c[i] = s[i] = bitsf(0x7fc00000u);
    }
}

// One set (queries or keys) of this launch: workgroups [b0, b0 + nb) take it.
// LP lanes a head, HB heads of one token a lane.  dim and rot multiples of 16.
template <bool BF, int LP, int HB>
__global__ __launch_bounds__(RT) void k_rope(RopeParams p) {
    const RopeSet& S = p.set[blockIdx.x < p.set[0].nb ? 0 : 1];
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
            store8<BF>(v[h], S.y, at + a);
            store8<BF>(v[h] + 8, S.y, at + b);
        }
    }
}

// Backward: the same lanes and chunks; a workgroup walks over its share of the
// set's tokens and keeps the weight gradient of its lanes in registers, joins
// them over its lanes in a fixed order and writes one partial row.
template <bool BF, int LP, int HB>
__global__ __launch_bounds__(RT) void k_rope_back(RopeParams p) {
    __shared__ float sh[RT / 64][16 * LP];
    const RopeSet& S = p.set[blockIdx.x < p.set[0].nb ? 0 : 1];
    const uint32_t block = blockIdx.x - S.b0;
    const int u = threadIdx.x % LP;
    const uint32_t groups = (S.heads + HB - 1) / HB;
    const uint32_t slots = (uint32_t)p.tokens * groups, stride = S.nb * (RT / LP);
    const bool live = u < p.dim / 16, turns = u < p.rot / 16;
    const int a = turns && !p.adjacent ? 8 * u : 16 * u;
    const int b = turns && !p.adjacent ? p.rot / 2 + 8 * u : 16 * u + 8;

    float w[16], dw[16];
#pragma unroll
    for (int e = 0; e < 16; e++) { w[e] = 0.f; dw[e] = 0.f; }
    if (S.w && live) load_w(w, S.w, p.w_bf16, a, b);

    for (uint32_t slot = block * (RT / LP) + threadIdx.x / LP; slot < slots; slot += stride) {
        const uint32_t token = slot / groups, h0 = (slot - token * groups) * HB;
        float x[HB][16], g[HB][16];
#pragma unroll
        for (int h = 0; h < HB; h++) {
            const uint32_t hh = h0 + h < S.heads ? h0 + h : S.heads - 1;
            if (live) {
                const int64_t ax = (int64_t)token * S.x_ts + (int64_t)hh * S.x_hs;
                const int64_t ag = (int64_t)token * S.g_ts + (int64_t)hh * S.g_hs;
                load8<BF>(g[h], S.g, ag + a);
                load8<BF>(g[h] + 8, S.g, ag + b);
                if (S.w) {
                    load8<BF>(x[h], S.x, ax + a);
                    load8<BF>(x[h] + 8, S.x, ax + b);
                }
            } else {
#pragma unroll
                for (int e = 0; e < 16; e++) { x[h][e] = 0.f; g[h][e] = 0.f; }
            }
        }
        if (turns) {
            float c[8], s[8];
            load_turn(p, token, 8 * u, c, s);
#pragma unroll
            for (int h = 0; h < HB; h++) turn<-1>(g[h], c, s, p.adjacent);
        }
        if (S.w) {
#pragma unroll
            for (int h = 0; h < HB; h++) {
                const bool own = h0 + h < S.heads;        // not the repeated last head
                float q = 0.f, m = 0.f;
#pragma unroll
                for (int e = 0; e < 16; e++) {
                    q += x[h][e] * x[h][e];
                    m += g[h][e] * w[e] * x[h][e];
                }
                const float rstd = 1.0f / sqrtf(group_sum<LP>(q) / (float)p.dim + p.eps);
                m = group_sum<LP>(m) / (float)p.dim * rstd;      // mean of h n
#pragma unroll
                for (int e = 0; e < 16; e++) {
                    const float n = x[h][e] * rstd;
                    if (own) dw[e] += g[h][e] * n;
                    g[h][e] = rstd * (g[h][e] * w[e] - n * m);
                }
            }
        }
        if (live) {
#pragma unroll
            for (int h = 0; h < HB; h++) {
                if (h0 + h >= S.heads) break;
                const int64_t at = (int64_t)token * S.y_ts + (int64_t)(h0 + h) * S.y_hs;
                store8<BF>(g[h], S.y, at + a);
                store8<BF>(g[h] + 8, S.y, at + b);
            }
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
    const RopeSet& S = p.set[blockIdx.x < p.set[0].nb ? 0 : 1];
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

// The partial rows of a set added up: 16 values a workgroup, 16 threads each
__global__ __launch_bounds__(RT) void k_rope_weights(RopeParams p) {
    __shared__ float sh[16][17];
    const RopeSet& S = p.set[blockIdx.y];
    if (!S.w) return;
    const int e = threadIdx.x % 16, k = threadIdx.x / 16, i = blockIdx.x * 16 + e;
    float t = 0.f;
    if (i < p.dim)
        for (uint32_t b = k; b < S.nb; b += 16) t += S.parts[(int64_t)b * p.dim + i];
    sh[k][e] = t;
    __syncthreads();
    if (k == 0 && i < p.dim) {
        t = 0.f;
#pragma unroll
        for (int j = 0; j < 16; j++) t += sh[j][e];
        S.dw[i] = t;
    }
}

// workgroups of each set: one per RT / LP slots, at most `cap`
uint32_t set_blocks(RopeParams& p, int lp, int hb, int64_t cap) {
    uint32_t at = 0;
    for (int i = 0; i < 2; i++) {
        RopeSet& S = p.set[i];
        int64_t n = 0;
        if (S.heads) {
            n = (p.tokens * ((S.heads + hb - 1) / hb) + RT / lp - 1) / (RT / lp);
            if (cap && n > cap) n = cap;
        }
        S.b0 = at;
        S.nb = (uint32_t)n;
        at += (uint32_t)n;
    }
    return at;
}

template <bool BF, int LP, int HB>
hipError_t go(RopeParams& p, bool back, hipStream_t s) {
    const uint32_t n = set_blocks(p, LP, HB, back ? ROPE_PARTS : 0);
    if (!n) return hipSuccess;
    if (back) k_rope_back<BF, LP, HB><<<n, RT, 0, s>>>(p);
    else k_rope<BF, LP, HB><<<n, RT, 0, s>>>(p);
    return hipGetLastError();
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
    if (units <= 4) return go<BF, 4, 2>(p, back, s);
    if (units <= 8) return go<BF, 8, 2>(p, back, s);
    if (units <= 16) return go<BF, 16, 2>(p, back, s);
    if (units <= 32) return go<BF, 32, 1>(p, back, s);
    return go<BF, 64, 1>(p, back, s);
}

}  // namespace

hipError_t launch_rope(RopeParams p, bool bf16, bool back, hipStream_t s) {
    // each set's weight partials lie after the other's
    p.set[1].parts = p.set[0].parts + (int64_t)ROPE_PARTS * p.dim;
    hipError_t e = bf16 ? pick<true>(p, back, s) : pick<false>(p, back, s);
    if (e != hipSuccess || !back || (!p.set[0].w && !p.set[1].w)) return e;
    k_rope_weights<<<dim3((unsigned)((p.dim + 15) / 16), 2), RT, 0, s>>>(p);
    return hipGetLastError();
}

}  // namespace mxk
