// matvec.hip -- y = x . deq(W)^T + bias for a few tokens x (bf16 or fp32) and
// a 4-bit weight W in row blocks.
//
// Mathematics.  A weight is q s (+ o): the code's value q, its block's scale s
// and, for asymmetric blocks, an offset o.  q s is exact in bf16: E2M1 has two
// significant bits, a scale at most four, an INT4 code u = 0 .. 15 four.  INT4
// is taken as u with an offset (the min/max offset, or -8 s for a symmetric
// two's complement nibble, whose u is the nibble with its top bit flipped), and
// sum_k (q s + o) x = sum_k (q s) x + sum_blocks o X, X the block's sum of x.
// The second sum runs on the same matrix instruction, one K position per bf16
// part of X (three parts hold all 24 bits) and block.  An fp32 x is the exact
// sum of three bf16 parts, one product each.
//
// Split.  A workgroup owns 16 rows of W and up to 16 tokens, so each weight is
// read once and nothing is joined between workgroups; its waves share K.  The
// 16 x 16 x 32 bf16 instruction takes W as its 16 rows and x as its 16
// columns: for fewer tokens the other columns repeat the last token and are
// not stored (columns are independent, so they cost nothing but instructions
// that are far from the limit).
// A lane (row r, group g) holds the 32 codes K = k0 + 32 g .. + 31 of a
// 128-wide step as one 16-byte load, and its j-th instruction takes codes 8 j
// .. 8 j + 7 (the order of K inside an instruction is free as long as both
// operands agree).  x is staged in LDS in exactly that order, [step][j][g][token]
// with 16 bytes each.
#include "mx_kernels.hpp"

namespace mxk {
using namespace mxd;

namespace {

typedef __bf16 bf8v __attribute__((ext_vector_type(8)));
typedef __bf16 bf2v __attribute__((ext_vector_type(2)));
typedef float f2v __attribute__((ext_vector_type(2)));
typedef float f4v __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4a4 __attribute__((ext_vector_type(4), aligned(4)));   // rows are 4-byte aligned

constexpr int WAVES = 8, THREADS = 64 * WAVES, ROWS = 16, TOK = 16, STEP = 128;
constexpr size_t LDS_MAX = 64 * 1024;      // two workgroups per CU

__device__ __forceinline__ float mv_scale(uint32_t c, int kind) {
    // E8M0 2^(c - 127); UE4M3 / UE5M3 unsigned minifloats with 3 mantissa bits
    if (kind == SC_E8M0) return c == 255u ? bitsf(0x7fc00000u) : bitsf(c ? c << 23 : 0x00400000u);
    const bool ue5 = kind == SC_UE5M3;
    if (c == (ue5 ? 0xffu : 0x7fu) || c > 0xffu) return bitsf(0x7fc00000u);
    return fp8_value(ue5, (int)c);
}

__device__ __forceinline__ bf8v join4(bf2v a, bf2v b, bf2v c, bf2v d) {
    bf8v v;
    v[0] = a[0]; v[1] = a[1]; v[2] = b[0]; v[3] = b[1];
    v[4] = c[0]; v[5] = c[1]; v[6] = d[0]; v[7] = d[1];
    return v;
}
__device__ __forceinline__ bf2v mul2(f2v q, float s) {
    const f2v p = {q[0] * s, q[1] * s};
    return __builtin_convertvector(p, bf2v);
}

// The eight codes of w times their scale as bf16.  INT4 codes are spread to
// bytes (even codes, then odd ones: x is staged in that order) and go through
// the FP8 converter: the E4M3 code u = 0 .. 15 stands for u 2^-9, so INT4
// results are 2^-9 too small; the caller multiplies its sums by 2^9.
template <bool INT, bool MUL>
__device__ __forceinline__ bf8v decode8w(uint32_t w, float s) {
    if constexpr (INT) {
        const int lo = (int)(w & 0x0f0f0f0fu), hi = (int)((w >> 4) & 0x0f0f0f0fu);
        if constexpr (MUL) {
            return join4(mul2(__builtin_amdgcn_cvt_scalef32_pk_f32_fp8(lo, 1.0f, false), s),
                         mul2(__builtin_amdgcn_cvt_scalef32_pk_f32_fp8(lo, 1.0f, true), s),
                         mul2(__builtin_amdgcn_cvt_scalef32_pk_f32_fp8(hi, 1.0f, false), s),
                         mul2(__builtin_amdgcn_cvt_scalef32_pk_f32_fp8(hi, 1.0f, true), s));
        } else {
            return join4(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, s, false),
                         __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, s, true),
                         __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, s, false),
                         __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, s, true));
        }
    } else if constexpr (MUL) {
        return join4(mul2(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0), s),
                     mul2(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1), s),
                     mul2(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2), s),
                     mul2(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3), s));
    } else {
        return join4(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0), __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1),
                     __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2), __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3));
    }
}

// x = h + m + l, each a bf16 (truncated, so that no part overflows): exact.
// Inf keeps zero lower parts, NaN stays NaN.
__device__ __forceinline__ void split3(float x, uint16_t& h, uint16_t& m, uint16_t& l) {
    const uint32_t u = fbits(x);
    if ((u & 0x7f800000u) == 0x7f800000u) {
        h = bf16_rne(x);
        m = l = 0;
        return;
    }
    const float r = x - bitsf(u & 0xffff0000u);
    const uint32_t v = fbits(r);
    h = (uint16_t)(u >> 16);
    m = (uint16_t)(v >> 16);
    l = (uint16_t)(fbits(r - bitsf(v & 0xffff0000u)) >> 16);
}

// LDS of one chunk of kc values of K: XP parts of x, 16 bytes per 8 values and
// token, then with offsets the three parts of each sub-block's sum, 8 bytes
size_t chunk_bytes(int64_t kc, int toks, int xp, bool off, int nsb) {
    return (size_t)(kc / 8) * toks * 16 * xp + (off ? (size_t)(kc / 32) * nsb * toks * 8 : 0);
}

template <bool INT, bool MUL, bool OFF, int NSB, int XP>
__global__ __launch_bounds__(THREADS) void k_matvec(MatvecParams p) {
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    constexpr int SB = 32 / NSB;                 // codes per scale inside a lane's 32
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, g = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * ROWS, t0 = (int64_t)blockIdx.y * TOK;
    const int toks = (int)(p.tokens - t0 < TOK ? p.tokens - t0 : TOK);
    const int64_t row = n0 + r < p.n ? n0 + r : p.n - 1;
    const int K = (int)p.k;
    const uint8_t* wrow = p.codes + row * (p.k / 2);
    const int64_t srow = row * (p.k / p.bc);
    const int tl = r < toks ? r : toks - 1;      // the token this lane's B operand holds

    f4v acc = {0.f, 0.f, 0.f, 0.f};
    for (int c0 = 0; c0 < K; c0 += p.kc) {
        const int kc = K - c0 < p.kc ? (K - c0 + STEP - 1) / STEP * STEP : p.kc;
        __syncthreads();
        // stage x[t][c0 .. c0 + kc): eight values a thread
        uint8_t* sums = smem + (size_t)(p.kc / 8) * toks * 16 * XP;
        for (int i = threadIdx.x; i < (kc / 8) * toks; i += THREADS) {
            const int t = i / (kc / 8), u = i - t * (kc / 8), k = c0 + 8 * u;
            float f[8];
            if (k < K) {
                if (p.x_bf16) {
                    const u32x4 v = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p.x) + (t0 + t) * p.ldx + k);
#pragma unroll
                    for (int e = 0; e < 4; e++) { f[2 * e] = bf16lo(v[e]); f[2 * e + 1] = bf16hi(v[e]); }
                } else {
                    const float4* src = reinterpret_cast<const float4*>(static_cast<const float*>(p.x) + (t0 + t) * p.ldx + k);
                    const float4 a = src[0], b = src[1];
                    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w; f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; e++) f[e] = 0.f;
            }
            const int step = u / 16, gg = (u % 16) / 4, j = u % 4;
#pragma unroll
            for (int part = 0; part < XP; part++) {
                uint32_t o[4];
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    // INT4 decodes the even codes first
                    const float a = INT ? f[e < 2 ? 4 * e : 4 * e - 7] : f[2 * e];
                    const float b = INT ? f[e < 2 ? 4 * e + 2 : 4 * e - 5] : f[2 * e + 1];
                    uint16_t ha, ma, la, hb, mb, lb;
                    if constexpr (XP == 1) {
                        o[e] = (fbits(a) >> 16) | (fbits(b) & 0xffff0000u);
                    } else {
                        split3(a, ha, ma, la);
                        split3(b, hb, mb, lb);
                        o[e] = part == 0 ? ha | (uint32_t)hb << 16 : part == 1 ? ma | (uint32_t)mb << 16 : la | (uint32_t)lb << 16;
                    }
                }
                uint8_t* dst = smem + ((size_t)part * (p.kc / 8) * toks + (size_t)(((step * 4 + j) * 4 + gg) * toks + t)) * 16;
                *reinterpret_cast<uint4*>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
            }
        }
        if constexpr (OFF) {
            // the sum of x over each sub-block, in three parts
            const int per = kc / SB;
            for (int i = threadIdx.x; i < per * toks; i += THREADS) {
                const int t = i / per, u = i - t * per, k = c0 + SB * u;
                float X = 0.f;
                for (int e = 0; e < SB && k + e < K; e++)
                    X += p.x_bf16 ? bf16f(static_cast<const uint16_t*>(p.x)[(t0 + t) * p.ldx + k + e])
                                  : static_cast<const float*>(p.x)[(t0 + t) * p.ldx + k + e];
                uint16_t h, m, l;
                split3(X, h, m, l);
                const int step = u / (4 * NSB), gg = (u / NSB) % 4, sb = u % NSB;
                *reinterpret_cast<uint2*>(sums + (size_t)(((step * 4 + gg) * toks + t) * NSB + sb) * 8) =
                    make_uint2(h | (uint32_t)m << 16, l);
            }
        }
        __syncthreads();

        for (int step = wave; step < kc / STEP; step += WAVES) {
            const int kb = c0 + step * STEP + 32 * g;       // this lane's first code
            uint32_t w[4] = {0u, 0u, 0u, 0u};
            if (kb + 32 <= K) {
                const u32x4a4 v = *reinterpret_cast<const u32x4a4*>(wrow + kb / 2);
#pragma unroll
                for (int j = 0; j < 4; j++) w[j] = v[j];
            } else {
#pragma unroll
                for (int j = 0; j < 4; j++)
                    if (kb + 8 * j < K) w[j] = *reinterpret_cast<const uint32_t*>(wrow + kb / 2 + 4 * j);
            }
            float s[NSB];
            uint32_t off[NSB];
#pragma unroll
            for (int b = 0; b < NSB; b++) {
                const int k = kb + SB * b;
                s[b] = 1.0f;
                off[b] = 0;
                if (k >= K) continue;
                const int blk = k / p.bc;
                s[b] = mv_scale(p.scales[srow + blk], p.scale);
                if (MUL && p.macro) s[b] *= mv_scale(p.macro[row * (p.k / 128) + k / 128], SC_UE4M3);
                if constexpr (OFF) {
                    // a power of two times a bf16: exact (INT4 sums are 2^-9 too small)
                    const float o = p.offsets ? bf16f(p.offsets[srow + blk]) * (INT ? 0x1p-9f : 1.0f) : s[b] * -0x1p-6f;
                    off[b] = fbits(o) >> 16;
                }
            }
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const bf8v a = decode8w<INT, MUL>(INT && !p.offsets ? w[j] ^ 0x88888888u : w[j], s[j * NSB / 4]);
#pragma unroll
                for (int part = 0; part < XP; part++) {
                    const bf8v b = *reinterpret_cast<const bf8v*>(
                        smem + ((size_t)part * (p.kc / 8) * toks + (size_t)(((step * 4 + j) * 4 + g) * toks + tl)) * 16);
                    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, acc, 0, 0, 0);
                }
            }
            if constexpr (OFF) {
                // o X: o in the first three of four K positions per sub-block
#pragma unroll
                for (int b = 0; b < NSB; b += 2) {
                    uint32_t ao[4], bo[4] = {0u, 0u, 0u, 0u};
                    const uint2* src = reinterpret_cast<const uint2*>(sums + (size_t)(((step * 4 + g) * toks + tl) * NSB + b) * 8);
                    const uint2 x0 = src[0];
                    bo[0] = x0.x; bo[1] = x0.y;
                    ao[0] = off[b] | off[b] << 16; ao[1] = off[b]; ao[2] = ao[3] = 0u;
                    if constexpr (NSB > 1) {
                        const uint2 x1 = src[1];
                        bo[2] = x1.x; bo[3] = x1.y;
                        ao[2] = off[b + 1] | off[b + 1] << 16; ao[3] = off[b + 1];
                    }
                    bf8v av, bv;
                    __builtin_memcpy(&av, ao, 16);
                    __builtin_memcpy(&bv, bo, 16);
                    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av, bv, acc, 0, 0, 0);
                }
            }
        }
    }

    // the waves' sums, added in wave order
    __syncthreads();
    float* red = reinterpret_cast<float*>(smem);
    *reinterpret_cast<f4v*>(red + wave * 256 + r * 16 + 4 * g) = acc;      // [token r][row 4 g ..]
    __syncthreads();
    const int t = threadIdx.x >> 4, i = threadIdx.x & 15;
    if (t < toks && n0 + i < p.n) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < WAVES; w++) v += red[w * 256 + t * 16 + i];
        if constexpr (INT) v *= 512.0f;
        if (p.tensor_scale) v *= *p.tensor_scale;
        if (p.bias) v += p.x_bf16 ? bf16f(static_cast<const uint16_t*>(p.bias)[n0 + i]) : static_cast<const float*>(p.bias)[n0 + i];
        const int64_t at = (t0 + t) * p.ldy + n0 + i;
        if (p.y_bf16) static_cast<uint16_t*>(p.y)[at] = bf16_rne(v);
        else static_cast<float*>(p.y)[at] = v;
    }
}

template <bool INT, bool MUL, bool OFF, int NSB, int XP>
hipError_t go(MatvecParams& p, hipStream_t s) {
    const int toks = (int)(p.tokens < TOK ? p.tokens : TOK);
    const int64_t unit = (int64_t)STEP * WAVES, kall = (p.k + STEP - 1) / STEP * STEP;
    int64_t kc = LDS_MAX / chunk_bytes(unit, toks, XP, OFF, NSB) * unit;   // one unit is at most 96 KiB + sums
    if (kc < unit) kc = unit;
    p.kc = (int)(kc < kall ? kc : kall);
    size_t lds = chunk_bytes(p.kc, toks, XP, OFF, NSB);
    if (lds < WAVES * 256 * sizeof(float)) lds = WAVES * 256 * sizeof(float);
    if (lds > LDS_MAX) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(k_matvec<INT, MUL, OFF, NSB, XP>),
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
        if (e != hipSuccess) return e;
    }
    const dim3 grid((unsigned)((p.n + ROWS - 1) / ROWS), (unsigned)((p.tokens + TOK - 1) / TOK));
    k_matvec<INT, MUL, OFF, NSB, XP><<<grid, THREADS, lds, s>>>(p);
    return hipGetLastError();
}

template <bool INT, bool MUL, bool OFF>
hipError_t pick(MatvecParams& p, hipStream_t s) {
    if (p.x_bf16) return p.bc >= 32 ? go<INT, MUL, OFF, 1, 1>(p, s) : p.bc == 16 ? go<INT, MUL, OFF, 2, 1>(p, s) : go<INT, MUL, OFF, 4, 1>(p, s);
    return p.bc >= 32 ? go<INT, MUL, OFF, 1, 3>(p, s) : p.bc == 16 ? go<INT, MUL, OFF, 2, 3>(p, s) : go<INT, MUL, OFF, 4, 3>(p, s);
}

}  // namespace

hipError_t launch_matvec(MatvecParams p, hipStream_t s) {
    const bool mul = p.scale != SC_E8M0 || p.macro;
    if (p.elem == INT4) return mul ? pick<true, true, true>(p, s) : pick<true, false, true>(p, s);
    if (p.offsets) return pick<false, false, true>(p, s);
    return mul ? pick<false, true, false>(p, s) : pick<false, false, false>(p, s);
}

}  // namespace mxk
