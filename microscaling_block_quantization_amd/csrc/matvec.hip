// matvec.hip -- y = x . deq(W)^T + bias for a few tokens x (bf16 or fp32) and
// a 4-bit weight W in row blocks.
//
// Mathematics.  A weight is q s (+ o): the code's value q, its block's scale s
// and, for asymmetric blocks, an offset o.  q s is exact in bf16 (down to its
// smallest step, 2^-133; 2^-129 for INT4, see decode8w): E2M1 has two
// significant bits, a scale at most four, an INT4 code u = 0 .. 15 four.  INT4
// is taken as u with an offset (the min/max offset, or -8 s for a symmetric
// two's complement nibble, whose u is the nibble with its top bit flipped), and
// sum_k (q s + o) x = sum_k (q s) x + sum_blocks o X, X the block's sum of x.
// The second sum runs on the same matrix instruction, one K position per bf16
// part of X (three parts hold all 24 bits) and block.  An fp32 x is the exact
// sum of three bf16 parts, one product each (what of it lies below 2^-133 is
// not: parts are bf16 numbers).  A symmetric INT4 block's terms are u s x and
// -8 s X, so its rounding goes by those and not by q s x.
//
// The 16 x 16 x 32 bf16 instruction takes W as its 16 rows and x as its 16
// columns: for fewer tokens the other columns repeat the last token and are
// not stored (columns are independent, so they cost nothing but instructions
// that are far from the limit).  A lane (row or token r, group g) holds the 32
// values K = k0 + 32 g .. + 31 of a 128-wide step: of W one 16-byte load, whose
// codes share their scales, of x the four operands of the step's instructions
// as loaded, instruction j taking values 8 j .. 8 j + 7 (the order of K inside
// an instruction is free as long as both operands agree).  A sub-block's sum X
// is then a sum of the lane's own values, and nothing passes through LDS until
// the waves' sums are added, in their order, at the end.
//
// Bound.  Each weight is used once: memory.  Two splits, both with all of K in
// one workgroup, so that nothing is joined between workgroups:
//  - k_tall (K of at least one span per wave): each wave keeps one span of K, its x
//    in registers, and goes down the workgroup's rows, so the loop loads codes
//    and scales alone.  x from L2 or LDS in the loop instead costs four loads
//    per load of codes, and the scales of one step at a time touch as many
//    lines as the codes: hence spans of several steps, whose scales are one
//    load, dealt to the steps by lane exchanges.
//  - k_short: the waves take every eighth step of K, x loaded with the codes.
// A launch that touches almost nothing takes 3.1 us (16 x 1000 x 1008) to 4.3
// (1 x 1024 x 4096): the chain of first loads, x, codes, sums.  Above that the
// codes stream: MXFP4 1 x 14336 x 4096 10.3 us (3.0 TB/s), 1 x 28672 x 8192 31.3
// (4.0); NVFP4 16 x 28672 x 8192 39.9 (3.3), where its exact fp32 decode (16
// vector operations per 8 codes) is half the vector unit's time.  Loading the
// same bytes alone takes 25 us.  Tried: x through LDS in chunks 58 us, x loaded
// per step 52 to 83, sixteen waves 42, codes two tiles ahead 42.  The next
// pass's x and codes under this pass's last tile: 12.3 us against 12.6 at MXFP4
// 1 x 4096 x 14336, and fp32 tokens out of registers.  fp32 tokens take 17.6 us at
// MXFP4 1 x 14336 x 4096; their three parts side by side in the columns instead of
// in three products: 20.9 against 18.2 for five tokens, 48 against 52 for NVFP4
// 2 x 28672 x 8192.
#include <type_traits>

#include "decode_kernels.hpp"

namespace mxk {
using namespace mxd;

namespace {

typedef __bf16 bf8v __attribute__((ext_vector_type(8)));
typedef __bf16 bf2v __attribute__((ext_vector_type(2)));
typedef float f2v __attribute__((ext_vector_type(2)));
typedef float f4v __attribute__((ext_vector_type(4)));
typedef __amdgpu_buffer_rsrc_t rsrc_t;

constexpr int TOK = 16, STEP = 128;

// Value of a scale code: E8M0 is 2^(c - 127); UE4M3 and UE5M3, unsigned
// minifloats with three mantissa bits, are the code as the top of an fp32's
// exponent and mantissa (subnormals included) times 2^(127 - bias).
struct ScaleDec {
    float mul;          // 2^(127 - bias); 0: E8M0
    uint32_t nan;       // the code that means NaN
};
__device__ __forceinline__ float mv_scale(uint32_t c, ScaleDec d) {
    const float v = d.mul == 0.f ? bitsf(c ? c << 23 : 0x00400000u) : bitsf(c << 20) * d.mul;
    return c == d.nan ? bitsf(0x7fc00000u) : v;
}

// A buffer of `left` bytes at p: loads take a lane's byte offset and a uniform
// one, so a load costs no address arithmetic per lane, and a load past the end
// gives zero.
__device__ __forceinline__ rsrc_t mv_buf(const void* p, int64_t left) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, (int)(left < 0x7fffffff ? left : 0x7fffffff), 0x00020000);
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
// the FP8 converter: the E4M3 code u = 0 .. 15 stands for u 2^-9.  INT4 results
// are held 2^-4 too small and the sums multiplied by 2^4 at the end: u s 2^-4
// is exact in bf16 at the smallest E8M0 scale (2^-131 is four of its smallest
// steps) and stays finite at the largest.  s here is what the converter takes,
// 2^5 of the scale for INT4 without MUL.
constexpr float INT_DOWN = 0x1p-4f, INT_CVT = 0x1p5f;
template <bool INT, bool MUL>
__device__ __forceinline__ bf8v decode8w(uint32_t w, float s) {
    if constexpr (INT) {
        const int lo = (int)(w & 0x0f0f0f0fu), hi = (int)((w >> 4) & 0x0f0f0f0fu);
        if constexpr (MUL) {
            return join4(mul2(__builtin_amdgcn_cvt_scalef32_pk_f32_fp8(lo, INT_CVT, false), s),
                         mul2(__builtin_amdgcn_cvt_scalef32_pk_f32_fp8(lo, INT_CVT, true), s),
                         mul2(__builtin_amdgcn_cvt_scalef32_pk_f32_fp8(hi, INT_CVT, false), s),
                         mul2(__builtin_amdgcn_cvt_scalef32_pk_f32_fp8(hi, INT_CVT, true), s));
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

// Block widths: 64 and wider, 32, 16, 8
enum { B_WIDE = 0, B_32 = 1, B_16 = 2, B_8 = 4 };
constexpr int scales_of(int bk) { return bk == B_WIDE ? 1 : bk; }    // scales of a lane's 32 codes

// A step of x as the instructions' columns, in the order the codes are decoded
// in, and the sums of its sub-blocks in three bf16 parts.
template <bool OFF, int BK, int XP>
struct Cols {
    bf8v b[4][XP];
    uint32_t sum[OFF ? scales_of(BK) : 1][2];
};
// v: the 32 values as loaded.  Beside INT4's given offsets, which enter as they
// are, the sums carry the operands' 2^-4.
template <bool INT, bool OFF, int BK, int XP>
__device__ __forceinline__ void make_cols(Cols<OFF, BK, XP>& c, const u32x4 (&v)[4][XP == 1 ? 1 : 2], bool offsets) {
    constexpr int NSB = scales_of(BK);
    float X[NSB];
#pragma unroll
    for (int b = 0; b < NSB; b++) X[b] = 0.f;
#pragma unroll
    for (int j = 0; j < 4; j++) {
        uint32_t o[XP][4];
        if constexpr (XP == 1) {
            const u32x4 w = v[j][0];
            if constexpr (OFF) {
#pragma unroll
                for (int e = 0; e < 4; e++) X[j * NSB / 4] += bf16lo(w[e]) + bf16hi(w[e]);
            }
            if constexpr (INT) {                              // even values, then odd ones
                o[0][0] = __builtin_amdgcn_perm(w[1], w[0], 0x05040100u);
                o[0][1] = __builtin_amdgcn_perm(w[3], w[2], 0x05040100u);
                o[0][2] = __builtin_amdgcn_perm(w[1], w[0], 0x07060302u);
                o[0][3] = __builtin_amdgcn_perm(w[3], w[2], 0x07060302u);
            } else {
                o[0][0] = w[0]; o[0][1] = w[1]; o[0][2] = w[2]; o[0][3] = w[3];
            }
        } else {
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; e++) f[e] = bitsf(v[j][XP == 1 ? 0 : e / 4][e & 3]);
            if constexpr (OFF) X[j * NSB / 4] += ((f[0] + f[1]) + (f[2] + f[3])) + ((f[4] + f[5]) + (f[6] + f[7]));
#pragma unroll
            for (int e = 0; e < 4; e++) {
                uint16_t ha, ma, la, hb, mb, lb;
                split3(INT ? f[e < 2 ? 4 * e : 4 * e - 7] : f[2 * e], ha, ma, la);
                split3(INT ? f[e < 2 ? 4 * e + 2 : 4 * e - 5] : f[2 * e + 1], hb, mb, lb);
                o[0][e] = ha | (uint32_t)hb << 16;
                o[XP - 2][e] = ma | (uint32_t)mb << 16;
                o[XP - 1][e] = la | (uint32_t)lb << 16;
            }
        }
#pragma unroll
        for (int part = 0; part < XP; part++) __builtin_memcpy(&c.b[j][part], o[part], 16);
    }
    if constexpr (OFF) {
#pragma unroll
        for (int b = 0; b < NSB; b++) {
            uint16_t h, m, l;
            split3(INT && offsets ? X[b] * INT_DOWN : X[b], h, m, l);
            c.sum[b][0] = h | (uint32_t)m << 16;
            c.sum[b][1] = l;
        }
    }
}

// What a lane's 32 codes have beside them: NSB scale bytes, the macro scale,
// bf16 offsets
template <bool OFF, int BK>
struct Side {
    uint32_t sc, mac;
    uint32_t off[OFF ? scales_of(BK) : 1];
};

// Not 0 where a scale byte holds a code of 248 or more (its upper five bits are
// all set): from code 250 on the converter's 2^5 s overflows, and INT4 codes go
// through fp32.
__device__ __forceinline__ uint32_t far_codes(uint32_t sc) {
    const uint32_t low = ~sc & 0xf8f8f8f8u;
    return (low - 0x01010101u) & ~low & 0x80808080u;
}

// acc += codes . x of one step.  far: whether a lane's step has such a scale,
// or 2 to look; the seldom path (FAR) is kept from spreading over the other's
// registers.
template <bool INT, bool MUL, bool OFF, int BK, int XP, bool FAR = false>
__device__ __forceinline__ void step_product(f4v& acc, u32x4 w, const Side<OFF, BK>& sd, const Cols<OFF, BK, XP>& x, ScaleDec dec,
                                             bool macro, bool offsets, int far = 2) {
    constexpr int NSB = scales_of(BK);
    constexpr bool CVT = INT && !MUL;
    if constexpr (CVT) {
        const uint32_t low = ~sd.sc & 0xf8f8f8f8u;
        if (far == 2 ? __any((low - 0x01010101u) & ~low & 0x80808080u) : far) {
            // as other values, so that none of this is formed before the branch
            Side<OFF, BK> d = sd;
            asm volatile("" : "+v"(w), "+v"(d.sc));
            step_product<INT, true, OFF, BK, XP, true>(acc, w, d, x, dec, false, offsets);
            return;
        }
    }
    float s[NSB];
    uint32_t off[NSB];
#pragma unroll
    for (int b = 0; b < NSB; b++) {
        const uint32_t code = (sd.sc >> (8 * b)) & 0xffu;
        s[b] = CVT ? bitsf((code + 5) << 23) : mv_scale(code, dec);      // CVT: 2^5 s, of code 0 too, and no NaN
        if (MUL && macro) s[b] *= mv_scale(sd.mac, ScaleDec{0x1p120f, 0x7fu});
        // -8 s 2^-4: a scale's four bits at most, exact in bf16
        if constexpr (OFF) off[b] = offsets ? sd.off[b] : fbits(s[b] * (-8.0f * INT_DOWN / (CVT ? INT_CVT : 1.0f))) >> 16;
    }
#pragma unroll
    for (int j = 0; j < 4; j++) {
        const uint32_t c = w[j];
        const bf8v a = decode8w<INT, MUL>(INT && !offsets ? c ^ 0x88888888u : c, s[j * NSB / 4]);
#pragma unroll
        for (int part = 0; part < XP; part++) acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, x.b[j][part], acc, 0, 0, 0);
        if (FAR) __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (OFF) {
        // o X: o in the first three of four K positions per sub-block
#pragma unroll
        for (int b = 0; b < NSB; b += 2) {
            uint32_t ao[4] = {off[b] | off[b] << 16, off[b], 0u, 0u}, xo[4] = {x.sum[b][0], x.sum[b][1], 0u, 0u};
            if constexpr (NSB > 1) {
                ao[2] = off[b + 1] | off[b + 1] << 16;
                ao[3] = off[b + 1];
                xo[2] = x.sum[b + 1][0];
                xo[3] = x.sum[b + 1][1];
            }
            bf8v av, xv;
            __builtin_memcpy(&av, ao, 16);
            __builtin_memcpy(&xv, xo, 16);
            acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av, xv, acc, 0, 0, 0);
        }
    }
}

// The rows of W a workgroup works on and this lane's place in them.
struct Rows {
    rsrc_t w, s, o, m;             // codes, scales, offsets, macro scales from row n0 on
    int rows, cb, sr, mb;          // rows left; row bytes of codes, scales and macro scales
};
__device__ __forceinline__ Rows rows_at(const MatvecParams& p, int64_t n0, int most) {
    const int64_t cb = p.k / 2, sr = p.k >> p.lgb, mb = p.k / 128;
    Rows R;
    R.rows = (int)(p.n - n0 < most ? p.n - n0 : most);
    R.cb = (int)cb;
    R.sr = (int)sr;
    R.mb = (int)mb;
    R.w = mv_buf(p.codes + n0 * cb, R.rows * cb);
    R.s = mv_buf(p.scales + n0 * sr, R.rows * sr);
    R.o = mv_buf(p.offsets ? p.offsets + n0 * sr : nullptr, p.offsets ? R.rows * sr * 2 : 0);
    R.m = mv_buf(p.macro ? p.macro + n0 * mb : nullptr, p.macro ? R.rows * mb : 0);
    return R;
}

// scales and offsets of row rr at one whole step
template <bool MUL, bool OFF, int BK>
__device__ __forceinline__ void load_side(Side<OFF, BK>& d, const Rows& R, int rr, int k0, int g, int lgb) {
    constexpr int NSB = scales_of(BK);
    const int ks = k0 >> lgb, v = rr * R.sr + (32 * g >> lgb);
    if constexpr (NSB == 1) d.sc = __builtin_amdgcn_raw_buffer_load_b8(R.s, v, ks, 0);
    else if constexpr (NSB == 2) d.sc = __builtin_amdgcn_raw_buffer_load_b16(R.s, v, ks, 0);
    else d.sc = __builtin_amdgcn_raw_buffer_load_b32(R.s, v, ks, 0);
    if constexpr (OFF) {
#pragma unroll
        for (int b = 0; b < NSB; b++) d.off[b] = __builtin_amdgcn_raw_buffer_load_b16(R.o, 2 * v + 2 * b, 2 * ks, 0);
    }
    if constexpr (MUL) d.mac = __builtin_amdgcn_raw_buffer_load_b8(R.m, rr * R.mb, k0 >> 7, 0);      // 0 without macro scales
}
// codes, scales and offsets of row rr at the end of K: what lies in it, eight
// values at a time
template <bool OFF, int BK>
__device__ __forceinline__ void load_end(u32x4& w, Side<OFF, BK>& d, const Rows& R, int rr, int k0, int left, int g, int lgb) {
    constexpr int NSB = scales_of(BK), SB = 32 / NSB;
    const int ks = k0 >> lgb, v = rr * R.sr + (32 * g >> lgb), vw = rr * R.cb + 16 * g;
#pragma unroll
    for (int j = 0; j < 4; j++) w[j] = left > 8 * j ? __builtin_amdgcn_raw_buffer_load_b32(R.w, vw + 4 * j, k0 >> 1, 0) : 0u;
    d.sc = 0;                                                 // which no format reads as NaN
    d.mac = 0;                                                // K is whole macro blocks where there are any
#pragma unroll
    for (int b = 0; b < NSB; b++) {
        const bool in = left > SB * b;
        d.sc |= (in ? (uint32_t)__builtin_amdgcn_raw_buffer_load_b8(R.s, v + b, ks, 0) : 0u) << (8 * b);
        if constexpr (OFF) d.off[b] = in ? __builtin_amdgcn_raw_buffer_load_b16(R.o, 2 * v + 2 * b, 2 * ks, 0) : 0;
    }
}

// a lane's 32 values of x at k0 (xrow: its token's values from 32 g on), and at
// the end of K
template <int XP>
__device__ __forceinline__ void load_x(u32x4 (&v)[4][XP == 1 ? 1 : 2], const char* xrow, int64_t k0) {
    const u32x4* x = reinterpret_cast<const u32x4*>(xrow + k0 * (XP == 1 ? 2 : 4));
#pragma unroll
    for (int j = 0; j < 4; j++)
#pragma unroll
        for (int h = 0; h < (XP == 1 ? 1 : 2); h++) v[j][h] = x[XP == 1 ? j : 2 * j + h];
}
template <int XP>
__device__ __forceinline__ void load_x_end(u32x4 (&v)[4][XP == 1 ? 1 : 2], const char* xrow, int64_t k0, int left) {
    const u32x4* x = reinterpret_cast<const u32x4*>(xrow + k0 * (XP == 1 ? 2 : 4));
#pragma unroll
    for (int j = 0; j < 4; j++)
#pragma unroll
        for (int h = 0; h < (XP == 1 ? 1 : 2); h++) v[j][h] = left > 8 * j ? x[XP == 1 ? j : 2 * j + h] : u32x4{0u, 0u, 0u, 0u};
}
template <int XP>
__device__ __forceinline__ const char* x_row(const MatvecParams& p, int64_t t0, int toks, int r, int g) {
    return static_cast<const char*>(p.x) + ((t0 + (r < toks ? r : toks - 1)) * p.ldx + 32 * g) * (XP == 1 ? 2 : 4);
}

// what every sum is multiplied by
template <bool INT>
__device__ __forceinline__ float last_scale(const MatvecParams& p) {
    return (p.tensor_scale ? *p.tensor_scale : 1.0f) * (INT ? 1.0f / INT_DOWN : 1.0f);
}
// y of token t and row n from its sum
template <bool INT, int XP>
__device__ __forceinline__ void put(const MatvecParams& p, int64_t t, int64_t n, float v, float scale) {
    v *= scale;
    if (p.bias) v += XP == 1 ? bf16f(static_cast<const uint16_t*>(p.bias)[n]) : static_cast<const float*>(p.bias)[n];
    if (p.y_bf16) static_cast<uint16_t*>(p.y)[t * p.ldy + n] = bf16_rne(v);
    else static_cast<float*>(p.y)[t * p.ldy + n] = v;
}

// Left to itself the scheduler moves loads behind the wait for older ones, and
// a branch around loads makes every later use wait for all of them.
#define MV_FENCE __builtin_amdgcn_sched_barrier(0)

// ---------------------------------------------------------------------------
// Short K: each wave takes every eighth step of K for RT tiles of 16 rows, the
// next step's codes, scales and x in registers while it multiplies this one's.
// INT4 in blocks of 8 is held to 128 registers, four waves a SIMD, which puts 16
// bytes of two tiles' state to memory (1 x 14336 x 4096 18.8 us, with 132
// registers 20.0; 8 x 40000 x 1024 14.2 and 17.6).
// ---------------------------------------------------------------------------
template <bool INT, bool MUL, bool OFF, int BK, int XP, int RT>
__global__ __launch_bounds__(512, INT && !MUL && BK == B_8 && XP == 1 ? 4 : 1) void k_short(MatvecParams p, ScaleDec dec) {
    constexpr int WAVES = 8, HOP = WAVES * STEP;
    __shared__ __attribute__((aligned(16))) float red[WAVES][RT][256];
    struct St {
        u32x4 w[RT], x[4][XP == 1 ? 1 : 2];
        Side<OFF, BK> d[RT];
    };
    const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), K = (int)p.k;
    const int64_t n0 = (int64_t)blockIdx.x * 16 * RT, t0 = (int64_t)blockIdx.y * TOK;
    const int toks = (int)(p.tokens - t0 < TOK ? p.tokens - t0 : TOK);
    const Rows R = rows_at(p, n0, 16 * RT);
    int rr[RT];                                               // rows past the end repeat the last
#pragma unroll
    for (int t = 0; t < RT; t++) rr[t] = 16 * t + r < R.rows ? 16 * t + r : R.rows - 1;
    const char* xrow = x_row<XP>(p, t0, toks, r, g);
    const bool macro = p.macro != nullptr, offsets = p.offsets != nullptr;
    const float scale = last_scale<INT>(p);

    auto load = [&](St& o, int k0) {
        load_x<XP>(o.x, xrow, k0);
#pragma unroll
        for (int t = 0; t < RT; t++) {
            o.w[t] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(R.w, rr[t] * R.cb + 16 * g, k0 >> 1, 0));
            load_side<MUL, OFF, BK>(o.d[t], R, rr[t], k0, g, p.lgb);
        }
    };
    f4v acc[RT];
#pragma unroll
    for (int t = 0; t < RT; t++) acc[t] = f4v{0.f, 0.f, 0.f, 0.f};
    auto multiply = [&](const St& o) {
        Cols<OFF, BK, XP> c;
        make_cols<INT>(c, o.x, offsets);
#pragma unroll
        for (int t = 0; t < RT; t++) step_product<INT, MUL, OFF, BK, XP>(acc[t], o.w[t], o.d[t], c, dec, macro, offsets);
    };

    const int whole = K / STEP, mine = (whole - wave + WAVES - 1) / WAVES;      // whole steps; this wave's
    int k0 = wave * STEP;
    St a, b;
    if (mine > 0) {
        load(a, k0);
        for (int i = mine; i > 2; i -= 2, k0 += 2 * HOP) {
            load(b, k0 + HOP);
            MV_FENCE;
            multiply(a);
            MV_FENCE;
            load(a, k0 + 2 * HOP);
            MV_FENCE;
            multiply(b);
            MV_FENCE;
        }
        if (mine % 2 == 0) {
            load(b, k0 + HOP);
            MV_FENCE;
            multiply(a);
            multiply(b);
        } else {
            multiply(a);
        }
    }
    if (whole * STEP < K && whole % WAVES == wave) {
        const int left = K - whole * STEP - 32 * g;
        load_x_end<XP>(a.x, xrow, whole * STEP, left);
#pragma unroll
        for (int t = 0; t < RT; t++) load_end(a.w[t], a.d[t], R, rr[t], whole * STEP, left, g, p.lgb);
        multiply(a);
    }

    // the waves' sums, added in their order
#pragma unroll
    for (int t = 0; t < RT; t++) *reinterpret_cast<f4v*>(&red[wave][t][r * 16 + 4 * g]) = acc[t];      // [token r][row 4 g ..]
    __syncthreads();
    for (int n = tid; n < 256 * RT; n += 64 * WAVES) {
        const int i = n % (16 * RT), t = n / (16 * RT);                    // row of the workgroup, token
        if (t >= toks || i >= R.rows) continue;
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < WAVES; w++) v += red[w][i / 16][t * 16 + i % 16];
        put<INT, XP>(p, t0 + t, n0 + i, v, scale);
    }
}

// ---------------------------------------------------------------------------
// Tall: eight waves side by side along K, a span of SS steps each, x of the
// span in registers; the workgroup's `tiles` tiles of 16 rows one after the
// other, each tile's codes loaded into the registers the one before has just
// freed.  Sums lie in LDS, a
// kilobyte per wave and tile.  Longer K takes further passes over the rows;
// the steps that fill no span are dealt out at the end.
// ---------------------------------------------------------------------------
// as many as the registers hold: x of a step is 16 registers, 48 in three parts
constexpr int span_steps(int xp, bool off) { return xp == 1 ? 4 : off ? 1 : 2; }
constexpr int KW = 8, TALL_TILES = 8;

template <bool INT, bool MUL, bool OFF, int BK, int XP>
__global__ __launch_bounds__(64 * KW, 2) void k_tall(MatvecParams p, ScaleDec dec, int tiles) {
    constexpr int SS = span_steps(XP, OFF), NSB = scales_of(BK), THREADS = 64 * KW;
    extern __shared__ __attribute__((aligned(16))) float red[];            // [tile][wave][token][row]
    typedef Side<OFF, BK> Sd;
    const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), K = (int)p.k;
    const int64_t n0 = (int64_t)blockIdx.x * 16 * tiles, t0 = (int64_t)blockIdx.y * TOK;
    const int toks = (int)(p.tokens - t0 < TOK ? p.tokens - t0 : TOK);
    const Rows R = rows_at(p, n0, 16 * tiles);
    const int nt = (R.rows + 15) / 16;
    const char* xrow = x_row<XP>(p, t0, toks, r, g);
    const bool macro = p.macro != nullptr, offsets = p.offsets != nullptr;
    const float scale = last_scale<INT>(p);
    const int gs = g % SS;                                    // the step whose scales this lane loads
    auto row_of = [&](int t) { const int v = 16 * t + r; return v < R.rows ? v : R.rows - 1; };

    // The scales of a span: lane (r, g) loads row r's of step g, and step i takes
    // them from lane (r, i).
    struct Span {
        uint32_t sc[NSB], off[OFF ? 2 * NSB : 1], mac;
    };
    auto load_span = [&](Span& o, int rr, int k0) {
        const int ks = k0 >> p.lgb, v = rr * R.sr + (STEP * gs >> p.lgb);
        if constexpr (BK == B_32) {
            o.sc[0] = __builtin_amdgcn_raw_buffer_load_b32(R.s, v, ks, 0);
        } else if constexpr (BK == B_16) {
            const auto d = __builtin_amdgcn_raw_buffer_load_b64(R.s, v, ks, 0);
            o.sc[0] = d[0];
            o.sc[NSB - 1] = d[1];
        } else {
            // one block, or (64) two
            o.sc[0] = __builtin_amdgcn_raw_buffer_load_b8(R.s, v, ks, 0);
            o.sc[0] |= (uint32_t)__builtin_amdgcn_raw_buffer_load_b8(R.s, v + (64 >> p.lgb), ks, 0) << 8;
        }
        if constexpr (OFF) {
            if constexpr (BK == B_32) {
                const auto d = __builtin_amdgcn_raw_buffer_load_b64(R.o, 2 * v, 2 * ks, 0);
                o.off[0] = d[0];
                o.off[1] = d[1];
            } else if constexpr (BK == B_16) {
                const auto d = __builtin_amdgcn_raw_buffer_load_b128(R.o, 2 * v, 2 * ks, 0);
#pragma unroll
                for (int e = 0; e < 4; e++) o.off[e % (2 * NSB)] = d[e];
            } else {
                o.off[0] = __builtin_amdgcn_raw_buffer_load_b16(R.o, 2 * v, 2 * ks, 0);
                o.off[1] = __builtin_amdgcn_raw_buffer_load_b16(R.o, 2 * v + 2 * (64 >> p.lgb), 2 * ks, 0);
            }
        }
        if constexpr (MUL) o.mac = __builtin_amdgcn_raw_buffer_load_b8(R.m, rr * R.mb + gs, k0 >> 7, 0);
    };
    auto side_of = [&](Sd& o, const Span& f, int i) {
        const int from = (16 * i + r) * 4;
        auto pull = [&](uint32_t v) { return (uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)v); };
        if constexpr (BK == B_32) {
            o.sc = (pull(f.sc[0]) >> (8 * g)) & 0xffu;
        } else if constexpr (BK == B_16) {
            const uint32_t a = pull(f.sc[0]), b = pull(f.sc[NSB - 1]);
            o.sc = ((g & 2) ? b : a) >> (16 * (g & 1)) & 0xffffu;
        } else {
            o.sc = (pull(f.sc[0]) >> (p.lgb == 6 ? 4 * (g & 2) : 0)) & 0xffu;
        }
        if constexpr (OFF) {
            if (offsets) {
                if constexpr (BK == B_32) {
                    const uint32_t a = pull(f.off[0]), b = pull(f.off[1]);
                    o.off[0] = ((g & 2) ? b : a) >> (16 * (g & 1)) & 0xffffu;
                } else if constexpr (BK == B_16) {
                    uint32_t d[4];
#pragma unroll
                    for (int e = 0; e < 4; e++) d[e] = pull(f.off[e % (2 * NSB)]);
                    const uint32_t w = (g & 2) ? ((g & 1) ? d[3] : d[2]) : ((g & 1) ? d[1] : d[0]);
                    o.off[0] = w & 0xffffu;
                    o.off[NSB - 1] = w >> 16;
                } else {
                    const uint32_t a = pull(f.off[0]), b = pull(f.off[1]);
                    o.off[0] = p.lgb == 6 && (g & 2) ? b : a;
                }
            }
        }
        if constexpr (MUL) {
            if (macro) o.mac = pull(f.mac);
        }
    };
    auto load_w = [&](int rr, int k0) {
        return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(R.w, rr * R.cb + 16 * g, k0 >> 1, 0));
    };
    auto sum_at = [&](int t) -> f4v& { return *reinterpret_cast<f4v*>(red + ((t * KW + wave) * 256 + r * 16 + 4 * g)); };

    const int whole = K / STEP, spans = whole / SS;
    for (int base = 0; base == 0 || base < spans; base += KW) {
        if (base + wave < spans) {
            const int k0 = (base + wave) * SS * STEP;
            u32x4 w[SS], xv[SS][4][XP == 1 ? 1 : 2];
            Span f;
            Cols<OFF, BK, XP> c[SS];
            // tile t, and the loads of tile t + 1 as its registers are used up
            auto use = [&](int t, auto again) {
                f4v acc = {0.f, 0.f, 0.f, 0.f};
                if (base) acc = sum_at(t);
                Sd d[SS];
#pragma unroll
                for (int i = 0; i < SS; i++) side_of(d[i], f, i);
                const int far = INT && !MUL ? __any(far_codes(f.sc[0]) | far_codes(f.sc[NSB - 1])) : 0;      // of all its steps
                const int next = row_of(t + 1);
                if constexpr (again.value) load_span(f, next, k0);
#pragma unroll
                for (int i = 0; i < SS; i++) {
                    step_product<INT, MUL, OFF, BK, XP>(acc, w[i], d[i], c[i], dec, macro, offsets, far);
                    if constexpr (again.value) w[i] = load_w(next, k0 + i * STEP);
                    MV_FENCE;
                }
                sum_at(t) = acc;
            };
#pragma unroll
            for (int i = 0; i < SS; i++) load_x<XP>(xv[i], xrow, k0 + i * STEP);
            load_span(f, row_of(0), k0);
#pragma unroll
            for (int i = 0; i < SS; i++) w[i] = load_w(row_of(0), k0 + i * STEP);
            MV_FENCE;
#pragma unroll
            for (int i = 0; i < SS; i++) make_cols<INT>(c[i], xv[i], offsets);
            for (int t = 0; t + 1 < nt; t++) use(t, std::integral_constant<bool, true>{});
            use(nt - 1, std::integral_constant<bool, false>{});
        } else if (base == 0) {
            for (int t = 0; t < nt; t++) sum_at(t) = f4v{0.f, 0.f, 0.f, 0.f};
        }
    }
    // what fills no span: whole steps, then the end of K
    for (int st = spans * SS + wave; st * STEP < K; st += KW) {
        const int k0 = st * STEP, left = K - k0 - 32 * g;
        u32x4 xv[4][XP == 1 ? 1 : 2];
        if (st < whole) load_x<XP>(xv, xrow, k0);
        else load_x_end<XP>(xv, xrow, k0, left);
        Cols<OFF, BK, XP> c;
        make_cols<INT>(c, xv, offsets);
        for (int t = 0; t < nt; t++) {
            u32x4 w;
            Sd d;
            if (st < whole) {
                w = load_w(row_of(t), k0);
                load_side<MUL, OFF, BK>(d, R, row_of(t), k0, g, p.lgb);
            } else {
                load_end(w, d, R, row_of(t), k0, left, g, p.lgb);
            }
            f4v acc = sum_at(t);
            step_product<INT, MUL, OFF, BK, XP>(acc, w, d, c, dec, macro, offsets);
            sum_at(t) = acc;
        }
    }
    __syncthreads();
    for (int n = tid; n < 256 * nt; n += THREADS) {
        const int i = n % (16 * nt), t = n / (16 * nt);                    // row of the workgroup, token
        if (t >= toks || i >= R.rows) continue;
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < KW; w++) v += red[(i / 16 * KW + w) * 256 + t * 16 + i % 16];
        put<INT, XP>(p, t0 + t, n0 + i, v, scale);
    }
}
#undef MV_FENCE

ScaleDec scale_dec(int scale) {
    return scale == SC_E8M0 ? ScaleDec{0.f, 0xffu} : scale == SC_UE5M3 ? ScaleDec{0x1p112f, 0xffu} : ScaleDec{0x1p120f, 0x7fu};
}

template <bool INT, bool MUL, bool OFF, int BK, int XP, int RT>
hipError_t go_short(const MatvecParams& p, hipStream_t s) {
    const int64_t n = (p.n + 16 * RT - 1) / (16 * RT);
    if (!grid_ok(n, 512)) return TOO_LARGE;
    const dim3 grid((unsigned)n, (unsigned)((p.tokens + TOK - 1) / TOK));
    k_short<INT, MUL, OFF, BK, XP, RT><<<grid, 512, 0, s>>>(p, scale_dec(p.scale));
    return hipGetLastError();
}

template <bool INT, bool MUL, bool OFF, int BK, int XP>
hipError_t go_tall(const MatvecParams& p, hipStream_t s) {
    // one workgroup per CU as far as the rows go
    const int64_t all = (p.n + 15) / 16;
    int64_t tiles = (all + 255) / 256;
    if (tiles > TALL_TILES) tiles = TALL_TILES;
    if (!grid_ok((all + tiles - 1) / tiles, 64 * KW)) return TOO_LARGE;
    const dim3 grid((unsigned)((all + tiles - 1) / tiles), (unsigned)((p.tokens + TOK - 1) / TOK));
    k_tall<INT, MUL, OFF, BK, XP><<<grid, 64 * KW, (int)tiles * KW * 1024, s>>>(p, scale_dec(p.scale), (int)tiles);
    return hipGetLastError();
}

template <bool INT, bool MUL, bool OFF, int BK, int XP>
hipError_t rows(const MatvecParams& p, hipStream_t s) {
    if constexpr (BK != B_8)
        if (p.k >= KW * span_steps(XP, OFF) * STEP) return go_tall<INT, MUL, OFF, BK, XP>(p, s);
    if (p.n <= 16 * 512) return go_short<INT, MUL, OFF, BK, XP, 1>(p, s);
    return go_short<INT, MUL, OFF, BK, XP, 2>(p, s);
}

template <bool INT, bool MUL, bool OFF, int XP>
hipError_t block(const MatvecParams& p, hipStream_t s) {
    if (p.lgb > 5) return rows<INT, MUL, OFF, B_WIDE, XP>(p, s);
    if (p.lgb == 5) return rows<INT, MUL, OFF, B_32, XP>(p, s);
    return p.lgb == 4 ? rows<INT, MUL, OFF, B_16, XP>(p, s) : rows<INT, MUL, OFF, B_8, XP>(p, s);
}

template <bool INT, bool MUL, bool OFF>
hipError_t pick(const MatvecParams& p, hipStream_t s) {
    return p.x_bf16 ? block<INT, MUL, OFF, 1>(p, s) : block<INT, MUL, OFF, 3>(p, s);
}

}  // namespace

hipError_t launch_matvec(const MatvecParams& p, hipStream_t s) {
    const bool mul = p.scale != SC_E8M0 || p.macro;
    if (p.elem == INT4) return mul ? pick<true, true, true>(p, s) : pick<true, false, true>(p, s);
    if (p.offsets) return pick<false, false, true>(p, s);
    return mul ? pick<false, true, false>(p, s) : pick<false, false, false>(p, s);
}

}  // namespace mxk
