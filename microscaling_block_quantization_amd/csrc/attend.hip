// attend.hip -- a paged key-value cache in bf16, MXFP8 (E4M3) or MXFP4: the
// write of new tokens, and the attention of one new token per sequence.
//
// Mathematics.  o = sum_t p_t v_t / sum_t p_t with p_t = 2^(z_t - m), z_t =
// scale log2(e) q.k_t and m any common maximum: one pass over the tokens keeps
// (m, sum p, sum p v) per query head and rescales the sums where m grows; two
// such triples of different tokens join by the same rescaling, which is how
// waves, then workgroups, share a long sequence.
//
// Bound.  Each cached value is used by the few query heads of its key-value
// head and never again: the pass is bound by memory, and both products run on
// the 16 x 16 x 32 bf16 matrix instruction only because it feeds from
// registers as loaded, with the cache as the 16-row operand and up to 16
// query heads as its columns.  No value goes through LDS:
//  - scores: rows are 16 tokens, K runs over the head dimension; a lane (token
//    r, group g) takes 8 values per instruction, and which ones is free as long
//    as the query is laid out alike, so every load is as wide as the type
//    allows (16 bytes: 8 bf16, 16 FP8, or the whole block of 32 FP4).
//  - the result has head = lane % 16, tokens 4 g .. 4 g + 3 per 16: exactly the
//    column operand of the second product when its K order is (tile of 16,
//    token), so probabilities never leave the lane.
//  - that product's rows are values of the head dimension and its K the 32
//    tokens: a lane reads, of its 8 tokens, the same 8 (4, 2) consecutive
//    values, 16 lanes covering whole rows, and pairs of tokens are interleaved
//    in registers (one byte permute per two values).
// FP8 and FP4 values times their block's power of two are exact in bf16 (down
// to bf16's own smallest values), so a quantized cache costs conversions only.
#include "mx_kernels.hpp"

namespace mxk {
using namespace mxd;

namespace {

typedef __bf16 bf8v __attribute__((ext_vector_type(8)));
typedef __bf16 bf2v __attribute__((ext_vector_type(2)));
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

// ---------------------------------------------------------------------------
// Write: eight values a lane, four lanes a block.  The scale rule and the
// conversions are the row quantizer's (round to nearest even; E4M3 clamped
// first, since its converter does not saturate), so codes and scales are the
// ones it writes.
// ---------------------------------------------------------------------------
constexpr int CT = 256;

template <int KIND, bool BF>
__global__ __launch_bounds__(CT) void k_cache_write(CacheWrite p) {
    const uint32_t units = p.c.dim / 8;
    const uint64_t i = (uint64_t)blockIdx.x * CT + threadIdx.x;
    const uint32_t item = (uint32_t)(i / units), u = (uint32_t)(i - (uint64_t)item * units);
    const uint32_t token = item / (2 * p.c.heads), hv = item - token * (2 * p.c.heads);
    if ((int64_t)token >= p.tokens) return;              // whole blocks of four lanes leave
    const bool isv = hv >= (uint32_t)p.c.heads;
    const int head = isv ? hv - p.c.heads : hv;
    const int64_t slot = p.slots[token];
    if (slot < 0 || slot >= p.c.pages * p.c.page) return;
    const int64_t src = (int64_t)token * (isv ? p.v_ts : p.k_ts) + (int64_t)head * (isv ? p.v_hs : p.k_hs) + 8 * u;
    const int64_t page = slot / p.c.page, row = (page * p.c.heads + head) * p.c.page + (slot - page * p.c.page);
    uint8_t* dst = (isv ? p.c.v : p.c.k);
    const void* in = isv ? p.v : p.k;
    float x[8];
    u32x4 raw = {0u, 0u, 0u, 0u};
    if constexpr (BF) {
        raw = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(in) + src);
#pragma unroll
        for (int e = 0; e < 4; e++) { x[2 * e] = bf16lo(raw[e]); x[2 * e + 1] = bf16hi(raw[e]); }
    } else {
        const float4* s = reinterpret_cast<const float4*>(static_cast<const float*>(in) + src);
        const float4 a = s[0], b = s[1];
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    }
    if constexpr (KIND == KV_BF16) {
        if constexpr (!BF) {
#pragma unroll
            for (int e = 0; e < 4; e++) raw[e] = (uint32_t)bf16_rne(x[2 * e]) | (uint32_t)bf16_rne(x[2 * e + 1]) << 16;
        }
        *reinterpret_cast<u32x4*>(dst + (row * p.c.dim + 8 * u) * 2) = raw;
    } else {
        uint32_t am = 0;
#pragma unroll
        for (int e = 0; e < 8; e++) am = max(am, fbits(x[e]) & 0x7fffffffu);
        am = max(am, (uint32_t)__shfl_xor((int)am, 1, 64));
        am = max(am, (uint32_t)__shfl_xor((int)am, 2, 64));
        const bool bad = am >= 0x7f800000u;
        const Elem E = make_elem(KIND == KV_FP8 ? E4M3 : E2M1, 0);
        const uint32_t code = bad ? 255u : (uint32_t)(e8m0_exp(p.rule, p.tau, E, bitsf(am)) + 127);
        const float scale = bitsf(code << 23);
        uint8_t* sc = (isv ? p.c.vs : p.c.ks) + row * (p.c.dim / 32) + u / 4;
        if constexpr (KIND == KV_FP8) {
            // 448 2^e; past the fp32 range no value exceeds it
            const float c = bitsf(code + 8 >= 255 ? 0x7f800000u : ((code + 8) << 23) | 0x600000u);
            uint32_t w[2];
#pragma unroll
            for (int h = 0; h < 2; h++) {
                s2v r = {0, 0};
                r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, __builtin_amdgcn_fmed3f(x[4 * h], -c, c),
                                                             __builtin_amdgcn_fmed3f(x[4 * h + 1], -c, c), scale, false);
                r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, __builtin_amdgcn_fmed3f(x[4 * h + 2], -c, c),
                                                             __builtin_amdgcn_fmed3f(x[4 * h + 3], -c, c), scale, true);
                __builtin_memcpy(&w[h], &r, 4);
            }
            *reinterpret_cast<uint2*>(dst + row * p.c.dim + 8 * u) = make_uint2(bad ? 0u : w[0], bad ? 0u : w[1]);
        } else {
            uint32_t w = 0;
            w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[0], x[1], scale, 0);
            w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[2], x[3], scale, 1);
            w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[4], x[5], scale, 2);
            w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[6], x[7], scale, 3);
            *reinterpret_cast<uint32_t*>(dst + row * (p.c.dim / 2) + 4 * u) = bad ? 0u : w;
        }
        if (u % 4 == 0) *sc = (uint8_t)code;
    }
}

// ---------------------------------------------------------------------------
// Attention
// ---------------------------------------------------------------------------
constexpr int AW = 4, AT = 64 * AW;    // waves, threads
constexpr int TILE = 32;               // tokens a wave takes at a time
constexpr int QH = 16;                 // query heads of one workgroup

// Bits of one value, and the widest run of the head dimension (a "unit") that
// 4 lanes of a token cover with one load of at most 16 bytes each.
constexpr int kind_bits(int kind) { return kind == KV_BF16 ? 16 : kind == KV_FP8 ? 8 : 4; }
constexpr int unit_max(int kind) { return 4 * 128 / kind_bits(kind); }
// the unit at `base`: the widest power of two that fits, at least 32
constexpr int unit_at(int D, int base, int most) {
    int u = most;
    while (u > D - base) u /= 2;
    return u;
}
constexpr int count_units(int D, int most) {
    int n = 0;
    for (int b = 0; b < D; b += unit_at(D, b, most)) n++;
    return n;
}
constexpr int unit_base(int D, int most, int i) {
    int b = 0;
    for (int k = 0; k < i; k++) b += unit_at(D, b, most);
    return b;
}

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

// a query value as its exact bf16 parts
__device__ __forceinline__ void parts_of(float x, uint32_t (&o)[3]) {
    const uint32_t u = fbits(x);
    if ((u & 0x7f800000u) == 0x7f800000u) {
        o[0] = bf16_rne(x);
        o[1] = o[2] = 0;
        return;
    }
    const float r = x - bitsf(u & 0xffff0000u);
    o[0] = u >> 16;
    o[1] = fbits(r) >> 16;
    o[2] = fbits(r - bitsf(fbits(r) & 0xffff0000u)) >> 16;
}

template <int D, int KIND, bool QF32, bool PAGE16>
__global__ __launch_bounds__(AT) void k_attend(AttendParams p) {
    constexpr int QP = QF32 ? 3 : 1;              // bf16 parts of a query
    constexpr int PP = QF32 ? 3 : 2;              // bf16 parts of a probability
    constexpr int BITS = kind_bits(KIND), ROWB = D * BITS / 8;
    constexpr int KU = count_units(D, unit_max(KIND));     // units of the score product
    constexpr int VU = count_units(D, 128);                // runs of 16 lanes of the second product
    constexpr int LD = D + 1;                              // LDS row of one head's sums
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, g = lane >> 4;
    const int group = p.q_heads / p.c.heads, tiles = (group + QH - 1) / QH;
    // workgroup -> split (fastest), head tile, key-value head, sequence
    uint32_t id = blockIdx.x;
    const int split = (int)(id % (uint32_t)p.splits);
    id /= (uint32_t)p.splits;
    const int tile = (int)(id % (uint32_t)tiles);
    id /= (uint32_t)tiles;
    const int kvh = (int)(id % (uint32_t)p.c.heads);
    const int64_t b = id / (uint32_t)p.c.heads;
    const int h0 = kvh * group + tile * QH;                // first query head
    const int nh = group - tile * QH < QH ? group - tile * QH : QH;

    const int64_t cap = p.cols * p.c.page;
    int64_t len64 = p.lengths[b];
    len64 = len64 < 0 ? 0 : len64 > cap ? cap : len64;
    const int len = (int)len64, t0 = split * p.chunk;
    if (t0 >= len && !(len == 0 && split == 0)) return;    // nothing here; the join does not read it
    const int tend = len < t0 + p.chunk ? len : t0 + p.chunk;

    // the query, laid out as the score product's columns
    uint32_t q[QP][D / 32][4];
    {
        const int64_t at = b * p.q_ts + (int64_t)(h0 + (r < nh ? r : nh - 1)) * p.q_hs;
        each<KU>([&](auto iu) {
            constexpr int BASE = unit_base(D, unit_max(KIND), iu.value), U = unit_at(D, BASE, unit_max(KIND));
#pragma unroll
            for (int f = 0; f < U / 32; f++) {
                const int64_t d = at + BASE + g * (U / 4) + 8 * f;
                if constexpr (QF32) {
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        uint32_t x[3], y[3];
                        parts_of(static_cast<const float*>(p.q)[d + 2 * e], x);
                        parts_of(static_cast<const float*>(p.q)[d + 2 * e + 1], y);
#pragma unroll
                        for (int k = 0; k < 3; k++) q[k][BASE / 32 + f][e] = x[k] | y[k] << 16;
                    }
                } else {
                    load_bytes<16>(q[0][BASE / 32 + f], reinterpret_cast<const uint8_t*>(static_cast<const uint16_t*>(p.q) + d));
                }
            }
        });
    }

    f4v acc[D / 16];
#pragma unroll
    for (int i = 0; i < D / 16; i++) acc[i] = f4v{0.f, 0.f, 0.f, 0.f};
    float m = -INFINITY, l = 0.f;                          // of head r; l: this lane's tokens
    bool bad = false;
    const float zs = p.scale * 1.44269504088896340736f;
    const int32_t* table = p.table + b * p.table_stride;

    // cache row of token t (page lookup); a bad page reads page 0
    auto row_of = [&](int t) -> int64_t {
        const uint32_t pg = (uint32_t)(((uint64_t)(uint32_t)t * p.page_mul) >> p.page_shift);
        int64_t n = table[pg];
        if (n < 0 || n >= p.c.pages) { n = 0; bad = true; }
        return (n * p.c.heads + kvh) * p.c.page + (t - (int)pg * p.c.page);
    };

    for (int tb = t0 + wave * TILE; tb < tend; tb += AW * TILE) {
        // rows of the key operand: token 16 h + r; of the value operand: 16 h + 4 g + i
        int64_t kr[2], vr[2][4];
#pragma unroll
        for (int h = 0; h < 2; h++) {
            if constexpr (PAGE16) {
                // 16 tokens lie in one page
                const int t = tb + 16 * h < tend ? tb + 16 * h : tb;
                const int64_t base = row_of(t);
                const int left = tend - 1 - t;             // last usable token from the base
                kr[h] = base + (r < left ? r : left);
#pragma unroll
                for (int i = 0; i < 4; i++) vr[h][i] = base + (4 * g + i < left ? 4 * g + i : left);
            } else {
                const int tk = tb + 16 * h + r;
                kr[h] = row_of(tk < tend ? tk : tend - 1);
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const int t = tb + 16 * h + 4 * g + i;
                    vr[h][i] = row_of(t < tend ? t : tend - 1);
                }
            }
        }

        // scores
        f4v z[2];
#pragma unroll
        for (int h = 0; h < 2; h++) {
            z[h] = f4v{0.f, 0.f, 0.f, 0.f};
            const uint8_t* krow = p.c.k + kr[h] * ROWB;
            each<KU>([&](auto iu) {
                constexpr int BASE = unit_base(D, unit_max(KIND), iu.value), U = unit_at(D, BASE, unit_max(KIND));
                uint32_t w[4];
                load_bytes<U * BITS / 32>(w, krow + (BASE + g * (U / 4)) * BITS / 8);
                float s = 1.f;
                if constexpr (KIND != KV_BF16) s = e8m0(p.c.ks[kr[h] * (D / 32) + (BASE + g * (U / 4)) / 32]);
                each<U / 32>([&](auto fi) {
                    constexpr int f = fi.value;
                    const bf8v a = frag(pair_of<KIND, 4 * f>(w, s), pair_of<KIND, 4 * f + 1>(w, s),
                                        pair_of<KIND, 4 * f + 2>(w, s), pair_of<KIND, 4 * f + 3>(w, s));
#pragma unroll
                    for (int k = 0; k < QP; k++) {
                        const uint32_t* qq = q[k][BASE / 32 + f];
                        z[h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, frag(qq[0], qq[1], qq[2], qq[3]), z[h], 0, 0, 0);
                    }
                });
            });
        }

        // softmax of this lane's 8 tokens of head r
        float zmax = -INFINITY;
#pragma unroll
        for (int h = 0; h < 2; h++)
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const float v = tb + 16 * h + 4 * g + i < tend ? z[h][i] * zs : -INFINITY;
                z[h][i] = v;
                zmax = fmaxf(zmax, v);
            }
        zmax = fmaxf(zmax, __shfl_xor(zmax, 16, 64));
        zmax = fmaxf(zmax, __shfl_xor(zmax, 32, 64));
        const float mn = fmaxf(m, zmax);
        const float ms = mn == -INFINITY ? 0.f : mn;       // every score so far is -inf
        const float grow = exp2f(m - ms);
        m = mn;
        l *= grow;
        uint32_t pw[PP][4];                                // probabilities as bf16 pairs
        float pr[8];
#pragma unroll
        for (int i = 0; i < 8; i++) {
            pr[i] = exp2f(z[i / 4][i % 4] - ms);
            l += pr[i];
        }
#pragma unroll
        for (int i = 0; i < 4; i++) {
            float x = pr[2 * i], y = pr[2 * i + 1];
#pragma unroll
            for (int k = 0; k < PP; k++) {
                const uint32_t a = bf16_rne(x), c = bf16_rne(y);
                pw[k][i] = a | c << 16;
                x -= bitsf(a << 16);
                y -= bitsf(c << 16);
            }
        }
#pragma unroll
        for (int i = 0; i < D / 16; i++) acc[i] *= grow;

        // sums of p v
        const bool part = tb + TILE > tend;
        each<VU>([&](auto iu) {
            constexpr int BASE = unit_base(D, 128, iu.value), W = unit_at(D, BASE, 128) / 16;
            constexpr int WB = W * BITS / 8;               // bytes a lane reads per token
            uint32_t v[8][WB < 4 ? 1 : WB / 4];
            float s[8];
#pragma unroll
            for (int i = 0; i < 8; i++) {
                load_bytes<WB>(v[i], p.c.v + vr[i / 4][i % 4] * ROWB + (BASE + r * W) * BITS / 8);
                if constexpr (KIND != KV_BF16) s[i] = e8m0(p.c.vs[vr[i / 4][i % 4] * (D / 32) + (BASE + r * W) / 32]);
                else s[i] = 1.f;
            }
            if (part) {
                // past the end: whatever the cache holds is taken as zero
#pragma unroll
                for (int i = 0; i < 8; i++)
                    if (tb + 16 * (i / 4) + 4 * g + i % 4 >= tend) {
                        s[i] = 1.f;
#pragma unroll
                        for (int k = 0; k < (WB < 4 ? 1 : WB / 4); k++) v[i][k] = 0u;
                    }
            }
            each<W / 2>([&](auto pi) {
                constexpr int I = pi.value;
                uint32_t t[8];
#pragma unroll
                for (int i = 0; i < 8; i++) t[i] = pair_of<KIND, I>(v[i], s[i]);
#pragma unroll
                for (int odd = 0; odd < 2; odd++) {
                    const uint32_t sel = odd ? 0x07060302u : 0x05040100u;
                    const bf8v a = frag(__builtin_amdgcn_perm(t[1], t[0], sel), __builtin_amdgcn_perm(t[3], t[2], sel),
                                        __builtin_amdgcn_perm(t[5], t[4], sel), __builtin_amdgcn_perm(t[7], t[6], sel));
                    f4v& o = acc[BASE / 16 + 2 * I + odd];
#pragma unroll
                    for (int k = 0; k < PP; k++)
                        o = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, frag(pw[k][0], pw[k][1], pw[k][2], pw[k][3]), o, 0, 0, 0);
                }
            });
        });
    }

    // the waves' triples, joined through LDS
    l += __shfl_xor(l, 16, 64);
    l += __shfl_xor(l, 32, 64);
    if (__any(bad)) l = bitsf(0x7fc00000u);
    float* sums = reinterpret_cast<float*>(smem);                  // [wave][head][LD]
    float* ml = sums + AW * QH * LD;                               // [wave][head][2]
    each<VU>([&](auto iu) {
        constexpr int BASE = unit_base(D, 128, iu.value), W = unit_at(D, BASE, 128) / 16;
#pragma unroll
        for (int i = 0; i < W; i++)
#pragma unroll
            for (int e = 0; e < 4; e++)
                sums[(wave * QH + r) * LD + BASE + (4 * g + e) * W + i] = acc[BASE / 16 + i][e];
    });
    if (g == 0) {
        ml[(wave * QH + r) * 2] = m;
        ml[(wave * QH + r) * 2 + 1] = l;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < nh * D; i += AT) {
        const int h = i / D, d = i - h * D;
        float M = -INFINITY, L = 0.f, o = 0.f;
#pragma unroll
        for (int w = 0; w < AW; w++) M = fmaxf(M, ml[(w * QH + h) * 2]);
        const float Ms = M == -INFINITY ? 0.f : M;
#pragma unroll
        for (int w = 0; w < AW; w++) {
            const float f = exp2f(ml[(w * QH + h) * 2] - Ms);
            L += f * ml[(w * QH + h) * 2 + 1];
            o += f * sums[(w * QH + h) * LD + d];
        }
        const int64_t bh = b * p.q_heads + h0 + h;
        if (p.splits > 1) {
            p.parts[(bh * p.splits + split) * D + d] = o;
            if (d == 0) {
                float* x = p.parts + p.batch * p.q_heads * p.splits * D + (bh * p.splits + split) * 2;
                x[0] = M;
                x[1] = L;
            }
        } else {
            const float v = L == 0.f ? 0.f : o / L;
            const int64_t at = b * p.o_ts + (int64_t)(h0 + h) * p.o_hs + d;
            if (QF32) static_cast<float*>(p.o)[at] = v;
            else static_cast<uint16_t*>(p.o)[at] = bf16_rne(v);
            if (p.lse && d == 0) p.lse[bh] = L == 0.f ? -INFINITY : (Ms + log2f(L)) * 0.69314718055994530942f;
        }
    }
}

// Joins the splits of one sequence and query head: a wave takes every fourth
// split, lanes the head dimension.
template <int D, bool QF32>
__global__ __launch_bounds__(256) void k_attend_join(AttendParams p) {
    constexpr int N = (D + 63) / 64;
    __shared__ float so[4][D], sl[4];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t bh = blockIdx.x, b = bh / p.q_heads;
    const int h = (int)(bh - b * p.q_heads);
    const int64_t cap = p.cols * p.c.page;
    int64_t len = p.lengths[b];
    len = len < 0 ? 0 : len > cap ? cap : len;
    int used = (int)((len + p.chunk - 1) / p.chunk);
    if (used < 1) used = 1;                          // an empty sequence's first workgroup leaves sum 0
    const float* o = p.parts + bh * p.splits * D;
    const float* x = p.parts + p.batch * p.q_heads * p.splits * D + bh * p.splits * 2;
    float M = -INFINITY;
    for (int i = lane; i < used; i += 64) M = fmaxf(M, x[2 * i]);
#pragma unroll
    for (int k = 1; k < 64; k <<= 1) M = fmaxf(M, __shfl_xor(M, k, 64));
    const float Ms = M == -INFINITY ? 0.f : M;
    float v[N], L = 0.f;
#pragma unroll
    for (int k = 0; k < N; k++) v[k] = 0.f;
    for (int i = wave; i < used; i += 4) {
        const float f = exp2f(x[2 * i] - Ms);
        L += f * x[2 * i + 1];
#pragma unroll
        for (int k = 0; k < N; k++)
            if (lane + 64 * k < D) v[k] += f * o[(int64_t)i * D + lane + 64 * k];
    }
#pragma unroll
    for (int k = 0; k < N; k++)
        if (lane + 64 * k < D) so[wave][lane + 64 * k] = v[k];
    if (lane == 0) sl[wave] = L;
    __syncthreads();
    L = sl[0] + sl[1] + sl[2] + sl[3];
    for (int d = threadIdx.x; d < D; d += 256) {
        const float s = so[0][d] + so[1][d] + so[2][d] + so[3][d];
        const float r = L == 0.f ? 0.f : s / L;
        const int64_t at = b * p.o_ts + (int64_t)h * p.o_hs + d;
        if (QF32) static_cast<float*>(p.o)[at] = r;
        else static_cast<uint16_t*>(p.o)[at] = bf16_rne(r);
        if (p.lse && d == 0) p.lse[bh] = L == 0.f ? -INFINITY : (Ms + log2f(L)) * 0.69314718055994530942f;
    }
}

template <int D, int KIND, bool QF32, bool PAGE16>
hipError_t go(const AttendParams& p, hipStream_t s) {
    const int group = p.q_heads / p.c.heads, tiles = (group + QH - 1) / QH;
    const int64_t n = p.batch * p.c.heads * tiles * p.splits;
    constexpr int lds = (AW * QH * (D + 1) + AW * QH * 2) * (int)sizeof(float);
    if (lds > 64 * 1024) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(k_attend<D, KIND, QF32, PAGE16>),
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, lds);
        if (e != hipSuccess) return e;
    }
    k_attend<D, KIND, QF32, PAGE16><<<(unsigned)n, AT, lds, s>>>(p);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.splits == 1) return e;
    k_attend_join<D, QF32><<<(unsigned)(p.batch * p.q_heads), 256, 0, s>>>(p);
    return hipGetLastError();
}

template <int D, bool QF32>
hipError_t pick(const AttendParams& p, hipStream_t s) {
    const bool p16 = p.c.page % 16 == 0;
    if (p.c.kind == KV_BF16) return p16 ? go<D, KV_BF16, QF32, true>(p, s) : go<D, KV_BF16, QF32, false>(p, s);
    if (p.c.kind == KV_FP8) return p16 ? go<D, KV_FP8, QF32, true>(p, s) : go<D, KV_FP8, QF32, false>(p, s);
    return p16 ? go<D, KV_FP4, QF32, true>(p, s) : go<D, KV_FP4, QF32, false>(p, s);
}

}  // namespace

hipError_t launch_cache_write(const CacheWrite& p, bool bf, hipStream_t s) {
    const int64_t n = p.tokens * 2 * p.c.heads * (p.c.dim / 8);
    const unsigned grid = (unsigned)((n + CT - 1) / CT);
    if (p.c.kind == KV_BF16) {
        if (bf) k_cache_write<KV_BF16, true><<<grid, CT, 0, s>>>(p);
        else k_cache_write<KV_BF16, false><<<grid, CT, 0, s>>>(p);
    } else if (p.c.kind == KV_FP8) {
        if (bf) k_cache_write<KV_FP8, true><<<grid, CT, 0, s>>>(p);
        else k_cache_write<KV_FP8, false><<<grid, CT, 0, s>>>(p);
    } else {
        if (bf) k_cache_write<KV_FP4, true><<<grid, CT, 0, s>>>(p);
        else k_cache_write<KV_FP4, false><<<grid, CT, 0, s>>>(p);
    }
    return hipGetLastError();
}

bool attend_dim_ok(int d) { return d == 64 || d == 96 || d == 128 || d == 192 || d == 256; }

// Splits: enough workgroups to fill the chip twice over, none shorter than one
// tile per wave.
void attend_plan(const KvCache& c, int64_t batch, int q_heads, int64_t cols, int* chunk, int* splits) {
    const int group = q_heads / c.heads, tiles = (group + QH - 1) / QH;
    const int64_t units = batch > 0 ? batch * c.heads * tiles : 1, longest = cols * c.page, least = AW * TILE;
    const int64_t want = 1024;
    int64_t n = units >= want ? 1 : (want + units - 1) / units;
    int64_t per = ((longest + n - 1) / n + least - 1) / least * least;
    if (per < least) per = least;
    *chunk = (int)per;
    *splits = longest > 0 ? (int)((longest + per - 1) / per) : 1;
}

hipError_t launch_attend(AttendParams p, bool bf, hipStream_t s) {
    // t / page by a multiply: mul = ceil(2^sh / page) with 2^sh >= 2^31 page,
    // exact for t < 2^31; mul < 2^32
    int lg = 0;
    while ((1 << lg) < p.c.page) lg++;
    p.page_shift = 31 + lg;
    p.page_mul = (uint32_t)((((uint64_t)1 << p.page_shift) + p.c.page - 1) / p.c.page);
    switch (p.c.dim) {
    case 64: return bf ? pick<64, false>(p, s) : pick<64, true>(p, s);
    case 96: return bf ? pick<96, false>(p, s) : pick<96, true>(p, s);
    case 128: return bf ? pick<128, false>(p, s) : pick<128, true>(p, s);
    case 192: return bf ? pick<192, false>(p, s) : pick<192, true>(p, s);
    default: return bf ? pick<256, false>(p, s) : pick<256, true>(p, s);
    }
}

}  // namespace mxk
