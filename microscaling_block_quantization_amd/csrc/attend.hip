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
// Measured (32 query and 8 key-value heads of 128): 32 sequences up to 8192
// tokens, bf16, 106 us, 5.3 TB/s of cache (a large copy reaches 5.1); one of
// 131072, bf16 100 us (5.4), MXFP8 64 us (4.3), MXFP4 47 us (3.0), where the
// conversions, the softmax and the waits between them no longer hide.
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

// ---------------------------------------------------------------------------
// Write: eight values a lane, four lanes a block.  The scale rule and the
// conversions are the row quantizer's (round to nearest even; E4M3 clamped
// first, since its converter does not saturate), so codes and scales are the
// ones it writes.
// ---------------------------------------------------------------------------
constexpr int CT = 256;

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

// D: the head dimension, known here because a division by a number that is not
// costs more than everything else a lane does.  A lane takes the key and the
// value of its place, both loads at once.
template <int D, int KIND, bool BF>
__global__ __launch_bounds__(CT) void k_cache_write(CacheWrite p) {
    constexpr uint32_t UNITS = D / 8, PER = CT / UNITS;           // lanes of a vector, vectors of a workgroup
    const uint32_t n = threadIdx.x / UNITS, u = threadIdx.x - n * UNITS;
    const uint32_t item = blockIdx.x * PER + n;                   // (token, head)
    const uint32_t token = over(item, p.per_token), head = item - token * p.c.heads;
    if (n >= PER || (int64_t)token >= p.tokens) return;           // whole blocks of four lanes leave
    u32x4 raw[2][BF ? 1 : 2];
#pragma unroll
    for (int v = 0; v < 2; v++) {
        const int64_t src = (int64_t)token * (v ? p.v_ts : p.k_ts) + (int64_t)head * (v ? p.v_hs : p.k_hs) + 8 * u;
        const u32x4* in = BF ? reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(v ? p.v : p.k) + src)
                             : reinterpret_cast<const u32x4*>(static_cast<const float*>(v ? p.v : p.k) + src);
#pragma unroll
        for (int i = 0; i < (BF ? 1 : 2); i++) raw[v][i] = in[i];
    }
    const int64_t slot = p.slots[token];
    if (slot < 0 || slot >= p.c.pages * p.c.page) return;
    const int64_t page = p.page_shift >= 0 ? slot >> p.page_shift : slot < (1ll << 31) ? over((uint32_t)slot, p.page_div) : slot / p.c.page;
    const int64_t row = (page * p.c.heads + head) * p.c.page + (slot - page * p.c.page);
#pragma unroll
    for (int v = 0; v < 2; v++) {
        uint8_t* dst = v ? p.c.v : p.c.k;
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; e++)
            x[e] = BF ? ((e & 1) ? bf16hi(raw[v][0][e / 2]) : bf16lo(raw[v][0][e / 2])) : bitsf(raw[v][BF ? 0 : e / 4][e % 4]);
        if constexpr (KIND == KV_BF16) {
            u32x4 o = raw[v][0];
            if constexpr (!BF) {
#pragma unroll
                for (int e = 0; e < 4; e++) o[e] = (uint32_t)bf16_rne(x[2 * e]) | (uint32_t)bf16_rne(x[2 * e + 1]) << 16;
            }
            *reinterpret_cast<u32x4*>(dst + (row * D + 8 * u) * 2) = o;
            continue;
        }
        uint32_t am = 0;
#pragma unroll
        for (int e = 0; e < 8; e++) am = max(am, fbits(x[e]) & 0x7fffffffu);
        am = max(am, (uint32_t)__shfl_xor((int)am, 1, 64));
        am = max(am, (uint32_t)__shfl_xor((int)am, 2, 64));
        const bool bad = am >= 0x7f800000u;
        const Elem E = make_elem(KIND == KV_FP8 ? E4M3 : E2M1, 0);
        const uint32_t code = bad ? 255u : (uint32_t)(e8m0_exp(p.rule, p.tau, E, bitsf(am)) + 127);
        const float scale = bitsf(code << 23);
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
            *reinterpret_cast<uint2*>(dst + row * D + 8 * u) = make_uint2(bad ? 0u : w[0], bad ? 0u : w[1]);
        } else {
            uint32_t w = 0;
            w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[0], x[1], scale, 0);
            w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[2], x[3], scale, 1);
            w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[4], x[5], scale, 2);
            w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[6], x[7], scale, 3);
            *reinterpret_cast<uint32_t*>(dst + row * (D / 2) + 4 * u) = bad ? 0u : w;
        }
        if (u % 4 == 0) (v ? p.c.vs : p.c.ks)[row * (D / 32) + u / 4] = (uint8_t)code;
    }
}

// ---------------------------------------------------------------------------
// Attention
// ---------------------------------------------------------------------------
constexpr int TILE = 32;               // tokens a wave takes at a time
constexpr int QH = 16;                 // query heads of one workgroup
constexpr int EIGHT_MAX = 128;         // largest head dimension whose registers leave room for eight waves

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

// Left to itself the scheduler moves loads behind the wait for older ones.
#define ISSUED __builtin_amdgcn_sched_barrier(0)

// How long sequences are shared out.  Lengths are known on the device alone and
// differ, so the workgroups of a plane ("workers") divide the tokens of all
// sequences, one after the other in units of 128, into equal ranges: worker w of
// W takes units [w T / W, (w + 1) T / W) of T (of the first T workers where there
// are more than units, so that no range is empty).  A range may hold the end of one
// sequence and the beginning of the next; a sequence within one range is
// finished there, the others' parts go to slot w + b of their heads (in order, a
// range's step moves w on and a sequence's step b, so no two share one).
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
// Worker w's range, the sequence its first unit lies in and the units before
// that sequence; false for an empty range.
template <int T, typename F>
__device__ __forceinline__ bool share_of(int64_t batch, uint32_t w, int workers, F&& units, int64_t& b, int64_t& before, int64_t& u,
                                         int64_t& u_end) {
    __shared__ int64_t sh[T / 64 + 2];
    const int tid = threadIdx.x, lane = tid & 63;
    // the same in every thread, and known to be
    auto uniform = [](int64_t v) {
        return (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(v >> 32)) << 32 |
                         (uint32_t)__builtin_amdgcn_readfirstlane((int)v));
    };
    if (batch <= 64) {                                     // each wave on its own, a sequence a lane (at most 2^29 units)
        const int n = lane < batch ? (int)units(lane) : 0;
        int upto = n;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int v = __shfl_up(upto, o, 64);
            if (lane >= o) upto += v;
        }
        const int t = __builtin_amdgcn_readlane(upto, 63), of = workers_used(t, workers);
        if ((int)w >= of) return false;
        u = (int64_t)w * t / of;
        u_end = (int64_t)(w + 1) * t / of;
        const int at = __ffsll((unsigned long long)__ballot(upto > u)) - 1;      // the first that reaches past unit u
        b = at;
        before = __builtin_amdgcn_readlane(upto - n, at);
        return true;
    }
    int64_t mine = 0;
    for (int64_t i = tid; i < batch; i += T) mine += units(i);
    const int64_t t = block_total<T>(mine, sh), of = workers_used(t, workers);
    if (w >= of) return false;
    u = w * t / of;
    u_end = (w + 1) * t / of;
    int64_t run = 0;
    for (int64_t base = 0;; base += T) {                   // some sequence holds unit u
        const int64_t n = base + tid < batch ? units(base + tid) : 0;
        int64_t upto = n;                                  // inclusive sums over the wave
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int64_t v = __shfl_up(upto, o, 64);
            if (lane >= o) upto += v;
        }
        if (lane == 63) sh[tid >> 6] = upto;
        __syncthreads();
        int64_t lead = run, all = 0;
#pragma unroll
        for (int i = 0; i < T / 64; i++) {
            if (i < (tid >> 6)) lead += sh[i];
            all += sh[i];
        }
        const int64_t from = lead + upto - n;
        if (from <= u && u < from + n) {
            sh[T / 64] = base + tid;
            sh[T / 64 + 1] = from;
        }
        __syncthreads();
        if (u < run + all) break;
        run += all;
    }
    b = uniform(sh[T / 64]);
    before = uniform(sh[T / 64 + 1]);
    u = uniform(u);
    u_end = uniform(u_end);
    return true;
}

// One wave takes every AW-th tile of 32 tokens of the workgroup's segment.  The
// loads of a tile's values go out before its scores are formed, those of the
// next tile's keys before its second product, so one of the two is always in
// flight.  PAGE16: pages of a multiple of 16 tokens, so that 16 tokens share a
// page, whose number is then one scalar load, and reading all 16 stays inside
// the page whatever the length.
template <int D, int KIND, bool QF32, bool PAGE16, int AW>
__global__ __launch_bounds__(64 * AW, D <= 128 ? 2 : 1) void k_attend(AttendParams p) {
    constexpr int QP = QF32 ? 3 : 1;              // bf16 parts of a query
    // bf16 parts of a probability: three hold all its 24 bits.  A bf16 query's
    // output has 8, and a probability's 16 move it by at most 2^-16 of sum p |v|
    // (one in a few hundred outputs rounds to its other bf16 neighbour; the error
    // against 64 bits is the same), for two products instead of three.
    constexpr int PP = QF32 ? 3 : 2;
    constexpr int BITS = kind_bits(KIND), ROWB = D * BITS / 8, NB = D / 32;
    constexpr int KU = count_units(D, unit_max(KIND));     // units of the score product
    constexpr int VU = count_units(D, 128);                // runs of 16 lanes of the second product
    constexpr int LD = D + 1;                              // LDS row of one head's sums
    // scales of a token (and of the value operand's four tokens) as whole dwords
    constexpr bool WIDE_SC = KIND != KV_BF16 && PAGE16 && (D == 64 || D % 128 == 0);
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, g = lane >> 4;
    const int group = p.q_heads / p.c.heads, tiles = (group + QH - 1) / QH;
    const uint32_t planes = (uint32_t)(p.c.heads * tiles);
    const int64_t cap = p.cols * p.c.page;
    auto len_of = [&](int64_t b) {
        const int64_t n = p.lengths[b];
        return (int)(n < 0 ? 0 : n > cap ? cap : n);
    };
    // This workgroup's plane (key-value head and head tile), first sequence and,
    // among workers, its share [u, u_end) of the units of all sequences in order;
    // `before` is the number of units before sequence b.
    uint32_t plane;
    int64_t b, u = 0, u_end = 0, before = 0;
    if (p.workers) {
        plane = blockIdx.x / (uint32_t)p.workers;
        const uint32_t w = blockIdx.x - plane * (uint32_t)p.workers;
        if (!share_of<64 * AW>(p.batch, w, p.workers, [&](int64_t i) { return units_of(len_of(i)); }, b, before, u, u_end)) return;
    } else {
        b = blockIdx.x / planes;
        plane = blockIdx.x - (uint32_t)b * planes;
    }
    const int tile = (int)(plane % (uint32_t)tiles), kvh = (int)(plane / (uint32_t)tiles);
    const int h0 = kvh * group + tile * QH;                // first query head
    const int nh = group - tile * QH < QH ? group - tile * QH : QH;
    const float zs = p.scale * 1.44269504088896340736f;

    while (true) {                                         // a segment of one sequence: tokens [t0, tend)
    const int len = len_of(b);
    const int64_t t1 = (u_end - before) * UNIT;
    const int t0 = p.workers ? (int)((u - before) * UNIT) : 0, tend = p.workers && t1 < len ? (int)t1 : len;
    const int32_t* table = p.table + b * p.table_stride;

    bool bad = false;
    // cache row of token t (page lookup); a bad page reads page 0
    auto row_of = [&](int t) -> int64_t {
        const uint32_t pg = over((uint32_t)t, p.page_div);
        int64_t n = table[pg];
        if (n < 0 || n >= p.c.pages) { n = 0; bad = true; }
        return (n * p.c.heads + kvh) * p.c.page + (t - (int)pg * p.c.page);
    };
    // rows of the operands of the tile at tb: keys 16 h + r, values 16 h + 4 g + i
    struct Place {
        int64_t base[2];           // PAGE16: the row of token 16 h
        int64_t k[PAGE16 ? 1 : 2], v[PAGE16 ? 1 : 2][4];
    };
    auto place = [&](Place& o, int tb) {
#pragma unroll
        for (int h = 0; h < 2; h++) {
            if constexpr (PAGE16) {
                o.base[h] = row_of(tb + 16 * h < tend ? tb + 16 * h : tb);
            } else {
                const int tk = tb + 16 * h + r;
                o.k[h] = row_of(tk < tend ? tk : tend - 1);
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const int t = tb + 16 * h + 4 * g + i;
                    o.v[h][i] = row_of(t < tend ? t : tend - 1);
                }
            }
        }
    };
    // bytes `at` of key row 16 h + r / value row 16 h + 4 g + i of an array of `per` bytes a row
    auto key_at = [&](const uint8_t* a, const Place& o, int h, int per, uint32_t at) -> const uint8_t* {
        if constexpr (PAGE16) return a + o.base[h] * per + (uint32_t)(r * per + at);
        else return a + o.k[h] * per + at;
    };
    auto value_at = [&](const uint8_t* a, const Place& o, int h, int i, int per, uint32_t at) -> const uint8_t* {
        if constexpr (PAGE16) return a + o.base[h] * per + (uint32_t)((4 * g + i) * per + at);
        else return a + o.v[h][i] * per + at;
    };

    // a tile's keys: 16-byte pieces by unit, and their scales
    struct Keys {
        uint32_t w[2][KU][4], sc[2][KIND == KV_BF16 ? 1 : WIDE_SC ? (NB + 3) / 4 : KU];
    };
    auto load_keys = [&](Keys& o, const Place& at) {
#pragma unroll
        for (int h = 0; h < 2; h++) {
            each<KU>([&](auto iu) {
                constexpr int BASE = unit_base(D, unit_max(KIND), iu.value), U = unit_at(D, BASE, unit_max(KIND));
                load_bytes<U * BITS / 32>(o.w[h][iu.value], key_at(p.c.k, at, h, ROWB, (BASE + g * (U / 4)) * BITS / 8));
                if constexpr (KIND != KV_BF16 && !WIDE_SC)
                    o.sc[h][iu.value] = *key_at(p.c.ks, at, h, NB, (BASE + g * (U / 4)) / 32);
            });
            if constexpr (WIDE_SC) load_bytes<NB>(o.sc[h], key_at(p.c.ks, at, h, NB, 0));
        }
    };
    // its values: runs of W per token, and their scales
    struct Values {
        uint32_t w[VU][8][4], sc[WIDE_SC ? 2 : VU][WIDE_SC ? NB : 8];
    };
    auto load_values = [&](Values& o, const Place& at) {
        each<VU>([&](auto iu) {
            constexpr int BASE = unit_base(D, 128, iu.value), W = unit_at(D, BASE, 128) / 16;
#pragma unroll
            for (int i = 0; i < 8; i++) {
                load_bytes<W * BITS / 8>(o.w[iu.value][i], value_at(p.c.v, at, i / 4, i % 4, ROWB, (BASE + r * W) * BITS / 8));
                if constexpr (KIND != KV_BF16 && !WIDE_SC)
                    o.sc[iu.value][i] = *value_at(p.c.vs, at, i / 4, i % 4, NB, (BASE + r * W) / 32);
            }
        });
        if constexpr (WIDE_SC) {
            // four tokens' scales, NB dwords
#pragma unroll
            for (int h = 0; h < 2; h++)
#pragma unroll
                for (int k = 0; k < NB; k += 4) load_bytes<(NB < 4 ? NB : 4) * 4>(&o.sc[h][k], value_at(p.c.vs, at, h, 0, NB, 4 * k));
        }
    };

    Place here, then;
    Keys keys;
    const int first = t0 + wave * TILE;
    if (first < tend) {
        place(here, first);
        load_keys(keys, here);
    }
    ISSUED;

    // the query, laid out as the score product's columns
    uint32_t q[QP][NB][4];
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
                        const Parts x = parts_of(static_cast<const float*>(p.q)[d + 2 * e]);
                        const Parts y = parts_of(static_cast<const float*>(p.q)[d + 2 * e + 1]);
                        q[0][BASE / 32 + f][e] = pack_hi(x.h, y.h);
                        q[QP - 2][BASE / 32 + f][e] = pack_hi(x.m, y.m);
                        q[QP - 1][BASE / 32 + f][e] = pack_hi(x.l, y.l);
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

    for (int tb = first; tb < tend; tb += AW * TILE) {
        Values val;
        load_values(val, here);
        const int next = tb + AW * TILE < tend ? tb + AW * TILE : tb;      // after the last tile: its keys again, unused
        place(then, next);
        ISSUED;

        // scores
        f4v z[2];
#pragma unroll
        for (int h = 0; h < 2; h++) {
            z[h] = f4v{0.f, 0.f, 0.f, 0.f};
            each<KU>([&](auto iu) {
                constexpr int BASE = unit_base(D, unit_max(KIND), iu.value), U = unit_at(D, BASE, unit_max(KIND));
                const uint32_t* w = keys.w[h][iu.value];
                float s = 1.f;
                if constexpr (WIDE_SC)
                    s = e8m0((keys.sc[h][BASE / 128] >> (BASE % 128 / 4)) >> (8 * (g * (U / 4) / 32)) & 0xffu);
                else if constexpr (KIND != KV_BF16)
                    s = e8m0(keys.sc[h][iu.value]);
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
        ISSUED;
        load_keys(keys, then);
        ISSUED;

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
        if (__any(zmax > m)) {                             // the maximum of some head grows
            const float mn = fmaxf(m, zmax);
            const float grow = exp2f(m - (mn == -INFINITY ? 0.f : mn));
            m = mn;
            l *= grow;
#pragma unroll
            for (int i = 0; i < D / 16; i++) acc[i] *= grow;
        }
        const float ms = m == -INFINITY ? 0.f : m;         // every score so far is -inf
        uint32_t pw[PP][4];                                // probabilities as bf16 pairs
#pragma unroll
        for (int i = 0; i < 4; i++) {
            float x = exp2f(z[i / 2][2 * (i % 2)] - ms), y = exp2f(z[i / 2][2 * (i % 2) + 1] - ms);
            l += x + y;
#pragma unroll
            for (int k = 0; k < PP; k++) {
                const f2v xy = {x, y};
                pw[k][i] = bits_of(__builtin_convertvector(xy, bf2v));
                x -= bitsf(pw[k][i] << 16);
                y -= bitsf(pw[k][i] & 0xffff0000u);
            }
        }

        // sums of p v
        const bool part = tb + TILE > tend;
        each<VU>([&](auto iu) {
            constexpr int BASE = unit_base(D, 128, iu.value), W = unit_at(D, BASE, 128) / 16;
            constexpr int WD = W * BITS / 8 < 4 ? 1 : W * BITS / 32;
            float s[8];
#pragma unroll
            for (int i = 0; i < 8; i++) {
                if constexpr (WIDE_SC) {
                    constexpr int NBW = NB;
                    const int n = (i % 4) * NBW + BASE / 32;               // byte of the first of this run's blocks
                    s[i] = e8m0((val.sc[i / 4][n / 4] >> (8 * (n % 4))) >> (8 * (r * W / 32)) & 0xffu);
                } else if constexpr (KIND != KV_BF16) {
                    s[i] = e8m0(val.sc[iu.value][i]);
                } else {
                    s[i] = 1.f;
                }
            }
            if (part) {
                // past the end: whatever the cache holds is taken as zero
#pragma unroll
                for (int i = 0; i < 8; i++)
                    if (tb + 16 * (i / 4) + 4 * g + i % 4 >= tend) {
                        s[i] = 1.f;
#pragma unroll
                        for (int k = 0; k < WD; k++) val.w[iu.value][i][k] = 0u;
                    }
            }
            each<W / 2>([&](auto pi) {
                constexpr int I = pi.value;
                uint32_t t[8];
#pragma unroll
                for (int i = 0; i < 8; i++) t[i] = pair_of<KIND, I>(val.w[iu.value][i], s[i]);
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
        here = then;
    }

    // the waves' triples, joined through LDS
    l += __shfl_xor(l, 16, 64);
    l += __shfl_xor(l, 32, 64);
    if (__any(bad)) l = bitsf(0x7fc00000u);
    float* sums = reinterpret_cast<float*>(smem);                  // [wave][head][LD]
    float* ml = sums + AW * nh * LD;                               // [wave][head][2]
    if (r < nh) {
        each<VU>([&](auto iu) {
            constexpr int BASE = unit_base(D, 128, iu.value), W = unit_at(D, BASE, 128) / 16;
#pragma unroll
            for (int i = 0; i < W; i++)
#pragma unroll
                for (int e = 0; e < 4; e++) sums[(wave * nh + r) * LD + BASE + (4 * g + e) * W + i] = acc[BASE / 16 + i][e];
        });
        if (g == 0) {
            ml[(wave * nh + r) * 2] = m;
            ml[(wave * nh + r) * 2 + 1] = l;
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < nh * D; i += 64 * AW) {
        const int h = i / D, d = i - h * D;
        float M = -INFINITY, L = 0.f, o = 0.f;
#pragma unroll
        for (int w = 0; w < AW; w++) M = fmaxf(M, ml[(w * nh + h) * 2]);
        const float Ms = M == -INFINITY ? 0.f : M;
#pragma unroll
        for (int w = 0; w < AW; w++) {
            const float f = exp2f(ml[(w * nh + h) * 2] - Ms);
            L += f * ml[(w * nh + h) * 2 + 1];
            o += f * sums[(w * nh + h) * LD + d];
        }
        const int64_t bh = b * p.q_heads + h0 + h;
        if (t0 == 0 && tend == len) {                      // the whole sequence
            const float v = L == 0.f ? 0.f : o / L;
            const int64_t at = b * p.o_ts + (int64_t)(h0 + h) * p.o_hs + d;
            if (QF32) static_cast<float*>(p.o)[at] = v;
            else static_cast<uint16_t*>(p.o)[at] = bf16_rne(v);
            if (p.lse && d == 0) p.lse[bh] = L == 0.f ? -INFINITY : (Ms + log2f(L)) * 0.69314718055994530942f;
        } else {
            const int64_t slots = p.workers + p.batch, at = (h0 + h) * slots + (int64_t)(blockIdx.x - plane * (uint32_t)p.workers) + b;
            p.parts[at * D + d] = o;
            if (d == 0) {
                float* x = p.parts + (int64_t)p.q_heads * slots * D + at * 2;
                x[0] = M;
                x[1] = L;
            }
        }
    }
    if (!p.workers) break;
    // the next sequence that holds anything
    u = before += units_of(len);
    if (u >= u_end) break;
    do b++; while (len_of(b) == 0);
    __syncthreads();                                       // the sums' LDS is used again
    }
}
#undef ISSUED

// Joins the parts of one sequence and query head, where it has several, and
// writes the empty ones: groups of D / 4 lanes (a power of two of them) take
// every JG-th part, four values a lane, then their
// triples are joined in order.
template <int D, bool QF32>
__global__ __launch_bounds__(256) void k_attend_join(AttendParams p) {
    constexpr int LG = D <= 64 ? 16 : D <= 128 ? 32 : 64, JG = 256 / LG, AHEAD = 4;
    __shared__ float so[JG][LG * 4], sm[JG], sl[JG];
    const int grp = threadIdx.x / LG, u = threadIdx.x % LG;
    const int64_t bh = blockIdx.x, b = bh / p.q_heads;
    const int h = (int)(bh - b * p.q_heads);
    const int64_t cap = p.cols * p.c.page;
    auto units = [&](int64_t i) {
        const int64_t n = p.lengths[i];
        return units_of((int)(n < 0 ? 0 : n > cap ? cap : n));
    };
    const int64_t n = units(b);
    int64_t t = n, before = 0;
    if (p.batch > 1) {
        __shared__ int64_t sh[256 / 64];
        int64_t mine = 0, less = 0;
        for (int64_t i = threadIdx.x; i < p.batch; i += 256) {
            const int64_t v = units(i);
            mine += v;
            if (i < b) less += v;
        }
        t = block_total<256>(mine, sh);
        before = block_total<256>(less, sh);
    }
    // the workers that hold its first and last unit
    const int64_t of = workers_used(t, p.workers);
    const int64_t from = n ? ((before + 1) * of - 1) / t : 0, to = n ? ((before + n) * of - 1) / t : 0;
    if (n && from == to) return;                     // finished there
    const int used = n ? (int)(to - from + 1) : 0;
    const int64_t slots = p.workers + p.batch, at0 = h * slots + from + b;
    const float* o = p.parts + at0 * D + (4 * u < D ? 4 * u : 0);
    const float* x = p.parts + (int64_t)p.q_heads * slots * D + at0 * 2;
    float M = -INFINITY, L = 0.f;
    f4v v = {0.f, 0.f, 0.f, 0.f};
    for (int i = grp; i < used; i += JG * AHEAD) {
        f4v a[AHEAD];
        float am[AHEAD], al[AHEAD];
#pragma unroll
        for (int k = 0; k < AHEAD; k++) {
            const int j = i + k * JG < used ? i + k * JG : i;
            a[k] = *reinterpret_cast<const f4v*>(o + (int64_t)j * D);
            am[k] = i + k * JG < used ? x[2 * j] : -INFINITY;
            al[k] = x[2 * j + 1];
        }
        float Mn = M;
#pragma unroll
        for (int k = 0; k < AHEAD; k++) Mn = fmaxf(Mn, am[k]);
        const float Ms = Mn == -INFINITY ? 0.f : Mn, old = exp2f(M - Ms);
        L *= old;
        v *= old;
#pragma unroll
        for (int k = 0; k < AHEAD; k++) {
            if (i + k * JG >= used) break;
            const float f = exp2f(am[k] - Ms);
            L += f * al[k];
            v += f * a[k];
        }
        M = Mn;
    }
    *reinterpret_cast<f4v*>(&so[grp][4 * u]) = v;
    if (u == 0) {
        sm[grp] = M;
        sl[grp] = L;
    }
    __syncthreads();
    if (threadIdx.x < D) {
        const int d = threadIdx.x;
        float Ma = -INFINITY, La = 0.f, s = 0.f;
#pragma unroll
        for (int k = 0; k < JG; k++) Ma = fmaxf(Ma, sm[k]);
        const float Ms = Ma == -INFINITY ? 0.f : Ma;
#pragma unroll
        for (int k = 0; k < JG; k++) {
            const float f = exp2f(sm[k] - Ms);
            La += f * sl[k];
            s += f * so[k][d];
        }
        const float r = La == 0.f ? 0.f : s / La;
        const int64_t at = b * p.o_ts + (int64_t)h * p.o_hs + d;
        if (QF32) static_cast<float*>(p.o)[at] = r;
        else static_cast<uint16_t*>(p.o)[at] = bf16_rne(r);
        if (p.lse && d == 0) p.lse[bh] = La == 0.f ? -INFINITY : (Ms + log2f(La)) * 0.69314718055994530942f;
    }
}

template <int D, int KIND, bool QF32, bool PAGE16, int AW>
hipError_t go(const AttendParams& p, hipStream_t s) {
    const int group = p.q_heads / p.c.heads, tiles = (group + QH - 1) / QH, rows = group < QH ? group : QH;
    const int64_t n = p.c.heads * tiles * (p.workers ? p.workers : p.batch);
    const int64_t joins = p.workers ? p.batch * p.q_heads : 0;
    if (!grid_ok(n, 64 * AW) || !grid_ok(joins, 256)) return TOO_LARGE;
    const int lds = AW * rows * (D + 3) * (int)sizeof(float);
    if (lds > 64 * 1024) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(k_attend<D, KIND, QF32, PAGE16, AW>),
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, lds);
        if (e != hipSuccess) return e;
    }
    k_attend<D, KIND, QF32, PAGE16, AW><<<(unsigned)n, 64 * AW, lds, s>>>(p);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !joins) return e;
    k_attend_join<D, QF32><<<(unsigned)joins, 256, 0, s>>>(p);
    return hipGetLastError();
}

template <int D, int KIND, bool QF32>
hipError_t pages(const AttendParams& p, hipStream_t s) {
    if constexpr (D <= EIGHT_MAX)
        if (p.waves == 8) return p.c.page % 16 ? go<D, KIND, QF32, false, 8>(p, s) : go<D, KIND, QF32, true, 8>(p, s);
    return p.c.page % 16 ? go<D, KIND, QF32, false, 4>(p, s) : go<D, KIND, QF32, true, 4>(p, s);
}
template <int D, bool QF32>
hipError_t pick(const AttendParams& p, hipStream_t s) {
    if (p.c.kind == KV_BF16) return pages<D, KV_BF16, QF32>(p, s);
    return p.c.kind == KV_FP8 ? pages<D, KV_FP8, QF32>(p, s) : pages<D, KV_FP4, QF32>(p, s);
}

template <int D, int KIND>
hipError_t write_as(const CacheWrite& p, bool bf, hipStream_t s) {
    constexpr int PER = CT / (D / 8);
    const int64_t n = p.tokens * p.c.heads;
    if (!grid_ok((n + PER - 1) / PER, CT)) return TOO_LARGE;
    const unsigned grid = (unsigned)((n + PER - 1) / PER);
    if (bf) k_cache_write<D, KIND, true><<<grid, CT, 0, s>>>(p);
    else k_cache_write<D, KIND, false><<<grid, CT, 0, s>>>(p);
    return hipGetLastError();
}
template <int D>
hipError_t write_dim(const CacheWrite& p, bool bf, hipStream_t s) {
    if (p.c.kind == KV_BF16) return write_as<D, KV_BF16>(p, bf, s);
    return p.c.kind == KV_FP8 ? write_as<D, KV_FP8>(p, bf, s) : write_as<D, KV_FP4>(p, bf, s);
}

}  // namespace

hipError_t launch_cache_write(CacheWrite p, bool bf, hipStream_t s) {
    p.per_token = div_by(p.c.heads);
    p.page_div = div_by(p.c.page);
    p.page_shift = -1;
    if ((p.c.page & (p.c.page - 1)) == 0) p.page_shift = __builtin_ctz((unsigned)p.c.page);
    switch (p.c.dim) {
    case 64: return write_dim<64>(p, bf, s);
    case 96: return write_dim<96>(p, bf, s);
    case 128: return write_dim<128>(p, bf, s);
    case 192: return write_dim<192>(p, bf, s);
    default: return write_dim<256>(p, bf, s);
    }
}

bool attend_dim_ok(int d) { return d == 64 || d == 96 || d == 128 || d == 192 || d == 256; }

// pairs of a key-value head and 16 of its query heads
static int64_t planes_of(const KvCache& c, int q_heads) { return (int64_t)c.heads * ((q_heads / c.heads + QH - 1) / QH); }
constexpr int64_t FULL = 256;          // whole sequences that fill the chip, one for each CU

// How a call is split.  Short sequences (one tile a wave, or four if there are
// enough of them to fill the chip): eight waves take a whole one and no join
// follows (32 sequences of 777: 17 us, shared out 25; one of 777: 12 us, shared
// out 9.8).  Others: workers, one workgroup of four waves for each CU where a
// token's row is 256 bytes or more, so that four waves keep enough in flight,
// three where it is less (us with 256 workgroups and with 768, 32 sequences up
// to 8192 tokens of 128 values: bf16 106 and 120, MXFP8 84 and 68, MXFP4 71 and
// 52; bf16 of 64 values, half the tokens: 44 and 37).  Those are pages of a
// multiple of 16 and bf16 queries, whose registers (up to 168) let a CU hold the
// three.  Of the 44 variants below 256 bytes 29 hold one or two (other pages or
// fp32 queries at 96 and 128 values, fp32 queries of other pages at 64, all at
// 192 and 256) and run the 768 in rounds; their counts were not measured.
AttendPlan attend_plan(const KvCache& c, int64_t batch, int q_heads, int64_t cols) {
    const int64_t planes = planes_of(c, q_heads), longest = cols * c.page;
    if (c.dim <= EIGHT_MAX && (longest <= 8 * TILE || (longest <= 8 * TILE * 4 && batch * planes >= FULL))) return AttendPlan{8, 0};
    const int64_t want = c.dim * kind_bits(c.kind) / 8 >= 256 ? 256 : 768;
    int64_t workers = (want + planes - 1) / planes;
    const int64_t most = batch * ((longest + UNIT - 1) / UNIT);
    if (workers > most) workers = most;
    return AttendPlan{4, (int)(workers < 1 ? 1 : workers)};
}

// Workers and slots grow with batch and columns, but for one step: a batch that
// fills the chip with whole sequences needs none where a smaller one does.
int64_t attend_slots(const KvCache& c, int64_t batch, int q_heads, int64_t cols) {
    AttendPlan a = attend_plan(c, batch, q_heads, cols);
    if (!a.workers) {
        const int64_t most = (FULL - 1) / planes_of(c, q_heads);
        if (batch > most) batch = most;
        a = attend_plan(c, batch, q_heads, cols);
    }
    return a.workers && batch ? a.workers + batch : 0;
}

hipError_t launch_attend(AttendParams p, bool bf, hipStream_t s) {
    p.page_div = div_by(p.c.page);
    switch (p.c.dim) {
    case 64: return bf ? pick<64, false>(p, s) : pick<64, true>(p, s);
    case 96: return bf ? pick<96, false>(p, s) : pick<96, true>(p, s);
    case 128: return bf ? pick<128, false>(p, s) : pick<128, true>(p, s);
    case 192: return bf ? pick<192, false>(p, s) : pick<192, true>(p, s);
    default: return bf ? pick<256, false>(p, s) : pick<256, true>(p, s);
    }
}

}  // namespace mxk
