// attend_shared.hip -- attention of one new token per sequence where the
// sequences share a long prefix.
//
// Mathematics.  A softmax over the prefix's and a sequence's own tokens joins
// from the triples (m, sum p, sum p v) of any split of them.  The prefix's keys
// and values are the same for every sequence, so for one key-value head the
// query heads of all sequences are the rows of one matrix product with them:
// `batch x group` rows, each cached value read once for all.  The own tokens
// are k_attend's, which leaves all its triples unjoined; k_shared_join adds
// both kinds up.
//
// Bound and measured (32 query and 8 key-value heads of 128).  Few rows: memory;
// 4 sequences behind 65536 bf16 tokens 61 us in all, 4.4 TB/s of cache.  Many:
// issue slots, most of them the vector unit's (softmax, conversion of cached
// values to bf16, two bf16 parts of every probability).  64 sequences behind 32768
// MXFP8 tokens: 63 us for the prefix (fp32 queries, three parts of both: 123), 830
// TFLOP/s of matrix instructions, of which the second part of the probabilities
// takes 11 (one part: 52 us; it would double the squared error against 64 bits,
// so it stays).  Of 148 thousand cycles a SIMD's matrix unit works 50 and its
// vector unit 53; a wave waits 37 % of its time for issue and 32 % for loads, LDS
// or a barrier.  Tried there: 4 waves to a workgroup, two of those on a CU, one
// copy of each tile and two barriers a step 66 us; two groups of waves half a
// period apart 72 to 80; instruction order by scheduling groups within 1 us of
// the compiler's.
#include "attend_device.hpp"

namespace mxk {
using namespace mxd;

namespace {

typedef float f16v __attribute__((ext_vector_type(16)));
typedef short s4v __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s4v lds_s4v;

// Waves of a workgroup: two on a SIMD where their registers let them.
constexpr int waves_of(int D, bool qf32, bool one = false) { return D <= 128 && !qf32 && !one ? 8 : 4; }
// Tokens of a tile: 32 for each wave side by side along them.
constexpr int tile_tokens(int waves, int rw) { return 32 * waves / rw; }
// Pages whose places are held at a time
constexpr int TABLE = 1024;
// Tokens that a range of the prefix is a multiple of
constexpr int UT = 64;
// Maxima beyond this take the score's product with the scale rounded on its own:
// a product that is not, less a maximum that was, is off by half the maximum's
// unit, 2^-4 here and past what 2^x holds from 2^31 on.
constexpr float FAR = 0x1p20f;
// LDS row strides in bytes.  Keys: 8 lanes of a 16-byte read take 8 rows, whose
// starts are then 4 banks apart or a multiple of it, all different.  Values: the
// transposing read takes 64 bytes of 4 rows, a quarter of the banks each.
constexpr int key_stride(int D) { return D * 2 + 16; }
constexpr int value_stride(int D) { return D * 2 + ((D * 2) % 128 == 0 ? 64 : 0); }
constexpr int tile_bytes(int D, int tk) { return tk * (key_stride(D) + value_stride(D)); }
// a wave's triples: D / 2 values and two statistics a lane
constexpr int triple_bytes(int D) { return 64 * 4 * (D / 2 + 2); }
constexpr int lds_bytes(int D, int waves, int rw) {
    const int tiles = 2 * tile_bytes(D, tile_tokens(waves, rw)), join = waves / 2 * triple_bytes(D);
    return rw == waves || tiles > join ? tiles : join;
}

// One tile of RW x 32 rows and one range of the prefix's tokens.
//
// RW of the W waves stand along the rows, W / RW along the tokens.  The
// 32 x 32 x 16 instruction takes tokens as rows and query rows as columns, so a
// lane holds 16 scores of one query row and the row's maximum is a maximum over
// registers and one exchange; the scores' layout is the column operand of the
// second product when its K order is (8-token run, half of the wave, token),
// which the transposing LDS read of the values follows.
//
// Keys and values lie in LDS twice over, so a step takes one barrier.  In step j
// a wave forms the scores of tile j + 1, the softmax of tile j and its sums, and
// converts its share of the values of tile j + 1 and the keys of tile j + 2 from
// the registers they were loaded to SLOTS steps before.  What is independent in
// that keeps the matrix and the vector unit busy at once.
//
// ONE: every range is one tile, so there is nothing to load ahead and four waves
// do (4 sequences behind 777 bf16 tokens: 7.2 us, with the other form 13).
template <int D, int KIND, bool QF32, int RW, bool ONE>
__global__ __launch_bounds__(64 * waves_of(D, QF32, ONE), waves_of(D, QF32, ONE) / 4) void k_prefix(SharedParams p) {
    constexpr int W = waves_of(D, QF32, ONE), ST = 64 * W, TW = W / RW, TK = tile_tokens(W, RW), RT = 32 * RW;
    constexpr int QP = QF32 ? 3 : 1, PP = QF32 ? 3 : 2;            // bf16 parts of a query and of a probability
    constexpr int BITS = kind_bits(KIND), ROWB = D * BITS / 8, NB = D / 32;
    constexpr int CPR = ROWB / 16, VALS = 128 / BITS;              // 16-byte chunks of a row, values of one
    constexpr int CHUNKS = TK * CPR, NC = (CHUNKS + ST - 1) / ST;
    constexpr int KS = key_stride(D), VS = value_stride(D);
    // tiles whose bytes are on their way: two where that takes 32 registers, else one (of at least as many bytes)
    constexpr int SLOTS = NC <= 2 ? 2 : 1;
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    __shared__ int bad_page;
    __shared__ int64_t table[TABLE];                               // where the pages' keys and values begin, in bytes

    const AttendParams& a = p.own;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int c = lane & 31, half = lane >> 5;
    const int rw = wave % RW, tw = wave / RW;
    uint8_t *sk = smem, *sv = smem + 2 * TK * KS;                  // tile j's lie at j % 2
    const int group = a.q_heads / a.c.heads;
    const uint32_t rows = (uint32_t)a.batch * (uint32_t)group, row_tiles = (rows + RT - 1) / RT;      // below 2^31
    // every eighth workgroup runs on the same XCD: a range's tiles of rows go
    // there one after the other, so that all but the first find it in its L2
    const uint32_t turn = blockIdx.x / 8u, eight = turn / row_tiles;
    const uint32_t rt = turn - eight * row_tiles, pair = eight * 8u + blockIdx.x % 8u;
    const int kvh = (int)(pair / (uint32_t)p.splits), split = (int)(pair - (uint32_t)kvh * (uint32_t)p.splits);
    const int64_t cap = p.prefix_cols * a.c.page;
    const int64_t n = *p.prefix_length;
    const int len = (int)(n < 0 ? 0 : n > cap ? cap : n);
    const int units = (len + UT - 1) / UT, of = units < p.splits ? units : p.splits;
    if (split >= of || kvh >= a.c.heads) return;
    const int t0 = (int)((int64_t)split * units / of) * UT;
    const int t1 = (int)((int64_t)(split + 1) * units / of) * UT, tend = t1 < len ? t1 : len;
    // a scale of 0 as one that rounds every finite score to 0: 0 times a masked
    // -Inf would be no mask
    const float zs = a.scale == 0.f ? 0x1p-149f : __builtin_fabsf(a.scale) * 1.44269504088896340736f;
    const uint32_t flip = a.scale < 0.f ? 0x80008000u : 0u;        // a negative scale's sign goes to the query
    const uint32_t row0 = rt * RT + 32 * rw;                       // this wave's first row
    const bool active = row0 < rows;
    if (threadIdx.x == 0) bad_page = 0;

    // A tile's cached bytes on their way to LDS; a row's place in the cache.
    struct Bytes {
        uint32_t w[NC][4], sc[KIND == KV_BF16 ? 1 : NC];
    };
    struct Places {
        int64_t at[NC];                                            // bytes from the first key or value
    };
    int c0 = 0, cend = 0, base = 0;                                // tokens whose pages the table holds, its first page
    auto at_of = [&](int j) { return c0 + j * TK; };               // first token of tile j
    auto chunk = [&](int i) { return CHUNKS % ST == 0 || tid + ST * i < CHUNKS ? tid + ST * i : CHUNKS - 1; };
    // a token past the end counts as the last
    auto place = [&](Places& o, int j) {
#pragma unroll
        for (int i = 0; i < NC; i++) {
            const int at = at_of(j) + chunk(i) / CPR, t = at < cend ? at : cend - 1;
            const uint32_t pg = over((uint32_t)t, a.page_div);
            o.at[i] = table[pg - base] + (uint32_t)((t - (int)pg * a.c.page) * ROWB + chunk(i) % CPR * 16);
        }
    };
    auto load = [&](Bytes& o, const Places& at, const uint8_t* codes, const uint8_t* scales) {
#pragma unroll
        for (int i = 0; i < NC; i++) {
            load_bytes<16>(o.w[i], codes + at.at[i]);
            if constexpr (KIND != KV_BF16) o.sc[i] = scales[at.at[i] >> (KIND == KV_FP8 ? 5 : 4)];      // a block's bytes
        }
    };
    auto store = [&](const Bytes& o, uint8_t* to, int stride) {
#pragma unroll
        for (int i = 0; i < NC; i++) {
            if (CHUNKS % ST && tid + ST * i >= CHUNKS) break;
            const int token = chunk(i) / CPR, ch = chunk(i) % CPR;
            const float s = KIND == KV_BF16 ? 1.f : e8m0(o.sc[KIND == KV_BF16 ? 0 : i]);
            each<VALS / 8>([&](auto jc) {
                constexpr int J = 4 * jc.value;
                *reinterpret_cast<u32x4*>(to + token * stride + ch * VALS * 2 + 4 * J) =
                    u32x4{pair_of<KIND, J>(o.w[i], s), pair_of<KIND, J + 1>(o.w[i], s), pair_of<KIND, J + 2>(o.w[i], s),
                          pair_of<KIND, J + 3>(o.w[i], s)};
            });
        }
    };
    // past the end: values count as zero
    auto cut = [&](Bytes& o, int j) {
        if (at_of(j) + TK <= cend) return;
#pragma unroll
        for (int i = 0; i < NC; i++)
            if (at_of(j) + chunk(i) / CPR >= cend) {
#pragma unroll
                for (int e = 0; e < 4; e++) o.w[i][e] = 0u;
                if constexpr (KIND != KV_BF16) o.sc[i] = 127u;
            }
    };

    // this lane's query row as the score product's columns
    uint32_t q[QP][D / 16][4];
    {
        const uint32_t m = row0 + c < rows ? row0 + c : rows - 1, b = m / (uint32_t)group;
        const int64_t at = b * a.q_ts + (int64_t)(kvh * group + (int)(m - b * group)) * a.q_hs + 8 * half;
#pragma unroll
        for (int k = 0; k < D / 16; k++) {
            if constexpr (QF32) {
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const Parts x = parts_of(static_cast<const float*>(a.q)[at + 16 * k + 2 * e]);
                    const Parts y = parts_of(static_cast<const float*>(a.q)[at + 16 * k + 2 * e + 1]);
                    q[0][k][e] = pack_hi(x.h, y.h) ^ flip;
                    q[QP - 2][k][e] = pack_hi(x.m, y.m) ^ flip;
                    q[QP - 1][k][e] = pack_hi(x.l, y.l) ^ flip;
                }
            } else {
                load_bytes<16>(q[0][k], reinterpret_cast<const uint8_t*>(static_cast<const uint16_t*>(a.q) + at + 16 * k));
#pragma unroll
                for (int e = 0; e < 4; e++) q[0][k][e] ^= flip;
            }
        }
    }

    f16v acc[D / 32], z[2];                                        // z: scores, tile j's at j % 2
#pragma unroll
    for (int i = 0; i < D / 32; i++)
#pragma unroll
        for (int e = 0; e < 16; e++) acc[i][e] = 0.f;
    float m = -INFINITY, l = 0.f;                                  // of row c; l: this lane's tokens
    bool far = false;                                              // some row's maximum lies beyond FAR
    uint32_t pw[PP][2][4];                                         // probabilities as bf16 pairs
    const int tk = 32 * tw;                                        // this wave's tokens in the tile

    // values of 16 tokens as the second product's rows: of 16 lanes, four at a row's 16 values
    const uint8_t* vat = sv + (tk + 4 * half + (c % 16) / 4) * VS + (c / 16) * 32 + (c % 4) * 8;
    const uint8_t* kat = sk + (tk + c) * KS + 16 * half;
    auto value = [&](int buf, int s, int i) {
        const uint8_t* at = vat + buf * TK * VS + 16 * s * VS + 64 * i;
        const s4v lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4v*)at);
        const s4v hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4v*)(at + 8 * VS));
        return __builtin_bit_cast(bf8v, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    };
    auto column = [&](const uint32_t (&w)[4]) { return frag(w[0], w[1], w[2], w[3]); };
    auto scores = [&](auto bc) {
        constexpr int B = bc.value;
#pragma unroll
        for (int e = 0; e < 16; e++) z[B][e] = 0.f;
#pragma unroll
        for (int k = 0; k < D / 16; k++) {
            const bf8v x = *reinterpret_cast<const bf8v*>(kat + B * TK * KS + 32 * k);
#pragma unroll
            for (int i = 0; i < QP; i++) z[B] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x, column(q[i][k]), z[B], 0, 0, 0);
        }
    };
    auto sums = [&](auto bc) {
#pragma unroll
        for (int s = 0; s < 2; s++)
#pragma unroll
            for (int i = 0; i < D / 32; i++) {
                const bf8v x = value(bc.value, s, i);
#pragma unroll
                for (int k = 0; k < PP; k++) acc[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x, column(pw[k][s]), acc[i], 0, 0, 0);
            }
    };
    // the row's maximum, and what it takes along when it moves
    auto peak = [&](auto bc, int j) {
        f16v& y = z[bc.value];
        const int first = at_of(j) + tk;
        if (first + 32 > cend) {
#pragma unroll
            for (int e = 0; e < 16; e++)
                if (first + 8 * (e / 4) + 4 * half + e % 4 >= cend) y[e] = -INFINITY;
        }
        float zmax = y[0];
#pragma unroll
        for (int e = 1; e < 16; e++) zmax = fmaxf(zmax, y[e]);
        // the other half's of the same row, without LDS
        const auto both = __builtin_amdgcn_permlane32_swap(fbits(zmax), fbits(zmax), false, false);
        zmax = fmaxf(bitsf(both[0]), bitsf(both[1])) * zs;
        // Any number from the maximum up to a little more does for m, so that no
        // probability is above 1.  It keeps 2^4 ahead and follows where a row's
        // maximum has outgrown it, seldom after the first tile (the 63 us are 69
        // to 71 with none, 63 to 65 with 2^2); what the exponential gives as 0,
        // below 2^-126, is then below 2^-122 of the likeliest.
        if (__any(zmax > m)) {
            const float mn = fmaxf(m, zmax + 4.f);
            const float grow = __builtin_amdgcn_exp2f(m - (mn == -INFINITY ? 0.f : mn));
            m = mn;
            far = __any(m != -INFINITY && __builtin_fabsf(m) > FAR);
            l *= grow;
#pragma unroll
            for (int i = 0; i < D / 32; i++) acc[i] *= grow;
        }
        if (far) {
            const float ms = m == -INFINITY ? 0.f : m;
#pragma unroll
            for (int e = 0; e < 16; e++) y[e] = y[e] * zs - ms;
        }
    };
    auto softmax = [&](auto bc) {
        const f16v& y = z[bc.value];
        const float by = far ? 1.f : zs;
        const float ms = far || m == -INFINITY ? 0.f : m;          // -inf: every score so far is
#pragma unroll
        for (int i = 0; i < 8; i++) {
            float u = __builtin_amdgcn_exp2f(__builtin_fmaf(y[2 * i], by, -ms));
            float v = __builtin_amdgcn_exp2f(__builtin_fmaf(y[2 * i + 1], by, -ms));
            l += u + v;
#pragma unroll
            for (int k = 0; k < PP; k++) {
                const f2v uv = {u, v};
                pw[k][i / 4][i % 4] = bits_of(__builtin_convertvector(uv, bf2v));
                u -= bitsf(pw[k][i / 4][i % 4] << 16);
                v -= bitsf(pw[k][i / 4][i % 4] & 0xffff0000u);
            }
        }
    };
    // The tiles of the tokens whose pages are in the table.  Every load is made,
    // those past the end of the last row again, so that the compiler can count
    // which are still under way; a tile past the end has no score above -Inf.
    auto run = [&](auto work, int steps) {
        constexpr bool WORK = work.value;
        // bytes of values from tile j + 1 on and of keys from tile j + 2 on, and
        // where the next ones lie
        Bytes keys[SLOTS], vals[SLOTS];
        Places now, next;
        {
            Places first;
            Bytes k0, k1, v0;
            place(first, 0);
            load(k0, first, a.c.k, a.c.ks);
            load(v0, first, a.c.v, a.c.vs);
            place(first, 1);
            load(k1, first, a.c.k, a.c.ks);
            load(vals[0], first, a.c.v, a.c.vs);
            place(first, 2);
            load(keys[0], first, a.c.k, a.c.ks);
            if constexpr (SLOTS > 1) {
                load(vals[SLOTS - 1], first, a.c.v, a.c.vs);
                place(first, 3);
                load(keys[SLOTS - 1], first, a.c.k, a.c.ks);
            }
            now = first;                                           // of tile SLOTS + 1
            cut(v0, 0);
            store(k0, sk, KS);
            store(v0, sv, VS);
            store(k1, sk + TK * KS, KS);
        }
        __syncthreads();
        if constexpr (WORK) scores(ic<0>{});
        __syncthreads();
        // S: j modulo SLOTS, B: j modulo 2
        auto step = [&](int j, auto sc, auto bc) {
            constexpr int S = sc.value, B = bc.value;
            place(next, j + SLOTS + 2);
            if constexpr (WORK) {
                peak(bc, j);
                scores(ic<1 - B>{});
                softmax(bc);
                sums(bc);
            }
            cut(vals[S], j + 1);
            store(vals[S], sv + (1 - B) * TK * VS, VS);            // of tile j + 1
            store(keys[S], sk + B * TK * KS, KS);                  // of tile j + 2
            load(vals[S], now, a.c.v, a.c.vs);
            load(keys[S], next, a.c.k, a.c.ks);
            now = next;
            __syncthreads();
        };
        for (int j = 0; j < steps; j += 2) {
            step(j, ic<0>{}, ic<0>{});
            if (j + 1 < steps) step(j + 1, ic<SLOTS - 1>{}, ic<1>{});
        }
    };
    for (c0 = t0; c0 < tend; c0 = cend) {
        const uint32_t first = over((uint32_t)c0, a.page_div);
        const int64_t most = (int64_t)(first + TABLE) * a.c.page / TK * TK;      // whole tiles, but for the last
        base = (int)first;
        cend = most < tend ? (int)most : tend;
        const int held = (int)over((uint32_t)(cend - 1), a.page_div) - base + 1;
        __syncthreads();                                           // nobody reads the table or a tile
        for (int i = threadIdx.x; i < held; i += ST) {
            int64_t page = p.prefix[base + i];
            if (page < 0 || page >= a.c.pages) {
                page = 0;
                bad_page = 1;
            }
            table[i] = (page * a.c.heads + kvh) * a.c.page * ROWB;
        }
        __syncthreads();
        const int steps = (cend - c0 + TK - 1) / TK;
        if constexpr (ONE) {
            Places first;
            Bytes k0, v0;
            place(first, 0);
            load(k0, first, a.c.k, a.c.ks);
            load(v0, first, a.c.v, a.c.vs);
            cut(v0, 0);
            store(k0, sk, KS);
            store(v0, sv, VS);
            __syncthreads();
            if (active) {
                scores(ic<0>{});
                peak(ic<0>{}, 0);
                softmax(ic<0>{});
                sums(ic<0>{});
            }
        } else if (active) {
            run(ic<1>{}, steps);
        } else {
            run(ic<0>{}, steps);
        }
    }
    l += __shfl_xor(l, 32, 64);
    __syncthreads();
    if (bad_page) l = bitsf(0x7fc00000u);

    // The waves along the tokens join in LDS, the upper half of them into the
    // lower until one is left; a lane's place is the same in all.
    constexpr int PER = 64 * (D / 2 + 2);
    float* st = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int left = TW / 2; left; left /= 2) {
        float* box = st + ((tw % left) * RW + rw) * PER + 4 * lane;
        float* ml = st + ((tw % left) * RW + rw) * PER + 64 * (D / 2) + lane;
        if (tw >= left && tw < 2 * left) {
#pragma unroll
            for (int i = 0; i < D / 32; i++)
#pragma unroll
                for (int e = 0; e < 16; e += 4)
                    *reinterpret_cast<f4v*>(box + (i * 4 + e / 4) * 256) = f4v{acc[i][e], acc[i][e + 1], acc[i][e + 2], acc[i][e + 3]};
            ml[0] = m;
            ml[64] = l;
        }
        __syncthreads();
        if (tw < left) {
            const float om = ml[0], ol = ml[64], M = fmaxf(m, om), Ms = M == -INFINITY ? 0.f : M;
            const float f = __builtin_amdgcn_exp2f(m - Ms), g = __builtin_amdgcn_exp2f(om - Ms);
            m = M;
            l = f * l + g * ol;
#pragma unroll
            for (int i = 0; i < D / 32; i++)
#pragma unroll
                for (int e = 0; e < 16; e += 4) {
                    const f4v o = *reinterpret_cast<const f4v*>(box + (i * 4 + e / 4) * 256);
#pragma unroll
                    for (int x = 0; x < 4; x++) acc[i][e + x] = f * acc[i][e + x] + g * o[x];
                }
        }
        __syncthreads();
    }
    if (tw == 0 && row0 + c < rows) {
        const int64_t wg = ((int64_t)kvh * row_tiles + rt) * p.splits + split;
        float* out = p.parts + wg * RT * D + (32 * rw + c) * D;
        float* ml = p.parts + (int64_t)a.c.heads * row_tiles * p.splits * (RT * D) + wg * RT * 2 + 2 * (32 * rw + c);
#pragma unroll
        for (int i = 0; i < D / 32; i++)
#pragma unroll
            for (int e = 0; e < 16; e += 4)
                *reinterpret_cast<f4v*>(out + 32 * i + 2 * e + 4 * half) = f4v{acc[i][e], acc[i][e + 1], acc[i][e + 2], acc[i][e + 3]};
        if (half == 0) {
            ml[0] = m;
            ml[1] = l;
        }
    }
}
// Joins the parts of one sequence and query head, those of the prefix and those
// of its own tokens: groups of D / 4 lanes (a power of two of them) take every
// JG-th part, four values a lane, then their triples are joined in order.
template <int D, bool QF32>
__global__ __launch_bounds__(256) void k_shared_join(SharedParams p) {
    constexpr int LG = D <= 64 ? 16 : D <= 128 ? 32 : 64, JG = 256 / LG, AHEAD = 4;
    __shared__ float so[JG][LG * 4], sm[JG], sl[JG];
    const AttendParams& a = p.own;
    const int grp = threadIdx.x / LG, u = threadIdx.x % LG;
    // 32 bits: a division of 64 takes longer than everything else here
    const uint32_t bh = blockIdx.x, b = bh / (uint32_t)a.q_heads;
    const int h = (int)(bh - b * (uint32_t)a.q_heads);
    // the prefix's
    const int group = a.q_heads / a.c.heads, kvh = h / group, RT = 32 * p.row_waves;
    const int lg = 5 + __builtin_ctz(p.row_waves);
    int front = 0;
    const float *fo = nullptr, *fx = nullptr;
    if (p.splits) {
        const int64_t cap = p.prefix_cols * a.c.page, n = *p.prefix_length;
        const int len = (int)(n < 0 ? 0 : n > cap ? cap : n), units = (len + UT - 1) / UT;
        front = units < p.splits ? units : p.splits;
        const uint32_t rows = (uint32_t)a.batch * (uint32_t)group, row_tiles = (rows + RT - 1) >> lg;
        const uint32_t m = b * group + (h - kvh * group), rt = m >> lg;
        const int64_t at = ((int64_t)kvh * row_tiles + rt) * p.splits * RT + (m - (rt << lg));
        fo = p.parts + at * D;
        fx = p.parts + (int64_t)a.c.heads * row_tiles * p.splits * RT * D + at * 2;
    }
    // its own
    const int64_t cap = a.cols * a.c.page;
    auto units = [&](int64_t i) {
        const int64_t n = a.lengths[i];
        return units_of((int)(n < 0 ? 0 : n > cap ? cap : n));
    };
    const int64_t n = units(b);
    int64_t from = 0;
    int back = n ? 1 : 0;
    if (a.workers) {
        __shared__ int64_t sh[256 / 64];
        int64_t mine = 0, less = 0;
        for (int64_t i = threadIdx.x; i < a.batch; i += 256) {
            const int64_t v = units(i);
            mine += v;
            if (i < b) less += v;
        }
        const int64_t t = block_total<256>(mine, sh), before = block_total<256>(less, sh);
        if (n) {                                     // the workers that hold its first and last unit
            const int64_t of = workers_used(t, a.workers);
            from = ((before + 1) * of - 1) / t;
            back = (int)(((before + n) * of - 1) / t - from + 1);
        }
    }
    const int64_t slots = a.workers + a.batch, at0 = h * slots + from + b;
    const float *bo = a.parts + at0 * D, *bx = a.parts + (int64_t)a.q_heads * slots * D + at0 * 2;
    const int used = front + back, d = 4 * u < D ? 4 * u : 0;

    float M = -INFINITY, L = 0.f;
    f4v v = {0.f, 0.f, 0.f, 0.f};
    for (int i = grp; i < used; i += JG * AHEAD) {
        f4v s[AHEAD];
        float am[AHEAD], al[AHEAD];
#pragma unroll
        for (int k = 0; k < AHEAD; k++) {
            const int j = i + k * JG < used ? i + k * JG : i;
            const float* o = j < front ? fo + (int64_t)j * RT * D : bo + (int64_t)(j - front) * D;
            const float* x = j < front ? fx + (int64_t)j * RT * 2 : bx + (int64_t)(j - front) * 2;
            s[k] = *reinterpret_cast<const f4v*>(o + d);
            am[k] = i + k * JG < used ? x[0] : -INFINITY;
            al[k] = x[1];
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
            v += f * s[k];
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
        const int e = threadIdx.x;
        float Ma = -INFINITY, La = 0.f, s = 0.f;
#pragma unroll
        for (int k = 0; k < JG; k++) Ma = fmaxf(Ma, sm[k]);
        const float Ms = Ma == -INFINITY ? 0.f : Ma;
#pragma unroll
        for (int k = 0; k < JG; k++) {
            const float f = exp2f(sm[k] - Ms);
            La += f * sl[k];
            s += f * so[k][e];
        }
        const float r = La == 0.f ? 0.f : s / La;
        const int64_t at = b * a.o_ts + (int64_t)h * a.o_hs + e;
        if (QF32) static_cast<float*>(a.o)[at] = r;
        else static_cast<uint16_t*>(a.o)[at] = bf16_rne(r);
        if (a.lse && e == 0) a.lse[bh] = La == 0.f ? -INFINITY : (Ms + log2f(La)) * 0.69314718055994530942f;
    }
}

int64_t prefix_blocks(const SharedParams& p) {
    const int64_t rows = p.own.batch * (p.own.q_heads / p.own.c.heads), rt = 32 * p.row_waves;
    return ((int64_t)p.own.c.heads * p.splits + 7) / 8 * 8 * ((rows + rt - 1) / rt);
}

template <int D, int KIND, bool QF32, int RW, bool ONE>
hipError_t go(const SharedParams& p, hipStream_t s) {
    constexpr int W = waves_of(D, QF32, ONE), lds = lds_bytes(D, W, RW);
    static_assert(lds + 8 * TABLE + 64 <= 160 * 1024, "LDS of a CU");
    if (lds + 8 * TABLE + 64 > 64 * 1024) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(k_prefix<D, KIND, QF32, RW, ONE>),
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, lds);
        if (e != hipSuccess) return e;
    }
    k_prefix<D, KIND, QF32, RW, ONE><<<(unsigned)prefix_blocks(p), 64 * W, lds, s>>>(p);
    return hipGetLastError();
}
template <int D, int KIND, bool QF32>
hipError_t rows(const SharedParams& p, hipStream_t s) {
    if constexpr (waves_of(D, QF32) == 8)
        if (p.row_waves == 8) return go<D, KIND, QF32, 8, false>(p, s);
    if (p.one) return go<D, KIND, QF32, 2, true>(p, s);
    if constexpr (KIND != KV_BF16)
        if (p.row_waves == 2) return go<D, KIND, QF32, 2, false>(p, s);
    return go<D, KIND, QF32, 4, false>(p, s);
}
template <int D, bool QF32>
hipError_t pick(const SharedParams& p, hipStream_t s) {
    if (p.splits) {
        const hipError_t e = p.own.c.kind == KV_BF16  ? rows<D, KV_BF16, QF32>(p, s)
                             : p.own.c.kind == KV_FP8 ? rows<D, KV_FP8, QF32>(p, s)
                                                      : rows<D, KV_FP4, QF32>(p, s);
        if (e != hipSuccess) return e;
    }
    k_shared_join<D, QF32><<<(unsigned)(p.own.batch * p.own.q_heads), 256, 0, s>>>(p);
    return hipGetLastError();
}

}  // namespace

constexpr int FULL = 256;              // workgroups that fill the chip: one for each CU

// Tiles of 64, 128 or 256 rows (waves of rows that do not exist stand idle, which
// few rows leave them time for), and as many ranges of tokens as fill the chip
// once.  64 rows stand with twice the tokens of 128 in a tile, for which a bf16
// cache lacks registers: 4 sequences (16 rows) behind 65536 tokens take 53 us so
// and 61 in tiles of 128 rows from MXFP8, 49 and 60 from MXFP4, but 63 and 61
// from bf16.  A prefix that 64-token ranges cover takes those.
// Ranges are whole, so where the tiles do not divide 256 some CUs stand idle: 8
// key-value heads of 256, 16 query heads each, 8192 bf16 tokens take 245 us for 96
// sequences (192 workgroups), 252 for 128 (256), 475 for 136 (136), 493 for 256.
SharedPlan shared_plan(const KvCache& c, int64_t batch, int q_heads, int64_t prefix_cols, bool q_bf16) {
    const int64_t rows = batch * (q_heads / c.heads), units = (prefix_cols * c.page + UT - 1) / UT;
    SharedPlan o;
    o.one = rows <= 64 && units <= FULL / c.heads;
    o.row_waves = o.one || (rows <= 64 && c.kind != KV_BF16) ? 2 : rows <= 128 || waves_of(c.dim, !q_bf16) == 4 ? 4 : 8;
    o.planes = c.heads * ((rows + 32 * o.row_waves - 1) / (32 * o.row_waves));
    int64_t splits = o.planes ? FULL / o.planes : 1;
    if (splits < 1) splits = 1;
    o.splits = (int)(splits < units ? splits : units);
    return o;
}

// Parts, in rows: planes x splits is at most FULL or the planes, and at most
// planes x units; the planes and the units (of 64 tokens) grow with their
// arguments, the rows of a tile with the batch (in fp32 they stop at 128).
int64_t shared_rows(const KvCache& c, int64_t batch, int q_heads, int64_t prefix_cols) {
    if (!batch || !prefix_cols) return 0;
    const int64_t units = (prefix_cols * c.page + UT - 1) / UT;
    int64_t most = 0;
    for (const bool bf : {true, false}) {
        const SharedPlan o = shared_plan(c, batch, q_heads, prefix_cols, bf);
        int64_t n = o.planes > FULL ? o.planes : FULL;
        if (n > o.planes * units) n = o.planes * units;
        if (n * 32 * o.row_waves > most) most = n * 32 * o.row_waves;
    }
    return most;
}

hipError_t launch_attend_shared(SharedParams p, bool bf, hipStream_t s) {
    if ((p.splits && !grid_ok(prefix_blocks(p), 512)) || !grid_ok(p.own.batch * p.own.q_heads, 256)) return TOO_LARGE;
    p.own.page_div = div_by(p.own.c.page);
    p.own.all_parts = 1;
    if (p.own.cols) {
        const hipError_t e = launch_attend(p.own, bf, s);
        if (e != hipSuccess) return e;
    }
    switch (p.own.c.dim) {
    case 64: return bf ? pick<64, false>(p, s) : pick<64, true>(p, s);
    case 96: return bf ? pick<96, false>(p, s) : pick<96, true>(p, s);
    case 128: return bf ? pick<128, false>(p, s) : pick<128, true>(p, s);
    case 192: return bf ? pick<192, false>(p, s) : pick<192, true>(p, s);
    default: return bf ? pick<256, false>(p, s) : pick<256, true>(p, s);
    }
}

}  // namespace mxk
