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
#include "attend_device.hpp"

namespace mxk {
using namespace mxd;

namespace {

typedef float f16v __attribute__((ext_vector_type(16)));
typedef short s4v __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s4v lds_s4v;

constexpr int WAVES = 4, ST = 64 * WAVES;

// tokens of a tile: 32 for each wave side by side along them, twice that where
// all waves stand side by side along the rows
constexpr int tile_tokens(int rw) { return rw == 1 ? 128 : 64; }
// LDS row strides in bytes.  Keys: 8 lanes of a 16-byte read take 8 rows, whose
// starts are then 4 banks apart or a multiple of it, all different.  Values: the
// transposing read takes 64 bytes of 4 rows, a quarter of the banks each.
constexpr int key_stride(int D) { return D * 2 + 16; }
constexpr int value_stride(int D) { return D * 2 + ((D * 2) % 128 == 0 ? 64 : 0); }
constexpr int sum_stride(int D) { return D + 4; }
constexpr int lds_bytes(int D, int rw) {
    const int tiles = tile_tokens(rw) * (key_stride(D) + value_stride(D));
    const int join = rw == WAVES ? 0 : WAVES * 32 * (sum_stride(D) + 2) * 4;
    return tiles > join ? tiles : join;
}

// Rows of one tile of RW x 32 and one range of the prefix's tokens.  RW waves
// stand along the rows, 4 / RW along the tokens.  The 32 x 32 x 16 instruction
// takes tokens as rows and query rows as columns, so a lane holds 16 scores of
// one query row and the row's maximum is a maximum over registers and one
// exchange; the scores' layout is the column operand of the second product when
// its K order is (8-token run, half of the wave, token), which the transposing
// LDS read of the values follows.
template <int D, int KIND, bool QF32, int RW>
__global__ __launch_bounds__(ST, D <= 128 && !QF32 ? 2 : 1) void k_prefix(SharedParams p) {
    constexpr int TW = WAVES / RW, TK = tile_tokens(RW), SUB = TK / TW / 32, RT = 32 * RW;
    constexpr int QP = QF32 ? 3 : 1, PP = QF32 ? 3 : 2;            // bf16 parts of a query and of a probability
    constexpr int BITS = kind_bits(KIND), ROWB = D * BITS / 8, NB = D / 32;
    constexpr int CPR = ROWB / 16, VALS = 128 / BITS;              // 16-byte chunks of a row, values of one
    constexpr int CHUNKS = TK * CPR, NC = (CHUNKS + ST - 1) / ST;
    constexpr int KS = key_stride(D), VS = value_stride(D);
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    __shared__ int bad_page;
    uint8_t *sk = smem, *sv = smem + TK * KS;

    const AttendParams& a = p.own;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int c = lane & 31, half = lane >> 5;
    const int rw = wave % RW, tw = wave / RW;
    const int group = a.q_heads / a.c.heads;
    const int64_t rows = a.batch * group, row_tiles = (rows + RT - 1) / RT;
    const int64_t pair = blockIdx.x / row_tiles, rt = blockIdx.x - pair * row_tiles;
    const int kvh = (int)(pair / p.splits), split = (int)(pair - (int64_t)kvh * p.splits);
    const int64_t cap = p.prefix_cols * a.c.page;
    const int64_t n = *p.prefix_length;
    const int len = (int)(n < 0 ? 0 : n > cap ? cap : n);
    const int units = (len + TK - 1) / TK, of = units < p.splits ? units : p.splits;
    if (split >= of) return;
    const int t0 = (int)((int64_t)split * units / of) * TK;
    const int t1 = (int)((int64_t)(split + 1) * units / of) * TK, tend = t1 < len ? t1 : len;
    const float zs = a.scale * 1.44269504088896340736f;
    const int64_t row0 = rt * RT + 32 * rw;                        // this wave's first row
    const bool active = row0 < rows;
    if (tid == 0) bad_page = 0;

    // this lane's query row as the score product's columns
    uint32_t q[QP][D / 16][4];
    {
        const int64_t m = row0 + c < rows ? row0 + c : rows - 1;
        const int64_t b = m / group, at = b * a.q_ts + (kvh * group + (m - b * group)) * a.q_hs + 8 * half;
#pragma unroll
        for (int k = 0; k < D / 16; k++) {
            if constexpr (QF32) {
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const Parts x = parts_of(static_cast<const float*>(a.q)[at + 16 * k + 2 * e]);
                    const Parts y = parts_of(static_cast<const float*>(a.q)[at + 16 * k + 2 * e + 1]);
                    q[0][k][e] = pack_hi(x.h, y.h);
                    q[QP - 2][k][e] = pack_hi(x.m, y.m);
                    q[QP - 1][k][e] = pack_hi(x.l, y.l);
                }
            } else {
                load_bytes<16>(q[0][k], reinterpret_cast<const uint8_t*>(static_cast<const uint16_t*>(a.q) + at + 16 * k));
            }
        }
    }

    // a tile's cached bytes on their way to LDS
    struct Tile {
        uint32_t k[NC][4], v[NC][4], ks[KIND == KV_BF16 ? 1 : NC], vs[KIND == KV_BF16 ? 1 : NC];
    };
    bool bad = false;
    auto load = [&](Tile& o, int tb) {
#pragma unroll
        for (int i = 0; i < NC; i++) {
            const int idx = tid + ST * i < CHUNKS ? tid + ST * i : CHUNKS - 1;
            const int token = idx / CPR, ch = idx - token * CPR;
            const int t = tb + token < tend ? tb + token : tend - 1;
            const uint32_t pg = over((uint32_t)t, a.page_div);
            int64_t page = p.prefix[pg];
            if (page < 0 || page >= a.c.pages) { page = 0; bad = true; }
            const int64_t row = (page * a.c.heads + kvh) * a.c.page + (t - (int)pg * a.c.page);
            load_bytes<16>(o.k[i], a.c.k + row * ROWB + 16 * ch);
            load_bytes<16>(o.v[i], a.c.v + row * ROWB + 16 * ch);
            if constexpr (KIND != KV_BF16) {
                o.ks[i] = a.c.ks[row * NB + ch * VALS / 32];
                o.vs[i] = a.c.vs[row * NB + ch * VALS / 32];
            }
        }
    };
    auto store = [&](const Tile& o, int tb) {
#pragma unroll
        for (int i = 0; i < NC; i++) {
            const int idx = tid + ST * i;
            if (CHUNKS % ST && idx >= CHUNKS) break;
            const int token = idx / CPR, ch = idx - token * CPR;
            const bool live = tb + token < tend;                   // past the end: values count as zero
            const float ks = KIND == KV_BF16 ? 1.f : e8m0(o.ks[KIND == KV_BF16 ? 0 : i]);
            const float vs = KIND == KV_BF16 ? 1.f : e8m0(o.vs[KIND == KV_BF16 ? 0 : i]);
            each<VALS / 8>([&](auto jc) {
                constexpr int J = 4 * jc.value;
                u32x4 x = {pair_of<KIND, J>(o.k[i], ks), pair_of<KIND, J + 1>(o.k[i], ks), pair_of<KIND, J + 2>(o.k[i], ks),
                           pair_of<KIND, J + 3>(o.k[i], ks)};
                *reinterpret_cast<u32x4*>(sk + token * KS + ch * VALS * 2 + 4 * J) = x;
                u32x4 y = {pair_of<KIND, J>(o.v[i], vs), pair_of<KIND, J + 1>(o.v[i], vs), pair_of<KIND, J + 2>(o.v[i], vs),
                           pair_of<KIND, J + 3>(o.v[i], vs)};
                if (!live) y = u32x4{0u, 0u, 0u, 0u};
                *reinterpret_cast<u32x4*>(sv + token * VS + ch * VALS * 2 + 4 * J) = y;
            });
        }
    };

    f16v acc[D / 32];
#pragma unroll
    for (int i = 0; i < D / 32; i++)
#pragma unroll
        for (int e = 0; e < 16; e++) acc[i][e] = 0.f;
    float m = -INFINITY, l = 0.f;                                  // of row c; l: this lane's tokens

    Tile tile;
    load(tile, t0);
    for (int tb = t0; tb < tend; tb += TK) {
        __syncthreads();                                           // the tile before has been read
        store(tile, tb);
        __syncthreads();
        if (tb + TK < tend) load(tile, tb + TK);
        if (!active) continue;
#pragma unroll
        for (int sub = 0; sub < SUB; sub++) {
            const int tk = (SUB * tw + sub) * 32;                  // first token in the tile
            if (tb + tk >= tend) break;
            f16v z;
#pragma unroll
            for (int e = 0; e < 16; e++) z[e] = 0.f;
#pragma unroll
            for (int k = 0; k < D / 16; k++) {
                const bf8v x = *reinterpret_cast<const bf8v*>(sk + (tk + c) * KS + 32 * k + 16 * half);
#pragma unroll
                for (int i = 0; i < QP; i++)
                    z = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x, frag(q[i][k][0], q[i][k][1], q[i][k][2], q[i][k][3]), z, 0, 0, 0);
            }
            float zmax = -INFINITY;
            const bool part = tb + tk + 32 > tend;
#pragma unroll
            for (int e = 0; e < 16; e++) {
                z[e] *= zs;
                if (part && tb + tk + 8 * (e / 4) + 4 * half + e % 4 >= tend) z[e] = -INFINITY;
                zmax = fmaxf(zmax, z[e]);
            }
            zmax = fmaxf(zmax, __shfl_xor(zmax, 32, 64));
            if (__any(zmax > m)) {                                 // the maximum of some row grows
                const float mn = fmaxf(m, zmax);
                const float grow = __builtin_amdgcn_exp2f(m - (mn == -INFINITY ? 0.f : mn));
                m = mn;
                l *= grow;
#pragma unroll
                for (int i = 0; i < D / 32; i++) acc[i] *= grow;
            }
            const float ms = m == -INFINITY ? 0.f : m;             // every score so far is -inf
            uint32_t pw[PP][2][4];                                 // probabilities as bf16 pairs
#pragma unroll
            for (int i = 0; i < 8; i++) {
                float x = __builtin_amdgcn_exp2f(z[2 * i] - ms), y = __builtin_amdgcn_exp2f(z[2 * i + 1] - ms);
                l += x + y;
#pragma unroll
                for (int k = 0; k < PP; k++) {
                    const f2v xy = {x, y};
                    pw[k][i / 4][i % 4] = bits_of(__builtin_convertvector(xy, bf2v));
                    x -= bitsf(pw[k][i / 4][i % 4] << 16);
                    y -= bitsf(pw[k][i / 4][i % 4] & 0xffff0000u);
                }
            }
            // sums of p v: of 16 lanes, four at a row's 16 values
            const uint8_t* at = sv + (tk + 4 * half + (c % 16) / 4) * VS + (c / 16) * 32 + (c % 4) * 8;
#pragma unroll
            for (int s = 0; s < 2; s++)
#pragma unroll
                for (int i = 0; i < D / 32; i++) {
                    s4v lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4v*)(at + 16 * s * VS + 64 * i));
                    s4v hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4v*)(at + (16 * s + 8) * VS + 64 * i));
                    const short w[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
                    bf8v x;
                    __builtin_memcpy(&x, w, 16);
#pragma unroll
                    for (int k = 0; k < PP; k++)
                        acc[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x, frag(pw[k][s][0], pw[k][s][1], pw[k][s][2], pw[k][s][3]),
                                                                         acc[i], 0, 0, 0);
                }
        }
    }
    l += __shfl_xor(l, 32, 64);
    if (bad) bad_page = 1;

    // the tile's triples; waves along the tokens are joined through LDS
    const int64_t wg = ((int64_t)kvh * row_tiles + rt) * p.splits + split;
    float* out = p.parts + wg * RT * D;
    float* ml = p.parts + (int64_t)a.c.heads * row_tiles * p.splits * RT * D + wg * RT * 2;
    __syncthreads();
    if (bad_page) l = bitsf(0x7fc00000u);
    if constexpr (TW == 1) {
        if (row0 + c < rows) {
#pragma unroll
            for (int i = 0; i < D / 32; i++)
#pragma unroll
                for (int e = 0; e < 16; e += 4)
                    *reinterpret_cast<f4v*>(out + (int64_t)(32 * rw + c) * D + 32 * i + 2 * e + 4 * half) =
                        f4v{acc[i][e], acc[i][e + 1], acc[i][e + 2], acc[i][e + 3]};
            if (half == 0) {
                ml[2 * (32 * rw + c)] = m;
                ml[2 * (32 * rw + c) + 1] = l;
            }
        }
    } else {
        constexpr int SS = sum_stride(D);
        float* sums = reinterpret_cast<float*>(smem);              // [token wave][row][SS]
        float* st = sums + WAVES * 32 * SS;
        const int at = tw * RT + 32 * rw + c;
#pragma unroll
        for (int i = 0; i < D / 32; i++)
#pragma unroll
            for (int e = 0; e < 16; e += 4)
                *reinterpret_cast<f4v*>(sums + at * SS + 32 * i + 2 * e + 4 * half) =
                    f4v{acc[i][e], acc[i][e + 1], acc[i][e + 2], acc[i][e + 3]};
        if (half == 0) {
            st[2 * at] = m;
            st[2 * at + 1] = l;
        }
        __syncthreads();
        const int held = (int)(rows - rt * RT < RT ? rows - rt * RT : RT);
        for (int i = tid; i < held * (D / 4); i += ST) {
            const int r = i / (D / 4), d = 4 * (i - r * (D / 4));
            float M = -INFINITY, L = 0.f;
            f4v o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int w = 0; w < TW; w++) M = fmaxf(M, st[2 * (w * RT + r)]);
            const float Ms = M == -INFINITY ? 0.f : M;
#pragma unroll
            for (int w = 0; w < TW; w++) {
                const float f = __builtin_amdgcn_exp2f(st[2 * (w * RT + r)] - Ms);
                L += f * st[2 * (w * RT + r) + 1];
                o += f * *reinterpret_cast<const f4v*>(sums + (w * RT + r) * SS + d);
            }
            *reinterpret_cast<f4v*>(out + (int64_t)r * D + d) = o;
            if (d == 0) {
                ml[2 * r] = M;
                ml[2 * r + 1] = L;
            }
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
    const int64_t bh = blockIdx.x, b = bh / a.q_heads;
    const int h = (int)(bh - b * a.q_heads);
    // the prefix's
    const int group = a.q_heads / a.c.heads, kvh = h / group, RT = 32 * p.row_waves, TK = tile_tokens(p.row_waves);
    int front = 0;
    const float *fo = nullptr, *fx = nullptr;
    if (p.splits) {
        const int64_t cap = p.prefix_cols * a.c.page, n = *p.prefix_length;
        const int len = (int)(n < 0 ? 0 : n > cap ? cap : n), units = (len + TK - 1) / TK;
        front = units < p.splits ? units : p.splits;
        const int64_t rows = a.batch * group, row_tiles = (rows + RT - 1) / RT, m = b * group + (h - kvh * group), rt = m / RT;
        const int64_t at = (kvh * row_tiles + rt) * p.splits * RT + (m - rt * RT);
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
    return (int64_t)p.own.c.heads * p.splits * ((rows + rt - 1) / rt);
}

template <int D, int KIND, bool QF32, int RW>
hipError_t go(const SharedParams& p, hipStream_t s) {
    constexpr int lds = lds_bytes(D, RW);
    if (lds > 64 * 1024) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(k_prefix<D, KIND, QF32, RW>),
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, lds);
        if (e != hipSuccess) return e;
    }
    k_prefix<D, KIND, QF32, RW><<<(unsigned)prefix_blocks(p), ST, lds, s>>>(p);
    return hipGetLastError();
}
template <int D, int KIND, bool QF32>
hipError_t rows(const SharedParams& p, hipStream_t s) {
    if constexpr (D <= 128)
        if (p.row_waves == 1) return go<D, KIND, QF32, 1>(p, s);
    return p.row_waves == 2 ? go<D, KIND, QF32, 2>(p, s) : go<D, KIND, QF32, 4>(p, s);
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

constexpr int FULL = 512;              // workgroups that fill the chip: two for each CU

// Tiles of 32, 64 or 128 rows, the smallest that holds them all (64 where the
// head dimension is above 128: a tile of 128 tokens' registers do not fit), and
// as many ranges of tokens as fill the chip once.
SharedPlan shared_plan(const KvCache& c, int64_t batch, int q_heads, int64_t prefix_cols, bool q_bf16) {
    const int64_t rows = batch * (q_heads / c.heads);
    SharedPlan o;
    o.row_waves = rows <= 32 && c.dim <= 128 ? 1 : rows <= 64 ? 2 : 4;
    o.planes = c.heads * ((rows + 32 * o.row_waves - 1) / (32 * o.row_waves));
    const int64_t units = (prefix_cols * c.page + tile_tokens(o.row_waves) - 1) / tile_tokens(o.row_waves);
    const int64_t want = c.dim <= 128 && q_bf16 ? FULL : FULL / 2;
    int64_t splits = o.planes ? want / o.planes : 1;
    if (splits < 1) splits = 1;
    o.splits = (int)(splits < units ? splits : units);
    return o;
}

// planes x splits is at most FULL or the planes, and at most planes x units;
// planes, units (in tiles of 64) and the tile's rows grow with their arguments.
int64_t shared_rows(const KvCache& c, int64_t batch, int q_heads, int64_t prefix_cols) {
    if (!batch || !prefix_cols) return 0;
    const SharedPlan o = shared_plan(c, batch, q_heads, prefix_cols, true);
    const int64_t units = (prefix_cols * c.page + 63) / 64, most = o.planes > FULL ? o.planes : FULL;
    return (most < o.planes * units ? most : o.planes * units) * 32 * o.row_waves;
}

hipError_t launch_attend_shared(SharedParams p, bool bf, hipStream_t s) {
    if ((p.splits && !grid_ok(prefix_blocks(p), ST)) || !grid_ok(p.own.batch * p.own.q_heads, 256)) return TOO_LARGE;
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
