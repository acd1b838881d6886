// lora.hip -- low-rank adapters of many requests beside a shared projection:
// y[t] = base[t] + s_a B_a (A_a x[t]), a the adapter that token t names.
//
// Mathematics.  Two products with a thin middle: h = A x (rank values a token)
// and B h.  Tokens come in tiles of 16, the columns of the 16 x 16 matrix
// instruction, whose rows are ranks (first product) or outputs (second).
// Columns are independent, so a tile whose tokens name several adapters runs
// once for each distinct one and keeps its own columns: a decode batch costs
// every adapter it uses once, a prompt of one adapter no more than a dense
// product, and tokens need no sorting.  bf16 operands: the 16 x 16 x 32 bf16
// instruction, h (fp32) as the exact sum of three bf16 parts side by side
// along K.  fp32 operands: the 16 x 16 x 4 fp32 instruction, products exact to
// its own rounding.
//
// Bound and measured (bf16).  Prompts: memory; 8192 tokens at 14336 x 4096, rank
// 16: 27 us for h and 119 for y (470 MB, 4.0 TB/s).  There the parts of h formed by
// every wave again, 156 to 176 us, took the vector unit longer than the base takes
// from memory; lanes that take 64 bytes of x each instead of four side by side, 34
// us for h.  fp32 operands, base and y: 55 + 255 us (3.9 TB/s).  A few tokens:
// chains of loads; 16 tokens of 16 adapters at 14336 x 4096 6.1 + 7.6 us (fp32
// 8.2 + 7.3), one at 1024 x 1024 3.6 + 4.7.
#include "decode_kernels.hpp"

namespace mxk {
using namespace mxd;

namespace {

typedef __bf16 bf8v __attribute__((ext_vector_type(8)));
typedef float f4v __attribute__((ext_vector_type(4)));
typedef float f2v __attribute__((ext_vector_type(2)));
typedef __bf16 bf2v __attribute__((ext_vector_type(2)));

constexpr int TOK = 16;

// ids of the tile's tokens, one for each of 16 lanes (-1: none, or no such
// adapter), and the set of lanes that are the first with theirs
struct Ids {
    int id;
    uint32_t first;
};
__device__ __forceinline__ Ids tile_ids(const LoraParams& p, int64_t t0, int c) {
    Ids o;
    o.id = t0 + c < p.tokens ? p.ids[t0 + c] : -1;
    if (o.id < 0 || o.id >= p.count) o.id = -1;
    const int id0 = __builtin_amdgcn_readfirstlane(o.id);
    if (__all(o.id == id0)) {                         // a prompt's tile
        o.first = id0 >= 0 ? 1u : 0u;
        return o;
    }
    bool again = o.id < 0;
#pragma unroll
    for (int i = 0; i < TOK - 1; i++) again |= i < c && __builtin_amdgcn_readlane(o.id, i) == o.id;
    o.first = (uint32_t)__ballot(!again) & 0xffffu;
    return o;
}

// x as three bf16 parts, truncated (exact; Inf and NaN keep their first)
__device__ __forceinline__ uint16_t part3(float x, int part) {
    const uint32_t u = fbits(x);
    if ((u & 0x7f800000u) == 0x7f800000u) return part ? 0 : bf16_rne(x);
    const float r = x - bitsf(u & 0xffff0000u);
    const uint32_t v = fbits(r);
    return (uint16_t)((part == 0 ? u : part == 1 ? v : fbits(r - bitsf(v & 0xffff0000u))) >> 16);
}

__device__ __forceinline__ f4v mfma_bf16(u32x4 a, u32x4 b, f4v c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8v, a), __builtin_bit_cast(bf8v, b), c, 0, 0, 0);
}
// the product of 16 K positions, four of a lane's each
__device__ __forceinline__ f4v mfma_f32(u32x4 a, u32x4 b, f4v c) {
#pragma unroll
    for (int e = 0; e < 4; e++) c = __builtin_amdgcn_mfma_f32_16x16x4f32(bitsf(a[e]), bitsf(b[e]), c, 0, 0, 0);
    return c;
}

// ---------------------------------------------------------------------------
// h = A x.  Eight waves share K in steps of 256 bytes, RT tiles of 16
// ranks each; a workgroup takes one of `splits` runs of K.  The waves' sums are
// added in LDS in their order and scaled, the runs' by the second product.  More
// than 16 tokens have one run, and their bf16 parts are formed here, once.
// ---------------------------------------------------------------------------
constexpr int SW = 8;

template <bool F32, int RT>
__global__ __launch_bounds__(64 * SW) void k_lora_down(LoraParams p) {
    constexpr int ES = F32 ? 4 : 2, STEP = 256 / ES;                     // values a wave takes at a time
    __shared__ __attribute__((aligned(16))) float red[SW][RT][256];
    const int tid = threadIdx.x, lane = tid & 63, c = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    uint32_t rest = blockIdx.x;
    const int split = (int)(rest % (uint32_t)p.splits);
    rest /= (uint32_t)p.splits;
    const int turn = (int)(rest % (uint32_t)p.spread);                   // which of the tile's adapters, where they are spread
    rest /= (uint32_t)p.spread;
    const int r0 = (int)(rest % (uint32_t)p.rank_groups) * 16 * RT;
    const int64_t t0 = (int64_t)(rest / (uint32_t)p.rank_groups) * TOK;
    const Ids ids = tile_ids(p, t0, c);
    const int k = (int)p.k, steps = (k + STEP - 1) / STEP;
    const int from = (int)((int64_t)split * steps / p.splits), to = (int)((int64_t)(split + 1) * steps / p.splits);
    const int64_t tok = t0 + c < p.tokens ? t0 + c : p.tokens - 1;
    const char* x = static_cast<const char*>(p.x) + tok * p.ldx * ES + 16 * g;

    f4v acc[RT];
#pragma unroll
    for (int i = 0; i < RT; i++) acc[i] = f4v{0.f, 0.f, 0.f, 0.f};
    int seen = 0;
    for (uint32_t left = ids.first; left; left &= left - 1, seen++) {
        if (p.spread > 1 && seen != turn) continue;
        const int a = __builtin_amdgcn_readlane(ids.id, __builtin_ctz(left));
        const char* w[RT];
#pragma unroll
        for (int i = 0; i < RT; i++) {
            const int r = r0 + 16 * i + c < p.rank ? r0 + 16 * i + c : p.rank - 1;
            w[i] = static_cast<const char*>(p.a) + ((int64_t)a * p.rank + r) * k * ES + 16 * g;
        }
        f4v sum[RT];
#pragma unroll
        for (int i = 0; i < RT; i++) sum[i] = f4v{0.f, 0.f, 0.f, 0.f};
        for (int s = from + wave; s < to; s += SW) {
            const int at = s * STEP * ES;                                // bytes; four lanes take 64 of a row at once
            u32x4 xv[4], wv[RT][4];
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const bool in = at + 64 * j + 16 * g < k * ES;
                xv[j] = in ? *reinterpret_cast<const u32x4*>(x + at + 64 * j) : u32x4{0u, 0u, 0u, 0u};
#pragma unroll
                for (int i = 0; i < RT; i++)
                    wv[i][j] = in ? *reinterpret_cast<const u32x4*>(w[i] + at + 64 * j) : u32x4{0u, 0u, 0u, 0u};
            }
#pragma unroll
            for (int j = 0; j < 4; j++)
#pragma unroll
                for (int i = 0; i < RT; i++) sum[i] = F32 ? mfma_f32(wv[i][j], xv[j], sum[i]) : mfma_bf16(wv[i][j], xv[j], sum[i]);
        }
#pragma unroll
        for (int i = 0; i < RT; i++)
            if (ids.id == a) acc[i] = sum[i];
    }
    if (p.spread > 1 && turn >= __builtin_popcount(ids.first)) return;       // the same in every wave
#pragma unroll
    for (int i = 0; i < RT; i++) *reinterpret_cast<f4v*>(&red[wave][i][c * 16 + 4 * g]) = acc[i];     // [token][rank]
    __syncthreads();
    int mine = 0;                                                        // the spread adapter's id
    if (p.spread > 1) {
        uint32_t left = ids.first;
        for (int i = 0; i < turn; i++) left &= left - 1;
        mine = __builtin_amdgcn_readlane(ids.id, __builtin_ctz(left));
    }
    for (int n = tid; n < 256 * RT; n += 64 * SW) {
        const int i = n % (16 * RT), t = n / (16 * RT);                  // rank, token
        const int id = __shfl(ids.id, t, 64);
        if (t0 + t >= p.tokens || r0 + i >= p.rank || id < 0 || (p.spread > 1 && id != mine)) continue;
        float v = 0.f;
#pragma unroll
        for (int q = 0; q < SW; q++) v += red[q][i / 16][t * 16 + i % 16];
        if (p.scales) v *= p.scales[id];
        if (!F32 && p.thirds) {
            uint16_t* h = reinterpret_cast<uint16_t*>(p.h) + (t0 + t) * 3 * p.rank + r0 + i;
#pragma unroll
            for (int part = 0; part < 3; part++) h[part * p.rank] = part3(v, part);
        } else {
            p.h[((int64_t)split * p.tokens + t0 + t) * p.rank + r0 + i] = v;
        }
    }
}

// ---------------------------------------------------------------------------
// y = base + B h.  A wave takes NT tiles of 16 outputs, whose rows are dealt so
// that a lane ends with 4 NT consecutive outputs of its token, and goes down
// `run` tiles of tokens with B in registers while they name the same adapter.
// ---------------------------------------------------------------------------
constexpr int UW = 4;

// N values of a token's row (4 or 16) as they lie in memory, and as numbers.
// Rows that do not all start at a multiple of 16 bytes go value by value: 8192
// tokens of 14337 outputs, bf16, 475 us where 14336 take 119; 16 tokens 8.0 and 7.6.
template <bool BF, int N>
struct Run {
    static constexpr int W = BF ? (N + 7) / 8 : N / 4;
    u32x4 w[W];
    __device__ __forceinline__ void load(const void* p, int64_t at, int have, bool vec) {
        const char* x = static_cast<const char*>(p) + at * (BF ? 2 : 4);
        if (vec && have >= N) {
            if constexpr (BF && N == 4) {
                const uint2 v = *reinterpret_cast<const uint2*>(x);
                w[0] = u32x4{v.x, v.y, 0u, 0u};
            } else {
#pragma unroll
                for (int i = 0; i < W; i++) w[i] = *reinterpret_cast<const u32x4*>(x + 16 * i);
            }
        } else {
#pragma unroll
            for (int i = 0; i < W; i++)
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    uint32_t v = 0u;
                    if constexpr (BF) {
                        if (8 * i + 2 * e < have) v = reinterpret_cast<const uint16_t*>(x)[8 * i + 2 * e];
                        if (8 * i + 2 * e + 1 < have) v |= (uint32_t)reinterpret_cast<const uint16_t*>(x)[8 * i + 2 * e + 1] << 16;
                    } else {
                        if (4 * i + e < have) v = reinterpret_cast<const uint32_t*>(x)[4 * i + e];
                    }
                    w[i][e] = v;
                }
        }
    }
    __device__ __forceinline__ float value(int i) const {
        if constexpr (BF) return (i & 1) ? bf16hi(w[i / 8][i / 2 % 4]) : bf16lo(w[i / 8][i / 2 % 4]);
        else return bitsf(w[i / 4][i % 4]);
    }
};
template <int N>
__device__ __forceinline__ void store_run(const float (&o)[N], void* p, int64_t at, int have, bool vec, bool bf) {
    if (bf) {
        uint16_t* x = static_cast<uint16_t*>(p) + at;
        if (vec && have >= N) {
#pragma unroll
            for (int i = 0; i < N; i += N < 8 ? 4 : 8) {
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < (N < 8 ? 2 : 4); e++) {
                    const f2v a = {o[i + 2 * e], o[i + 2 * e + 1]};
                    w[e] = __builtin_bit_cast(uint32_t, __builtin_convertvector(a, bf2v));
                }
                if constexpr (N < 8) *reinterpret_cast<uint2*>(x + i) = make_uint2(w[0], w[1]);
                else *reinterpret_cast<u32x4*>(x + i) = u32x4{w[0], w[1], w[2], w[3]};
            }
        } else {
#pragma unroll
            for (int i = 0; i < N; i++)
                if (i < have) x[i] = bf16_rne(o[i]);
        }
    } else {
        float* x = static_cast<float*>(p) + at;
        if (vec && have >= N) {
#pragma unroll
            for (int i = 0; i < N; i += 4) *reinterpret_cast<f4v*>(x + i) = f4v{o[i], o[i + 1], o[i + 2], o[i + 3]};
        } else {
#pragma unroll
            for (int i = 0; i < N; i++)
                if (i < have) x[i] = o[i];
        }
    }
}

// R8: runs of 8 ranks of a group (1, 2, 4 or 8), further groups of 64 in turn
template <bool F32, int R8, int NT, bool BB>
__global__ __launch_bounds__(64 * UW) void k_lora_up(LoraParams p) {
    constexpr int ES = F32 ? 4 : 2, N = 4 * NT;
    // bf16: K slot 8 (4 j + g) holds run (4 j + g) % R8 of part (4 j + g) / R8;
    // fp32: slot 4 (4 j + g) the four ranks there
    constexpr int J = F32 ? (R8 + 1) / 2 : (3 * R8 + 3) / 4;
    constexpr int FR = F32 ? J : R8 <= 4 ? 1 : R8 / 4;                   // distinct pieces of B's row a lane holds
    const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t n0 = ((int64_t)blockIdx.x * UW + wave) * 16 * NT;
    if (n0 >= p.n) return;
    const int64_t tiles = (p.tokens + TOK - 1) / TOK;
    const int64_t first = (int64_t)blockIdx.y * p.run, last = first + p.run < tiles ? first + p.run : tiles;
    const int64_t n = n0 + N * g;                                        // this lane's outputs
    const int have = (int)(p.n - n < N ? p.n - n : N);                   // may be negative
    const int groups = (p.rank + 8 * R8 - 1) / (8 * R8);

    // B's rows of group q: row i of tile s is output n0 + N (i / 4) + 4 s + i % 4
    struct Rows {
        u32x4 w[NT][FR];
    };
    auto load_b = [&](Rows& o, int a, int q) {
#pragma unroll
        for (int s = 0; s < NT; s++) {
            const int64_t row = n0 + N * (c / 4) + 4 * s + c % 4;
            const char* b = static_cast<const char*>(p.b) + ((int64_t)a * p.n + (row < p.n ? row : p.n - 1)) * p.rank * ES;
#pragma unroll
            for (int f = 0; f < FR; f++) {
                const int r = q * 8 * R8 + (F32 ? 16 * f + 4 * g : R8 <= 4 ? 8 * (g % R8) : 32 * f + 8 * g);
                o.w[s][f] = r < p.rank ? *reinterpret_cast<const u32x4*>(b + r * ES) : u32x4{0u, 0u, 0u, 0u};
            }
        }
    };
    // What a tile of tokens brings along, loaded a tile ahead.  h of a token
    // without an adapter is whatever the workspace held, and not kept.
    constexpr bool THIRDS = !F32 && NT > 1;                              // h comes in its bf16 parts
    constexpr int V = F32 ? 4 : 8, HV = THIRDS ? 1 : V / 4;
    struct Tokens {
        Ids ids;
        Run<BB, N> base;
        f4v h[J][HV];
    };
    auto load_h = [&](f4v (&h)[J][HV], int64_t tok, int q) {
#pragma unroll
        for (int j = 0; j < J; j++) {
            const int slot = 4 * j + g, r = q * 8 * R8 + (F32 ? 4 * slot : 8 * (slot % R8));
            const bool in = (F32 || slot < 3 * R8) && r < p.rank;
#pragma unroll
            for (int e = 0; e < HV; e++) h[j][e] = f4v{0.f, 0.f, 0.f, 0.f};
            if constexpr (THIRDS) {
                const uint16_t* from = reinterpret_cast<const uint16_t*>(p.h) + (tok * 3 + slot / R8) * p.rank + r;
                if (in) h[j][0] = *reinterpret_cast<const f4v*>(from);
                continue;
            }
            for (int s = 0; in && s < p.splits; s++) {
                const f4v* from = reinterpret_cast<const f4v*>(p.h + ((int64_t)s * p.tokens + tok) * p.rank + r);
#pragma unroll
                for (int e = 0; e < HV; e++) h[j][e] = s ? h[j][e] + from[e] : from[e];
            }
        }
    };
    auto token_of = [&](int64_t tile) { return tile * TOK + c < p.tokens ? tile * TOK + c : p.tokens - 1; };
    auto load_tokens = [&](Tokens& o, int64_t tile) {
        const int64_t tok = token_of(tile);
        o.ids = tile_ids(p, tile * TOK, c);
        // without a base: nothing is there to load, and zeros are loaded
        o.base.load(p.base, tok * p.ld_base + n, p.base ? have : 0, p.vec_base);
        load_h(o.h, tok, 0);
    };
    // adapters whose rows are asked for at once: a decode tile names many
    constexpr int AT = NT == 1 && R8 <= 4 ? 4 : 1;
    Rows w[AT];
    int held = -1;
    Tokens now, next;
    load_tokens(now, first);
    for (int64_t tile = first; tile < last; tile++) {
        if (tile + 1 < last) load_tokens(next, tile + 1);
        f4v acc[NT];
#pragma unroll
        for (int s = 0; s < NT; s++) acc[s] = f4v{0.f, 0.f, 0.f, 0.f};
        for (int q = 0; q < groups; q++) {
            if (q) load_h(now.h, token_of(tile), q);
            // the token's h as columns
            u32x4 h[J];
#pragma unroll
            for (int j = 0; j < J; j++)
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    if constexpr (F32 || THIRDS) {
                        h[j][e] = fbits(now.h[j][0][e]);
                    } else {
                        const int part = (4 * j + g) / R8;
                        const f4v v = now.h[j][e / 2 % HV];
                        h[j][e] = part < 3 ? part3(v[2 * e % 4], part) | (uint32_t)part3(v[(2 * e + 1) % 4], part) << 16 : 0u;
                    }
                }
            for (uint32_t left = now.ids.first; left;) {
                int a[AT];
#pragma unroll
                for (int i = 0; i < AT; i++) {                           // -2: no further one
                    a[i] = left ? __builtin_amdgcn_readlane(now.ids.id, __builtin_ctz(left)) : -2;
                    left = left ? left & (left - 1) : 0u;
                    if (a[i] >= 0 && (AT > 1 || a[i] != held || groups > 1)) load_b(w[i], a[i], q);
                }
                held = a[0];
#pragma unroll
                for (int i = 0; i < AT; i++) {
                    if (a[i] < 0) break;
                    // of its own tokens alone, by selection: what another adapter's
                    // weights hold, a NaN say, reaches nobody else
#pragma unroll
                    for (int s = 0; s < NT; s++) {
                        f4v sum = acc[s];
#pragma unroll
                        for (int j = 0; j < J; j++) {
                            if (F32) sum = mfma_f32(w[i].w[s][j % FR], h[j], sum);
                            else sum = mfma_bf16(w[i].w[s][j % FR], h[j], sum);
                        }
                        if (now.ids.id == a[i]) acc[s] = sum;
                    }
                }
            }
        }
        if (tile * TOK + c < p.tokens && have > 0) {
            float y[N];
#pragma unroll
            for (int i = 0; i < N; i++) y[i] = now.base.value(i) + acc[i / 4][i % 4];
            store_run(y, p.y, token_of(tile) * p.ldy + n, have, p.vec_y, p.y_bf16);
        }
        now = next;
    }
}

template <bool F32, int RT>
hipError_t down(const LoraParams& p, hipStream_t s) {
    const int64_t n = (p.tokens + TOK - 1) / TOK * p.rank_groups * p.spread * p.splits;
    k_lora_down<F32, RT><<<(unsigned)n, 64 * SW, 0, s>>>(p);
    return hipGetLastError();
}
template <bool F32, int R8, int NT>
hipError_t up(const LoraParams& p, hipStream_t s) {
    const int64_t n = (p.n + 16 * NT * UW - 1) / (16 * NT * UW), tiles = (p.tokens + TOK - 1) / TOK;
    const dim3 grid((unsigned)n, (unsigned)((tiles + p.run - 1) / p.run));
    if (p.base_bf16) k_lora_up<F32, R8, NT, true><<<grid, 64 * UW, 0, s>>>(p);
    else k_lora_up<F32, R8, NT, false><<<grid, 64 * UW, 0, s>>>(p);
    return hipGetLastError();
}
template <bool F32, int NT>
hipError_t up_rank(const LoraParams& p, hipStream_t s) {
    if (p.rank <= 8) return up<F32, 1, NT>(p, s);
    if (p.rank <= 16) return up<F32, 2, NT>(p, s);
    return p.rank <= 32 ? up<F32, 4, NT>(p, s) : up<F32, 8, NT>(p, s);
}
template <bool F32>
hipError_t both(LoraParams p, hipStream_t s) {
    p.rank_groups = (p.rank + 63) / 64;
    // both grids, before either is launched
    const int64_t tiles = (p.tokens + TOK - 1) / TOK, wide = 16 * UW * (p.tokens <= TOK ? 1 : 4);
    if (!grid_ok(tiles * p.rank_groups * p.spread * p.splits, 64 * SW) ||
        !grid_ok((p.n + wide - 1) / wide * ((tiles + p.run - 1) / p.run), 64 * UW))
        return TOO_LARGE;
    const hipError_t e = p.rank <= 16 ? down<F32, 1>(p, s) : p.rank <= 32 ? down<F32, 2>(p, s) : down<F32, 4>(p, s);
    if (e != hipSuccess) return e;
    return p.tokens <= TOK ? up_rank<F32, 1>(p, s) : up_rank<F32, 4>(p, s);
}

}  // namespace

// Runs of K for few tokens, whose first product is a chain of loads.  More than
// one tile of tokens has no runs, and outputs in fours of tiles: at 14336 x 4096,
// rank 16, 32 adapters, 16 tokens take 6.1 + 7.8 us and 17, 32, 64 and 128 take
// 11.3 + 9.2, 11.4 + 10.0, 11.6 + 10.3 and 11.7 + 12.8.
constexpr int MOST_SPLITS = 8;
int lora_splits(int64_t tokens, int64_t k) {
    if (tokens > TOK) return 1;
    const int64_t n = k / 1024;
    return (int)(n < 1 ? 1 : n > MOST_SPLITS ? MOST_SPLITS : n);
}
// three bf16 parts, or an fp32 for each run, of each token
int64_t lora_bytes(int64_t tokens, int64_t rank) {
    const int64_t few = (tokens < TOK ? tokens : TOK) * MOST_SPLITS * 4, many = tokens * 6;
    return (few > many ? few : many) * rank;
}

hipError_t launch_lora(LoraParams p, hipStream_t s) {
    const int64_t tiles = (p.tokens + TOK - 1) / TOK;
    p.splits = lora_splits(p.tokens, p.k);
    p.thirds = p.bf16 && p.tokens > TOK;
    p.spread = p.tokens <= 1024 ? (int)(p.tokens < TOK ? p.tokens : TOK) : 1;
    if (p.spread > p.count) p.spread = p.count > 0 ? p.count : 1;
    // tiles of tokens a workgroup goes down: about 2048 workgroups
    const int64_t n = (p.n + 64 * UW - 1) / (64 * UW), run = tiles * n / 2048;
    p.run = (int)(run < 1 ? 1 : run > 64 ? 64 : run);
    if ((tiles + p.run - 1) / p.run > 65535) p.run = (int)((tiles + 65534) / 65535);
    return p.bf16 ? both<false>(p, s) : both<true>(p, s);
}

}  // namespace mxk
