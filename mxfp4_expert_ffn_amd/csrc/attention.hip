// Attention over the paged cache (MXFP4 or bf16): single tokens, drafted
// blocks and prompts, causal or not, with a sliding window and first tokens
// that stay visible.
//
// Online softmax over tiles of 32 keys.  For a tile of 16 query rows the
// scores are formed transposed, S^T = K Q^T, and so is the product, O^T = V^T
// P^T, with v_mfma_f32_16x16x32_bf16: then a lane holds one query row (l % 16)
// throughout, row statistics and rescaling are lane-local, and the scores come
// out of the first product in the lane that the second product's operand wants
// them in.  For that, row m of the half tile t of keys is key 8 (m / 4) + 4 t +
// m % 4, so that lane group g = l / 16 ends up with the 8 keys 8 g .. 8 g + 7 of
// its row: a k-group of the operand, nothing moves between lanes.
//
// The reduction index of the first product may be in any order that K and Q
// share: group g takes elements [g D/4, (g+1) D/4), which are 16 contiguous
// bytes of an MXFP4 key row of 128 and one MX block.  V^T's row m of the
// product's tile tau is element m D/16 + tau, so a lane needs D/16 consecutive elements of
// its 8 keys, decodes pairs of elements with their key's scale and regroups
// halves of registers by key.  Both operands come straight from memory into
// registers; V's codes are stored so that these are 16-byte loads.
//
// Decoding E2M1 x E8M0 to bf16 is exact, queries are bf16 as given, scores and
// statistics float32; the softmax weights are rounded to bf16 for the second
// product (a relative 2^-9 each, as the operand type asks).  The row maximum
// is only a reference point: it is moved when some score of the tile passes it
// by 2^8, so most tiles need neither a lane exchange nor a rescaling.
//
// Four waves of a workgroup take every fourth tile of the workgroup's share
// of the keys and join their sums through LDS.  Where there are few (sequence,
// head) pairs the keys are shared by several workgroups, which leave float32
// sums that k_attn_join adds up in order.
#include <type_traits>

#include "kv_cache.hpp"

namespace moe {
namespace {

constexpr int kWaves = 4;
constexpr int kThreads = kWaves * kWave;
constexpr int kTile = 32;                          // keys per tile
constexpr float kSlack = 8.0f;                     // log2 a score may pass the reference by

struct AttnArgs {
    const uint16_t* q;
    uint16_t* out;
    const int32_t *table, *cu_q, *kv_lens;
    const uint8_t *k, *v, *ks, *vs;
    float *part, *stat;                            // sums [T H][nsplit][D], (reference, sum of weights) [T H][nsplit][2]
    int64_t qs, os;
    int32_t B, T, H, Hk, G, W, shift, num_pages, causal, window, sinks;
    int32_t share, nsplit, row_tiles;              // tiles per workgroup; workgroups along the keys, along the rows
    float c;                                       // scale * log2(e)
};

// A sequence: first row, rows, cached tokens (clamped to what there is).
struct Seq {
    int start, n, kv;
};
__device__ __forceinline__ Seq sequence(const AttnArgs& a, int b) {
    Seq s;
    s.start = min(max(a.cu_q[b], 0), a.T);
    s.n = min(max(a.cu_q[b + 1], s.start), a.T) - s.start;
    s.kv = (int)min((int64_t)max(a.kv_lens[b], 0), (int64_t)a.W << a.shift);
    return s;
}

// The key tiles that the rows of positions p0 .. p1 see: tiles 0 .. head-1
// (first tokens), then lo .. lo + total - head - 1.
struct Range {
    int head, lo, total;
};
__device__ __forceinline__ Range tiles_of(const AttnArgs& a, int p0, int p1, int kv) {
    Range r{0, 0, 0};
    const int end = p1 < 0 ? 0 : a.causal ? min(p1 + 1, kv) : kv;      // one past the last visible key
    int first = 0;
    if (a.window > 0) {
        first = (int)max((int64_t)p0 - a.window + 1, (int64_t)0);
        r.lo = first / kTile;
        r.head = min((int)(((int64_t)min(a.sinks, min(first, end)) + kTile - 1) / kTile), r.lo);
    }
    r.total = r.head + max((int)(((int64_t)end + kTile - 1) / kTile) - r.lo, 0);
    return r;
}

// MFMA operands of one tile of keys before decoding.
template <int FMT, int D> struct Raw;
template <int D> struct Raw<MOE_KV_MXFP4, D> {
    uint32_t k[2][D / 32];                         // D/4 codes of this lane's key in each half tile
    uint32_t kb[2];                                // their scale bytes
    uint32_t v[D / 16];                            // D/16 codes of this lane's 8 keys
    uint32_t vb[2];                                // their 8 scale bytes
};
template <int D> struct Raw<MOE_KV_BF16, D> {
    u32x4_t k[2][D / 32];
    uint32_t v[8][D / 32];
};

template <int N>
__device__ __forceinline__ void load_words(uint32_t* dst, const uint8_t* src) {
    if constexpr (N % 4 == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const u32x4_t x = *reinterpret_cast<const u32x4_t*>(src + 4 * i);
            dst[i] = x[0]; dst[i + 1] = x[1]; dst[i + 2] = x[2]; dst[i + 3] = x[3];
        }
    } else {
        static_assert(N == 2, "");
        const uint2 x = *reinterpret_cast<const uint2*>(src);
        dst[0] = x.x; dst[1] = x.y;
    }
}

// Pages of a tile's two halves of 16 keys; -1: outside the cache or behind the
// last key.
struct Pages {
    int p[2];
};
__device__ __forceinline__ Pages pages_of(const AttnArgs& a, const int32_t* row, int tile, int kv) {
    Pages pg;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int key = tile * kTile + 16 * h;
        int p = -1;
        if (key < kv) p = row[key >> a.shift];     // key < kv <= W pages
        pg.p[h] = p >= 0 && p < a.num_pages ? p : -1;
    }
    return pg;
}

template <int FMT, int D>
__device__ __forceinline__ void load_tile(Raw<FMT, D>& r, const AttnArgs& a, const Pages& pg, int tile, int hk, int lane) {
    const int m = lane % 16, g = lane / 16;
    const int mask = (1 << a.shift) - 1;
    const int pa = max(pg.p[0], 0), pb = max(pg.p[1], 0);               // page 0 stands in: read, then not used
    const int64_t ka = ((int64_t)(m < 8 ? pa : pb) * a.Hk + hk) << a.shift;
    const int64_t va = ((int64_t)(g < 2 ? pa : pb) * a.Hk + hk) << a.shift;
    const int vrow = (tile * kTile + 8 * g) & mask;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const int64_t row = ka + ((tile * kTile + 8 * (m / 4) + 4 * t + m % 4) & mask);
        if constexpr (FMT == MOE_KV_MXFP4) {
            load_words<D / 32>(r.k[t], a.k + row * (D / 2) + g * (D / 8));
            r.kb[t] = a.ks[row * (D / 32) + g * D / 128];
        } else {
            const u32x4_t* src = reinterpret_cast<const u32x4_t*>(a.k + (row * D + g * (D / 4)) * 2);
#pragma unroll
            for (int i = 0; i < D / 32; ++i) r.k[t][i] = src[i];
        }
    }
    if constexpr (FMT == MOE_KV_MXFP4) {
        constexpr int KG = v_keys_per_piece(D);
#pragma unroll
        for (int i = 0; i < 8 / KG; ++i)
            load_words<4>(r.v + 4 * i, a.v + va * (D / 2) + (vrow / KG + i) * (KG * D / 2) + m * 16);
        const uint2 b = *reinterpret_cast<const uint2*>(a.vs + va * (D / 32) + vrow * (D / 32) + (m * D / 512) * 8);
        r.vb[0] = b.x; r.vb[1] = b.y;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) load_words<D / 32>(r.v[j], a.v + ((va + vrow + j) * D + m * (D / 16)) * 2);
    }
}

// K operand of half tile t, step s: 8 elements of this lane's key.
template <int FMT, int D>
__device__ __forceinline__ bf16x8_t k_operand(const Raw<FMT, D>& r, int t, int s) {
    if constexpr (FMT == MOE_KV_MXFP4) return decode8_bf16(r.k[t][s], e8m0_as_scale(r.kb[t]));
    else return __builtin_bit_cast(bf16x8_t, r.k[t][s]);
}

template <int SEL>
__device__ __forceinline__ uint32_t decode2(uint32_t w, float scale) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, SEL));
}

// V^T operands of tiles 2u and 2u+1: pairs of elements of 8 keys -> the
// pairs' first and second elements by key.  live: which of the 8 keys count
// (the others' values become 0).
template <int FMT, int D, int U>
__device__ __forceinline__ void v_operand(const Raw<FMT, D>& r, uint32_t live, bf16x8_t& first, bf16x8_t& second) {
    uint32_t w[8];
    if constexpr (FMT == MOE_KV_MXFP4) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float sc = e8m0_as_scale((r.vb[j / 4] >> (8 * (j % 4))) & 0xFF);
            const int at = j * (D / 32) + U;       // byte of the lane's codes
            const uint32_t word = r.v[at / 4];
            w[j] = at % 4 == 0 ? decode2<0>(word, sc) : at % 4 == 1 ? decode2<1>(word, sc)
                 : at % 4 == 2 ? decode2<2>(word, sc) : decode2<3>(word, sc);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = r.v[j][U];
    }
    if (live != 0xFF) {
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = (live >> j) & 1 ? w[j] : 0;
    }
    u32x4_t lo, hi;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        lo[i] = __builtin_amdgcn_perm(w[2 * i + 1], w[2 * i], 0x05040100u);
        hi[i] = __builtin_amdgcn_perm(w[2 * i + 1], w[2 * i], 0x07060302u);
    }
    first = __builtin_bit_cast(bf16x8_t, lo);
    second = __builtin_bit_cast(bf16x8_t, hi);
}

__device__ __forceinline__ bool wild_pair(uint32_t w) {                 // infinite or NaN bf16 in either half
    return (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u;
}

// Whether a live key of this lane has an infinite or NaN value (MXFP4: a
// scale with which 6 passes float32's range, or NaN).
template <int FMT, int D>
__device__ __forceinline__ bool wild_values(const Raw<FMT, D>& r, uint32_t live) {
    bool wild = false;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        bool x = false;
        if constexpr (FMT == MOE_KV_MXFP4) {
            x = ((r.vb[j / 4] >> (8 * (j % 4))) & 0xFF) >= 253;
        } else {
#pragma unroll
            for (int u = 0; u < D / 32; ++u) x |= wild_pair(r.v[j][u]);
        }
        wild |= x && ((live >> j) & 1);
    }
    return wild;
}

// One element of a cached value, as the operands decode it.
template <int FMT, int D>
__device__ __forceinline__ float value_at(const AttnArgs& a, int64_t base, int row, int d) {
    if constexpr (FMT == MOE_KV_BF16) {
        return bf16_to_f32(reinterpret_cast<const uint16_t*>(a.v)[(base + row) * D + d]);
    } else {
        constexpr int KG = v_keys_per_piece(D), C = D / 32;
        const int byte = d / 2;
        const uint32_t w = a.v[base * (D / 2) + (row / KG) * (KG * D / 2) + (byte / C) * 16 + (row % KG) * C + byte % C];
        const uint32_t sb = a.vs[base * C + (row / 8) * (8 * C) + (d / 32) * 8 + row % 8];
        const uint32_t pair = decode2<0>(w, e8m0_as_scale(sb));
        return __uint_as_float(d & 1 ? pair & 0xFFFF0000u : pair << 16);
    }
}

// What a row sees: keys j < up with j >= lo or j < sinks (none if up <= 0).
struct View {
    int up, lo;
};

__device__ __forceinline__ uint32_t pack_bf16(float x, float y) {
    bf16x2_t r;
    r[0] = (__bf16)x;
    r[1] = (__bf16)y;
    return __builtin_bit_cast(uint32_t, r);
}

// MT tiles of 16 rows per wave.
template <int FMT, int D, int MT>
__global__ __launch_bounds__(kThreads) void k_attn(AttnArgs a) {
    constexpr int NT = D / 16, KS = D / 32, ROWS = 16 * MT;
    __shared__ float sh_o[kWaves][16][D + 4];
    __shared__ float sh_m[kWaves][16], sh_l[kWaves][16];
    const int tid = threadIdx.x, lane = tid % kWave, wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int m = lane % 16, g = lane / 16;
    int id = blockIdx.x;
    const int rt0 = id % a.row_tiles; id /= a.row_tiles;
    const int split = id % a.nsplit; id /= a.nsplit;
    const int hk = id % a.Hk, b = id / a.Hk;
    const Seq sq = sequence(a, b);
    const int32_t* trow = a.table + (size_t)b * a.W;
    const int rows = sq.n * a.G;                   // (token, head of the group) pairs, token-major

    for (int r0 = rt0 * ROWS; r0 < rows; r0 += a.row_tiles * ROWS) {
        const int p0 = sq.kv - sq.n + r0 / a.G, p1 = sq.kv - sq.n + (min(r0 + ROWS, rows) - 1) / a.G;
        const Range rg = tiles_of(a, p0, p1, sq.kv);
        const bool alone = rg.total <= a.share || a.nsplit == 1;
        const int c0 = split * a.share;
        if (split > 0 && (alone || c0 >= rg.total)) continue;
        // the last workgroup along the keys takes what is left
        const int c1 = alone || split == a.nsplit - 1 ? rg.total : min(c0 + a.share, rg.total);

        // queries and views of this lane's row in each 16-row tile
        bf16x8_t qf[MT][KS];
        View vw[MT];
#pragma unroll
        for (int q = 0; q < MT; ++q) {
            const int r = r0 + 16 * q + m;
            const bool in = r < rows;
            const int tok = in ? r / a.G : 0, h = in ? hk * a.G + r % a.G : 0;
            const int p = sq.kv - sq.n + tok;
            vw[q].up = !in || p < 0 ? 0 : a.causal ? min(p + 1, sq.kv) : sq.kv;
            vw[q].lo = a.window > 0 ? (int)max((int64_t)p - a.window + 1, (int64_t)0) : 0;
            const uint16_t* src = a.q + (int64_t)(sq.start + tok) * a.qs + (int64_t)h * D + g * (D / 4);
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                u32x4_t x{0, 0, 0, 0};
                if (in) x = *reinterpret_cast<const u32x4_t*>(src + 8 * s);
                qf[q][s] = __builtin_bit_cast(bf16x8_t, x);
            }
        }
        // keys that every row of the tile sees: [all_lo, all_up) and below all_sink
        const int all_up = p0 < 0 ? 0 : a.causal ? min(p0 + 1, sq.kv) : sq.kv;
        const int all_lo = a.window > 0 ? (int)max((int64_t)p1 - a.window + 1, (int64_t)0) : 0;

        f32x4_t o[MT][NT];
        float mx[MT], ls[MT];
#pragma unroll
        for (int q = 0; q < MT; ++q) {
            mx[q] = -INFINITY;
            ls[q] = 0.f;
#pragma unroll
            for (int n = 0; n < NT; ++n) o[q][n] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        }

        Raw<FMT, D> cur, nxt;
        Pages pc{}, pn{};
        int c = c0 + wave;
        auto tile_at = [&](int x) { return x < rg.head ? x : rg.lo + x - rg.head; };
        if (c < c1) {
            pc = pages_of(a, trow, tile_at(c), sq.kv);
            load_tile<FMT, D>(cur, a, pc, tile_at(c), hk, lane);
        }
        for (; c < c1; c += kWaves) {
            const int tile = tile_at(c), key0 = tile * kTile;
            if (c + kWaves < c1) {
                const int tn = tile_at(c + kWaves);
                pn = pages_of(a, trow, tn, sq.kv);
                load_tile<FMT, D>(nxt, a, pn, tn, hk, lane);
            }
            // scores
            f32x4_t sc[MT][2];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
#pragma unroll
                for (int q = 0; q < MT; ++q) sc[q][t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int s = 0; s < KS; ++s) {
                    const bf16x8_t kf = k_operand<FMT, D>(cur, t, s);
#pragma unroll
                    for (int q = 0; q < MT; ++q)
                        sc[q][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, qf[q][s], sc[q][t], 0, 0, 0);
                }
            }
            // A tile that every row sees whole needs no mask.  Else: keys in
            // no page or behind the last are dead (their values count as 0), the rest is
            // masked row by row.
            const bool whole = pc.p[0] >= 0 && pc.p[1] >= 0 && key0 + kTile <= all_up &&
                               (key0 >= all_lo || key0 + kTile <= a.sinks);
            uint32_t live = 0xFF;                  // of keys key0 + 8 g + j
            uint32_t seen[MT];
            bool slow = false;
            if (!whole) {
                const int kg = key0 + 8 * g;
                const int left = (g < 2 ? pc.p[0] : pc.p[1]) >= 0 ? min(max(sq.kv - kg, 0), 8) : 0;
                live = (1u << left) - 1;
#pragma unroll
                for (int q = 0; q < MT; ++q) {
                    uint32_t see = 0;
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        see |= (uint32_t)(kg + j < vw[q].up && (kg + j >= vw[q].lo || kg + j < a.sinks)) << j;
                    seen[q] = see & live;
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (!((seen[q] >> j) & 1)) sc[q][j / 4][j % 4] = -INFINITY;
                }
                slow = __any(wild_values<FMT, D>(cur, live));
            }
            // softmax weights, in the lane and order of the second product's operand
            bf16x8_t pf[MT];
            float pw[MT][8];
            bool up = false;
            float tm[MT];
#pragma unroll
            for (int q = 0; q < MT; ++q) {
                tm[q] = sc[q][0][0];
#pragma unroll
                for (int j = 1; j < 8; ++j) tm[q] = fmaxf(tm[q], sc[q][j / 4][j % 4]);
                tm[q] *= a.c;
                up |= tm[q] > mx[q] + kSlack;
            }
            if (__any(up)) {
#pragma unroll
                for (int q = 0; q < MT; ++q) {
                    float t = fmaxf(tm[q], __shfl_xor(tm[q], 16));
                    t = fmaxf(t, __shfl_xor(t, 32));
                    const float mn = fmaxf(mx[q], t);
                    const float f = mn == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(mx[q] - mn);
                    mx[q] = mn;
                    ls[q] *= f;
#pragma unroll
                    for (int n = 0; n < NT; ++n) o[q][n] *= f;
                }
            }
#pragma unroll
            for (int q = 0; q < MT; ++q) {
                const float ref = mx[q] == -INFINITY ? 0.f : mx[q];
                u32x4_t w;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    pw[q][j] = __builtin_amdgcn_exp2f(fmaf(sc[q][j / 4][j % 4], a.c, -ref));
                    ls[q] += pw[q][j];
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) w[i] = pack_bf16(pw[q][2 * i], pw[q][2 * i + 1]);
                pf[q] = __builtin_bit_cast(bf16x8_t, w);
            }
            if (!slow) {
                auto pv = [&](auto U) {
                    constexpr int u = decltype(U)::value;
                    bf16x8_t va, vb;
                    v_operand<FMT, D, u>(cur, live, va, vb);
#pragma unroll
                    for (int q = 0; q < MT; ++q) {
                        o[q][2 * u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(va, pf[q], o[q][2 * u], 0, 0, 0);
                        o[q][2 * u + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vb, pf[q], o[q][2 * u + 1], 0, 0, 0);
                    }
                };
                pv(std::integral_constant<int, 0>{});
                pv(std::integral_constant<int, 1>{});
                if constexpr (D == 128) {
                    pv(std::integral_constant<int, 2>{});
                    pv(std::integral_constant<int, 3>{});
                }
            } else {
                // A partly visible tile with an infinite or NaN value: the
                // matrix product would spread 0 x inf to rows that do not see
                // it, so only the rows that see a key add it, one key at a time.
                for (int gs = 0; gs < 4; ++gs) {
                    const int64_t base = ((int64_t)max(pc.p[gs / 2], 0) * a.Hk + hk) << a.shift;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int row = (key0 + 8 * gs + j) & ((1 << a.shift) - 1);
#pragma unroll
                        for (int q = 0; q < MT; ++q) {
                            const float w = __shfl(pw[q][j], m + 16 * gs);
                            const bool sees = (__shfl(seen[q], m + 16 * gs) >> j) & 1;
                            if (!__any(sees)) continue;
#pragma unroll
                            for (int n = 0; n < NT; ++n)
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    const float x = value_at<FMT, D>(a, base, row, (4 * g + i) * NT + n);
                                    if (sees) o[q][n][i] = fmaf(w, x, o[q][n][i]);
                                }
                        }
                    }
                }
            }
            cur = nxt;
            pc = pn;
        }

        // join the four waves, 16 rows at a time; a thread takes D/16
        // elements of one row
#pragma unroll
        for (int q = 0; q < MT; ++q) {
            float l = ls[q] + __shfl_xor(ls[q], 16);
            l += __shfl_xor(l, 32);
            __syncthreads();
            if (g == 0) {
                sh_m[wave][m] = mx[q];
                sh_l[wave][m] = l;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int n = 0; n < NT; n += 4)
                    *reinterpret_cast<f32x4_t*>(&sh_o[wave][m][(4 * g + i) * NT + n]) =
                        f32x4_t{o[q][n][i], o[q][n + 1][i], o[q][n + 2][i], o[q][n + 3][i]};
            __syncthreads();
            const int rr = tid / 16, d0 = (tid % 16) * NT;
            const int r = r0 + 16 * q + rr;
            if (r < rows) {
                float top = sh_m[0][rr];
#pragma unroll
                for (int w = 1; w < kWaves; ++w) top = fmaxf(top, sh_m[w][rr]);
                const float ref = top == -INFINITY ? 0.f : top;
                float acc[NT], lt = 0.f;
#pragma unroll
                for (int n = 0; n < NT; ++n) acc[n] = 0.f;
#pragma unroll
                for (int w = 0; w < kWaves; ++w) {
                    const float f = __builtin_amdgcn_exp2f(sh_m[w][rr] - ref);
                    lt += f * sh_l[w][rr];
#pragma unroll
                    for (int n = 0; n < NT; ++n) acc[n] += f * sh_o[w][rr][d0 + n];
                }
                const int t = sq.start + r / a.G, h = hk * a.G + r % a.G;
                if (alone) {
                    const float inv = lt == 0.f ? 0.f : 1.f / lt;
                    uint32_t w[NT / 2];
#pragma unroll
                    for (int n = 0; n < NT / 2; ++n) w[n] = pack_bf16(acc[2 * n] * inv, acc[2 * n + 1] * inv);
                    uint32_t* dst = reinterpret_cast<uint32_t*>(a.out + (int64_t)t * a.os + (int64_t)h * D + d0);
                    if constexpr (NT == 8) *reinterpret_cast<u32x4_t*>(dst) = u32x4_t{w[0], w[1], w[2], w[3]};
                    else *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
                } else {
                    const int64_t at = ((int64_t)t * a.H + h) * a.nsplit + split;
#pragma unroll
                    for (int n = 0; n < NT; n += 4)
                        *reinterpret_cast<f32x4_t*>(a.part + at * D + d0 + n) =
                            f32x4_t{acc[n], acc[n + 1], acc[n + 2], acc[n + 3]};
                    if (d0 == 0) *reinterpret_cast<float2*>(a.stat + at * 2) = make_float2(top, lt);
                }
            }
        }
    }
}

// Rows whose keys several workgroups shared: out = sum 2^(m_s - m) O_s / sum
// 2^(m_s - m) l_s over the shares in order.  A wave per row.
template <int D>
__device__ __forceinline__ void join_row(const AttnArgs& a, int rows_per_tile, int64_t row, int lane) {
    constexpr int E = D / 64;                      // elements per lane
    const int t = (int)(row / a.H), h = (int)(row % a.H);
    // the sequence of row t: the last that starts at or before it
    int lo = 0, hi = a.B;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.cu_q[mid] <= t) lo = mid; else hi = mid;
    }
    const Seq sq = sequence(a, lo);
    if (t < sq.start || t >= sq.start + sq.n) return;
    const int rows = sq.n * a.G, r = (t - sq.start) * a.G + h % a.G;
    const int r0 = r / rows_per_tile * rows_per_tile;
    const Range rg = tiles_of(a, sq.kv - sq.n + r0 / a.G, sq.kv - sq.n + (min(r0 + rows_per_tile, rows) - 1) / a.G, sq.kv);
    if (rg.total <= a.share) return;               // written by its one workgroup
    const int used = min((rg.total + a.share - 1) / a.share, a.nsplit);
    const float* stat = a.stat + row * a.nsplit * 2;
    float top = -INFINITY;
    for (int s = lane; s < used; s += kWave) top = fmaxf(top, stat[2 * s]);
#pragma unroll
    for (int off = kWave / 2; off >= 1; off >>= 1) top = fmaxf(top, __shfl_xor(top, off));
    const float ref = top == -INFINITY ? 0.f : top;
    const float* part = a.part + row * a.nsplit * D + lane * E;
    float acc[E] = {}, l = 0.f;
    for (int s = 0; s < used; ++s) {
        const float f = __builtin_amdgcn_exp2f(stat[2 * s] - ref);
        l += f * stat[2 * s + 1];
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] += f * part[(int64_t)s * D + e];
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    uint16_t* dst = a.out + (int64_t)t * a.os + (int64_t)h * D + lane * E;
    if constexpr (E == 2) *reinterpret_cast<uint32_t*>(dst) = pack_bf16(acc[0] * inv, acc[1] * inv);
    else *dst = (uint16_t)(pack_bf16(acc[0] * inv, 0.f) & 0xFFFF);
}

template <int D>
__global__ __launch_bounds__(kThreads) void k_attn_join(AttnArgs a, int rows_per_tile) {
    const int lane = threadIdx.x % kWave;
    for (int64_t row = (int64_t)blockIdx.x * kWaves + threadIdx.x / kWave; row < (int64_t)a.T * a.H;
         row += (int64_t)gridDim.x * kWaves)
        join_row<D>(a, rows_per_tile, row, lane);
}

// Launch shape: a function of the sizes alone, so that the workspace's size
// and the launch agree.
struct Shape {
    int mt, row_tiles, share, nsplit;
};
Shape shape_of(const moe_mxfp4_attn_args& p, const moe_mxfp4_kv_cache& c) {
    Shape s{};
    const int64_t G = p.heads / c.kv_heads;
    const int64_t mq = p.max_q < p.num_tokens ? p.max_q : p.num_tokens;
    const int64_t rows = mq * G;
    s.mt = rows <= 16 ? 1 : rows <= 32 ? 2 : 4;
    int64_t tiles = (rows + 16 * s.mt - 1) / (16 * s.mt);
    int64_t keys = p.max_kv;
    if (p.window > 0) {
        const int64_t w = (int64_t)p.window + 16 * s.mt / G + 1 + p.sinks + 2 * kTile;
        if (w < keys) keys = w;
    }
    const int64_t kt = (keys + kTile - 1) / kTile;
    const int64_t pairs = (int64_t)p.batch * c.kv_heads;
    // the grid stays below 2^22 workgroups: more row tiles than fit are walked by a loop
    const int64_t most = (1 << 22) / pairs > 0 ? (1 << 22) / pairs : 1;
    if (tiles > most) tiles = most;
    const int64_t want = 1024, base = pairs * tiles;
    int64_t n = want / base;
    const int64_t cap = kt / (2 * kWaves);         // two tiles a wave at least
    if (n > cap) n = cap;
    if (n > 64) n = 64;
    if (n < 1) n = 1;
    int64_t share = (kt + n - 1) / n;
    share = (share + kWaves - 1) / kWaves * kWaves;
    n = (kt + share - 1) / share;
    s.row_tiles = (int)tiles;
    s.share = (int)share;
    s.nsplit = (int)n;
    return s;
}

template <int FMT, int D>
hipError_t launch_fmt(const AttnArgs& a, const Shape& sh, hipStream_t s) {
    const dim3 grid((unsigned)((int64_t)a.B * a.Hk * sh.nsplit * sh.row_tiles)), block(kThreads);
    if (sh.mt == 1) hipLaunchKernelGGL((k_attn<FMT, D, 1>), grid, block, 0, s, a);
    else if (sh.mt == 2) hipLaunchKernelGGL((k_attn<FMT, D, 2>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((k_attn<FMT, D, 4>), grid, block, 0, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || sh.nsplit == 1) return e;
    const int64_t wgs = ((int64_t)a.T * a.H + kWaves - 1) / kWaves;
    hipLaunchKernelGGL((k_attn_join<D>), dim3((unsigned)(wgs < 65536 ? wgs : 65536)), block, 0, s, a, 16 * sh.mt);
    return hipGetLastError();
}

size_t sums_bytes(const moe_mxfp4_attn_args& p, const moe_mxfp4_kv_cache& c, const Shape& s) {
    return (size_t)p.num_tokens * p.heads * s.nsplit * c.head_dim * sizeof(float);
}

}  // namespace

size_t attention_workspace_bytes(const moe_mxfp4_attn_args& p, const moe_mxfp4_kv_cache& c) {
    const Shape s = shape_of(p, c);
    if (s.nsplit == 1) return 0;
    return sums_bytes(p, c, s) + (size_t)p.num_tokens * p.heads * s.nsplit * 2 * sizeof(float);
}

hipError_t launch_attention(const moe_mxfp4_attn_args& p, const moe_mxfp4_kv_cache& c, void* workspace,
                            hipStream_t s) {
    const Shape sh = shape_of(p, c);
    AttnArgs a{};
    a.q = static_cast<const uint16_t*>(p.q); a.out = static_cast<uint16_t*>(p.out);
    a.table = p.block_table; a.cu_q = p.cu_q; a.kv_lens = p.kv_lens;
    a.k = static_cast<const uint8_t*>(c.k); a.v = static_cast<const uint8_t*>(c.v);
    a.ks = c.k_scale; a.vs = c.v_scale;
    a.part = static_cast<float*>(workspace);
    a.stat = sh.nsplit > 1 ? a.part + sums_bytes(p, c, sh) / sizeof(float) : nullptr;
    a.qs = p.q_stride; a.os = p.out_stride;
    a.B = p.batch; a.T = p.num_tokens; a.H = p.heads; a.Hk = c.kv_heads; a.G = p.heads / c.kv_heads;
    a.W = p.max_blocks; a.shift = log2_of(c.page_size); a.num_pages = c.num_pages;
    a.causal = p.causal != 0; a.window = p.window; a.sinks = p.sinks;
    a.share = sh.share; a.nsplit = sh.nsplit; a.row_tiles = sh.row_tiles;
    a.c = p.scale * 1.4426950408889634f;
    if (c.format == MOE_KV_MXFP4)
        return c.head_dim == 128 ? launch_fmt<MOE_KV_MXFP4, 128>(a, sh, s) : launch_fmt<MOE_KV_MXFP4, 64>(a, sh, s);
    return c.head_dim == 128 ? launch_fmt<MOE_KV_BF16, 128>(a, sh, s) : launch_fmt<MOE_KV_BF16, 64>(a, sh, s);
}

}  // namespace moe
