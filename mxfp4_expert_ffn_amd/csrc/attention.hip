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
// halves of registers by key; V's codes are stored so that these are 16-byte
// reads.
//
// Decoding E2M1 x E8M0 to bf16 is exact, queries are bf16 as given, scores and
// statistics float32; the softmax weights are rounded to bf16 for the second
// product (a relative 2^-9 each, as the operand type asks), and their sum is
// taken from the rounded ones.  The row maximum is only a reference point: it
// is moved when some score of the tile passes it by 2^8, so most tiles need
// neither a lane exchange nor a rescaling.
//
// Tiles go from memory to LDS without registers, a tile or two ahead of their
// use.  Up to 64 rows: four waves take every fourth tile of the workgroup's
// keys, each through a ring of its own, read it as stored and decode it in
// registers, and their sums are joined through LDS.  Those kernels are bound
// by the cache's bytes (64 sequences, one token each, 0.7 GB of MXFP4: 146-149
// us, 4.8-4.9 TB/s; a window of 1000 in bf16, 0.14 GB: 30 us, 4.7 TB/s) and,
// with more rows a key, by decoding (32 sequences, 8 tokens each: 57-61 us; the
// decode of a tile is 64 converts and 32 permutes whatever the rows).  More
// rows: the four waves take 48 rows each (64 of D = 64) and share every tile,
// decoded once into operands in LDS, so that its cost is divided by 192 rows.
// Those are bound by the matrix cores and by the LDS reads that feed them
// (2048 tokens behind 6144, 48 heads: 353 us a call, 1.02 PFLOP/s).
//
// Where there are few (sequence, head, set of rows) the keys of all of them
// are divided evenly over the workgroups the GPU holds, which leave float32
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
    float *part, *stat;                            // pieces: sums [workgroup][2][rows][D], (reference, sum of weights)
    int32_t* joins;                                // [workgroup][kJoinInts]: the rows that its last piece begins
    int64_t qs, os;
    int32_t B, T, H, Hk, G, W, shift, num_pages, causal, window, sinks;
    int32_t row_tiles;                             // even: workgroups along the rows of a sequence and head
    float c;                                       // scale * log2(e)
};

// A sequence: first row, rows, cached tokens (clamped to what there is).
struct Seq {
    int start, n, kv;
};
// Arrays read through the scalar cache.
typedef const __attribute__((address_space(4))) int32_t* ScalarInts;
template <typename Ints>
__device__ __forceinline__ Seq sequence(const AttnArgs& a, int b, Ints cu_q, Ints kv_lens) {
    Seq s;
    s.start = min(max(cu_q[b], 0), a.T);
    s.n = min(max(cu_q[b + 1], s.start), a.T) - s.start;
    s.kv = (int)min((int64_t)max(kv_lens[b], 0), (int64_t)a.W << a.shift);
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

// Keeps the compiler from moving the decoding of V out of a loop, where the
// decoded tile would take registers from the common path.
template <int D>
__device__ __forceinline__ void decode_anew(Raw<MOE_KV_MXFP4, D>& r) {
#pragma unroll
    for (int i = 0; i < D / 16; ++i) asm volatile("" : "+v"(r.v[i]));
}
template <int D>
__device__ __forceinline__ void decode_anew(Raw<MOE_KV_BF16, D>& r) {
#pragma unroll
    for (int i = 0; i < 8 * (D / 32); ++i) asm volatile("" : "+v"(r.v[i / (D / 32)][i % (D / 32)]));
}

// A tile of 32 keys in LDS as a wave fetches it: keys, values and (MXFP4)
// their scales, in the cache's order but for a permutation of the 16-byte
// chunks of a key row, chosen so that the 16 lanes that read the same chunk
// of 16 rows find it in different banks.
template <int FMT, int D> struct Tile {
    static constexpr int kRowBytes = FMT == MOE_KV_MXFP4 ? D / 2 : D * 2;
    static constexpr int kKeys = 0, kValues = kTile * kRowBytes, kScales = 2 * kValues;
    static constexpr int kBytes = kScales + (FMT == MOE_KV_MXFP4 ? 256 : 0);
    static constexpr int kFetches = 2 * kValues / 1024 + (FMT == MOE_KV_MXFP4 ? 1 : 0);   // loads of a wave
};

template <int N>
__device__ __forceinline__ void load_words(uint32_t* dst, const uint8_t* src) {
    if constexpr (N % 4 == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const u32x4_t x = *reinterpret_cast<const u32x4_t*>(src + 4 * i);
            dst[i] = x[0]; dst[i + 1] = x[1]; dst[i + 2] = x[2]; dst[i + 3] = x[3];
        }
    } else if constexpr (N == 1) {
        dst[0] = *reinterpret_cast<const uint32_t*>(src);
    } else {
        static_assert(N == 2, "");
        const uint2 x = *reinterpret_cast<const uint2*>(src);
        dst[0] = x.x; dst[1] = x.y;
    }
}

// A tile and the block table entries of its two halves of 16 keys, as they
// stand.  They are read through the scalar cache, and looked at only where they
// are used, a tile or more later, so that nothing waits for them.
struct Pages {
    int tile, a, b;
};
// row: the sequence's entries; last: its last key's
__device__ __forceinline__ Pages pages_of(const AttnArgs& a, ScalarInts row, int tile, int last) {
    const int first = (tile * kTile) >> a.shift, second = min(first + (a.shift == 4), last);
    typedef const __attribute__((address_space(4))) uint8_t* Bytes;
    return Pages{tile, *(ScalarInts)((Bytes)row + (uint32_t)(4 * first)), *(ScalarInts)((Bytes)row + (uint32_t)(4 * second))};
}
__device__ __forceinline__ bool in_cache(const AttnArgs& a, int page) { return (unsigned)page < (unsigned)a.num_pages; }

typedef __attribute__((address_space(3))) void lds_void;

// 16 (or 4) bytes per lane from base + off (base the same for all lanes)
// straight into LDS: lane L's go to lds + 16 L (4 L).  These loads write no
// register, so nothing the compiler allocates can be under way; it does not
// count them either, which is the point: of a ring slot chosen at run time it
// would assume that any load under way may write it, and wait for all of them
// before a read.  wait_loads() below does the waiting, before every read.
// m0 holds the LDS address; the compiler writes m0 only right before its own
// uses, of which there are none in this file, so it is not preserved.
// ONCE: no other wave reads these bytes, so they need not stay in the caches
// (nt): 5.6 against 4.7 TB/s of such loads alone over 0.7 GB of MXFP4 keys.
template <bool ONCE>
__device__ __forceinline__ void lds_dma16(const uint8_t* base, uint32_t off, uint32_t lds) {
    const uint64_t b = (uint64_t)(uintptr_t)base;
    const uint64_t s = (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(b >> 32)) << 32 |
                       (uint32_t)__builtin_amdgcn_readfirstlane((int)b);
    const uint32_t m = __builtin_amdgcn_readfirstlane((int)lds);
    if constexpr (ONCE)
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2 nt" ::"s"(m), "v"(off), "s"(s) : "memory");
    else
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(m), "v"(off), "s"(s) : "memory");
}
__device__ __forceinline__ void lds_dma16(const uint8_t* src, uint32_t lds) {
    const uint32_t m = __builtin_amdgcn_readfirstlane((int)lds);
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(m), "v"(src) : "memory");
}
__device__ __forceinline__ void lds_dma4(const uint8_t* src, uint32_t lds) {
    const uint32_t m = __builtin_amdgcn_readfirstlane((int)lds);
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(m), "v"(src) : "memory");
}

// The first LANES lanes' only, of all 64 that are active here.
template <int LANES, int BYTES>
__device__ __forceinline__ void lds_dma_low(const uint8_t* base, uint32_t off, uint32_t lds) {
    const uint64_t b = (uint64_t)(uintptr_t)base;
    const uint64_t s = (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(b >> 32)) << 32 |
                       (uint32_t)__builtin_amdgcn_readfirstlane((int)b);
    const uint32_t m = __builtin_amdgcn_readfirstlane((int)lds);
    const uint64_t on = ((uint64_t)1 << LANES) - 1;
    if constexpr (BYTES == 16)
        asm volatile("s_mov_b32 m0, %0\n\ts_mov_b64 exec, %3\n\tglobal_load_lds_dwordx4 %1, %2\n\ts_mov_b64 exec, -1"
                     ::"s"(m), "v"(off), "s"(s), "s"(on) : "memory");
    else
        asm volatile("s_mov_b32 m0, %0\n\ts_mov_b64 exec, %3\n\tglobal_load_lds_dword %1, %2\n\ts_mov_b64 exec, -1"
                     ::"s"(m), "v"(off), "s"(s), "s"(on) : "memory");
}

// Of a bf16 tile that waves share, chunk c of value row r is stored at c ^ this:
// a transposing read takes two neighbouring chunks of rows 8 g + k, k = 0..3,
// of all four g at once, and finds them in twice all banks.
__device__ constexpr int value_swizzle(int D, int r) {
    return D == 128 ? 2 * (r % 4 + 4 * (r / 8 % 2)) : 2 * (r % 4 / 2 + 2 * (r / 8 % 2));
}

// First row of a half tile's keys in the cache; page 0 stands in for none: read,
// then not used.
__device__ __forceinline__ int64_t half_row(const AttnArgs& a, int page, int key, int hk) {
    return (((int64_t)(in_cache(a, page) ? page : 0) * a.Hk + hk) << a.shift) + (key & ((1 << a.shift) - 1));
}

// Starts the loads of a tile into its slot dst (an LDS address, the same for
// all lanes).  What this wave read from the slot before has arrived.
template <int FMT, int D, bool ONCE>
__device__ __forceinline__ void fetch(uint32_t dst, const AttnArgs& a, const Pages& pg, int hk, int lane) {
    using T = Tile<FMT, D>;
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    const int64_t b0 = half_row(a, pg.a, pg.tile * kTile, hk), b1 = half_row(a, pg.b, pg.tile * kTile + 16, hk);
    if constexpr (FMT == MOE_KV_MXFP4 && D == 128) {
        // chunk c of row r is stored at c ^ (r / 8)
#pragma unroll
        for (int h = 0; h < 2; ++h)
            lds_dma16<ONCE>(a.k + (h ? b1 : b0) * 64, lane / 4 * 64 + ((lane % 4) ^ (2 * h + lane / 32)) * 16, dst + h * 1024);
#pragma unroll
        for (int h = 0; h < 2; ++h) lds_dma16<ONCE>(a.v + (h ? b1 : b0) * 64, lane * 16, dst + T::kValues + h * 1024);
        const uint8_t* sc = lane < 32 ? a.ks : a.vs;
        lds_dma4(sc + (lane & 16 ? b1 : b0) * 4 + lane % 16 * 4, dst + T::kScales);
    } else if constexpr (FMT == MOE_KV_MXFP4) {
        const int64_t base = lane < 32 ? b0 : b1;
        const int chunk = (lane % 2) ^ ((lane / 16) & 1);               // chunk c of row r at c ^ (r / 8 mod 2)
        lds_dma16(a.k + base * 32 + (lane / 2 % 16 * 32 + chunk * 16), dst);
        lds_dma16(a.v + base * 32 + lane % 32 * 16, dst + T::kValues);
        const uint8_t* sc = lane & 16 ? a.vs : a.ks;                    // lanes 32.. repeat lanes 0..31
        lds_dma4(sc + (lane & 8 ? b1 : b0) * 2 + lane % 8 * 4, dst + T::kScales);
    } else {
        constexpr int C = D / 8, R = 64 / C, N = kTile / R;             // chunks per row, rows per load, loads
#pragma unroll
        for (int i = 0; i < N; ++i) {
            // chunk c of row r at c ^ (its lane m = 4 (r / 8) + r mod 4)
            const int row = i * R + lane / C, mm = 4 * (row / 8) + row % 4;
            lds_dma16<ONCE>(a.k + (i < 16 / R ? b0 : b1) * (2 * D), row % 16 * (2 * D) + ((lane % C) ^ (mm % C)) * 16, dst + i * 1024);
        }
#pragma unroll
        for (int i = 0; i < N; ++i)
            lds_dma16<ONCE>(a.v + (i < 16 / R ? b0 : b1) * (2 * D) + i % (16 / R) * 1024, lane * 16, dst + T::kValues + i * 1024);
    }
}

// The same where the workgroup's four waves share the tile: wave `part` starts
// its loads, each of one half.  MXFP4: from these arrays, chosen once (chosen
// anew, they would be read from the arguments for every tile).
struct PartOf {
    const uint8_t *data, *scale;
    __device__ __forceinline__ PartOf(const AttnArgs& a, int part) {
        data = part < 2 ? a.k : a.v;
        scale = part < 2 ? a.ks : a.vs;
        asm volatile("" : "+s"(data), "+s"(scale));
    }
};
template <int FMT, int D>
__device__ __forceinline__ void fetch_part(uint32_t dst, const AttnArgs& a, const PartOf& from, const Pages& pg, int hk, int lane,
                                           int part) {
    using T = Tile<FMT, D>;
    if constexpr (FMT == MOE_KV_MXFP4) {
        const int h = part % 2;                    // keys or values of half h
        const bool keys = part < 2;
        const int64_t b = half_row(a, h ? pg.b : pg.a, pg.tile * kTile + 16 * h, hk);
        const uint8_t* src = from.data + b * (D / 2);
        const uint32_t to = dst + (keys ? 0 : T::kValues) + h * (8 * D);
        if constexpr (D == 128) {
            const int chunk = keys ? (lane % 4) ^ (2 * h + lane / 32) : lane % 4;
            lds_dma16<false>(src, lane / 4 * 64 + chunk * 16, to);
            lds_dma_low<16, 4>(from.scale + b * 4, lane * 4, dst + T::kScales + part * 64);
        } else {
            const int chunk = keys ? (lane % 2) ^ ((lane / 16) & 1) : lane % 2;
            lds_dma_low<32, 16>(src, lane / 2 * 32 + chunk * 16, to);
            lds_dma_low<8, 4>(from.scale + b * 2, lane * 4, dst + T::kScales + part * 32);
        }
    } else {
        constexpr int C = D / 8, R = 64 / C, N = kTile / R / kWaves;    // chunks per row, rows per load, loads
        const int h = part / 2;
        const int64_t b = half_row(a, h ? pg.b : pg.a, pg.tile * kTile + 16 * h, hk);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int row = (part * N + i) * R + lane / C, mm = 4 * (row / 8) + row % 4;
            lds_dma16<false>(a.k + b * (2 * D), row % 16 * (2 * D) + ((lane % C) ^ (mm % C)) * 16, dst + (part * N + i) * 1024);
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int row = (part * N + i) * R + lane / C;              // chunk c at c ^ value_swizzle
            lds_dma16<false>(a.v + b * (2 * D), row % 16 * (2 * D) + ((lane % C) ^ value_swizzle(D, row)) * 16,
                             dst + T::kValues + (part * N + i) * 1024);
        }
    }
}

// Waits until at most N loads of this wave are under way (they end in order).
template <int N>
__device__ __forceinline__ void wait_loads() {
    static_assert(N >= 0 && N < 64, "vmcnt range");
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

template <int FMT, int D>
__device__ __forceinline__ void read_keys(Raw<FMT, D>& r, const uint8_t* src, int lane) {
    const int m = lane % 16, g = lane / 16;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const int row = 8 * (m / 4) + 4 * t + m % 4;
        const uint8_t* p = src + row * Tile<FMT, D>::kRowBytes;
        if constexpr (FMT == MOE_KV_MXFP4) {
            if constexpr (D == 128) load_words<4>(r.k[t], p + (g ^ (m / 4)) * 16);
            else load_words<2>(r.k[t], p + ((g / 2) ^ ((m / 4) & 1)) * 16 + g % 2 * 8);
            r.kb[t] = src[Tile<FMT, D>::kScales + row * (D / 32) + g * D / 128];
        } else {
#pragma unroll
            for (int i = 0; i < D / 32; ++i)
                r.k[t][i] = *reinterpret_cast<const u32x4_t*>(p + ((g * (D / 32) + i) ^ (m % (D / 8))) * 16);
        }
    }
}

template <int FMT, int D>
__device__ __forceinline__ void read_values(Raw<FMT, D>& r, const uint8_t* src, int lane) {
    using T = Tile<FMT, D>;
    const int m = lane % 16, g = lane / 16;
    if constexpr (FMT == MOE_KV_MXFP4) {
        constexpr int KG = v_keys_per_piece(D);
#pragma unroll
        for (int i = 0; i < 8 / KG; ++i) load_words<4>(r.v + 4 * i, src + T::kValues + ((8 / KG) * g + i) * 256 + m * 16);
        const uint2 b = *reinterpret_cast<const uint2*>(src + T::kScales + kTile * (D / 32) + (g * (D / 32) + m * D / 512) * 8);
        r.vb[0] = b.x; r.vb[1] = b.y;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) load_words<D / 32>(r.v[j], src + T::kValues + (8 * g + j) * (2 * D) + m * (D / 8));
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
            // the convert reads the exponent field of its scale only, so the
            // other bytes around it may stay
            const uint32_t b = r.vb[j / 4];
            const float sc = __uint_as_float(j % 4 == 3 ? b >> 1 : b << (23 - 8 * (j % 4)));
            const int at = j * (D / 32) + U;       // byte of the lane's codes
            const uint32_t word = r.v[at / 4];
            w[j] = at % 4 == 0 ? decode2<0>(word, sc) : at % 4 == 1 ? decode2<1>(word, sc)
                 : at % 4 == 2 ? decode2<2>(word, sc) : decode2<3>(word, sc);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = r.v[j][U];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = (live >> j) & 1 ? w[j] : 0;     // nothing where live is the constant 0xFF
    u32x4_t lo, hi;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        lo[i] = __builtin_amdgcn_perm(w[2 * i + 1], w[2 * i], 0x05040100u);
        hi[i] = __builtin_amdgcn_perm(w[2 * i + 1], w[2 * i], 0x07060302u);
    }
    first = __builtin_bit_cast(bf16x8_t, lo);
    second = __builtin_bit_cast(bf16x8_t, hi);
}

// Two bf16 at once: a bit of 0x80008000 is set where one's exponent, kept by
// mask (0x7F80 of it), is all ones.
__device__ __forceinline__ uint32_t wild2(uint32_t w, uint32_t mask) { return (w & mask) + 0x00800080u; }

// Whether a live key of this lane has an infinite or NaN value (MXFP4: a
// scale with which 6 passes float32's range, or NaN).
template <int FMT, int D>
__device__ __forceinline__ bool wild_values(const Raw<FMT, D>& r, uint32_t live) {
    uint32_t wild = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const bool on = (live >> j) & 1;
        if constexpr (FMT == MOE_KV_MXFP4) {
            wild |= on && ((r.vb[j / 4] >> (8 * (j % 4))) & 0xFF) >= 253 ? 0x8000u : 0u;
        } else {
#pragma unroll
            for (int u = 0; u < D / 32; ++u) wild |= wild2(r.v[j][u], on ? 0x7F807F80u : 0u);
        }
    }
    return (wild & 0x80008000u) != 0;
}

__device__ __forceinline__ f32x4_t mfma(const bf16x8_t& x, const bf16x8_t& y, const f32x4_t& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, y, c, 0, 0, 0);
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

// The lowest n of 8 bits, n clamped to 0..8.
__device__ __forceinline__ uint32_t low_bits(int n) { return (1u << min(max(n, 0), 8)) - 1; }

// A wave's running softmax of MT tiles of 16 rows.
template <int D, int MT>
struct Sums {
    f32x4_t o[MT][D / 16];                         // O^T
    float l[MT];                                   // the weights' sum, of row lane % 16
    float m[MT];                                   // the reference, of row lane % 16
};

// The eight V^T operands of a tile, each handed to f(number, operand).
template <int FMT, int D, typename F>
__device__ __forceinline__ void each_v(const Raw<FMT, D>& r, uint32_t live, F f) {
    auto pair = [&](auto U) {
        bf16x8_t x, y;
        v_operand<FMT, D, decltype(U)::value>(r, live, x, y);
        f(2 * decltype(U)::value, x);
        f(2 * decltype(U)::value + 1, y);
    };
    pair(std::integral_constant<int, 0>{});
    pair(std::integral_constant<int, 1>{});
    if constexpr (D == 128) {
        pair(std::integral_constant<int, 2>{});
        pair(std::integral_constant<int, 3>{});
    }
}

// S^T of a tile; key(t, s): the operand of half tile t, step s.
template <int D, int MT, typename Key>
__device__ __forceinline__ void scores(f32x4_t (&sc)[MT][2], Key key, const bf16x8_t (&qf)[MT][D / 32]) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
#pragma unroll
        for (int q = 0; q < MT; ++q) sc[q][t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < D / 32; ++s) {
            const bf16x8_t kf = key(t, s);
#pragma unroll
            for (int q = 0; q < MT; ++q) sc[q][t] = mfma(kf, qf[q][s], sc[q][t]);
        }
    }
}

// This lane's largest score of each row, in the exponent's units.
template <int MT>
__device__ __forceinline__ void tops(float (&t)[MT], const f32x4_t (&sc)[MT][2], float c) {
#pragma unroll
    for (int q = 0; q < MT; ++q) {
        float x = fmaxf(fmaxf(sc[q][0][0], sc[q][0][1]), sc[q][0][2]);
        x = fmaxf(fmaxf(x, sc[q][0][3]), sc[q][1][0]);
        x = fmaxf(fmaxf(x, sc[q][1][1]), sc[q][1][2]);
        t[q] = fmaxf(x, sc[q][1][3]) * c;
    }
}

// Softmax weights, in the lane and order of the second product's operand.
// Their sum comes from the same rounded weights, as one more product, with ones.
template <int D, int MT>
__device__ __forceinline__ void weights(Sums<D, MT>& a, bf16x8_t (&pf)[MT], const f32x4_t (&sc)[MT][2], float c) {
    const uint32_t one2 = 0x3F803F80u;
    const bf16x8_t ones = __builtin_bit_cast(bf16x8_t, u32x4_t{one2, one2, one2, one2});
#pragma unroll
    for (int q = 0; q < MT; ++q) {
        const float ref = a.m[q] == -INFINITY ? 0.f : a.m[q];
        float p[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) p[j] = __builtin_amdgcn_exp2f(fmaf(sc[q][j / 4][j % 4], c, -ref));
        u32x4_t w;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = pack_bf16(p[2 * i], p[2 * i + 1]);
        pf[q] = __builtin_bit_cast(bf16x8_t, w);
        // all four registers of the product are the same; one is kept
        a.l[q] += mfma(ones, pf[q], f32x4_t{0.f, 0.f, 0.f, 0.f})[0];
    }
}

// A tile as the waves along the keys hold it: in registers as stored, decoded
// on use.
template <int FMT, int D> struct RawTile {
    Raw<FMT, D> r;
    __device__ __forceinline__ RawTile(const uint8_t* src, int lane) {
        read_keys<FMT, D>(r, src, lane);
        read_values<FMT, D>(r, src, lane);
    }
    __device__ __forceinline__ bf16x8_t key(int t, int s) const { return k_operand<FMT, D>(r, t, s); }
    // f(n, operand of tile n), of the keys in `keep`
    template <typename F> __device__ __forceinline__ void values(uint32_t keep, F f) const { each_v<FMT, D>(r, keep, f); }
    __device__ __forceinline__ bool wild(uint32_t live) const { return wild_values<FMT, D>(r, live); }
    __device__ __forceinline__ void anew() { decode_anew(r); }
};

// A tile as the waves along the rows share it: operands in LDS, 16 bytes per
// lane, dead keys' values already 0.
template <int D> struct SharedTile {
    const uint8_t* f;                              // + 16 lane
    static constexpr int kBytes = (2 * (D / 32) + D / 16) * 1024;
    __device__ __forceinline__ bf16x8_t at(int i) const { return *reinterpret_cast<const bf16x8_t*>(f + i * 1024); }
    __device__ __forceinline__ bf16x8_t key(int t, int s) const { return at(t * (D / 32) + s); }
    __device__ __forceinline__ bf16x8_t value(int n) const { return at(2 * (D / 32) + n); }
};

// A bf16 tile needs no decoding, so the waves along the rows read it as
// fetched: rows of keys are operands as they stand, rows of values become
// operands by the LDS's transposing reads.  Its tile n holds elements 16 n ..
// 16 n + 15 in order.
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef const __attribute__((address_space(3))) uint8_t* LdsBytes;
template <int D> struct DirectTile {
    LdsBytes k[2], v;                              // this lane's key rows, and where its first transposing read begins
    int m;
    __device__ __forceinline__ DirectTile(LdsBytes tile, int lane) : m(lane % 16) {
        const int g = lane / 16, row = 8 * g + m / 4;
#pragma unroll
        for (int t = 0; t < 2; ++t) k[t] = tile + (8 * (m / 4) + 4 * t + m % 4) * (2 * D);
        v = tile + Tile<MOE_KV_BF16, D>::kValues + row * (2 * D) + ((m % 4 / 2) ^ value_swizzle(D, row)) * 16 + m % 2 * 8;
        m = ((lane / 16) * (D / 32)) ^ (m % (D / 8));
    }
    __device__ __forceinline__ bf16x8_t key(int t, int s) const {
        return *reinterpret_cast<const __attribute__((address_space(3))) bf16x8_t*>(k[t] + (m ^ s) * 16);
    }
    __device__ __forceinline__ bf16x8_t value(int n) const {
        // bits 5 and up of the address select the pair of chunks within a row
        LdsBytes p = (LdsBytes)(uintptr_t)((uint32_t)(uintptr_t)v ^ (uint32_t)(32 * n));
        const s16x4_t a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4_t*)p);
        const s16x4_t b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4_t*)(p + 4 * (2 * D)));
        return __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
    }
};

// Such tiles for attend_part.
template <int D, typename Tile_> struct Masked : Tile_ {
    using Tile_::Tile_;
    __device__ __forceinline__ Masked(const Tile_& t) : Tile_(t) {}
    template <typename F> __device__ __forceinline__ void values(uint32_t keep, F f) const {
#pragma unroll
        for (int n = 0; n < D / 16; ++n) {
            u32x4_t w = __builtin_bit_cast(u32x4_t, this->value(n));
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] &= ((keep >> (2 * i)) & 1 ? 0xFFFFu : 0u) | ((keep >> (2 * i + 1)) & 1 ? 0xFFFF0000u : 0u);
            f(n, __builtin_bit_cast(bf16x8_t, w));
        }
    }
    // whether one of the lane group's live keys has an infinite or NaN value
    __device__ __forceinline__ bool wild(uint32_t live) const {
        uint32_t mask[4], x = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            mask[i] = ((live >> (2 * i)) & 1 ? 0x7F80u : 0u) | ((live >> (2 * i + 1)) & 1 ? 0x7F800000u : 0u);
#pragma unroll
        for (int n = 0; n < D / 16; ++n) {
            const u32x4_t w = __builtin_bit_cast(u32x4_t, this->value(n));
#pragma unroll
            for (int i = 0; i < 4; ++i) x |= wild2(w[i], mask[i]);
        }
        return (x & 0x80008000u) != 0;
    }
    __device__ __forceinline__ void anew() {}
};

// After a loop that is left from its middle too: keeps the compiler from telling
// the ways out apart.  Of a loop with several exits it would carry all sums,
// as before the tile and as after, to one common end: twice the registers.
__device__ __forceinline__ void one_exit(int& x, int& y) { asm volatile("" : "+s"(x), "+s"(y)); }

__device__ __forceinline__ void pin() { __builtin_amdgcn_sched_barrier(0); }

// The common tile: every row sees every key.  False, with the sums untouched,
// if a reference has to move.
template <int D, int MT, typename Src>
__device__ __forceinline__ bool attend_whole(Sums<D, MT>& sums, const Src& src, const bf16x8_t (&qf)[MT][D / 32], float c) {
    f32x4_t sc[MT][2];
    scores<D, MT>(sc, [&](int t, int s) { return src.key(t, s); }, qf);
    float top[MT];
    tops<MT>(top, sc, c);
    bool move = false;
#pragma unroll
    for (int q = 0; q < MT; ++q) move |= top[q] > sums.m[q] + kSlack;
    if (__any(move)) return false;
    bf16x8_t pf[MT];
    weights<D, MT>(sums, pf, sc, c);
    src.values(0xFF, [&](int n, const bf16x8_t& v) {
#pragma unroll
        for (int q = 0; q < MT; ++q) sums.o[q][n] = mfma(v, pf[q], sums.o[q][n]);
    });
    return true;
}

// The same of a shared tile, operands asked for kAhead steps before their
// product: read on use, each would wait for LDS longer than its MT matrix
// instructions last.  The first values' reads pass under the softmax.
constexpr int kAhead = 4;
template <int D, int MT, typename Src>
__device__ __forceinline__ bool attend_shared(Sums<D, MT>& sums, const Src& src, const bf16x8_t (&qf)[MT][D / 32], float c) {
    constexpr int KS = D / 32, NT = D / 16;
    bf16x8_t x[kAhead];
    f32x4_t sc[MT][2];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) x[i] = src.key(i / KS, i % KS);
    pin();
#pragma unroll
    for (int i = 0; i < 2 * KS; ++i) {
        const int t = i / KS, s = i % KS;
#pragma unroll
        for (int q = 0; q < MT; ++q) sc[q][t] = mfma(x[i % kAhead], qf[q][s], s == 0 ? f32x4_t{0.f, 0.f, 0.f, 0.f} : sc[q][t]);
        const int next = i + kAhead;
        if (next < 2 * KS) x[i % kAhead] = src.key(next / KS, next % KS);
        else x[i % kAhead] = src.value(next - 2 * KS);
        pin();
    }
    float top[MT];
    tops<MT>(top, sc, c);
    bool move = false;
#pragma unroll
    for (int q = 0; q < MT; ++q) move |= top[q] > sums.m[q] + kSlack;
    if (__any(move)) return false;
    bf16x8_t pf[MT];
    weights<D, MT>(sums, pf, sc, c);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int q = 0; q < MT; ++q) sums.o[q][n] = mfma(x[n % kAhead], pf[q], sums.o[q][n]);
        if (n + kAhead < NT) x[n % kAhead] = src.value(n + kAhead);
        pin();
    }
    return true;
}

// Any tile.  live: which of the lane group's 8 keys exist; kg: the first of
// them.  WILD: some value is infinite or NaN.
template <int D, int MT, bool WILD, typename Src>
__device__ __forceinline__ void attend_part(Sums<D, MT>& a, const Src& src, const bf16x8_t (&qf)[MT][D / 32],
                                            const View (&vw)[MT], int kg, uint32_t live, int sinks, float c) {
    f32x4_t sc[MT][2];
    scores<D, MT>(sc, [&](int t, int s) { return src.key(t, s); }, qf);
    uint32_t seen[MT];
#pragma unroll
    for (int q = 0; q < MT; ++q) {
        seen[q] = low_bits(vw[q].up - kg) & (~low_bits(vw[q].lo - kg) | low_bits(sinks - kg)) & live;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (!((seen[q] >> j) & 1)) sc[q][j / 4][j % 4] = -INFINITY;
    }
    float tm[MT];
    tops<MT>(tm, sc, c);
#pragma unroll
    for (int q = 0; q < MT; ++q) {
        float t = fmaxf(tm[q], __shfl_xor(tm[q], 16));
        t = fmaxf(t, __shfl_xor(t, 32));
        if (!__any(t > a.m[q] + kSlack)) continue;
        const float mn = fmaxf(a.m[q], t);
        const float f = mn == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(a.m[q] - mn);
        a.m[q] = mn;
        a.l[q] *= f;
#pragma unroll
        for (int n = 0; n < D / 16; ++n) a.o[q][n] *= f;
    }
    bf16x8_t pf[MT];
    weights<D, MT>(a, pf, sc, c);
    if constexpr (WILD) {
        // One product would spread 0 x inf to rows that do not see the key.
        // So a product per row, with the values that this row sees, of which
        // only that row is kept.
        for (int n = 0; n < 16; ++n) {
            Src x = src;
            x.anew();
#pragma unroll
            for (int q = 0; q < MT; ++q) {
                const uint32_t own = __shfl(seen[q], (threadIdx.x & 48) + n);
                const bool mine = (threadIdx.x & 15) == (unsigned)n;
                x.values(own, [&](int k, const bf16x8_t& v) {
                    const f32x4_t y = mfma(v, pf[q], f32x4_t{0.f, 0.f, 0.f, 0.f});
                    if (mine) a.o[q][k] += y;
                });
            }
        }
    } else {
        src.values(live, [&](int k, const bf16x8_t& v) {
#pragma unroll
            for (int q = 0; q < MT; ++q) a.o[q][k] = mfma(v, pf[q], a.o[q][k]);
        });
    }
}

// A wave's share of turning a tile as fetched (raw) into operands (dst): waves 0
// and 1 take the keys of a half tile each, 2 and 3 half of the elements of the
// values.  live: which of the lane group's 8 keys exist.
template <int FMT, int D, int HALF>
__device__ __forceinline__ void share_keys(const uint8_t* raw, uint8_t* dst, int lane) {
    const int m = lane % 16, g = lane / 16, row = 8 * (m / 4) + 4 * HALF + m % 4;
    const uint8_t* p = raw + row * Tile<FMT, D>::kRowBytes;
    uint8_t* to = dst + HALF * (D / 32) * 1024 + lane * 16;
    if constexpr (FMT == MOE_KV_MXFP4) {
        uint32_t w[D / 32];
        if constexpr (D == 128) load_words<4>(w, p + (g ^ (m / 4)) * 16);
        else load_words<2>(w, p + ((g / 2) ^ ((m / 4) & 1)) * 16 + g % 2 * 8);
        const float sc = e8m0_as_scale(raw[Tile<FMT, D>::kScales + row * (D / 32) + g * D / 128]);
#pragma unroll
        for (int s = 0; s < D / 32; ++s) *reinterpret_cast<bf16x8_t*>(to + s * 1024) = decode8_bf16(w[s], sc);
    } else {
#pragma unroll
        for (int s = 0; s < D / 32; ++s)
            *reinterpret_cast<u32x4_t*>(to + s * 1024) = *reinterpret_cast<const u32x4_t*>(p + ((g * (D / 32) + s) ^ (m % (D / 8))) * 16);
    }
}
template <int FMT, int D, int HALF>
__device__ __forceinline__ void share_values(const uint8_t* raw, uint8_t* dst, uint32_t live, int lane) {
    Raw<FMT, D> r;
    read_values<FMT, D>(r, raw, lane);
    uint8_t* to = dst + 2 * (D / 32) * 1024 + lane * 16;
    auto pair = [&](auto U) {
        constexpr int u = decltype(U)::value;
        bf16x8_t x, y;
        v_operand<FMT, D, u>(r, live, x, y);
        *reinterpret_cast<bf16x8_t*>(to + 2 * u * 1024) = x;
        *reinterpret_cast<bf16x8_t*>(to + (2 * u + 1) * 1024) = y;
    };
    pair(std::integral_constant<int, HALF * (D / 64)>{});
    if constexpr (D == 128) pair(std::integral_constant<int, HALF * (D / 64) + 1>{});
}
template <int FMT, int D>
__device__ __forceinline__ void share_out(const uint8_t* raw, uint8_t* dst, uint32_t live, bool all_live, int wave, int lane) {
    if (wave == 0) {
        share_keys<FMT, D, 0>(raw, dst, lane);
    } else if (wave == 1) {
        share_keys<FMT, D, 1>(raw, dst, lane);
    } else if (wave == 2) {
        if (all_live) share_values<FMT, D, 0>(raw, dst, 0xFF, lane);
        else share_values<FMT, D, 0>(raw, dst, live, lane);
    } else {
        if (all_live) share_values<FMT, D, 1>(raw, dst, 0xFF, lane);
        else share_values<FMT, D, 1>(raw, dst, live, lane);
    }
}

// A workgroup barrier that waits for this wave's LDS operations only: loads
// from memory stay under way.
__device__ __forceinline__ void lds_barrier() {
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// How the work is divided.  kEven: a workgroup per sequence, head and set of
// rows.  kQuota: all (sequence, head, set of rows) are laid end to end, a unit
// per tile of keys, and every workgroup takes the same number of units, which
// may begin and end inside one: such pieces leave float32 sums that k_attn_join
// adds up.  The workgroups find their units themselves, by a prefix sum over
// the sequences, since only the device knows the lengths.
enum { kEven, kQuota };
constexpr int kQuotaBatch = 1024;                  // sequences kQuota handles: four per thread, their sums in LDS
constexpr int kJoinInts = 8;
constexpr int kQuotaLeast = 16;                    // units a workgroup takes at least, where a sequence has them

// A sequence's sets of `per` rows, and the units each counts: as many tiles of
// keys as any of the sets sees, and one at least, so that every row is
// written.
struct Units {
    int tiles, sets;
};
__device__ __forceinline__ Units units_of(const AttnArgs& a, const Seq& sq, int per) {
    const int rows = sq.n * a.G;
    if (rows == 0) return Units{0, 0};
    int64_t t = ((int64_t)sq.kv + kTile - 1) / kTile;
    if (a.window > 0) {
        // a set's rows are of at most (per - 1) / G + 2 tokens; an interval of
        // keys touches (length + 2 (kTile - 1)) / kTile tiles at most
        const int64_t len = (int64_t)a.window + (a.causal ? (min(per, rows) - 1) / a.G + 1 : sq.n);
        t = min(t, (int64_t)((a.sinks + (int64_t)kTile - 1) / kTile + (len + 2 * (kTile - 1)) / kTile));
    }
    return Units{max((int)t, 1), (rows + per - 1) / per};
}

// A workgroup's 4 waves: WR along the rows (MT tiles of 16 each), 4 / WR along
// the keys.  WPE: waves per SIMD.
template <int FMT, int D, int MT, int WR, int WPE, int MODE>
__global__ __launch_bounds__(kThreads, WPE) void k_attn(AttnArgs a) {
    constexpr int NT = D / 16, KS = D / 32, WK = kWaves / WR, ROWS = 16 * MT * WR;
    constexpr int TPR = 16 / WR, E = D / TPR;      // threads per row and elements per thread in the join
    constexpr bool ONCE = WR == 1;                 // each key is read by one wave only
    constexpr bool SHARED = WR == kWaves;          // or by all four, at the same time
    using T = Tile<FMT, D>;
    typedef float JoinRows[kWaves][16][D + 4];
    constexpr bool DIRECT = SHARED && FMT == MOE_KV_BF16;      // as fetched
    constexpr int kRing = SHARED ? 0 : 2 * T::kBytes;
    constexpr int kTiles = DIRECT ? 3 * T::kBytes : SHARED ? 2 * (SharedTile<D>::kBytes + T::kBytes) : kWaves * kRing;
    constexpr int kLds = kTiles > (int)sizeof(JoinRows) ? kTiles : sizeof(JoinRows);
    __shared__ __align__(1024) uint8_t lds[kLds];
    __shared__ float sh_m[kWaves][16], sh_l[kWaves][16];
    __shared__ int64_t sh_start[MODE == kQuota ? kQuotaBatch + 1 : 1];
    __shared__ int64_t sh_sum[kWaves];
    __shared__ int sh_top[kWaves];
    JoinRows& sh_o = *reinterpret_cast<JoinRows*>(lds);
    const int tid = threadIdx.x, lane = tid % kWave, wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int wr = wave % WR, wk = wave / WR;
    const uint8_t* const base = lds + wave * kRing;
    const uint32_t lds_at = (uint32_t)(uintptr_t)(lds_void*)lds, mine = lds_at + wave * kRing;
    const int m = lane % 16, g = lane / 16;
    const ScalarInts cu_q = (ScalarInts)(uintptr_t)a.cu_q, kv_lens = (ScalarInts)(uintptr_t)a.kv_lens;

    // this workgroup's units [unit, last)
    int64_t unit, last, quota = 1;
    int joined = 0;                                // pieces of the rows that the last piece here begins
    int join_start = 0, join_r0 = 0, join_rows = 0, join_hk = 0;
    if constexpr (MODE == kQuota) {
        int64_t before[4], sum = 0;
        int most = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int b = tid * 4 + i;
            before[i] = sum;
            if (b < a.B) {
                const Units u = units_of(a, sequence(a, b, a.cu_q, a.kv_lens), ROWS);
                sum += (int64_t)u.sets * u.tiles;
                most = max(most, u.tiles);
            }
        }
        int64_t incl = sum;
#pragma unroll
        for (int off = 1; off < kWave; off <<= 1) {
            const int64_t o = __shfl_up(incl, off);
            if (lane >= off) incl += o;
            most = max(most, __shfl_xor(most, off));
        }
        if (lane == kWave - 1) {
            sh_sum[wave] = incl;
            sh_top[wave] = most;
        }
        __syncthreads();
        int64_t all = 0, ahead = 0;
        most = 0;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            if (w < wave) ahead += sh_sum[w];
            all += sh_sum[w];
            most = max(most, sh_top[w]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (tid * 4 + i <= a.B) sh_start[tid * 4 + i] = ahead + incl - sum + before[i];
        if (tid == 0) sh_start[a.B] = all;
        const int64_t share = (all * a.Hk + gridDim.x - 1) / gridDim.x;
        quota = max(share, (int64_t)min(most, kQuotaLeast));
        unit = blockIdx.x * quota;
        last = min(unit + quota, all * a.Hk);
        __syncthreads();
    } else {
        unit = blockIdx.x;                         // set of rows, then by row_tiles
        last = INT64_MAX;
    }

    while (unit < last) {
        int b, hk, set, c0, c1;
        bool complete;                             // all of its keys are taken here
        if constexpr (MODE == kQuota) {
            int lo = 0, hi = a.B;                  // the last sequence that starts at or before the unit
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (sh_start[mid] * a.Hk <= unit) lo = mid; else hi = mid;
            }
            b = __builtin_amdgcn_readfirstlane(lo);
        } else {
            b = (int)(blockIdx.x / (unsigned)(a.row_tiles * a.Hk));
        }
        const Seq sq = sequence(a, b, cu_q, kv_lens);
        const int rows = sq.n * a.G;               // (token, head of the group) pairs, token-major
        if constexpr (MODE == kQuota) {
            const Units u = units_of(a, sq, ROWS);
            const int64_t in = unit - sh_start[b] * a.Hk, per = (int64_t)u.sets * u.tiles;
            hk = __builtin_amdgcn_readfirstlane((int)(in / per));
            const int64_t rest = in - hk * per;
            set = __builtin_amdgcn_readfirstlane((int)(rest / u.tiles));
            c0 = __builtin_amdgcn_readfirstlane((int)(rest - (int64_t)set * u.tiles));
            c1 = (int)min((int64_t)u.tiles, c0 + (last - unit));
            complete = c0 == 0 && c1 == u.tiles;
            if (c0 == 0 && !complete) {
                joined = (int)((unit + u.tiles - 1) / quota) - (int)blockIdx.x + 1;
                join_start = sq.start;
                join_r0 = set * ROWS;
                join_rows = rows;
                join_hk = hk;
            }
            unit += c1 - c0;
        } else {
            const int in = (int)(blockIdx.x % (unsigned)(a.row_tiles * a.Hk));
            hk = in % a.Hk;                        // sets of one head on one XCD, where it has a multiple of 8
            // the last first: they see most keys where attention is causal (a
            // 2048-token chunk behind 6144: 457 -> 421 us)
            set = a.row_tiles - 1 - in / a.Hk + (int)(unit - blockIdx.x);
            if ((int64_t)set * ROWS >= rows) return;
            c0 = 0;
            c1 = INT32_MAX;
            complete = true;
            unit += a.row_tiles;
        }
        const int r0 = set * ROWS;
        const ScalarInts trow = (ScalarInts)(uintptr_t)(a.table + (size_t)b * a.W);
        const int p0 = sq.kv - sq.n + r0 / a.G, p1 = sq.kv - sq.n + (min(r0 + ROWS, rows) - 1) / a.G;
        const Range rg = tiles_of(a, p0, p1, sq.kv);
        c1 = complete ? rg.total : min(c1, rg.total);
        const int rw = r0 + 16 * MT * wr;          // this wave's first row

        // queries of this lane's row in each 16-row tile
        bf16x8_t qf[MT][KS];
#pragma unroll
        for (int q = 0; q < MT; ++q) {
            const int r = rw + 16 * q + m;
            const bool in = r < rows;
            const int tok = in ? r / a.G : 0, h = in ? hk * a.G + r % a.G : 0;
            const uint16_t* src = a.q + (int64_t)(sq.start + tok) * a.qs + (int64_t)h * D + g * (D / 4);
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                u32x4_t x{0, 0, 0, 0};
                if (in) x = *reinterpret_cast<const u32x4_t*>(src + 8 * s);
                qf[q][s] = __builtin_bit_cast(bf16x8_t, x);
            }
        }
        // what they see; found anew for each tile that needs it, since kept it
        // would cost the common tiles registers
        const int tok0 = rw / a.G, in0 = rw % a.G;
        const float per_token = 1.0f / (float)a.G;
        auto views = [&](View (&vw)[MT]) {
            int first = m;
            asm volatile("" : "+v"(first));
#pragma unroll
            for (int q = 0; q < MT; ++q) {
                // (x + 1/2) / G is at least 1 / 2G from a whole number, and x below 2^15
                const int x = first + 16 * q, t = (int)(((float)(in0 + x) + 0.5f) * per_token), p = sq.kv - sq.n + tok0 + t;
                vw[q].up = rw + x >= rows || p < 0 ? 0 : a.causal ? min(p + 1, sq.kv) : sq.kv;
                vw[q].lo = a.window > 0 ? (int)max((int64_t)p - a.window + 1, (int64_t)0) : 0;
            }
        };
        // keys that every row of this wave sees, [all_lo, all_up) and below
        // sinks, and that any of them does (a wave without rows: none)
        const int pw0 = sq.kv - sq.n + min(rw, rows - 1) / a.G;
        const int pw1 = sq.kv - sq.n + (min(rw + 16 * MT, rows) - 1) / a.G;
        const int all_up = pw0 < 0 ? 0 : a.causal ? min(pw0 + 1, sq.kv) : sq.kv;
        const int all_lo = a.window > 0 ? (int)max((int64_t)pw1 - a.window + 1, (int64_t)0) : 0;
        const int last_page = (sq.kv - 1) >> a.shift;

        Sums<D, MT> sums;
#pragma unroll
        for (int q = 0; q < MT; ++q) {
            // a lane without a row (queries of 0, scores of 0) never moves
            sums.m[q] = rw + 16 * q + m < rows ? -INFINITY : 0.f;
            sums.l[q] = 0.f;
#pragma unroll
            for (int n = 0; n < NT; ++n) sums.o[q][n] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        }

        // tiles c0 + wk, c0 + wk + WK, ...
        auto tile_at = [&](int x) { return x < rg.head ? x : rg.lo + x - rg.head; };
        auto pages_for = [&](int x) { return pages_of(a, trow, tile_at(min(x, c1 - 1)), last_page); };
        // A tile that every row sees whole needs no mask.  Else keys in no page
        // or behind the last are dead (their values count as 0) and the others
        // are masked row by row.
        const int whole_up = all_up / kTile, whole_lo = all_lo / kTile + (all_lo % kTile != 0), whole_sinks = a.sinks / kTile;
        auto whole = [&](const Pages& p) {
            return in_cache(a, p.a) && in_cache(a, p.b) && p.tile < whole_up && (p.tile >= whole_lo || p.tile < whole_sinks);
        };
        auto live_in = [&](const Pages& p) {
            const bool ok0 = in_cache(a, p.a), ok1 = in_cache(a, p.b);
            return (g < 2 ? ok0 : ok1) ? low_bits(sq.kv - p.tile * kTile - 8 * g) : 0u;
        };
        if constexpr (SHARED) {
            // The waves along the rows share every tile.  Between two barriers
            // they start the loads of the tile after the next and read this one;
            // MXFP4: and turn the next one, which has arrived, into operands.
            const int any_up = rw >= rows || pw1 < 0 ? 0 : a.causal ? min(pw1 + 1, sq.kv) : sq.kv;
            const int any_lo = a.window > 0 ? (int)max((int64_t)pw0 - a.window + 1, (int64_t)0) : 0;
            constexpr int kRaws = DIRECT ? 0 : 2 * SharedTile<D>::kBytes;
            uint8_t* const raws = lds + kRaws;
            const uint32_t raw_at = lds_at + kRaws;
            auto turn = [&](int slot, const Pages& p) {
                const bool all = in_cache(a, p.a) && in_cache(a, p.b) && p.tile < sq.kv / kTile;
                share_out<FMT, D>(raws + slot * T::kBytes, lds + slot * SharedTile<D>::kBytes, all ? 0u : live_in(p), all, wave, lane);
            };
            const PartOf from(a, wave);
            int c = c0, buf = 0;                   // tile and its slot
            Pages pg0{}, pg1{}, pg2{};             // of tiles c, c + 1, c + 2
            auto begin = [&] {
                c = c0;
                buf = 0;
                if (c >= c1) return;
                pg0 = pages_for(c);
                pg1 = pages_for(c + 1);
                pg2 = pages_for(c + 2);
                fetch_part<FMT, D>(raw_at, a, from, pg0, hk, lane, wave);
                fetch_part<FMT, D>(raw_at + T::kBytes, a, from, pg1, hk, lane, wave);
                if constexpr (!DIRECT) {
                    wait_loads<0>();
                    lds_barrier();
                    turn(0, pg0);
                }
            };
            auto share = [&] {
                if constexpr (DIRECT) {
                    wait_loads<T::kFetches / kWaves>();        // tile c has arrived, this wave's part of it
                    lds_barrier();                 // and the others'; tile c - 1 is read
                    fetch_part<FMT, D>(raw_at + (buf == 0 ? 2 : buf - 1) * T::kBytes, a, from, pg2, hk, lane, wave);
                } else {
                    wait_loads<0>();               // tile c + 1 has arrived, this wave's part of it
                    lds_barrier();                 // and the others'; tile c is operands, c - 1 read
                    fetch_part<FMT, D>(raw_at + buf * T::kBytes, a, from, pg2, hk, lane, wave);
                    turn(buf ^ 1, pg1);
                }
            };
            auto next = [&] {
                ++c;
                if constexpr (DIRECT) buf = buf == 2 ? 0 : buf + 1;
                else buf ^= 1;
                pg0 = pg1;
                pg1 = pg2;
                pg2 = pages_for(c + 2);
            };
            auto tile_here = [&] {
                if constexpr (DIRECT) return DirectTile<D>((LdsBytes)(lds_void*)lds + buf * T::kBytes, lane);
                else return SharedTile<D>{lds + buf * SharedTile<D>::kBytes + lane * 16};
            };
            typedef Masked<D, decltype(tile_here())> Any;
            auto seen_here = [&] {                 // by any row of this wave
                const int key0 = pg0.tile * kTile;
                return key0 < any_up && (key0 + kTile > any_lo || key0 < a.sinks);
            };
            int wild = 0;
            begin();
            while (c < c1) {
                int shared = 0;
                while (__builtin_expect(c < c1 && whole(pg0), 1)) {
                    share();
                    if (__builtin_expect(!attend_shared<D, MT>(sums, tile_here(), qf, a.c), 0)) {
                        shared = 1;
                        break;
                    }
                    next();
                }
                one_exit(c, shared);
                if (c >= c1) break;
                if (!shared) share();
                if (seen_here()) {
                    const Any tile(tile_here());
                    const uint32_t live = live_in(pg0);
                    if (!whole(pg0) && __any(tile.wild(live))) {
                        wild = 1;
                    } else {
                        View vw[MT];
                        views(vw);
                        attend_part<D, MT, false>(sums, tile, qf, vw, pg0.tile * kTile + 8 * g, live, a.sinks, a.c);
                    }
                }
                next();
            }
            wait_loads<0>();
            // tiles put off, as below; the waves go through them together
            if (__syncthreads_or(wild)) {
                begin();
                while (c < c1) {
                    share();
                    if (!whole(pg0) && seen_here()) {
                        const Any tile(tile_here());
                        const uint32_t live = live_in(pg0);
                        View vw[MT];
                        views(vw);
                        if (__any(tile.wild(live)))
                            attend_part<D, MT, true>(sums, tile, qf, vw, pg0.tile * kTile + 8 * g, live, a.sinks, a.c);
                    }
                    next();
                }
                wait_loads<0>();
                __syncthreads();
            }
        } else {
            // Two tiles per wave in LDS, one on its way while the other is read (a
            // third did not help).  The loop over common tiles (every row sees every key, no
            // reference moves) has no other branch in it, so that the sums stay in
            // their registers; anything else leaves it before the sums are touched.
            // Loads past the end ask for the last tile again, so that the number
            // under way is always the same.
            bool wild = false;
            int c = c0 + wk;
            uint32_t at = 0;                       // tile c's slot
            Pages pg0{}, pg1{}, pg2{};             // of tiles c, c + WK, c + 2 WK
            if (c < c1) {
                pg0 = pages_for(c);
                pg1 = pages_for(c + WK);
                pg2 = pages_for(c + 2 * WK);
                fetch<FMT, D, ONCE>(mine, a, pg0, hk, lane);
                fetch<FMT, D, ONCE>(mine + T::kBytes, a, pg1, hk, lane);
            }
            // the queries are used here, so that the wait for them is not left to
            // the loops below, where it would be for the tiles' loads too
#pragma unroll
            for (int q = 0; q < MT; ++q)
#pragma unroll
                for (int s = 0; s < KS; ++s) {
                    u32x4_t x = __builtin_bit_cast(u32x4_t, qf[q][s]);
                    asm volatile("" : "+v"(x));
                    qf[q][s] = __builtin_bit_cast(bf16x8_t, x);
                }
            // tile c is done with: its slot takes the next but one
            auto advance = [&] {
                fetch<FMT, D, ONCE>(mine + at, a, pg2, hk, lane);
                c += WK;
                at ^= T::kBytes;
                pg0 = pg1;
                pg1 = pg2;
                pg2 = pages_for(c + 2 * WK);
            };
            constexpr int kUnder = T::kFetches;
            while (c < c1) {
                while (c < c1 && whole(pg0)) {
                    wait_loads<kUnder>();
                    if (!attend_whole<D, MT>(sums, RawTile<FMT, D>(base + at, lane), qf, a.c)) break;
                    advance();
                }
                int same = 0;
                one_exit(c, same);
                if (c >= c1) break;
                // any tile
                wait_loads<kUnder>();
                const RawTile<FMT, D> r(base + at, lane);
                const uint32_t live = live_in(pg0);
                if (!whole(pg0) && __any(r.wild(live))) {
                    wild = true;
                } else {
                    View vw[MT];
                    views(vw);
                    attend_part<D, MT, false>(sums, r, qf, vw, pg0.tile * kTile + 8 * g, live, a.sinks, a.c);
                }
                advance();
            }
            // tiles put off: those that rows see in part and that hold an infinite
            // or NaN value.  Rare, and kept out of the loop above so that it costs
            // that loop no registers.
            if (wild) {
                for (c = c0 + wk; c < c1; c += WK) {
                    const Pages pc = pages_for(c);
                    if (whole(pc)) continue;
                    wait_loads<0>();
                    fetch<FMT, D, ONCE>(mine, a, pc, hk, lane);
                    wait_loads<0>();
                    const RawTile<FMT, D> r(base, lane);
                    const uint32_t live = live_in(pc);
                    View vw[MT];
                    views(vw);
                    if (__any(r.wild(live)))
                        attend_part<D, MT, true>(sums, r, qf, vw, pc.tile * kTile + 8 * g, live, a.sinks, a.c);
                }
            }
            wait_loads<0>();                       // the ring's memory is used again below
        }

        // join the waves along the keys, 16 rows of each row wave at a time
#pragma unroll
        for (int q = 0; q < MT; ++q) {
            if (WK > 1 || q == 0) __syncthreads();
            else asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            if (g == 0) {
                sh_m[wave][m] = sums.m[q];
                sh_l[wave][m] = sums.l[q];
            }
            float* row = sh_o[wave][m];
            if constexpr (DIRECT) {
#pragma unroll
                for (int n = 0; n < NT; ++n) *reinterpret_cast<f32x4_t*>(row + 16 * n + 4 * g) = sums.o[q][n];
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int n = 0; n < NT; n += 4)
                        *reinterpret_cast<f32x4_t*>(row + (4 * g + i) * NT + n) =
                            f32x4_t{sums.o[q][n][i], sums.o[q][n + 1][i], sums.o[q][n + 2][i], sums.o[q][n + 3][i]};
            }
            if constexpr (WK > 1) __syncthreads();
            else asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");    // a wave reads what it wrote
            const int wj = tid / TPR / 16, rr = tid / TPR % 16, d0 = tid % TPR * E;
            const int r = r0 + 16 * MT * wj + 16 * q + rr;
            if (r < rows) {
                float top = sh_m[wj][rr];
#pragma unroll
                for (int w = 1; w < WK; ++w) top = fmaxf(top, sh_m[wj + w * WR][rr]);
                const float ref = top == -INFINITY ? 0.f : top;
                float acc[E], lt = 0.f;
#pragma unroll
                for (int n = 0; n < E; ++n) acc[n] = 0.f;
#pragma unroll
                for (int w = 0; w < WK; ++w) {
                    const float f = __builtin_amdgcn_exp2f(sh_m[wj + w * WR][rr] - ref);
                    const float* part = sh_o[wj + w * WR][rr] + d0;
                    lt += f * sh_l[wj + w * WR][rr];
#pragma unroll
                    for (int n = 0; n < E; ++n) acc[n] += f * part[n];
                }
                const int t = sq.start + r / a.G, h = hk * a.G + r % a.G;
                if (complete) {
                    const float inv = lt == 0.f ? 0.f : 1.f / lt;
                    uint32_t* dst = reinterpret_cast<uint32_t*>(a.out + (int64_t)t * a.os + (int64_t)h * D + d0);
                    if constexpr (E == 4) {
                        *reinterpret_cast<uint2*>(dst) =
                            make_uint2(pack_bf16(acc[0] * inv, acc[1] * inv), pack_bf16(acc[2] * inv, acc[3] * inv));
                    } else {
#pragma unroll
                        for (int n = 0; n < E; n += 8)
                            *reinterpret_cast<u32x4_t*>(dst + n / 2) =
                                u32x4_t{pack_bf16(acc[n] * inv, acc[n + 1] * inv), pack_bf16(acc[n + 2] * inv, acc[n + 3] * inv),
                                        pack_bf16(acc[n + 4] * inv, acc[n + 5] * inv),
                                        pack_bf16(acc[n + 6] * inv, acc[n + 7] * inv)};
                    }
                } else {
                    // a piece that begins inside its units is the workgroup's
                    // first, one that begins with them and ends early its last
                    const int64_t at = ((int64_t)blockIdx.x * 2 + (c0 == 0)) * ROWS + (r - r0);
#pragma unroll
                    for (int n = 0; n < E; n += 4)
                        *reinterpret_cast<f32x4_t*>(a.part + at * D + d0 + n) =
                            f32x4_t{acc[n], acc[n + 1], acc[n + 2], acc[n + 3]};
                    if (d0 == 0) *reinterpret_cast<float2*>(a.stat + at * 2) = make_float2(top, lt);
                }
            }
        }
        __syncthreads();                           // the next rows' tiles come where the join was read
    }
    if (MODE == kQuota && tid == 0) {
        int32_t* j = a.joins + (int64_t)blockIdx.x * kJoinInts;
        j[0] = joined;
        j[1] = join_start;
        j[2] = join_r0;
        j[3] = join_rows;
        j[4] = join_hk;
    }
}

// Rows whose units several workgroups shared: out = sum 2^(m_s - m) O_s / sum
// 2^(m_s - m) l_s over the pieces in order.  They begin as the last piece of
// workgroup w and go on as the first of each that follows, so blockIdx.y = w
// finds them in one record; blockIdx.x takes 4 `each` of its rows, a wave one
// after the other.  This way round, a long sequence's rows are spread over the
// XCDs: begun every 64th workgroup, they would else all be read by one.
template <int D>
__global__ __launch_bounds__(kThreads) void k_attn_join(AttnArgs a, int per, int each) {
    const int w = blockIdx.y, lane = threadIdx.x % kWave;
    const int32_t* j = a.joins + (int64_t)w * kJoinInts;
    const int used = j[0];
    if (used == 0) return;
    const int start = j[1], r0 = j[2], rows = j[3], hk = j[4];
    const int first = (blockIdx.x * kWaves + threadIdx.x / kWave) * each;
    for (int in = first; in < min(first + each, per); ++in) {
        const int r = r0 + in;
        if (r >= rows) return;
        auto at = [&](int s) { return ((int64_t)(w + s) * 2 + (s == 0)) * per + in; };
        float top = -INFINITY;
        for (int s = lane; s < used; s += kWave) top = fmaxf(top, a.stat[at(s) * 2]);
#pragma unroll
        for (int off = kWave / 2; off >= 1; off >>= 1) top = fmaxf(top, __shfl_xor(top, off));
        const float ref = top == -INFINITY ? 0.f : top;
        // D/4 lanes take 4 elements each of a piece, the wave 256/D pieces at a
        // time and 4 or 8 such rounds under way (16 take registers that cost
        // the short joins more than the long ones gain)
        constexpr int L = D / 4, P = kWave / L;
        const int sub = lane / L, d0 = lane % L * 4;
        f32x4_t acc{0.f, 0.f, 0.f, 0.f};
        float l = 0.f;
        auto add = [&](auto N, int s0) {
            f32x4_t x[N];
            float2 ml[N];
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int s = min(s0 + i * P + sub, used - 1);
                ml[i] = *reinterpret_cast<const float2*>(a.stat + at(s) * 2);
                x[i] = *reinterpret_cast<const f32x4_t*>(a.part + at(s) * D + d0);
            }
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float f = s0 + i * P + sub < used ? __builtin_amdgcn_exp2f(ml[i].x - ref) : 0.f;
                l += f * ml[i].y;
                acc += f * x[i];
            }
        };
        if (used <= 4 * P) add(std::integral_constant<int, 4>{}, 0);
        else for (int s0 = 0; s0 < used; s0 += 8 * P) add(std::integral_constant<int, 8>{}, s0);
#pragma unroll
        for (int off = L; off < kWave; off <<= 1) {
            l += __shfl_xor(l, off);
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[e] += __shfl_xor(acc[e], off);
        }
        if (sub != 0) continue;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        *reinterpret_cast<uint2*>(a.out + (int64_t)(start + r / a.G) * a.os + (int64_t)(hk * a.G + r % a.G) * D + d0) =
            make_uint2(pack_bf16(acc[0] * inv, acc[1] * inv), pack_bf16(acc[2] * inv, acc[3] * inv));
    }
}

// Launch shape: a function of the sizes alone, so that the workspace's size
// and the launch agree.
// 16-row tiles of a wave where four waves along the rows share each tile of
// keys: what 256 registers hold.  Two, with three workgroups a CU: 443 against
// 424 us (MXFP4 chunk) and 228 against 201 us (bf16 windowed prompts).
constexpr int shared_mt(int D) { return D == 128 ? 3 : 4; }
struct Shape {
    int mode, mt, wr, row_tiles, grid;
};
Shape shape_of(const moe_mxfp4_attn_args& p, const moe_mxfp4_kv_cache& c) {
    Shape s{};
    const bool fp4 = c.format == MOE_KV_MXFP4, wide = !fp4 && c.head_dim == 128;
    const int64_t G = p.heads / c.kv_heads;
    const int64_t mq = p.max_q < p.num_tokens ? p.max_q : p.num_tokens;
    const int64_t rows = mq * G;
    if (rows <= 64) {
        // waves along the keys: 16 rows a wave, or 32; above that two waves
        // along the rows, or four (bf16 rows of 128: 16 a wave always)
        s.mt = rows <= 16 || wide ? 1 : 2;
        s.wr = rows <= 16 * s.mt ? 1 : 2;
    } else {
        s.mt = shared_mt(c.head_dim);
        s.wr = kWaves;
    }
    const int64_t per = 16 * s.mt * s.wr;
    int64_t tiles = (rows + per - 1) / per;
    int64_t keys = p.max_kv;
    if (p.window > 0) {
        const int64_t w = (int64_t)p.window + per / G + 1 + p.sinks + 2 * kTile;
        if (w < keys) keys = w;
    }
    const int64_t pairs = (int64_t)p.batch * c.kv_heads;
    // Quotas where sequences are long enough to be divided and too few sets of
    // rows to fill the GPU, of which ragged ones would leave it early (a
    // 2048-token chunk, 512 sets: 446 us without, 474 + 32 for the join with
    // quotas); not where a window makes them all alike and there are enough of
    // them (64 sequences x 8 heads of a window of 1000: 30 us, 38 + 18 with).
    const int64_t held = 256 * (wide && s.wr < kWaves ? 1 : s.mt == 1 && fp4 ? 3 : 2);   // workgroups the GPU holds at once
    const bool alike = p.window > 0 && keys < p.max_kv && pairs * tiles >= held;
    if (p.batch <= kQuotaBatch && pairs * tiles < held && (keys + kTile - 1) / kTile > kQuotaLeast && !alike) {
        s.mode = kQuota;
        s.grid = (int)held;
        return s;
    }
    s.mode = kEven;
    // the grid stays below 2^22 workgroups: more sets of rows than fit are walked by a loop
    const int64_t most = (1 << 22) / pairs > 0 ? (1 << 22) / pairs : 1;
    s.row_tiles = (int)(tiles < most ? tiles : most);
    s.grid = (int)(pairs * s.row_tiles);
    return s;
}

template <int FMT, int D, int MODE>
void launch_mode(const AttnArgs& a, const Shape& sh, hipStream_t s) {
    // waves per SIMD: what the registers of MT tiles leave
    constexpr bool fp4 = FMT == MOE_KV_MXFP4;
    constexpr bool wide = !fp4 && D == 128;       // whose tiles fill the LDS with one workgroup
    constexpr int MT = wide ? 1 : 2, W1 = wide ? 1 : !fp4 ? 2 : D == 128 ? 3 : 4, W2 = wide ? 1 : !fp4 || D == 128 ? 2 : 3;
    const dim3 grid(sh.grid), block(kThreads);
    if (sh.mt == 1 && sh.wr == 1) hipLaunchKernelGGL((k_attn<FMT, D, 1, 1, W1, MODE>), grid, block, 0, s, a);
    else if (sh.wr == 1) hipLaunchKernelGGL((k_attn<FMT, D, MT, 1, W2, MODE>), grid, block, 0, s, a);
    else if (sh.wr == 2) hipLaunchKernelGGL((k_attn<FMT, D, MT, 2, W2, MODE>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((k_attn<FMT, D, shared_mt(D), kWaves, 2, MODE>), grid, block, 0, s, a);
}

template <int FMT, int D>
hipError_t launch_fmt(const AttnArgs& a, const Shape& sh, hipStream_t s) {
    if (sh.mode == kEven) {
        launch_mode<FMT, D, kEven>(a, sh, s);
        return hipGetLastError();
    }
    launch_mode<FMT, D, kQuota>(a, sh, s);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int per = 16 * sh.mt * sh.wr, each = per > 64 ? 4 : 1;        // many rows have few pieces
    hipLaunchKernelGGL((k_attn_join<D>), dim3((per + kWaves * each - 1) / (kWaves * each), sh.grid), dim3(kThreads), 0, s, a,
                       per, each);
    return hipGetLastError();
}

// Pieces of a quota launch: rows of sums, two pieces a workgroup.
int64_t piece_rows(const Shape& s) { return (int64_t)s.grid * 2 * 16 * s.mt * s.wr; }

}  // namespace

size_t attention_workspace_bytes(const moe_mxfp4_attn_args& p, const moe_mxfp4_kv_cache& c) {
    const Shape s = shape_of(p, c);
    if (s.mode == kEven) return 0;
    return piece_rows(s) * (c.head_dim + 2) * sizeof(float) + (size_t)s.grid * kJoinInts * sizeof(int32_t);
}

hipError_t launch_attention(const moe_mxfp4_attn_args& p, const moe_mxfp4_kv_cache& c, void* workspace,
                            hipStream_t s) {
    const Shape sh = shape_of(p, c);
    AttnArgs a{};
    a.q = static_cast<const uint16_t*>(p.q); a.out = static_cast<uint16_t*>(p.out);
    a.table = p.block_table; a.cu_q = p.cu_q; a.kv_lens = p.kv_lens;
    a.k = static_cast<const uint8_t*>(c.k); a.v = static_cast<const uint8_t*>(c.v);
    a.ks = c.k_scale; a.vs = c.v_scale;
    if (sh.mode == kQuota) {
        a.part = static_cast<float*>(workspace);
        a.stat = a.part + piece_rows(sh) * c.head_dim;
        a.joins = reinterpret_cast<int32_t*>(a.stat + piece_rows(sh) * 2);
    }
    a.qs = p.q_stride; a.os = p.out_stride;
    a.B = p.batch; a.T = p.num_tokens; a.H = p.heads; a.Hk = c.kv_heads; a.G = p.heads / c.kv_heads;
    a.W = p.max_blocks; a.shift = log2_of(c.page_size); a.num_pages = c.num_pages;
    a.causal = p.causal != 0; a.window = p.window; a.sinks = p.sinks;
    a.row_tiles = sh.row_tiles;
    a.c = p.scale * 1.4426950408889634f;
    if (c.format == MOE_KV_MXFP4)
        return c.head_dim == 128 ? launch_fmt<MOE_KV_MXFP4, 128>(a, sh, s) : launch_fmt<MOE_KV_MXFP4, 64>(a, sh, s);
    return c.head_dim == 128 ? launch_fmt<MOE_KV_BF16, 128>(a, sh, s) : launch_fmt<MOE_KV_BF16, 64>(a, sh, s);
}

}  // namespace moe
