// Norms of queries and keys for each head, the position rotation and the
// cache write in one pass over the projection's output; and the read-back of
// cached rows.
//
// y = x * rsqrt(mean(x^2) + eps) * w per head, then the first R elements in
// pairs (a, b) -> (a cos - b sin, b cos + a sin), all in float32 and rounded
// once, to bf16 or to the cache's format.  A head is D/8 lanes of 8 elements
// (one 16-byte load each), so a wave holds 4 heads of 128 or 8 of 64; the sum
// of squares takes log2(D/8) lane exchanges, the partner of the half-split
// pairing sits R/16 lanes away, and an MX block of 32 is 4 lanes.  The angle
// pos * freq is formed in turns in 64 bits, where a position of a million
// still leaves 2^-33 of a turn, and only its fraction goes to float32; the
// R/2 angles of a token are computed once per workgroup, one a thread, into
// LDS.
//
// Bound by bytes (2 (2 Hq + 2 Hkv) D a token and the cache row): 5570
// tokens of 48 + 8 + 8 heads of 128, 165 MB, 40 us, 4.1 TB/s.  Few tokens: bound by the launch and one chain of
// loads (8 tokens 4.2 us, 512 tokens 6.8 us); a token's heads are split over
// up to four workgroups, so that every wave has one load round instead of four
// in sequence.
#include "kv_cache.hpp"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;

struct RopeArgs {
    const uint16_t *q, *k, *v, *wq, *wk;
    const double* freq;
    const int32_t *pos, *slots;
    uint16_t *q_out, *k_out;
    uint8_t *ck, *cv, *cks, *cvs;                  // the cache, ck null without one
    int64_t qs, ks, vs;
    int32_t Hq, Hk, HT, rot, nslots, shift, iters;
    float eps;
};

__device__ __forceinline__ void unpack8(const u32x4_t& raw, float f[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(raw[i] << 16);
        f[2 * i + 1] = __uint_as_float(raw[i] & 0xFFFF0000u);
    }
}

// Two floats -> two bf16, nearest even; NaN stays NaN.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    bf16x2_t r;
    r[0] = (__bf16)a;
    r[1] = (__bf16)b;
    return __builtin_bit_cast(uint32_t, r);
}

__device__ __forceinline__ u32x4_t pack8(const float f[8]) {
    u32x4_t r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = pack_bf16(f[2 * i], f[2 * i + 1]);
    return r;
}

// E2M1 code of |x| <= anything finite, already divided by its scale: the
// number of rounding borders passed.  A border belongs to the even of its two
// codes (ties to even), so it is passed by > below an even code's border and
// by >= below an odd one's.
__device__ __forceinline__ uint32_t e2m1(float x) {
    const float a = fabsf(x);
    const uint32_t c = (uint32_t)(a > 0.25f) + (a >= 0.75f) + (a > 1.25f) + (a >= 1.75f) + (a > 2.5f) + (a >= 3.5f) +
                       (a > 5.0f);
    return c | (__float_as_uint(x) >> 31 << 3);
}

// The 8 elements of this lane quantised within their block of 32 (4 lanes):
// codes (one dword) and the block's scale byte.
__device__ __forceinline__ uint32_t quant8(const float f[8], uint32_t& scale) {
    float amax = 0.f;
    bool wild = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        amax = fmaxf(amax, fabsf(f[i]));
        wild |= (__float_as_uint(f[i]) & 0x7F800000u) == 0x7F800000u;
    }
    if (wild) amax = INFINITY;                     // fmaxf would drop a NaN
    amax = fmaxf(amax, __shfl_xor(amax, 1));
    amax = fmaxf(amax, __shfl_xor(amax, 2));
    if (amax == INFINITY) {
        scale = 0xFF;
        return 0;
    }
    const int se = mx_scale_exp(amax, 2);
    scale = (uint32_t)(se + 127);
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) w |= e2m1(ldexpf(f[i], -se)) << (4 * i);
    return w;
}

// One head of a token into the cache: this lane's 8 elements, at 8 sub.
template <int D>
__device__ __forceinline__ void cache_store(const RopeArgs& a, bool value, int head, int slot, int sub,
                                            const float f[8]) {
    const int page = slot >> a.shift, row = slot & ((1 << a.shift) - 1);
    const int64_t base = ((int64_t)page * a.Hk + head) << a.shift;     // first row of the page's head
    uint8_t* dst = value ? a.cv : a.ck;
    uint8_t* dsc = value ? a.cvs : a.cks;
    if (!dsc) {
        *reinterpret_cast<u32x4_t*>(dst + ((base + row) * D + sub * 8) * 2) = pack8(f);
        return;
    }
    uint32_t scale;
    const uint32_t w = quant8(f, scale);
    if (!value) {
        *reinterpret_cast<uint32_t*>(dst + (base + row) * (D / 2) + sub * 4) = w;
        if ((sub & 3) == 0) dsc[(base + row) * (D / 32) + sub / 4] = (uint8_t)scale;
        return;
    }
    constexpr int KG = v_keys_per_piece(D), C = D / 32;                // a row's bytes in a piece
    uint8_t* piece = dst + base * (D / 2) + (row / KG) * (KG * D / 2) + (row % KG) * C;
    if constexpr (C == 4) {
        *reinterpret_cast<uint32_t*>(piece + sub * 16) = w;
    } else {
        *reinterpret_cast<uint16_t*>(piece + (2 * sub) * 16) = (uint16_t)w;
        *reinterpret_cast<uint16_t*>(piece + (2 * sub + 1) * 16) = (uint16_t)(w >> 16);
    }
    if ((sub & 3) == 0) dsc[base * (D / 32) + (row / 8) * (8 * (D / 32)) + (sub / 4) * 8 + row % 8] = (uint8_t)scale;
}

template <int D, bool INTER>
__global__ __launch_bounds__(kThreads) void k_rope(RopeArgs a) {
    constexpr int L = D / 8;                       // lanes per head
    constexpr int HPW = kWave / L;                 // heads per wave and round
    __shared__ float2 turn[D / 2];
    const int t = blockIdx.x, tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
    const int pos = a.pos[t];
    if (pos < 0) return;
    const int sub = lane % L;
    const int half = a.rot / 2;
    const int h0 = (blockIdx.y * kWaves + wave) * a.iters * HPW + lane / L;
    if (tid < half) {
        const double rev = (double)pos * a.freq[tid] * 0.15915494309189533577;   // turns
        float s, c;
        sincospif(2.0f * (float)(rev - rint(rev)), &s, &c);
        turn[tid] = make_float2(c, s);
    }
    const int slot = a.ck ? a.slots[t] : -1;
    __syncthreads();
    // cos and sin of this lane's 8 elements: half-split, element 8 sub + e is
    // of pair (8 sub + e) mod half; interleaved, of pair 4 sub + e / 2
    const bool rotates = sub * 8 < a.rot;
    float cs[8], sn[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int i = INTER ? sub * 4 + e / 2 : sub * 8 + e - (sub * 8 >= half ? half : 0);
        const float2 w = rotates ? turn[i] : make_float2(1.f, 0.f);
        cs[e] = w.x;
        sn[e] = w.y;
    }
    const bool low = sub * 8 < half;               // half-split: this lane holds a's, else b's
    const int partner = rotates ? lane + (low ? half / 8 : -(half / 8)) : lane;
    for (int it = 0; it < a.iters; ++it) {
        const int h = h0 + it * HPW;
        const bool isq = h < a.Hq, isk = !isq && h < a.Hq + a.Hk, in = h < a.HT;
        const uint16_t* src = isq ? a.q + t * a.qs + (int64_t)h * D
                            : isk ? a.k + t * a.ks + (int64_t)(h - a.Hq) * D
                                  : a.v + t * a.vs + (int64_t)(h - a.Hq - a.Hk) * D;
        u32x4_t raw{0, 0, 0, 0};
        if (in) raw = *reinterpret_cast<const u32x4_t*>(src + sub * 8);
        float f[8];
        unpack8(raw, f);
        const uint16_t* w = isq ? a.wq : isk ? a.wk : nullptr;
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(f[e], f[e], ss);
#pragma unroll
        for (int off = 1; off < L; off <<= 1) ss += __shfl_xor(ss, off);
        if (w) {
            const float inv = 1.0f / sqrtf(ss * (1.0f / D) + a.eps);
            float g[8];
            unpack8(*reinterpret_cast<const u32x4_t*>(w + sub * 8), g);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = f[e] * inv * g[e];
        }
        if (isq || isk) {
            if constexpr (INTER) {
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    const float x = f[e], y = f[e + 1];
                    if (rotates) {
                        f[e] = x * cs[e] - y * sn[e];
                        f[e + 1] = y * cs[e] + x * sn[e];
                    }
                }
            }
        }
        if constexpr (!INTER) {
            float o[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = __shfl(f[e], partner);      // every lane takes part
            if ((isq || isk) && rotates) {
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] = low ? f[e] * cs[e] - o[e] * sn[e] : f[e] * cs[e] + o[e] * sn[e];
            }
        }
        if (isq) {
            *reinterpret_cast<u32x4_t*>(a.q_out + ((int64_t)t * a.Hq + h) * D + sub * 8) = pack8(f);
        } else if (in) {
            const int hk = isk ? h - a.Hq : h - a.Hq - a.Hk;
            if (isk && a.k_out)
                *reinterpret_cast<u32x4_t*>(a.k_out + ((int64_t)t * a.Hk + hk) * D + sub * 8) = pack8(f);
            // the head's lanes go together: all of a block's lanes are here or none
            if (slot >= 0 && slot < a.nslots) cache_store<D>(a, !isk, hk, slot, sub, f);
        }
    }
}

struct ReadArgs {
    const uint8_t *k, *v, *ks, *vs;
    const int32_t* slots;
    uint16_t *ko, *vo;
    int32_t Hk, nslots, shift, first;              // first: 0 keys (then values), 1 values only
    int64_t rows;                                  // slots x heads
};

// A head row per L lanes: 8 elements a lane.
template <int D>
__global__ __launch_bounds__(kThreads) void k_kv_read(ReadArgs a) {
    constexpr int L = D / 8;
    const int64_t gid = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int64_t r = gid / L;
    const int sub = (int)(gid % L);
    if (r >= a.rows) return;
    const bool value = blockIdx.y + a.first != 0;
    const int64_t i = r / a.Hk;
    const int head = (int)(r % a.Hk), slot = a.slots[i];
    uint16_t* out = (value ? a.vo : a.ko) + r * D + sub * 8;
    u32x4_t w{0, 0, 0, 0};
    if (slot >= 0 && slot < a.nslots) {
        const int64_t base = ((int64_t)(slot >> a.shift) * a.Hk + head) << a.shift;
        const int row = slot & ((1 << a.shift) - 1);
        const uint8_t* src = value ? a.v : a.k;
        const uint8_t* sc = value ? a.vs : a.ks;
        if (!sc) {
            w = *reinterpret_cast<const u32x4_t*>(src + ((base + row) * D + sub * 8) * 2);
        } else {
            uint32_t codes, byte;
            if (!value) {
                codes = *reinterpret_cast<const uint32_t*>(src + (base + row) * (D / 2) + sub * 4);
                byte = sc[(base + row) * (D / 32) + sub / 4];
            } else {
                constexpr int KG = v_keys_per_piece(D), C = D / 32;
                const uint8_t* piece = src + base * (D / 2) + (row / KG) * (KG * D / 2) + (row % KG) * C;
                if constexpr (C == 4) {
                    codes = *reinterpret_cast<const uint32_t*>(piece + sub * 16);
                } else {
                    codes = *reinterpret_cast<const uint16_t*>(piece + (2 * sub) * 16) |
                            ((uint32_t)*reinterpret_cast<const uint16_t*>(piece + (2 * sub + 1) * 16) << 16);
                }
                byte = sc[base * (D / 32) + (row / 8) * (8 * (D / 32)) + (sub / 4) * 8 + row % 8];
            }
            if (byte == 0xFF) {
                w = u32x4_t{0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u};
            } else {
                w = __builtin_bit_cast(u32x4_t, decode8_bf16(codes, e8m0_as_scale(byte)));
            }
        }
    }
    *reinterpret_cast<u32x4_t*>(out) = w;
}

}  // namespace

hipError_t launch_qk_norm_rope(const moe_mxfp4_rope_args& p, const moe_mxfp4_kv_cache* c, hipStream_t s) {
    RopeArgs a{};
    a.q = static_cast<const uint16_t*>(p.q); a.k = static_cast<const uint16_t*>(p.k);
    a.v = static_cast<const uint16_t*>(p.v);
    a.wq = static_cast<const uint16_t*>(p.q_weight); a.wk = static_cast<const uint16_t*>(p.k_weight);
    a.freq = p.inv_freq; a.pos = p.positions; a.slots = p.slots;
    a.q_out = static_cast<uint16_t*>(p.q_out); a.k_out = static_cast<uint16_t*>(p.k_out);
    a.qs = p.q_stride; a.ks = p.k_stride; a.vs = p.v_stride;
    a.Hq = p.heads; a.Hk = p.kv_heads; a.HT = p.heads + p.kv_heads * (c ? 2 : 1);
    a.rot = p.rot_dim; a.eps = p.eps;
    if (c) {
        a.ck = static_cast<uint8_t*>(c->k); a.cv = static_cast<uint8_t*>(c->v);
        a.cks = c->format == MOE_KV_MXFP4 ? c->k_scale : nullptr;
        a.cvs = c->format == MOE_KV_MXFP4 ? c->v_scale : nullptr;
        a.nslots = c->num_pages * c->page_size;
        a.shift = log2_of(c->page_size);
    }
    const int per = kWaves * (kWave / (p.head_dim / 8));               // heads of a workgroup's round
    const int rounds = (a.HT + per - 1) / per;
    // up to 256 workgroups of few tokens; with more tokens than that the
    // chip is full and a token's rounds share one table of angles
    int parts = 256 / (p.num_tokens < 256 ? p.num_tokens : 256);
    parts = parts > rounds ? rounds : parts;
    a.iters = (rounds + parts - 1) / parts;
    parts = (rounds + a.iters - 1) / a.iters;
    const dim3 grid(p.num_tokens, parts), block(kThreads);
    if (p.head_dim == 128) {
        if (p.interleaved) hipLaunchKernelGGL((k_rope<128, true>), grid, block, 0, s, a);
        else hipLaunchKernelGGL((k_rope<128, false>), grid, block, 0, s, a);
    } else {
        if (p.interleaved) hipLaunchKernelGGL((k_rope<64, true>), grid, block, 0, s, a);
        else hipLaunchKernelGGL((k_rope<64, false>), grid, block, 0, s, a);
    }
    return hipGetLastError();
}

hipError_t launch_kv_read(const moe_mxfp4_kv_cache& c, const int32_t* slots, int32_t n, void* k, void* v,
                          hipStream_t s) {
    ReadArgs a{};
    a.k = static_cast<const uint8_t*>(c.k); a.v = static_cast<const uint8_t*>(c.v);
    a.ks = c.format == MOE_KV_MXFP4 ? c.k_scale : nullptr;
    a.vs = c.format == MOE_KV_MXFP4 ? c.v_scale : nullptr;
    a.slots = slots; a.ko = static_cast<uint16_t*>(k); a.vo = static_cast<uint16_t*>(v);
    a.Hk = c.kv_heads; a.nslots = c.num_pages * c.page_size; a.shift = log2_of(c.page_size);
    a.rows = (int64_t)n * c.kv_heads;
    a.first = k ? 0 : 1;
    const int64_t lanes = a.rows * (c.head_dim / 8);
    const dim3 grid((unsigned)((lanes + kThreads - 1) / kThreads), k && v ? 2 : 1), block(kThreads);
    if (c.head_dim == 128) hipLaunchKernelGGL(k_kv_read<128>, grid, block, 0, s, a);
    else hipLaunchKernelGGL(k_kv_read<64>, grid, block, 0, s, a);
    return hipGetLastError();
}

}  // namespace moe
