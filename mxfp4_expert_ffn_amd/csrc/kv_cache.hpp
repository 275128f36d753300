// Declarations of the attention half of a verify step: the paged cache's
// layout (moe_mxfp4.h states it byte by byte), its plan, the norms and
// rotation that write it, and the attention that reads it.
#pragma once

#include "common.hpp"

namespace moe {

constexpr int kPlanMaxBatch = 4096;    // the plan keeps three ints a request in LDS
constexpr int kKvMaxHeads = 1024;

// Keys that share a 16-byte piece of the MXFP4 V codes: D/32 bytes each.
constexpr int v_keys_per_piece(int D) { return 512 / D; }

inline bool kv_page_size_ok(int32_t ps) { return ps == 16 || ps == 32 || ps == 64 || ps == 128 || ps == 256; }
inline int log2_of(int32_t p) { return 31 - __builtin_clz((unsigned)p); }

hipError_t launch_cache_plan(const moe_mxfp4_plan_args& a, hipStream_t s);
hipError_t launch_qk_norm_rope(const moe_mxfp4_rope_args& a, const moe_mxfp4_kv_cache* c, hipStream_t s);
hipError_t launch_kv_read(const moe_mxfp4_kv_cache& c, const int32_t* slots, int32_t n, void* k, void* v,
                          hipStream_t s);
size_t attention_workspace_bytes(const moe_mxfp4_attn_args& a, const moe_mxfp4_kv_cache& c);
hipError_t launch_attention(const moe_mxfp4_attn_args& a, const moe_mxfp4_kv_cache& c, void* workspace,
                            hipStream_t s);

}  // namespace moe
