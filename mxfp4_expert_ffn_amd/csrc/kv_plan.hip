// Cache plan: block tables, slot map and positions from request lengths.
//
// What a request gets depends on the requests before it through three prefix
// sums only: rows, pages needed and pages given back (moe_mxfp4.h).  Every
// workgroup forms all three itself, into LDS (B <= 4096: three ints each),
// and then writes its share of the rows and of the moved pages, so the call
// is one launch with no wait between workgroups.  That is safe because
// nothing a workgroup reads is written by the launch: the small state arrays
// have separate outputs, new table entries lie behind the held ones, and
// pages taken from the ring and pages appended to it are different entries
// (count + given back <= num_pages, so the append never wraps onto an entry
// that is read).  Bound by latency: loads, three scans and the writes in
// sequence, 8.0 us for 32 requests of 8 rows and 8.3 us for 256 prompts, 310
// thousand rows.
#include "kv_cache.hpp"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kPer = 4;                            // requests per thread and round
constexpr int kRound = kThreads * kPer;
constexpr int kRowsPer = 4;                        // rows per thread and step

struct PlanArgs {
    const int32_t *ctx, *nw, *held, *state;
    int32_t *table, *held_out, *ring, *state_out, *cu_q, *kv_lens, *slots, *positions, *refused;
    int32_t B, T, W, N, shift;
};

// Inclusive sum over the workgroup's threads; total: the sum of all.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* sh, int tid, int64_t& total) {
    const int lane = tid % kWave, wave = tid / kWave;
#pragma unroll
    for (int off = 1; off < kWave; off <<= 1) {
        const int64_t o = __shfl_up(v, off);
        if (lane >= off) v += o;
    }
    __syncthreads();                               // the last scan's sums have been read
    if (lane == kWave - 1) sh[wave] = v;
    __syncthreads();
    total = 0;
    int64_t before = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        if (w < wave) before += sh[w];
        total += sh[w];
    }
    return v + before;
}

// Ring position x in [0, 2 n) -> [0, n).
__device__ __forceinline__ int32_t wrap(int32_t x, int32_t n) { return x >= n ? x - n : x; }

// Last i in [0, n) with start[i] <= x (start ascending, start[0] <= x): the
// range that holds x, empty ranges skipped.
__device__ __forceinline__ int find_range(const int32_t* start, int n, int32_t x) {
    int lo = 0, hi = n;                            // start[lo] <= x < start[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (start[mid] <= x) lo = mid; else hi = mid;
    }
    return lo;
}

__global__ __launch_bounds__(kThreads) void k_plan(PlanArgs a) {
    extern __shared__ int32_t sh[];
    __shared__ int64_t part[kWaves];
    __shared__ int sh_refused;
    int32_t* row0 = sh;                            // [B] first row of a request (min with T)
    int32_t* take0 = sh + a.B;                     // [B] pages taken before it, ~that if it is refused
    int32_t* back0 = sh + 2 * a.B;                 // [B] pages given back before it
    const int tid = threadIdx.x;
    const bool first = blockIdx.x == 0;
    int32_t head = a.state[0], count = a.state[1];
    const bool state_ok = head >= 0 && head < a.N && count >= 0 && count <= a.N;
    const int32_t state0 = head, state1 = count;
    if (!state_ok) head = count = 0;
    if (tid == 0) sh_refused = 0;
    const int32_t ps1 = (1 << a.shift) - 1;
    const int64_t room = (int64_t)a.W << a.shift;
    int64_t rows = 0, needs = 0, backs = 0;        // of the rounds before
    int32_t taken = 0, given = 0;                  // granted
    for (int r0 = 0; r0 < a.B; r0 += kRound) {
        int32_t ctx[kPer], nw[kPer], held[kPer];
        int64_t n = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int b = r0 + tid * kPer + i;
            const bool in = b < a.B;
            ctx[i] = in ? a.ctx[b] : 0;
            nw[i] = in ? a.nw[b] : 0;
            held[i] = in ? a.held[b] : 0;
            n += max(nw[i], 0);
        }
        int64_t total;
        int64_t at = rows + block_scan(n, part, tid, total) - n;      // rows before this thread's requests
        rows += total;
        int32_t need[kPer], back[kPer];
        int64_t cu[kPer], sn = 0, sb = 0;
        bool good[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            cu[i] = at;
            at += max(nw[i], 0);
            const bool held_ok = held[i] >= 0 && held[i] <= a.W;
            const int64_t len = (int64_t)ctx[i] + nw[i];
            good[i] = held_ok && (nw[i] == -1 || (ctx[i] >= 0 && nw[i] >= 0 && len <= room && at <= a.T));
            need[i] = good[i] && nw[i] >= 0 ? max((int32_t)((len + ps1) >> a.shift) - held[i], 0) : 0;
            back[i] = good[i] && nw[i] == -1 ? held[i] : 0;
            sn += need[i];
            sb += back[i];
        }
        int64_t tn, tb;
        int64_t pn = needs + block_scan(sn, part, tid, tn) - sn;
        int64_t pb = backs + block_scan(sb, part, tid, tb) - sb;
        needs += tn;
        backs += tb;
        int32_t bad = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int b = r0 + tid * kPer + i;
            const bool ends = nw[i] == -1;
            const bool ok = good[i] && (ends ? back[i] == 0 || (state_ok && count + pb + back[i] <= a.N)
                                             : need[i] == 0 || pn + need[i] <= count);
            if (b < a.B) {
                // sums past the limits belong to refused requests, which move nothing
                row0[b] = (int32_t)min(cu[i], (int64_t)a.T);
                const int32_t t0 = (int32_t)min(pn, (int64_t)count);
                take0[b] = ok ? t0 : ~t0;
                back0[b] = (int32_t)min(pb, (int64_t)a.N);
                if (first) {
                    a.cu_q[b] = row0[b];
                    a.kv_lens[b] = ok && !ends ? ctx[i] + nw[i] : 0;
                    a.held_out[b] = ok ? held[i] + need[i] - back[i] : held[i];
                    bad += !ok;
                }
            }
            pn += need[i];
            pb += back[i];
        }
        if (bad) atomicAdd(&sh_refused, bad);      // an integer count: order does not matter
    }
    __syncthreads();
    const int32_t rows_end = (int32_t)min(rows, (int64_t)a.T);
    // pages, a wave per request.  head < N and both sums stay within N for
    // what is granted, so a ring position needs one conditional subtraction.
    for (int b = blockIdx.x * kWaves + tid / kWave; b < a.B; b += gridDim.x * kWaves) {
        const int32_t t0 = take0[b];
        if (t0 < 0) continue;                      // refused
        const int32_t nw = a.nw[b], held = a.held[b];
        int32_t* row = a.table + (size_t)b * a.W;
        if (nw == -1) {
            for (int k = tid % kWave; k < held; k += kWave) a.ring[wrap(head + count + back0[b] + k, a.N)] = row[k];
        } else {
            const int32_t need = (int32_t)(((int64_t)a.ctx[b] + nw + ps1) >> a.shift) - held;
            for (int k = tid % kWave; k < need; k += kWave) row[held + k] = a.ring[wrap(head + t0 + k, a.N)];
        }
    }
    // rows: four in a row per thread, their request found by bisection
    const int nstep = gridDim.x * kThreads * kRowsPer;
    for (int t = (blockIdx.x * kThreads + tid) * kRowsPer; t < a.T; t += nstep) {
        int b = 0;
        if (t < rows_end) b = find_range(row0, a.B, t);
        int32_t slot[kRowsPer], pos[kRowsPer];
#pragma unroll
        for (int i = 0; i < kRowsPer; ++i) {
            const int r = t + i;
            slot[i] = pos[i] = -1;
            if (r < rows_end) {
                while (b + 1 < a.B && row0[b + 1] <= r) ++b;
                const int32_t t0 = take0[b];
                if (t0 >= 0) {
                    const int32_t p = a.ctx[b] + (r - row0[b]), k = p >> a.shift, held = a.held[b];
                    const int32_t page = k < held ? a.table[(size_t)b * a.W + k] : a.ring[wrap(head + t0 + k - held, a.N)];
                    pos[i] = p;
                    if (page >= 0 && page < a.N) slot[i] = (page << a.shift) | (p & ps1);
                }
            }
        }
        if (t + kRowsPer <= a.T) {
            *reinterpret_cast<int4*>(a.slots + t) = make_int4(slot[0], slot[1], slot[2], slot[3]);
            *reinterpret_cast<int4*>(a.positions + t) = make_int4(pos[0], pos[1], pos[2], pos[3]);
        } else {
#pragma unroll
            for (int i = 0; i < kRowsPer; ++i)
                if (t + i < a.T) {
                    a.slots[t + i] = slot[i];
                    a.positions[t + i] = pos[i];
                }
        }
    }
    if (!first) return;
    // the state after the call: granted requests that move pages come before
    // the first whose pages do not fit, so the last of them ends both sums
    for (int b = tid; b < a.B; b += kThreads) {
        const int32_t t0 = take0[b], held = a.held[b];
        if (t0 < 0) continue;
        if (a.nw[b] == -1) {
            if (held > 0) given = max(given, back0[b] + held);
        } else {
            const int32_t need = (int32_t)(((int64_t)a.ctx[b] + a.nw[b] + ps1) >> a.shift) - held;
            if (need > 0) taken = max(taken, t0 + need);
        }
    }
#pragma unroll
    for (int off = kWave / 2; off >= 1; off >>= 1) {
        taken = max(taken, __shfl_xor(taken, off));
        given = max(given, __shfl_xor(given, off));
    }
    __syncthreads();
    if (tid % kWave == 0) part[tid / kWave] = ((int64_t)taken << 32) | (uint32_t)given;
    __syncthreads();
    if (tid == 0) {
        for (int w = 0; w < kWaves; ++w) {
            taken = max(taken, (int32_t)(part[w] >> 32));
            given = max(given, (int32_t)(uint32_t)part[w]);
        }
        a.cu_q[a.B] = rows_end;
        *a.refused = sh_refused;
        a.state_out[0] = state_ok ? wrap(head + taken, a.N) : state0;
        a.state_out[1] = state_ok ? count - taken + given : state1;
    }
}

}  // namespace

hipError_t launch_cache_plan(const moe_mxfp4_plan_args& p, hipStream_t s) {
    PlanArgs a{};
    a.ctx = p.ctx_lens; a.nw = p.new_lens; a.held = p.held; a.state = p.free_state;
    a.table = p.block_table; a.held_out = p.held_out; a.ring = p.free_ring; a.state_out = p.free_state_out;
    a.cu_q = p.cu_q; a.kv_lens = p.kv_lens; a.slots = p.slots; a.positions = p.positions; a.refused = p.refused;
    a.B = p.batch; a.T = p.num_tokens; a.W = p.max_blocks; a.N = p.num_pages; a.shift = log2_of(p.page_size);
    // a workgroup per 1024 rows (one step of it) or 16 requests (four steps), whichever asks for more
    const int64_t by_rows = ((int64_t)a.T + kThreads * kRowsPer - 1) / (kThreads * kRowsPer);
    const int64_t by_reqs = (a.B + 4 * kWaves - 1) / (4 * kWaves);
    int64_t grid = by_rows > by_reqs ? by_rows : by_reqs;
    grid = grid < 1 ? 1 : grid > 512 ? 512 : grid;
    const size_t lds = (size_t)(a.B > 0 ? a.B : 1) * 3 * sizeof(int32_t);
    hipLaunchKernelGGL(k_plan, dim3((unsigned)grid), dim3(kThreads), lds, s, a);
    return hipGetLastError();
}

}  // namespace moe
