"""Plain 64-bit forms of the attention half of a verify step, and the cache
layout of the C header written out on the host.  Nothing here uses the
library; MXFP4 quantisation is the CPU oracle's."""
from __future__ import annotations

import dataclasses

import numpy as np

import oracle
import synth

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def bf16_round(x):
    """float -> the nearest bf16, as float64 (NaN and infinities kept)."""
    x = np.asarray(x, np.float32)
    return np.where(np.isfinite(x), synth.bf16_bits_to_f32(synth.bf16_bits_from_f32(np.where(np.isfinite(x), x, 0))), x).astype(np.float64)


# ------------------------------------------------------------------ plan

def plan(ctx, new, table, held, ring, state, ps, T):
    """One request after another."""
    B, W = table.shape
    N = len(ring)
    head, count = int(state[0]), int(state[1])
    state_ok = 0 <= head < N and 0 <= count <= N
    offered = count if state_ok else 0
    table, ring, held_out = table.copy(), ring.copy(), held.copy()
    old_ring, old_table = ring.copy(), table.copy()
    cu, kv, refused = [0], np.zeros(B, np.int32), 0
    slots, positions = np.full(T, -1, np.int32), np.full(T, -1, np.int32)
    at, needs, backs, taken, given = 0, 0, 0, 0, 0
    for b in range(B):
        c, n, h = int(ctx[b]), int(new[b]), int(held[b])
        first, at = at, at + max(n, 0)
        cu.append(min(at, T))
        ok = 0 <= h <= W
        if n == -1:
            if ok:
                backs += h
                ok = h == 0 or (state_ok and offered + backs <= N)
            if ok:
                for k in range(h):
                    ring[(head + offered + backs - h + k) % N] = old_table[b, k]
                held_out[b] = 0
                given += h
            refused += not ok
            continue
        ok = ok and c >= 0 and n >= 0 and c + n <= W * ps and at <= T
        if ok:
            need = max(0, -(-(c + n) // ps) - h)
            needs += need
            ok = need == 0 or needs <= offered
        if not ok:
            refused += 1
            continue
        for k in range(need):
            table[b, h + k] = old_ring[(head + needs - need + k) % N]
        taken += need
        held_out[b] = h + need
        kv[b] = c + n
        for i in range(n):
            pos = c + i
            page = int(table[b, pos // ps])
            positions[first + i] = pos
            if 0 <= page < N:
                slots[first + i] = page * ps + pos % ps
    state_out = np.array([(head + taken) % N, count - taken + given] if state_ok else state, np.int32)
    return dict(table=table, ring=ring, held=held_out, free_state=state_out, cu_q=np.array(cu, np.int32), kv_lens=kv,
                slots=slots, positions=positions, refused=np.array([refused], np.int32))


# ------------------------------------------------------------------ the cache's layout

@dataclasses.dataclass
class HostCache:
    """Buffers of a cache and the float64 values they stand for, [page, head, row, D]."""
    fp4: bool
    k: np.ndarray
    v: np.ndarray
    k_scale: np.ndarray | None
    v_scale: np.ndarray | None
    kx: np.ndarray
    vx: np.ndarray


def quantise(x):
    """float [..., D] -> (codes [..., D/2], scales [..., D/32]) by the oracle's rule."""
    x = np.ascontiguousarray(x, np.float32)
    p, s = oracle.quant_mxfp4(x.reshape(-1, x.shape[-1]))
    return p.reshape(*x.shape[:-1], -1), s.reshape(*x.shape[:-1], -1)


def values(codes, scales):
    """E2M1 codes and E8M0 bytes -> float64 (0xFF: NaN)."""
    c = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)
    x = np.where(c >= 8, -E2M1[c & 7], E2M1[c & 7])
    s = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127))
    return x * np.repeat(s, 32, -1)


def v_pack(codes, scales):
    """Row-major V codes [P, H, ps, D/2] and scales -> the header's order, element by element of its formula."""
    P, H, ps, half = codes.shape
    C = half // 16
    n = 512 // (2 * half)
    out, so = np.empty_like(codes), np.empty_like(scales)
    flat, sflat = out.reshape(P, H, -1), so.reshape(P, H, -1)
    for row in range(ps):
        for c in range(half):
            flat[:, :, (row // n) * (n * half) + (c // C) * 16 + (row % n) * C + c % C] = codes[:, :, row, c]
        for b in range(C):
            sflat[:, :, (row // 8) * (8 * C) + b * 8 + row % 8] = scales[:, :, row, b]
    return out, so


def v_unpack(codes, scales):
    """The inverse of v_pack."""
    idx_c, idx_s = np.arange(codes[0, 0].size), np.arange(scales[0, 0].size)
    pc, psc = v_pack(idx_c.reshape(1, 1, *codes.shape[2:]), idx_s.reshape(1, 1, *scales.shape[2:]))
    out, so = np.empty_like(codes), np.empty_like(scales)
    out.reshape(*codes.shape[:2], -1)[..., pc.reshape(-1)] = codes.reshape(*codes.shape[:2], -1)
    so.reshape(*scales.shape[:2], -1)[..., psc.reshape(-1)] = scales.reshape(*scales.shape[:2], -1)
    return out, so


def host_cache(rng, fp4, pages, heads, ps, D, k=None, v=None):
    """A cache of N(0, 1) contents (or of the given float arrays)."""
    shape = (pages, heads, ps, D)
    k = rng.standard_normal(shape) if k is None else k
    v = rng.standard_normal(shape) if v is None else v
    if not fp4:
        kx, vx = bf16_round(k), bf16_round(v)
        bits = [(np.ascontiguousarray(x, np.float32).view(np.uint32) >> 16).astype(np.uint16) for x in (kx, vx)]
        return HostCache(False, *bits, None, None, kx, vx)
    (kc, ks), (vc, vs) = quantise(k), quantise(v)
    pv, psv = v_pack(vc, vs)
    return HostCache(True, kc, pv, ks, psv, values(kc, ks), values(vc, vs))


# ------------------------------------------------------------------ norms and rotation

def norm_rope(x, weight, pos, freq, eps, interleaved):
    """x [T, H, D] float64 -> (rotated, |a| + |b| of each element's pair)."""
    y = np.asarray(x, np.float64)
    if weight is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    half = len(freq)
    i = np.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    ang = np.asarray(pos, np.float64)[:, None, None] * np.asarray(freq, np.float64)
    out, size = y.copy(), np.abs(y)
    out[..., a] = y[..., a] * np.cos(ang) - y[..., b] * np.sin(ang)
    out[..., b] = y[..., b] * np.cos(ang) + y[..., a] * np.sin(ang)
    both = np.abs(y[..., a]) + np.abs(y[..., b])
    size[..., a] = both
    size[..., b] = both
    return out, size


# ------------------------------------------------------------------ attention

def visible(p, kv, causal, window, sinks):
    """Keys 0 .. kv-1 that a row at position p sees."""
    j = np.arange(kv)
    if p < 0:
        return np.zeros(kv, bool)
    see = j <= p if causal else np.ones(kv, bool)
    if window:
        see &= (p - j < window) | (j < sinks)
    return see


def attention(q, kx, vx, table, cu, lens, ps, *, scale, causal, window, sinks):
    """(out, bound): float64 attention of the packed rows, and how far a kernel may be off that
    rounds its softmax weights and its output to bf16 and computes in float32.

    bound = 2^-8 |out| (the output's rounding) + A (2^-8 + exp(2 e) - 1 + (n + 64) 2^-24), A = sum p_j |v_j|:
    2^-8 for the weights' rounding; e, the absolute error of a score in units of the exponent:
    (D + 8) 2^-24 scale sum |q k| for the products' float32 sum, and 8 x 2^-24 max |score| for the scaling,
    the reference and the exponential's argument; a weight and the sum of weights are each off by a
    factor within exp(+-e); (n + 64) 2^-24 for the float32 sums over n keys.
    Rows that no sequence has stay NaN in out.
    """
    T, H, D = q.shape
    HK = kx.shape[1]
    G = H // HK
    out = np.full((T, H, D), np.nan)
    bound = np.zeros((T, H, D))
    pages = kx.shape[0]
    for b in range(len(lens)):
        kv, n = int(lens[b]), int(cu[b + 1] - cu[b])
        if n == 0:
            continue
        j = np.arange(kv)
        pg = table[b][j // ps] if kv else j
        there = (pg >= 0) & (pg < pages)
        K = kx[np.where(there, pg, 0), :, j % ps]              # [kv, HK, D]
        V = vx[np.where(there, pg, 0), :, j % ps]
        for i in range(n):
            see = visible(kv - n + i, kv, causal, window, sinks) & there
            t = cu[b] + i
            if not see.any():
                out[t] = 0
                continue
            for h in range(HK):
                k, v, x = K[see, h], V[see, h], q[t, h * G:(h + 1) * G]
                s = x @ k.T * scale
                w = np.exp(s - s.max(-1, keepdims=True))
                w /= w.sum(-1, keepdims=True)
                o = w @ v
                e = ((D + 8) * scale * (np.abs(x) @ np.abs(k).T).max(-1) + 8 * np.abs(s).max(-1)) * 2.0 ** -24
                A = w @ np.abs(v)
                out[t, h * G:(h + 1) * G] = o
                bound[t, h * G:(h + 1) * G] = 2.0 ** -8 * np.abs(o) + A * (2.0 ** -8 + np.expm1(2 * e[:, None]) + (see.sum() + 64) * 2.0 ** -24)
    return out, bound
