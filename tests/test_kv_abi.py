"""The attention half of a verify step refuses what it does not handle, on the
host, before anything is queued; and the host-side forms the GPU tests check
against hold by themselves (CPU only)."""
import ctypes

import numpy as np
import pytest

import mxfp4_expert_ffn_amd as moe
from tests import kv_reference as ref

torch = pytest.importorskip("torch")

FAKE = 1 << 20          # a 16-byte-aligned stand-in device address (never dereferenced)
OK, INVALID, SHAPE, ALIGN, WORKSPACE, HIP = 0, 1, 2, 4, 5, 6


def _with(struct, base, kw):
    s = struct(**{**base, **kw})
    s.struct_size = kw.get("struct_size", ctypes.sizeof(struct))
    return s


CACHE = dict(format=1, num_pages=8, page_size=64, kv_heads=2, head_dim=128, k=FAKE, v=FAKE, k_scale=FAKE, v_scale=FAKE)


def cache(**kw):
    return _with(moe.KvCacheStruct, CACHE, kw)


@pytest.fixture
def no_launch(monkeypatch):
    """A call that gets past its checks stops at its launch site, as a failed launch (MOE_ERR_HIP)."""
    return lambda name: monkeypatch.setenv("MOE_MXFP4_FAULT", name)


@pytest.mark.parametrize("kw,status", [
    (dict(), OK), (dict(format=0), OK), (dict(format=2), INVALID), (dict(struct_size=4), INVALID),
    (dict(num_pages=0), INVALID), (dict(page_size=0), INVALID), (dict(kv_heads=0), INVALID), (dict(head_dim=0), INVALID),
    (dict(page_size=8), SHAPE), (dict(page_size=48), SHAPE), (dict(page_size=512), SHAPE), (dict(page_size=256), OK),
    (dict(head_dim=96), SHAPE), (dict(head_dim=256), SHAPE), (dict(head_dim=64), OK), (dict(kv_heads=1025), SHAPE),
    (dict(num_pages=1 << 25), SHAPE), (dict(num_pages=(1 << 25) - 1), OK),
    (dict(k=None, v=None, k_scale=None, v_scale=None), OK),                    # pointers are not looked at
])
def test_cache_bytes(kw, status):
    d, s = ctypes.c_size_t(7), ctypes.c_size_t(7)
    c = cache(**kw)
    f = moe.lib().moe_mxfp4_kv_cache_bytes
    assert f(ctypes.byref(c), ctypes.byref(d), ctypes.byref(s)) == status
    if status == OK:
        rows = c.num_pages * c.page_size * c.kv_heads
        assert (d.value, s.value) == ((rows * c.head_dim // 2, rows * c.head_dim // 32) if c.format else (rows * c.head_dim * 2, 0))
    else:
        assert (d.value, s.value) == (7, 7)
    assert f(None, ctypes.byref(d), ctypes.byref(s)) == INVALID
    assert f(ctypes.byref(cache()), None, ctypes.byref(s)) == INVALID and f(ctypes.byref(cache()), ctypes.byref(d), None) == INVALID


def _each(values):
    """FAKE addresses, all different."""
    return {n: FAKE * (2 + i) for i, n in enumerate(values)}


PLAN_PTRS = [n for n, t in moe.PlanArgs._fields_ if t is ctypes.c_void_p]
PLAN = dict(batch=3, num_tokens=24, max_blocks=4, page_size=64, num_pages=32, **_each(PLAN_PTRS))


@pytest.mark.parametrize("kw,status", [
    (dict(), HIP), (dict(struct_size=8), INVALID), (dict(batch=-1), INVALID), (dict(num_tokens=-1), INVALID),
    (dict(max_blocks=0), INVALID), (dict(page_size=0), INVALID), (dict(num_pages=0), INVALID),
    (dict(batch=4096), HIP), (dict(batch=4097), SHAPE), (dict(page_size=24), SHAPE), (dict(num_tokens=(1 << 30) + 1), SHAPE),
    (dict(num_pages=1 << 25), SHAPE), (dict(max_blocks=1 << 25), SHAPE),
    (dict(held_out=PLAN["held"]), INVALID), (dict(free_state_out=PLAN["free_state"]), INVALID),
    *[({n: None}, INVALID) for n in PLAN_PTRS], *[({n: PLAN[n] + 4}, ALIGN) for n in PLAN_PTRS],
    # no requests: nothing of theirs is needed; no rows: no slots
    (dict(batch=0, ctx_lens=None, new_lens=None, block_table=None, held=None, held_out=None, kv_lens=None), HIP),
    (dict(num_tokens=0, slots=None, positions=None), HIP),
])
def test_plan_refusals(kw, status, no_launch):
    no_launch("plan")
    a = _with(moe.PlanArgs, PLAN, kw)
    assert moe.lib().moe_mxfp4_cache_plan(ctypes.byref(a), None) == status
    assert moe.lib().moe_mxfp4_cache_plan(None, None) == INVALID


ROPE_PTRS = [n for n, t in moe.RopeArgs._fields_ if t is ctypes.c_void_p]
ROPE = dict(num_tokens=5, heads=4, kv_heads=2, head_dim=128, rot_dim=128, interleaved=0, eps=1e-6, q_stride=512,
            k_stride=256, v_stride=256, **_each(ROPE_PTRS))


@pytest.mark.parametrize("kw,ckw,status", [
    (dict(), {}, HIP), (dict(), None, HIP), (dict(struct_size=8), {}, INVALID), (dict(num_tokens=-1), {}, INVALID),
    (dict(num_tokens=0, q=None, k=None, v=None, positions=None, slots=None, q_out=None), {}, OK),
    (dict(heads=0), {}, INVALID), (dict(kv_heads=0), {}, INVALID), (dict(head_dim=0), {}, INVALID),
    (dict(rot_dim=-16), {}, INVALID), (dict(rot_dim=144), {}, INVALID), (dict(rot_dim=24), {}, SHAPE), (dict(rot_dim=64), {}, HIP),
    (dict(rot_dim=0, inv_freq=None), {}, HIP), (dict(inv_freq=None), {}, INVALID),
    (dict(eps=-1.0), {}, INVALID), (dict(eps=float("nan")), {}, INVALID), (dict(eps=float("inf")), {}, INVALID), (dict(eps=0.0), {}, HIP),
    (dict(head_dim=32, rot_dim=32), {}, SHAPE), (dict(heads=1025, q_stride=1025 * 128), {}, SHAPE), (dict(num_tokens=1 << 24), {}, SHAPE),
    (dict(q_stride=504), {}, INVALID), (dict(q_stride=513), {}, INVALID), (dict(k_stride=248), {}, INVALID),
    (dict(v_stride=248), {}, INVALID), (dict(v_stride=260), {}, INVALID), (dict(v_stride=0, v=None, slots=None), None, HIP),
    (dict(), dict(kv_heads=4), INVALID), (dict(), dict(head_dim=64), INVALID), (dict(), dict(k=None), INVALID),
    (dict(), dict(v_scale=None), INVALID), (dict(), dict(k_scale=FAKE + 8), ALIGN), (dict(), dict(format=0, k_scale=None, v_scale=None), HIP),
    (dict(q=None), {}, INVALID), (dict(k=None), {}, INVALID), (dict(v=None), {}, INVALID), (dict(positions=None), {}, INVALID),
    (dict(slots=None), {}, INVALID), (dict(q_out=None), {}, INVALID), (dict(k_out=None), {}, HIP), (dict(k_out=None), None, INVALID),
    (dict(q_weight=None, k_weight=None), {}, HIP),
    (dict(q_out=ROPE["q"]), {}, HIP), (dict(q_out=ROPE["q"], q_stride=520), {}, INVALID),
    (dict(k_out=ROPE["k"]), {}, HIP), (dict(k_out=ROPE["k"], k_stride=264), {}, INVALID),
    *[({n: ROPE[n] + 8}, {}, ALIGN) for n in ROPE_PTRS],
])
def test_rope_refusals(kw, ckw, status, no_launch):
    no_launch("rope")
    a = _with(moe.RopeArgs, ROPE, kw)
    c = None if ckw is None else ctypes.byref(cache(**ckw))
    assert moe.lib().moe_mxfp4_qk_norm_rope(ctypes.byref(a), c, None) == status
    assert moe.lib().moe_mxfp4_qk_norm_rope(None, c, None) == INVALID


def test_kv_read_refusals(no_launch):
    no_launch("kvread")
    f = moe.lib().moe_mxfp4_kv_read
    c = ctypes.byref(cache())
    assert f(c, FAKE, 4, FAKE, FAKE, None) == HIP and f(c, FAKE, 4, None, FAKE, None) == HIP and f(c, FAKE, 4, FAKE, None, None) == HIP
    assert f(c, None, 0, None, None, None) == OK and f(c, FAKE, -1, FAKE, FAKE, None) == INVALID
    assert f(c, None, 4, FAKE, FAKE, None) == INVALID and f(c, FAKE, 4, None, None, None) == INVALID
    assert f(c, FAKE + 4, 4, FAKE, FAKE, None) == ALIGN and f(c, FAKE, 4, FAKE + 2, FAKE, None) == ALIGN
    assert f(c, FAKE, 1 << 27, FAKE, FAKE, None) == SHAPE
    assert f(None, FAKE, 4, FAKE, FAKE, None) == INVALID and f(ctypes.byref(cache(v=None)), FAKE, 4, FAKE, FAKE, None) == INVALID


ATTN_PTRS = [n for n, t in moe.AttnArgs._fields_ if t is ctypes.c_void_p]
ATTN = dict(batch=2, num_tokens=16, heads=8, max_q=8, max_kv=100, max_blocks=4, causal=1, window=0, sinks=0, scale=0.1,
            q_stride=1024, out_stride=1024, **_each(ATTN_PTRS))


@pytest.mark.parametrize("kw,ckw,status", [
    (dict(), {}, HIP), (dict(struct_size=8), {}, INVALID), (dict(batch=-1), {}, INVALID), (dict(num_tokens=-1), {}, INVALID),
    (dict(batch=0, q=None, out=None), {}, OK), (dict(num_tokens=0, q=None, out=None), {}, OK),
    (dict(heads=0), {}, INVALID), (dict(heads=7, q_stride=896, out_stride=896), {}, INVALID), (dict(max_q=0), {}, INVALID),
    (dict(max_kv=0), {}, INVALID), (dict(max_blocks=0), {}, INVALID), (dict(window=-1), {}, INVALID), (dict(sinks=-1, window=4), {}, INVALID),
    (dict(sinks=4), {}, INVALID), (dict(sinks=4, window=1), {}, HIP), (dict(scale=0.0), {}, INVALID), (dict(scale=-1.0), {}, INVALID),
    (dict(scale=float("nan")), {}, INVALID), (dict(scale=float("inf")), {}, INVALID),
    (dict(q_stride=1016), {}, INVALID), (dict(q_stride=1028), {}, INVALID), (dict(out_stride=1016), {}, INVALID),
    (dict(out_stride=1030), {}, INVALID), (dict(q_stride=2048, out_stride=1032), {}, HIP),
    (dict(batch=65536), {}, SHAPE), (dict(num_tokens=1 << 27), {}, SHAPE), (dict(batch=65535), dict(kv_heads=32), INVALID),
    (dict(batch=65535, heads=32, q_stride=4096, out_stride=4096), dict(kv_heads=32), SHAPE),
    (dict(), dict(head_dim=96), SHAPE), (dict(), dict(v=None), INVALID), (dict(), dict(v=FAKE + 1), ALIGN),
    (dict(out=ATTN["q"]), {}, INVALID),
    *[({n: None}, {}, INVALID) for n in ATTN_PTRS], *[({n: ATTN[n] + 4}, {}, ALIGN) for n in ATTN_PTRS],
])
def test_attention_refusals(kw, ckw, status, no_launch):
    no_launch("attn")
    a, c = _with(moe.AttnArgs, ATTN, kw), cache(**ckw)
    assert moe.lib().moe_mxfp4_attention(ctypes.byref(a), ctypes.byref(c), FAKE, 1 << 40, None) == status
    assert moe.lib().moe_mxfp4_attention(None, ctypes.byref(c), FAKE, 1 << 40, None) == INVALID
    assert moe.lib().moe_mxfp4_attention(ctypes.byref(a), None, FAKE, 1 << 40, None) == INVALID


def test_attention_workspace(no_launch):
    no_launch("attn")
    L = moe.lib()
    a, c = _with(moe.AttnArgs, ATTN, dict(max_kv=100000)), cache()
    need = L.moe_mxfp4_attention_workspace_bytes(ctypes.byref(a), ctypes.byref(c))
    assert need > 0
    f = L.moe_mxfp4_attention
    assert f(ctypes.byref(a), ctypes.byref(c), FAKE, need, None) == HIP
    assert f(ctypes.byref(a), ctypes.byref(c), FAKE, need - 1, None) == WORKSPACE
    assert f(ctypes.byref(a), ctypes.byref(c), None, need, None) == WORKSPACE
    assert f(ctypes.byref(a), ctypes.byref(c), FAKE + 8, need, None) == ALIGN
    for bad in (dict(batch=0), dict(scale=0.0), dict(heads=7)):
        b = _with(moe.AttnArgs, ATTN, bad)
        assert L.moe_mxfp4_attention_workspace_bytes(ctypes.byref(b), ctypes.byref(c)) == 0
    one = _with(moe.AttnArgs, ATTN, dict(max_kv=64))
    assert L.moe_mxfp4_attention_workspace_bytes(ctypes.byref(one), ctypes.byref(c)) == 0
    assert f(ctypes.byref(one), ctypes.byref(c), None, 0, None) == HIP


def test_binding_refuses_wrong_tensors():
    c = moe.KvCache(4, 16, 2, 64, device="cpu")
    assert c.k.shape == (4, 2, 16, 32) and c.v_scale.shape == (4, 2, 16, 2) and c.fmt == moe.KV_MXFP4
    with pytest.raises(moe.MoeError):
        moe.KvCache(4, 24, 2, 64, device="cpu")
    with pytest.raises(ValueError):
        moe.KvCache(4, 16, 2, 64, fmt=3, device="cpu")
    with pytest.raises(ValueError):
        moe.KvCache.wrap(c.k, c.v[:2], c.k_scale, c.v_scale)
    with pytest.raises(ValueError):
        moe.KvCache.wrap(c.k, c.v)                              # uint8 codes without scales
    q = torch.zeros((3, 4, 64), dtype=torch.bfloat16)
    i32 = dict(dtype=torch.int32)
    table, cu, lens = torch.zeros((1, 4), **i32), torch.zeros(2, **i32), torch.zeros(1, **i32)
    with pytest.raises(ValueError, match="CUDA"):               # CPU tensors
        moe.attention(q, c, table, cu, lens, max_q=3, max_kv=8)
    with pytest.raises(ValueError, match="cu_q"):
        moe.attention(q, c, table, lens, lens, max_q=3, max_kv=8)
    with pytest.raises(ValueError, match="q:"):
        moe.attention(q.float(), c, table, cu, lens, max_q=3, max_kv=8)
    with pytest.raises(ValueError, match="q:"):
        moe.attention(q.transpose(0, 1), c, table, cu, lens, max_q=3, max_kv=8)
    pos, freq = torch.zeros(3, **i32), torch.zeros(32, dtype=torch.float64)
    with pytest.raises(ValueError, match="CUDA"):
        moe.qk_norm_rope(q, q[:, :2], None, pos, freq)
    with pytest.raises(ValueError, match="inv_freq"):
        moe.qk_norm_rope(q, q[:, :2], None, pos, freq.float())
    with pytest.raises(ValueError, match="slots"):
        moe.qk_norm_rope(q, q[:, :2], q[:, :2], pos, freq, cache=c)
    with pytest.raises(ValueError, match="CUDA"):
        moe.cache_plan(lens, lens, table, lens, torch.zeros(4, **i32), torch.zeros(2, **i32), page_size=16, num_tokens=0)
    with pytest.raises(ValueError, match="CUDA"):
        moe.kv_read(c, lens)


def test_reference_layout_round_trips_and_values():
    rng = np.random.default_rng(11)
    for D, ps in ((64, 16), (128, 16), (128, 64)):
        codes = rng.integers(0, 256, (2, 3, ps, D // 2), dtype=np.uint8)
        scales = rng.integers(100, 140, (2, 3, ps, D // 32), dtype=np.uint8)
        p, s = ref.v_pack(codes, scales)
        assert sorted(p[1, 2].reshape(-1)) == sorted(codes[1, 2].reshape(-1))
        u, us = ref.v_unpack(p, s)
        assert np.array_equal(u, codes) and np.array_equal(us, scales)
        # 16 bytes of a piece: the same D/16 elements of 512/D rows
        n, C = 512 // D, D // 32
        assert np.array_equal(p[0, 0].reshape(-1)[16:32].reshape(n, C), codes[0, 0, :n, C:2 * C])
    assert ref.values(np.array([[0x21] + [0] * 15], np.uint8), np.array([[128]], np.uint8))[0, :2].tolist() == [1.0, 2.0]


def test_reference_attention_against_plain_softmax():
    """The reference with everything visible is torch's softmax product; with a window, a masked one."""
    rng = np.random.default_rng(12)
    D, ps, HK, G = 64, 16, 2, 3
    kx, vx = rng.standard_normal((2, 4, HK, ps, D))
    q = rng.standard_normal((5, HK * G, D))
    table = np.array([[2, 0, 3]])
    for causal, window, sinks in ((True, 0, 0), (False, 0, 0), (True, 7, 2), (False, 9, 0)):
        out, bound = ref.attention(q, kx, vx, table, [0, 5], [39], ps, scale=0.125, causal=causal, window=window, sinks=sinks)
        k = torch.from_numpy(kx[[2, 0, 3]].transpose(1, 0, 2, 3).reshape(HK, 48, D)[:, :39])
        v = torch.from_numpy(vx[[2, 0, 3]].transpose(1, 0, 2, 3).reshape(HK, 48, D)[:, :39])
        p, j = torch.arange(34, 39)[:, None], torch.arange(39)
        see = (j <= p) if causal else torch.ones(5, 39, dtype=torch.bool)
        if window:
            see = see & ((p - j < window) | (j < sinks))
        x = torch.from_numpy(q).view(5, HK, G, D).permute(1, 2, 0, 3) @ k[:, None].transpose(2, 3) * 0.125
        want = (x.masked_fill(~see, float("-inf")).softmax(-1) @ v[:, None]).permute(2, 0, 1, 3).reshape(5, HK * G, D)
        assert np.abs(out - want.numpy()).max() < 1e-12 and np.isfinite(bound).all()


def test_reference_plan_invariants():
    """Over random steps no page is ever in two places, and none is lost."""
    rng = np.random.default_rng(13)
    B, W, ps, N = 9, 12, 16, 60
    table, held = np.full((B, W), -1, np.int32), np.zeros(B, np.int32)
    ring, state = rng.permutation(N).astype(np.int32), np.array([17, N], np.int32)
    ctx = np.zeros(B, np.int32)
    refused = 0
    for step in range(200):
        new = rng.integers(0, 40, B).astype(np.int32)
        new[rng.random(B) < 0.2] = -1
        r = ref.plan(ctx, new, table, held, ring, state, ps, int(np.maximum(new, 0).sum()))
        refused += int(r["refused"][0])
        table, held, ring, state = r["table"], r["held"], r["ring"], r["free_state"]
        free = [int(ring[(state[0] + i) % N]) for i in range(state[1])]
        used = [int(table[b, k]) for b in range(B) for k in range(held[b])]
        assert sorted(free + used) == list(range(N))
        ctx = np.where(new == -1, 0, np.where(r["kv_lens"] > 0, np.maximum(r["kv_lens"] - rng.integers(0, 8, B), 0), ctx)).astype(np.int32)
    assert refused > 0
