"""GPU parity of attention over the paged cache against the 64-bit reference,
whose bound counts the roundings to bf16 of the weights and the output and the
float32 steps (kv_reference.attention)."""
import numpy as np
import pytest

import synth
from tests import kv_reference as ref
from tests import problems

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def _moe():
    import mxfp4_expert_ffn_amd as moe
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible")
    return moe


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).cuda().bfloat16()


def host(t):
    return t.double().cpu().numpy()


def to_device(moe, hc):
    bufs = [dev(x) if hc.fp4 else dev(x.view(np.int16)).view(torch.bfloat16) for x in (hc.k, hc.v)]
    return moe.KvCache.wrap(*bufs, *([dev(hc.k_scale), dev(hc.v_scale)] if hc.fp4 else []))


def problem(rng, fp4, D, HK, G, ps, new, tot, extra_rows=0):
    """Queries, a cache with its pages in random order, and a block table (unused entries name no page)."""
    blocks = [-(-t // ps) for t in tot]
    W, pages = max(max(blocks), 1) + 1, sum(blocks) + 2
    order = rng.permutation(pages).astype(np.int32)
    table = np.full((len(tot), W), -1, np.int32)
    at = 0
    for b, n in enumerate(blocks):
        table[b, :n] = order[at:at + n]
        at += n
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    T = int(cu[-1]) + extra_rows
    q = ref.bf16_round(rng.standard_normal((T, HK * G, D)) * 1.5)
    return dict(q=q, hc=ref.host_cache(rng, fp4, pages, HK, ps, D), table=table, cu=cu, lens=np.array(tot, np.int32), ps=ps)


def check(moe, p, *, scale=None, causal=True, window=0, sinks=0, max_q=None, max_kv=None, label="", cache=None, out=None):
    D = p["q"].shape[2]
    s = D ** -0.5 if scale is None else scale
    n = np.diff(p["cu"])
    cache = to_device(moe, p["hc"]) if cache is None else cache
    got = moe.attention(bf16(p["q"]), cache, dev(p["table"]), dev(p["cu"]), dev(p["lens"]),
                        max_q=int(max(n.max(), 1)) if max_q is None else max_q,
                        max_kv=int(max(p["lens"].max(), 1)) if max_kv is None else max_kv,
                        scale=scale, causal=causal, window=window, sinks=sinks, out=out)
    torch.cuda.synchronize()
    want, bound = ref.attention(p["q"], p["hc"].kx, p["hc"].vx, p["table"], p["cu"], p["lens"], p["ps"], scale=float(np.float32(s)),
                                causal=causal, window=window, sinks=sinks)
    g = host(got)
    rows = ~np.isnan(want).all((1, 2))
    over = np.abs(g - want)[rows] > bound[rows]
    assert not over.any() and np.isfinite(g[rows]).all(), (label, over.sum(), np.abs(g - want)[rows].max())
    return got, want, bound


CASES = [
    # D, kv_heads, G, page, new, tot, causal, window, sinks
    (128, 1, 1, 16, [1], [1], True, 0, 0),
    (64, 1, 1, 16, [1], [1], True, 0, 0),
    (128, 2, 4, 64, [1], [77], True, 0, 0),
    (64, 2, 3, 32, [1, 1, 1], [31, 32, 33], True, 0, 0),
    (128, 2, 4, 16, [8, 8], [8, 200], True, 0, 0),
    (128, 1, 8, 128, [9], [1500], True, 0, 0),                     # 72 rows, several workgroups along the keys
    (64, 1, 16, 16, [5, 1, 7], [900, 17, 333], True, 0, 0),
    (128, 8, 6, 32, [1] * 5, [5, 64, 1000, 127, 2], True, 0, 0),
    (128, 1, 5, 256, [3, 0, 4], [700, 50, 4], True, 0, 0),         # a sequence without rows
    (64, 2, 2, 64, [70], [70], True, 0, 0),                        # a prompt
    (128, 2, 4, 64, [100, 37], [300, 37], True, 0, 0),
    (128, 1, 7, 16, [8, 8, 8], [40, 400, 8], False, 0, 0),         # a block whose rows see each other
    (64, 4, 8, 16, [8, 8], [1200, 90], False, 100, 4),
    (128, 2, 2, 32, [1, 8], [600, 601], True, 1, 0),               # a window of one key
    (128, 2, 2, 32, [1, 8], [600, 601], True, 33, 1),
    (64, 2, 4, 64, [64, 9], [500, 800], True, 50, 40),             # sinks past a tile
    (128, 1, 4, 16, [90], [90], True, 20, 16),
    (128, 1, 2, 64, [6], [2000], True, 5000, 7),                   # a window longer than the context
    (64, 1, 1, 128, [300], [1000], True, 0, 0),
]


@pytest.mark.parametrize("fp4", [False, True], ids=["bf16", "mxfp4"])
@pytest.mark.parametrize("D,HK,G,ps,new,tot,causal,window,sinks", CASES)
def test_attention_matches_reference(fp4, D, HK, G, ps, new, tot, causal, window, sinks):
    moe = _moe()
    rng = np.random.default_rng(5000 + D + HK * G + sum(tot) + window)
    check(moe, problem(rng, fp4, D, HK, G, ps, new, tot), causal=causal, window=window, sinks=sinks)


@pytest.mark.parametrize("fp4", [False, True], ids=["bf16", "mxfp4"])
def test_long_context_shared_by_many_workgroups(fp4):
    moe = _moe()
    rng = np.random.default_rng(5100)
    p = problem(rng, fp4, 128, 1, 4, 64, [2, 1], [20011, 4097])
    check(moe, p)
    check(moe, p, window=9000, sinks=3)


@pytest.mark.parametrize("fp4", [False, True], ids=["bf16", "mxfp4"])
def test_hints_do_not_change_what_is_computed(fp4):
    """max_q and max_kv far too small and far too large."""
    moe = _moe()
    rng = np.random.default_rng(5200)
    p = problem(rng, fp4, 64, 2, 3, 16, [40, 3], [700, 1300])
    for mq, mk in ((1, 1), (1, 5000), (1000, 1), (100000, 2 ** 31 - 1), (2 ** 31 - 1, 900)):
        check(moe, p, max_q=mq, max_kv=mk, label=(mq, mk))
        check(moe, p, max_q=mq, max_kv=mk, window=90, sinks=5, label=(mq, mk, "window"))


@pytest.mark.parametrize("fp4", [False, True], ids=["bf16", "mxfp4"])
def test_rows_without_keys_and_rows_of_nobody(fp4):
    """Refused requests (kv 0), more rows than cached tokens, and rows behind the last sequence."""
    moe = _moe()
    rng = np.random.default_rng(5300)
    p = problem(rng, fp4, 128, 2, 2, 16, [3, 5, 2], [0, 3, 40], extra_rows=4)
    for causal in (True, False):
        out = torch.full(p["q"].shape, 7.0, dtype=torch.bfloat16, device="cuda")
        got, want, _ = check(moe, p, causal=causal, out=out)
        g = host(got)
        assert (g[:3] == 0).all() and (g[3:5] == 0).all() and (g[10:] == 7.0).all()
    # all sequences empty
    p["lens"][:] = 0
    got, _, _ = check(moe, p, out=out)
    assert (host(got)[:10] == 0).all() and (host(got)[10:] == 7.0).all()


@pytest.mark.parametrize("fp4", [False, True], ids=["bf16", "mxfp4"])
def test_pages_outside_the_cache_are_not_seen(fp4):
    moe = _moe()
    rng = np.random.default_rng(5400)
    p = problem(rng, fp4, 64, 1, 4, 16, [4, 1], [200, 90])
    t = p["table"]
    t[0, 2], t[0, 5], t[0, 7], t[1, 0] = -1, p["hc"].kx.shape[0], 2 ** 31 - 1, -2 ** 31
    check(moe, p)
    t[1, :] = -9                                     # nothing left at all
    got, _, _ = check(moe, p)
    assert (host(got)[4] == 0).all()


@pytest.mark.parametrize("fp4", [False, True], ids=["bf16", "mxfp4"])
@pytest.mark.parametrize("value", [np.nan, np.inf, -np.inf])
def test_what_is_not_visible_has_no_influence(fp4, value):
    """NaN and infinities behind the last token, before the window and in later rows of the block: those
    rows that do not see them are as if they were not there, those that do see them are not finite."""
    moe = _moe()
    rng = np.random.default_rng(5500)
    D, ps = 128, 16
    p = problem(rng, fp4, D, 2, 2, ps, [6], [310])
    hc = p["hc"]
    def poison(key, row_too=True):
        page, r = p["table"][0][key // ps], key % ps
        if not fp4:
            bits = (np.array([value], np.float32).view(np.uint32) >> 16).astype(np.uint16)[0]
            hc.k[page, :, r], hc.v[page, :, r] = bits, bits
        else:                                        # the scale byte for NaN; the largest one overflows to infinity
            s, sv = hc.k_scale, ref.v_unpack(hc.v, hc.v_scale)
            byte = 255 if np.isnan(value) else 254
            s[page, :, r] = byte
            hc.k[page, :, r] = 0x77 if value > 0 else 0xFF
            sv[0][page, :, r] = 0x77 if not value < 0 else 0xFF
            sv[1][page, :, r] = byte
            hc.v[...], hc.v_scale[...] = ref.v_pack(*sv)
    # behind the last token (page rows never written), all of them
    for key in range(310, 320):
        poison(key)
    check(moe, p)
    # before the window
    poison(100)
    poison(310 - 6 - 50)
    check(moe, p, window=50, sinks=4)
    # the block's fourth row: the first three are unharmed
    poison(307)
    want, bound = ref.attention(p["q"][:3], hc.kx, hc.vx, p["table"], [0, 3], [307], ps, scale=float(np.float32(D ** -0.5)),
                                causal=True, window=50, sinks=4)
    got = host(moe.attention(bf16(p["q"]), to_device(moe, hc), dev(p["table"]), dev(p["cu"]), dev(p["lens"]), max_q=6, max_kv=310,
                             window=50, sinks=4))
    assert (np.abs(got[:3] - want) <= bound).all()
    assert not np.isfinite(got[3:]).all(-1).any()


def test_visible_nan_and_large_scores():
    """A visible NaN makes its rows NaN; scores of very different size do not overflow the softmax."""
    moe = _moe()
    rng = np.random.default_rng(5600)
    p = problem(rng, False, 128, 1, 2, 16, [2], [500])
    p["q"] *= 64.0
    p["q"] = ref.bf16_round(p["q"])
    check(moe, p, scale=4.0)                         # scores of thousands
    check(moe, p, scale=1e-4)
    page = p["table"][0][3]
    p["hc"].k[page, 0, 1, 5] = 0x7FC0
    got = host(moe.attention(bf16(p["q"]), to_device(moe, p["hc"]), dev(p["table"]), dev(p["cu"]), dev(p["lens"]), max_q=2, max_kv=500))
    assert np.isnan(got).all()


def test_strides_streams_workspace_and_determinism():
    moe = _moe()
    rng = np.random.default_rng(5700)
    p = problem(rng, True, 128, 2, 4, 64, [8, 8, 8], [3000, 5000, 700])
    T, H, D = p["q"].shape
    cache = to_device(moe, p["hc"])
    args = (cache, dev(p["table"]), dev(p["cu"]), dev(p["lens"]))
    want, _, _ = check(moe, p, cache=cache)
    # queries and outputs inside wider rows
    wide = torch.full((T, (H + 5) * D), 3.0, dtype=torch.bfloat16, device="cuda")
    wide[:, D:(H + 1) * D] = bf16(p["q"]).flatten(1)
    o = torch.full((T, (H + 2) * D), 9.0, dtype=torch.bfloat16, device="cuda")
    moe.attention(wide[:, D:(H + 1) * D].unflatten(1, (H, D)), *args, max_q=8, max_kv=5000, out=o[:, D:(H + 1) * D].unflatten(1, (H, D)))
    assert torch.equal(o[:, D:(H + 1) * D].unflatten(1, (H, D)), want) and (o[:, :D] == 9).all() and (o[:, (H + 1) * D:] == 9).all()
    # on a side stream behind other work, with a caller's workspace full of NaN; again and again the same bits
    ws = torch.full((moe.attention_workspace_bytes(cache, T, H, 3, max_q=8, max_kv=5000),), 0xFF, dtype=torch.uint8, device="cuda")
    assert ws.numel() > 0
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    qd = bf16(p["q"])
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        got = moe.attention(qd, *args, max_q=8, max_kv=5000, workspace=ws, stream=side)
        side.synchronize()
        assert torch.equal(got, want)
    with pytest.raises(moe.MoeError):
        moe.attention(qd, *args, max_q=8, max_kv=5000, workspace=ws[:-1])


def test_attention_replays_from_a_hip_graph():
    """One graph, captured once, serves steps of other lengths and contents."""
    moe = _moe()
    rng = np.random.default_rng(5800)
    B, HK, G, D, ps = 3, 2, 4, 64, 16
    first = problem(rng, True, D, HK, G, ps, [8] * B, [400, 300, 200])
    W, T = first["table"].shape[1], 8 * B
    cache = moe.KvCache(first["hc"].kx.shape[0], ps, HK, D)
    q, table = torch.zeros((T, HK * G, D), dtype=torch.bfloat16, device="cuda"), dev(first["table"])
    cu, lens = dev(first["cu"]), dev(first["lens"])
    out = torch.zeros_like(q)
    ws = torch.empty(moe.attention_workspace_bytes(cache, T, HK * G, B, max_q=8, max_kv=400), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.attention(q, cache, table, cu, lens, max_q=8, max_kv=400, out=out, workspace=ws)
    for i, tot in enumerate(([400, 300, 200], [8, 399, 30], [120, 64, 401])):
        p = problem(rng, True, D, HK, G, ps, [8] * B, tot)
        need = p["table"].shape[1]
        assert p["table"].max() < cache.num_pages
        full = ref.host_cache(rng, True, cache.num_pages, HK, ps, D)
        p["hc"] = full
        tab = np.full((B, W), -1, np.int32)
        tab[:, :min(W, need)] = p["table"][:, :W]
        p["table"] = tab
        for t, x in ((cache.k, full.k), (cache.v, full.v), (cache.k_scale, full.k_scale), (cache.v_scale, full.v_scale), (table, tab),
                     (cu, p["cu"]), (lens, p["lens"])):
            t.copy_(dev(x))
        q.copy_(bf16(p["q"]))
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        eager, want, bound = check(moe, p, cache=cache, max_q=8, max_kv=400)
        assert torch.equal(out, eager), i


def test_cache_past_four_gigabytes():
    """Keys in pages whose bytes lie past 2^32 of the buffers."""
    moe = _moe()
    rng = np.random.default_rng(5900)
    D, HK, ps, pages = 128, 8, 64, 40000
    p = problem(rng, False, D, HK, 2, ps, [3], [150])
    small = p["hc"]
    k, v = (torch.zeros((pages, HK, ps, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    at = np.array([39999, 35000, 33001, 12, 34567], np.int32)[:small.kx.shape[0]]
    for dst, src in ((k, small.k), (v, small.v)):
        dst[torch.from_numpy(at.astype(np.int64)).cuda()] = dev(src.view(np.int16)).view(torch.bfloat16)
    cache = moe.KvCache.wrap(k, v)
    q = dict(p, table=np.where(p["table"] >= 0, at[np.maximum(p["table"], 0)], -1).astype(np.int32))
    want, bound = ref.attention(p["q"], small.kx, small.vx, p["table"], p["cu"], p["lens"], ps, scale=float(np.float32(D ** -0.5)),
                                causal=True, window=0, sinks=0)
    got = host(moe.attention(bf16(p["q"]), cache, dev(q["table"]), dev(p["cu"]), dev(p["lens"]), max_q=3, max_kv=150))
    assert (np.abs(got - want) <= bound).all()


@pytest.mark.parametrize("fp4", [False, True], ids=["bf16", "mxfp4"])
def test_verify_steps_end_to_end(fp4):
    """Plan, norms and cache write, attention, expert layer and acceptance as a verify loop runs them: prompts,
    then drafted blocks with rollbacks, every attention output against the 64-bit form of the whole history."""
    moe = _moe()
    rng = np.random.default_rng(6000)
    B, HK, G, D, ps, W, N = 3, 1, 2, 128, 16, 12, 40
    H, block = HK * G, 4
    w = synth.Workload("step", 64, H * D, 256, 8, 2, "bf16", "none", 6001)
    layer = moe.MoeMxfp4(problems.to_device(problems.pack_experts(w)), w.E, w.d, w.f, w.k, max_tokens=128)
    router = torch.from_numpy(synth.router_weights_bf16(w).view(np.int16)).cuda().view(torch.bfloat16)
    cache = moe.KvCache(N, ps, HK, D, fmt=moe.KV_MXFP4 if fp4 else moe.KV_BF16)
    freq = 10000.0 ** (-np.arange(D // 2) * 2.0 / D)
    wq, wk = ref.bf16_round(1 + 0.1 * rng.standard_normal((2, D)))
    i32 = dict(dtype=torch.int32, device="cuda")
    table, ring = torch.full((B, W), -1, **i32), torch.arange(N, **i32)
    held, held2 = torch.zeros(B, **i32), torch.zeros(B, **i32)
    state, state2 = torch.tensor([0, N], **i32), torch.zeros(2, **i32)
    ctx = np.zeros(B, np.int64)
    hist = [dict(k=np.zeros((0, HK, D)), v=np.zeros((0, HK, D))) for _ in range(B)]
    for step, new in enumerate(([20, 33, 7], [block] * 3, [block, 0, block], [block] * 3)):
        T = sum(new)
        plan = moe.cache_plan(dev(ctx.astype(np.int32)), torch.tensor(new, **i32), table, held, ring, state, page_size=ps,
                              num_tokens=T, held_out=held2, free_out=state2)
        held, held2, state, state2 = held2, held, state2, state
        x = ref.bf16_round(rng.standard_normal((T, (H + 2 * HK) * D)))
        xt = bf16(x)
        qt, kt, vt = xt[:, :H * D].unflatten(1, (H, D)), xt[:, H * D:(H + HK) * D].unflatten(1, (HK, D)), xt[:, (H + HK) * D:].unflatten(1, (HK, D))
        q, _ = moe.qk_norm_rope(qt, kt, vt, plan.positions, dev(freq), q_weight=bf16(wq), k_weight=bf16(wk), cache=cache, slots=plan.slots)
        a = moe.attention(q, cache, table, plan.cu_q, plan.kv_lens, max_q=max(new), max_kv=W * ps)
        y = layer(a.flatten(1), None, w_router=router)
        torch.cuda.synchronize()
        assert int(plan.refused.cpu()) == 0 and torch.isfinite(y).all()
        # the history as the cache should hold it: what kv_read gives for the new slots
        rk, rv = (host(t) for t in moe.kv_read(cache, plan.slots))
        at = 0
        for b, n in enumerate(new):
            h = hist[b]
            h["k"], h["v"] = np.concatenate([h["k"][:ctx[b]], rk[at:at + n]]), np.concatenate([h["v"][:ctx[b]], rv[at:at + n]])
            wantk, _ = ref.norm_rope(x[at:at + n, H * D:(H + HK) * D].reshape(n, HK, D), wk, ctx[b] + np.arange(n), freq, 1e-6, False)
            if n:                                    # 4 bits: at most a quarter of the block's largest; bf16: its rounding
                err = np.abs(rk[at:at + n] - wantk)
                assert (err <= (0.26 * np.abs(wantk).max() if fp4 else 2.0 ** -7 * np.abs(wantk) + 1e-5)).all()
            if n:
                pad = -(-len(h["k"]) // ps) * ps
                kk, vv = (np.pad(t, ((0, pad - len(t)), (0, 0), (0, 0))).reshape(-1, ps, HK, D).transpose(0, 2, 1, 3) for t in (h["k"], h["v"]))
                want, bound = ref.attention(host(q)[at:at + n], kk, vv, np.arange(len(kk))[None], [0, n], [len(h["k"])], ps,
                                            scale=float(np.float32(D ** -0.5)), causal=True, window=0, sinks=0)
                assert (np.abs(host(a)[at:at + n] - want) <= bound).all(), (step, b)
            at += n
            ctx[b] += n
        if step:                                     # acceptance: rows past the accepted ones are rolled back
            d = synth.dflash_batch(B, block, 500, seed=6100 + step, eps=1.0)
            acc, _ = moe.dflash_accept(*[dev(d[n]) for n in ("draft", "p_draft", "p_target", "u", "r")])
            acc = acc.cpu().numpy()
            ctx -= np.where(np.array(new) > 0, block - np.maximum(acc, 1), 0)
