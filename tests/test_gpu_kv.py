"""GPU parity of the paged cache: its plan (exact), the norms and rotation that
write it, and its read-back, against the 64-bit forms in kv_reference."""
import numpy as np
import pytest

import oracle
from tests import kv_reference as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

PLAN_KEYS = ("cu_q", "kv_lens", "slots", "positions", "refused")


def _moe():
    import mxfp4_expert_ffn_amd as moe
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible")
    return moe


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def bf16(x):
    """float array -> bf16 CUDA tensor."""
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).cuda().bfloat16()


def host(t):
    return t.double().cpu().numpy()


# ------------------------------------------------------------------ plan

def _plan_case(rng, B, W, ps, N, T=None, faults=False, new_max=None):
    """A consistent state (pages of the requests and the ring are distinct) and lengths."""
    order = rng.permutation(N).astype(np.int32)
    held = np.minimum(rng.integers(0, W + 1, B), max(0, N // max(B, 1))).astype(np.int32)
    table = np.full((B, W), -1, np.int32)
    at = 0
    for b in range(B):
        table[b, :held[b]] = order[at:at + held[b]]
        at += held[b]
    head = int(rng.integers(0, N))
    ring = np.full(N, -5, np.int32)
    ring[(head + np.arange(N - at)) % N] = order[at:]
    ctx = (held * ps * rng.random(B)).astype(np.int32)
    new = rng.integers(0, (new_max or 2 * ps) + 1, B).astype(np.int32)
    new[rng.random(B) < 0.15] = -1
    if faults:
        for what in range(5):
            b = int(rng.integers(0, B))
            if what == 0:
                ctx[b] = -3
            elif what == 1:
                new[b] = -2
            elif what == 2:
                ctx[b] = W * ps
            elif what == 3:
                held[b] = W + 1
            else:
                table[b, 0] = N + 7
    total = int(np.maximum(new, 0).sum())
    return dict(ctx=ctx, new=new, table=table, held=held, ring=ring, state=np.array([head, N - at], np.int32), ps=ps,
                T=total + int(rng.integers(0, 5)) if T is None else T)


def _run_plan(moe, c):
    table, ring = dev(c["table"]), dev(c["ring"])
    r = moe.cache_plan(dev(c["ctx"]), dev(c["new"]), table, dev(c["held"]), ring, dev(c["state"]), page_size=c["ps"],
                       num_tokens=c["T"])
    torch.cuda.synchronize()
    return dict(table=table.cpu().numpy(), ring=ring.cpu().numpy(), **{n: t.cpu().numpy() for n, t in r._asdict().items()})


def _check_plan(moe, c, label):
    got, want = _run_plan(moe, c), ref.plan(c["ctx"], c["new"], c["table"], c["held"], c["ring"], c["state"], c["ps"], c["T"])
    for n, w in want.items():
        assert np.array_equal(got[n], w), (label, n, np.nonzero(got[n] != w)[0][:8])


@pytest.mark.parametrize("B,W,ps,N,faults", [
    (1, 1, 16, 1, False), (1, 64, 64, 100, False), (3, 5, 128, 40, True), (32, 130, 64, 5000, False), (63, 9, 16, 600, True),
    (64, 4, 256, 300, False), (257, 40, 32, 9000, True), (1025, 3, 16, 4000, False), (4096, 17, 32, 50000, True),
])
def test_plan_matches_reference(B, W, ps, N, faults):
    moe = _moe()
    rng = np.random.default_rng(3000 + B + W)
    for k in range(3):
        _check_plan(moe, _plan_case(rng, B, W, ps, N, faults=faults), (B, W, ps, N, k))


def test_plan_edges():
    moe = _moe()
    rng = np.random.default_rng(3100)
    base = _plan_case(rng, 20, 8, 16, 200)
    # too few free pages: in order, the first requests get theirs
    short = dict(base, state=np.array([base["state"][0], 7], np.int32))
    _check_plan(moe, short, "short")
    _check_plan(moe, dict(base, state=np.array([base["state"][0], 0], np.int32)), "none free")
    # rows that do not fit, none at all, and far fewer requests' rows than rows
    total = int(np.maximum(base["new"], 0).sum())
    for T in (0, 1, 3, total - 1, total, total + 1000):
        _check_plan(moe, dict(base, T=T), ("rows", T))
    # a state outside the ring offers nothing
    for state in ([-1, 5], [200, 5], [3, -1], [3, 201], [2 ** 31 - 1, 2 ** 31 - 1]):
        _check_plan(moe, dict(base, state=np.array(state, np.int32)), ("state", state))
    # lengths at the ends of int32
    wild = dict(base, ctx=base["ctx"].copy(), new=base["new"].copy())
    wild["ctx"][3], wild["new"][5], wild["ctx"][7], wild["new"][7], wild["new"][9] = 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1, -2 ** 31
    _check_plan(moe, dict(wild, T=64), "wild")
    # every request ends; every request idles
    _check_plan(moe, dict(base, new=np.full(20, -1, np.int32), T=4), "all end")
    _check_plan(moe, dict(base, new=np.zeros(20, np.int32), T=0), "idle")
    # no requests: the rows are all marked
    none = dict(base, ctx=base["ctx"][:0], new=base["new"][:0], held=base["held"][:0], table=base["table"][:0], T=9)
    _check_plan(moe, none, "no requests")
    # long prompts
    _check_plan(moe, _plan_case(rng, 40, 700, 16, 30000, new_max=5000), "prompts")


def test_plan_repeats_and_replays_from_a_graph():
    """The call repeated on the same inputs, eagerly and from a graph, repeats its result; a replay sees new lengths."""
    moe = _moe()
    rng = np.random.default_rng(3200)
    B, W, ps, N, T = 17, 10, 16, 400, 200
    c = _plan_case(rng, B, W, ps, N, T=T, new_max=11)
    t = {n: dev(c[n]) for n in ("ctx", "new", "table", "held", "ring", "state")}
    call = lambda out=None: moe.cache_plan(t["ctx"], t["new"], t["table"], t["held"], t["ring"], t["state"],  # noqa: E731
                                           page_size=ps, num_tokens=T, out=out)
    out = call()
    want = {n: x.clone() for n, x in out._asdict().items()}
    call(out)
    assert all(torch.equal(want[n], x) for n, x in out._asdict().items())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        call(out)
    for i in range(3):
        d = _plan_case(rng, B, W, ps, N, T=T, new_max=11)
        for n in t:
            t[n].copy_(dev(d[n]))
        g.replay()
        torch.cuda.synchronize()
        w = ref.plan(d["ctx"], d["new"], d["table"], d["held"], d["ring"], d["state"], ps, T)
        got = dict(table=t["table"], ring=t["ring"], **out._asdict())
        for n in w:
            assert np.array_equal(got[n].cpu().numpy(), w[n]), (i, n)


# ------------------------------------------------------------------ norms, rotation, cache write

def _between(got, lo, hi):
    return (got >= lo) & (got <= hi)


def _check_fp4_key(got, codes_scale, want, tol, label):
    """Each block is a quantisation of something within tol of want: its scale byte is one that the
    largest magnitude, within tol, can have, and its elements lie between the roundings of want -+ tol."""
    T, H, D = want.shape
    w, t, x = (a.reshape(T, H, D // 32, 32) for a in (want, tol, got))
    s = codes_scale.astype(np.int64) - 127
    top_lo, top_hi = (np.abs(w) - t).max(-1), (np.abs(w) + t).max(-1)
    e = lambda a: np.where(a > 0, np.floor(np.log2(np.maximum(a, 1e-300))), -125).clip(-125, 129) - 2  # noqa: E731
    assert (_between(s, e(top_lo), e(top_hi))).all(), label
    scale = np.exp2(s.astype(np.float64))[..., None]

    def rnd(a):                                     # nearest of the grid, either way at a tie
        m = np.minimum(np.abs(a) / scale, 6.0)
        grid = ref.E2M1
        d = np.abs(m[..., None] - grid)
        return np.sign(a) * grid[d.argmin(-1)] * scale
    eps = 1e-9 * scale
    assert _between(x, rnd(w - t - eps), rnd(w + t + eps)).all(), label


ROPE_CASES = [
    # T, heads, kv_heads, D, rot, interleaved, fp4 (None: no cache), page, norms, far
    (1, 1, 1, 64, 64, False, True, 16, True, False),
    (1, 32, 8, 128, 128, False, True, 64, True, True),
    (3, 5, 1, 128, 16, True, True, 16, True, False),
    (7, 48, 8, 128, 96, False, False, 32, True, True),
    (9, 3, 3, 64, 48, True, True, 128, False, True),
    (37, 16, 2, 64, 32, False, True, 64, True, False),
    (5, 8, 8, 128, 0, False, True, 16, False, False),
    (64, 7, 7, 64, 64, False, False, 256, True, False),
    (300, 32, 8, 128, 128, True, True, 64, True, True),
    (11, 4, 2, 128, 128, False, None, 16, True, True),
    (4, 33, 11, 64, 16, False, None, 16, False, False),
]


@pytest.mark.parametrize("T,H,HK,D,rot,inter,fp4,ps,norms,far", ROPE_CASES)
def test_rope_matches_reference(T, H, HK, D, rot, inter, fp4, ps, norms, far):
    """q_out: 2^-8 of the value for its rounding, and 2^-19 (|a| + |b|) of its pair: the norm's factor and
    product are within 2^-20 relatively (a sum of up to 16 partial steps, a root, a division, two products: 12 x 2^-24), cos
    and sin within 2^-21 (the turn's fraction is off by 2^-25 of a turn, 2^-22.3 radians, and the function by
    2^-22), the two products and the sum by 3 x 2^-24."""
    moe = _moe()
    rng = np.random.default_rng(4000 + T * 7 + H + D + rot)
    width = (H + 2 * HK) * D
    proj = ref.bf16_round(rng.standard_normal((T, width + 8)) * np.exp(rng.standard_normal((T, 1))))
    pt = bf16(proj)[:, :width]                       # rows at a stride of their own
    q, k, v = (x.reshape(T, -1, D) for x in np.split(proj[:, :width], [H * D, (H + HK) * D], 1))
    qt, kt, vt = pt[:, :H * D].unflatten(1, (H, D)), pt[:, H * D:(H + HK) * D].unflatten(1, (HK, D)), pt[:, (H + HK) * D:].unflatten(1, (HK, D))
    pos = rng.integers(0, 1_000_000 if far else 4096, T).astype(np.int32)
    if T > 4:
        pos[T // 2] = -1                             # a row that no request has
    freq = 10000.0 ** (-np.arange(rot // 2) * 2.0 / max(rot, 1))
    wq, wk = (ref.bf16_round(1 + 0.2 * rng.standard_normal(D)) if norms else None for _ in range(2))
    pages = T // ps + 3
    cache = hc = slots = None
    if fp4 is not None:
        hc = ref.host_cache(rng, fp4, pages, HK, ps, D)
        bufs = [dev(x.view(np.int16)).view(torch.bfloat16) if x.dtype == np.uint16 else dev(x) for x in (hc.k, hc.v)]
        cache = moe.KvCache.wrap(*bufs, *([dev(hc.k_scale), dev(hc.v_scale)] if fp4 else []))
        slots = rng.permutation(pages * ps)[:T].astype(np.int32)
        if T > 6:
            slots[0], slots[1] = -1, pages * ps      # outside the cache: not written
    qo = torch.full((T, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
    ko = torch.full((T, HK, D), 7.0, dtype=torch.bfloat16, device="cuda")
    args = dict(q_weight=None if wq is None else bf16(wq), k_weight=None if wk is None else bf16(wk), eps=1e-5, interleaved=inter)
    moe.qk_norm_rope(qt, kt, vt, dev(pos), dev(freq), cache=cache, slots=None if slots is None else dev(slots), q_out=qo,
                     k_out=ko, **args)
    torch.cuda.synchronize()
    live = pos >= 0
    for got, x, w in ((host(qo), q, wq), (host(ko), k, wk)):
        want, size = ref.norm_rope(x, w, pos, freq, 1e-5, inter)
        tol = 2.0 ** -8 * np.abs(want) + 2.0 ** -19 * size + 2.0 ** -133
        assert (np.abs(got - want) <= tol)[live].all(), np.abs(got - want)[live].max()
        assert (got[~live] == 7.0).all()             # left as it was
    if fp4 is None:
        return
    # the whole cache: written slots hold the new rows, every other byte is what it was
    if fp4:
        kc, ks, (vc, vs) = cache.k.cpu().numpy(), cache.k_scale.cpu().numpy(), ref.v_unpack(cache.v.cpu().numpy(), cache.v_scale.cpu().numpy())
        oc, (ovc, ovs) = (hc.k, hc.k_scale), ref.v_unpack(hc.v, hc.v_scale)
        new = [kc.transpose(0, 2, 1, 3).reshape(pages * ps, HK, -1), ks.transpose(0, 2, 1, 3).reshape(pages * ps, HK, -1),
               vc.transpose(0, 2, 1, 3).reshape(pages * ps, HK, -1), vs.transpose(0, 2, 1, 3).reshape(pages * ps, HK, -1)]
        old = [x.transpose(0, 2, 1, 3).reshape(pages * ps, HK, -1) for x in (*oc, ovc, ovs)]
    else:
        new = [x.view(torch.int16).cpu().numpy().transpose(0, 2, 1, 3).reshape(pages * ps, HK, D) for x in (cache.k, cache.v)]
        old = [x.view(np.int16).transpose(0, 2, 1, 3).reshape(pages * ps, HK, D) for x in (hc.k, hc.v)]
    put = live & (slots >= 0) & (slots < pages * ps)
    rest = np.ones(pages * ps, bool)
    rest[slots[put]] = False
    assert all(np.array_equal(n[rest], o[rest]) for n, o in zip(new, old))
    at = slots[put]
    want, size = ref.norm_rope(k, wk, pos, freq, 1e-5, inter)
    want, size = want[put], size[put]
    rk, rv = moe.kv_read(cache, dev(slots))
    rk, rv = host(rk), host(rv)
    outside = (slots < 0) | (slots >= pages * ps)
    assert (rk[outside] == 0).all() and (rv[outside] == 0).all()
    if fp4:
        qc, qs = ref.quantise(v[put])                # values are quantised as they are
        assert np.array_equal(new[2][at], qc) and np.array_equal(new[3][at], qs)
        got = ref.values(new[0][at], new[1][at])
        _check_fp4_key(got, new[1][at], want, 2.0 ** -19 * size, "key")
        if wk is None and rot == 0:                  # nothing computed: exact
            qc, qs = ref.quantise(k[put])
            assert np.array_equal(new[0][at], qc) and np.array_equal(new[1][at], qs)
        assert np.array_equal(rk[put], got) and np.array_equal(rv[put], ref.values(new[2][at], new[3][at]))
    else:
        assert np.array_equal(rk[put], host(ko)[put]) and np.array_equal(rv[put], v[put])


def test_rope_in_place_other_stream_and_device_state():
    moe = _moe()
    rng = np.random.default_rng(4100)
    T, H, HK, D = 6, 8, 2, 128
    q, k = bf16(rng.standard_normal((T, H, D))), bf16(rng.standard_normal((T, HK, D)))
    pos, freq = dev(np.arange(T, dtype=np.int32)), dev(10000.0 ** (-np.arange(64) / 64.0))
    w = bf16(np.ones(D))
    want = moe.qk_norm_rope(q, k, None, pos, freq, q_weight=w, k_weight=w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = moe.qk_norm_rope(q, k, None, pos, freq, q_weight=w, k_weight=w, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    moe.qk_norm_rope(q, k, None, pos, freq, q_weight=w, k_weight=w, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])


def test_cache_write_of_wild_values():
    """Infinities and NaN: their block reads as NaN, the row's other blocks as themselves; zeros keep their sign;
    subnormal and largest magnitudes take the smallest and largest scales."""
    moe = _moe()
    D, HK, ps = 128, 1, 16
    x = np.zeros((6, HK, D), np.float32)
    x[0, 0, 3] = np.inf
    x[1, 0, 40] = np.nan
    x[2, 0, 100] = -np.inf
    x[3, 0, :] = 2.0 ** -133
    x[4, 0, :] = 3.0e38
    x[5, 0, ::2] = -0.0
    x[:3, 0, 70] = 1.5
    t = torch.from_numpy(x).cuda().bfloat16()
    cache = moe.KvCache(1, ps, HK, D)
    zero = torch.zeros(0, dtype=torch.float64, device="cuda")
    pos = torch.zeros(6, dtype=torch.int32, device="cuda")
    slots = torch.arange(6, dtype=torch.int32, device="cuda")
    qo, _ = moe.qk_norm_rope(t, t, t, pos, zero, cache=cache, slots=slots)
    assert torch.equal(qo.view(torch.int16), t.view(torch.int16))
    k, v = moe.kv_read(cache, slots)
    assert torch.equal(k.view(torch.int16), v.view(torch.int16))
    k = host(k)[:, 0].reshape(6, 4, 32)
    for r, blk in ((0, 0), (1, 1), (2, 3)):
        bad = np.isnan(k[r]).all(-1)
        assert bad[blk] and bad.sum() == 1 and k[r, 2, 6] == 1.5
    want = host(t)[3:, 0]
    qc, qs = ref.quantise(want)
    assert np.array_equal(k[3:].reshape(3, D), ref.values(qc, qs).astype(np.float64))
    vc, vs = ref.v_unpack(cache.v.cpu().numpy(), cache.v_scale.cpu().numpy())
    assert np.array_equal(vc[0, 0, 3:6], qc) and np.array_equal(vs[0, 0, 3:6], qs)


def test_cache_past_four_gigabytes():
    """Slots whose bytes lie past 2^32 of the buffers."""
    moe = _moe()
    D, HK, ps, pages = 128, 8, 64, 40000            # 5.2 GB of bf16 each
    k, v = (torch.empty((pages, HK, ps, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    cache = moe.KvCache.wrap(k, v)
    rng = np.random.default_rng(4300)
    x = bf16(rng.standard_normal((4, HK, D)))
    slots = dev(np.array([pages * ps - 1, pages * ps - 64, 33000 * ps + 5, 17], np.int32))
    zero, pos = torch.zeros(0, dtype=torch.float64, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
    moe.qk_norm_rope(x, x, x, pos, zero, cache=cache, slots=slots)
    rk, rv = moe.kv_read(cache, slots)
    assert torch.equal(rk, x) and torch.equal(rv, x)
    assert torch.equal(k[pages - 1, :, ps - 1], x[0]) and torch.equal(k[33000, :, 5], x[2])
