"""GPU parity of attention where there are many rows or many sequences: sets of
rows whose waves share each tile of keys, whole or in pieces, against the
64-bit reference and its bound (kv_reference.attention)."""
import numpy as np
import pytest

from tests import kv_reference as ref
from tests.test_gpu_attention import bf16, check, dev, host, problem, to_device

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def _moe():
    import mxfp4_expert_ffn_amd as moe
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible")
    return moe


SETS = [
    # kv_heads, G, page, new, tot, causal, window, sinks
    (1, 1, 16, [193], [193], True, 0, 0),                          # one row more than a set of 192
    (2, 5, 32, [150, 1, 0, 77], [500, 33, 20, 77], True, 0, 0),    # sets that end inside a token's heads
    (1, 3, 128, [260], [1900], True, 0, 0),                        # pieces
    (2, 6, 64, [100, 31], [1500, 1031], True, 700, 33),
    (1, 8, 16, [97], [640], True, 1, 0),                           # every tile cut twice by its rows
    (1, 4, 256, [300], [300], False, 0, 0),
    (4, 2, 16, [120, 40], [800, 2000], False, 90, 5),
    (1, 16, 64, [70, 9], [40, 9], True, 0, 0),                     # more rows than cached tokens
]


@pytest.mark.parametrize("fp4", [False, True], ids=["bf16", "mxfp4"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("HK,G,ps,new,tot,causal,window,sinks", SETS)
def test_many_rows_match_reference(fp4, D, HK, G, ps, new, tot, causal, window, sinks):
    moe = _moe()
    rng = np.random.default_rng(7000 + D + HK * G + sum(tot) + window)
    check(moe, problem(rng, fp4, D, HK, G, ps, new, tot), causal=causal, window=window, sinks=sinks)


@pytest.mark.parametrize("fp4", [False, True], ids=["bf16", "mxfp4"])
@pytest.mark.parametrize("D", [64, 128])
def test_scores_that_keep_growing(fp4, D):
    """Keys that score higher the later they stand, so that the reference moves again and again."""
    moe = _moe()
    rng = np.random.default_rng(7100 + D)
    p = problem(rng, fp4, D, 1, 2, 32, [120, 3], [700, 900])
    q = np.abs(p["q"]) * 0.25
    p["q"] = ref.bf16_round(q)
    where = {int(page): b * 100000 + i for b in range(2) for i, page in enumerate(p["table"][b]) if page >= 0}
    k = np.ones(p["hc"].kx.shape)
    for page, i in where.items():
        k[page] *= (i % 100000 + 1) * 0.5
    p["hc"] = ref.host_cache(rng, fp4, k.shape[0], 1, 32, D, k=k)
    check(moe, p)
    check(moe, p, window=200, sinks=20)


@pytest.mark.parametrize("fp4", [False, True], ids=["bf16", "mxfp4"])
@pytest.mark.parametrize("D", [64, 128])
def test_many_rows_and_pages_outside_the_cache(fp4, D):
    moe = _moe()
    rng = np.random.default_rng(7200 + D)
    for ps in (16, 64):
        p = problem(rng, fp4, D, 1, 4, ps, [60, 40], [700, 300])
        t = p["table"]
        t[0, 1], t[0, 4], t[0, 700 // ps], t[1, 0] = -1, p["hc"].kx.shape[0], -2 ** 31, 2 ** 31 - 1
        check(moe, p, label=ps)
        check(moe, p, window=150, sinks=30, label=(ps, "window"))
        t[1, :] = -1
        got, _, _ = check(moe, p, label=(ps, "none"))
        assert (host(got)[60:] == 0).all()


@pytest.mark.parametrize("fp4", [False, True], ids=["bf16", "mxfp4"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("value", [np.nan, np.inf])
def test_later_rows_values_do_not_reach_earlier_ones(fp4, D, value):
    """A prompt in which one token's value is not finite: the rows before it, and those whose window has
    passed it, are as if it were not there."""
    moe = _moe()
    rng = np.random.default_rng(7300 + D)
    n, ps, at, window = 130, 16, 75, 40
    p = problem(rng, fp4, D, 2, 2, ps, [n], [n])
    hc = p["hc"]
    page, r = p["table"][0][at // ps], at % ps
    clean = hc.vx.copy()
    if not fp4:
        hc.v[page, :, r] = 0x7FC0 if np.isnan(value) else 0x7F80
    else:
        codes, scales = ref.v_unpack(hc.v, hc.v_scale)
        codes[page, :, r], scales[page, :, r] = 0x77, 255 if np.isnan(value) else 254
        hc.v[...], hc.v_scale[...] = ref.v_pack(codes, scales)
    clean[page, :, r] = 0
    cache = to_device(moe, hc)
    for w in (0, window):
        got = host(moe.attention(bf16(p["q"]), cache, dev(p["table"]), dev(p["cu"]), dev(p["lens"]), max_q=n, max_kv=n, window=w))
        want, bound = ref.attention(p["q"], hc.kx, clean, p["table"], p["cu"], p["lens"], ps, scale=float(np.float32(D ** -0.5)),
                                    causal=True, window=w, sinks=0)
        blind = np.array([i < at or (w and i - w + 1 > at) for i in range(n)])
        assert (np.abs(got - want) <= bound)[blind].all(), w
        assert not np.isfinite(got[~blind]).any(), w


@pytest.mark.parametrize("B", [7, 1024, 1025])
def test_many_ragged_sequences(B):
    """Up to 1024 sequences are divided by their lengths, more one workgroup each."""
    moe = _moe()
    rng = np.random.default_rng(7400 + B)
    tot = rng.integers(1, 40, B)
    tot[rng.integers(0, B, 3)] = (600, 900, 1300)
    new = np.minimum(rng.integers(0, 3, B), tot)
    p = problem(rng, True, 64, 1, 2, 16, list(new), list(tot))
    check(moe, p, max_q=2, max_kv=1300)
    check(moe, p, max_q=2, max_kv=1300, window=64, sinks=2)


def test_sizes_drawn_at_random():
    moe = _moe()
    rng = np.random.default_rng(7500)
    for i in range(48):
        D, ps = int(rng.choice([64, 128])), int(rng.choice([16, 32, 64, 128, 256]))
        HK, G, B = int(rng.integers(1, 4)), int(rng.integers(1, 9)), int(rng.integers(1, 6))
        tot = np.exp(rng.uniform(0, 7.2, B)).astype(int)
        new = np.minimum(np.exp(rng.uniform(0, rng.choice([0.5, 2.5, 5.0]), B)).astype(int), tot)
        window = int(rng.choice([0, 0, 1, 31, 200]))
        sinks = int(rng.integers(0, 50)) if window else 0
        causal, fp4 = bool(rng.integers(0, 2)), bool(rng.integers(0, 2))
        label = (i, D, ps, HK, G, list(new), list(tot), window, sinks, causal, fp4)
        print(label, flush=True)
        check(moe, problem(rng, fp4, D, HK, G, ps, list(new), list(tot)), causal=causal, window=window, sinks=sinks, label=label)


def test_two_graphs_of_two_workspaces_and_eager_calls_between():
    """Calls in flight at once, each with its own workspace, on two streams."""
    moe = _moe()
    rng = np.random.default_rng(7600)
    ps = [problem(rng, True, 128, 2, 4, 32, new, tot) for new, tot in (([8, 8], [2500, 700]), ([90], [1700]))]
    runs = []
    for p in ps:
        n = int(np.diff(p["cu"]).max())
        T, H, _ = p["q"].shape
        cache = to_device(moe, p["hc"])
        r = dict(q=bf16(p["q"]), table=dev(p["table"]), cu=dev(p["cu"]), lens=dev(p["lens"]), cache=cache, n=n,
                 ws=torch.empty(max(moe.attention_workspace_bytes(cache, T, H, len(p["lens"]), max_q=n, max_kv=2500), 16),
                                dtype=torch.uint8, device="cuda"))
        r["out"] = torch.empty_like(r["q"])
        r["want"], _, _ = check(moe, p, max_kv=2500, cache=cache)
        r["graph"] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(r["graph"]):
            moe.attention(r["q"], cache, r["table"], r["cu"], r["lens"], max_q=n, max_kv=2500, out=r["out"], workspace=r["ws"])
        runs.append(r)
    streams = [torch.cuda.Stream() for _ in runs]
    for turn in range(4):
        for r in runs:
            r["out"].fill_(5.0)
        torch.cuda.synchronize()
        for r, s in zip(runs, streams):
            with torch.cuda.stream(s):
                r["graph"].replay()
        eager = [moe.attention(r["q"], r["cache"], r["table"], r["cu"], r["lens"], max_q=r["n"], max_kv=2500) for r in runs]
        torch.cuda.synchronize()
        for r, e in zip(runs, eager):
            assert torch.equal(r["out"], r["want"]) and torch.equal(e, r["want"]), turn


def test_workspace_that_is_not_one_piece_is_refused():
    """Bytes counted through strides need not be there."""
    moe = _moe()
    rng = np.random.default_rng(7700)
    p = problem(rng, True, 64, 1, 2, 16, [2], [900])
    cache, q = to_device(moe, p["hc"]), bf16(p["q"])
    args = (q, cache, dev(p["table"]), dev(p["cu"]), dev(p["lens"]))
    need = moe.attention_workspace_bytes(cache, 2, 2, 1, max_q=2, max_kv=900)
    assert need > 0
    whole = torch.empty(2 * need, dtype=torch.uint8, device="cuda")
    for ws in (whole[:16].view(1, 16).expand(need, 16), whole[::2], whole[:need].cpu()):
        with pytest.raises(ValueError, match="workspace"):
            moe.attention(*args, max_q=2, max_kv=900, workspace=ws)
    with pytest.raises(moe.MoeError):
        moe.attention(*args, max_q=2, max_kv=900, workspace=whole[1:])          # not on a 16-byte boundary
    want, _, _ = check(moe, p, cache=cache)
    assert torch.equal(moe.attention(*args, max_q=2, max_kv=900, workspace=whole), want)
