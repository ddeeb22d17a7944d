"""Attention over a tree of drafted tokens (kvc_attn_tree) against a plain 64-bit form over the rows that the oracle stored."""
import math

import numpy as np
import pytest

import oracle
from block_ref import exact_kv, values
from draft_ref import attend, attend_bound, tree_sees
from twin import Twin, kv_inputs

pytestmark = pytest.mark.gpu


Q8, F16, Q4 = oracle.Q8_0, oracle.F16, oracle.Q4_0
KINDS = {"q8": (Q8, Q8), "f16": (F16, F16), "q8q4": (Q8, Q4)}


KERNEL = 0


@pytest.fixture(autouse=True, params=[0, 1, 2], ids=["by_size", "mma", "tcgen05"])
def kernel(request):
    """Every test on the kernel that the sizes choose and on each of the two for 16-bit queries."""
    global KERNEL
    act = request.node.callspec.params.get("act") if hasattr(request.node, "callspec") else None
    if request.param and act == "f32":
        pytest.skip("32-bit queries have one kernel")
    KERNEL = request.param
    yield request.param
    KERNEL = 0


def _force(tw):
    tw.kvc.kvc_debug_block_kernel(tw.gpu.ctx, KERNEL)
    return tw


def _types():
    import torch

    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def _queries(rng, T, H, D, act, sigma=1.0):
    import torch

    return torch.from_numpy((rng.standard_normal((T, H, D)) * sigma).astype(np.float32)).to("cuda:0", _types()[act])


def _parents(rng, T, reach=6):
    return np.array([-1 if t == 0 else rng.integers(max(-1, t - reach), t) for t in range(T)], np.int32)


def _run(tw, ids, n_q, q, scale, parent=None, layer=0):
    import torch

    out = torch.full_like(q, float("nan"))
    p = None if parent is None else torch.from_numpy(np.ascontiguousarray(parent, np.int32)).to(q.device)
    tw.gpu.attn_tree(layer, ids, n_q, q, out, scale, parent=p)
    torch.cuda.synchronize()
    assert tw.kvc.kvc_check_device_error(tw.gpu.ctx) == 0
    return out


def _compare(tw, ids, n_q, q, scale, parent, got, act, layer=0, exact=False):
    qa, o, t0 = q.double().cpu().numpy(), got.double().cpu().numpy(), 0
    for i, T in zip(ids, n_q):
        s = tw.ref.seqs[i]
        K, V = values(s.K[layer]), values(s.V[layer])
        sl = slice(t0, t0 + T)
        par = None if parent is None else parent[sl]
        want, mag, size = attend(qa[sl], K, V, float(np.float32(scale)), tree_sees(par, len(K), T))
        bound = attend_bound(mag, size, len(K), q.shape[-1], act, exact)
        err = np.abs(o[sl] - want)
        assert np.all(err <= bound), "sequence %d: off by %.3g, %.2f of its bound" % (i, err.max(), (err / bound).max())
        t0 += T


def _cache(kind, H, Hk, D, lens, page=64, seed=1, layers=1, exact=False, extra=64):
    tk, tv = KINDS[kind]
    tw = _force(Twin(layers, H, Hk, D, sum(lens) + extra, n_seq_max=max(1, len(lens)), type_=tk, type_v=tv, page_rows=page))
    rng = np.random.default_rng(seed)
    for i, n in enumerate(lens):
        for layer in range(layers):
            if not n:
                continue
            if exact:
                tw.append(layer, i, 0, exact_kv(rng, n, Hk, D), exact_kv(rng, n, Hk, D))
            else:
                k, v = kv_inputs(seed, layer, n, Hk, D, pos0=1000003 * i, sigma=0.5)
                tw.append(layer, i, 0, k, v)
    return tw


@pytest.mark.parametrize("act", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("kind,D", [("q8", 64), ("f16", 64), ("q8", 128), ("f16", 128), ("q8q4", 128)])
@pytest.mark.parametrize("T,n", [(1, 1), (1, 300), (3, 3), (3, 65), (6, 130), (13, 1000), (37, 700)])
def test_tree_types_and_lengths(kind, D, act, T, n):
    """10 heads of 2 KV heads: tiles of 16 (T 1, 3), 32 (6) and 64 query rows (13: two tiles, 37: three)."""
    tw = _cache(kind, 10, 2, D, [n], page=48)
    try:
        rng = np.random.default_rng(3)
        q = _queries(rng, T, 10, D, act)
        par = _parents(rng, T)
        got = _run(tw, [0], [T], q, 1 / math.sqrt(D), par)
        _compare(tw, [0], [T], q, 1 / math.sqrt(D), par, got, act)
        assert bool((_run(tw, [0], [T], q, 1 / math.sqrt(D), par) == got).all())  # bitwise repeatable
    finally:
        tw.close()


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["q8", "f16"])
@pytest.mark.parametrize("H,Hk,D", [(8, 8, 64), (16, 2, 128), (6, 2, 128), (8, 1, 64)])
@pytest.mark.parametrize("shape", ["tree", "chain", "none", "roots", "odd"])
def test_tree_masks_on_exact_values(kind, act, H, Hk, D, shape):
    """K and V that the cache holds exactly and scores of some size: a row too many or too few shows.  A random tree, a
    chain given and not given, roots only, and parents that are no earlier tokens (roots too)."""
    n, T = 333, 41
    tw = _cache(kind, H, Hk, D, [n], exact=True)
    try:
        rng = np.random.default_rng(5)
        q = _queries(rng, T, H, D, act, 0.3)
        par = {"tree": _parents(rng, T), "chain": np.arange(T, dtype=np.int32) - 1, "none": None,
               "roots": np.full(T, -1, np.int32), "odd": _parents(rng, T)}[shape]
        if shape == "odd":
            par[[3, 9, 17, 30]] = [3, 40, 2**31 - 1, -2**31]
        got = _run(tw, [0], [T], q, 0.07, par)
        _compare(tw, [0], [T], q, 0.07, par, got, act, exact=True)
        if shape == "none":
            assert bool((_run(tw, [0], [T], q, 0.07, np.arange(T) - 1) == got).all())
    finally:
        tw.close()


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["q8", "f16"])
@pytest.mark.parametrize("T", [32, 33, 64, 65, 255, 256])
def test_tree_of_many_tokens(kind, act, T):
    """Masks of up to eight words, a tree that spans several steps, one that is the whole sequence."""
    for n in (T, T + 190):
        tw = _cache(kind, 4, 2, 64, [n], page=32, exact=True)
        try:
            rng = np.random.default_rng(T)
            q = _queries(rng, T, 4, 64, act, 0.3)
            par = _parents(rng, T, 40)
            got = _run(tw, [0], [T], q, 0.05, par)
            _compare(tw, [0], [T], q, 0.05, par, got, act, exact=True)
        finally:
            tw.close()


@pytest.mark.parametrize("act", ["f32", "f16"])
@pytest.mark.parametrize("kind", ["q8", "f16"])
def test_tree_ragged_batch(kind, act):
    lens = [5, 0, 700, 64, 2100]
    tw = _cache(kind, 8, 2, 64, lens, page=32)
    try:
        rng = np.random.default_rng(7)
        ids, n_q = [4, 1, 2, 4, 0, 3], [3, 0, 0, 19, 5, 9]  # an id twice, one without rows or tokens, a whole sequence
        T = sum(n_q)
        q = _queries(rng, T, 8, 64, act)
        par = np.concatenate([_parents(rng, t) for t in n_q])
        got = _run(tw, ids, n_q, q, 0.125, par)
        _compare(tw, [4, 4, 0, 3], [3, 19, 5, 9], q, 0.125, par, got, act)
    finally:
        tw.close()


@pytest.mark.parametrize("act", ["f16", "bf16"])
@pytest.mark.parametrize("kind,D", [("q8", 64), ("f16", 128), ("q8q4", 128)])
@pytest.mark.parametrize("n_q", [[52], [76], [77], [103, 5], [20, 52, 154, 77, 1]])
def test_tree_last_tile_of_few_rows(kind, D, act, n_q):
    """Blocks whose query rows (5 a token) end shortly behind a tile, at its half and behind that."""
    H, Hk = 10, 2
    lens = [max(n_q) + 37 * (i + 1) + 900 * (i % 2) for i in range(len(n_q))]
    tw = _force(_cache(kind, H, Hk, D, lens))
    try:
        rng = np.random.default_rng(13)
        q = _queries(rng, sum(n_q), H, D, act)
        par = np.concatenate([_parents(rng, t) for t in n_q])
        ids = list(range(len(n_q)))
        _compare(tw, ids, n_q, q, 0.11, par, _run(tw, ids, n_q, q, 0.11, par), act)
    finally:
        tw.close()


def test_tree_more_last_tiles_than_a_launch_has_room_for():
    """40 sequences of two tiles a KV head each, then 25 of one in the same call."""
    H, Hk, D = 10, 2, 64
    tw = _force(_cache("q8", H, Hk, D, [60 + 5 * i for i in range(40)]))
    try:
        rng = np.random.default_rng(14)
        ids, n_q = list(range(40)) + list(range(25)), [52] * 40 + [3] * 25
        q = _queries(rng, sum(n_q), H, D, "bf16")
        par = np.concatenate([_parents(rng, t) for t in n_q])
        _compare(tw, ids, n_q, q, 0.11, par, _run(tw, ids, n_q, q, 0.11, par), "bf16")
    finally:
        tw.close()


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("kind,lens", [("q8", [90, 1500, 64, 2200, 333]), ("f16", [1, 700, 40, 1300, 2])])
def test_tree_order_of_the_sequences_changes_no_bit(kind, lens, act):
    """Short and long sequences in either order: the kernel begins with the longest, a sequence's result is its own."""
    import torch

    H, Hk, D = 8, 2, 64
    tw = _force(_cache(kind, H, Hk, D, lens))
    try:
        rng = np.random.default_rng(11)
        n_q = [6, 3, 33, 1, 2]
        n_q = [min(t, n) for t, n in zip(n_q, lens)]
        qs = [_queries(rng, t, H, D, act) for t in n_q]
        ps = [_parents(rng, t) for t in n_q]
        results = []
        for order in ([0, 1, 2, 3, 4], [4, 3, 2, 1, 0], [2, 4, 1, 0, 3]):
            q, m = torch.cat([qs[i] for i in order]), [n_q[i] for i in order]
            parent = np.concatenate([ps[i] for i in order])
            got = _run(tw, order, m, q, 0.125, parent)
            _compare(tw, order, m, q, 0.125, parent, got, act)
            results.append(dict(zip(order, got.split(m))))
        for i in range(5):
            for r in results[1:]:
                assert torch.equal(r[i].view(torch.uint8), results[0][i].view(torch.uint8))
    finally:
        tw.close()


def test_tree_more_sequences_than_a_launch_holds():
    import torch

    n_seq = 70
    tw = _cache("q8", 4, 2, 64, [20 + i for i in range(n_seq)], page=16)
    try:
        rng = np.random.default_rng(9)
        ids = [int(i) for i in rng.permutation(n_seq)]
        n_q = [1 + i % 5 for i in range(n_seq)]
        q = _queries(rng, sum(n_q), 4, 64, "f32")
        par = np.concatenate([_parents(rng, t) for t in n_q])
        got = _run(tw, ids, n_q, q, 0.125, par)
        _compare(tw, ids, n_q, q, 0.125, par, got, "f32")
        out = torch.full((sum(n_q) + 5, 4, 64), 7.0, device="cuda:0")  # nothing behind the last token is written
        tw.gpu.attn_tree(0, ids, n_q, q, out, 0.125, parent=torch.from_numpy(par).to(q.device))
        torch.cuda.synchronize()
        assert bool((out[sum(n_q):] == 7.0).all()) and bool((out[:sum(n_q)] == got).all())
    finally:
        tw.close()


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["q8", "f16", "q8q4"])
@pytest.mark.parametrize("T", [2, 6, 30])
def test_tree_long_rows(kind, act, T):
    """Rings that go round several times, parts of many steps, pages that end inside a step."""
    n, D = 9000, 128
    tw = _cache(kind, 10, 2, D, [n], page=1008)
    try:
        rng = np.random.default_rng(21)
        q = _queries(rng, T, 10, D, act)
        par = _parents(rng, T)
        got = _run(tw, [0], [T], q, 0.0884, par)
        _compare(tw, [0], [T], q, 0.0884, par, got, act)
    finally:
        tw.close()


@pytest.mark.parametrize("cut", [1, 7, 16, 33, 100])
def test_tree_rows_that_start_inside_a_page(cut):
    """A prefix left: the first row lies anywhere in its page, and the rows before it belong to nobody."""
    tw = _cache("f16", 8, 2, 64, [400], page=64)
    try:
        tw.gpu.seq_rm(0, 0, cut)
        tw.ref.seq_rm(0, 0, cut)
        rng = np.random.default_rng(cut)
        T = 9
        q = _queries(rng, T, 8, 64, "f32")
        par = _parents(rng, T)
        got = _run(tw, [0], [T], q, 0.125, par)
        _compare(tw, [0], [T], q, 0.125, par, got, "f32")
    finally:
        tw.close()


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["q8", "f16", "q8q4"])
@pytest.mark.parametrize("T", [4, 20])
def test_tree_unseen_rows_never_reach_a_token(kind, act, T):
    """Infinities and NaN in rows before the first, behind the last and of other branches change nothing."""
    import torch

    n, D, H, Hk, cut = 300, 128, 4, 2, 21
    tk, tv = KINDS[kind]
    rng = np.random.default_rng(13)
    k, v = kv_inputs(13, 0, n, Hk, D)
    q = _queries(rng, T, H, D, act)
    par = np.full(T, -1, np.int32)  # siblings: token 1's row and token 3's are spoilt, the others must not notice
    par[2] = 0
    spoilt = [1, 3]
    outs = []
    for spoil in (False, True):
        tw = _force(Twin(1, H, Hk, D, n + 64, type_=tk, type_v=tv, page_rows=64))
        try:
            kk, vv = k.copy(), v.copy()
            tail = np.ones((30, Hk, D), np.float32)
            if spoil:
                kk[:cut], vv[:cut] = np.inf, np.nan
                vv[3, :, ::2] = np.inf
                for t in spoilt:
                    kk[n - T + t], vv[n - T + t] = np.inf, np.inf
                    vv[n - T + t, :, ::3] = np.nan
                tail[:] = np.nan
                tail[::2] = np.inf
            t = torch.from_numpy
            tw.gpu.append(0, 0, 0, t(kk).to(tw.dev), t(vv).to(tw.dev))
            tw.gpu.append(0, 0, n, t(tail).to(tw.dev), t(tail).to(tw.dev))
            tw.gpu.seq_rm(0, n, -1)  # what is left of these lies behind the last row
            tw.gpu.seq_rm(0, 0, cut)  # and before the first
            outs.append(_run(tw, [0], [T], q, 0.09, par))
        finally:
            tw.close()
    keep = [t for t in range(T) if t not in spoilt]
    assert bool(torch.isfinite(outs[0].float()).all())
    assert bool((outs[0][keep] == outs[1][keep]).all())
    assert not bool(torch.isfinite(outs[1][spoilt].float()).any(-1).any())  # each sees its own row


@pytest.mark.parametrize("act", ["f32", "f16"])
@pytest.mark.parametrize("T", [3, 30])
def test_tree_infinite_values_of_seen_rows(act, T):
    import torch

    n, D = 500, 64
    k, v = kv_inputs(17, 0, n, 2, D)
    v[100, 0, 3], v[101, 0, 4], v[102, 1, 5] = np.inf, -np.inf, np.nan
    v[n - T, 0, 7] = np.inf  # the root of all: a row of a step that not all tokens see wholly
    v[n - 1, 1, 9] = -np.inf  # the last token's own
    tw = _force(Twin(1, 4, 2, D, n + 64, type_=F16, page_rows=64))
    try:
        tw.gpu.append(0, 0, 0, torch.from_numpy(k).to(tw.dev), torch.from_numpy(v).to(tw.dev))
        q = _queries(np.random.default_rng(1), T, 4, D, act)
        par = np.zeros(T, np.int32)
        par[0] = -1
        o = _run(tw, [0], [T], q, 0.125, par).float()
        inf = float("inf")
        assert bool((o[:, :2, 3] == inf).all()) and bool((o[:, :2, 4] == -inf).all()) and bool((o[:, :2, 7] == inf).all())
        assert bool(torch.isnan(o[:, 2:, 5]).all()) and bool((o[-1, 2:, 9] == -inf).all())
        o[:, :2, 3] = o[:, :2, 4] = o[:, :2, 7] = 0
        o[:, 2:, 5] = 0
        o[-1, 2:, 9] = 0
        assert bool(torch.isfinite(o).all())
        # the other values, against a cache without them
        for i in (100, 101, 102, n - T, n - 1):
            v[i][~np.isfinite(v[i])] = 0
        tw2 = _force(Twin(1, 4, 2, D, n + 64, type_=F16, page_rows=64))
        try:
            tw2.append(0, 0, 0, k, v)
            plain = _run(tw2, [0], [T], q, 0.125, par)
            _compare(tw2, [0], [T], q, 0.125, par, plain, act)
            p = plain.float()
            p[:, :2, 3] = p[:, :2, 4] = p[:, :2, 7] = 0
            p[:, 2:, 5] = 0
            p[-1, 2:, 9] = 0
            assert float((o - p).abs().max()) <= (2.0**-18 if act == "f32" else 2.0**-9)
        finally:
            tw2.close()
    finally:
        tw.close()


@pytest.mark.parametrize("kind", ["q8", "f16"])
@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_tree_values_of_any_size(kind, act):
    """Scales far apart between rows, queries of very small and very large magnitude, a scale of zero and below."""
    import torch

    n, T, D = 400, 20, 64
    tw = _force(Twin(1, 4, 2, D, n + 64, type_=KINDS[kind][0], page_rows=64))
    try:
        rng = np.random.default_rng(11)
        k = rng.standard_normal((n, 2, D)).astype(np.float32)
        v = rng.standard_normal((n, 2, D)).astype(np.float32)
        f = (10.0 ** np.linspace(-3, 4, n)).astype(np.float32)[:, None, None]
        tw.append(0, 0, 0, k / np.sqrt(f), v * f)
        q = _queries(rng, T, 4, D, act)
        mult = [2.0**-30, 1.0, 2.0**9] + [1.0] * (T - 3)
        q = (q.float() * torch.tensor(mult, device=q.device)[:, None, None]).to(q.dtype)
        par = _parents(rng, T)
        for scale in (0.01, 0.0, -0.02):
            got = _run(tw, [0], [T], q, scale, par)
            _compare(tw, [0], [T], q, scale, par, got, act)
    finally:
        tw.close()


@pytest.mark.parametrize("act", ["f32", "f16"])
def test_tree_peaked_softmax(act):
    """Maxima that keep rising along the rows, and one row that takes nearly all the weight."""
    n, T, D = 1500, 7, 128
    tw = _force(Twin(1, 8, 2, D, n + 64, type_=Q8, page_rows=64))
    try:
        rng = np.random.default_rng(19)
        u = rng.standard_normal((1, 2, D))
        k = (rng.standard_normal((n, 2, D)) * 0.1 + u * np.linspace(0, 6, n)[:, None, None]).astype(np.float32)
        v = rng.standard_normal((n, 2, D)).astype(np.float32)
        tw.append(0, 0, 0, k, v)
        import torch

        q = torch.from_numpy((np.repeat(u, 4, 1) + rng.standard_normal((T, 8, D)) * 0.2).astype(np.float32)).to("cuda:0", _types()[act])
        par = _parents(rng, T)
        got = _run(tw, [0], [T], q, 0.0884, par)
        _compare(tw, [0], [T], q, 0.0884, par, got, act)
    finally:
        tw.close()


def test_tree_one_token_is_the_decode_attention():
    import torch

    tw = _cache("q8", 40, 8, 128, [1500])
    try:
        q = _queries(np.random.default_rng(2), 1, 40, 128, "f32")
        got = _run(tw, [0], [1], q, 0.088)
        out = torch.empty(1, 40, 128, device="cuda:0")
        tw.gpu.attn_decode(0, [0], q, out, 0.088)
        torch.cuda.synchronize()
        assert float((got - out).abs().max()) <= 2e-6
    finally:
        tw.close()


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_tree_in_a_graph_on_another_stream(act):
    """Two captured graphs share the work space; the parents of a replay are those that the tensor holds then."""
    import torch

    tw = _cache("q8", 8, 2, 128, [2000, 900], layers=2)
    try:
        rng = np.random.default_rng(4)
        qs = [_queries(rng, 9, 8, 128, act), _queries(rng, 30, 8, 128, act)]
        calls = [(0, [0, 1], [4, 5]), (1, [1], [30])]
        pars = [[np.concatenate([_parents(rng, t) for t in nq]) for _, _, nq in calls] for _ in range(2)]
        want = [[_run(tw, ids, nq, q, 0.09, par, layer=layer) for (layer, ids, nq), q, par in zip(calls, qs, ps)] for ps in pars]
        par_d = [torch.from_numpy(p).to("cuda:0") for p in pars[0]]
        outs = [torch.empty_like(q) for q in qs]
        st = torch.cuda.Stream()
        graphs = []
        for (layer, ids, nq), q, out, par in zip(calls, qs, outs, par_d):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=st):
                tw.gpu.attn_tree(layer, ids, nq, q, out, 0.09, parent=par)
            graphs.append(g)
        for which in (0, 1, 0):
            for p, src in zip(par_d, pars[which]):
                p.copy_(torch.from_numpy(src))
            torch.cuda.synchronize()
            with torch.cuda.stream(st):
                for g in graphs:
                    g.replay()
            torch.cuda.synchronize()
            for o, w in zip(outs, want[which]):
                assert bool((o == w).all())
    finally:
        tw.close()


def test_tree_first_call_in_a_capture_is_refused():
    import torch

    tw = _cache("q8", 8, 2, 64, [100])
    try:
        q = _queries(np.random.default_rng(4), 2, 8, 64, "f32")
        out = torch.empty_like(q)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out.zero_()
            with pytest.raises(tw.kvc.KvcError) as e:
                tw.gpu.attn_tree(0, [0], [2], q, out, 0.125)
        assert e.value.status == tw.kvc.KVC_EINVAL
        g.replay()
        _compare(tw, [0], [2], q, 0.125, None, _run(tw, [0], [2], q, 0.125), "f32")
    finally:
        tw.close()


def test_tree_refusals():
    import torch

    tw = _cache("q8", 8, 2, 64, [300, 3])
    kvc = tw.kvc
    try:
        q = _queries(np.random.default_rng(4), 4, 8, 64, "f32")
        out = torch.empty_like(q)
        ok = dict(layer=0, seq_ids=[0], n_q=[4], act=0, q=q, out=out, kq_scale=0.1)
        bad = [dict(layer=1), dict(layer=-1), dict(seq_ids=[2]), dict(seq_ids=[-1]), dict(n_q=[-1]), dict(act=3),
               dict(act=-1), dict(q=None), dict(out=None), dict(q=q.data_ptr() + 4), dict(out=out.data_ptr() + 8),
               dict(kq_scale=float("nan")), dict(kq_scale=float("inf")), dict(out=q), dict(out=q.data_ptr() + 256),
               dict(seq_ids=[], n_q=[]), dict(parent=out.data_ptr() + 1), dict(n_q=[257]), dict(seq_ids=[1]),
               dict(n_q=[2**31 - 1])]
        for b in bad:
            with pytest.raises(kvc.KvcError) as e:
                kvc.kvc_attn_tree(tw.gpu.ctx, **{**ok, **b})
            assert e.value.status == kvc.KVC_EINVAL, b
        kvc.kvc_attn_tree(tw.gpu.ctx, **{**ok, "n_q": [0]})  # no tokens: nothing to do
        good = dict(layer=0, seq_ids=[0], n_q=[4], q=q, out=out, kq_scale=0.1)
        for b in (dict(q=q.double()), dict(q=q.cpu()), dict(out=out.half()), dict(q=q.transpose(0, 1)), dict(n_q=[5]),
                  dict(parent=torch.zeros(4, device="cuda:0")), dict(parent=torch.zeros(3, dtype=torch.int32, device="cuda:0")),
                  dict(parent=torch.zeros(4, dtype=torch.int32))):
            with pytest.raises(kvc.KvcError) as e:
                tw.gpu.attn_tree(**{**good, **b})
            assert e.value.status == kvc.KVC_EINVAL, b
        host = kvc.KVCache(1, 8, 2, 64, 512, residency=kvc.KVC_HOST_PINNED)
        try:
            with pytest.raises(kvc.KvcError) as e:
                host.attn_tree(**good)
            assert e.value.status == kvc.KVC_EINVAL
        finally:
            host.close()
        kvc.kvc_debug_fail_alloc_after(tw.gpu.ctx, 0)
        with pytest.raises(kvc.KvcError) as e:
            tw.gpu.attn_tree(**good)  # its work space
        assert e.value.status == kvc.KVC_ENOMEM
        kvc.kvc_debug_fail_alloc_after(tw.gpu.ctx, -1)
        _compare(tw, [0], [4], q, 0.1, None, _run(tw, [0], [4], q, 0.1), "f32")
    finally:
        tw.close()
