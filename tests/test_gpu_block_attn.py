"""Block attention (kvc_attn_cross) against a plain 64-bit form over the rows that the oracle stored."""
import math

import numpy as np
import pytest

import oracle
from block_ref import cross, cross_bound, exact_kv, values
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


def _run(tw, ids, n_q, q, scale, vis=None, layer=0, lse=True, out=None):
    import torch

    out = torch.full_like(q, float("nan")) if out is None else out
    z = torch.full(q.shape[:2], float("nan"), device=q.device) if lse else None
    v = None if vis is None else torch.as_tensor(np.asarray(vis), dtype=torch.int32).to(q.device)
    tw.gpu.attn_cross(layer, ids, n_q, q, out, scale, lse=z, n_vis=v)
    torch.cuda.synchronize()
    assert tw.kvc.kvc_check_device_error(tw.gpu.ctx) == 0
    return out, z


def _compare(tw, ids, n_q, q, scale, vis, got, z, act, layer=0, bits=None, exact_kv_=False):
    """bits: significant bits of the products' operands (22 or more for 32-bit queries, 11 for others; K and V that
    fp16 holds exactly lose nothing, the probabilities still do)."""
    qa = q.double().cpu().numpy()
    o, s = got.double().cpu().numpy(), z.double().cpu().numpy()
    t0 = 0
    for i, T in zip(ids, n_q):
        K, V = values(tw.ref.seqs[i].K[layer]), values(tw.ref.seqs[i].V[layer])
        sl = slice(t0, t0 + T)
        vv = np.full(T, len(K)) if vis is None else np.asarray(vis)[sl]
        want, wz, mag, size = cross(qa[sl], K, V, scale, vv)
        sb, vb = (20, 20) if act == "f32" else ((22, 11) if exact_kv_ else (11, 11))
        bo, bz = cross_bound(mag, size, len(K), q.shape[-1], act, sb, vb)
        err = np.abs(o[sl] - want)
        assert np.all(err <= bo), "sequence %d: out off by %.3g, %.2f of its bound" % (i, err.max(), (err / bo).max())
        empty = vv <= 0
        assert np.all(np.isneginf(s[sl][empty])) and np.all(o[sl][empty] == 0)
        if (~empty).any():
            d = np.abs(s[sl][~empty] - wz[~empty])
            assert np.all(d <= bz[~empty]), "sequence %d: lse off by %.3g, %.2f of its bound" % (
                i, d.max(), (d / bz[~empty]).max())
        t0 += T


def _cache(kind, H, Hk, D, lens, page=64, seed=1, layers=1, exact=False, sigma=0.5):
    tk, tv = KINDS[kind]
    tw = _force(Twin(layers, H, Hk, D, sum(lens) + 64, n_seq_max=max(1, len(lens)), type_=tk, type_v=tv, page_rows=page))
    rng = np.random.default_rng(seed)
    for i, n in enumerate(lens):
        for layer in range(layers):
            if not n:
                continue
            if exact:
                tw.append(layer, i, 0, exact_kv(rng, n, Hk, D), exact_kv(rng, n, Hk, D))
            else:
                k, v = kv_inputs(seed, layer, n, Hk, D, pos0=1000003 * i, sigma=sigma)
                tw.append(layer, i, 0, k, v)
    return tw


@pytest.mark.parametrize("act", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("kind,D", [("q8", 64), ("f16", 64), ("q8", 128), ("f16", 128), ("q8q4", 128)])
@pytest.mark.parametrize("T,n", [(1, 1), (1, 300), (3, 65), (37, 130), (70, 1000)])
def test_cross_types_and_lengths(kind, D, act, T, n):
    tw = _cache(kind, 10, 2, D, [n], page=48)
    try:
        rng = np.random.default_rng(3)
        q = _queries(rng, T, 10, D, act)
        got, z = _run(tw, [0], [T], q, 1 / math.sqrt(D))
        _compare(tw, [0], [T], q, float(np.float32(1 / math.sqrt(D))), None, got, z, act)
    finally:
        tw.close()


@pytest.mark.parametrize("act", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("kind", ["q8", "f16"])
@pytest.mark.parametrize("H,Hk,D", [(8, 8, 64), (16, 2, 128), (6, 2, 128), (9, 3, 64)])
def test_cross_masks_on_exact_values(kind, act, H, Hk, D):
    """K and V that the cache holds exactly: the score's error is that of fp32 sums alone, so one row too many or too few
    shows.  Tokens that see nothing, one row, a part, all, and counts out of range."""
    n, T = 333, 41
    tw = _cache(kind, H, Hk, D, [n], exact=True)
    try:
        rng = np.random.default_rng(5)
        q = _queries(rng, T, H, D, act, 0.3)
        vis = rng.integers(0, n + 1, T)
        vis[:8] = [0, 1, 63, 64, 65, -7, n + 100, 2**31 - 1]
        got, z = _run(tw, [0], [T], q, 0.07, vis)
        _compare(tw, [0], [T], q, float(np.float32(0.07)), vis, got, z, act, exact_kv_=True)
        none = np.zeros(T, int)
        got, z = _run(tw, [0], [T], q, 0.07, none)
        assert bool((got == 0).all()) and bool((z == -float("inf")).all())
    finally:
        tw.close()


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["q8", "f16"])
def test_cross_ragged_batch_shared_and_empty_sequences(kind, act):
    lens = [5, 0, 700, 64, 2100]
    tw = _cache(kind, 8, 2, 64, lens, page=32)
    try:
        rng = np.random.default_rng(7)
        ids, n_q = [4, 1, 2, 4, 0, 3], [3, 2, 0, 19, 1, 5]  # an id twice, a sequence without rows, one without tokens
        T = sum(n_q)
        q = _queries(rng, T, 8, 64, act)
        vis = rng.integers(0, 2200, T)
        for v in (None, vis):
            got, z = _run(tw, ids, n_q, q, 0.125, v)
            vv = np.full(T, 2**31 - 1) if v is None else v
            t0 = 0
            for i, t in zip(ids, n_q):
                if lens[i] == 0:
                    assert bool((got[t0:t0 + t] == 0).all())
                    assert bool((z[t0:t0 + t] == -float("inf")).all())
                elif t:
                    _compare(tw, [i], [t], q[t0:t0 + t], 0.125, vv[t0:t0 + t], got[t0:t0 + t], z[t0:t0 + t], act)
                t0 += t
        again, z2 = _run(tw, ids, n_q, q, 0.125, vis)
        assert bool((again == got).all()) and bool((z2 == z).all())  # bitwise repeatable
    finally:
        tw.close()


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["q8", "f16"])
@pytest.mark.parametrize("scale", [0.0, -0.3])
def test_cross_scales_of_zero_and_below(scale, kind, act):
    n, T = 300, 37
    tw = _cache(kind, 8, 2, 64, [n], exact=True)
    try:
        rng = np.random.default_rng(15)
        q = _queries(rng, T, 8, 64, act, 0.3)
        vis = rng.integers(0, n + 1, T)
        got, z = _run(tw, [0], [T], q, scale, vis)
        _compare(tw, [0], [T], q, float(np.float32(scale)), vis, got, z, act, exact_kv_=True)
    finally:
        tw.close()


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["q8", "f16"])
@pytest.mark.parametrize("T", [6, 90])
def test_cross_long_rows_in_few_pages(kind, act, T):
    """Many steps in a part, whole units beside cut ones, a page that ends inside a step."""
    n = 9000
    tw = _cache(kind, 8, 2, 64, [n], page=1008)
    try:
        rng = np.random.default_rng(21)
        q = _queries(rng, T, 8, 64, act)
        vis = np.sort(rng.integers(n - 300, n + 1, T))
        got, z = _run(tw, [0], [T], q, 0.125, vis)
        _compare(tw, [0], [T], q, 0.125, vis, got, z, act)
    finally:
        tw.close()


def test_cross_more_sequences_than_a_launch_holds():
    import torch

    n_seq = 70
    tw = _cache("q8", 4, 2, 64, [20 + i for i in range(n_seq)], page=16)
    try:
        rng = np.random.default_rng(9)
        ids = list(rng.permutation(n_seq))
        n_q = [1 + i % 3 for i in range(n_seq)]
        q = _queries(rng, sum(n_q), 4, 64, "f32")
        got, z = _run(tw, ids, n_q, q, 0.125)
        _compare(tw, ids, n_q, q, 0.125, None, got, z, "f32")
        # nothing behind the last token is written
        out = torch.full((sum(n_q) + 5, 4, 64), 7.0, device="cuda:0")
        tw.gpu.attn_cross(0, ids, n_q, q, out, 0.125)
        torch.cuda.synchronize()
        assert bool((out[sum(n_q):] == 7.0).all()) and bool((out[:sum(n_q)] == got).all())
    finally:
        tw.close()


@pytest.mark.parametrize("act", ["f32", "f16", "bf16"])
def test_cross_one_token_is_the_decode_attention(act):
    import torch

    tw = _cache("q8", 40, 8, 128, [1500])
    try:
        q = _queries(np.random.default_rng(2), 1, 40, 128, act)
        got, z = _run(tw, [0], [1], q, 0.088)
        out = torch.empty(1, 40, 128, device="cuda:0")
        tw.gpu.attn_decode(0, [0], q.float(), out, 0.088)
        torch.cuda.synchronize()
        _compare(tw, [0], [1], q, float(np.float32(0.088)), None, got, z, act)
        if act == "f32":
            assert float((got - out).abs().max()) <= 2e-6
    finally:
        tw.close()


@pytest.mark.parametrize("kind", ["q8", "f16"])
@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_cross_values_of_any_size(kind, act):
    """Scales far apart between rows and tiles, queries of very small and very large magnitude."""
    n, T, D = 400, 20, 64
    tw = _force(Twin(1, 4, 2, D, n + 64, type_=KINDS[kind][0], page_rows=64))
    try:
        rng = np.random.default_rng(11)
        k = rng.standard_normal((n, 2, D)).astype(np.float32)
        v = rng.standard_normal((n, 2, D)).astype(np.float32)
        # values grow from 1e-3 to 1e4 along the rows, K shrinks
        f = (10.0 ** np.linspace(-3, 4, n)).astype(np.float32)[:, None, None]
        tw.append(0, 0, 0, k / np.sqrt(f), v * f)
        q = _queries(rng, T, 4, D, act)
        mult = [2.0**-30, 1.0, 2.0**9] + [1.0] * (T - 3)
        import torch

        q = (q.float() * torch.tensor(mult, device=q.device)[:, None, None]).to(q.dtype)
        vis = [n, n, n] + list(rng.integers(1, n + 1, T - 3))
        got, z = _run(tw, [0], [T], q, 0.01, vis)
        # V's range: 16-bit results are exact to 11 bits of the largest value met (20 bits for 32-bit ones)
        K, V = values(tw.ref.seqs[0].K[0]), values(tw.ref.seqs[0].V[0])
        want, wz, mag, size = cross(q.double().cpu().numpy(), K, V, float(np.float32(0.01)), np.asarray(vis))
        sb, vb = (20, 20) if act == "f32" else (11, 11)
        bo, bz = cross_bound(mag, size, n, D, act, sb, vb)
        assert np.all(np.abs(got.double().cpu().numpy() - want) <= bo)
        assert np.all(np.abs(z.double().cpu().numpy() - wz) <= bz)
    finally:
        tw.close()


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["q8", "f16"])
@pytest.mark.parametrize("T", [3, 40, 150])
def test_cross_unseen_rows_never_reach_a_token(kind, act, T):
    """Infinities and NaN in K and V of rows that a token does not see change nothing; in rows that it sees they
    come through."""
    import torch

    n, D, H, Hk = 700, 64, 4, 2
    rng = np.random.default_rng(13)
    k, v = kv_inputs(13, 0, n, Hk, D)
    bad = [600, 610, 640, 699]
    outs = []
    q = _queries(rng, T, H, D, act)
    vis = rng.integers(0, 600, T)
    vis[0] = 600
    for spoil in (False, True):
        tw = _force(Twin(1, H, Hk, D, n + 64, type_=KINDS[kind][0], page_rows=64))
        try:
            kk, vv = k.copy(), v.copy()
            if spoil:
                kk[bad], vv[bad] = np.float32(np.inf), np.float32(np.nan)
                vv[610, :, ::2], kk[640] = -np.inf, np.nan
            t = torch.from_numpy
            tw.gpu.append(0, 0, 0, t(kk).to(tw.dev), t(vv).to(tw.dev))
            got, z = _run(tw, [0], [T], q, 0.125, vis)
            outs.append((got, z))
            if spoil:
                # the last token sees row 600 too: its K is infinite, so its weights are not numbers
                w = vis.copy()
                w[-1] = 601
                got, z = _run(tw, [0], [T], q, 0.125, w)
                assert not bool(torch.isfinite(got[-1].float()).all())
                assert bool((got[:-1] == outs[1][0][:-1]).all())
        finally:
            tw.close()
    assert bool((outs[0][0] == outs[1][0]).all()) and bool((outs[0][1] == outs[1][1]).all())


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("T", [2, 60])
def test_cross_infinite_value_of_a_seen_row(act, T):
    import torch

    n, D = 500, 64
    k, v = kv_inputs(17, 0, n, 2, D)
    v[100, 0, 3], v[101, 0, 4], v[102, 1, 5] = np.inf, -np.inf, np.nan
    v[400, 0, 3] = -np.inf
    tw = _force(Twin(1, 4, 2, D, n + 64, type_=F16, page_rows=64))
    try:
        tw.gpu.append(0, 0, 0, torch.from_numpy(k).to(tw.dev), torch.from_numpy(v).to(tw.dev))
        q = _queries(np.random.default_rng(1), T, 4, D, act)
        got, _ = _run(tw, [0], [T], q, 0.125, [300] * T)
        o = got.float()
        inf = float("inf")
        assert bool((o[:, :2, 3] == inf).all()) and bool((o[:, :2, 4] == -inf).all())
        assert bool(torch.isnan(o[:, 2:, 5]).all())
        o[:, :2, 3] = o[:, :2, 4] = 0
        o[:, 2:, 5] = 0
        assert bool(torch.isfinite(o).all())
        got, _ = _run(tw, [0], [T], q, 0.125, [450] * T)
        assert bool(torch.isnan(got.float()[:, :2, 3]).all())  # +inf and -inf
    finally:
        tw.close()


def test_cross_splits_agree_with_one_part():
    """The same rows attended alone (split over items) and among enough query tiles (one part each)."""
    tw = _cache("q8", 8, 8, 64, [3000], page=256)
    try:
        q = _queries(np.random.default_rng(3), 700, 8, 64, "f32")
        many, _ = _run(tw, [0], [700], q, 0.125)
        few, z = _run(tw, [0], [3], q[:3].contiguous(), 0.125)
        _compare(tw, [0], [3], q[:3], 0.125, None, few, z, "f32")
        assert float((many[:3] - few).abs().max()) <= 3e-6
    finally:
        tw.close()


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_cross_in_a_graph_on_another_stream(act):
    """Two captured graphs of one context share its work space; replayed in turn they give what eager calls give."""
    import torch

    tw = _cache("q8", 8, 2, 128, [2000, 900], layers=2)
    try:
        rng = np.random.default_rng(4)
        qs = [_queries(rng, 5, 8, 128, act), _queries(rng, 90, 8, 128, act)]
        calls = [(0, [0, 1], [2, 3], qs[0]), (1, [1], [90], qs[1])]
        outs = [torch.empty_like(q) for q in qs]
        want = [_run(tw, ids, nq, q, 0.09, layer=layer)[0] for layer, ids, nq, q in calls]
        st = torch.cuda.Stream()
        graphs = []
        for (layer, ids, nq, q), out in zip(calls, outs):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=st):
                tw.gpu.attn_cross(layer, ids, nq, q, out, 0.09)
            graphs.append(g)
        for _ in range(3):
            for o in outs:
                o.zero_()
            torch.cuda.synchronize()
            with torch.cuda.stream(st):
                for g in graphs:
                    g.replay()
            torch.cuda.synchronize()
            for o, w in zip(outs, want):
                assert bool((o == w).all())
    finally:
        tw.close()


def test_cross_first_call_in_a_capture_is_refused():
    import torch

    tw = _cache("q8", 8, 2, 64, [100])
    try:
        q = _queries(np.random.default_rng(4), 2, 8, 64, "f32")
        out = torch.empty_like(q)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out.zero_()
            with pytest.raises(tw.kvc.KvcError) as e:
                tw.gpu.attn_cross(0, [0], [2], q, out, 0.125)
        assert e.value.status == tw.kvc.KVC_EINVAL
        g.replay()
        got, z = _run(tw, [0], [2], q, 0.125)
        _compare(tw, [0], [2], q, 0.125, None, got, z, "f32")
    finally:
        tw.close()


def test_cross_refusals():
    import torch

    kvc_tw = _cache("q8", 8, 2, 64, [100, 50])
    try:
        tw, kvc = kvc_tw, kvc_tw.kvc
        q = _queries(np.random.default_rng(4), 4, 8, 64, "f32")
        out = torch.empty_like(q)
        ok = dict(layer=0, seq_ids=[0], n_q=[4], act=0, q=q, out=out, kq_scale=0.1)
        bad = [dict(layer=1), dict(layer=-1), dict(seq_ids=[2]), dict(seq_ids=[-1]), dict(n_q=[-1]), dict(act=3),
               dict(act=-1), dict(q=None), dict(out=None), dict(q=q.data_ptr() + 4), dict(out=out.data_ptr() + 8),
               dict(kq_scale=float("nan")), dict(kq_scale=float("inf")), dict(out=q), dict(out=q.data_ptr() + 256),
               dict(seq_ids=[], n_q=[]), dict(lse=out.data_ptr() + 2), dict(n_vis=out.data_ptr() + 1),
               dict(n_q=[2**31 - 1])]
        for b in bad:
            with pytest.raises(kvc.KvcError) as e:
                kvc.kvc_attn_cross(tw.gpu.ctx, **{**ok, **b})
            assert e.value.status == kvc.KVC_EINVAL, b
        kvc.kvc_attn_cross(tw.gpu.ctx, **{**ok, "n_q": [0]})  # no tokens: nothing to do
        good = dict(layer=0, seq_ids=[0], n_q=[4], q=q, out=out, kq_scale=0.1)
        for b in (dict(q=q.double()), dict(q=q.cpu()), dict(out=out.half()), dict(q=q.transpose(0, 1)), dict(n_q=[5]),
                  dict(lse=torch.empty(4, 7, device="cuda:0")), dict(n_vis=torch.zeros(4, device="cuda:0")),
                  dict(n_vis=torch.zeros(4, dtype=torch.int32))):
            with pytest.raises(kvc.KvcError) as e:
                tw.gpu.attn_cross(**{**good, **b})
            assert e.value.status == kvc.KVC_EINVAL, b
        host = kvc.KVCache(1, 8, 2, 64, 512, residency=kvc.KVC_HOST_PINNED)
        try:
            with pytest.raises(kvc.KvcError) as e:
                host.attn_cross(**good)
            assert e.value.status == kvc.KVC_EINVAL
        finally:
            host.close()
    finally:
        kvc_tw.close()


def test_cross_work_space_allocation_failure():
    import torch

    tw = _cache("q8", 8, 2, 64, [100])
    try:
        q = _queries(np.random.default_rng(4), 2, 8, 64, "f32")
        out = torch.empty_like(q)
        tw.kvc.kvc_debug_fail_alloc_after(tw.gpu.ctx, 0)
        with pytest.raises(tw.kvc.KvcError) as e:
            tw.gpu.attn_cross(0, [0], [2], q, out, 0.125)
        assert e.value.status == tw.kvc.KVC_ENOMEM
        tw.kvc.kvc_debug_fail_alloc_after(tw.gpu.ctx, -1)
        got, z = _run(tw, [0], [2], q, 0.125)
        _compare(tw, [0], [2], q, 0.125, None, got, z, "f32")
    finally:
        tw.close()
