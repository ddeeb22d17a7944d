"""Row weights (kvc_attn_weight) and the eviction by them (kvc_seq_evict_weight) against plain forms."""
import numpy as np
import pytest

import oracle
from block_ref import cross, evict, values, weight
from test_gpu_block_attn import KINDS, _cache, _queries, _run
from twin import Twin, assert_attn_close, kv_inputs, q_inputs

pytestmark = pytest.mark.gpu

Q8, F16, Q4 = oracle.Q8_0, oracle.F16, oracle.Q4_0


def _lse(tw, ids, n_q, q, scale, vis, layer=0):
    """The statistics in 64 bits, rounded once."""
    qa, t0, out = q.double().cpu().numpy(), 0, []
    for i, T in zip(ids, n_q):
        K, V = values(tw.ref.seqs[i].K[layer]), values(tw.ref.seqs[i].V[layer])
        out.append(cross(qa[t0:t0 + T], K, V, scale, vis[t0:t0 + T])[1])
        t0 += T
    return np.concatenate(out).astype(np.float32)


def _check_weight(tw, ids, n_q, q, scale, vis, pad=5, layer=0, masked=True):
    import torch

    scale = float(np.float32(scale))
    lse = _lse(tw, ids, n_q, q, scale, vis, layer)
    lens = [len(values(tw.ref.seqs[i].K[layer])) for i in ids]
    rng = np.random.default_rng(99)
    w0 = rng.random((len(ids), tw.Hk, max(lens) + pad)).astype(np.float32)
    w = torch.from_numpy(w0).to("cuda:0")
    z = torch.from_numpy(lse).to("cuda:0")
    nv = torch.from_numpy(np.asarray(vis, np.int32)).to("cuda:0") if masked else None
    tw.gpu.attn_weight(layer, ids, n_q, q, z, w, scale, n_vis=nv)
    torch.cuda.synchronize()
    assert tw.kvc.kvc_check_device_error(tw.gpu.ctx) == 0
    got, t0 = w.cpu().numpy(), 0
    for i, (s, T) in enumerate(zip(ids, n_q)):
        K = values(tw.ref.seqs[s].K[layer])
        add, bound = weight(q[t0:t0 + T].double().cpu().numpy(), K, scale, vis[t0:t0 + T], lse[t0:t0 + T].astype(np.float64))
        n = len(K)
        err = np.abs(got[i, :, :n] - (w0[i, :, :n].astype(np.float64) + add))
        # the accumulators take the query rows in groups of 128 or 256: an addition, rounded by half a step (2^-24), for each
        # group, on a sum that no addition makes smaller; and one more for w0 + add here
        groups = -(-T * (q.shape[1] // tw.Hk) // 128)
        lim = bound + (groups + 1) * 2.0**-24 * (w0[i, :, :n] + add)
        assert np.all(err <= lim), "entry %d: off by %.3g, %.2f of its bound" % (i, err.max(), (err / lim).max())
        assert np.array_equal(got[i, :, n:], w0[i, :, n:])  # behind the rows: as it was
        t0 += T
    return got


@pytest.mark.parametrize("act", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("kind,H,Hk,D", [("q8", 8, 2, 64), ("f16", 6, 2, 64), ("q8", 40, 8, 128), ("f16", 4, 4, 128),
                                         ("q8q4", 8, 1, 128)])
@pytest.mark.parametrize("T,n", [(1, 1), (1, 333), (17, 130), (40, 1000)])
def test_weight_types_and_lengths(kind, H, Hk, D, act, T, n):
    tw = _cache(kind, H, Hk, D, [n], page=48)
    try:
        rng = np.random.default_rng(3)
        q = _queries(rng, T, H, D, act)
        vis = np.maximum(0, np.arange(n - T + 1, n + 1))  # causal; the first tokens of a short prompt see nothing
        _check_weight(tw, [0], [T], q, D**-0.5, vis)
        _check_weight(tw, [0], [T], q, D**-0.5, np.full(T, n), masked=False)
    finally:
        tw.close()


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_weight_ragged_batch(act):
    lens = [5, 0, 700, 64]
    tw = _cache("q8", 8, 2, 64, lens, page=32)
    try:
        rng = np.random.default_rng(7)
        ids, n_q = [2, 0, 2, 3], [3, 20, 0, 5]
        q = _queries(rng, sum(n_q), 8, 64, act)
        vis = rng.integers(0, 800, sum(n_q))
        vis[:2] = [-3, 0]
        a = _check_weight(tw, ids, n_q, q, 0.125, vis)
        b = _check_weight(tw, ids, n_q, q, 0.125, vis)
        assert np.array_equal(a, b)  # bitwise repeatable
    finally:
        tw.close()


@pytest.mark.parametrize("kind", ["q8", "f16"])
@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_weight_more_query_rows_than_fit_at_a_time(kind, act):
    """Several groups of query rows over an odd number of steps; scales far apart between the steps."""
    n, T = 700, 75  # 600 query rows of a KV head
    tw = Twin(1, 8, 1, 64, n + 64, type_=KINDS[kind][0], page_rows=48)
    try:
        rng = np.random.default_rng(31)
        f = (2.0 ** rng.integers(-8, 9, (n // 100, 1, 1))).astype(np.float32).repeat(100, 0)
        k = rng.standard_normal((n, 1, 64)).astype(np.float32) * f
        tw.append(0, 0, 0, k, k)
        q = _queries(rng, T, 8, 64, act)
        vis = rng.integers(0, n + 1, T)
        _check_weight(tw, [0], [T], q, 0.01, vis)
        _check_weight(tw, [0], [T], q, -0.01, np.full(T, n), masked=False)
    finally:
        tw.close()


def test_weight_in_a_graph_on_another_stream():
    import torch

    tw = _cache("q8", 8, 2, 64, [900])
    try:
        q = _queries(np.random.default_rng(3), 9, 8, 64, "bf16")
        _, z = _run(tw, [0], [9], q, 0.125)
        w, eager = (torch.zeros(1, 2, 900, device="cuda:0") for _ in range(2))
        st, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            tw.gpu.attn_weight(0, [0], [9], q, z, w, 0.125)
        for _ in range(3):
            g.replay()
            tw.gpu.attn_weight(0, [0], [9], q, z, eager, 0.125)
        torch.cuda.synchronize()
        assert bool((w == eager).all()) and float(w.sum()) > 0
    finally:
        tw.close()


def test_weights_of_a_block_sum_to_its_tokens():
    """Every query row's weights sum to one, so the accumulators of a KV head sum to tokens x group."""
    import torch

    tw = _cache("q8", 40, 8, 128, [4000])
    try:
        q = _queries(np.random.default_rng(3), 32, 40, 128, "bf16")
        _, z = _run(tw, [0], [32], q, 0.088)
        w = torch.zeros(1, 8, 4000, device="cuda:0")
        tw.gpu.attn_weight(0, [0], [32], q, z, w, 0.088)
        # lse of 16-bit queries is off by the scores' operand rounding, averaged: far below 1e-3
        assert float((w.double().sum(2) - 160).abs().max()) <= 0.16
    finally:
        tw.close()


def test_weight_unseen_rows():
    """Infinities and NaN in K of rows that no token sees leave their accumulators and the others alone."""
    import torch

    n, D = 200, 64
    k, v = kv_inputs(13, 0, n, 2, D)
    k[150], k[160] = np.inf, np.nan
    tw = Twin(1, 4, 2, D, n + 64, type_=F16, page_rows=64)
    try:
        tw.gpu.append(0, 0, 0, torch.from_numpy(k).to(tw.dev), torch.from_numpy(v).to(tw.dev))
        q = _queries(np.random.default_rng(1), 30, 4, D, "f32")
        vis = torch.full((30,), 150, dtype=torch.int32, device="cuda:0")
        vis[3] = 0
        z = torch.empty(30, 4, device="cuda:0")
        out = torch.empty_like(q)
        tw.gpu.attn_cross(0, [0], [30], q, out, 0.125, lse=z, n_vis=vis)
        w = torch.zeros(1, 2, n, device="cuda:0")
        tw.gpu.attn_weight(0, [0], [30], q, z, w, 0.125, n_vis=vis)
        assert bool((w[:, :, 150:] == 0).all())
        assert float((w.double().sum(2) - 58).abs().max()) <= 1e-3
    finally:
        tw.close()


def test_weight_and_evict_refusals():
    import torch

    tw = _cache("q8", 8, 2, 64, [100, 50], layers=2)
    try:
        kvc = tw.kvc
        q = _queries(np.random.default_rng(4), 4, 8, 64, "f32")
        z, w = torch.zeros(4, 8, device="cuda:0"), torch.zeros(1, 2, 100, device="cuda:0")
        ok = dict(layer=0, seq_ids=[0], n_q=[4], act=0, q=q, lse=z, w=w, w_stride=100, kq_scale=0.1)
        for b in (dict(layer=2), dict(seq_ids=[2]), dict(n_q=[-1]), dict(act=7), dict(q=None), dict(lse=None),
                  dict(w=None), dict(w_stride=99), dict(kq_scale=float("nan")), dict(w=w.data_ptr() + 2),
                  dict(lse=z.data_ptr() + 1), dict(q=q.data_ptr() + 4)):
            with pytest.raises(kvc.KvcError) as e:
                kvc.kvc_attn_weight(tw.gpu.ctx, **{**ok, **b})
            assert e.value.status == kvc.KVC_EINVAL, b
        good = dict(layer=0, seq_ids=[0], n_q=[4], q=q, lse=z, w=w, kq_scale=0.1)
        for b in (dict(w=w[0]), dict(w=w.double()), dict(w=w[:, :, ::2]), dict(w=w[:, :1]), dict(lse=z.half()),
                  dict(w=torch.zeros(1, 2, 99, device="cuda:0")), dict(w=w.cpu())):
            with pytest.raises(kvc.KvcError) as e:
                tw.gpu.attn_weight(**{**good, **b})
            assert e.value.status == kvc.KVC_EINVAL, b
        assert bool((w == 0).all())
        ok = dict(seq=0, p0=0, p1=-1, n_remove=3, w=w, w_stride=100)
        for b in (dict(seq=2), dict(seq=-1), dict(n_remove=-1), dict(w=None), dict(w_stride=99), dict(w=w.data_ptr() + 1)):
            with pytest.raises(kvc.KvcError) as e:
                kvc.kvc_seq_evict_weight(tw.gpu.ctx, **{**ok, **b})
            assert e.value.status == kvc.KVC_EINVAL, b
        with pytest.raises(kvc.KvcError):
            tw.gpu.evict_weight(0, 0, -1, 3, w)  # three axes
        assert tw.gpu.n_tokens(0) == 100
        k, v = kv_inputs(5, 0, 1, 2, 64)
        tw.gpu.append(0, 0, 100, torch.from_numpy(k).to(tw.dev), torch.from_numpy(v).to(tw.dev))
        with pytest.raises(kvc.KvcError) as e:  # a step's appends are incomplete
            tw.gpu.evict_weight(0, 0, -1, 3, torch.zeros(2, 200, device="cuda:0"))
        assert e.value.status == kvc.KVC_EINVAL
    finally:
        tw.close()


def _state(blob, tw):
    return tw.ref.parse_state(blob)


def _evict_and_check(tw, seq, p0, p1, k, w0):
    """Evict on the device, and compare positions, weights and every layer's stored bytes with the plain form."""
    import torch

    before = _state(tw.gpu.state_get(seq, -1, -1), tw)
    pos = before[0]
    n = len(pos)
    lo, hi = (0 if p0 < 0 else p0), (2**31 if p1 < 0 else p1)
    cand = [j for j in range(n) if lo <= pos[j] < hi]
    order, gone = evict(w0[:, :n], cand, n, k)
    w = torch.from_numpy(w0.copy()).to("cuda:0")
    removed = tw.gpu.evict_weight(seq, p0, p1, k, w)
    assert removed == len(gone) == min(k, len(cand))
    assert tw.gpu.n_tokens(seq) == n - removed
    assert np.array_equal(tw.gpu.positions(seq), pos[order])
    want = w0.copy()
    want[:, :len(order)] = w0[:, order]
    want[:, len(order):n] = 0
    if removed == 0:
        want = w0
    assert np.array_equal(w.cpu().numpy(), want, equal_nan=True)
    after = _state(tw.gpu.state_get(seq, -1, -1), tw)
    assert np.array_equal(after[0], pos[order])
    for a, b in ((before[1], after[1]), (before[2], after[2])):
        for x, y in zip(a, b):
            assert np.array_equal(x.a[order], y.a)
            assert x.s is None or np.array_equal(x.s[order], y.s)
    return order, w


@pytest.mark.parametrize("kind,D", [("q8", 64), ("f16", 64), ("q8", 128), ("f16", 128), ("q8q4", 128)])
@pytest.mark.parametrize("n,k,page", [(1, 1, 16), (70, 5, 16), (300, 290, 64), (1000, 137, 256), (1000, 1000, 48)])
def test_evict_against_the_plain_form(kind, D, n, k, page):
    tw = _cache(kind, 8, 2, D, [40, n], page=page, layers=3)
    try:
        rng = np.random.default_rng(n + k)
        _evict_and_check(tw, 1, -1, -1, k, rng.random((2, n + 9)).astype(np.float32))
        assert tw.gpu.n_tokens(0) == 40
    finally:
        tw.close()


def test_evict_order_of_weights():
    """Ties, zeros of both signs, negative values, infinities and NaN; ranges that protect rows; nothing to do."""
    n = 500
    rng = np.random.default_rng(5)
    w = rng.integers(0, 4, (2, n)).astype(np.float32)  # many equal weights
    odd = w.copy()
    odd[:, 10], odd[0, 11], odd[1, 12], odd[0, 13] = -0.0, -5.0, np.inf, np.nan
    odd[:, 14], odd[0, 15], odd[1, 15] = -np.inf, np.inf, -np.inf
    odd[0, 16] = -np.nan
    for name, ww, p0, p1, k in (("ties", w, -1, -1, 123), ("all equal", np.zeros_like(w), -1, -1, 77),
                                ("odd", odd, -1, -1, 200), ("odd, all but two", odd, -1, -1, 498),
                                ("range", w, 4, 400, 300), ("more than there are", w, 100, 120, 50),
                                ("last rows only", w, 450, -1, 30), ("none", w, -1, -1, 0), ("empty range", w, 900, -1, 5)):
        tw = _cache("q8", 8, 2, 64, [n], page=32)
        try:
            _evict_and_check(tw, 0, p0, p1, k, ww)
        finally:
            tw.close()


def test_evict_again_and_again_among_other_operations():
    """A sequence whose first page is partly used and whose rows are out of position order: evictions, removals,
    copies, shifts and appends in turn, the attention after each against the oracle's over the same stored rows."""
    import torch

    tw = _cache("q8", 8, 2, 64, [700], page=32, layers=2)
    try:
        rng = np.random.default_rng(8)
        tw.gpu.seq_rm(0, 0, 21)
        nxt = 700
        for step in range(6):
            n = tw.gpu.n_tokens(0)
            top = int(tw.gpu.positions(0).max()) - 40
            _evict_and_check(tw, 0, 30, top, 60, rng.random((2, n + 3)).astype(np.float32))
            if step == 2:
                tw.gpu.seq_rm(0, 100, 150)
            if step == 3:
                tw.gpu.seq_cp(0, 0, 60, 60)
                tw.gpu.seq_add(0, 300, 400, -7)
            for layer in range(2):
                k, v = kv_inputs(step, layer, 35, 2, 64, pos0=nxt)
                tw.gpu.append(layer, 0, nxt, torch.from_numpy(k).to(tw.dev), torch.from_numpy(v).to(tw.dev))
            nxt += 35
            blob = tw.gpu.state_get(0, -1, -1)
            ref = oracle.OracleCache(2, 8, 2, 64, Q8, Q8)
            ref.state_set(0, blob)
            q = q_inputs(step, 0, 1, 8, 64)
            for layer in range(2):
                out = torch.empty(1, 8, 64, device="cuda:0")
                qd = torch.from_numpy(q).to("cuda:0")
                tw.gpu.attn_decode(layer, [0], qd, out, 0.125)
                assert_attn_close(out.cpu().numpy().astype(np.float64), ref.attn(layer, [0], q, 0.125), "decode")
                tw.gpu.attn_cross(layer, [0], [1], qd, out, 0.125)
                assert_attn_close(out.cpu().numpy().astype(np.float64), ref.attn(layer, [0], q, 0.125), "block")
        scores = tw.gpu.key_scores(0, 0)
        assert len(scores) == tw.gpu.n_tokens(0) and np.isfinite(scores).all()
        assert tw.gpu.evict_window(0, 0, 10, 50, 50) >= 0
    finally:
        tw.close()


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_serving_loop_keeps_a_prompt_within_its_budget(act):
    """The operators as they are used: a prompt comes in blocks, each attends over the rows before it and itself (causal),
    its weights are added to the rows', and the cache is cut back to its budget; then tokens are decoded."""
    import torch

    H, Hk, D, budget, block, layers = 8, 2, 64, 256, 96, 2
    tw = Twin(layers, H, Hk, D, 1024, type_=Q8, page_rows=64)
    try:
        rng = np.random.default_rng(12)
        w = torch.zeros(1, Hk, budget + block, device="cuda:0")
        kept = np.zeros(0, np.int64)  # positions, in row order, by the plain form
        w_ref = np.zeros((Hk, budget + block), np.float32)
        scale = 0.125
        for b in range(5):
            pos0 = b * block
            for layer in range(layers):
                k, v = kv_inputs(b, layer, block, Hk, D)
                tw.gpu.append(layer, 0, pos0, torch.from_numpy(k).to(tw.dev), torch.from_numpy(v).to(tw.dev))
            before = len(kept)
            vis = torch.arange(before + 1, before + block + 1, dtype=torch.int32, device="cuda:0")
            ref = oracle.OracleCache(layers, H, Hk, D, Q8, Q8)
            ref.state_set(0, tw.gpu.state_get(0, -1, -1))
            for layer in range(layers):
                q = _queries(rng, block, H, D, act)
                out, z = torch.empty_like(q), torch.empty(block, H, device="cuda:0")
                tw.gpu.attn_cross(layer, [0], [block], q, out, scale, lse=z, n_vis=vis)
                tw.gpu.attn_weight(layer, [0], [block], q, z, w, scale, n_vis=vis)
                K, V = values(ref.seqs[0].K[layer]), values(ref.seqs[0].V[layer])
                want, wz, _, _ = cross(q.double().cpu().numpy(), K, V, scale, vis.cpu().numpy())
                assert float(np.abs(out.double().cpu().numpy() - want).max()) <= (1e-5 if act == "f32" else 0.03)
                add, _ = weight(q.double().cpu().numpy(), K, scale, vis.cpu().numpy(), wz)
                w_ref[:, :len(K)] += add
            assert float(np.abs(w[0].cpu().numpy() - w_ref).max()) <= 2e-2
            kept = np.concatenate([kept, np.arange(pos0, pos0 + block)])
            over = len(kept) - budget
            if over > 0:
                # the device's own weights decide (near ties may differ in 64 bits)
                ww = w[0].cpu().numpy()
                cand = [j for j in range(len(kept)) if 4 <= kept[j] < pos0]
                order, _ = evict(ww[:, :len(kept)], cand, len(kept), over)
                assert tw.gpu.evict_weight(0, 4, pos0, over, w[0]) == over
                w_ref[:, :len(order)] = w_ref[:, order]
                w_ref[:, len(order):] = 0
                kept = kept[order]
                assert np.array_equal(tw.gpu.positions(0), kept)
            assert set(range(4)) <= set(kept.tolist())
        ref = oracle.OracleCache(layers, H, Hk, D, Q8, Q8)
        ref.state_set(0, tw.gpu.state_get(0, -1, -1))
        for t in range(3):
            for layer in range(layers):
                k, v = kv_inputs(50 + t, layer, 1, Hk, D)
                q = q_inputs(50 + t, layer, 1, H, D)
                out = torch.empty(1, H, D, device="cuda:0")
                t_ = lambda x: torch.from_numpy(x).to("cuda:0")  # noqa: E731
                tw.gpu.decode_step(layer, [0], [5 * block + t], t_(k), t_(v), t_(q), out, scale)
                ref.append(layer, 0, 5 * block + t, k, v)
                assert_attn_close(out.cpu().numpy().astype(np.float64), ref.attn(layer, [0], q, scale), "decode step")
    finally:
        tw.close()


def test_evict_allocation_failure_leaves_the_cache():
    import torch

    tw = _cache("q8", 8, 2, 64, [300])
    try:
        blob = tw.gpu.state_get(0, -1, -1)
        w = torch.rand(2, 300, device="cuda:0")
        w0 = w.clone()
        tw.kvc.kvc_debug_fail_alloc_after(tw.gpu.ctx, 0)
        with pytest.raises(tw.kvc.KvcError) as e:
            tw.gpu.evict_weight(0, -1, -1, 20, w)
        assert e.value.status == tw.kvc.KVC_ENOMEM
        tw.kvc.kvc_debug_fail_alloc_after(tw.gpu.ctx, -1)
        assert tw.gpu.state_get(0, -1, -1) == blob and bool((w == w0).all())
        assert tw.gpu.evict_weight(0, -1, -1, 20, w) == 20
    finally:
        tw.close()


def test_tables_of_weights_that_are_no_tensors_are_refused():
    import torch

    tw = _cache("q8", 8, 2, 64, [20])
    try:
        q = _queries(np.random.default_rng(4), 1, 8, 64, "f32")
        z, w = torch.zeros(1, 8, device="cuda:0"), torch.zeros(1, 2, 20, device="cuda:0")
        for bad in (None, w.data_ptr(), w.cpu().numpy()):
            with pytest.raises(tw.kvc.KvcError) as e:
                tw.gpu.attn_weight(0, [0], [1], q, z, bad, 0.1)
            assert e.value.status == tw.kvc.KVC_EINVAL
            with pytest.raises(tw.kvc.KvcError) as e:
                tw.gpu.evict_weight(0, 0, -1, 3, bad)
            assert e.value.status == tw.kvc.KVC_EINVAL
        assert tw.gpu.n_tokens(0) == 20
    finally:
        tw.close()
