"""Rows as a model's projections leave them into the cache (kvc_append_rope), the rows that stay of a drafted block
(kvc_seq_keep), and a block's whole step, against plain 64-bit forms."""
import math

import numpy as np
import pytest

import oracle
from draft_ref import EPS_OF, attend, attend_bound, stored, tree_sees, turned

pytestmark = pytest.mark.gpu

Q8, F16, Q4 = oracle.Q8_0, oracle.F16, oracle.Q4_0
KINDS = {"q8": (Q8, Q8), "f16": (F16, F16), "q8q4": (Q8, Q4)}
EPS = 1e-6


def _types():
    import torch

    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def _cache(kind, H, Hk, D, n_ctx, n_seq=1, layers=1, page=64, base=10000.0, neox=True):
    from kv_cache_decode_flash_gb300 import kvc

    tk, tv = KINDS[kind]
    return kvc.KVCache(layers, H, Hk, D, n_ctx, n_seq, tk, tv, base, kvc.KVC_ROPE_NEOX if neox else kvc.KVC_ROPE_NORM,
                       page_rows=page)


def _rows(rng, T, H, Hk, D, act, fused=True, sigma=1.0):
    """Queries, keys and values as one projection leaves them, or apart."""
    import torch

    x = torch.from_numpy((rng.standard_normal((T, H + 2 * Hk, D)) * sigma).astype(np.float32)).to("cuda:0", _types()[act])
    parts = x.split([H, Hk, Hk], 1)
    return parts if fused else [p.contiguous() for p in parts]


def _weights(rng, D):
    import torch

    return torch.from_numpy((1 + 0.2 * rng.standard_normal(D)).astype(np.float32)).to("cuda:0")


def _np(t):
    return t.double().cpu().numpy()


def _check_rows(got, step, want, slack, kind):
    """Stored values [Hk][T][D] against want [T][Hk][D], computed within `slack` of it before they are rounded."""
    want, slack = want.transpose(1, 0, 2), slack.transpose(1, 0, 2)
    if kind == F16:
        # half a step, 2^-11 of the value or half of the smallest subnormal
        bound = slack + np.maximum(np.abs(want) * 2.0**-11, 2.0**-25) * (1 + 2.0**-8)
    elif kind == Q8:
        # half a step of the code; the scale's rounding to fp16 (2^-11 of the value, or of 127 codes at 2^-25 each); d is off
        # by the slack of the block's largest value, which half a step takes in with 1 + 2^-8
        bound = slack + step * (0.5 + 2.0**-8) + np.abs(want) * 2.0**-11 + 127 * 2.0**-25
    else:
        # trunc(x / d + 8.5) - 8 is off by half a step, by a whole one where 16 is cut to 15
        bound = slack + step * (1 + 2.0**-6) + np.abs(want) * 2.0**-11 + 8 * 2.0**-25
    err = np.abs(got - want)
    assert np.all(err <= bound), "rows off by %.3g, %.2f of their bound" % (err.max(), (err / bound).max())


def _call(c, layer, ids, n_tok, pos, qkv, qw=None, kw=None, out=None):
    import torch

    q, k, v = qkv
    out = torch.full((sum(n_tok), q.shape[1], q.shape[2]), float("nan"), device=q.device, dtype=q.dtype) if out is None else out
    c.append_rope(layer, ids, n_tok, pos, q, k, v, out, q_norm=qw, k_norm=kw, eps=EPS)
    torch.cuda.synchronize()
    from kv_cache_decode_flash_gb300 import kvc

    assert kvc.kvc_check_device_error(c.ctx) == 0
    return out


@pytest.mark.parametrize("act", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("kind,D", [("q8", 64), ("f16", 64), ("q8", 128), ("f16", 128), ("q8q4", 128)])
@pytest.mark.parametrize("T,H,Hk,norm,neox,fused", [(1, 10, 2, True, True, True), (1, 7, 7, False, False, True),
                                                    (37, 8, 1, True, False, False), (130, 6, 2, False, True, True),
                                                    (3, 9, 3, True, True, False)])
def test_append_rope_types_and_shapes(kind, D, act, T, H, Hk, norm, neox, fused):
    """Odd head counts (a warp's last head-rows are not there), both pairings, strided and separate rows."""
    rng = np.random.default_rng(T + H)
    tk, tv = KINDS[kind]
    c = _cache(kind, H, Hk, D, 200, page=48, neox=neox)
    try:
        qkv = _rows(rng, T, H, Hk, D, act, fused)
        w = (_weights(rng, D), _weights(rng, D)) if norm else (None, None)
        pos = rng.integers(0, 5000, T).astype(np.int32)
        out = _call(c, 0, [0], [T], pos, qkv, *w)
        y, s = turned(_np(qkv[0]), pos, 10000.0, neox, _np(w[0]) if norm else None, EPS)
        assert np.all(np.abs(_np(out) - y) <= s * (1 + 2.0**-7) + np.abs(y) * EPS_OF[act] + 2.0**-25)
        p, layers = stored(c.state_get(0, -1, -1), 1, Hk, D, tk, tv)
        assert list(p) == list(pos) and list(c.positions(0)) == list(pos)
        k, ks, v, vs = layers[0]
        yk, sk = turned(_np(qkv[1]), pos, 10000.0, neox, _np(w[1]) if norm else None, EPS)
        _check_rows(k, ks, yk, sk, tk)
        _check_rows(v, vs, _np(qkv[2]), np.zeros_like(sk), tv)
    finally:
        c.close()


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("base", [10000.0, 1000000.0])
def test_append_rope_far_positions(act, base):
    """Angles of positions up to 2^31 - 1 keep their 32 bits (the 64-bit form's own are off by 2^-22 there)."""
    H, Hk, D = 4, 2, 128
    pos = np.array([0, 1, 2**20 - 1, 2**20, 1500000, 2**24 + 1, 2**30 + 12345, 2**31 - 1], np.int32)
    rng = np.random.default_rng(3)
    c = _cache("f16", H, Hk, D, 100, base=base)
    try:
        qkv = _rows(rng, len(pos), H, Hk, D, act)
        out = _call(c, 0, [0], [len(pos)], pos, qkv)
        y, s = turned(_np(qkv[0]), pos, base, True)
        # pos * theta in 64 bits is off by half a unit of 2^-53 relatively, and theta by one: 3 x 2^-54 of the angle
        far = (pos.astype(np.float64) * 3 * 2.0**-54)[:, None, None] * (s / (24 * 2.0**-24))
        assert np.all(np.abs(_np(out) - y) <= s * (1 + 2.0**-7) + far + np.abs(y) * EPS_OF[act] + 2.0**-25)
    finally:
        c.close()


@pytest.mark.parametrize("kind,D", [("q8", 64), ("f16", 64), ("q8", 128), ("f16", 128), ("q8q4", 128)])
@pytest.mark.parametrize("neox", [True, False])
def test_append_rope_without_turn_is_the_plain_append(kind, D, neox):
    """Position 0, no norm: the stored bytes are kvc_append's and the queries come back as they were."""
    import torch

    H, Hk, T = 6, 3, 90
    rng = np.random.default_rng(5)
    a, b = _cache(kind, H, Hk, D, 200, page=32, neox=neox), _cache(kind, H, Hk, D, 200, page=32, neox=neox)
    try:
        x = rng.standard_normal((T, H + 2 * Hk, D)).astype(np.float32)
        x[3], x[4, :, :40], x[5] = 0, 0, 1e-30
        x[6] *= 1e4
        x = torch.from_numpy(x).to("cuda:0")
        qkv = x.split([H, Hk, Hk], 1)
        for act in ("f32", "f16"):
            rows = [p.to(_types()[act]) for p in qkv]
            out = _call(a, 0, [0], [T], np.zeros(T, np.int32), rows)
            assert bool((out == rows[0]).all())
            for t in range(T):  # (one position at a time: its positions are consecutive)
                b.append(0, 0, 0, rows[1][t:t + 1].float().contiguous(), rows[2][t:t + 1].float().contiguous())
            assert a.state_get(0, -1, -1) == b.state_get(0, -1, -1)
            a.seq_rm(0, -1, -1)
            b.seq_rm(0, -1, -1)
    finally:
        a.close()
        b.close()


def test_append_rope_turn_is_seq_adds():
    """Rows turned to p on the way in, and rows put in at 0 and moved to p by kvc_seq_add, differ by roundings only."""
    H, Hk, D, T, delta = 4, 2, 128, 50, 777
    rng = np.random.default_rng(6)
    a, b = _cache("f16", H, Hk, D, 100), _cache("f16", H, Hk, D, 100)
    try:
        qkv = _rows(rng, T, H, Hk, D, "f16")
        _call(a, 0, [0], [T], np.arange(T) + delta, qkv)
        _call(b, 0, [0], [T], np.arange(T), qkv)
        b.seq_add(0, 0, -1, delta)
        (pa, (la,)), (pb, (lb,)) = (stored(c.state_get(0, -1, -1), 1, Hk, D, F16, F16) for c in (a, b))
        assert list(pa) == list(pb)
        # two roundings to f16 (2^-11 of values of at most |a| + |b| <= 1.42 x the pair's length) against one
        size = np.sqrt(la[0][..., :64] ** 2 + la[0][..., 64:] ** 2)
        assert np.all(np.abs(la[0] - lb[0]) <= np.concatenate([size, size], -1) * 3.5 * 2.0**-11)
        assert np.array_equal(la[2], lb[2])
    finally:
        a.close()
        b.close()


@pytest.mark.parametrize("kind", ["q8", "f16"])
def test_append_rope_batch_over_pages_and_layers(kind):
    """A ragged batch in two layers after other rows, one sequence's first row inside its page, one without tokens, small
    pages; then the same tokens' attention over the tree, and a second block behind it."""
    H, Hk, D, L = 8, 2, 64, 2
    tk, tv = KINDS[kind]
    rng = np.random.default_rng(8)
    c = _cache(kind, H, Hk, D, 600, n_seq=4, layers=L, page=16)
    try:
        import torch

        before = [0, 40, 33, 7]
        for i, n in enumerate(before):
            if n:
                for l in range(L):
                    k = torch.randn(n, Hk, D, device="cuda:0", generator=torch.Generator("cuda:0").manual_seed(10 * i + l))
                    c.append(l, i, 0, k, k * 2)
        c.seq_rm(1, 0, 5)
        had = [stored(c.state_get(i, -1, -1), L, Hk, D, tk, tv) if n else None for i, n in enumerate(before)]
        ids = [2, 0, 3, 1]
        for block in range(2):
            n_tok = [[5, 19, 0, 37], [1, 2, 30, 3]][block]
            T = sum(n_tok)
            pos = np.concatenate([100 * block + rng.integers(0, 90, t) for t in n_tok]).astype(np.int32)
            for l in range(L):
                qkv = _rows(rng, T, H, Hk, D, "bf16")
                out = _call(c, l, ids, n_tok, pos, qkv)
                y, s = turned(_np(qkv[0]), pos, 10000.0, True)
                assert np.all(np.abs(_np(out) - y) <= s * (1 + 2.0**-7) + np.abs(y) * EPS_OF["bf16"] + 2.0**-25)
                yk, sk = turned(_np(qkv[1]), pos, 10000.0, True)
                if l + 1 < L:
                    kept = (yk, sk, _np(qkv[2]))
                    with pytest.raises(Exception) as e:  # a layer's rows are missing
                        c.keep(ids, n_tok, [[] for _ in ids])
                    assert "sync" in str(e.value)
            t0 = 0
            for i, t in zip(ids, n_tok):
                p, layers = stored(c.state_get(i, -1, -1), L, Hk, D, tk, tv)
                m = 0 if had[i] is None else len(had[i][0])
                assert list(p[m:]) == list(pos[t0:t0 + t]) and (m == 0 or list(p[:m]) == list(had[i][0]))
                for l, (k, ks, v, vs) in enumerate(layers):
                    a, b, w = kept if l == 0 else (yk, sk, _np(qkv[2]))
                    step = [None if x is None else x[:, m:] for x in (ks, vs)]
                    _check_rows(k[:, m:], step[0], a[t0:t0 + t], b[t0:t0 + t], tk)
                    _check_rows(v[:, m:], step[1], w[t0:t0 + t], np.zeros_like(w[t0:t0 + t]), tv)
                    if m:  # the rows before the block are as they were
                        assert np.array_equal(k[:, :m], had[i][1][l][0]) and np.array_equal(v[:, :m], had[i][1][l][2])
                had[i] = (p, layers)
                t0 += t
    finally:
        c.close()


def test_append_rope_many_sequences_and_listed_positions():
    """More sequences than a launch carries, and more positions that are no run than one lists."""
    H, Hk, D = 2, 1, 64
    rng = np.random.default_rng(9)
    n_tok = [1 + int(rng.integers(0, 12)) for _ in range(150)]
    n_tok[20], n_tok[70], n_tok[71] = 700, 400, 0
    T = sum(n_tok)
    c = _cache("f16", H, Hk, D, T, n_seq=150, page=16)
    try:
        pos = np.concatenate([np.arange(t) + 3 if i % 3 == 0 else rng.integers(0, 4000, t) for i, t in enumerate(n_tok)]).astype(np.int32)
        ids = [int(i) for i in rng.permutation(150)]
        qkv = _rows(rng, T, H, Hk, D, "f32")
        out = _call(c, 0, ids, n_tok, pos, qkv)
        y, s = turned(_np(qkv[0]), pos, 10000.0, True)
        assert np.all(np.abs(_np(out) - y) <= s * (1 + 2.0**-7) + np.abs(y) * EPS_OF["f32"] + 2.0**-25)
        yk, sk = turned(_np(qkv[1]), pos, 10000.0, True)
        t0 = 0
        for i, t in zip(ids, n_tok):
            if t:
                p, ((k, ks, v, vs),) = stored(c.state_get(i, -1, -1), 1, Hk, D, F16, F16)
                assert list(p) == list(pos[t0:t0 + t])
                _check_rows(k, ks, yk[t0:t0 + t], sk[t0:t0 + t], F16)
            t0 += t
    finally:
        c.close()


def test_append_rope_in_place_without_queries_and_behind_the_last_token():
    import torch

    H, Hk, D, T = 4, 2, 128, 9
    rng = np.random.default_rng(10)
    c = _cache("q8", H, Hk, D, 100)
    try:
        pos = np.arange(T, dtype=np.int32)
        q, k, v = _rows(rng, T, H, Hk, D, "bf16", fused=False)
        apart = _call(c, 0, [0], [T], pos, (q, k, v))
        blob = c.state_get(0, -1, -1)
        c.seq_rm(0, -1, -1)
        room = torch.full((T + 3, H, D), 7.0, device=q.device, dtype=q.dtype)
        _call(c, 0, [0], [T], pos, (q, k, v), out=room)
        assert bool((room[:T] == apart).all()) and bool((room[T:] == 7.0).all())
        c.seq_rm(0, -1, -1)
        _call(c, 0, [0], [T], pos, (q, k, v), out=q)  # in place
        assert bool((q == apart).all()) and c.state_get(0, -1, -1) == blob
        c.seq_rm(0, -1, -1)
        c.append_rope(0, [0], [T], pos, None, k, v, None)
        assert c.state_get(0, -1, -1) == blob
    finally:
        c.close()


def test_append_rope_zero_rows_and_large_values():
    """Rows of zeros stay zeros under a norm; values at the ends of the types' ranges."""
    import torch

    H, Hk, D = 2, 1, 64
    c = _cache("f16", H, Hk, D, 100)
    try:
        x = torch.zeros(4, H + 2 * Hk, D, device="cuda:0")
        x[1] = 3e4
        x[2, :, ::2] = 1e-20
        x[3, :, 5] = 1e15
        w = torch.ones(D, device="cuda:0")
        qkv = x.split([H, Hk, Hk], 1)
        pos = np.arange(4, dtype=np.int32)
        out = _call(c, 0, [0], [4], pos, qkv, w, w)
        y, s = turned(_np(qkv[0]), pos, 10000.0, True, np.ones(D), EPS)
        assert np.all(np.abs(_np(out) - y) <= s * (1 + 2.0**-7) + np.abs(y) * 2.0**-24 + 2.0**-140)
        assert bool((out[0] == 0).all())
    finally:
        c.close()


def test_append_rope_in_a_graph_on_another_stream():
    """A captured append and its block's attention: a replay writes the same cells from what the tensors hold then."""
    import torch

    H, Hk, D, T = 8, 2, 64, 6
    rng = np.random.default_rng(12)
    c = _cache("q8", H, Hk, D, 200)
    ref = _cache("q8", H, Hk, D, 200)
    try:
        first = [_rows(rng, 50, H, Hk, D, "bf16") for _ in range(1)][0]
        for x in (c, ref):
            _call(x, 0, [0], [50], np.arange(50), first)
        probe = first[0][:1].contiguous()
        c.attn_tree(0, [0], [1], probe, torch.empty_like(probe), 0.125)  # (the work space)
        pos = np.array([50, 51, 51, 52, 52, 53], np.int32)
        blocks = [_rows(rng, T, H, Hk, D, "bf16", fused=False) for _ in range(3)]
        par = torch.tensor([-1, 0, 0, 1, 2, 3], dtype=torch.int32, device="cuda:0")
        live = [b.clone() for b in blocks[0]]
        q_out, out = torch.empty_like(live[0]), torch.empty_like(live[0])
        st = torch.cuda.Stream()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            c.append_rope(0, [0], [T], pos, *live, q_out)
            c.attn_tree(0, [0], [T], q_out, out, 0.125, parent=par)
        for b in (1, 2, 0):
            for dst, src in zip(live, blocks[b]):
                dst.copy_(src)
            torch.cuda.synchronize()
            with torch.cuda.stream(st):
                g.replay()
            torch.cuda.synchronize()
            want_q = _call(ref, 0, [0], [T], pos, blocks[b])
            want = torch.empty_like(want_q)
            ref.attn_tree(0, [0], [T], want_q, want, 0.125, parent=par)
            torch.cuda.synchronize()
            assert bool((q_out == want_q).all()) and bool((out == want).all())
            assert c.state_get(0, -1, -1) == ref.state_get(0, -1, -1)
            ref.keep([0], [T], [[]])
    finally:
        c.close()
        ref.close()


def test_append_rope_refusals():
    import torch

    from kv_cache_decode_flash_gb300 import kvc

    H, Hk, D, T = 4, 2, 64, 5
    c = _cache("q8", H, Hk, D, 64, n_seq=2, layers=2, page=16)
    try:
        rng = np.random.default_rng(4)
        q, k, v = _rows(rng, T, H, Hk, D, "f32", fused=False)
        w = _weights(rng, D)
        out = torch.empty_like(q)
        pos = list(range(T))
        ok = dict(layer=0, seq_ids=[0], n_tok=[T], pos=pos, act=0, q=q, q_stride=H * D, k=k, k_stride=Hk * D, v=v,
                  v_stride=Hk * D, q_out=out, q_norm=w, k_norm=w, eps=1e-6)
        inval = [dict(layer=2), dict(layer=-1), dict(seq_ids=[2]), dict(seq_ids=[-1]), dict(seq_ids=[0, 0], n_tok=[2, 3]),
                 dict(n_tok=[-1]), dict(act=3), dict(k=None), dict(v=None), dict(q_out=None), dict(q=None),
                 dict(q=q.data_ptr() + 4), dict(k=k.data_ptr() + 8), dict(v=v.data_ptr() + 4), dict(q_out=out.data_ptr() + 8),
                 dict(q_norm=w.data_ptr() + 4), dict(k_norm=w.data_ptr() + 8), dict(q_stride=H * D - 4), dict(k_stride=Hk * D + 2),
                 dict(v_stride=-Hk * D), dict(q_stride=2**40), dict(eps=-1.0), dict(eps=float("nan")), dict(q_out=q.data_ptr() + 16),
                 dict(q_out=k), dict(q_out=v), dict(q_out=q, q_stride=2 * H * D, n_tok=[2]), dict(seq_ids=[], n_tok=[]),
                 dict(n_tok=[2**31 - 1], pos=np.zeros(0, np.int32))]
        for b in inval:
            with pytest.raises(kvc.KvcError) as e:
                kvc.kvc_append_rope(c.ctx, **{**ok, **b})
            assert e.value.status == kvc.KVC_EINVAL, b
        for b, status in ((dict(pos=[0, 1, 2, 3, -1]), kvc.KVC_ERANGE), (dict(pos=[0, 1, 2, 3, 2**31]), kvc.KVC_ERANGE),
                          (dict(pos=[0, 1]), kvc.KVC_EINVAL)):
            with pytest.raises(kvc.KvcError) as e:
                kvc.kvc_append_rope(c.ctx, **{**ok, **b})
            assert e.value.status == status, b
        assert c.n_tokens(0) == 0 and c.stats()["pages_free"] == c.stats()["pages_total"]
        kvc.kvc_append_rope(c.ctx, **{**ok, "n_tok": [0], "pos": []})  # no tokens: nothing to do
        kvc.kvc_append_rope(c.ctx, **ok)
        # the other layer must append the same positions, and no more of them
        for b in (dict(layer=1, pos=[0, 1, 2, 3, 5]), dict(layer=1, seq_ids=[1, 0], n_tok=[1, 4], pos=[0, 1, 2, 3, 4])):
            with pytest.raises(kvc.KvcError) as e:
                kvc.kvc_append_rope(c.ctx, **{**ok, **b})
            assert e.value.status == kvc.KVC_EINVAL, b
        assert c.n_tokens(1) == 0  # (its part of the call did not happen either)
        kvc.kvc_append_rope(c.ctx, **{**ok, "layer": 1})
        # no room: nothing happens to either sequence
        big = 100
        qb, kb, vb = _rows(rng, big + 1, H, Hk, D, "f32", fused=False)
        with pytest.raises(kvc.KvcError) as e:
            c.append_rope(0, [1, 0], [1, big], np.arange(big + 1), qb, kb, vb, torch.empty_like(qb))
        assert e.value.status == kvc.KVC_ENOSPC
        assert c.n_tokens(1) == 0 and c.n_tokens(0) == T
        good = dict(layer=0, seq_ids=[0], n_tok=[T], pos=pos, q=q, k=k, v=v, q_out=out)
        for b in (dict(q=q.half()), dict(k=k.double()), dict(q=q.cpu()), dict(q_out=out.half()), dict(k=k.transpose(1, 2)),
                  dict(v=v[:, :1]), dict(k=k[:3]), dict(q=None), dict(q_norm=w.half()), dict(k_norm=w[:32]), dict(k=k[..., ::2])):
            with pytest.raises(kvc.KvcError) as e:
                c.append_rope(**{**good, **b})
            assert e.value.status == kvc.KVC_EINVAL, b
        host = kvc.KVCache(1, H, Hk, D, 512, residency=kvc.KVC_HOST_PINNED)
        try:
            with pytest.raises(kvc.KvcError) as e:
                host.append_rope(**good)
            assert e.value.status == kvc.KVC_EINVAL
            with pytest.raises(kvc.KvcError) as e:
                host.keep([0], [0], [[]])
            assert e.value.status == kvc.KVC_EINVAL
        finally:
            host.close()
    finally:
        c.close()


# ------------------------------------------------------------------ keep --
def _pair(kind, D, lens, layers=2, page=16):
    """A cache with rows of every sequence, and its exported states."""
    import torch

    c = _cache(kind, 4, 2, D, sum(lens) + 64, n_seq=len(lens), layers=layers, page=page)
    for i, n in enumerate(lens):
        for l in range(layers):
            gen = torch.Generator("cuda:0").manual_seed(100 * i + l)
            k = torch.randn(n, 2, D, device="cuda:0", generator=gen)
            v = torch.randn(n, 2, D, device="cuda:0", generator=gen)
            c.append(l, i, 10, k, v)
    return c


def _states(c, kind, D, layers, n):
    tk, tv = KINDS[kind]
    return [stored(c.state_get(i, -1, -1), layers, 2, D, tk, tv) for i in range(n)]


@pytest.mark.parametrize("kind,D", [("q8", 64), ("f16", 64), ("q8", 128), ("f16", 128), ("q8q4", 128)])
@pytest.mark.parametrize("page", [16, 64])
def test_keep_rows_of_a_block(kind, D, page):
    lens = [70, 200, 33, 64]
    c = _pair(kind, D, lens, page=page)
    try:
        c.seq_rm(1, 10, 23)  # a first row inside its page
        lens[1] -= 13
        before = _states(c, kind, D, 2, 4)
        rng = np.random.default_rng(D)
        ids, last = [3, 0, 1], [64, 20, 100]
        keep = [[0, 1, 2, 30, 31, 63], [], sorted(rng.choice(100, 60, replace=False).tolist())]
        c.keep(ids, last, keep)
        after = _states(c, kind, D, 2, 4)
        for i in range(4):
            order = list(range(lens[i]))
            if i in ids:
                j = ids.index(i)
                base = lens[i] - last[j]
                order = order[:base] + [base + a for a in keep[j]]
            assert list(after[i][0]) == list(before[i][0][order])
            for a, b in zip(after[i][1], before[i][1]):
                assert np.array_equal(a[0], b[0][:, order]) and np.array_equal(a[2], b[2][:, order])
        pages = c.stats()
        assert pages["pages_free"] == pages["pages_total"] - sum(
            -(-(len(after[i][0]) + (13 % page if i == 1 else 0)) // page) for i in range(4))
    finally:
        c.close()


def test_keep_all_none_and_long_lists():
    lens = [1500, 40]
    c = _pair("q8", 64, lens, layers=1)
    try:
        before = _states(c, "q8", 64, 1, 2)
        c.keep([0, 1], [1500, 0], [list(range(1500)), []])
        assert all(np.array_equal(a[1][0][0], b[1][0][0]) for a, b in zip(_states(c, "q8", 64, 1, 2), before))
        odd = list(range(1, 1500, 2))  # more moves than a launch carries
        c.keep([0], [1500], [odd])
        (p, ((k, _, v, _),)) = _states(c, "q8", 64, 1, 1)[0]
        assert list(p) == [10 + i for i in odd]
        assert np.array_equal(k, before[0][1][0][0][:, odd]) and np.array_equal(v, before[0][1][0][2][:, odd])
        c.keep([0, 1], [750, 40], [[], [39]])
        assert c.n_tokens(0) == 0 and list(c.positions(1)) == [49]
    finally:
        c.close()


def test_keep_restores_position_order():
    """A drafted block with shared positions, then its accepted path: position ranges work again as for a plain sequence."""
    c = _cache("f16", 4, 2, 64, 400, layers=1)
    try:
        rng = np.random.default_rng(2)
        _call(c, 0, [0], [100], np.arange(100), _rows(rng, 100, 4, 2, 64, "f16"))
        _call(c, 0, [0], [6], np.array([100, 101, 101, 102, 102, 103]), _rows(rng, 6, 4, 2, 64, "f16"))
        c.keep([0], [6], [[0, 2, 4, 5]])
        assert list(c.positions(0)) == list(range(104))
        c.seq_rm(0, 0, 10)
        c.seq_add(0, 10, -1, -10)
        assert list(c.positions(0)) == list(range(94))
        with pytest.raises(Exception):
            c.keep([0], [3], [[2, 1]])
        assert c.n_tokens(0) == 94
    finally:
        c.close()


def test_keep_refusals():
    from kv_cache_decode_flash_gb300 import kvc

    c = _pair("q8", 64, [30, 5], layers=1)
    try:
        blob = [c.state_get(i, -1, -1) for i in range(2)]
        for a in (([2], [1], [[]]), ([-1], [1], [[]]), ([0, 0], [1, 1], [[], []]), ([0], [31], [[]]), ([0], [-1], [[]]),
                  ([0], [3], [[3]]), ([0], [3], [[-1]]), ([0], [3], [[1, 1]]), ([0], [3], [[2, 0]]), ([0], [1], [[0, 1]]),
                  ([0, 1], [3, 6], [[0], []]), ([], [], []), ([0], [1], [])):
            with pytest.raises(kvc.KvcError) as e:
                c.keep(*a)
            assert e.value.status == kvc.KVC_EINVAL, a
        assert [c.state_get(i, -1, -1) for i in range(2)] == blob
    finally:
        c.close()


# ------------------------------------------------------------------ step --
@pytest.mark.parametrize("kind,act,D,page", [("q8", "bf16", 128, 64), ("f16", "f16", 64, 16), ("q8q4", "bf16", 128, 16),
                                             ("q8", "f16", 64, 256)])
def test_drafted_steps_one_after_the_other(kind, act, D, page):
    """Several steps of a ragged batch: append, attention over the trees, the accepted paths stay, the next token's decode
    step behind them; everything against the plain forms over the rows that the cache holds then."""
    import torch

    H, Hk, L = 8, 2, 2
    tk, tv = KINDS[kind]
    rng = np.random.default_rng(31)
    lens = [90, 17, 300]
    c = _cache(kind, H, Hk, D, 1200, n_seq=3, layers=L, page=page)
    scale = float(np.float32(1 / math.sqrt(D)))
    try:
        w = _weights(rng, D), _weights(rng, D)
        for i, n in enumerate(lens):
            for l in range(L):
                _call(c, l, [i], [n], np.arange(n), _rows(rng, n, H, Hk, D, act), *w)
        nxt = list(lens)
        for step in range(4):
            n_tok = [int(rng.integers(1, 14)) for _ in lens]
            par = [np.array([-1 if t == 0 else rng.integers(max(-1, t - 4), t) for t in range(n)], np.int32) for n in n_tok]
            depth = []
            for p in par:
                d = []
                for t, u in enumerate(p):
                    d.append(0 if u < 0 else d[u] + 1)
                depth.append(d)
            pos = np.concatenate([nxt[i] + np.array(d) for i, d in enumerate(depth)]).astype(np.int32)
            parent = torch.from_numpy(np.concatenate(par)).to("cuda:0")
            outs = []
            for l in range(L):
                qkv = _rows(rng, sum(n_tok), H, Hk, D, act)
                q = torch.empty(sum(n_tok), H, D, device="cuda:0", dtype=_types()[act])
                o = torch.empty_like(q)
                c.append_rope(l, [0, 1, 2], n_tok, pos, *qkv, q, q_norm=w[0], k_norm=w[1], eps=EPS)
                c.attn_tree(l, [0, 1, 2], n_tok, q, o, scale, parent=parent)
                outs.append((q, o))
            torch.cuda.synchronize()
            state = [stored(c.state_get(i, -1, -1), L, Hk, D, tk, tv) for i in range(3)]
            for l, (q, o) in enumerate(outs):
                t0 = 0
                for i, t in enumerate(n_tok):
                    K, V = (state[i][1][l][j].transpose(1, 0, 2) for j in (0, 2))
                    want, mag, size = attend(_np(q)[t0:t0 + t], K, V, scale, tree_sees(par[i], len(K), t))
                    err = np.abs(_np(o)[t0:t0 + t] - want)
                    assert np.all(err <= attend_bound(mag, size, len(K), D, act)), (step, l, i, err.max())
                    t0 += t
            path = []
            for p, d in zip(par, depth):
                at, chain = int(np.argmax(d)), []
                while at >= 0:
                    chain.append(at)
                    at = int(p[at])
                path.append(chain[::-1])
            c.keep([0, 1, 2], n_tok, path)
            nxt = [n + len(p) for n, p in zip(nxt, path)]
            # the next token by the decode step, straight behind it on the stream
            for l in range(L):
                k1, v1, q1 = (torch.randn(3, h, D, device="cuda:0") for h in (Hk, Hk, H))
                o1 = torch.empty_like(q1)
                c.decode_step(l, [0, 1, 2], nxt, k1, v1, q1, o1, scale)
                outs[l] = (q1, o1)
            torch.cuda.synchronize()
            nxt = [n + 1 for n in nxt]
            for i in range(3):
                p, layers = stored(c.state_get(i, -1, -1), L, Hk, D, tk, tv)
                assert list(p) == list(range(nxt[i]))
                for l, (q1, o1) in enumerate(outs):
                    K, V = (layers[l][j].transpose(1, 0, 2) for j in (0, 2))
                    want, _, _ = attend(_np(q1)[i:i + 1], K, V, scale, np.ones((1, len(K)), bool))
                    assert np.abs(_np(o1)[i:i + 1] - want).max() <= 1e-3
                n = len(state[i][0]) - n_tok[i]
                order = list(range(n)) + [n + a for a in path[i]]
                for l in range(L):  # the rows that stayed are the rows that were there
                    for j in (0, 2):
                        assert np.array_equal(layers[l][j][:, :len(order)], state[i][1][l][j][:, order])
    finally:
        c.close()
