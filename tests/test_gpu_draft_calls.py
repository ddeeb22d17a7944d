"""The calls of a drafted block's step among others: queued without waits, over pages that change hands, on streams of two
contexts, beside the sequence operations; against contexts that are waited for after every call."""
import numpy as np
import pytest

import oracle

pytestmark = pytest.mark.gpu

KINDS = {"q8": (oracle.Q8_0, oracle.Q8_0), "f16": (oracle.F16, oracle.F16), "q8q4": (oracle.Q8_0, oracle.Q4_0)}


def _cache(kind, D, n_ctx, n_seq=1, layers=1, page=16, H=8, Hk=2):
    from kv_cache_decode_flash_gb300 import kvc

    tk, tv = KINDS[kind]
    return kvc.KVCache(layers, H, Hk, D, n_ctx, n_seq, tk, tv, page_rows=page)


def _draws(rng, T, H, Hk, D, dtype):
    import torch

    return torch.from_numpy(rng.standard_normal((T, H + 2 * Hk, D)).astype(np.float32)).to("cuda:0", dtype)


class Steps:
    """Drafted steps of one or more sequences: the same draws for every cache that runs them."""

    def __init__(self, cache, seed, D, dtype, wait, H=8, Hk=2, layers=1):
        import torch

        self.torch, self.c, self.rng, self.D, self.dtype, self.wait = torch, cache, np.random.default_rng(seed), D, dtype, wait
        self.H, self.Hk, self.L = H, Hk, layers
        self.outs, self.held = [], []

    def done(self):
        if self.wait:
            self.torch.cuda.synchronize()

    def step(self, ids, start, most=12, decode=True):
        torch, rng, H, Hk, D = self.torch, self.rng, self.H, self.Hk, self.D
        n_tok = [int(rng.integers(1, most)) for _ in ids]
        par = [np.array([-1 if t == 0 else rng.integers(max(-1, t - 4), t) for t in range(n)], np.int32) for n in n_tok]
        pos, path = [], []
        for i, p in zip(ids, par):
            d = []
            for u in p:
                d.append(0 if u < 0 else d[u] + 1)
            pos += [start[i] + x for x in d]
            at, chain = int(np.argmax(d)), []
            while at >= 0:
                chain.append(at)
                at = int(p[at])
            path.append(chain[::-1])
        parent = torch.from_numpy(np.concatenate(par)).to("cuda:0")
        for layer in range(self.L):
            x = _draws(rng, sum(n_tok), H, Hk, D, self.dtype)
            q = torch.empty(sum(n_tok), H, D, device="cuda:0", dtype=self.dtype)
            o = torch.empty_like(q)
            self.done()
            self.c.append_rope(layer, ids, n_tok, pos, x[:, :H], x[:, H:H + Hk], x[:, H + Hk:], q)
            self.done()
            self.c.attn_tree(layer, ids, n_tok, q, o, 0.11, parent=parent)
            self.done()
            self.outs.append(o)
            self.held.append((x, q, parent))
        self.c.keep(ids, n_tok, path)
        self.done()
        for i, p in zip(ids, path):
            start[i] += len(p)
        if decode:  # the next kernels start under the end of those before them and read rows that were just moved
            for layer in range(self.L):
                k, v, q = (torch.from_numpy(rng.standard_normal((len(ids), h, D)).astype(np.float32)).to("cuda:0")
                           for h in (Hk, Hk, H))
                o = torch.empty_like(q)
                self.done()
                self.c.decode_step(layer, ids, [start[i] for i in ids], k, v, q, o, 0.11)
                self.done()
                self.c.attn_decode(layer, ids, q, o, 0.11)
                self.done()
                self.outs.append(o)
                self.held.append((k, v, q))
            for i in ids:
                start[i] += 1


@pytest.mark.parametrize("kind,D", [("q8", 128), ("f16", 64), ("q8q4", 128)])
@pytest.mark.parametrize("n_seq,page", [(1, 16), (3, 64)])
def test_queued_steps_are_the_waited_for_ones(kind, D, n_seq, page):
    """Forty steps queued at once, with moves, pages that come and go and the fused decode step behind them, bit for bit."""
    import torch

    runs = []
    for wait in (True, False):
        c = _cache(kind, D, 3000, n_seq, layers=2, page=page)
        try:
            s = Steps(c, 5, D, torch.bfloat16, wait, layers=2)
            start = [0] * n_seq
            for _ in range(40):
                s.step(list(range(n_seq)), start)
            torch.cuda.synchronize()
            from kv_cache_decode_flash_gb300 import kvc

            assert kvc.kvc_check_device_error(c.ctx) == 0
            runs.append((s.outs, [c.state_get(i, -1, -1) for i in range(n_seq)]))
            for i in range(n_seq):
                assert list(c.positions(i)) == list(range(start[i]))
        finally:
            c.close()
    assert len(runs[0][0]) == len(runs[1][0])
    for a, b in zip(runs[0][0], runs[1][0]):
        assert bool((a == b).all()) and bool(torch.isfinite(a.float()).all())
    assert runs[0][1] == runs[1][1]


def test_pages_that_change_hands():
    """Two sequences take each other's freed pages: the device's table follows, whichever call had written it."""
    import torch

    from kv_cache_decode_flash_gb300 import kvc

    c = _cache("f16", 64, 96, 2, page=16)
    rng = np.random.default_rng(3)
    want = [[], []]  # the values appended, by sequence
    nxt = [0, 0]
    try:
        def add(i, n, plain):
            x = _draws(rng, n, 8, 2, 64, torch.float16)
            k, v = x[:, 8:10].contiguous(), x[:, 10:].contiguous()
            if plain:
                c.append(0, i, nxt[i], k.float(), v.float())
            else:
                c.append_rope(0, [i], [n], [0] * n, None, k, v, None)  # (position 0: nothing turns)
            want[i] += list(v.cpu().numpy())
            nxt[i] += n

        def drop(i, n):
            c.keep([i], [n], [[]])
            del want[i][len(want[i]) - n:]
            nxt[i] -= n

        for turn in range(60):
            i = int(rng.integers(0, 2))
            room = 90 - len(want[0]) - len(want[1])
            n = int(rng.integers(1, 30))
            if n <= room:
                add(i, n, bool(rng.integers(0, 2)))
            if len(want[1 - i]):
                drop(1 - i, int(rng.integers(1, len(want[1 - i]) + 1)))
            if turn % 7 == 3 and len(want[i]) > 3:  # the synchronous operations send the table too
                blob = c.state_get(i, -1, -1)
                c.seq_rm(i, -1, -1)
                c.state_set(i, blob)
            for j in range(2):
                if not want[j]:
                    continue
                # what the kernels see: a query of zeros weighs every row alike
                q = torch.zeros(1, 8, 64, device="cuda:0")
                o = torch.empty_like(q)
                c.attn_tree(0, [j], [1], q, o, 1.0)
                mean = np.mean(np.array(want[j], np.float64), 0)
                assert np.abs(o[0].double().cpu().numpy() - np.repeat(mean, 4, 0)).max() <= 2.0**-18, (turn, j)
        torch.cuda.synchronize()
        assert kvc.kvc_check_device_error(c.ctx) == 0
    finally:
        c.close()


def test_two_contexts_on_two_streams():
    """Steps of two contexts side by side on streams of their own give what each gives alone."""
    import torch

    def alone(kind, seed):
        c = _cache(kind, 128, 2000)
        s = Steps(c, seed, 128, torch.float16, True)
        start = [0]
        for _ in range(12):
            s.step([0], start)
        return c, s

    refs = [alone("q8", 1), alone("f16", 2)]
    caches = [_cache("q8", 128, 2000), _cache("f16", 128, 2000)]
    try:
        runs, starts = [Steps(c, i + 1, 128, torch.float16, False) for i, c in enumerate(caches)], [[0], [0]]
        streams = [torch.cuda.Stream() for _ in caches]
        torch.cuda.synchronize()
        for _ in range(12):
            for s, st, start in zip(runs, streams, starts):
                with torch.cuda.stream(st):
                    s.step([0], start)
        torch.cuda.synchronize()
        for (_, ref), s in zip(refs, runs):
            assert len(ref.outs) == len(s.outs)
            for a, b in zip(ref.outs, s.outs):
                assert bool((a == b).all())
    finally:
        for c in caches + [r[0] for r in refs]:
            c.close()


@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_a_whole_step_captured_and_replayed(act):
    """Append, tree attention and keep of two layers in one graph that leaves the sequence as it found it: replays give what
    eager calls give for the tensors' contents of the moment."""
    import torch

    dtype = {"bf16": torch.bfloat16, "f32": torch.float32}[act]
    rng = np.random.default_rng(4)
    H, Hk, D, T, L = 8, 2, 128, 10, 2
    c = _cache("q8", D, 700, layers=L, page=64)
    try:
        base = _draws(rng, 300, H, Hk, D, dtype)
        for layer in range(L):
            c.append_rope(layer, [0], [300], np.arange(300, dtype=np.int32), None, base[:, H:H + Hk], base[:, H + Hk:], None)
        par = torch.tensor([-1, 0, 0, 1, 1, 2, 3, -1, 7, 6], dtype=torch.int32, device="cuda:0")
        pos = np.array([300, 301, 301, 302, 302, 302, 303, 300, 301, 304], np.int32)
        live = torch.empty(L, T, H + 2 * Hk, D, device="cuda:0", dtype=dtype)
        q, out, after = (torch.empty(L, n, H, D, device="cuda:0", dtype=dtype) for n in (T, T, 1))
        probe = _draws(rng, 1, H, 0, D, dtype)

        def step():
            for layer in range(L):
                x = live[layer]
                c.append_rope(layer, [0], [T], pos, x[:, :H], x[:, H:H + Hk], x[:, H + Hk:], q[layer])
                c.attn_tree(layer, [0], [T], q[layer], out[layer], 0.0884, parent=par)
            c.keep([0], [T], [[0, 1, 3, 6, 9]])
            for layer in range(L):
                c.attn_tree(layer, [0], [1], probe, after[layer], 0.0884)
            c.keep([0], [5], [[]])

        draws = [_draws(rng, L * T, H, Hk, D, dtype).view(L, T, H + 2 * Hk, D) for _ in range(3)]
        want = []
        for x in draws:
            live.copy_(x)
            step()
            want.append([t.clone() for t in (q, out, after)])
        st = torch.cuda.Stream()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            step()
        for i in (1, 0, 2, 2):
            live.copy_(draws[i])
            torch.cuda.synchronize()
            with torch.cuda.stream(st):
                g.replay()
            torch.cuda.synchronize()
            for a, b in zip((q, out, after), want[i]):
                assert bool((a == b).all())
        assert c.n_tokens(0) == 300
    finally:
        c.close()


def test_steps_beside_the_sequence_operations():
    """Removal, shifts, copies, eviction by weight and export between drafted steps, against a cache that got the same rows by
    plain appends in the order that they ended up in."""
    import torch

    c = _cache("f16", 64, 900, 2, page=32)
    rng = np.random.default_rng(8)
    try:
        s = Steps(c, 3, 64, torch.float16, False)
        start = [0, 0]
        for _ in range(15):
            s.step([0], start, decode=False)
        n = c.n_tokens(0)
        assert list(c.positions(0)) == list(range(n)) and n == start[0]
        c.seq_rm(0, 3, 9)
        c.seq_add(0, 9, -1, -6)
        start[0] = n - 6
        assert list(c.positions(0)) == list(range(n - 6))
        w = torch.rand(2, 900, device="cuda:0")
        c.evict_weight(0, 2, -1, 5, w)
        for _ in range(6):  # rows are out of position order from here on; the steps do not mind
            s.step([0], start, decode=False)
        left = c.n_tokens(0)
        blob = c.state_get(0, -1, -1)
        c.seq_cp(0, 1, -1, -1)
        q = torch.from_numpy(rng.standard_normal((2, 8, 64)).astype(np.float32)).to("cuda:0")
        o = torch.empty_like(q)
        c.attn_tree(0, [0, 1], [1, 1], torch.cat([q[:1], q[:1]]), o, 0.125)
        torch.cuda.synchronize()
        assert bool((o[0] == o[1]).all()) and c.n_tokens(1) == left
        d = _cache("f16", 64, 900, 1, page=16)
        try:
            d.state_set(0, blob)
            o2 = torch.empty_like(q[:1])
            d.attn_decode(0, [0], q[:1], o2, 0.125)
            torch.cuda.synchronize()
            assert float((o2[0] - o[0]).abs().max()) <= 2e-6
        finally:
            d.close()
    finally:
        c.close()
