"""Entries of the device's page tables that captured, released and failed appends write or leave: whatever of these came
before, a call's rows reach the pages that the sequence has, and no other sequence's."""
import ctypes

import numpy as np
import pytest

import oracle

pytestmark = pytest.mark.gpu

H, Hk, D, PAGE = 4, 2, 64, 16


class Cache:
    """Two sequences of 16-bit rows in small pages; draws by number, so that two caches can be given the same ones."""

    def __init__(self, layers=1):
        import torch

        from kv_cache_decode_flash_gb300 import kvc

        self.torch, self.kvc = torch, kvc
        self.c = kvc.KVCache(layers, H, Hk, D, 192, 2, oracle.F16, oracle.F16, page_rows=PAGE)
        self.held = []

    def draw(self, number, n):
        x = np.random.default_rng(number).standard_normal((n, H + 2 * Hk, D)).astype(np.float32)
        t = self.torch.from_numpy(x).to("cuda:0", self.torch.float16)
        self.held.append(t)
        return t

    def rope(self, seq, x, pos0, q_out=None):
        n = len(x)
        self.c.append_rope(0, [seq], [n], list(range(pos0, pos0 + n)), None if q_out is None else x[:, :H], x[:, H:H + Hk],
                           x[:, H + Hk:], q_out)

    def plain(self, seq, x, pos0):
        k, v = x[:, H:H + Hk].float().contiguous(), x[:, H + Hk:].float().contiguous()
        self.held.append((k, v))
        return lambda: self.c.append(0, seq, pos0, k, v)

    def drop(self, seq, n):
        self.c.keep([seq], [n], [[]])

    def tree(self, seq, q, out):
        self.c.attn_tree(0, [seq], [len(q)], q, out, 0.125)

    def rows(self, number=99):
        """What either sequence's rows hold, and what the kernels find by the device's table: attention of one query."""
        q = self.draw(number, 1)[:, :H].contiguous()
        outs = []
        for seq in range(2):
            if self.c.n_tokens(seq):
                o = self.torch.empty_like(q)
                self.tree(seq, q, o)
                outs.append(o)
        self.torch.cuda.synchronize()
        assert self.kvc.kvc_check_device_error(self.c.ctx) == 0
        return [self.c.state_get(i, -1, -1) for i in range(2)], [o.cpu() for o in outs]

    def start(self):
        """Sequence 0 fills its first page; sequence 1 has five, the pool's first ones among them."""
        self.rope(1, self.draw(1, 5 * PAGE), 0)
        self.rope(0, self.draw(2, PAGE), 0)
        self.rows()  # (the work space, which no capture can allocate)
        return self

    def capture(self, fn):
        g, st = self.torch.cuda.CUDAGraph(), self.torch.cuda.Stream()
        self.torch.cuda.synchronize()
        with self.torch.cuda.graph(g, stream=st):
            fn()
        return g

    def step(self, x, q, out):
        """A drafted block on sequence 0 of which no row stays."""
        def run():
            self.rope(0, x, PAGE, q)
            self.tree(0, q, out)
            self.drop(0, len(x))
        return run


@pytest.fixture
def two():
    caches = [Cache(), Cache()]
    yield caches
    for c in caches:
        c.c.close()


def same(a, b):
    (sa, oa), (sb, ob) = a, b
    assert sa == sb
    assert len(oa) == len(ob) and all(bool((x == y).all()) for x, y in zip(oa, ob))


def buffers(c, n):
    q = c.torch.empty(n, H, D, device="cuda:0", dtype=c.torch.float16)
    c.held.append(q)
    return q, c.torch.full_like(q, float("nan"))


@pytest.mark.parametrize("how", ["rope", "plain"])
def test_an_eager_append_behind_a_captured_step_that_was_not_replayed(two, how):
    """The step takes a page and gives it back, in a capture; the page then is the eager append's."""
    a, b = (c.start() for c in two)
    x = a.draw(3, 5)
    a.capture(a.step(x, *buffers(a, 5)))
    for c in (a, b):
        y = c.draw(4, 7)
        if how == "rope":
            c.rope(0, y, PAGE)
        else:
            c.plain(0, y, PAGE)()
    same(a.rows(), b.rows())


@pytest.mark.parametrize("first", ["rope", "plain"])
@pytest.mark.parametrize("then", ["rope", "plain"])
def test_an_eager_append_into_the_page_that_a_captured_one_took(two, first, then):
    """Captured rows stay, rows behind them in the same page are appended before the capture is replayed."""
    a, b = (c.start() for c in two)

    def rows(c, how, number, n, pos0):
        x = c.draw(number, n)
        return (lambda: c.rope(0, x, pos0)) if how == "rope" else c.plain(0, x, pos0)

    g = a.capture(rows(a, first, 3, 5, PAGE))
    rows(b, first, 3, 5, PAGE)()
    for c in (a, b):
        rows(c, then, 4, 2, PAGE + 5)()
    g.replay()
    same(a.rows(), b.rows())


@pytest.mark.parametrize("order", [(0, 1), (1, 0), (1, 1, 0), (1,)])
def test_two_captured_steps_replayed_in_any_order(two, order):
    """Graphs for blocks of two sizes, each over the page that the other takes too."""
    a, b = (c.start() for c in two)
    xs, bufs = [a.draw(3, 5), a.draw(4, 9)], [buffers(a, 5), buffers(a, 9)]
    graphs = [a.capture(a.step(x, *qo)) for x, qo in zip(xs, bufs)]
    want = []
    for x in xs:
        qo = buffers(b, len(x))
        b.step(x, *qo)()
        want.append(qo)
    for i in order:
        graphs[i].replay()
        a.torch.cuda.synchronize()
        assert all(bool((got == w).all()) for got, w in zip(bufs[i], want[i]))
    same(a.rows(), b.rows())


def test_pages_exchanged_between_captured_and_eager_steps(two):
    """A replay sets an entry back to the page that its capture had: an eager append that takes another one says so again."""
    a, b = (c.start() for c in two)
    x = a.draw(3, 5)
    g = a.capture(a.step(x, *buffers(a, 5)))

    def both(c, first):
        c.rope(1, c.draw(10 + first, PAGE), 5 * PAGE)  # takes the page that the step had
        c.rope(0, c.draw(20 + first, 6), PAGE)         # the one below it

    for c in (a, b):
        both(c, 0)
        c.drop(0, 6)
        c.drop(1, PAGE)
    g.replay()
    for c in (a, b):
        both(c, 1)
    same(a.rows(), b.rows())


def test_a_capture_of_several_appends_sends_an_entry_once(two):
    """Rows appended one after the other in one capture, over two page ends, all behind a single replay."""
    a, b = (c.start() for c in two)

    def run(c):
        xs = [c.draw(30 + i, 3) for i in range(8)]

        def steps():
            for i, x in enumerate(xs):
                c.rope(0, x, PAGE + 3 * i)
        return steps

    g = a.capture(run(a))
    run(b)()
    g.replay()
    same(a.rows(), b.rows())
    for c in (a, b):
        c.rope(0, c.draw(50, 20), PAGE + 24)
    same(a.rows(), b.rows())


@pytest.mark.parametrize("then", ["rope", "plain"])
def test_an_append_whose_launch_failed_leaves_no_entry_behind(two, then):
    """A capture that is no longer valid refuses the launches of an append; the next one must not rely on them."""
    a, b = (c.start() for c in two)
    torch, kvc = a.torch, a.kvc
    x, y = a.draw(3, 5), b.draw(4, 7)
    free = a.c.stats()["pages_free"]
    cu = ctypes.CDLL("libcuda.so.1")
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    stream, graph = ctypes.c_void_p(st.cuda_stream), ctypes.c_void_p()
    assert cu.cuStreamBeginCapture_v2(stream, 2) == 0  # relaxed: no other stream is concerned
    assert cu.cuStreamSynchronize(stream) != 0         # not allowed there: the capture is void
    with pytest.raises(kvc.KvcError) as e:
        a.c.append_rope(0, [0], [5], list(range(PAGE, PAGE + 5)), None, x[:, H:H + Hk], x[:, H + Hk:], None, stream=st)
    assert e.value.status == kvc.KVC_ECUDA
    assert cu.cuStreamEndCapture(stream, ctypes.byref(graph)) != 0
    assert a.c.n_tokens(0) == PAGE and a.c.stats()["pages_free"] == free
    for c in (a, b):
        if then == "rope":
            c.rope(0, y, PAGE)
        else:
            c.plain(0, y, PAGE)()
    same(a.rows(), b.rows())


@pytest.mark.parametrize("then", ["rope", "plain"])
def test_a_failed_launch_is_reported_once(two, then):
    """An append into a page that is there, refused by a void capture; the next one, which takes a page, is not told of it."""
    a, b = (c.start() for c in two)
    torch, kvc = a.torch, a.kvc
    for c in (a, b):
        c.rope(0, c.draw(6, 2), PAGE)
    x, y = a.draw(3, 5), b.draw(4, 20)
    cu = ctypes.CDLL("libcuda.so.1")
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    stream, graph = ctypes.c_void_p(st.cuda_stream), ctypes.c_void_p()
    assert cu.cuStreamBeginCapture_v2(stream, 2) == 0
    assert cu.cuStreamSynchronize(stream) != 0
    with pytest.raises(kvc.KvcError) as e:
        a.c.append_rope(0, [0], [5], list(range(PAGE + 2, PAGE + 7)), None, x[:, H:H + Hk], x[:, H + Hk:], None, stream=st)
    assert e.value.status == kvc.KVC_ECUDA
    assert cu.cuStreamEndCapture(stream, ctypes.byref(graph)) != 0
    assert a.c.n_tokens(0) == PAGE + 2
    for c in (a, b):
        if then == "rope":
            c.rope(0, y, PAGE + 2)
        else:
            c.plain(0, y, PAGE + 2)()
    same(a.rows(), b.rows())


@pytest.mark.parametrize("first", ["rope", "plain"])
@pytest.mark.parametrize("then", ["rope", "plain", "step"])
def test_another_layers_append_behind_a_captured_one(first, then):
    """The first layer's append takes a page in a capture; the second layer's rows of the same tokens come outside it, ahead of
    the replay."""
    a, b = caches = [Cache(2), Cache(2)]
    try:
        n = 1 if then == "step" else 5

        def rows(c, how, layer, number):
            x = c.draw(number, n)
            k, v = x[:, H:H + Hk].float().contiguous(), x[:, H + Hk:].float().contiguous()
            q = x[:, :H].float().contiguous()
            c.held.append((k, v, q))
            if how == "rope":
                return lambda: c.c.append_rope(layer, [0], [n], list(range(PAGE, PAGE + n)), None, x[:, H:H + Hk],
                                               x[:, H + Hk:], None)
            if how == "plain":
                return lambda: c.c.append(layer, 0, PAGE, k, v)
            return lambda: c.c.decode_step(layer, [0], [PAGE], k, v, q, c.torch.empty_like(q), 0.125)

        for c in caches:
            for seq, m in ((1, 5 * PAGE), (0, PAGE)):
                for layer in range(2):
                    x = c.draw(10 * seq + layer, m)
                    c.c.append_rope(layer, [seq], [m], list(range(m)), None, x[:, H:H + Hk], x[:, H + Hk:], None)
            c.rows()
        g = a.capture(rows(a, first, 0, 30))
        rows(b, first, 0, 30)()
        for c in caches:
            rows(c, then, 1, 31)()
        g.replay()
        same(a.rows(), b.rows())
    finally:
        for c in caches:
            c.c.close()
