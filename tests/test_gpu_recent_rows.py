"""Rows that a decode attention may not yet request ahead of its wait, in a loop of drafted steps: those that the kernels since
the last attention wrote, and no more of them than there are."""
import numpy as np
import pytest

import oracle

pytestmark = pytest.mark.gpu

H, Hk, D = 4, 2, 64


@pytest.fixture
def cache():
    from kv_cache_decode_flash_gb300 import kvc

    c = kvc.KVCache(2, H, Hk, D, 400, 2, oracle.F16, oracle.F16, page_rows=16)
    yield c, lambda layer=0, seq=0: kvc.kvc_debug_recent_rows(c.ctx, layer, seq)
    c.close()


def _append(c, layer, seq, n, pos0=0, plain=False):
    import torch

    x = torch.from_numpy(np.random.default_rng(n).standard_normal((n, 2 * Hk, D)).astype(np.float32)).to("cuda:0")
    if plain:
        c.append(layer, seq, pos0, x[:, :Hk].contiguous(), x[:, Hk:].contiguous())
    else:
        c.append_rope(layer, [seq], [n], list(range(pos0, pos0 + n)), None, x[:, :Hk], x[:, Hk:], None)


def _attend(c, n=1, layer=0, seq=0):
    import torch

    q = torch.zeros(n, H, D, device="cuda:0")
    c.attn_tree(layer, [seq], [n], q, torch.empty_like(q), 0.125)
    return q


@pytest.mark.parametrize("plain", [False, True])
def test_steps_without_an_attention_never_count_more_rows_than_there_are(cache, plain):
    c, recent = cache
    for _ in range(200):
        for layer in range(2):
            _append(c, layer, 0, 20, plain=plain)
        assert recent(0) == recent(1) == 20
        c.keep([0], [20], [[]])
        assert recent(0) == recent(1) == 0


def test_rows_that_leave_are_no_longer_counted_and_moved_ones_are(cache):
    c, recent = cache
    for layer in range(2):
        _append(c, layer, 0, 30)
        _append(c, layer, 1, 7)
    assert recent(0, 0) == recent(1, 0) == 30 and recent(0, 1) == 7
    c.keep([0], [10], [[0, 3]])  # 22 left, all of them new
    assert recent() == 22 and recent(0, 1) == 7
    _attend(c)
    assert recent() == recent(1) == recent(0, 1) == 0
    for layer in range(2):
        _append(c, layer, 0, 9, 22)
    c.keep([0], [12], [[1, 4, 11]])  # three old rows among the last ones: what stays of the twelve moved
    assert c.n_tokens(0) == 22 and recent() == recent(1) == 3
    c.keep([0], [2], [[0, 1]])
    assert recent() == 3
    c.keep([0], [2], [[]])
    assert recent() == 1
    c.seq_rm(0, -1, -1)
    assert recent() == 0


def test_a_captured_attention_is_no_wait(cache):
    """What it waits for it waits for at its replays: appends in flight at the capture still count."""
    import torch

    c, recent = cache
    for layer in range(2):
        _append(c, layer, 0, 8)
    _attend(c)
    for layer in range(2):
        _append(c, layer, 0, 5, 8)
    g = torch.cuda.CUDAGraph()
    q = torch.zeros(1, H, D, device="cuda:0")
    out = torch.empty_like(q)
    with torch.cuda.graph(g):
        c.attn_tree(0, [0], [1], q, out, 0.125)
    assert recent() == recent(1) == 5
    g.replay()
    _attend(c)
    assert recent() == 0
