"""The plan of a tree attention, the angles of an append and the binding's refusals, without a GPU."""
import decimal

import numpy as np
import pytest


def _kvc():
    from kv_cache_decode_flash_gb300 import kvc

    return kvc


@pytest.mark.parametrize("H,Hk", [(8, 2), (40, 8), (32, 8), (8, 8), (6, 2), (8, 1)])
def test_tree_plans_cover_every_row_within_the_work_space(H, Hk):
    rng = np.random.default_rng(1)
    r = H // Hk
    for _ in range(300):
        n_seq = int(rng.choice([1, 1, 2, 5, 33, 64]))
        n_q = [int(x) for x in np.exp(rng.uniform(0, np.log(257), n_seq)).astype(int)]
        rows = [t + int(np.exp(rng.uniform(0, np.log(200000)))) - 1 for t in n_q]
        off = [int(x) for x in rng.integers(0, 300, n_seq)]
        p = _kvc().kvc_debug_tree_plan(H, Hk, 152, rows, off, n_q)
        assert p["tile_m"] == 32
        items = 0
        for n, o, t, w, s, length in zip(rows, off, n_q, p["whole"], p["splits"], p["split_rows"]):
            # rows are counted from the 16-row boundary below the first; parts are whole steps of 64
            assert s >= 1 and length % 64 == 0 and s * length >= n + o % 16
            units = -(-t * r // p["tile_m"]) * Hk
            assert 0 <= w <= units and (s > 1 or w == units)
            items += w + (units - w) * s
        assert items == p["items"]
        assert p["part_rows"] <= p["part_cap"]


@pytest.mark.parametrize("bad", [dict(n_q=[0]), dict(n_q=[257]), dict(n_q=[101]), dict(off=[-1]), dict(H=7), dict(H=72)])
def test_tree_plan_refusals(bad):
    kvc = _kvc()
    a = {**dict(H=8, rows=[100], off=[0], n_q=[5]), **bad}
    with pytest.raises(kvc.KvcError):
        kvc.kvc_debug_tree_plan(a["H"], 2, 152, a["rows"], a["off"], a["n_q"])


def _pi(digits):
    """pi by Machin's formula."""
    decimal.getcontext().prec = digits + 10

    def arctan_inv(x):
        x = decimal.Decimal(x)
        total, term, k = decimal.Decimal(0), 1 / x, 1
        while abs(term) > decimal.Decimal(10) ** -(digits + 5):
            total += term / k if k % 4 == 1 else -term / k
            term /= x * x
            k += 2
        return total

    return 4 * (4 * arctan_inv(5) - arctan_inv(239))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("base", [1.0000002, 10000.0, 500000.0, 1000000.0, 3.0e38])
def test_turns_of_a_position_are_exact_to_64_bits(base, D):
    """Each is base^(-2i/D) / (2 pi) of the double that kvc_seq_add's angles are made from, rounded to 2^-64."""
    pi = _pi(60)
    got = _kvc().kvc_debug_rope_turns(base, D)
    assert len(got) == D // 2
    b = float(np.float32(base))
    for i, t in enumerate(got):
        theta = decimal.Decimal(b ** (-2.0 * i / D))
        want = theta / (2 * pi) * 2**64
        # pow may differ by a unit in the last place between libraries: 2^-52 of the value beside half a unit
        assert abs(t - want) <= 1 + abs(want) * decimal.Decimal(2.0**-52)


@pytest.mark.parametrize("base,D", [(1.0, 64), (float("inf"), 64), (float("nan"), 128), (10000.0, 96)])
def test_turns_refusals(base, D):
    kvc = _kvc()
    with pytest.raises(kvc.KvcError):
        kvc.kvc_debug_rope_turns(base, D)


def test_calls_without_a_context_are_refused():
    kvc = _kvc()
    lib = kvc.load()
    assert lib.kvc_attn_tree(None, 0, 1, None, None, 0, None, None, None, 1.0, None) == kvc.KVC_EINVAL
    assert lib.kvc_append_rope(None, 0, 1, None, None, None, 0, None, 0, None, 0, None, 0, None, None, 0.0, None,
                               None) == kvc.KVC_EINVAL
    assert lib.kvc_seq_keep(None, 1, None, None, None, None, None) == kvc.KVC_EINVAL


def test_positions_that_do_not_fit_are_refused_by_the_binding():
    kvc = _kvc()
    for pos in ([2**31], [-2**31 - 1], np.array([2**40])):
        with pytest.raises(kvc.KvcError):
            kvc._host_ints(pos)
    at, n, a = kvc._host_ints(np.arange(10)[::2])
    assert n == 5 and list(a) == [0, 2, 4, 6, 8] and a.dtype == np.int32 and at == a.ctypes.data
    for x in ([3, -1], (3, -1), iter([3, -1]), [np.int64(3), np.int32(-1)], [3.0, -1.0]):
        at, n, a = kvc._host_ints(x)
        assert n == 2 and list(a) == [3, -1]
