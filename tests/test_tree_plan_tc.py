"""The plan of a tree attention on the tcgen05 kernel, without a GPU: entries for short last tiles, weighted parts, their order."""
import numpy as np
import pytest


def _kvc():
    from kv_cache_decode_flash_gb300 import kvc

    return kvc


def _check(H, Hk, rows, n_q):
    p = _kvc().kvc_debug_tree_plan_tc(H, Hk, 152, rows, n_q)
    r = H // Hk
    assert p["tile_m"] == 256 and len(rows) <= len(p["entries"]) <= 64
    items = part_row = cut = 0
    tiles = {i: [] for i in range(len(rows))}
    for e in p["entries"]:  # in the launch's order: items, partial rows and cut units follow each other without a gap
        assert e["item0"] == items and e["part_row0"] == part_row and e["cut0"] == cut
        units = e["tiles"] * Hk
        assert e["tiles"] >= 1 and e["splits"] >= 1 and 0 <= e["whole"] <= units and (e["splits"] > 1 or e["whole"] == units)
        assert e["split_rows"] % 128 == 0 and e["splits"] * e["split_rows"] >= rows[e["id"]]
        widest = min(256, max(n_q) * r)  # partial rows of an item
        assert e["part_rows"] == (units - e["whole"]) * e["splits"] * widest
        items += e["whole"] + (units - e["whole"]) * e["splits"]
        part_row += e["part_rows"]
        cut += units - e["whole"]
        tiles[e["id"]] += range(e["tile0"], e["tile0"] + e["tiles"])
    assert items == p["items"] and part_row == p["part_rows"] <= p["part_cap"]
    for i, t in enumerate(n_q):  # every tile of every sequence once
        assert sorted(tiles[i]) == list(range(-(-t * r // 256)))
    return p


@pytest.mark.parametrize("H,Hk", [(8, 2), (40, 8), (32, 8), (8, 8), (6, 2), (8, 1), (64, 8)])
def test_plans_cover_every_tile_and_row_once_within_the_work_space(H, Hk):
    rng = np.random.default_rng(1)
    for _ in range(400):
        n_seq = int(rng.choice([1, 1, 2, 4, 5, 33, 40, 63, 64]))
        n_q = [int(x) for x in np.exp(rng.uniform(0, np.log(257), n_seq)).astype(int)]
        if rng.random() < 0.5:  # blocks that end shortly behind a tile
            n_q = [int(x) for x in rng.integers(256 // (H // Hk) + 1, 257, n_seq)] if H // Hk > 1 else n_q
        rows = [t + int(np.exp(rng.uniform(0, np.log(200000)))) - 1 for t in n_q]
        _check(H, Hk, rows, n_q)


def test_a_short_last_tile_is_an_entry_of_its_own_with_longer_parts():
    p = _check(40, 8, [32832], [64])  # 320 query rows of a KV head: 256 and 64
    a, b = p["entries"]
    assert {(e["tile0"], e["tiles"]) for e in (a, b)} == {(0, 1), (1, 1)}
    short, full = sorted((a, b), key=lambda e: -e["tile0"])
    assert short["splits"] < full["splits"]


@pytest.mark.parametrize("n_seq,entries", [(31, 62), (32, 64), (33, 64), (50, 64), (63, 64), (64, 64)])
def test_more_short_last_tiles_than_a_launch_has_room_for(n_seq, entries):
    p = _check(10, 2, [60 + 5 * i for i in range(n_seq)], [52] * n_seq)  # 260 query rows each
    assert len(p["entries"]) == entries


def test_entries_are_in_the_order_of_their_parts_cost():
    rng = np.random.default_rng(3)
    for _ in range(50):
        n_q = [int(x) for x in rng.integers(20, 81, 32)]
        rows = [int(x) for x in rng.integers(1024, 8001, 32)]
        cost = []
        for e in _check(40, 8, rows, n_q)["entries"]:
            half = n_q[e["id"]] * 5 - e["tile0"] * 256 <= 128  # at 5/8 of another's a step
            cost.append(rows[e["id"]] * (5 if half else 8) / e["splits"])
        assert all(x >= y for x, y in zip(cost, cost[1:]))


@pytest.mark.parametrize("bad", [dict(n_q=[0]), dict(n_q=[257]), dict(n_q=[101]), dict(H=7), dict(H=72), dict(rows=[1] * 65, n_q=[1] * 65),
                                 dict(rows=[], n_q=[])])
def test_refusals(bad):
    kvc = _kvc()
    a = {**dict(H=8, rows=[100], n_q=[5]), **bad}
    with pytest.raises(kvc.KvcError):
        kvc.kvc_debug_tree_plan_tc(a["H"], 2, 152, a["rows"], a["n_q"])
