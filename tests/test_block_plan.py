"""The work plan of the block attention and the binding's refusals, without a GPU."""
import numpy as np
import pytest


def _plan(H, Hk, D, act, rows, n_q, sms=152):
    from kv_cache_decode_flash_gb300 import kvc

    return kvc.kvc_debug_block_plan(H, Hk, D, act, sms, rows, n_q)


@pytest.mark.parametrize("H,Hk,D", [(8, 2, 64), (40, 8, 128), (32, 8, 128), (8, 8, 64), (6, 2, 128)])
@pytest.mark.parametrize("act", [0, 1, 2])
def test_plans_cover_every_row_within_the_work_space(H, Hk, D, act):
    rng = np.random.default_rng(1)
    r = H // Hk
    for _ in range(300):
        n_seq = int(rng.choice([1, 1, 2, 5, 33, 64]))
        rows = [int(x) for x in np.exp(rng.uniform(0, np.log(200000), n_seq)).astype(int) - 1]
        n_q = [int(x) for x in np.exp(rng.uniform(0, np.log(600), n_seq)).astype(int) - 1]
        p = _plan(H, Hk, D, act, rows, n_q)
        items = 0
        for n, t, w, s, length in zip(rows, n_q, p["whole"], p["splits"], p["split_rows"]):
            assert s >= 1 and length >= 1 and s * length >= n  # every row is in a part
            units = -(-t * r // p["tile_m"]) * Hk
            assert 0 <= w <= units and (s > 1 or w == units)
            items += w + (units - w) * s
        assert items == p["items"]
        assert p["part_rows"] <= p["part_cap"]


def test_plan_refusals():
    from kv_cache_decode_flash_gb300 import kvc

    for args in ((8, 3, 64, 0, [1], [1]), (8, 2, 96, 0, [1], [1]), (8, 2, 64, 3, [1], [1]), (8, 2, 64, 0, [-1], [1]),
                 (8, 2, 64, 0, [1], [-1]), (8, 2, 64, 0, [], []), (8, 2, 64, 0, [1] * 65, [1] * 65),
                 (8, 2, 64, 0, [1], [2**31 - 1]), (64, 2, 64, 0, [1], [1])):
        with pytest.raises(kvc.KvcError):
            _plan(*args)


def test_null_context_is_refused():
    from kv_cache_decode_flash_gb300 import kvc

    L = kvc.load()
    assert L.kvc_attn_cross(None, 0, 1, None, None, 0, None, None, None, None, 1.0, None) == kvc.KVC_EINVAL
    assert L.kvc_attn_weight(None, 0, 1, None, None, 0, None, None, None, 1.0, None, 0, None) == kvc.KVC_EINVAL
    assert L.kvc_seq_evict_weight(None, 0, 0, 0, 0, None, 0, None) == kvc.KVC_EINVAL


def test_binding_refuses_tensors_it_would_misread():
    import torch

    from kv_cache_decode_flash_gb300 import kvc

    with pytest.raises(kvc.KvcError):
        kvc._act(torch.zeros(1, dtype=torch.float64))
    with pytest.raises(kvc.KvcError):
        kvc._block_tensor("q", torch.zeros(4), 0, torch.float32, 4)  # not on the device
    with pytest.raises(kvc.KvcError):
        kvc._block([0, 1], [1])
