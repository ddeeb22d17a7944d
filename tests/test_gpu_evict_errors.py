"""Eviction by weight where a device error was reported: the call fails and nothing has changed."""
import numpy as np
import pytest

from test_gpu_row_weight import _cache, _evict_and_check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["q8", "f16"])
@pytest.mark.parametrize("n,k", [(300, 20), (300, 300), (9000, 700)])  # one CTA does it all, and several kernels
def test_evict_with_a_device_error_reported_changes_nothing(n, k, kind):
    import torch

    tw = _cache(kind, 8, 2, 64, [n], layers=2)
    try:
        blob, pos = tw.gpu.state_get(0, -1, -1), tw.gpu.positions(0)
        w0 = np.random.default_rng(n).random((2, n + 7)).astype(np.float32)
        w = torch.from_numpy(w0.copy()).to("cuda:0")
        for _ in range(2):  # and again: the word stays until it is asked for
            tw.kvc.kvc_debug_set_device_error(tw.gpu.ctx, 8)
            with pytest.raises(tw.kvc.KvcError) as e:
                tw.gpu.evict_weight(0, -1, -1, k, w)
            assert e.value.status == tw.kvc.KVC_EINTERNAL
            assert np.array_equal(w.cpu().numpy(), w0)
            assert tw.gpu.n_tokens(0) == n and np.array_equal(tw.gpu.positions(0), pos)
        assert tw.kvc.kvc_check_device_error(tw.gpu.ctx) == 8
        assert tw.gpu.state_get(0, -1, -1) == blob
        _evict_and_check(tw, 0, -1, -1, k, w0)
    finally:
        tw.close()


def test_evict_without_host_memory_says_so():
    """The list of candidates that are not consecutive rows cannot be allocated: KVC_ENOMEM with a message of its own, and
    nothing has changed."""
    import torch

    tw = _cache("q8", 8, 2, 64, [300])
    try:
        w = torch.rand(2, 300, device="cuda:0")
        assert tw.gpu.evict_weight(0, -1, -1, 20, w) == 20  # (the rows are out of order from here on)
        blob, w0 = tw.gpu.state_get(0, -1, -1), w.clone()
        with pytest.raises(tw.kvc.KvcError):
            tw.gpu.evict_weight(5, -1, -1, 20, w)  # leaves another message
        tw.kvc.kvc_debug_fail_alloc_after(tw.gpu.ctx, 0)
        with pytest.raises(tw.kvc.KvcError) as e:
            tw.gpu.evict_weight(0, 0, 290, 20, w)
        assert e.value.status == tw.kvc.KVC_ENOMEM and "no host memory" in str(e.value)
        tw.kvc.kvc_debug_fail_alloc_after(tw.gpu.ctx, -1)
        assert tw.gpu.state_get(0, -1, -1) == blob and bool((w == w0).all())
        assert tw.gpu.evict_weight(0, 0, 290, 20, w) == 20
    finally:
        tw.close()
