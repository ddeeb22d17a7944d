"""Host values and streams that the binding takes for a drafted block's calls, without a GPU."""
import numpy as np
import pytest


def _kvc():
    from kv_cache_decode_flash_gb300 import kvc

    return kvc


@pytest.mark.parametrize("x", [[1.7, 2.2], (0.5,), [2**40 + 0.5], [float("nan")], [float("inf")], [1, -float("inf")], [2.0**31],
                               [-2.0**31 - 1], [np.float32(1.5)], [np.float64("nan")], [np.int64(2**31)], iter([1.5]),
                               np.array([1.7, 2.2]), np.array([np.nan]), [1, None], ["2.5"]])
def test_numbers_that_are_not_whole_or_too_large_are_refused(x):
    kvc = _kvc()
    with np.errstate(invalid="ignore"):
        with pytest.raises((kvc.KvcError, TypeError)) as e:
            kvc._host_ints(x)
    if e.type is kvc.KvcError:
        assert e.value.status == kvc.KVC_ERANGE
    else:
        assert None in x  # no number at all


@pytest.mark.parametrize("x", [[3.0, -1.0], [2.0**31 - 1, -2.0**31], (np.float32(3), np.int8(-1)), [True, False],
                               np.array([3.0, -1.0]), np.array([[3], [-1]])])
def test_whole_numbers_of_any_type_are_taken(x):
    _, n, a = _kvc()._host_ints(x)
    assert n == 2 and [int(v) for v in np.asarray(a).ravel()] == [int(v) for v in np.asarray(x).ravel()]


@pytest.mark.parametrize("device", [0, 1, None, "cuda:0", np.int64(0)])
def test_current_stream_of_any_device_that_torch_takes(device, monkeypatch):
    """A device number by the short way, anything else (the current device, torch.device, a name) by torch's own."""
    import torch

    kvc = _kvc()
    if isinstance(device, str):
        device = torch.device(device)

    class Stream:
        cuda_stream = 77

    asked = []
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: asked.append(d) or Stream())
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 70 + (asked.append(d) or 7) if type(d) is int else 1 / 0)
    for known in (None, torch._C._cuda_getCurrentRawStream):
        monkeypatch.setattr(kvc, "_raw_stream", known)
        assert kvc._stream(None, device) == 77
        assert kvc._stream(5, device) == 5 and kvc._stream(Stream(), device) == 77
    assert len(asked) == 2 and all(d is device for d in asked)
