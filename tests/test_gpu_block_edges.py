"""Block attention and row weights where a call's corners meet: tiles whose tokens see nothing, values that are not finite
beside tokens that do not see them, tokens of few rows, peaked softmaxes."""
import math

import numpy as np
import pytest

import oracle
from block_ref import cross, cross_bound, values
from twin import Twin, kv_inputs

pytestmark = pytest.mark.gpu

Q8, F16, Q4 = oracle.Q8_0, oracle.F16, oracle.Q4_0
KINDS = {"q8": (Q8, Q8), "f16": (F16, F16), "q8q4": (Q8, Q4)}
MMA, TC = 1, 2  # kernels of 16-bit queries (kvc_debug_block_kernel)


def _twin(kind, H, Hk, D, n_ctx, n_seq=1, page=64, layers=1):
    tk, tv = KINDS[kind]
    return Twin(layers, H, Hk, D, n_ctx, n_seq_max=n_seq, type_=tk, type_v=tv, page_rows=page)


def _tensor(x, act="f32"):
    import torch

    dt = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[act]
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to("cuda:0", dt)


def _attend(tw, kernel, ids, n_q, q, scale, vis=None, lse=True):
    import torch

    tw.kvc.kvc_debug_block_kernel(tw.gpu.ctx, kernel)
    out = torch.full_like(q, float("nan"))
    z = torch.full(q.shape[:2], float("nan"), device=q.device) if lse else None
    v = None if vis is None else torch.as_tensor(np.asarray(vis), dtype=torch.int32).to(q.device)
    tw.gpu.attn_cross(0, ids, n_q, q, out, scale, lse=z, n_vis=v)
    torch.cuda.synchronize()
    assert tw.kvc.kvc_check_device_error(tw.gpu.ctx) == 0
    return out, z


@pytest.mark.parametrize("act", ["f16", "bf16"])
@pytest.mark.parametrize("kind,D", [("f16", 64), ("f16", 128), ("q8", 128)])
@pytest.mark.parametrize("T", [10, 64, 150])
@pytest.mark.parametrize("kernel", [MMA, TC])
def test_tiles_whose_tokens_see_nothing(kernel, T, kind, D, act):
    """A batch in which every other sequence's tokens, and one sequence's last tokens, see no row, among others that see
    all of theirs: whole query tiles (narrow: 40 query rows, wide: 256) have nothing to do while rows that hold large
    values were asked for.  Their results are 0 and -inf, every time."""
    import torch

    H, Hk, n_seq, n = 8, 2, 8, 300
    tw = _twin(kind, H, Hk, D, n_seq * n + 64, n_seq)
    try:
        rng = np.random.default_rng(T)
        for i in range(n_seq):
            big = (1000.0 + rng.random((n, Hk, D))).astype(np.float32)
            tw.gpu.append(0, i, 0, _tensor(big * 2.0**-10), _tensor(big))
        ids, n_q = list(range(n_seq)) + [1], [T] * n_seq + [2 * 64 + T]
        q = _tensor(rng.standard_normal((sum(n_q), H, D)), act)
        vis = np.concatenate([np.full(T, n if i % 2 == 0 else 0) for i in range(n_seq)] + [np.repeat([n, 0], [64, 64 + T])])
        none = torch.from_numpy(vis == 0).to(q.device)
        for _ in range(20):
            got, z = _attend(tw, kernel, ids, n_q, q, D**-0.5, vis)
            assert bool((got[none] == 0).all()) and bool((z[none] == -math.inf).all())
            assert bool((got[~none].float() >= 999).all()) and bool(torch.isfinite(z[~none]).all())
    finally:
        tw.close()
