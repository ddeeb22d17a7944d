"""Block attention (kvc_attn_cross): V values that are not finite in rows of no weight, on each of the two kernels."""
import numpy as np
import pytest

import oracle
from twin import Twin

pytestmark = pytest.mark.gpu

Q8, F16, Q4 = oracle.Q8_0, oracle.F16, oracle.Q4_0
KINDS = {"q8": (Q8, Q8), "f16": (F16, F16), "q8q4": (Q8, Q4)}
MMA, TCGEN05 = 1, 2


@pytest.mark.parametrize("kernel", [MMA, TCGEN05], ids=["mma", "tcgen05"])
@pytest.mark.parametrize("act", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("kind,D", [("q8", 64), ("f16", 64), ("q8", 128), ("f16", 128), ("q8q4", 128)])
@pytest.mark.parametrize("T", [2, 30, 150])
@pytest.mark.parametrize("n,low", [(700, 0), (6000, 3000)])
def test_values_that_are_not_finite_in_rows_of_no_weight(kind, D, act, T, n, low, kernel):
    """Seen rows whose scores lie 600 below the others' weigh 0 in 32 bits; an infinite V there reaches the tokens that see it
    (as an infinity or as 0 x inf) and no other.  One row that all see (alone, or among 3000 like it, whole parts of the rows),
    one that only the last token sees; a q8_0 or q4_0 value spoils its block of 32."""
    if act == "f32" and kernel == TCGEN05:
        pytest.skip("32-bit queries have one kernel")
    import torch

    H, Hk = 4, 2
    rng = np.random.default_rng(41)
    k = rng.standard_normal((n, Hk, D)).astype(np.float32) * 0.1
    v = rng.standard_normal((n, Hk, D)).astype(np.float32)
    k[:low] = -40
    k[[100, n - 1]] = -40
    v[100, 0, 3], v[n - 1, 1, 40] = np.inf, -np.inf
    tk, tv = KINDS[kind]
    tw = Twin(1, H, Hk, D, n + 64, type_=tk, type_v=tv, page_rows=64)
    try:
        tw.kvc.kvc_debug_block_kernel(tw.gpu.ctx, kernel)
        tw.gpu.append(0, 0, 0, torch.from_numpy(k).to(tw.dev), torch.from_numpy(v).to(tw.dev))
        dtype = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[act]
        q = (15 + torch.rand(T, H, D, generator=torch.Generator().manual_seed(5))).to("cuda:0", dtype)
        vis = torch.full((T,), n - 1, dtype=torch.int32, device="cuda:0")
        vis[-1] = n
        out = torch.full_like(q, float("nan"))
        tw.gpu.attn_cross(0, [0], [T], q, out, 1.0 / D, n_vis=vis)
        torch.cuda.synchronize()
        assert tw.kvc.kvc_check_device_error(tw.gpu.ctx) == 0
        spoil = np.zeros((T, H, D), bool)
        spoil[:, :2, slice(3, 4) if kind == "f16" else slice(0, 32)] = True
        spoil[-1, 2:, slice(40, 41) if kind == "f16" else slice(32, 64)] = True
        assert np.array_equal(~np.isfinite(out.float().cpu().numpy()), spoil)
    finally:
        tw.close()
