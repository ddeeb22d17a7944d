"""Tree attention (kvc_attn_tree) on values where bits or rows are easily lost: keys that are no 11-bit numbers under a
softmax of large scores, and V values that are not finite in rows of next to no weight.  On each of the two kernels."""
import numpy as np
import pytest

import oracle
from block_ref import values
from draft_ref import attend, attend_bound, tree_sees
from twin import Twin

pytestmark = pytest.mark.gpu

Q8, F16, Q4 = oracle.Q8_0, oracle.F16, oracle.Q4_0
KINDS = {"q8": (Q8, Q8), "f16": (F16, F16), "q8q4": (Q8, Q4)}
MMA, TCGEN05 = 1, 2


def _types():
    import torch

    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def _twin(kind, H, Hk, D, n, k, v, kernel, page=64, ref=True):
    tk, tv = KINDS[kind]
    tw = Twin(1, H, Hk, D, n + 64, type_=tk, type_v=tv, page_rows=page)
    tw.kvc.kvc_debug_block_kernel(tw.gpu.ctx, kernel)
    import torch

    if ref:
        tw.append(0, 0, 0, k, v)
    else:
        tw.gpu.append(0, 0, 0, torch.from_numpy(k).to(tw.dev), torch.from_numpy(v).to(tw.dev))
    return tw


def _run(tw, T, q, scale, parent):
    import torch

    out = torch.full_like(q, float("nan"))
    tw.gpu.attn_tree(0, [0], [T], q, out, scale, parent=torch.from_numpy(parent).to(q.device))
    torch.cuda.synchronize()
    assert tw.kvc.kvc_check_device_error(tw.gpu.ctx) == 0
    return out


def _level_rows(rng, n, Hk, D, spread):
    """Rows whose keys are alike but for the first of every 32, which gives the block its scale and which the queries leave out:
    a code of 90 to 126, another one in every row, times a scale of 11 bits, 1 to 1 + spread together.  Rounding a row's keys to
    11 bits then goes the same way in every product of its score; V's sign is that of this rounding."""
    a, c = 1 + spread * rng.random((n, Hk, 1)), rng.integers(90, 127, (n, Hk, 1))
    k = np.broadcast_to(a, (n, Hk, D)).astype(np.float32)
    k[..., ::32] = (127 * a / c).astype(np.float32)
    held = np.float16(a / c).astype(np.float64) * c
    sign = np.where(np.float16(held).astype(np.float64) > held, 1.0, -1.0)
    v = sign * (1 + 0.1 * rng.random((n, Hk, D)))
    return k, v.astype(np.float32)


# The bound is attend_bound's with operands of 20 bits or more: both kernels take the codes of K exactly (mma.sync) or as two
# fp16 parts (tcgen05: 18 bits, all that a code times its scale has).  One part of 11 bits is off by up to 2^-12 of a score of
# 100, 0.02, where the bound has 100 (2^-20 + 132 x 2^-24) = 0.0009, and the results move by as much with V as it is here.
@pytest.mark.parametrize("kernel", [MMA, TCGEN05], ids=["mma", "tcgen05"])
@pytest.mark.parametrize("act", ["f16", "bf16"])
@pytest.mark.parametrize("kind,D", [("q8", 64), ("q8", 128), ("q8q4", 128)])
@pytest.mark.parametrize("T,n", [(9, 300), (30, 1500), (70, 900)])
@pytest.mark.parametrize("score,spread", [(30, 0.05), (100, 0.02), (300, 0.01)])
def test_keys_keep_their_bits_under_large_scores(kind, D, act, T, n, score, spread, kernel):
    H, Hk = 10, 2
    rng = np.random.default_rng(31)
    k, v = _level_rows(rng, n, Hk, D, spread)
    tw = _twin(kind, H, Hk, D, n, k, v, kernel)
    try:
        import torch

        one = np.ones((T, H, D))
        one[..., ::32] = 0
        q = torch.from_numpy(one).to("cuda:0", _types()[act])
        par = np.array([-1 if t == 0 else rng.integers(max(-1, t - 6), t) for t in range(T)], np.int32)
        scale = float(np.float32(score / D))
        got = _run(tw, T, q, scale, par).double().cpu().numpy()
        s = tw.ref.seqs[0]
        K, V = values(s.K[0]), values(s.V[0])
        want, mag, size = attend(one, K, V, scale, tree_sees(par, n, T))
        bound = attend_bound(mag, size, n, D, act, exact=True)
        ratio = np.abs(got - want) / bound
        assert ratio.max() <= 1, "%.2f of its bound" % ratio.max()
    finally:
        tw.close()


@pytest.mark.parametrize("kernel", [MMA, TCGEN05], ids=["mma", "tcgen05"])
@pytest.mark.parametrize("act", ["f16", "bf16"])
@pytest.mark.parametrize("kind,D", [("q8", 64), ("q8", 128), ("q8q4", 128)])
def test_keys_beside_an_unseen_one_of_a_million_times_their_size(kind, D, act, kernel):
    """A step's codes of K share a power of two on tcgen05: both parts of a code times its scale are whole up to 2^21 below the
    step's largest scale, also one of a row that most tokens do not see."""
    import torch

    H, Hk, T, n = 10, 2, 30, 600
    rng = np.random.default_rng(43)
    k, v = _level_rows(rng, n, Hk, D, 0.02)
    k *= 2.0**-6
    k[n - T + 1] = 2.0**14  # token 1's, a sibling of all but itself
    tw = _twin(kind, H, Hk, D, n, k, v, kernel)
    try:
        one = np.full((T, H, D), 2.0**6)
        one[..., ::32] = 0
        par = np.zeros(T, np.int32)
        par[:2] = -1
        scale = float(np.float32(100 / D))
        got = _run(tw, T, torch.from_numpy(one).to("cuda:0", _types()[act]), scale, par).double().cpu().numpy()
        s = tw.ref.seqs[0]
        want, mag, size = attend(one, values(s.K[0]), values(s.V[0]), scale, tree_sees(par, n, T))
        bound = attend_bound(mag, size, n, D, act, exact=True)
        ratio = (np.abs(got - want) / bound)[[t for t in range(T) if t != 1]]
        assert ratio.max() <= 1, "%.2f of its bound" % ratio.max()
    finally:
        tw.close()


@pytest.mark.parametrize("kernel", [MMA, TCGEN05], ids=["mma", "tcgen05"])
@pytest.mark.parametrize("act", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("kind,D", [("q8", 64), ("f16", 64), ("q8", 128), ("f16", 128), ("q8q4", 128)])
@pytest.mark.parametrize("T", [3, 30, 70])
@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
@pytest.mark.parametrize("n,low", [(700, 0), (6000, 3000)])
def test_values_that_are_not_finite_in_rows_of_no_weight(kind, D, act, T, n, low, bad, kernel):
    """A seen row whose score lies 600 below the others': its weight is 0 in 32 bits, and what its V holds reaches the tokens
    that see it all the same (as an infinity or as 0 x inf).  One row far before the block (alone, or among 3000 like it, whole
    parts of the rows that are nothing beside the others), one just before it and one of the block that some of its tokens do
    not see; a q8_0 or q4_0 value spoils its block of 32."""
    if act == "f32" and kernel == TCGEN05:
        pytest.skip("32-bit queries have one kernel")
    if kind != "f16" and np.isnan(bad):
        pytest.skip("codes hold no NaN: a block's scale is formed without it")
    H, Hk = 4, 2
    rng = np.random.default_rng(37)
    k = rng.standard_normal((n, Hk, D)).astype(np.float32) * 0.1
    v = rng.standard_normal((n, Hk, D)).astype(np.float32)
    k[:low] = -40
    spoilt = {100: (0, 3), n - T - 2: (1, 35), n - T + 1: (0, 40)}  # row: (KV head, dim)
    for row, (g, d) in spoilt.items():
        k[row] = -40
        v[row, g, d] = bad
    tw = _twin(kind, H, Hk, D, n, k, v, kernel, ref=False)
    try:
        import torch

        q = (15 + torch.rand(T, H, D, generator=torch.Generator().manual_seed(5))).to("cuda:0", _types()[act])
        par = np.array([-1, 0] + [0 if t % 3 else 1 for t in range(2, T)], np.int32)[:T]
        o = _run(tw, T, q, 1.0 / D, par).float().cpu().numpy()
        sees = tree_sees(par, n, T)
        spoil = np.zeros((T, H, D), bool)
        for row, (g, d) in spoilt.items():
            dims = slice(d, d + 1) if kind == "f16" else slice(d // 32 * 32, d // 32 * 32 + 32)
            spoil[sees[:, row], g * 2:g * 2 + 2, dims] = True
        assert sees[:, n - T + 1].any() and not sees[:, n - T + 1].all()
        assert np.array_equal(~np.isfinite(o), spoil)
    finally:
        tw.close()
