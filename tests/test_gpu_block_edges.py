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


@pytest.mark.parametrize("act", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("unseen", [0, 1, 5])
@pytest.mark.parametrize("T", [12, 40, 130])
@pytest.mark.parametrize("kernel", [MMA, TC])
def test_values_that_are_not_finite_reach_the_tokens_that_see_them(kernel, T, unseen, D, act):
    """Infinities and NaN in V of rows that all but the block's first tokens see (those see nothing, or the rows before the
    first of them): they come through for every token that sees them, whatever its neighbours see, and for no other."""
    import torch

    n, H, Hk = 500, 8, 2
    inf = float("inf")
    k, v = kv_inputs(19, 0, n, Hk, D, sigma=0.5)
    v[100, 0, 3], v[170, 0, 35], v[299, 1, 5], v[400, 0, 3] = inf, -inf, np.nan, inf
    tw = _twin("f16", H, Hk, D, n + 64)
    try:
        tw.gpu.append(0, 0, 0, _tensor(k), _tensor(v))
        q = _tensor(np.random.default_rng(2).standard_normal((T, H, D)), act)
        for few in (0, 100):  # none of them at all, or the rows before the first one that is not finite
            vis = np.full(T, n)
            vis[:unseen] = few
            got, z = _attend(tw, kernel, [0], [T], q, 0.125, vis)
            o = got.float()
            assert bool(torch.isfinite(o[:unseen]).all())
            assert few or bool((o[:unseen] == 0).all())
            o = o[unseen:]
            assert bool((o[:, :4, 3] == inf).all()) and bool((o[:, :4, 35] == -inf).all())
            assert bool(torch.isnan(o[:, 4:, 5]).all())
            o[:, :4, 3] = o[:, :4, 35] = o[:, 4:, 5] = 0
            assert bool(torch.isfinite(o).all()) and bool(torch.isfinite(z[unseen:]).all())
    finally:
        tw.close()


@pytest.mark.parametrize("kind", ["q8", "q8q4"])
@pytest.mark.parametrize("T", [12, 130])
@pytest.mark.parametrize("kernel", [MMA, TC])
def test_scales_that_are_not_finite_reach_the_tokens_that_see_them(kernel, T, kind):
    """A block of V whose scale is infinite or NaN (values beyond fp16's scales) is not a number for the tokens that see
    its row, and nothing for those that do not."""
    import torch

    n, H, Hk, D = 500, 8, 2, 128
    k, v = kv_inputs(23, 0, n, Hk, D, sigma=0.5)
    v[200, 1, 70], v[390, 0, 7] = np.float32(3e38), np.float32(np.nan)
    tw = _twin(kind, H, Hk, D, n + 64)
    try:
        tw.gpu.append(0, 0, 0, _tensor(k), _tensor(v))
        q = _tensor(np.random.default_rng(2).standard_normal((T, H, D)), "bf16")
        vis = np.full(T, n)
        vis[:3] = [0, 200, 390]
        got, _ = _attend(tw, kernel, [0], [T], q, 0.125, vis)
        fin = torch.isfinite(got.float())
        assert bool(fin[:2].all()) and bool(fin[:, :4, 32:].all())  # (heads 0-3 read KV head 0: only its block 0 is spoilt)
        assert not bool(fin[2:, 4:, 64:96].all(2).any())
        assert bool(fin[:, 4:, :64].all()) and bool(fin[:, 4:, 96:].all())
    finally:
        tw.close()


@pytest.mark.parametrize("act", ["f16", "bf16"])
@pytest.mark.parametrize("T", [2, 60])
@pytest.mark.parametrize("kernel", [MMA, TC])
def test_infinite_value_of_a_row_of_little_weight(kernel, T, act):
    """A row's weight of e^-40 is a positive number, too small for fp16: an infinite value there is infinite in the result, not
    the NaN of 0 x inf (which the tcgen05 kernel may give where all tokens see the row)."""
    import torch

    n, H, Hk, D = 300, 4, 2, 64
    k, v = kv_inputs(29, 0, n, Hk, D, sigma=0.5)
    k[:] = 0
    k[37, :, 0] = -40.0  # its score
    v[37, 0, 3], v[37, 1, 40] = np.inf, -np.inf
    tw = _twin("f16", H, Hk, D, n + 64)
    try:
        tw.gpu.append(0, 0, 0, _tensor(k), _tensor(v))
        q = np.zeros((T, H, D))
        q[:, :, 0] = 1.0
        for vis in (None, [n] * (T - 1) + [30]):
            got, _ = _attend(tw, kernel, [0], [T], _tensor(q, act), 1.0, vis)
            o = got.float()[:T - 1]
            if kernel == TC and vis is None:
                assert not bool(torch.isfinite(o[:, :2, 3]).any()) and not bool(torch.isfinite(o[:, 2:, 40]).any())
            else:
                assert bool((o[:, :2, 3] == math.inf).all()) and bool((o[:, 2:, 40] == -math.inf).all())
            o[:, :2, 3] = o[:, 2:, 40] = 0
            assert bool(torch.isfinite(o).all())
    finally:
        tw.close()


@pytest.mark.parametrize("act", ["f16", "bf16"])
@pytest.mark.parametrize("T", [1, 70, 9728])
@pytest.mark.parametrize("nats", [14, 16, 17, 20])
@pytest.mark.parametrize("kernel", [MMA, TC])
def test_many_small_weights_beside_a_great_one(kernel, nats, T, act):
    """An attention sink: the first row's score lies `nats` above those of 32767 others, which hold most of the values.
    With the most tokens a work item walks all rows, so that every small weight is formed beside the great one.

    Off by: half a step of the result and of P (2^-11 each: weights may be rounded alike, so nothing averages out); P below
    its normal range, 2^-32 of the largest weight a row; the exponential (2^-22) and the scores' sums, (D + 4) 2^-24 of
    |q| |k| = nats + 1, twice; a chain of n / 16 sums of positive numbers in the products, each losing at most 2^-23 of
    what is summed there (the denominator's is shorter)."""
    n, H, Hk, D = 32768, 4, 2, 64
    rng = np.random.default_rng(nats)
    k, v = np.zeros((n, Hk, D), np.float32), (0.5 + rng.random((n, Hk, D))).astype(np.float32)
    k[:, :, 1] = rng.integers(-8, 9, (n, Hk)) / 16.0
    k[0, :, 0], k[0, :, 1], v[0] = nats, 0, 2.0**-9
    tw = _twin("f16", H, Hk, D, n + 64, page=256)
    try:
        tw.gpu.append(0, 0, 0, _tensor(k), _tensor(v))
        few = min(T, 7)  # different tokens
        q = np.zeros((few, H, D), np.float32)
        q[:, :, 0], q[:, :, 1] = 1.0, np.linspace(-1, 1, few * H).reshape(few, H)
        qt = _tensor(q, act)
        got, z = _attend(tw, kernel, [0], [T], qt.repeat(-(-T // few), 1, 1)[:T].contiguous(), 1.0)
        K, V = k.astype(np.float64), v.astype(np.float16).astype(np.float64)
        want, wz, mag, _ = cross(qt.double().cpu().numpy(), K, V, 1.0, np.full(few, n))
        half = {"f16": 2.0**-11, "bf16": 2.0**-8}[act]
        score = 2.0**-22 + (nats + 1) * (D + 4) * 2.0**-24
        sums = n / 16 * 2.0**-23
        lim = mag * (half + 2.0**-11 + 2 * score + sums) + n * 2.0**-32 * np.abs(V).max()
        got, z = got.double().cpu().numpy(), z.double().cpu().numpy()
        for t in range(0, T, few):
            m = min(few, T - t)
            err = np.abs(got[t:t + m] - want[:m])
            assert np.all(err <= lim[:m]), "off by %.3g, %.2f of its bound" % (err.max(), (err / lim[:m]).max())
            assert np.abs(z[t:t + m] - wz[:m]).max() <= score + sums + 2.0**-23 * 2 * nats
    finally:
        tw.close()


@pytest.mark.parametrize("act", ["f16", "bf16"])
@pytest.mark.parametrize("kind,D", [("q8", 64), ("q8", 128), ("q8q4", 128), ("f16", 128)])
@pytest.mark.parametrize("sigma", [1.0, 8.0])
@pytest.mark.parametrize("T", [9, 100])
@pytest.mark.parametrize("kernel", [MMA, TC])
def test_lse_holds_32_bits_whatever_a_token_sees(kernel, T, sigma, kind, D, act):
    """The log-sum-exp of tokens that see one row, four, 64 and all of a long sequence, of flat and of peaked softmaxes, on
    either kernel: within the bound of operands of 20 bits; and the rows' weights that are formed from it sum to one for every
    query row that sees any, within the bounds of both."""
    import torch

    n, H, Hk, scale = 4096, 8, 2, float(np.float32(D**-0.5))
    tw = _twin(kind, H, Hk, D, n + 64, page=256)
    try:
        k, v = kv_inputs(31, 0, n, Hk, D, sigma=0.5)
        tw.append(0, 0, 0, k, v)
        q = _tensor(np.random.default_rng(T).standard_normal((T, H, D)) * sigma, act)
        vis = np.resize([1, 4, 64, n, 2, 1, 129, 0, 3000], T)
        got, z = _attend(tw, kernel, [0], [T], q, scale, vis)
        K, V = values(tw.ref.seqs[0].K[0]), values(tw.ref.seqs[0].V[0])
        qd = q.double().cpu().numpy()
        want, wz, mag, size = cross(qd, K, V, scale, vis)
        bo, bz = cross_bound(mag, size, n, D, act, 20, 11)
        zz = z.double().cpu().numpy()
        seen = vis > 0
        err = np.abs(zz[seen] - wz[seen])
        assert np.all(err <= bz[seen]), "lse off by %.3g, %.2f of its bound" % (err.max(), (err / bz[seen]).max())
        # out: P and V lose 11 bits each, K nothing.  A peaked softmax whose row holds a 0 leaves results of next to nothing:
        # below f16's normal range (2^-14) a result is off by half of 2^-24, whatever its size, and the weights of at most n
        # rows, where fp16 has no bits left for them, by 2^-32 of the largest each
        out = np.abs(got.double().cpu().numpy() - want)
        bo = bo + (2.0**-25 if act == "f16" else 0) + n * 2.0**-32 * np.abs(V).max()
        assert np.all(out <= bo), "out off by %.3g, %.2f of its bound" % (out.max(), (out / bo).max())
        w = torch.zeros(1, Hk, n, device="cuda:0")
        nv = torch.from_numpy(vis.astype(np.int32)).to("cuda:0")
        tw.gpu.attn_weight(0, [0], [T], q, z, w, scale, n_vis=nv)
        total = w.double().sum(2).cpu().numpy()[0]
        for g in range(Hk):
            hs = slice(g * H // Hk, (g + 1) * H // Hk)
            rows = seen.sum() * H // Hk
            # each query row's weights: e^(lse's error), e^(a score's error) and the sums' (T r + 4) 2^-24
            lim = (2 * bz[seen, hs]).sum() + rows * (T * H // Hk + 4) * 2.0**-24
            assert abs(total[g] - rows) <= lim, "weights sum to %.6f of %d" % (total[g], rows)
    finally:
        tw.close()


@pytest.mark.parametrize("act", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("kind,D", [("q8", 64), ("q8", 128), ("q8q4", 128), ("f16", 64)])
@pytest.mark.parametrize("T", [3, 150])
@pytest.mark.parametrize("kernel", [MMA, TC])
def test_large_values_that_nobody_sees_change_nothing(kernel, T, kind, D, act):
    """Rows behind the last one that any token sees, whatever finite values they hold, leave results, log-sum-exps and weights
    as they are without them, bit by bit: the operands' powers of two come from rows that are seen."""
    import torch

    if act == "f32" and kernel == TC:
        pytest.skip("32-bit queries have one kernel")
    n, seen, H, Hk = 300, 150, 4, 2
    k, v = kv_inputs(37, 0, n, Hk, D, sigma=0.1)
    rng = np.random.default_rng(T)
    q = _tensor(rng.standard_normal((T, H, D)), act)
    vis = rng.integers(1, seen + 1, T)
    vis[0] = seen
    got = []
    for big in (1.0, 6e4 if kind == "f16" else 6e6):  # (q8_0 and q4_0 hold up to 127 and 8 x 65504, of either sign)
        kk, vv = k.copy(), v.copy()
        kk[seen:] *= np.float32(big) / np.abs(kk[seen:]).max()
        vv[seen:] *= np.float32(min(big, 5e5) if kind == "q8q4" else big) / np.abs(vv[seen:]).max()
        tw = _twin(kind, H, Hk, D, n + 64)
        try:
            tw.gpu.append(0, 0, 0, _tensor(kk), _tensor(vv))
            o, z = _attend(tw, kernel, [0], [T], q, D**-0.5, vis)
            w = torch.zeros(1, Hk, n, device="cuda:0")
            tw.gpu.attn_weight(0, [0], [T], q, z, w, D**-0.5, n_vis=torch.from_numpy(vis.astype(np.int32)).to("cuda:0"))
            got.append((o, z, w))
            assert tw.kvc.kvc_check_device_error(tw.gpu.ctx) == 0
        finally:
            tw.close()
    for a, b in zip(*got):
        assert bool(torch.isfinite(a.float()).all()) and bool((a == b).all())
    assert bool((got[0][2][:, :, seen:] == 0).all())
