"""Cases of the attention operators over the quantised KV cache: what is measured, and their plain forms.

Three operators, used one after the other by a program that serves long prompts from the cache:

  cross   every token of a block attends over the rows of a sequence (an encoder's states, an image's, a
          prompt's), each token over its own number of leading rows; the natural logarithm of the softmax's
          sum comes with it                                                           (kvc.KVCache.attn_cross)
  weight  the softmax weight that each cached row receives from a block of tokens, summed per KV head into
          accumulators                                                               (kvc.KVCache.attn_weight)
  evict   the rows of the least accumulated weight leave the cache, every layer's and head's, and the last
          rows take their places                                               (kvc.KVCache.evict_weight)

`own` False computes them from the stored codes and scales in plain torch operations in 32 bits; True calls
the library.  K and V rows are stored as q8_0, f16, or q8_0 K with q4_0 V, and are quantised by the steps
that include/kvc.h gives for its types.
"""
import functools
import math
import random

import torch

own = False

Q8_0, F16, Q8_Q4 = "q8_0", "f16", "q8_0/q4_0"
ACTS = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ cases --
def _attn(op, name, heads, heads_kv, dim, kv, act, seqs, rows, tok, see="all", page=256):
    """rows and tok: "lo:hi", each sequence's drawn between them (by `mix`); see: the leading rows that a token
    sees: all of them, causal (the block's tokens are the sequence's last rows), or ragged (any number, none too)."""
    return {"name": name, "op": op, "heads": heads, "heads_kv": heads_kv, "dim": dim, "kv": kv, "act": act,
            "seqs": seqs, "rows": rows, "tok": tok, "see": see, "page": page, "mix": 7}


def _evict(name, heads, heads_kv, dim, kv, layers, rows, block, page=256):
    return {"name": name, "op": "evict", "heads": heads, "heads_kv": heads_kv, "dim": dim, "kv": kv,
            "layers": layers, "rows": rows, "block": block, "page": page}


def listed():
    return [
        # one decoder token over a short encoder's states: latency alone
        _attn("cross", "cross one token 512", 8, 2, 64, Q8_0, "f32", 1, "512:512", "1:1"),
        # a few drafted tokens verified over a long context
        _attn("cross", "cross 5 tokens 16k", 40, 8, 128, Q8_0, "bf16", 1, "16384:16384", "5:5", "causal"),
        # a batch of decoders, each over a prompt of its own length, a few tokens each
        _attn("cross", "cross ragged batch f16", 32, 8, 128, F16, "f16", 32, "1024:32768", "1:8"),
        # a prompt over an encoder's 1500 states
        _attn("cross", "cross 512 x 1500 f16", 32, 8, 128, F16, "f16", 1, "1500:1500", "512:512"),
        # the last 2048 tokens of a 16k prompt
        _attn("cross", "cross 2048 x 16k causal", 40, 8, 128, Q8_0, "bf16", 1, "16384:16384", "2048:2048", "causal"),
        # a padded block in 32 bits over the asymmetric cache; some tokens see nothing
        _attn("cross", "cross 257 x 4999 f32", 40, 8, 128, Q8_Q4, "f32", 1, "4999:4999", "257:257", "ragged"),
        # a decode step's weights
        _attn("weight", "weight one token 16k", 40, 8, 128, Q8_0, "f32", 1, "16384:16384", "1:1"),
        # a prompt's last 32 tokens say which of 131072 rows matter
        _attn("weight", "weight 32 tokens 128k", 40, 8, 128, Q8_0, "bf16", 1, "131072:131072", "32:32", "causal"),
        # a small ragged batch of short odd prompts
        _attn("weight", "weight ragged f16", 8, 2, 64, F16, "f16", 4, "400:1300", "3:40", "causal", 64),
        # one layer of a short cache at its limit: a block comes, as many rows go
        _evict("evict 64 of 512", 8, 2, 64, F16, 1, 512, 64, 64),
        # sixteen layers at their limit of 32768 rows: a block of 1024 tokens comes, as many rows go
        _evict("evict 1024 of 32k x 16", 40, 8, 128, Q8_0, 16, 32768, 1024),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["cross", "cross", "weight", "evict"])
    heads, heads_kv, dim = rng.choice([(8, 2, 64), (40, 8, 128), (32, 8, 128), (8, 8, 64), (6, 2, 128), (16, 2, 64)])
    kv = rng.choice([Q8_0, F16, Q8_Q4] if dim == 128 else [Q8_0, F16])
    page = rng.choice([16, 64, 256])
    if op == "evict":
        rows = _log(rng, 100, 32768)
        layers = rng.randint(1, max(1, min(16, 16 * 32768 * 8 // (rows * heads_kv * 4))))
        case = _evict("", heads, heads_kv, dim, kv, layers, rows, _log(rng, 1, max(1, rows // 8)), page)
        del case["name"]
        return case
    act = rng.choice(["f32", "f16", "bf16"])
    seqs = rng.choice([1, 1, 1, 2, 5, 16])
    hi = _log(rng, 64, 131072 // seqs)
    lo = hi if seqs == 1 else max(1, hi // rng.randint(1, 16))
    most = 2048 if op == "cross" else 64
    tok = _log(rng, 1, max(1, min(most, 2048 * 16384 // (hi * seqs))))
    case = _attn(op, "", heads, heads_kv, dim, kv, act, seqs, "%d:%d" % (lo, hi), "%d:%d" % (max(1, tok // 2), tok),
                 rng.choice(["all", "causal", "ragged"]), page)
    del case["name"]
    case["mix"] = rng.randrange(1 << 20)
    return case


def _lengths(case):
    rng = random.Random(case["mix"])
    span = [tuple(int(x) for x in case[k].split(":")) for k in ("rows", "tok")]
    return [[rng.randint(*s) for _ in range(case["seqs"])] for s in span]


# ----------------------------------------------------------------- inputs --
def _types(kv):
    return (Q8_0, "q4_0") if kv == Q8_Q4 else (kv, kv)


def _round_away(x):
    """To the nearest integer, halves away from zero (the sum is exact in 64 bits)."""
    return torch.sign(x) * torch.floor(x.abs().double() + 0.5)


def _store(x, kind):
    """x [..., dim] in 32 bits as its stored form: halves, or codes and one fp16 scale for each 32 values."""
    if kind == F16:
        return {"half": x.half()}
    b = x.unflatten(-1, (-1, 32))
    if kind == Q8_0:
        top = b.abs().amax(-1, keepdim=True)
        d = top / torch.full_like(top, 127.0)  # by a tensor: a division by a number is a product with its inverse
        inv = torch.where(d != 0, 1.0 / d, torch.zeros_like(d))
        codes = _round_away(b * inv).to(torch.int8)
    else:
        top = b.gather(-1, b.abs().argmax(-1, keepdim=True))
        d = top / -8.0
        inv = torch.where(d != 0, 1.0 / d, torch.zeros_like(d))
        codes = (b * inv + 8.5).trunc().clamp(max=15.0).to(torch.int8) - 8
    return {"codes": codes.flatten(-2), "scale": d.squeeze(-1).half()}


def _value(s):
    """The stored values in 32 bits (exact: a code of at most 8 bits times a scale of 11)."""
    if "half" in s:
        return s["half"].float()
    return (s["codes"].float().unflatten(-1, (-1, 32)) * s["scale"].float().unsqueeze(-1)).flatten(-2)


def _kvc_types(kvc, kv):
    return {Q8_0: (kvc.KVC_Q8_0, kvc.KVC_Q8_0), F16: (kvc.KVC_F16, kvc.KVC_F16),
            Q8_Q4: (kvc.KVC_Q8_0, kvc.KVC_Q4_0)}[kv]


def _cache(case, layers, n_ctx, seqs):
    from kv_cache_decode_flash_gb300 import kvc

    tk, tv = _kvc_types(kvc, case["kv"])
    return kvc.KVCache(layers, case["heads"], case["heads_kv"], case["dim"], n_ctx=n_ctx, n_seq_max=seqs, type_k=tk,
                       type_v=tv, page_rows=case["page"])


def _inputs(case, seed):
    """The inputs of an attention case: K and V [seqs, rows, heads_kv, dim] in 32 bits (padded to the longest
    sequence), the tokens' queries packed one sequence after the other, and where they belong."""
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    rows, tok = _lengths(case)
    rnd = functools.partial(torch.randn, generator=gen, device=dev)
    top = max(rows)
    k = rnd(len(rows), top, case["heads_kv"], case["dim"]) * 0.5
    v = rnd(len(rows), top, case["heads_kv"], case["dim"]) * 0.5
    total = sum(tok)
    q = rnd(total, case["heads"], case["dim"]).to(ACTS[case["act"]])
    seq_of = torch.repeat_interleave(torch.arange(len(tok), device=dev), torch.tensor(tok, device=dev))
    tok_of = torch.cat([torch.arange(t, device=dev) for t in tok])
    rows_d, tok_d = torch.tensor(rows, device=dev), torch.tensor(tok, device=dev)
    if case["see"] == "causal":
        vis = (rows_d[seq_of] - tok_d[seq_of] + tok_of + 1).clamp(min=0)
    elif case["see"] == "ragged":
        some = torch.rand(total, generator=gen, device=dev)
        vis = torch.where(some < 0.1, torch.zeros_like(some), some * (rows_d[seq_of] + 1)).floor()
    else:
        vis = rows_d[seq_of]
    return {"k": k, "v": v, "q": q, "rows": rows, "tok": tok, "seq_of": seq_of, "tok_of": tok_of,
            "vis": vis.to(torch.int32), "scale": 1.0 / math.sqrt(case["dim"]), "gen": gen}


def _earlier(case, x):
    """Weights that earlier blocks of the same size left: half of what this one brings, on average."""
    share = max(x["tok"]) * case["heads"] / case["heads_kv"] / max(x["rows"])
    return torch.rand(len(x["rows"]), case["heads_kv"], max(x["rows"]), generator=x["gen"], device=x["q"].device) * share


def prepare(case, seed):
    if case["op"] == "evict":
        return _prepare_evict(case, seed)
    x = _inputs(case, seed)
    s = {"op": case["op"], "heads_kv": case["heads_kv"], "tok": x["tok"], "rows": x["rows"], "q": x["q"],
         "vis": None if case["see"] == "all" else x["vis"], "scale": x["scale"], "seq_of": x["seq_of"],
         "tok_of": x["tok_of"], "lengths": torch.tensor(x["rows"], device=x["q"].device, dtype=torch.int32)}
    tk, tv = _types(case["kv"])
    if case["op"] == "weight":
        # the block's statistics, as the attention of the same tokens left them, and the weights of earlier blocks
        sc = _scores(dict(s, k=_store(x["k"], tk)))
        s["lse"] = torch.logsumexp(sc.double(), -1).float()[s["seq_of"], :, s["tok_of"]].contiguous()
        del sc
        s["w"] = _earlier(case, x)
    if not own:
        s["k"] = _store(x["k"], tk)
        if case["op"] == "cross":
            s["v"] = _store(x["v"], tv)
        return s
    s["cache"] = _cache(case, 1, sum(x["rows"]), len(x["rows"]))
    for i, n in enumerate(x["rows"]):
        s["cache"].append(0, i, 0, x["k"][i, :n], x["v"][i, :n])
    s["ids"] = list(range(len(x["rows"])))
    return s


def _prepare_evict(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    rnd = functools.partial(torch.randn, generator=gen, device=dev)
    n, m, layers, hk, dim = case["rows"], case["block"], case["layers"], case["heads_kv"], case["dim"]
    tk, tv = _types(case["kv"])
    s = {"op": "evict", "layers": layers, "n": n, "block": m, "keep": min(n // 8, 64), "next": n,
         "scale": 1.0 / math.sqrt(dim), "heads_kv": hk, "types": (tk, tv)}
    if own:
        s["cache"] = _cache(case, layers, n + m, 1)
    else:
        s["pos"] = torch.cat([torch.arange(n, device=dev), torch.zeros(m, device=dev, dtype=torch.long)]).to(torch.int32)
    parts = []
    for layer in range(layers):
        k, v = rnd(n, hk, dim) * 0.5, rnd(n, hk, dim) * 0.5
        if own:
            s["cache"].append(layer, 0, 0, k, v)
        else:
            room = (0, 0, 0, 0, 0, m)  # room for the block behind the rows
            parts.append([{a: torch.nn.functional.pad(b, room) for a, b in _store(t, kind).items()}
                          for t, kind in ((k, tk), (v, tv))])
    if not own:
        s["k"], s["v"] = ({a: torch.stack([p[i][a] for p in parts]) for a in parts[0][i]} for i in (0, 1))
    # the block's keys and values and the next token's queries, by layer; the weights accumulated so far
    s["kn"], s["vn"] = rnd(layers, m, hk, dim) * 0.5, rnd(layers, m, hk, dim) * 0.5
    s["q"] = rnd(layers, 1, case["heads"], dim)
    s["w"] = torch.cat([torch.rand(hk, n, generator=gen, device=dev).square(), torch.zeros(hk, m, device=dev)], 1)
    return s


# ------------------------------------------------------------ plain forms --
def _scores(s):
    """Scaled scores [seqs, heads, tokens, rows] of the padded blocks, -inf where a token does not see a row."""
    k = _value(s["k"])
    seqs, top = k.shape[0], k.shape[1]
    heads, dim = s["q"].shape[1:]
    q = torch.zeros(seqs, max(s["tok"]), heads, dim, device=k.device)
    q[s["seq_of"], s["tok_of"]] = s["q"].float()
    r = heads // s["heads_kv"]
    q = q.view(seqs, -1, s["heads_kv"], r, dim).permute(0, 2, 3, 1, 4).reshape(seqs, s["heads_kv"], -1, dim)
    sc = (q @ k.permute(0, 2, 3, 1)).mul_(s["scale"]).view(seqs, heads, -1, top)
    sees = torch.zeros(seqs, max(s["tok"]), device=k.device, dtype=torch.int32)
    sees[s["seq_of"], s["tok_of"]] = s["lengths"][s["seq_of"]] if s["vis"] is None else s["vis"]
    return sc.masked_fill_((torch.arange(top, device=k.device) >= sees[..., None])[:, None], float("-inf"))


def _plain_cross(s):
    sc = _scores(s)
    seqs, heads, tokens, top = sc.shape
    m = sc.amax(-1, keepdim=True)
    m = torch.where(m == float("-inf"), torch.zeros_like(m), m)
    p = sc.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    v = _value(s["v"]).permute(0, 2, 1, 3)
    o = (p.view(seqs, s["heads_kv"], -1, top) @ v).view(seqs, heads, tokens, -1)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    lse = (m + total.log()).squeeze(-1)
    at = (s["seq_of"], slice(None), s["tok_of"])
    return o[at].to(s["q"].dtype), lse[at]


def _plain_weight(s):
    sc = _scores(s)
    lse = torch.zeros(sc.shape[:3], device=sc.device)
    lse[s["seq_of"], :, s["tok_of"]] = s["lse"]
    p = sc.sub_(torch.where(lse == float("-inf"), torch.zeros_like(lse), lse)[..., None]).exp_()
    live = torch.zeros(sc.shape[0], sc.shape[2], device=sc.device)
    live[s["seq_of"], s["tok_of"]] = 1.0
    p = p.mul_(live[:, None, :, None])
    s["w"] += p.view(p.shape[0], s["heads_kv"], -1, p.shape[-1]).sum(2)
    return s["w"]


def _plain_evict(s):
    n, m = s["n"], s["block"]
    tk, tv = s["types"]
    new_k, new_v = _store(s["kn"], tk), _store(s["vn"], tv)
    for part, new in ((s["k"], new_k), (s["v"], new_v)):
        for a in part:
            part[a][:, n:] = new[a]
    s["pos"][n:] = torch.arange(s["next"], s["next"] + m, device=s["pos"].device, dtype=torch.int32)
    s["next"] += m
    weight = functools.reduce(torch.add, s["w"].unbind(0))
    open_ = (s["pos"] >= s["keep"]) & (s["pos"] < s["next"] - m)
    order = torch.sort(torch.where(open_, weight, torch.full_like(weight, float("inf"))), stable=True).indices
    gone = torch.zeros(n + m, device=order.device, dtype=torch.bool)
    gone[order[:m]] = True
    holes, movers = gone[:n].nonzero().squeeze(1), n + (~gone[n:]).nonzero().squeeze(1)
    for part in (s["k"], s["v"]):
        for a in part:
            part[a][:, holes] = part[a][:, movers]
    s["pos"][holes] = s["pos"][movers]
    s["w"][:, holes] = s["w"][:, movers]
    s["w"][:, n:] = 0.0
    k, v = ({a: t[:, :n] for a, t in part.items()} for part in (s["k"], s["v"]))
    layers, _, heads, dim = s["q"].shape
    q = s["q"].view(layers, s["heads_kv"], -1, dim)
    sc = (q @ _value(k).permute(0, 2, 3, 1)) * s["scale"]
    p = (sc - sc.amax(-1, keepdim=True)).exp()
    o = (p @ _value(v).permute(0, 2, 1, 3)) / p.sum(-1, keepdim=True)
    return s["pos"][:n].clone(), s["w"], o.view(layers, 1, heads, dim)


def run(s):
    if not own:
        return {"cross": _plain_cross, "weight": _plain_weight, "evict": _plain_evict}[s["op"]](s)
    cache = s["cache"]
    if s["op"] == "cross":
        out = torch.empty_like(s["q"])
        lse = torch.empty(s["q"].shape[:2], device=out.device)
        cache.attn_cross(0, s["ids"], s["tok"], s["q"], out, s["scale"], lse=lse, n_vis=s["vis"])
        return out, lse
    if s["op"] == "weight":
        cache.attn_weight(0, s["ids"], s["tok"], s["q"], s["lse"], s["w"], s["scale"], n_vis=s["vis"])
        return s["w"]
    # a cache at its limit: a block of tokens comes, as many rows of the least weight go (neither the first rows
    # nor the block itself), and the next token attends over what is left
    first = s["next"]
    s["next"] += s["block"]
    out = torch.empty_like(s["q"])
    for layer in range(s["layers"]):
        cache.append(layer, 0, first, s["kn"][layer], s["vn"][layer])
    cache.evict_weight(0, s["keep"], first, s["block"], s["w"])
    for layer in range(s["layers"]):
        cache.attn_decode(layer, [0], s["q"][layer], out[layer], s["scale"])
    return cache.positions(0), s["w"], out


# ------------------------------------------------------------------- work --
def _row_bytes(kind, dim):
    return {F16: 2 * dim, Q8_0: dim + dim // 16, "q4_0": dim // 2 + dim // 16}[kind]


def work(case):
    tk, tv = _types(case["kv"])
    hk, dim, heads = case["heads_kv"], case["dim"], case["heads"]
    kb, vb = hk * _row_bytes(tk, dim), hk * _row_bytes(tv, dim)
    if case["op"] == "evict":
        n, m, layers = case["rows"], case["block"], case["layers"]
        # the block is read in 32 bits and stored, the holes are filled, and every row is read by the attention
        return {"bytes": layers * (m * hk * dim * 8 + 3 * m * (kb + vb) + n * (kb + vb) + 8 * heads * dim)
                + 4 * hk * (n + m), "flops": layers * 4 * n * heads * dim}
    rows, tok = _lengths(case)
    act = 4 if case["act"] == "f32" else 2
    share = 0.45 if case["see"] == "ragged" else 1.0  # of the (token, row) pairs
    pairs = sum(r * t * share - (t * (t - 1) / 2 if case["see"] == "causal" else 0) for r, t in zip(rows, tok))
    pairs = max(pairs, sum(tok))
    total = sum(tok) * heads * dim
    if case["op"] == "weight":
        return {"bytes": sum(rows) * (kb + 8 * hk) + total * act + 4 * sum(tok) * heads, "flops": 2 * pairs * heads * dim}
    return {"bytes": sum(rows) * (kb + vb) + 2 * total * act + 4 * sum(tok) * heads, "flops": 4 * pairs * heads * dim}


# ------------------------------------------------- in 64 bits, from the definition --
def _exact_value(x, kind):
    """Stored values of x [..., dim] in 64 bits: each 32-bit step of the types' definition is a 64-bit one, rounded."""
    f = lambda t: t.float().double()  # noqa: E731
    x = x.double()
    if kind == F16:
        return x.half().double()
    b = x.reshape(*x.shape[:-1], -1, 32)
    if kind == Q8_0:
        d = f(b.abs().max(-1, keepdim=True).values / 127)
        y = f(b * torch.where(d > 0, f(1 / d), d))
        code = torch.where(y < 0, torch.ceil(y - 0.5), torch.floor(y + 0.5))
    else:
        place = torch.arange(32, device=b.device).expand_as(b)
        first = torch.where(b.abs() == b.abs().max(-1, keepdim=True).values, place, 32).min(-1, keepdim=True).values
        top = torch.where(place == first, b, torch.zeros_like(b)).sum(-1, keepdim=True)
        d = f(top / -8)
        y = f(f(b * torch.where(d != 0, f(1 / d), d)) + 8.5)
        code = torch.minimum(torch.trunc(y), torch.full_like(y, 15)) - 8
    return (code * d.half().double()).reshape(x.shape)


def exact(case, seed):
    if case["op"] == "evict":
        return _exact_evict(case, seed)
    x = _inputs(case, seed)
    tk, tv = _types(case["kv"])
    hk, r = case["heads_kv"], case["heads"] // case["heads_kv"]
    w = None
    if case["op"] == "weight":
        # as in prepare(): the accumulators are the next numbers of the same generator
        w = _earlier(case, x).double()
        state = {"q": x["q"], "heads_kv": hk, "tok": x["tok"], "scale": x["scale"], "vis": x["vis"],
                 "seq_of": x["seq_of"], "tok_of": x["tok_of"], "k": _store(x["k"], tk)}
        given = torch.logsumexp(_scores(state).double(), -1).float()[x["seq_of"], :, x["tok_of"]].double()
    outs, sums, t0 = [], [], 0
    for i, (n, t) in enumerate(zip(x["rows"], x["tok"])):
        k = _exact_value(x["k"][i, :n], tk)
        q = x["q"][t0:t0 + t].double().view(t, hk, r, -1)
        sees = torch.arange(n, device=k.device)[None, :] < x["vis"][t0:t0 + t, None]
        if w is not None:
            for g in range(hk):
                sc = torch.einsum("tjd,nd->tjn", q[:, g], k[:, g]) * x["scale"]
                e = torch.exp(sc - given[t0:t0 + t].view(t, hk, r)[:, g, :, None])
                w[i, g, :n] += torch.where(sees[:, None], e, torch.zeros_like(e)).sum((0, 1))
        else:
            v = _exact_value(x["v"][i, :n], tv)
            o, z = [], []
            for g in range(hk):
                sc = torch.einsum("tjd,nd->tjn", q[:, g], k[:, g]) * x["scale"]
                sc = torch.where(sees[:, None], sc, torch.full_like(sc, float("-inf")))
                one = torch.logsumexp(sc, -1)
                o.append(torch.exp(sc - one[..., None]).nan_to_num(nan=0.0) @ v[:, g])
                z.append(one)
            outs.append(torch.stack(o, 1).reshape(t, hk * r, -1))
            sums.append(torch.stack(z, 1).reshape(t, hk * r))
        t0 += t
    return w if w is not None else (torch.cat(outs), torch.cat(sums))


def _exact_evict(case, seed):
    keep_own = own
    try:
        globals()["own"] = False
        s = _prepare_evict(case, seed)
    finally:
        globals()["own"] = keep_own
    n, m, hk, layers = case["rows"], case["block"], case["heads_kv"], case["layers"]
    w = s["w"].cpu()
    weight = w[0].clone()
    for g in range(1, hk):  # the sum over the heads is defined in 32 bits, in their order
        weight += w[g]
    rank = sorted(range(s["keep"], n), key=lambda i: (float(weight[i]), i))
    gone = set(rank[:m])
    stay = [i for i in range(n + m) if i not in gone]
    tail, place = [i for i in stay if i >= n], [i for i in range(n) if i not in gone]
    at = list(range(n))
    for hole, mover in zip(sorted(g for g in gone if g < n), tail):
        at[hole] = mover
    assert len(place) + len(tail) == n
    at = torch.tensor(at, device=s["q"].device)
    after = torch.zeros_like(s["w"], dtype=torch.float64)
    after[:, :n] = s["w"].double()[:, at]
    outs = []
    for layer in range(layers):
        old = [{a: b[layer, :n] for a, b in s[p].items()} for p in ("k", "v")]
        k, v = (torch.cat([_value(o).double(), _exact_value(s[x][layer], kind)])[at]
                for o, x, kind in zip(old, ("kn", "vn"), s["types"]))
        q = s["q"][layer].double().view(hk, -1, case["dim"])
        a = torch.softmax(torch.einsum("gjd,ngd->gjn", q, k) * s["scale"], -1)
        outs.append(torch.einsum("gjn,ngd->gjd", a, v).reshape(1, case["heads"], -1))
    return None, after, torch.stack(outs)
