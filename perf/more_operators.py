"""Cases of a drafted block's step over the quantised KV cache: what is measured, and their plain forms.

Three operators, used one after the other by a program that decodes with drafted tokens (and the first of them by one
that reads prompts):

  append  new tokens' queries and keys as the projections leave them, each head normalised and turned to its token's
          position; keys and values quantised into the cache, queries handed back   (kvc.KVCache.append_rope)
  tree    each drafted token attends over the rows before the block, its ancestors in the block's tree and itself
                                                                                    (kvc.KVCache.attn_tree)
  keep    the rows of the accepted path stay, the block's others leave              (kvc.KVCache.keep)

`own` False computes them from the stored codes and scales in plain torch operations in 32 bits (angles in 64); True
calls the library.  K and V rows are stored as q8_0, f16, or q8_0 K with q4_0 V, and are quantised by the steps that
include/kvc.h gives for its types.
"""
import functools
import math
import random

import numpy as np
import torch

own = False

Q8_0, F16, Q8_Q4 = "q8_0", "f16", "q8_0/q4_0"
ACTS = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-6


# ------------------------------------------------------------------ cases --
def _case(op, name, shape, kv, act, seqs, rows, tok, layers=1, norm=True, fused=True, rope="neox", base=1e6, start=0,
          page=256):
    """rows and tok: "lo:hi", each sequence's drawn between them (by `mix`): rows in the cache before the block, the
    block's tokens.  fused: queries, keys and values lie side by side, as one projection leaves them.  start: the
    position of a sequence's first row."""
    heads, heads_kv, dim = shape
    return {"name": name, "op": op, "heads": heads, "heads_kv": heads_kv, "dim": dim, "kv": kv, "act": act,
            "seqs": seqs, "rows": rows, "tok": tok, "layers": layers, "norm": norm, "fused": fused, "rope": rope,
            "base": base, "start": start, "page": page, "mix": 11}


SMALL, BIG, FOUR = (8, 2, 64), (40, 8, 128), (32, 8, 128)


def listed():
    return [
        # one new token of one sequence (its query and the cached rows are read back by a token's attention): latency
        _case("append", "append one token", BIG, Q8_0, "bf16", 1, "100:100", "1:1"),
        # a batch of decoders, a token each
        _case("append", "append 32 sequences f16", FOUR, F16, "f16", 32, "64:400", "1:1", norm=False, page=64),
        # a prompt's block, far into a long text
        _case("append", "append 2048 tokens", BIG, Q8_0, "bf16", 1, "512:512", "2048:2048", start=100000),
        # an odd block in 32 bits over the asymmetric cache, adjacent pairs turned, positions beyond a million
        _case("append", "append 777 tokens f32", BIG, Q8_Q4, "f32", 1, "33:33", "777:777", fused=False, rope="norm",
              start=1500000),
        # a handful of drafted tokens over a short text: latency
        _case("tree", "tree 6 tokens 512 f32", SMALL, Q8_0, "f32", 1, "512:512", "6:6"),
        # a usual tree over a long context
        _case("tree", "tree 26 tokens 16k", BIG, Q8_0, "bf16", 1, "16384:16384", "26:26"),
        # a batch of trees, each over a context of its own length
        _case("tree", "tree ragged batch f16", FOUR, F16, "f16", 32, "1024:32768", "4:16"),
        # a large tree over a long context
        _case("tree", "tree 64 tokens 32k", BIG, Q8_0, "bf16", 1, "32768:32768", "64:64"),
        # 32-bit queries over the asymmetric cache
        _case("tree", "tree 33 x 4999 f32", BIG, Q8_Q4, "f32", 1, "4999:4999", "33:33"),
        # the whole step of a small model's layer
        _case("step", "step 4 tokens 300", SMALL, F16, "bf16", 1, "300:300", "4:4", norm=False, base=1e4, page=64),
        # eight layers of a usual tree's step, and the next token's attention
        _case("step", "step 26 tokens 16k x 8", BIG, Q8_0, "bf16", 1, "16384:16384", "26:26", layers=8),
        # two layers of a ragged batch over small pages
        _case("step", "step ragged batch", FOUR, Q8_0, "f16", 16, "300:3000", "3:9", layers=2, page=16),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "tree", "tree", "step"])
    shape = rng.choice([SMALL, BIG, FOUR, (8, 8, 64), (6, 2, 128), (16, 2, 64)])
    kv = rng.choice([Q8_0, F16, Q8_Q4] if shape[2] == 128 else [Q8_0, F16])
    # (rows that a step computes and quantises itself are read back in 16 bits)
    act = rng.choice(["f16", "bf16"] if op == "step" else ["f32", "f16", "bf16"])
    seqs = rng.choice([1, 1, 1, 2, 5, 16])
    if op == "append":
        hi, tok, layers = _log(rng, 1, 1024), _log(rng, 1, 2048 // seqs), 1
    elif op == "tree":
        hi, layers = _log(rng, 64, 65536 // seqs), 1
        tok = _log(rng, 1, max(1, min(128, 64 * 32768 // (hi * seqs))))
    else:
        hi, tok = _log(rng, 64, 16384 // seqs), _log(rng, 1, 32)
        layers = rng.randint(1, max(1, min(6, 65536 // (hi * seqs))))
    lo = hi if seqs == 1 else max(1, hi // rng.randint(1, 16))
    case = _case(op, "", shape, kv, act, seqs, "%d:%d" % (lo, hi), "%d:%d" % (max(1, tok // 2), tok), layers,
                 norm=rng.random() < 0.6, fused=rng.random() < 0.7, rope=rng.choice(["neox", "norm"]),
                 base=rng.choice([1e4, 1e6]), start=rng.choice([0, rng.randrange(1 << 12), rng.randrange(1 << 21)]),
                 page=rng.choice([16, 64, 256]))
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


def _tree(seed, n):
    """A drafted tree of n tokens: each token's parent (-1: none), its depth, and a path from a root to a leaf."""
    rng = random.Random(seed)
    parent = [-1 if t == 0 else rng.randint(max(-1, t - 6), t - 1) for t in range(n)]
    depth = []
    for p in parent:
        depth.append(0 if p < 0 else depth[p] + 1)
    path, at = [], depth.index(max(depth))
    while at >= 0:
        path.append(at)
        at = parent[at]
    return parent, depth, path[::-1]


def _inputs(case, seed):
    """Context rows [layers, seqs, rows, heads_kv, dim] in 32 bits (padded to the longest), the block's raw queries,
    keys and values [layers, tokens, ...] packed one sequence after the other, the trees and the places."""
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    rows, tok = _lengths(case)
    rnd = functools.partial(torch.randn, generator=gen, device=dev)
    layers, heads, hk, dim, act = case["layers"], case["heads"], case["heads_kv"], case["dim"], ACTS[case["act"]]
    total = sum(tok)
    x = {"k": rnd(layers, len(rows), max(rows), hk, dim) * 0.5, "v": rnd(layers, len(rows), max(rows), hk, dim) * 0.5}
    raw = rnd(layers, total, heads + 2 * hk, dim).to(act)
    parts = raw.split([heads, hk, hk], 2)  # a projection's columns: tokens are heads + 2 hk head-rows apart
    x["qn"], x["kn"], x["vn"] = parts if case["fused"] else [p.contiguous() for p in parts]
    x["q_norm"] = 1 + 0.1 * rnd(dim) if case["norm"] else None
    x["k_norm"] = 1 + 0.1 * rnd(dim) if case["norm"] else None
    x["next"] = rnd(layers, len(rows), heads, dim)  # the next token's queries, already turned
    trees = [_tree(seed * 1000003 + i, t) for i, t in enumerate(tok)]
    flat = lambda k: [p for t in trees for p in t[k]]  # noqa: E731
    chain = [t for n in tok for t in range(n)]
    x["parent"] = torch.tensor(flat(0), device=dev, dtype=torch.int32)
    x["path"] = [t[2] for t in trees]
    first = [case["start"] + n for n in rows]
    seq = [i for i, n in enumerate(tok) for _ in range(n)]
    at = chain if case["op"] == "append" else flat(1)
    x["pos"] = np.array([first[i] + a for i, a in zip(seq, at)], np.int32)
    x["seq_of"], x["tok_of"] = torch.tensor(seq, device=dev), torch.tensor(chain, device=dev)
    x["rows"], x["tok"], x["scale"] = rows, tok, 1.0 / math.sqrt(dim)
    return x


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


def prepare(case, seed):
    x = _inputs(case, seed)
    rows, tok, dev = x["rows"], x["tok"], x["next"].device
    s = {k: x[k] for k in ("qn", "kn", "vn", "q_norm", "k_norm", "next", "parent", "path", "pos", "rows", "tok",
                           "scale", "seq_of", "tok_of")}
    s.update(op=case["op"], layers=case["layers"], heads_kv=case["heads_kv"], rope=case["rope"], base=case["base"],
             types=_types(case["kv"]), act=ACTS[case["act"]])
    s["n"] = torch.tensor(rows, device=dev)
    s["n_tok"] = torch.tensor(tok, device=dev)
    tk, tv = s["types"]
    k, v = x["k"], x["v"]
    if case["op"] == "tree":
        # the block's rows are in the cache, as an append of the same tokens left them; the queries come from it too
        block = _turned(s, x["kn"], x["k_norm"]), x["vn"].float()
        s["q"] = _turned(s, x["qn"], x["q_norm"]).to(s["act"])[0]
    if not own:
        room = (0, 0, 0, 0, 0, max(tok))
        s["k"], s["v"] = ({a: t.contiguous() for a, t in _store(torch.nn.functional.pad(t, room), kind).items()}
                          for t, kind in ((k, tk), (v, tv)))
        if case["op"] == "tree":
            _put(s, *block)
        else:
            moves = [(i, rows[i] + a, rows[i] + b) for i, p in enumerate(s["path"]) for b, a in enumerate(p)]
            s["moves"] = torch.tensor(moves, device=dev).T
            s["kept"] = torch.tensor([len(p) for p in s["path"]], device=dev)
        return s
    from kv_cache_decode_flash_gb300 import kvc

    kinds = {Q8_0: kvc.KVC_Q8_0, F16: kvc.KVC_F16, "q4_0": kvc.KVC_Q4_0}
    cache = kvc.KVCache(case["layers"], case["heads"], case["heads_kv"], case["dim"], n_ctx=sum(rows) + sum(tok),
                        n_seq_max=len(rows), type_k=kinds[tk], type_v=kinds[tv], rope_base=case["base"],
                        rope_mode=kvc.KVC_ROPE_NEOX if case["rope"] == "neox" else kvc.KVC_ROPE_NORM,
                        page_rows=case["page"])
    t0 = 0
    for i, n in enumerate(rows):
        for layer in range(case["layers"]):
            cache.append(layer, i, case["start"], k[layer, i, :n], v[layer, i, :n])
        if case["op"] == "tree":
            kb, vb = (b[0, t0:t0 + tok[i]].contiguous() for b in block)
            cache.append(0, i, case["start"] + n, kb, vb)
            t0 += tok[i]
    s["cache"], s["ids"] = cache, list(range(len(rows)))
    s["none"] = [[] for _ in rows]
    s["one"] = [1] * len(rows)
    s["n_kept"] = [len(p) for p in s["path"]]
    return s


# ------------------------------------------------------------ plain forms --
def _turned(s, x, weight):
    """Heads normalised (where there is a weight) and turned to their tokens' positions, in 32 bits."""
    x = x.float()
    dim = x.shape[-1]
    if weight is not None:
        x = x * (x.square().mean(-1, keepdim=True) + EPS).rsqrt() * weight
    theta = s["base"] ** (-2.0 * torch.arange(dim // 2, device=x.device, dtype=torch.float64) / dim)
    angle = torch.from_numpy(s["pos"]).to(x.device)[:, None, None] * theta
    cos, sin = angle.cos().float(), angle.sin().float()
    if s["rope"] == "neox":
        a, b = x[..., :dim // 2], x[..., dim // 2:]
        return torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)


def _put_part(s, part, new):
    at = (slice(None), s["seq_of"], s["n"][s["seq_of"]] + s["tok_of"])
    for a in part:
        part[a][at] = new[a]


def _put(s, k, v):
    """The block's keys and values, quantised, behind each sequence's rows."""
    _put_part(s, s["k"], _store(k, s["types"][0]))
    _put_part(s, s["v"], _store(v, s["types"][1]))


def _attend(s, q, sees):
    """q [layers, seqs, tokens, heads, dim] over the stored rows that it sees [seqs, tokens, rows]; 0 where none."""
    k, v = _value(s["k"]).permute(0, 1, 3, 2, 4), _value(s["v"]).permute(0, 1, 3, 2, 4)
    layers, seqs, tokens, heads, dim = q.shape
    q = q.float().unflatten(3, (s["heads_kv"], -1)).permute(0, 1, 3, 4, 2, 5).flatten(3, 4)
    sc = (q @ k.transpose(-1, -2)).mul_(s["scale"]).unflatten(3, (-1, tokens))
    sc = sc.masked_fill_(~sees[:, None, None], float("-inf"))
    m = sc.amax(-1, keepdim=True)
    p = sc.sub_(torch.where(m == float("-inf"), torch.zeros_like(m), m)).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.flatten(3, 4) @ v).unflatten(3, (-1, tokens))
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    return o.permute(0, 1, 4, 2, 3, 5).reshape(layers, seqs, tokens, heads, dim)


def _plain_tree(s, q):
    """q [layers, tokens, heads, dim], packed."""
    top, width = next(iter(s["k"].values())).shape[2], max(s["tok"])
    seqs, dev = len(s["tok"]), q.device
    # token t's ancestors and itself: paths of any length along the parents, by doubling
    one = torch.eye(width, device=dev).expand(seqs, -1, -1).clone()
    t = (s["parent"] >= 0).nonzero().squeeze(1)
    one[s["seq_of"][t], s["tok_of"][t], s["parent"][t].long()] = 1.0
    line = functools.reduce(lambda m, _: (m @ m).clamp_(max=1.0), range(max(1, width.bit_length())), one) > 0
    at = torch.arange(top, device=dev)[None] - s["n"][:, None]
    inside = (at >= 0) & (at < s["n_tok"][:, None])
    sees = line.gather(2, at.clamp(0, width - 1)[:, None].expand(-1, width, -1)) & inside[:, None]
    sees |= (at < 0)[:, None]
    padded = torch.zeros(q.shape[0], seqs, width, *q.shape[2:], device=dev)
    padded[:, s["seq_of"], s["tok_of"]] = q.float()
    return _attend(s, padded, sees)[:, s["seq_of"], s["tok_of"]].to(s["act"])


def _plain_next(s, q, n):
    """A token of every sequence over its leading n rows."""
    at = torch.arange(next(iter(s["k"].values())).shape[2], device=q.device)
    return _attend(s, q[:, :, None], (at < n[:, None])[:, None])[:, :, 0]


def _plain_append(s):
    _put(s, _turned(s, s["kn"], s["k_norm"]), s["vn"].float())
    return _turned(s, s["qn"], s["q_norm"]).to(s["act"])


def _plain_step(s):
    q = _plain_append(s)
    out = _plain_tree(s, q)
    seq, src, dst = s["moves"]
    for part in (s["k"], s["v"]):
        for a in part:
            part[a][:, seq, dst] = part[a][:, seq, src]
    return q, out, _plain_next(s, s["next"].to(s["act"]), s["n"] + s["kept"]).to(s["act"])


def run(s):
    if not own:
        if s["op"] == "tree":
            return _plain_tree(s, s["q"][None])[0]
        if s["op"] == "append":
            q = _plain_append(s)
            return q, _plain_next(s, s["next"].bfloat16(), s["n"] + s["n_tok"]).bfloat16()
        return _plain_step(s)
    cache, ids, tok = s["cache"], s["ids"], s["tok"]
    if s["op"] == "tree":
        out = torch.empty_like(s["q"])
        cache.attn_tree(0, ids, tok, s["q"], out, s["scale"], parent=s["parent"])
        return out
    q = torch.empty(s["qn"].shape, device=s["qn"].device, dtype=s["act"])
    if s["op"] == "append":
        # the rows are read back by a token of every sequence, then leave, so that the next pass finds the same cache
        cache.append_rope(0, ids, tok, s["pos"], s["qn"][0], s["kn"][0], s["vn"][0], q[0], q_norm=s["q_norm"],
                          k_norm=s["k_norm"], eps=EPS)
        probe = s["next"].bfloat16()
        back = torch.empty_like(probe)
        cache.attn_tree(0, ids, s["one"], probe[0], back[0], s["scale"])
        cache.keep(ids, tok, s["none"])
        return q, back
    out = torch.empty_like(q)
    for layer in range(s["layers"]):
        cache.append_rope(layer, ids, tok, s["pos"], s["qn"][layer], s["kn"][layer], s["vn"][layer], q[layer],
                          q_norm=s["q_norm"], k_norm=s["k_norm"], eps=EPS)
        cache.attn_tree(layer, ids, tok, q[layer], out[layer], s["scale"], parent=s["parent"])
    cache.keep(ids, tok, s["path"])
    # the next token of every sequence, over what is left
    after_q = s["next"].to(s["act"])
    after = torch.empty_like(after_q)
    for layer in range(s["layers"]):
        cache.attn_tree(layer, ids, s["one"], after_q[layer], after[layer], s["scale"])
    cache.keep(ids, s["n_kept"], s["none"])  # as it was, for the next pass
    return q, out, after


# ------------------------------------------------------------------- work --
def _row_bytes(kind, dim):
    return {F16: 2 * dim, Q8_0: dim + dim // 16, "q4_0": dim // 2 + dim // 16}[kind]


def work(case):
    tk, tv = _types(case["kv"])
    hk, dim, heads, layers = case["heads_kv"], case["dim"], case["heads"], case["layers"]
    row = hk * (_row_bytes(tk, dim) + _row_bytes(tv, dim))
    rows, tok = _lengths(case)
    act = 4 if case["act"] == "f32" else 2
    total, n = sum(tok), sum(rows)
    pairs = sum(r * t for r, t in zip(rows, tok)) + 4 * total  # (a token has a few ancestors)
    block = total * (2 * heads + 2 * hk) * dim * act + total * row + 4 * total  # projections in, queries and rows out
    tree = (n + total) * row + 2 * total * heads * dim * act + 4 * total
    if case["op"] == "tree":
        return {"bytes": tree, "flops": 4 * pairs * heads * dim}
    if case["op"] == "append":
        probe = (n + total) * row + len(rows) * heads * dim * 4
        return {"bytes": block + probe, "flops": 10 * total * (heads + hk) * dim + 4 * (n + total) * heads * dim}
    kept = sum(len(_tree(i, t)[2]) for i, t in enumerate(tok))
    after = (n + kept) * row + 4 * len(rows) * heads * dim
    return {"bytes": layers * (block + tree + 2 * kept * row + after),
            "flops": layers * (10 * total * (heads + hk) * dim + 4 * pairs * heads * dim + 4 * (n + kept) * heads * dim)}


# ------------------------------------------------- in 64 bits, from the definition --
def _exact_value(x, kind):
    """Stored values of x [..., dim] in 64 bits: each 32-bit step of the types' definition is a 64-bit one, rounded."""
    f = lambda t: t.float().double()  # noqa: E731
    x = f(x)
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


def _exact_turn(case, pos, x, weight):
    x = x.double()
    dim = x.shape[-1]
    if weight is not None:
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / dim + EPS) * weight.double()
    pos = torch.tensor(pos.tolist(), device=x.device, dtype=torch.float64)
    out = torch.empty_like(x)
    for i in range(dim // 2):
        w = pos * math.exp(-2.0 * i / dim * math.log(case["base"]))
        c, s = torch.cos(w)[:, None], torch.sin(w)[:, None]
        u, v = (i, i + dim // 2) if case["rope"] == "neox" else (2 * i, 2 * i + 1)
        out[..., u] = x[..., u] * c - x[..., v] * s
        out[..., v] = x[..., u] * s + x[..., v] * c
    return out


def _exact_attn(q, k, v, sees, scale):
    """q [tokens, heads, dim], k and v [rows, heads_kv, dim], sees [tokens, rows], all in 64 bits."""
    t, heads, dim = q.shape
    hk = k.shape[1]
    outs = []
    for g in range(hk):
        sc = torch.einsum("tjd,nd->tjn", q.view(t, hk, -1, dim)[:, g], k[:, g]) * scale
        sc = torch.where(sees[:, None], sc, torch.full_like(sc, float("-inf")))
        outs.append(torch.softmax(sc, -1) @ v[:, g])
    return torch.stack(outs, 1).reshape(t, heads, dim)


def exact(case, seed):
    x = _inputs(case, seed)
    tk, tv = _types(case["kv"])
    act = ACTS[case["act"]]
    parent = x["parent"].tolist()
    turned, outs, after = [], [], []
    for layer in range(case["layers"]):
        qn = _exact_turn(case, x["pos"], x["qn"][layer], x["q_norm"])
        kn = _exact_value(_exact_turn(case, x["pos"], x["kn"][layer], x["k_norm"]), tk)
        vn = _exact_value(x["vn"][layer], tv)
        turned.append(qn)
        if case["op"] == "tree":  # the cache and the queries are inputs: as prepare() made them, in 32 bits
            s = {"pos": x["pos"], "rope": case["rope"], "base": case["base"]}
            kn = _exact_value(_turned(s, x["kn"], x["k_norm"])[0], tk)
            qn = _turned(s, x["qn"], x["q_norm"])[0].to(act).double()
        else:
            qn = qn.to(act).double()  # handed over in the activations' type
        t0 = 0
        for i, (n, t) in enumerate(zip(x["rows"], x["tok"])):
            k = torch.cat([_exact_value(x["k"][layer, i, :n], tk), kn[t0:t0 + t]])
            v = torch.cat([_exact_value(x["v"][layer, i, :n], tv), vn[t0:t0 + t]])
            if case["op"] != "append":
                sees = torch.zeros(t, n + t, dtype=torch.bool)
                sees[:, :n] = True
                for a in range(t):
                    up = a
                    while up >= 0:
                        sees[a, n + up] = True
                        up = parent[t0 + up]
                outs.append(_exact_attn(qn[t0:t0 + t], k, v, sees.to(k.device), x["scale"]))
            if case["op"] != "tree":
                stay = list(range(n + t)) if case["op"] == "append" else list(range(n)) + [n + a for a in x["path"][i]]
                stay = torch.tensor(stay, device=k.device)
                nq = x["next"][layer, i]
                nq = nq.to(torch.bfloat16 if case["op"] == "append" else act).double()[None]
                every = torch.ones(1, len(stay), dtype=torch.bool, device=k.device)
                after.append(_exact_attn(nq, k[stay], v[stay], every, x["scale"])[0])
            t0 += t
    shape = (case["layers"], case["seqs"], case["heads"], case["dim"])
    if case["op"] == "tree":
        return torch.cat(outs)
    if case["op"] == "append":
        return torch.stack(turned), torch.stack(after).view(shape)
    total = sum(x["tok"])
    return torch.stack(turned), torch.cat(outs).view(case["layers"], total, *shape[2:]), torch.stack(after).view(shape)
