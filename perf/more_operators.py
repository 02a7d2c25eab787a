"""Measured cases of the 8-bit key-value cache and of attention with changed scores: the append
that quantises, the read-back, attention over the quantised cache, the step that does both, and
attention whose scores are capped, biased by distance or masked by a prefix.

Each case runs one operator in plain torch operations (fp32, rounded once at the end), or, with
`own` set, through the package's entry points.  Batches are drawn like workloads.py draws them:
a ragged token axis, a shuffled page pool, block tables.  What the append stores is read back
(its tokens' values, as bf16), so that the outputs are the values that the codes stand for.
"""
from __future__ import annotations

import math
import random

import torch

own = False

_LOW, _HIGH = -32, 31  # exponents of a row's scale


# ------------------------------------------------------------------------------------- cases
def _case(name, op, decodes, chunks, chunk, ctx, heads, d, bs, layout, spread="uniform", rot=0,
          interleaved=False, packed=False, cap=0.0, distance=False, visible=False):
    return dict(name=name, op=op, decodes=decodes, chunks=chunks, chunk=chunk, ctx=ctx,
                hq=heads[0], hkv=heads[1], d=d, bs=bs, layout=layout, spread=spread, rot=rot,
                interleaved=interleaved, packed=packed, cap=cap, distance=distance,
                visible=visible)


def listed():
    return [
        # one token of one request on a toy model, rotated and stored: the latency of a call
        _case("append one token", "append", 1, 0, 0, 100, (4, 2), 64, 16, 1, rot=64),
        # a prefill-heavy step: 8 prompts of about 1024 tokens beside 16 decodes
        _case("append chunks 8x1024", "append", 16, 8, 1024, 2048, (64, 8), 128, 64, 2, rot=128,
              packed=True),
        # short ragged requests read back (to be stored in another cache), odd heads
        _case("read back 37 requests", "gather", 37, 0, 0, 500, (15, 5), 64, 16, 3),
        # a few long contexts read back, each from some key on
        _case("read back long contexts", "gather", 6, 0, 0, 30000, (32, 8), 128, 32, 4),
        # decode-only batches: 64 requests of middling lengths
        _case("attend decode 64", "attend", 64, 0, 0, 4096, (32, 8), 128, 32, 5),
        # 256 requests, most short, some very long
        _case("attend long tail 256", "attend", 256, 0, 0, 2048, (64, 8), 128, 64, 6,
              spread="lognormal"),
        # chunked prefill: 8 chunks of 512 tokens after up to 8192 keys, 16 decodes
        _case("attend chunks 8x512", "attend", 16, 8, 512, 8192, (32, 8), 128, 64, 7),
        # a layer's whole step on a toy model: three decodes and a prompt of 32 tokens
        _case("step tiny", "step", 3, 1, 32, 100, (4, 2), 64, 16, 8, rot=64),
        # a mixed continuous-batching step at 2048 tokens: 120 decodes and a long chunk
        _case("step mixed 2048", "step", 120, 1, 1928, 8192, (32, 8), 128, 32, 9, rot=128,
              packed=True),
        # a model with capped scores: decode on the 16-bit cache
        _case("scored cap decode 48", "scored", 48, 0, 0, 3000, (32, 16), 128, 16, 10, cap=50.0),
        # a model without position embedding, its scores biased by distance: mixed batch
        _case("scored distance mixed", "scored", 32, 3, 700, 4000, (32, 8), 128, 32, 11,
              distance=True),
        # prompts whose first part (an image, an instruction) sees itself both ways, capped
        _case("scored prefix prompts", "scored", 4, 6, 900, 300, (16, 8), 64, 16, 12, cap=30.0,
              visible=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw_once(rng):
    op = rng.choice(["append", "gather", "attend", "attend", "step", "scored", "scored"])
    hkv = rng.choice([1, 2, 3, 4, 5, 8, 8, 16])
    g = rng.choice([1, 2, 3, 4, 4, 5, 7, 8, 8, 16])
    if g > 8 and hkv > 4 and hkv % 4 or hkv > 64 // g:
        hkv = 4
    d = rng.choice([64, 128, 128])
    c = _case("", op, _log(rng, 1, 257) - 1, rng.choice([0, 0, 1, 1, 2, 5, 9]), _log(rng, 2, 1000),
              _log(rng, 1, 16384) - 1, (hkv * g, hkv), d,
              rng.choice([4, 8, 16, 16, 24, 32, 32, 64, 100, 128]), rng.randrange(1 << 30),
              spread=rng.choice(["uniform", "lognormal"]))
    del c["name"]
    if op == "gather":
        c["chunks"] = 0
    if c["decodes"] + c["chunks"] == 0:
        c["decodes"] = 1
    if op in ("append", "step"):
        c.update(rot=16 * rng.randint(0, d // 16), interleaved=rng.random() < 0.5,
                 packed=rng.random() < 0.5)
    if op in ("attend", "scored"):
        kind = rng.choice([0, 1, 2, 3, 4]) if op == "scored" else rng.choice([0, 0, 0, 1, 2, 3])
        c.update(cap=rng.choice([5.0, 30.0, 50.0]) if kind in (1, 4) else 0.0,
                 distance=kind in (2, 4), visible=kind in (3, 4))
    return c


def draw(rng):
    """A case of the same ranges that costs no more than the largest listed one of its operator,
    neither in its own work nor in the plain form's padded scores and gathered keys."""
    most = {}
    for c in listed():
        most[c["op"]] = [max(v) for v in zip(most.get(c["op"], [0] * 4), _cost(c))]
    while True:
        c = _draw_once(rng)
        if all(x <= m for x, m in zip(_cost(c), most[c["op"]])):
            return c


def _cost(case):
    w, lay = work(case), _layout(case)
    pairs = keys = 0
    for group in _groups(lay):
        n, k = max(lay["q"][i] for i in group), max(lay["kv"][i] for i in group)
        pairs += len(group) * n * k * case["hq"]
        keys += len(group) * k * case["hkv"] * case["d"]
    if case["op"] in ("append", "gather"):
        pairs = 0
    return w["bytes"], w["flops"], pairs, keys


# ---------------------------------------------------------------------------------- lengths
def _layout(case):
    """Per sequence: q (query tokens), kv (keys after the append), visible (keys that every query
    sees) and start (the first key that is read back)."""
    r = random.Random(case["layout"])
    q = [1] * case["decodes"]
    q += [max(1, case["chunk"] - r.randrange(1 + case["chunk"] // 8)) for _ in range(case["chunks"])]
    kv = []
    for n in q:
        if case["spread"] == "uniform":
            ctx = r.randint(case["ctx"] // 8, case["ctx"])
        else:
            ctx = min(16384, int(case["ctx"] * math.exp(r.gauss(0.0, 1.0))))
        kv.append(ctx + n)
    visible = [r.randint(0, k) if case["visible"] else 0 for k in kv]
    start = [r.randint(0, k // 4) for k in kv]
    return dict(q=q, kv=kv, visible=visible, start=start)


def _groups(lay):
    """Sequences of one query token, and those of more."""
    return [g for g in ([i for i, n in enumerate(lay["q"]) if n == 1],
                        [i for i, n in enumerate(lay["q"]) if n > 1]) if g]


def _pairs(lay):
    """(query, key) pairs that the masks leave."""
    total = 0
    for n, k, v in zip(lay["q"], lay["kv"], lay["visible"]):
        c = k - n  # query i sees max(c + i + 1, v) keys
        first = min(n, max(0, v - c - 1))  # the queries that see v
        total += first * v + (c + 1 + first + c + n) * (n - first) // 2
    return total


def work(case):
    lay = _layout(case)
    t, hq, hkv, d, op = sum(lay["q"]), case["hq"], case["hkv"], case["d"], case["op"]
    wide, narrow = hkv * d * 4, hkv * (2 * d + 2)  # bytes of one token's K and V: bf16; codes, scales
    if op == "gather":
        n = sum(k - s for k, s in zip(lay["kv"], lay["start"]))
        return {"bytes": n * (wide + narrow), "flops": 2 * n * hkv * d}
    nbytes = flops = 0
    if op in ("append", "step"):  # read, stored, read back and returned
        at = {k - n + i for n, k in zip(lay["q"], lay["kv"]) for i in range(n)}
        nbytes += t * (2 * wide + 2 * narrow) + len(at) * case["rot"] * 4
        flops += 3 * t * (hq + hkv) * case["rot"] + 8 * t * hkv * d
        if case["rot"]:
            nbytes += 2 * t * hq * d * 2 if op == "append" else t * hq * d * 2
    if op in ("attend", "step", "scored"):
        keys = sum(lay["kv"]) - (t if op == "step" else 0)
        nbytes += keys * (wide if op == "scored" else narrow) + (0 if op == "step" else t * hq * 4)
        nbytes += t * hq * d * 2 * (1 if op == "step" and case["rot"] else 2)
        flops += 4 * d * hq * _pairs(lay)
    return {"bytes": nbytes, "flops": flops}


# ----------------------------------------------------------------------------------- inputs
def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    r = random.Random(seed)
    lay = _layout(case)
    hq, hkv, d, bs, op = case["hq"], case["hkv"], case["d"], case["bs"], case["op"]
    t = sum(lay["q"])
    nblk = [-(-k // bs) for k in lay["kv"]]
    pages = sum(nblk) + max(1, sum(nblk) // 16)
    ids = list(range(pages))
    r.shuffle(ids)
    width = max(nblk) + 2
    rows, at = [], 0
    for n in nblk:
        rows.append(ids[at:at + n] + [-1] * (width - n))
        at += n
    cu = [0]
    for n in lay["q"]:
        cu.append(cu[-1] + n)

    def i32(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    def rand(*shape):
        return torch.empty(shape, dtype=torch.bfloat16, device=dev).normal_(generator=gen)

    def tokens(*shape):  # keys and values: tokens of different norms
        x = torch.empty(shape, dtype=torch.float32, device=dev).normal_(generator=gen)
        return (x * (0.5 * x.new_empty(shape[:-1] + (1,)).normal_(generator=gen)).exp()).bfloat16()

    st = dict(case=case, block_size=bs, scale=d ** -0.5, block_table=i32(rows),
              cu_seqlens_q=i32(cu), kv_lens=i32(lay["kv"]), tokens=t)
    k, v = tokens(pages, bs, hkv, d), tokens(pages, bs, hkv, d)
    if op == "scored":
        st["k_pages"], st["v_pages"] = k, v
    else:
        st["k_pages"], ek = _quantise(k.float())
        st["v_pages"], ev = _quantise(v.float())
        st["kv_scales"] = torch.stack((ek, ev), -1).contiguous()
    del k, v
    # what is read back: the tokens appended here, or a gather's ranges
    start = lay["start"] if op == "gather" else [a - n for a, n in zip(lay["kv"], lay["q"])]
    cuk = [0]
    for a, b in zip(start, lay["kv"]):
        cuk.append(cuk[-1] + b - a)
    st["key_starts"], st["cu_seqlens_k"], st["keys"] = i32(start), i32(cuk), cuk[-1]
    if op in ("append", "step"):
        if case["packed"]:  # views of the projection's output, token rows (hq + 2 hkv) d apart
            qkv = rand(t, hq + 2 * hkv, d)
            st["q"], st["k_new"], st["v_new"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
            if op == "step" and not case["rot"]:
                st["q"] = st["q"].contiguous()
        else:
            st["q"], st["k_new"], st["v_new"] = rand(t, hq, d), tokens(t, hkv, d), tokens(t, hkv, d)
        if case["rot"]:
            half = case["rot"] // 2
            pos = torch.arange(max(lay["kv"]) + 1, device=dev, dtype=torch.float64)
            freq = 10000.0 ** (-torch.arange(half, device=dev, dtype=torch.float64) / half)
            ang = pos[:, None] * freq
            st["cos_sin"] = torch.cat((ang.cos(), ang.sin()), 1).float().contiguous()
    elif op != "gather":
        st["q"] = rand(t, hq, d)
    if case["distance"]:  # a geometric sequence, like the method's: 2^-(8 i / heads)
        st["slopes"] = torch.exp2(-8.0 * torch.arange(1, hq + 1, device=dev) / hq).float()
    if case["visible"]:
        st["visible_lens"] = i32(lay["visible"])
    st["groups"] = []
    for group in _groups(lay):
        tok = [cu[i] + j for i in group for j in range(lay["q"][i])]
        seq = [x for x, i in enumerate(group) for _ in range(lay["q"][i])]
        col = [j for i in group for j in range(lay["q"][i])]
        st["groups"].append(dict(
            ids=i32(group).long(), tok=i32(tok).long(), seq=i32(seq).long(), col=i32(col).long(),
            q_max=max(lay["q"][i] for i in group), blocks=max(nblk[i] for i in group)))
    return st


# --------------------------------------------------------------------------- the plain forms
def _quantise(x):
    """x [..., D] fp32: e4m3 codes, and per row the exponent e (+ 127) of its scale: the smallest
    one with max |x| <= 448 * 2^e."""
    top = x.abs().amax(-1)
    m, e = torch.frexp(top)  # top = m * 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
    e = (e - 9 + (m > 0.875)).clamp(_LOW, _HIGH)
    e = torch.where(top == 0, torch.full_like(e, _LOW), e)
    y = torch.ldexp(x, -e[..., None]).clamp(-448.0, 448.0)
    return y.to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def _values(codes, scales):
    return torch.ldexp(codes.float(), (scales.int() - 127)[..., None])


def _rotate(x, cos, sin, interleaved):
    """x [T, H, D] fp32 with its first 2 * cos.shape[1] elements rotated."""
    half = cos.shape[1]
    y = x.float()
    c, s = cos[:, None], sin[:, None]
    if interleaved:
        a, b = y[..., 0:2 * half:2], y[..., 1:2 * half:2]
        turned = torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    else:
        a, b = y[..., :half], y[..., half:2 * half]
        turned = torch.cat((a * c - b * s, b * c + a * s), -1)
    return torch.cat((turned, y[..., 2 * half:]), -1)


def _slots(st, cu, first, n):
    """Cache slots of n packed rows: row cu[s] + i is key first[s] + i of sequence s."""
    cu, bs = cu.long(), st["block_size"]
    t = torch.arange(n, device=cu.device)
    seq = torch.searchsorted(cu, t, right=True) - 1
    pos = first.long()[seq] + t - cu[seq]
    block = st["block_table"].long()[seq, torch.div(pos, bs, rounding_mode="floor")]
    return block * bs + pos % bs, pos


def _pool(x):
    """A pool as rows of tokens, codes as bytes (indexing takes no 8-bit floats)."""
    x = x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x
    return x.view(-1, *x.shape[2:])


def _append_plain(st):
    slot, pos = _slots(st, st["cu_seqlens_q"], st["key_starts"], st["tokens"])
    q, k = None, st["k_new"].float()
    if "cos_sin" in st:
        rows = st["cos_sin"][pos]
        half = rows.shape[1] // 2
        cos, sin = rows[:, :half], rows[:, half:]
        k = _rotate(k, cos, sin, st["case"]["interleaved"])
        q = _rotate(st["q"], cos, sin, st["case"]["interleaved"]).to(st["q"].dtype)
    kc, ke = _quantise(k)
    vc, ve = _quantise(st["v_new"].float())
    _pool(st["k_pages"])[slot] = kc.view(torch.uint8)
    _pool(st["v_pages"])[slot] = vc.view(torch.uint8)
    _pool(st["kv_scales"])[slot] = torch.stack((ke, ve), -1)
    return q


def _gather_plain(st):
    slot, _ = _slots(st, st["cu_seqlens_k"], st["key_starts"], st["keys"])
    scales = _pool(st["kv_scales"])[slot]
    k = _values(_pool(st["k_pages"])[slot].view(torch.float8_e4m3fn), scales[..., 0])
    v = _values(_pool(st["v_pages"])[slot].view(torch.float8_e4m3fn), scales[..., 1])
    return k.bfloat16(), v.bfloat16()


def _keys(st, group, name, which):
    """A group's keys (or values), every sequence's gathered whole: fp32 [s, keys, hkv, d]."""
    table = st["block_table"][group["ids"], :group["blocks"]].long().clamp(min=0)
    pages = st[name]
    if pages.dtype == torch.float8_e4m3fn:
        x = _values(pages.view(torch.uint8)[table].view(pages.dtype), st["kv_scales"][table][..., which])
    else:
        x = pages[table].float()
    return x.view(table.shape[0], -1, *pages.shape[2:])


def _attend_group(st, q, group, out, lse):
    hq, d = q.shape[1:]
    hkv = st["k_pages"].shape[2]
    cu, kv = st["cu_seqlens_q"].long(), st["kv_lens"].long()[group["ids"]]
    c0 = cu[group["ids"]]
    n = cu[group["ids"] + 1] - c0
    s, q_max = kv.shape[0], group["q_max"]
    col = torch.arange(q_max, device=q.device)
    rows = (c0[:, None] + col).clamp(max=q.shape[0] - 1)
    qs = q[rows].float().view(s, q_max, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4)
    k = _keys(st, group, "k_pages", 0).permute(0, 2, 3, 1)
    x = torch.matmul(qs.reshape(s, hkv, -1, d), k).mul_(st["scale"])  # [s, hkv, heads * q_max, keys]
    del k
    x = x.view(s, hkv, hq // hkv, q_max, -1)
    pos = (kv - n)[:, None] + col  # [s, q_max]
    key = torch.arange(x.shape[-1], device=q.device)
    if st["case"]["cap"]:
        x = x.div_(st["case"]["cap"]).tanh_().mul_(st["case"]["cap"])
    if "slopes" in st:
        away = (key - pos[..., None]).float()[:, None, None]
        x = x.add_(st["slopes"].view(1, hkv, -1, 1, 1) * away)
    last = pos if "visible_lens" not in st else torch.maximum(
        pos, st["visible_lens"].long()[group["ids"], None] - 1)
    x = x.masked_fill_((key > last[..., None])[:, None, None], float("-inf"))
    m = x.amax(-1, keepdim=True)
    p = x.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    v = _keys(st, group, "v_pages", 1).permute(0, 2, 1, 3)
    o = torch.matmul(p.view(s, hkv, -1, p.shape[-1]), v).view(s, hkv, hq // hkv, q_max, d) / total
    norm = (m + total.log()).squeeze(-1)
    at = group["seq"], group["col"]
    out[group["tok"]] = o.permute(0, 3, 1, 2, 4)[at].reshape(-1, hq, d).to(out.dtype)
    lse[group["tok"]] = norm.permute(0, 3, 1, 2)[at].reshape(-1, hq)


def _attend_plain(st, q):
    out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
    for group in st["groups"]:
        _attend_group(st, q, group, out, lse)
    return out, lse


def run(state):
    st, op = state, state["case"]["op"]
    if own:
        import continuous_batching_paged_gb300 as cb
        if op == "scored":
            out, lse = cb.scored_attention(
                st["q"], st["k_pages"], st["v_pages"], st["block_table"], st["cu_seqlens_q"],
                st["kv_lens"], st["block_size"], st["scale"], softcap=st["case"]["cap"],
                slopes=st.get("slopes"), visible_lens=st.get("visible_lens"), lse=True)
            return {"out": out, "lse": lse}
        pools = (st["k_pages"], st["v_pages"], st["kv_scales"])
        where = (st["block_table"], st["cu_seqlens_q"], st["kv_lens"], st["block_size"])
        res = {}
        if op == "append":
            q = cb.quant_append(st["q"] if "cos_sin" in st else None, st["k_new"], st["v_new"],
                                *pools, *where, cos_sin=st.get("cos_sin"),
                                interleaved=st["case"]["interleaved"])
            if q is not None:
                res["q"] = q
        elif op == "step":
            res["out"] = cb.quant_append_attention(
                st["q"], st["k_new"], st["v_new"], *pools, *where, st["scale"],
                cos_sin=st.get("cos_sin"), interleaved=st["case"]["interleaved"])
        elif op == "attend":
            out, lse = cb.quant_attention(
                st["q"], *pools, *where, st["scale"], softcap=st["case"]["cap"],
                slopes=st.get("slopes"), visible_lens=st.get("visible_lens"), lse=True)
            return {"out": out, "lse": lse}
        res["k"], res["v"] = cb.quant_gather(*pools, st["block_table"], st["cu_seqlens_k"],
                                             st["block_size"], st["keys"],
                                             key_starts=st["key_starts"])
        return res
    res = {}
    if op in ("append", "step"):
        q = _append_plain(st)
        if op == "append" and q is not None:
            res["q"] = q
        if op == "step":
            res["out"], _ = _attend_plain(st, st["q"] if q is None else q)
    if op in ("attend", "scored"):
        out, lse = _attend_plain(st, st["q"])
        return {"out": out, "lse": lse}
    res["k"], res["v"] = _gather_plain(st)
    return res


# ------------------------------------------------------------------------ the values in 64 bits
def _stored(x):
    """What the cache holds of x [..., D] (64 bits): each row in steps of its own scale."""
    top = x.abs().max(-1, keepdim=True).values
    e = torch.ceil(torch.log2(top.clamp(min=1e-300) / 448.0))
    e = e + (top > 448.0 * 2.0 ** e).double() - (top <= 448.0 * 2.0 ** (e - 1)).double()  # log2 rounds
    e = e.clamp(_LOW, _HIGH)
    y = (x / 2.0 ** e).clamp(-448.0, 448.0)
    step = 2.0 ** (torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step * 2.0 ** e  # (round: halves to even)


def exact(case, seed):
    """The operators' definitions, sequence by sequence in 64 bits.  A step's attention reads
    what the step stores, and its rotated queries rounded to bf16."""
    st = prepare(case, seed)
    lay, op = _layout(case), case["op"]
    bs, hq, hkv, d = case["bs"], case["hq"], case["hkv"], case["d"]
    if op in ("attend", "step", "scored") and _pairs(lay) * hq * d > 2e11:
        return None
    dev = st["k_pages"].device
    table = st["block_table"].tolist()

    def cached(i, name, which, first, last):
        pos = torch.arange(first, last, device=dev)
        blk = torch.tensor(table[i], device=dev)[pos // bs]
        if op == "scored":
            return st[name][blk, pos % bs].double()
        codes = st[name].view(torch.uint8)[blk, pos % bs].view(torch.float8_e4m3fn).double()
        return codes * 2.0 ** (st["kv_scales"][blk, pos % bs, :, which].double() - 127.0)[..., None]

    if op == "gather":
        ranges = list(zip(lay["start"], lay["kv"]))
        return {n: torch.cat([cached(i, m, w, a, b) for i, (a, b) in enumerate(ranges)])
                for n, m, w in (("k", "k_pages", 0), ("v", "v_pages", 1))}
    qs, ks, vs, outs, lses, at = [], [], [], [], [], 0
    first, second = slice(0, case["rot"] // 2), slice(case["rot"] // 2, case["rot"])
    if case["interleaved"]:
        first, second = slice(0, case["rot"], 2), slice(1, case["rot"], 2)

    def rotated(x, pos):
        if not case["rot"]:
            return x.double()
        half = case["rot"] // 2
        x, w = x.double().clone(), st["cos_sin"][pos].double()
        z = torch.complex(x[..., first].contiguous(), x[..., second].contiguous())
        z = z * torch.complex(w[:, :half].contiguous(), w[:, half:].contiguous())[:, None]
        x[..., first], x[..., second] = z.real, z.imag
        return x

    for i, (n, k, seen) in enumerate(zip(lay["q"], lay["kv"], lay["visible"])):
        pos = torch.arange(k - n, k, device=dev)
        if op in ("append", "step"):
            qs.append(rotated(st["q"][at:at + n], pos))
            ks.append(_stored(rotated(st["k_new"][at:at + n], pos)))
            vs.append(_stored(st["v_new"][at:at + n].double()))
        if op != "append":
            old = k - n if op == "step" else k
            keys, vals = (cached(i, m, w, 0, old) for m, w in (("k_pages", 0), ("v_pages", 1)))
            q = st["q"][at:at + n].double()
            if op == "step":
                keys, vals = torch.cat((keys, ks[-1])), torch.cat((vals, vs[-1]))
                q = qs[-1].bfloat16().double()
            q = q.view(n, hkv, -1, d).permute(1, 2, 0, 3)
            x = q @ keys.permute(1, 2, 0)[:, None] * st["scale"]  # [hkv, heads, n, keys]
            j = torch.arange(k, device=dev)
            if case["cap"]:
                x = case["cap"] * torch.tanh(x / case["cap"])
            if case["distance"]:
                x = x + st["slopes"].double().view(hkv, -1, 1, 1) * (j - pos[:, None])
            ok = (j <= pos[:, None]) | (j < seen)
            x = torch.where(ok, x, torch.full_like(x, -math.inf))
            z = torch.logsumexp(x, -1, keepdim=True)
            o = torch.exp(x - z) @ vals.transpose(0, 1)[:, None]
            outs.append(o.permute(2, 0, 1, 3).reshape(n, hq, d))
            lses.append(z.squeeze(-1).permute(2, 0, 1).reshape(n, hq))
        at += n
    if op in ("attend", "scored"):
        return {"out": torch.cat(outs), "lse": torch.cat(lses)}
    res = {"k": torch.cat(ks), "v": torch.cat(vs)}
    if op == "step":
        res["out"] = torch.cat(outs)
    elif case["rot"]:
        res["q"] = torch.cat(qs)
    return res
