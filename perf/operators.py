"""Measured cases of the serving-step operators: the rotary KV append, attention over batches
that share prefixes, and the step that does both.

Each case runs one operator in plain torch operations (fp32, rounded once at the end), or, with
`own` set, through the package's entry points.  Batches are drawn like workloads.py draws them:
a ragged token axis, a shuffled page pool, block tables; sequences that share a prefix point at
the same physical blocks for it.
"""
from __future__ import annotations

import math
import random

import torch

own = False

_LOG2E = 1.4426950408889634


# ------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one token of one request on a toy model: the latency of a call
        dict(name="rope one token", op="rope", decodes=1, chunks=0, chunk=0, ctx=100, hq=4, hkv=2,
             d=64, bs=16, rot=64, interleaved=False, packed=False, layout=1),
        # a mixed continuous-batching step at 2048 tokens: 120 decodes and one long chunk, q/k/v
        # as views of the fused projection's output
        dict(name="rope mixed 2048", op="rope", decodes=120, chunks=1, chunk=1928, ctx=4096, hq=32,
             hkv=8, d=128, bs=32, rot=128, interleaved=False, packed=True, layout=2),
        # a prefill-heavy step, 64 query heads, half of each head rotated, neighbouring pairs
        dict(name="rope chunks 8x1024", op="rope", decodes=16, chunks=8, chunk=1024, ctx=2048, hq=64,
             hkv=8, d=128, bs=64, rot=64, interleaved=True, packed=False, layout=3),
        # odd head counts and ragged chunks: 15 query heads over 5, 32 of 64 elements rotated
        dict(name="rope odd heads", op="rope", decodes=37, chunks=5, chunk=149, ctx=777, hq=15,
             hkv=5, d=64, bs=16, rot=32, interleaved=True, packed=True, layout=4),
        # four samples of one prompt on the toy model: the smallest sharing batch
        dict(name="prefix 4 samples", op="prefix", seqs=4, members=4, groups=1, prefix=500, own=24,
             spec=1, chunk=0, hq=4, hkv=2, d=64, bs=16, layout=5),
        # long-tail decode where a quarter of the batch shares 1024 tokens
        dict(name="prefix long tail 256", op="prefix", seqs=256, members=64, groups=1, prefix=1024,
             own=2048, spec=1, chunk=0, hq=64, hkv=8, d=128, bs=64, layout=6),
        # chat serving: every request starts with the same system prompt
        dict(name="prefix system prompt", op="prefix", seqs=128, members=128, groups=1, prefix=4096,
             own=300, spec=1, chunk=0, hq=32, hkv=8, d=128, bs=32, layout=7),
        # parallel sampling: 16 prompts of different lengths, 8 samples each
        dict(name="prefix 16x8 samples", op="prefix", seqs=128, members=128, groups=16, prefix=8000,
             own=200, spec=1, chunk=0, hq=32, hkv=8, d=128, bs=32, layout=8),
        # questions about one long document
        dict(name="prefix document 64k", op="prefix", seqs=24, members=24, groups=1, prefix=65536,
             own=150, spec=1, chunk=0, hq=32, hkv=8, d=128, bs=64, layout=9),
        # speculative decoding: up to 8 tokens to verify per request under one system prompt
        dict(name="prefix verify 8", op="prefix", seqs=48, members=48, groups=1, prefix=2048,
             own=250, spec=8, chunk=0, hq=32, hkv=8, d=128, bs=16, layout=10),
        # one layer's whole step: rotate, append and attend, 64 decodes under one prompt
        dict(name="step decode 64", op="step", seqs=64, members=64, groups=1, prefix=1024, own=400,
             spec=1, chunk=0, hq=32, hkv=8, d=128, bs=32, rot=128, interleaved=False, packed=True,
             layout=11),
        # the same with a request whose prompt is still being read in (a chunk of 256)
        dict(name="step mixed", op="step", seqs=33, members=25, groups=2, prefix=2000, own=700,
             spec=1, chunk=256, hq=32, hkv=4, d=128, bs=32, rot=64, interleaved=False, packed=True,
             layout=12),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw_once(rng):
    op = rng.choice(["rope", "rope", "prefix", "prefix", "prefix", "step"])
    hkv = rng.choice([1, 2, 3, 4, 5, 8, 8, 16])
    g = rng.choice([1, 2, 3, 4, 4, 5, 7, 8, 8, 16])
    if g > 8 and hkv > 4 and hkv % 4 or hkv > 64 // g:
        hkv = 4
    c = dict(op=op, hq=hkv * g, hkv=hkv, d=rng.choice([64, 128, 128]),
             bs=rng.choice([4, 8, 16, 16, 32, 32, 64, 128]), layout=rng.randrange(1 << 30))
    if op == "rope":
        c.update(decodes=_log(rng, 1, 257) - 1, chunks=rng.choice([0, 1, 1, 2, 5, 9]),
                 chunk=_log(rng, 2, 1024), ctx=_log(rng, 1, 4096))
        if c["decodes"] + c["chunks"] == 0:
            c["decodes"] = 1
    else:
        members = _log(rng, 2, 160)
        c.update(members=members, seqs=members + rng.choice([0, 0, 1, 3, 17]),
                 groups=min(members // 2, rng.choice([1, 1, 1, 2, 3, 9])),
                 prefix=_log(rng, 64, 16384), own=_log(rng, 1, 2000),
                 spec=rng.choice([1, 1, 1, 2, 4, 8]), chunk=0)
        if rng.random() < 0.25:
            c["chunk"] = _log(rng, 9, 200)
    if op != "prefix":
        c.update(rot=16 * rng.randint(1, c["d"] // 16), interleaved=rng.random() < 0.5,
                 packed=rng.random() < 0.5)
    return c


def draw(rng):
    """A case of the same ranges that costs no more than the largest listed one, neither in its
    own work nor in the plain form's padded scores and gathered keys."""
    most = {op: [max(v) for v in zip(*(_cost(c) for c in listed() if c["op"] == op))]
            for op in ("rope", "prefix", "step")}
    while True:
        c = _draw_once(rng)
        if all(x <= m for x, m in zip(_cost(c), most[c["op"]])):
            return c


def _cost(case):
    w = work(case)
    lay = _layout(case)
    s, qm, km = len(lay["q"]), max(lay["q"]), max(lay["kv"])
    if case["op"] == "rope":
        return w["bytes"], sum(lay["kv"]) * case["hkv"] * case["d"]
    return w["bytes"], w["flops"], s * qm * km * case["hq"], s * km * case["hkv"] * case["d"]


# ---------------------------------------------------------------------------------- lengths
def _layout(case):
    """Lengths and groups of a case: q (query tokens), kv (keys after the append), group (-1:
    shares with nobody) per sequence, and each group's prefix length."""
    r = random.Random(case["layout"])
    if case["op"] == "rope":
        kinds = [1] * case["decodes"] + [0] * case["chunks"]
        q = [1 if k else max(1, case["chunk"] - r.randrange(1 + case["chunk"] // 8)) for k in kinds]
        kv = [n + r.randint(0, case["ctx"]) for n in q]
        return dict(q=q, kv=kv, group=[-1] * len(q), prefix=[])
    s, m, ng, bs = case["seqs"], case["members"], case["groups"], case["bs"]
    prefix = [case["prefix"]] if ng == 1 else [r.randint(case["prefix"] // 4, case["prefix"])
                                               for _ in range(ng)]
    group = [i % ng for i in range(m)] + [-1] * (s - m)
    r.shuffle(group)  # requests come in any order
    q = [r.randint(1, case["spec"]) for _ in range(s)]
    if case["chunk"]:
        q[r.randrange(s)] = case["chunk"]
    kv = []
    for i in range(s):
        tail = min(16384, max(0, int(case["own"] * math.exp(r.gauss(0.0, 0.8)))))
        base = -(-prefix[group[i]] // bs) * bs if group[i] >= 0 else 0
        kv.append(base + tail + q[i])
    return dict(q=q, kv=kv, group=group, prefix=prefix)


def work(case):
    lay = _layout(case)
    t, hq, hkv, d = sum(lay["q"]), case["hq"], case["hkv"], case["d"]
    row = hkv * d * 2  # bytes of one token's keys (or values)
    nbytes = flops = 0
    if case["op"] != "prefix":  # k, v read and written, the table's rows of the tokens' positions
        at = {k - n + i for n, k in zip(lay["q"], lay["kv"]) for i in range(n)}
        nbytes += 4 * t * row + len(at) * case["rot"] * 4
        flops += 3 * t * (hq + hkv) * case["rot"]
    nbytes += 2 * t * hq * d * 2  # q read; its rotation or the output written
    if case["op"] != "rope":
        # the prefix of each group once, every other key of each sequence, the tokens appended in
        # this very step not read again
        keys = sum(lay["prefix"]) + sum(k - (lay["prefix"][g] if g >= 0 else 0)
                                        for k, g in zip(lay["kv"], lay["group"]))
        keys -= t if case["op"] == "step" else 0
        nbytes += 2 * keys * row + t * hq * 4
        flops += sum(4 * d * hq * (n * (k - n) + n * (n + 1) // 2)
                     for n, k in zip(lay["q"], lay["kv"]))
    return {"bytes": nbytes, "flops": flops}


# ----------------------------------------------------------------------------------- inputs
def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    r = random.Random(seed)
    lay = _layout(case)
    hq, hkv, d, bs = case["hq"], case["hkv"], case["d"], case["bs"]
    s, t = len(lay["q"]), sum(lay["q"])
    nblk = [-(-k // bs) for k in lay["kv"]]
    shared = [-(-n // bs) for n in lay["prefix"]]  # blocks that a group's members have in common
    need = sum(shared) + sum(n - (shared[g] if g >= 0 else 0) for n, g in zip(nblk, lay["group"]))
    pages = need + max(1, need // 8)
    ids = list(range(pages))
    r.shuffle(ids)
    common = []
    for n in shared:
        common.append(ids[:n])
        ids = ids[n:]
    width = max(nblk) + 2
    rows, at = [], 0
    for n, g in zip(nblk, lay["group"]):
        head = common[g] if g >= 0 else []
        rows.append(head + ids[at:at + n - len(head)] + [-1] * (width - n))
        at += n - len(head)
    cu = [0]
    for n in lay["q"]:
        cu.append(cu[-1] + n)

    def i32(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    def rand(*shape):
        return torch.empty(shape, dtype=torch.bfloat16, device=dev).normal_(generator=gen)

    st = dict(case=case, block_size=bs, scale=d ** -0.5, q_max=max(lay["q"]), blocks=max(nblk),
              block_table=i32(rows), cu_seqlens_q=i32(cu), kv_lens=i32(lay["kv"]),
              k_pages=rand(pages, bs, hkv, d), v_pages=rand(pages, bs, hkv, d))
    if case["op"] == "prefix":
        st["q"] = rand(t, hq, d)
    elif case["packed"]:  # views of the projection's output, token rows (hq + 2 hkv) d apart
        qkv = rand(t, hq + 2 * hkv, d)
        st["q"], st["k_new"], st["v_new"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    else:
        st["q"], st["k_new"], st["v_new"] = rand(t, hq, d), rand(t, hkv, d), rand(t, hkv, d)
    if case["op"] != "rope":
        st["prefix_group"], st["prefix_lens"] = i32(lay["group"]), i32(lay["prefix"])
    if case["op"] != "prefix":
        half = case["rot"] // 2
        pos = torch.arange(max(lay["kv"]) + 1, device=dev, dtype=torch.float64)
        freq = 10000.0 ** (-torch.arange(half, device=dev, dtype=torch.float64) / half)
        ang = pos[:, None] * freq
        st["cos_sin"] = torch.cat((ang.cos(), ang.sin()), 1).float().contiguous()
        st["interleaved"] = case["interleaved"]
    return st


# --------------------------------------------------------------------------- the plain forms
def _places(st):
    """Per packed token: its sequence, its index among the sequence's tokens, its position."""
    cu = st["cu_seqlens_q"].long()
    t = torch.arange(st["q"].shape[0], device=cu.device)
    seq = torch.searchsorted(cu, t, right=True) - 1
    i = t - cu[seq]
    n = cu[1:] - cu[:-1]
    return seq, i, (st["kv_lens"].long() - n)[seq] + i


def _rotate(x, cos, sin, interleaved):
    """x [T, H, D] rounded to bf16 with its first 2 * cos.shape[1] elements rotated."""
    half = cos.shape[1]
    y = x.float()
    c, s = cos[:, None], sin[:, None]
    if interleaved:
        a, b = y[..., 0:2 * half:2], y[..., 1:2 * half:2]
        turned = torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    else:
        a, b = y[..., :half], y[..., half:2 * half]
        turned = torch.cat((a * c - b * s, b * c + a * s), -1)
    return torch.cat((turned, y[..., 2 * half:]), -1).to(x.dtype)


def _rope_plain(st):
    seq, _, pos = _places(st)
    rows = st["cos_sin"][pos]
    half = rows.shape[1] // 2
    cos, sin = rows[:, :half], rows[:, half:]
    bs = st["block_size"]
    block = st["block_table"].long()[seq, torch.div(pos, bs, rounding_mode="floor")]
    slot = block * bs + pos % bs
    hkv, d = st["k_pages"].shape[2:]
    st["k_pages"].view(-1, hkv, d)[slot] = _rotate(st["k_new"], cos, sin, st["interleaved"])
    st["v_pages"].view(-1, hkv, d)[slot] = st["v_new"]
    return _rotate(st["q"], cos, sin, st["interleaved"])


def _attend_plain(st, q):
    """Every sequence's keys gathered whole, a mask, softmax, a sum: out bf16 and lse fp32."""
    hq, d = q.shape[1:]
    hkv = st["k_pages"].shape[2]
    cu, kv = st["cu_seqlens_q"].long(), st["kv_lens"].long()
    n = cu[1:] - cu[:-1]
    s = kv.shape[0]
    col = torch.arange(st["q_max"], device=q.device)
    rows = (cu[:-1, None] + col).clamp(max=q.shape[0] - 1)
    qs = q[rows].float().view(s, st["q_max"], hkv, hq // hkv, d).permute(0, 2, 3, 1, 4)
    qs = qs.reshape(s, hkv, -1, d)
    table = st["block_table"][:, :st["blocks"]].long().clamp(min=0)
    k = st["k_pages"][table].view(s, -1, hkv, d).float().permute(0, 2, 3, 1)
    x = torch.matmul(qs, k).mul_(st["scale"])  # [s, hkv, heads * q_max, keys]
    del k
    x = x.view(s, hkv, hq // hkv, st["q_max"], -1)
    last = (kv - n)[:, None] + col  # the last key that each query sees
    dead = torch.arange(x.shape[-1], device=q.device) > last[..., None]
    x = x.masked_fill_(dead[:, None, None], float("-inf"))
    m = x.amax(-1, keepdim=True)
    p = x.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    v = st["v_pages"][table].view(s, -1, hkv, d).float().permute(0, 2, 1, 3)
    o = torch.matmul(p.view(s, hkv, -1, p.shape[-1]), v).view(s, hkv, hq // hkv, -1, d) / total
    lse = (m + total.log()).squeeze(-1)
    seq, i, _ = _places(st)
    out = o.permute(0, 3, 1, 2, 4)[seq, i].reshape(-1, hq, d)
    return out.to(q.dtype), lse.permute(0, 3, 1, 2)[seq, i].reshape(-1, hq)


def run(state):
    st, op = state, state["case"]["op"]
    if own:
        import continuous_batching_paged_gb300 as cb
        where = (st["k_pages"], st["v_pages"], st["block_table"], st["cu_seqlens_q"],
                 st["kv_lens"], st["block_size"])
        if op == "rope":
            q = cb.rope_append(st["q"], st["k_new"], st["v_new"], *where, st["cos_sin"],
                               interleaved=st["interleaved"])
            return {"q": q, "k_pages": st["k_pages"], "v_pages": st["v_pages"]}
        if op == "prefix":
            out, lse = cb.shared_prefix_attention(st["q"], *where, st["scale"],
                                                  st["prefix_group"], st["prefix_lens"], lse=True)
            return {"out": out, "lse": lse}
        out, lse = cb.rope_append_attention(st["q"], st["k_new"], st["v_new"], *where,
                                            st["scale"], st["cos_sin"],
                                            interleaved=st["interleaved"],
                                            prefix_group=st["prefix_group"],
                                            prefix_lens=st["prefix_lens"], lse=True)
        return {"out": out, "lse": lse, "k_pages": st["k_pages"], "v_pages": st["v_pages"]}
    if op == "prefix":
        out, lse = _attend_plain(st, st["q"])
        return {"out": out, "lse": lse}
    q = _rope_plain(st)
    if op == "rope":
        return {"q": q, "k_pages": st["k_pages"], "v_pages": st["v_pages"]}
    out, lse = _attend_plain(st, q)
    return {"out": out, "lse": lse, "k_pages": st["k_pages"], "v_pages": st["v_pages"]}


# ------------------------------------------------------------------------ the values in 64 bits
def exact(case, seed):
    """The operators' definitions, sequence by sequence in 64 bits.  A step's attention reads
    what the step stores: the rotated queries and keys rounded to bf16."""
    st = prepare(case, seed)
    lay = _layout(case)
    bs, hq, hkv, d = case["bs"], case["hq"], case["hkv"], case["d"]
    if case["op"] != "rope" and sum(n * k for n, k in zip(lay["q"], lay["kv"])) * hq * d > 4e10:
        return None
    table = st["block_table"].tolist()
    res, q_all, kp, vp = {}, st["q"], st["k_pages"], st["v_pages"]
    if case["op"] != "prefix":
        half = case["rot"] // 2
        turn = torch.complex(st["cos_sin"][:, :half].double(), st["cos_sin"][:, half:].double())
        first, second = ((slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if case["interleaved"]
                         else (slice(0, half), slice(half, 2 * half)))

        def rotated(x, pos):
            x = x.double().clone()
            w = torch.complex(x[..., first].contiguous(), x[..., second].contiguous())
            w = w * turn[pos][:, None]
            x[..., first], x[..., second] = w.real, w.imag
            return x

        kp, vp = kp.double(), vp.double()
        q_all = torch.empty(st["q"].shape, dtype=torch.float64, device=kp.device)
        at = 0
        for i, (n, k) in enumerate(zip(lay["q"], lay["kv"])):
            pos = torch.arange(k - n, k, device=kp.device)
            blk = torch.tensor([table[i][p // bs] for p in range(k - n, k)], device=kp.device)
            kp[blk, pos % bs] = rotated(st["k_new"][at:at + n], pos)
            vp[blk, pos % bs] = st["v_new"][at:at + n].double()
            q_all[at:at + n] = rotated(st["q"][at:at + n], pos)
            at += n
        res = {"k_pages": kp, "v_pages": vp}
        if case["op"] == "rope":
            return {"q": q_all, **res}
        q_all, kp = q_all.to(torch.bfloat16), kp.to(torch.bfloat16)
    outs, lses, at = [], [], 0
    for i, (n, k) in enumerate(zip(lay["q"], lay["kv"])):
        blocks = torch.tensor(table[i][:-(-k // bs)], device=q_all.device)
        keys = kp[blocks].reshape(-1, hkv, d)[:k].double().transpose(0, 1)
        vals = vp[blocks].reshape(-1, hkv, d)[:k].double().transpose(0, 1)
        q = q_all[at:at + n].double().view(n, hkv, -1, d).permute(1, 2, 0, 3)
        x = q @ keys[:, None].transpose(-1, -2) * _LOG2E * st["scale"]
        ok = torch.ones(n, k, dtype=torch.bool, device=x.device).tril(k - n)
        x = torch.where(ok, x, torch.full_like(x, -math.inf))
        top = x.max(-1, keepdim=True).values
        p = torch.exp2(x - top)
        norm = p.sum(-1, keepdim=True)
        outs.append((p / norm @ vals[:, None]).permute(2, 0, 1, 3).reshape(n, hq, d))
        lses.append(((top + norm.log2()) / _LOG2E).squeeze(-1).permute(2, 0, 1).reshape(n, hq))
        at += n
    return {"out": torch.cat(outs), "lse": torch.cat(lses), **res}
