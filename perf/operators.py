"""Rotation and key/value cache operators: what is measured, and their plain forms.

A pack's queries and keys are rotated by their positions (``rope``), prompts and
single tokens are appended to a paged cache of bf16 or 4-bit rows (``append``),
cached rows are read back as a contiguous pack (``read``), and a few new tokens
of each sequence attend to everything that it has cached (``attn``); ``step`` is
one decoding step, an append and the attention that reads it.

With ``own`` false ``run`` computes them with elementary torch operations in
32 bits; with ``own`` true it calls the package.
"""
import math
import random

import torch

own = False

# (query heads, kv heads, head_dim) of the package's own workloads, and one
# without shared heads
HEADS = [(32, 8, 128), (14, 2, 64), (16, 4, 128), (4, 4, 64), (8, 8, 128)]


def listed():
    return [
        # rotation of the queries and keys of one 131072-token pack of documents before its attention
        dict(name="rope_pack_128k", op="rope", tokens=131072, longest=65536, hq=32, hkv=8, d=128,
             rot=128, inter=False, inverse=False, fp32=False, mix=11),
        # gradients of a long-tail pack taken back through the rotation, in fp32 as the backward pass gives them
        dict(name="rope_grad_longtail", op="rope", tokens=32768, longest=16384, hq=14, hkv=2, d=64,
             rot=64, inter=True, inverse=True, fp32=True, mix=12),
        # one user's next token goes into the cache: pure latency
        dict(name="append_one", op="append", cache="bf16", batch=1, least=700, ctx=700, new=1,
             hq=32, hkv=8, d=128, rot=128, inter=False, page=16, mix=21),
        # prompts of one prefill batch go into the cache, rotated on the way
        dict(name="append_prompts", op="append", cache="bf16", batch=9, least=131, ctx=8192, new=8192,
             hq=32, hkv=8, d=128, rot=128, inter=False, page=64, mix=22),
        # the next chunk of several prompts goes into a 4-bit cache, and the whole contexts come back for the attention over the pack
        dict(name="append_read_int4", op="read", cache="int4", batch=6, least=600, ctx=12000, new=2048,
             hq=16, hkv=4, d=128, rot=64, inter=False, page=32, mix=23),
        # the same for a bf16 cache, long contexts with short chunks
        dict(name="append_read_bf16", op="read", cache="bf16", batch=4, least=9000, ctx=40000, new=300,
             hq=14, hkv=2, d=64, rot=64, inter=True, page=128, mix=24),
        # one user's next token against a short context: latency
        dict(name="attn_one", op="attn", cache="bf16", batch=1, least=4000, ctx=4000, new=1,
             hq=32, hkv=8, d=128, window=0, page=16, mix=31),
        # a full batch of decoding users with contexts of all lengths
        dict(name="attn_batch", op="attn", cache="bf16", batch=64, least=1024, ctx=16384, new=1,
             hq=32, hkv=8, d=128, window=0, page=64, mix=32),
        # drafts of up to 4 tokens a user are checked under a sliding window
        dict(name="attn_drafts_window", op="attn", cache="bf16", batch=48, least=1, ctx=9001, new=4,
             hq=14, hkv=2, d=64, window=4096, page=32, mix=33),
        # few users with very long contexts over a 4-bit cache
        dict(name="attn_int4_long", op="attn", cache="int4", batch=3, least=100000, ctx=131072, new=1,
             hq=32, hkv=8, d=128, window=0, page=64, mix=34),
        # a batch of decoding users over a 4-bit cache: append the token, then attend
        dict(name="step_int4", op="step", cache="int4", batch=96, least=200, ctx=16000, new=1,
             hq=16, hkv=4, d=128, window=0, rot=128, inter=False, page=16, mix=35),
        # short drafts of a small model over a 4-bit cache, each key head read by its own query head
        dict(name="step_int4_drafts", op="step", cache="int4", batch=7, least=33, ctx=2500, new=6,
             hq=4, hkv=4, d=64, window=0, rot=32, inter=True, page=16, mix=36),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    hq, hkv, d = rng.choice(HEADS)
    op = rng.choice(["rope", "append", "read", "attn", "attn", "step"])
    mix = rng.randrange(1 << 30)
    rot = rng.choice([d, d // 2])
    inter = rng.random() < 0.5
    if op == "rope":
        tokens = _log(rng, 1, min(131072, (131072 * 40 * 128) // ((hq + hkv) * d * 2)))
        return dict(op=op, tokens=tokens, longest=_log(rng, 1, tokens), hq=hq, hkv=hkv, d=d, rot=rot,
                    inter=inter, inverse=rng.random() < 0.5, fp32=rng.random() < 0.4, mix=mix)
    cache = rng.choice(["bf16", "int4"])
    page = rng.choice([16, 32, 64, 128, 256])
    c = dict(op=op, cache=cache, hq=hq, hkv=hkv, d=d, page=page, mix=mix)
    if op in ("append", "read"):
        batch = _log(rng, 1, 64)
        ctx = _log(rng, 1, max(2, min(65536, 160000 // batch)))
        new = min(ctx, _log(rng, 1, 8192))
        # a 4-bit cache is always read back: what it holds is seen through its values
        return dict(c, op="read" if cache == "int4" else op, batch=batch, least=_log(rng, 1, ctx), ctx=ctx, new=new,
                    rot=rot, inter=inter)
    batch = _log(rng, 1, 256)
    ctx = _log(rng, 1, max(2, min(131072, (64 * 16384 * 8 * 128) // (batch * hkv * d))))
    new = min(ctx, rng.choice([1, 1, 1, 2, 3, 5, 8, 16]))
    c = dict(c, batch=batch, least=_log(rng, 1, ctx), ctx=ctx, new=new,
             window=rng.choice([0, 0, _log(rng, 1, 2 * ctx)]))
    return dict(c, rot=rot, inter=inter) if op == "step" else c


def _shape(case):
    """Lengths that the case stands for: cached tokens of each sequence (the new ones among them), and new tokens."""
    rng = random.Random(case["mix"])
    if case["op"] == "rope":
        docs, left = [], case["tokens"]
        while left:
            docs.append(min(left, _log(rng, 1, case["longest"])))
            left -= docs[-1]
        return docs, docs
    lens = [_log(rng, case["least"], case["ctx"]) for _ in range(case["batch"])]
    lens[0] = case["ctx"]
    return lens, [min(n, _log(rng, 1, case["new"])) for n in lens]


def _ends(counts, device):
    return torch.tensor([0] + counts, dtype=torch.int32).cumsum(0).to(torch.int32).to(device)


def _angles(rows, rot, device):
    """(cos, sin) of every position and pair, from 64 bits: [rows, rot / 2, 2]."""
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=device) / rot)
    a = torch.arange(rows, dtype=torch.float64, device=device)[:, None] * inv
    return torch.stack((a.cos(), a.sin()), -1).float()


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    lens, news = _shape(case)
    hq, hkv, d, t = case["hq"], case["hkv"], case["d"], sum(news)
    s = dict(case=case, cu=_ends(news, dev))

    def randn(*shape):
        return torch.randn(shape, generator=g, device=dev)

    if case["op"] == "rope":
        kind = torch.float32 if case["fp32"] else torch.bfloat16
        s["table"] = _angles(max(lens), case["rot"], dev)
        s["q"], s["k"] = randn(t, hq, d).to(kind), randn(t, hkv, d).to(kind)
        s["q_out"], s["k_out"] = torch.empty_like(s["q"]), torch.empty_like(s["k"])
        return s
    page, batch = case["page"], case["batch"]
    used = [-(-n // page) for n in lens]
    width, count = max(used), sum(used) + 3
    # sequences own pages in no order; unused entries of the table name no page
    order = torch.randperm(count, generator=g, device=dev).to(torch.int32)
    s["pages"] = torch.full((batch, width), -1, dtype=torch.int32, device=dev)
    own_page = torch.arange(width, device=dev) < torch.tensor(used, device=dev)[:, None]
    s["pages"][own_page] = order[:sum(used)]
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    s["longest"] = max(lens)
    # what the projection of a layer gives: queries, keys and values of a token side by side
    qkv = randn(t, hq + 2 * hkv, d).to(torch.bfloat16)
    s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    shape = (count, hkv, page)
    if case["cache"] == "bf16":
        s["k_pages"], s["v_pages"] = (torch.empty(shape + (d,), dtype=torch.bfloat16, device=dev).normal_(generator=g) for _ in "kv")
    else:
        for x in "kv":
            rows = torch.empty(shape + (d,), dtype=torch.bfloat16, device=dev).normal_(generator=g)
            s[x + "_pages"], s[x + "_scales"] = _quantise(rows)
            del rows
    if "rot" in case:
        s["table"] = _angles(s["longest"], case["rot"], dev)
        s["q_rot"] = torch.empty((t, hq, d), dtype=torch.bfloat16, device=dev)
    if case["op"] == "read":
        s["cu_all"] = _ends(lens, dev)
        s["k_all"], s["v_all"] = (torch.empty((sum(lens), hkv, d), dtype=torch.bfloat16, device=dev) for _ in "kv")
    if case["op"] in ("attn", "step"):
        s["out"] = torch.empty((t, hq, d), dtype=torch.bfloat16, device=dev)
        s["lse"] = torch.empty((hq, t), dtype=torch.float32, device=dev)
    if own:  # the handle of the cache and the workspace that a serving program keeps
        from packed_varlen_attention_cu_gb300 import api
        s["cache"] = api.KVCache(s["k_pages"], s["v_pages"], s.get("k_scales"), s.get("v_scales"))
        if case["op"] in ("attn", "step"):
            s["work"] = api.alloc_cache_workspace(batch, hq, hkv, d, max_new=case["new"], device=dev)
    return s


# ------------------------------------------------------------ plain forms

def _rotate(x, turn, inter):
    """x [tokens, heads, d] fp32 turned by (cos, sin) [tokens, pairs, 2]; dims past the pairs stay."""
    r = 2 * turn.shape[1]
    c, s = turn[:, None, :, 0], turn[:, None, :, 1]
    if inter:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y = torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        y = torch.cat((a * c - b * s, b * c + a * s), -1)
    return torch.cat((y, x[..., r:]), -1)


def _quantise(rows):
    """bf16 rows [..., d] as (bytes [..., d / 2], (scale, lowest) [..., d / 64, 2] bf16): 64 values share a scale,
    value = lowest + code * scale.  Eight dims share a 32-bit word: dim i of the eight at bit 4 * (i / 2) + 16 * (i % 2);
    word w of a row holds eight dims of group w % groups."""
    d = rows.shape[-1]
    x = rows.float().unflatten(-1, (d // 64, 64))
    low, high = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    scale = ((high - low) * (1.0 / 15.0)).to(torch.bfloat16).float()
    inv = torch.where(scale == 0, torch.zeros_like(scale), 1.0 / scale)
    code = ((x - low) * inv).round().clamp(0, 15).to(torch.int32)
    shift = torch.tensor([0, 16, 4, 20, 8, 24, 12, 28], dtype=torch.int32, device=rows.device)
    word = (code.unflatten(-1, (8, 8)) << shift).sum(-1, dtype=torch.int32)  # [..., groups, 8]
    packed = word.transpose(-1, -2).flatten(-2).contiguous().view(torch.uint8)
    return packed, torch.cat((scale, low), -1).to(torch.bfloat16).contiguous()


def _values(packed, scales):
    """The values in fp32 that 4-bit rows stand for."""
    groups = scales.shape[-2]
    word = packed.contiguous().view(torch.int32).unflatten(-1, (8, groups)).transpose(-1, -2)
    shift = torch.tensor([0, 16, 4, 20, 8, 24, 12, 28], dtype=torch.int32, device=packed.device)
    code = ((word[..., None] >> shift) & 15).flatten(-2).float()  # [..., groups, 64]
    sc = scales.float()
    return (sc[..., 1:] + code * sc[..., :1]).flatten(-2)


def _owner(cu, rows):
    at = torch.arange(rows, device=cu.device, dtype=torch.int32)
    seq = torch.bucketize(at, cu[1:], right=True, out_int32=True)
    return seq, at - cu[seq]


def _append(s):
    case = s["case"]
    seq, i = _owner(s["cu"], s["q"].shape[0])
    pos = s["lens"][seq] - (s["cu"][seq + 1] - s["cu"][seq]) + i
    turn = s["table"][pos]
    q = _rotate(s["q"].float(), turn, case["inter"]).to(torch.bfloat16)
    k = _rotate(s["k"].float(), turn, case["inter"]).to(torch.bfloat16)
    page, slot = s["pages"][seq, pos // case["page"]], pos % case["page"]
    if case["cache"] == "bf16":
        s["k_pages"][page, :, slot], s["v_pages"][page, :, slot] = k, s["v"]
    else:
        s["k_pages"][page, :, slot], s["k_scales"][page, :, slot] = _quantise(k)
        s["v_pages"][page, :, slot], s["v_scales"][page, :, slot] = _quantise(s["v"])
    return q


def _rows(s, x, page, slot):
    """Cached rows in fp32 at page and slot."""
    if s["case"]["cache"] == "bf16":
        return s[x + "_pages"][page, :, slot].float()
    return _values(s[x + "_pages"][page, :, slot], s[x + "_scales"][page, :, slot])


def _attend(s, q):
    case = s["case"]
    batch, hkv, new, d = case["batch"], case["hkv"], case["new"], case["d"]
    group = case["hq"] // hkv
    cu, dev = s["cu"], q.device
    seq, i = _owner(cu, q.shape[0])
    count = cu[1:] - cu[:-1]
    padded = torch.zeros((batch, new, hkv, group, d), device=dev)
    padded[seq, i] = q.float().unflatten(1, (hkv, group))
    j = torch.arange(s["longest"], device=dev)
    page = s["pages"][:, j // case["page"]].clamp(min=0)
    slot = (j % case["page"]).expand_as(page)
    k, v = (_rows(s, x, page, slot) for x in "kv")
    pos = (s["lens"] - count)[:, None] + torch.arange(new, device=dev)
    seen = j <= pos[..., None]
    if case["window"]:
        seen &= j > pos[..., None] - case["window"]
    # rows past a sequence's last new token see its first key: their results are not taken
    seen[..., 0] |= torch.arange(new, device=dev) >= count[:, None]
    score = padded.permute(0, 2, 1, 3, 4).flatten(2, 3) @ k.permute(0, 2, 3, 1)
    score = (score * d ** -0.5).unflatten(2, (new, group)).masked_fill(~seen[:, None, :, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = (score - top).exp()
    total = p.sum(-1, keepdim=True)
    o = (p.flatten(2, 3) @ v.permute(0, 2, 1, 3)).unflatten(2, (new, group)) / total
    lse = (top + total.log())[..., 0]
    o, lse = o.permute(0, 2, 1, 3, 4)[seq, i], lse.permute(0, 2, 1, 3)[seq, i]
    return {"out": o.flatten(1, 2).to(torch.bfloat16), "lse": lse.flatten(1, 2).t().contiguous()}


def _run_plain(s):
    case = s["case"]
    if case["op"] == "rope":
        _, pos = _owner(s["cu"], s["q"].shape[0])
        turn = s["table"][pos]
        if case["inverse"]:
            turn = torch.stack((turn[..., 0], -turn[..., 1]), -1)
        return {"q": _rotate(s["q"].float(), turn, case["inter"]).to(s["q"].dtype),
                "k": _rotate(s["k"].float(), turn, case["inter"]).to(s["k"].dtype)}
    if case["op"] == "attn":
        return _attend(s, s["q"])
    q = _append(s)
    if case["op"] == "append":
        return {"q": q, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    if case["op"] == "step":
        return _attend(s, q)
    seq, j = _owner(s["cu_all"], s["k_all"].shape[0])
    page, slot = s["pages"][seq, j // case["page"]], j % case["page"]
    return {"q": q, "k": _rows(s, "k", page, slot).to(torch.bfloat16), "v": _rows(s, "v", page, slot).to(torch.bfloat16)}


# ------------------------------------------------------------ the package

def _run_own(s):
    from packed_varlen_attention_cu_gb300 import api
    case = s["case"]
    if case["op"] == "rope":
        api.rope(s["q"], s["k"], s["table"], s["q_out"], s["k_out"], cu_seqlens=s["cu"],
                 interleaved=case["inter"], inverse=case["inverse"])
        return {"q": s["q_out"], "k": s["k_out"]}
    q = s["q"]
    # one token for every sequence needs no table of offsets
    cu = None if case["new"] == 1 else s["cu"]
    if case["op"] != "attn":
        api.cache_append(s["cache"], s["k"], s["v"], s["pages"], s["lens"], cu_new=cu, table=s["table"],
                         q=q, q_out=s["q_rot"], interleaved=case["inter"])
        q = s["q_rot"]
    if case["op"] == "append":
        return {"q": q, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    if case["op"] == "read":
        api.cache_read(s["cache"], s["pages"], s["cu_all"], s["k_all"], s["v_all"])
        return {"q": q, "k": s["k_all"], "v": s["v_all"]}
    api.cache_attn(s["cache"], q, s["pages"], s["lens"], s["out"], s["lse"], s["work"], cu_new=cu,
                   max_new=case["new"], window=case["window"])
    return {"out": s["out"], "lse": s["lse"]}


def run(state):
    return _run_own(state) if own else _run_plain(state)


def work(case):
    lens, news = _shape(case)
    hq, hkv, d, t = case["hq"], case["hkv"], case["d"], sum(news)
    if case["op"] == "rope":
        size = 4 if case["fp32"] else 2
        table = max(lens) * case["rot"] * 4
        return {"bytes": 2 * t * (hq + hkv) * d * size + table, "flops": 3 * t * (hq + hkv) * case["rot"]}
    row = 2 * d if case["cache"] == "bf16" else d // 2 + d // 16  # a cached row of one head: its values or codes and scales
    done = {"bytes": 0, "flops": 0}
    if case["op"] != "attn":
        done["bytes"] += t * ((2 * hq + 2 * hkv) * d * 2 + 2 * hkv * row)
        done["flops"] += 3 * t * (hq + hkv) * case["rot"]
    if case["op"] == "read":
        done["bytes"] += sum(lens) * 2 * hkv * (row + 2 * d)
        done["flops"] += 0 if case["cache"] == "bf16" else sum(lens) * 4 * hkv * d
    if case["op"] in ("attn", "step"):
        w = case["window"]
        keys = sum(min(n, w + m - 1) if w else n for n, m in zip(lens, news))
        pairs = sum((min(n - m + i + 1, w) if w else n - m + i + 1) for n, m in zip(lens, news) for i in range(m))
        done["bytes"] += keys * 2 * hkv * row + t * hq * (4 * d + 4)
        done["flops"] += 4 * pairs * hq * d
    return done


# ------------------------------------------------------------ 64 bits

def exact(case, seed):
    """The operators by their definitions, sequence by sequence, in 64 bits."""
    s = prepare(case, seed)
    lens, news = _shape(case)
    hkv, d = case["hkv"], case["d"]
    half = case.get("rot", 0) // 2
    sign = -1.0 if case.get("inverse") else 1.0

    def turned(x, at):
        """Complex rotation of pair p of the tokens at positions `at` by the table's angle."""
        x = x.double()
        z = torch.view_as_complex(s["table"][at].double().contiguous())[:, None]
        z = torch.complex(z.real, sign * z.imag)
        left, right = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if case["inter"] else (slice(0, half), slice(half, 2 * half))
        w = torch.complex(x[..., left].contiguous(), x[..., right].contiguous()) * z
        y = x.clone()
        y[..., left], y[..., right] = w.real, w.imag
        return y

    if case["op"] == "rope":
        at = torch.tensor([t for n in news for t in range(n)], device=s["q"].device)
        return {"q": turned(s["q"], at), "k": turned(s["k"], at)}

    def rounded4(x):
        """The nearest of the 16 values that its group of 64 allows, for every value."""
        out = torch.empty_like(x)
        for a in range(0, d, 64):
            part = x[..., a:a + 64]
            low, high = part.min(-1, keepdim=True).values, part.max(-1, keepdim=True).values
            step = ((high - low) / 15).to(torch.float32).to(torch.bfloat16).double()
            n = torch.where(step > 0, torch.round((part - low) / torch.where(step > 0, step, torch.ones_like(step))), torch.zeros_like(part))
            out[..., a:a + 64] = low + n.clamp(0, 15) * step
        return out

    def cached(x, b):
        """All cached rows of sequence b: [len, heads, d]."""
        table = s["pages"][b, :-(-lens[b] // case["page"])].long()
        rows = s[x + "_pages"][table].transpose(1, 2).flatten(0, 1)[:lens[b]]
        if case["cache"] == "bf16":
            return rows.double()
        sc = s[x + "_scales"][table].transpose(1, 2).flatten(0, 1)[:lens[b]].double()
        out = torch.empty(rows.shape[:-1] + (d,), dtype=torch.float64, device=rows.device)
        groups = d // 64
        for i in range(d):
            # dim i: which byte and which half of it
            word, bit = (i % 64) // 8 * groups + i // 64, 4 * (i % 8 // 2) + 16 * (i % 2)
            byte = rows[..., 4 * word + bit // 8].long()
            code = (byte >> 4) if bit % 8 else (byte & 15)
            out[..., i] = sc[..., i // 64, 1] + code * sc[..., i // 64, 0]
        return out

    q_new, outs, lses, ks, vs, a = [], [], [], [], [], 0
    for b, (n, m) in enumerate(zip(lens, news)):
        q = s["q"][a:a + m].double()
        k, v = cached("k", b), cached("v", b)
        if case["op"] != "attn":
            at = torch.arange(n - m, n, device=k.device)
            q, kn, vn = turned(s["q"][a:a + m], at), turned(s["k"][a:a + m], at), s["v"][a:a + m].double()
            if case["op"] != "append":  # what is read again was rounded to what the cache holds
                kn = kn.to(torch.float32).to(torch.bfloat16).double()
                if case["cache"] == "int4":
                    kn, vn = rounded4(kn), rounded4(vn)
            k[n - m:], v[n - m:] = kn, vn
            q_new.append(q)
        a += m
        if case["op"] in ("read", "append"):
            ks.append(k)
            vs.append(v)
            continue
        if case["op"] == "step":
            q = q.to(torch.float32).to(torch.bfloat16).double()
        at = torch.arange(n - m, n, device=q.device)[:, None]
        j = torch.arange(n, device=q.device)[None]
        ok = (j <= at) & ((j > at - case["window"]) if case["window"] else (j >= 0))
        sc = torch.einsum("mhgd,lhd->hgml", q.unflatten(1, (hkv, -1)), k) / math.sqrt(d)
        sc = sc.masked_fill(~ok, -math.inf)
        lse = torch.logsumexp(sc, -1)
        outs.append(torch.einsum("hgml,lhd->mhgd", (sc - lse[..., None]).exp(), v).flatten(1, 2))
        lses.append(lse.flatten(0, 1))
    if outs:
        return {"out": torch.cat(outs), "lse": torch.cat(lses, -1)}
    if case["op"] == "read":
        return {"q": torch.cat(q_new), "k": torch.cat(ks), "v": torch.cat(vs)}
    kp, vp = s["k_pages"].double(), s["v_pages"].double()
    for b, (n, m) in enumerate(zip(lens, news)):
        for pages, rows in ((kp, ks[b]), (vp, vs[b])):
            at = torch.arange(n - m, n, device=rows.device)
            pages[s["pages"][b, at // case["page"]].long(), :, at % case["page"]] = rows[n - m:]
    return {"q": torch.cat(q_new), "k_pages": kp, "v_pages": vp}
