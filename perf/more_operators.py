"""Operators of models that answer about a source: what is measured, and their plain forms.

Packs of targets attend to packs of sources (``fwd``, and ``train`` with the
gradients), beams attend to a source's cached keys and values (``attend``), the
best continuations of every group of beams are chosen from their logits
(``select``), and caches and states follow the chosen parents (``reorder``);
``step`` is one decoding step of all of them: selection, reordering, the append
of the new token, and its attention to its own past and to the source.

With ``own`` false ``run`` computes them with elementary torch operations in
32 bits (64 where candidates are ranked); with ``own`` true it calls the package.
"""
import math
import random

import torch

own = False

# (query heads, kv heads, head_dim) of the package's own workloads, and two
# without shared heads
HEADS = [(32, 8, 128), (14, 2, 64), (16, 4, 128), (4, 4, 64), (8, 8, 128)]


def listed():
    return [
        # many short pairs (sentences and their sources) in one training pack
        dict(name="train_short_pairs", op="train", docs=512, q_least=4, q_most=90, k_least=5, k_most=120,
             hq=16, hkv=4, d=128, mix=11),
        # a training pack of longer answers to long sources
        dict(name="train_long", op="train", docs=12, q_least=256, q_most=2048, k_least=512, k_most=4096,
             hq=32, hkv=8, d=128, mix=12),
        # one forced prefix against one source of a few windows of sound: latency
        dict(name="fwd_one", op="fwd", docs=1, q_least=77, q_most=77, k_least=1500, k_most=1500,
             hq=8, hkv=8, d=128, mix=13),
        # one user's beams look at their source: latency
        dict(name="attend_one", op="attend", cache="bf16", batch=1, beams=5, least=1500, ctx=1500,
             hq=8, hkv=8, d=128, page=64, mix=21),
        # a full batch of users with sources of all lengths
        dict(name="attend_batch", op="attend", cache="bf16", batch=64, beams=4, least=500, ctx=8192,
             hq=32, hkv=8, d=128, page=64, mix=22),
        # many beams over long sources kept in 4 bits
        dict(name="attend_int4", op="attend", cache="int4", batch=24, beams=8, least=2000, ctx=30000,
             hq=16, hkv=4, d=128, page=32, mix=23),
        # one user's beams: latency
        dict(name="select_one", op="select", kind="bf16", groups=1, beams=4, vocab=32000, k=8, pad=0, done=False, mix=31),
        # a full batch of users over a large vocabulary of odd size
        dict(name="select_batch", op="select", kind="bf16", groups=64, beams=8, vocab=131071, k=16, pad=1, done=False, mix=32),
        # fp32 logits, some beams are finished, and lengths weigh the scores
        dict(name="select_fp32", op="select", kind="fp32", groups=24, beams=5, vocab=50021, k=5, pad=0, done=True, mix=33),
        # one user's beams change places in a few layers: latency
        dict(name="reorder_one", op="reorder", layers=6, groups=1, beams=4, least=700, ctx=700, gen=60, hist=256, state=1024,
             hkv=8, d=128, page=16, mix=41),
        # a full batch of users and layers, with a recurrent state for every beam
        dict(name="reorder_batch", op="reorder", layers=12, groups=32, beams=5, least=64, ctx=900, gen=120, hist=512, state=16384,
             hkv=4, d=128, page=64, mix=42),
        # one decoding step of one layer, caches in 4 bits
        dict(name="step_int4", op="step", kind="bf16", cache="int4", groups=16, beams=4, vocab=65537, k=4, pad=0, layers=1,
             least=200, ctx=2000, gen=150, hq=16, hkv=4, d=128, page=32, src_least=300, src=6000, mix=51),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    hq, hkv, d = rng.choice(HEADS)
    op = rng.choice(["train", "train", "fwd", "attend", "attend", "select", "select", "reorder", "step"])
    c = dict(op=op, mix=rng.randrange(1 << 30))
    if op in ("train", "fwd"):
        q, k = _log(rng, 1, 4096), _log(rng, 1, 8192)
        most = 12 * 2048 * 4096 * 32 * 128 // (q * k * hq * d)
        return dict(c, docs=_log(rng, 1, max(2, min(1000, most, 65536 // q, 65536 // k))), q_least=_log(rng, 1, q), q_most=q,
                    k_least=_log(rng, 1, k), k_most=k, hq=hq, hkv=hkv, d=d)
    cache = rng.choice(["bf16", "int4"])
    page = rng.choice([16, 32, 64, 128, 256])
    if op == "attend":
        batch, beams = _log(rng, 1, 128), rng.choice([1, 2, 3, 4, 5, 8, 12])
        ctx = _log(rng, 1, max(2, min(65536, (64 * 8192 * 8 * 128) // (batch * hkv * d))))
        return dict(c, cache=cache, batch=batch, beams=beams, least=_log(rng, 1, ctx), ctx=ctx, hq=hq, hkv=hkv, d=d, page=page)
    beams = rng.choice([1, 2, 3, 4, 5, 8, 16])
    groups, ctx, src = _log(rng, 1, 64), _log(rng, 1, 3000), _log(rng, 1, 8192)
    if op == "step":
        groups = min(groups, max(1, (64 * 8192 * 8 * 128) // (beams * ctx * hkv * d)))
    if op in ("select", "step"):
        kind = rng.choice(["bf16", "bf16", "fp32"])
        most = (64 * 8 * 131071 * 2) // (groups * beams * (2 if kind == "bf16" else 4))
        c.update(kind=kind, groups=groups, beams=beams, vocab=_log(rng, 200, min(262144, most)), pad=rng.choice([0, 0, 1, 24]))
        if op == "select":
            return dict(c, k=rng.choice([beams, 2 * beams]), done=rng.random() < 0.4)
        return dict(c, k=beams, cache=cache, layers=1, least=_log(rng, 1, ctx), ctx=ctx, gen=_log(rng, 1, 200), hq=hq, hkv=hkv, d=d,
                    page=page, src_least=_log(rng, 1, src), src=src)
    most = (32 * 5 * 12 * 4 * 64 * 128) // (beams * hkv * page * d)
    groups = min(groups, most)
    layers = _log(rng, 1, max(1, min(24, most // groups)))
    return dict(c, layers=layers, groups=groups, beams=beams, least=_log(rng, 1, ctx), ctx=ctx, gen=_log(rng, 1, 200),
                hist=_log(rng, 1, 1024), state=4 * _log(rng, 1, 4096), hkv=hkv, d=d, page=page)


def _lengths(rng, count, least, most):
    lens = [_log(rng, least, most) for _ in range(count)]
    lens[0] = most
    return lens


def _shape(case):
    """Lengths that the case stands for: (targets, sources) of a pack; sources; cached tokens and parents of every group."""
    rng = random.Random(case["mix"])
    op = case["op"]
    if op in ("train", "fwd"):
        return _lengths(rng, case["docs"], case["q_least"], case["q_most"]), _lengths(rng, case["docs"], case["k_least"], case["k_most"])
    if op == "attend":
        return _lengths(rng, case["batch"], case["least"], case["ctx"])
    if op == "select":
        return None
    groups, beams = case["groups"], case["beams"]
    lens = _lengths(rng, groups, case["least"], case["ctx"])
    # some beams live on in their places, each followed by its other continuations: reordering twice is reordering once
    roots = [[0] + [j for j in range(1, beams) if rng.random() < 0.5] for _ in range(groups)]
    parents = [[max(r for r in up if r <= j) for j in range(beams)] for up in roots]
    return lens, parents, (_lengths(rng, groups, case["src_least"], case["src"]) if op == "step" else None)


def _ends(counts, device):
    return torch.tensor([0] + counts, dtype=torch.int32).cumsum(0).to(torch.int32).to(device)


def _angles(rows, rot, device):
    """(cos, sin) of every position and pair, from 64 bits: [rows, rot / 2, 2]."""
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=device) / rot)
    a = torch.arange(rows, dtype=torch.float64, device=device)[:, None] * inv
    return torch.stack((a.cos(), a.sin()), -1).float()


def _cache(s, name, int4, layers, count, hkv, page, d, g):
    """Pages of all layers under s[name + "_k"] and so on, 4-bit rows with their scales."""
    dev = g.device
    for x in "kv":
        rows = torch.empty((layers, count, hkv, page, d), dtype=torch.bfloat16, device=dev).normal_(generator=g)
        if int4:
            s[name + "_" + x], s[name + "_" + x + "s"] = _quantise(rows)
        else:
            s[name + "_" + x] = rows


def _pages_of(used, width, order, device):
    """A page table whose sequence b owns the next used[b] pages of `order`; other entries name no page."""
    table = torch.full((len(used), width), -1, dtype=torch.int32, device=device)
    table[torch.arange(width, device=device) < torch.tensor(used, device=device)[:, None]] = order[:sum(used)]
    return table


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    op = case["op"]
    s = dict(case=case)

    def randn(*shape):
        return torch.randn(shape, generator=g, device=dev)

    if op in ("train", "fwd"):
        qn, kn = _shape(case)
        hq, hkv, d = case["hq"], case["hkv"], case["d"]
        s["cu"], s["cu_keys"], s["q_most"], s["k_most"] = _ends(qn, dev), _ends(kn, dev), max(qn), max(kn)
        s["q"], s["dout"] = (randn(sum(qn), hq, d).to(torch.bfloat16) for _ in range(2))
        s["k"], s["v"] = (randn(sum(kn), hkv, d).to(torch.bfloat16) for _ in range(2))
        s["out"], s["lse"] = torch.empty_like(s["q"]), torch.empty((hq, sum(qn)), device=dev)
        s["dq"], s["dk"], s["dv"] = (torch.empty_like(s[x]) for x in "qkv")
        if own:  # what a training program plans once for a pack and all its layers
            from packed_varlen_attention_cu_gb300 import api
            s["mask"] = api.make_mask(api.MASK_CROSS, sum(qn), sum(kn), cu_keys=s["cu_keys"])
            s["params"] = api.make_params(hq, hkv, c_tile=api.default_c_tile(d), pack_docs=1)
            s["worklist"] = api.alloc_worklist(len(qn), s["mask"], s["params"], dev)
            api.build_worklist(s["cu"], s["mask"], s["params"], s["worklist"])
            if op == "train":
                s["plan"] = api.alloc_bwd_plan(len(qn), s["mask"], s["params"], dev)
                api.build_bwd_plan(s["worklist"], len(qn), s["mask"], s["params"], s["plan"])
        return s
    if op == "attend":
        _sources(s, _shape(case), case["beams"], case, g, randn)
        if own:
            _own_sources(s, case)
        return s
    groups, beams = case["groups"], case["beams"]
    rows = groups * beams
    if op in ("select", "step"):
        v, k = case["vocab"], case["k"]
        x = randn(rows, v + case["pad"]) * 2.5
        scores = -3 * randn(groups, beams).abs()
        if op == "select":
            if beams > 1:
                scores[0, beams // 2] = -math.inf  # a beam that died
        else:
            # strong tokens, so that the parents are those that the case stands for
            _, parents, _ = _shape(case)
            strong = [(b * beams + p, j) for b, row in enumerate(parents) for j, p in enumerate(row)]
            at = torch.tensor(strong, device=dev)
            place = torch.rand((rows, 1), generator=g, device=dev)
            token = ((at[:, 1:] + place) / beams * v).long().clamp(max=v - 1)
            x[at[:, 0], token[:, 0]] = 120 - 0.5 * at[:, 1]
            is_root = torch.tensor([[p == j for j, p in enumerate(row)] for row in parents], device=dev)
            scores = torch.where(is_root, -6.0 * torch.arange(beams, device=dev) + 0.01 * scores, scores - 6.0 * beams - 60)
        s["scores"] = scores.float().contiguous()
        s["logits"] = x.to(torch.bfloat16 if case["kind"] == "bf16" else torch.float32)[:, :v]
        s["out_scores"] = torch.empty((groups, k), device=dev)
        s["out_beams"], s["out_tokens"] = (torch.empty((groups, k), dtype=torch.int32, device=dev) for _ in range(2))
        if case.get("done"):
            s["finished"] = (torch.rand((groups, beams), generator=g, device=dev) < 0.25).to(torch.uint8)
            s["norms"] = (5 + torch.randint(0, 200, (groups, beams), generator=g, device=dev).float()) ** -0.6
            s["out_finished"] = torch.empty((groups, k), dtype=torch.uint8, device=dev)
        if own:
            from packed_varlen_attention_cu_gb300 import api
            s["beam_work"] = api.alloc_beam_workspace(groups, beams, v, k, device=dev)
        if op == "select":
            return s
    # caches of the beams: a group's prompt lies in pages that its beams share, what was generated in pages of each beam
    lens, parents, src = _shape(case)
    page, hkv, d = case["page"], case["hkv"], case["d"]
    used = [n // page + 1 for n in lens]
    first = [max(n - case["gen"], 0) // page for n in lens]
    width = max(used)
    count = sum(f + beams * (u - f) for u, f in zip(used, first)) + 3
    order = torch.randperm(count, generator=g, device=dev).to(torch.int32)
    shared = _pages_of(first, width, order, dev).repeat_interleave(beams, 0)
    private = _pages_of([u - f for u, f in zip(used, first) for _ in range(beams)], width, order[sum(first):], dev)
    column = torch.arange(width, device=dev) - torch.tensor(first, device=dev).repeat_interleave(beams)[:, None]
    s["pages"] = torch.where(column < 0, shared, private.gather(1, column.clamp(min=0))).contiguous()
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev).repeat_interleave(beams)
    s["longest"] = max(lens) + 1
    _cache(s, "self", case.get("cache") == "int4", case["layers"], count, hkv, page, d, g)
    if op == "reorder":
        s["parents"] = torch.tensor(parents, dtype=torch.int32, device=dev)
        s["history"] = torch.randint(0, 1 << 30, (rows, case["hist"]), generator=g, device=dev, dtype=torch.int32)
        s["state"] = randn(rows, case["state"] // 4)
    else:
        hq = case["hq"]
        qkv = randn(rows, hq + 2 * hkv, d).to(torch.bfloat16)
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        s["table"], s["lens_new"] = _angles(s["longest"], d, dev), s["lens"] + 1
        s["q_rot"], s["self_out"] = (torch.empty((rows, hq, d), dtype=torch.bfloat16, device=dev) for _ in range(2))
        s["self_lse"] = torch.empty((hq, rows), device=dev)
        _sources(s, src, beams, case, g, randn)
    if own:
        from packed_varlen_attention_cu_gb300 import api
        s["caches"] = [api.KVCache(*(s[x][i] if x in s else None for x in ("self_k", "self_v", "self_ks", "self_vs")))
                       for i in range(case["layers"])]
        if op == "step":
            s["self_work"] = api.alloc_cache_workspace(rows, case["hq"], hkv, d, device=dev)
            _own_sources(s, case)
    return s


def _sources(s, lens, beams, case, g, randn):
    """Cached keys and values of sources, and the queries of their beams."""
    hq, hkv, d, page, dev = case["hq"], case["hkv"], case["d"], case["page"], g.device
    used = [-(-n // page) for n in lens]
    count = sum(used) + 2
    s["src_pages"] = _pages_of(used, max(used), torch.randperm(count, generator=g, device=dev).to(torch.int32), dev)
    s["src_lens"], s["src_most"] = torch.tensor(lens, dtype=torch.int32, device=dev), max(lens)
    s["src_cu"] = torch.arange(0, len(lens) + 1, device=dev, dtype=torch.int32) * beams
    _cache(s, "src", case["cache"] == "int4", 1, count, hkv, page, d, g)
    rows = len(lens) * beams
    s["src_q"] = randn(rows, hq, d).to(torch.bfloat16)
    s["src_out"], s["src_lse"] = torch.empty((rows, hq, d), dtype=torch.bfloat16, device=dev), torch.empty((hq, rows), device=dev)


def _own_sources(s, case):
    from packed_varlen_attention_cu_gb300 import api
    s["src_cache"] = api.KVCache(*(s[x][0] if x in s else None for x in ("src_k", "src_v", "src_ks", "src_vs")))
    s["src_work"] = api.alloc_cache_workspace(s["src_lens"].numel(), case["hq"], case["hkv"], case["d"], max_new=case["beams"],
                                              device=s["src_q"].device)


# ------------------------------------------------------------ plain forms

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


def _rows(s, x, page, slot):
    """Rows of the first layer's cache in fp32 at page and slot."""
    if x + "s" in s:
        return _values(s[x][0][page, :, slot], s[x + "s"][0][page, :, slot])
    return s[x][0][page, :, slot].float()


def _padded(x, cu, most):
    """Rows of a pack in fp32 by document: [docs, most, heads, d], rows past a document's end 0, and which rows are there."""
    n = (cu[1:] - cu[:-1])[:, None]
    i = torch.arange(most, device=cu.device)
    there = i < n
    at = torch.where(there, cu[:-1, None] + i, 0)
    return torch.where(there[..., None, None], x[at].float(), 0.0), there


def _cross(s):
    case = s["case"]
    hkv, d = case["hkv"], case["d"]
    group, scale = case["hq"] // hkv, d ** -0.5
    q, q_there = _padded(s["q"], s["cu"], s["q_most"])
    k, k_there = _padded(s["k"], s["cu_keys"], s["k_most"])
    v, _ = _padded(s["v"], s["cu_keys"], s["k_most"])

    def by_head(x):  # [docs, kv heads, group * rows, d]: the rows of a kv head's query heads below each other
        return x.unflatten(2, (hkv, group)).permute(0, 2, 3, 1, 4).flatten(2, 3)

    def as_pack(x):  # back, and only the rows that are there
        return x.unflatten(2, (group, -1)).permute(0, 3, 1, 2, 4).flatten(2, 3)[q_there]

    q, k, v = by_head(q), k.transpose(1, 2), v.transpose(1, 2)
    p = (q * scale) @ k.transpose(2, 3)
    p.masked_fill_(~k_there[:, None, None], -math.inf)
    top = p.amax(-1, keepdim=True)
    p.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    p.div_(total)
    o = p @ v
    out = {"out": as_pack(o).to(torch.bfloat16), "lse": as_pack(top + total.log())[..., 0].t().contiguous()}
    if case["op"] == "fwd":
        return out
    do = by_head(_padded(s["dout"], s["cu"], s["q_most"])[0])
    dv = p.transpose(2, 3) @ do
    ds = do @ v.transpose(2, 3)
    ds.sub_((do * o).sum(-1, keepdim=True)).mul_(p).mul_(scale)
    dq, dk = ds @ k, ds.transpose(2, 3) @ q
    return dict(out, dq=as_pack(dq).to(torch.bfloat16), dk=dk.transpose(1, 2)[k_there].to(torch.bfloat16),
                dv=dv.transpose(1, 2)[k_there].to(torch.bfloat16))


def _attend(s, name, q, pages, lens, most, beams):
    """Every query of a sequence's beams over all that it has cached."""
    case = s["case"]
    hkv, d = case["hkv"], case["d"]
    j = torch.arange(most, device=q.device)
    page = pages[:, j // case["page"]].clamp(min=0)
    slot = (j % case["page"]).expand_as(page)
    k, v = (_rows(s, name + "_" + x, page, slot) for x in "kv")  # [sequences, keys, kv heads, d]
    there = (j < lens[:, None])[:, None, None]
    v = v * there[:, 0, 0, :, None, None]
    x = q.float().unflatten(0, (-1, beams)).unflatten(2, (hkv, -1)).permute(0, 2, 1, 3, 4)  # [sequences, kv heads, beams, group, d]
    score = (x.flatten(2, 3) * d ** -0.5) @ k.permute(0, 2, 3, 1)
    score = score.masked_fill(~there, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = (score - top).exp()
    total = p.sum(-1, keepdim=True)
    o = (p @ v.transpose(1, 2)) / total
    o, lse = (y.unflatten(2, (beams, -1)).permute(0, 2, 1, 3, 4).flatten(2, 3).flatten(0, 1) for y in (o, top + total.log()))
    return o.to(torch.bfloat16), lse[..., 0].t().contiguous()


def _select(s):
    case = s["case"]
    k, v = case["k"], case["vocab"]
    groups, beams = s["scores"].shape
    x = s["logits"].double()
    top = x.amax(-1, keepdim=True)
    lse = (x - top).exp().sum(-1).log() + top[:, 0]
    value, token = s["logits"].float().sort(dim=-1, descending=True, stable=True)
    value, token = value[:, :k], token[:, :k]
    score = (s["scores"].double().flatten() - lse)[:, None] + value.double()
    if "finished" in s:  # a finished beam has one candidate: itself
        done = s["finished"].flatten().bool()[:, None]
        first = torch.arange(score.shape[1], device=x.device) == 0
        itself = torch.where(first, s["scores"].double().flatten()[:, None], -math.inf)
        score, token = torch.where(done, itself, score), torch.where(done, 2, token)
    rank = score if "norms" not in s else score * s["norms"].double().flatten()[:, None]
    rank = rank.unflatten(0, (groups, beams)).flatten(1).sort(dim=-1, descending=True, stable=True)
    rank, at = rank.values[:, :k], rank.indices[:, :k]
    good = rank > -math.inf
    out = {"scores": score.unflatten(0, (groups, beams)).flatten(1).gather(1, at).float(),
           "beams": torch.where(good, at // token.shape[1], -1).int(),
           "tokens": torch.where(good, token.unflatten(0, (groups, beams)).flatten(1).gather(1, at), -1).int()}
    if "finished" in s:
        out["finished"] = (good & ((out["tokens"] == 2) | s["finished"].bool().gather(1, out["beams"].long().clamp(min=0)))).to(torch.uint8)
    return out


def _reorder(s, parents):
    """Pages and states follow the parents, in place."""
    case = s["case"]
    page, beams = case["page"], case["beams"]
    rows = torch.arange(parents.numel(), device=parents.device)
    source = rows // beams * beams + parents.flatten()
    last, part = s["lens"] // page, s["lens"] % page
    full = torch.arange(s["pages"].shape[1], device=rows.device) < last[:, None]
    frm, to = s["pages"][source, last], s["pages"][rows, last]
    mine = torch.arange(page, device=rows.device) < part[:, None]
    for x in ("self_k", "self_v", "self_ks", "self_vs"):
        if x in s:
            width = (slice(None), None, slice(None)) + (None,) * (s[x].ndim - 4)  # [rows, 1, slots, 1 ..]
            s[x][:, to] = torch.where(mine[width], s[x][:, frm], s[x][:, to])
    s["pages"].copy_(torch.where(full, s["pages"][source], s["pages"]))
    for x in ("history", "state"):
        if x in s:
            s[x].copy_(s[x][source])


def _append(s):
    """The new token's key and value go behind what is cached; its query, turned by its position."""
    case = s["case"]
    half = case["d"] // 2
    turn = s["table"][s["lens"]]
    c, n = turn[:, None, :, 0], turn[:, None, :, 1]

    def turned(x):
        a, b = x[..., :half].float(), x[..., half:].float()
        return torch.cat((a * c - b * n, b * c + a * n), -1).to(torch.bfloat16)

    rows = torch.arange(s["lens"].numel(), device=turn.device)
    page, slot = s["pages"][rows, s["lens"] // case["page"]], s["lens"] % case["page"]
    for x, new in (("self_k", turned(s["k"])), ("self_v", s["v"])):
        if x + "s" in s:
            s[x][0][page, :, slot], s[x + "s"][0][page, :, slot] = _quantise(new)
        else:
            s[x][0][page, :, slot] = new
    return turned(s["q"])


def _state(s):
    return {x: s[x] for x in ("pages", "self_k", "self_v", "history", "state")}


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op in ("train", "fwd"):
        return _cross(s)
    if op == "attend":
        out, lse = _attend(s, "src", s["src_q"], s["src_pages"], s["src_lens"], s["src_most"], case["beams"])
        return {"out": out, "lse": lse}
    if op == "select":
        return _select(s)
    if op == "reorder":
        _reorder(s, s["parents"])
        return _state(s)
    best = _select(s)
    _reorder(s, best["beams"])
    q = _append(s)
    best["self"] = _attend(s, "self", q, s["pages"], s["lens_new"], s["longest"], 1)
    best["source"] = _attend(s, "src", s["src_q"], s["src_pages"], s["src_lens"], s["src_most"], case["beams"])
    return best


# ------------------------------------------------------------ the package

def _run_own(s):
    from packed_varlen_attention_cu_gb300 import api
    case = s["case"]
    op = case["op"]
    if op in ("train", "fwd"):
        api.attn_fwd(s["q"], s["k"], s["v"], s["cu"], s["mask"], s["params"], s["worklist"], s["out"], s["lse"])
        out = {"out": s["out"], "lse": s["lse"]}
        if op == "fwd":
            return out
        api.attn_bwd(s["q"], s["k"], s["v"], s["out"], s["lse"], s["dout"], s["cu"], case["docs"], s["mask"], s["params"],
                     s["worklist"], s["plan"], s["dq"], s["dk"], s["dv"])
        return dict(out, dq=s["dq"], dk=s["dk"], dv=s["dv"])
    if op in ("select", "step"):
        api.beam_select(s["logits"], s["scores"], s["out_scores"], s["out_beams"], s["out_tokens"], s["beam_work"],
                        end_token=2, finished=s.get("finished"), norms=s.get("norms"), out_finished=s.get("out_finished"))
        out = {"scores": s["out_scores"], "beams": s["out_beams"], "tokens": s["out_tokens"]}
        if op == "select":
            return dict(out, finished=s["out_finished"]) if "finished" in s else out
    if op == "reorder":
        api.beam_reorder(s["parents"], s["caches"], s["pages"], s["lens"], states=(s["history"], s["state"]))
        return _state(s)
    if op == "step":
        cache = s["caches"][0]
        api.beam_reorder(s["out_beams"], s["caches"], s["pages"], s["lens"])
        api.cache_append(cache, s["k"], s["v"], s["pages"], s["lens_new"], table=s["table"], q=s["q"], q_out=s["q_rot"])
        api.cache_attn(cache, s["q_rot"], s["pages"], s["lens_new"], s["self_out"], s["self_lse"], s["self_work"])
        out["self"] = s["self_out"], s["self_lse"]
    api.cache_cross_attn(s["src_cache"], s["src_q"], s["src_pages"], s["src_lens"], s["src_out"], s["src_lse"], s["src_work"],
                         cu_new=s["src_cu"], max_new=case["beams"])
    if op == "step":
        out["source"] = s["src_out"], s["src_lse"]
        return out
    return {"out": s["src_out"], "lse": s["src_lse"]}


def run(state):
    return _run_own(state) if own else _run_plain(state)


def work(case):
    op = case["op"]
    done = {"bytes": 0, "flops": 0}
    shape = _shape(case)

    def row(c):  # a cached row of one head: its values, or codes and scales
        return 2 * c["d"] if c.get("cache") != "int4" else c["d"] // 2 + c["d"] // 16

    def attend(lens, rows):
        done["bytes"] += sum(lens) * 2 * case["hkv"] * row(case) + len(lens) * rows * case["hq"] * (4 * case["d"] + 4)
        done["flops"] += 4 * sum(lens) * rows * case["hq"] * case["d"]

    if op in ("train", "fwd"):
        hq, hkv, d = case["hq"], case["hkv"], case["d"]
        q, k = sum(shape[0]) * hq, sum(shape[1]) * hkv * d * 2
        pairs = sum(a * b for a, b in zip(*shape))
        train = op == "train"
        return {"bytes": q * (d * 2 * (4 if train else 2) + 4) + k * (4 if train else 2), "flops": (14 if train else 4) * pairs * hq * d}
    if op == "attend":
        attend(shape, case["beams"])
        return done
    rows = case["groups"] * case["beams"]
    if op in ("select", "step"):
        done["bytes"] += rows * (case["vocab"] * (2 if case["kind"] == "bf16" else 4) + 4) + case["groups"] * case["k"] * 12
        done["flops"] += 4 * rows * case["vocab"]
        if op == "select":
            return done
    lens, parents, src = shape
    page = case["page"]
    for n, up in zip(lens, parents):
        moved = sum(p != j for j, p in enumerate(up))
        read = len({p for j, p in enumerate(up) if p != j})
        each = n % page * case["layers"] * 2 * case["hkv"] * row(case) + n // page * 4
        if op == "reorder":
            each += 4 * case["hist"] + case["state"]
        done["bytes"] += (moved + read) * each + 8 * case["beams"]
    if op == "step":
        hq, hkv, d = case["hq"], case["hkv"], case["d"]
        done["bytes"] += rows * ((2 * hq + 2 * hkv) * d * 2 + 2 * hkv * row(case))
        # a group's beams share what lies before their own pages
        for n in lens:
            first = max(n - case["gen"], 0) // page * page
            done["bytes"] += (first + case["beams"] * (n + 1 - first)) * 2 * hkv * row(case) + case["beams"] * hq * (4 * d + 4)
            done["flops"] += 4 * case["beams"] * (n + 1) * hq * d
        attend(src, case["beams"])
    return done


# ------------------------------------------------------------ 64 bits

def exact(case, seed):
    """The operators by their definitions, sequence by sequence, in 64 bits."""
    op = case["op"]
    if op == "step" and case["groups"] * case["beams"] > 256:
        return None
    s = prepare(case, seed)
    shape = _shape(case)
    if op in ("train", "fwd"):
        hkv = case["hkv"]
        names = ("out", "lse", "dq", "dk", "dv") if op == "train" else ("out", "lse")
        got = {x: [] for x in names}
        a = c = 0
        for m, n in zip(*shape):
            q, k, v = (t[i:i + r].double().requires_grad_(op == "train") for t, i, r in ((s["q"], a, m), (s["k"], c, n), (s["v"], c, n)))
            sc = torch.einsum("mhgd,lhd->hgml", q.unflatten(1, (hkv, -1)), k) / math.sqrt(case["d"])
            lse = torch.logsumexp(sc, -1)
            o = torch.einsum("hgml,lhd->mhgd", (sc - lse[..., None]).exp(), v).flatten(1, 2)
            if op == "train":
                for x, grad in zip(("dq", "dk", "dv"), torch.autograd.grad(o, (q, k, v), s["dout"][a:a + m].double())):
                    got[x].append(grad)
            got["out"].append(o.detach())
            got["lse"].append(lse.detach().flatten(0, 1))
            del sc, o, lse
            a, c = a + m, c + n
        return {x: torch.cat(y, -1 if x == "lse" else 0) for x, y in got.items()}

    def held(name, pages, n):
        """All cached rows of one sequence: [n, heads, d]."""
        at = pages[:-(-n // case["page"])].long()
        rows = s[name][0][at].transpose(1, 2).flatten(0, 1)[:n]
        if name + "s" not in s:
            return rows.double()
        sc = s[name + "s"][0][at].transpose(1, 2).flatten(0, 1)[:n].double()
        groups = case["d"] // 64
        out = torch.empty(rows.shape[:-1] + (case["d"],), dtype=torch.float64, device=rows.device)
        for i in range(case["d"]):
            # dim i: which byte and which half of it
            word, bit = (i % 64) // 8 * groups + i // 64, 4 * (i % 8 // 2) + 16 * (i % 2)
            byte = rows[..., 4 * word + bit // 8].long()
            out[..., i] = sc[..., i // 64, 1] + ((byte >> 4) if bit % 8 else (byte & 15)) * sc[..., i // 64, 0]
        return out

    def attention(q, k, v):
        """[m, heads, d] over [n, kv heads, d], nothing masked: the result and [heads, m] of logarithms."""
        sc = torch.einsum("mhgd,lhd->hgml", q.unflatten(1, (case["hkv"], -1)), k) / math.sqrt(case["d"])
        lse = torch.logsumexp(sc, -1)
        return torch.einsum("hgml,lhd->mhgd", (sc - lse[..., None]).exp(), v).flatten(1, 2), lse.flatten(0, 1)

    def over_sources(lens):
        both = [attention(s["src_q"][b * case["beams"]:(b + 1) * case["beams"]].double(), *(held("src_" + x, s["src_pages"][b], n) for x in "kv"))
                for b, n in enumerate(lens)]
        return torch.cat([o for o, _ in both]), torch.cat([e for _, e in both], -1)

    if op == "attend":
        out, lse = over_sources(shape)
        return {"out": out, "lse": lse}
    beams = case["beams"]
    if op in ("select", "step"):
        logp = torch.log_softmax(s["logits"].double(), -1) + s["scores"].double().flatten()[:, None]
        if "finished" in s:
            done = s["finished"].flatten().bool()
            alone = torch.full_like(logp, -math.inf)
            alone[:, 2] = s["scores"].double().flatten()
            logp = torch.where(done[:, None], alone, logp)
        key = logp if "norms" not in s else logp * s["norms"].double().flatten()[:, None]
        key, logp = key.view(case["groups"], -1), logp.view(case["groups"], -1)
        at = torch.stack([key[b].sort(dim=-1, descending=True, stable=True).indices[:case["k"]] for b in range(case["groups"])])
        best = {"scores": logp.gather(1, at), "beams": (at // case["vocab"]).int(), "tokens": (at % case["vocab"]).int()}
        none = ~torch.isfinite(best["scores"])
        best["beams"][none] = best["tokens"][none] = -1
        if "finished" in s:
            was = s["finished"].bool().gather(1, best["beams"].clamp(min=0).long())
            best["finished"] = ((was | (best["tokens"] == 2)) & ~none).to(torch.uint8)
        del logp, key
        if op == "select":
            return best
    lens, parents, src = shape
    page = case["page"]
    up = torch.tensor(parents) if op == "reorder" else best["beams"].cpu()
    old_pages = s["pages"].clone()
    frm = {x: s[x].clone() for x in ("self_k", "self_v", "self_ks", "self_vs", "history", "state") if x in s}
    for b, n in enumerate(lens):
        for j in range(beams):
            row, parent = b * beams + j, b * beams + int(up[b, j])
            s["pages"][row, :n // page] = old_pages[parent, :n // page]
            here, there = int(old_pages[row, n // page]), int(old_pages[parent, n // page])
            for x in ("self_k", "self_v", "self_ks", "self_vs"):
                if x in s:
                    s[x][:, here, :, :n % page] = frm[x][:, there, :, :n % page]
            for x in ("history", "state"):
                if x in s:
                    s[x][row] = frm[x][parent]
    if op == "reorder":
        return {x: (s[x].double() if s[x].is_floating_point() else s[x]) for x in ("pages", "self_k", "self_v", "history", "state")}

    def rounded(x, int4):
        """What the cache holds of new rows."""
        x = x.to(torch.float32).to(torch.bfloat16).double()
        if not int4:
            return x
        part = x.unflatten(-1, (-1, 64))
        low, high = part.min(-1, keepdim=True).values, part.max(-1, keepdim=True).values
        step = ((high - low) / 15).to(torch.float32).to(torch.bfloat16).double()
        n = torch.where(step > 0, torch.round((part - low) / torch.where(step > 0, step, torch.ones_like(step))), torch.zeros_like(part))
        return (low + n.clamp(0, 15) * step).flatten(-2)

    def turned(x, at):
        """Complex rotation of the pairs by the table's angles at one position."""
        x, half = x.double(), case["d"] // 2
        w = torch.complex(x[..., :half].contiguous(), x[..., half:].contiguous()) * torch.view_as_complex(s["table"][at].double())
        return torch.cat((w.real, w.imag), -1)

    int4, outs, lses = case["cache"] == "int4", [], []
    for b, n in enumerate(lens):
        for j in range(beams):
            row = b * beams + j
            k, v = (torch.cat((held("self_" + x, s["pages"][row], n), rounded(new, int4)[None]))
                    for x, new in (("k", turned(s["k"][row], n)), ("v", s["v"][row].double())))
            o, lse = attention(rounded(turned(s["q"][row], n), False)[None], k, v)
            outs.append(o)
            lses.append(lse)
    return dict(best, self=(torch.cat(outs), torch.cat(lses, -1)), source=over_sources(src))
