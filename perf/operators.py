"""Cases and plain forms of the operators around the verification step.

Five operators, in the order a serving program uses them:

  tables  block tables and slot maps of admitted requests, from their lengths
  write   packed K/V rows scattered into the pages through a slot map
  prompt  causal attention of packed prompts over their pages
  prefix  verification attention of a batch that shares a long prefix
  logits  penalties, biases and grammar masks on the target's logits

``run`` computes an operator in elementary torch operations, or, where ``own``
is true, through the framework's own entry points.  Lengths follow from the
case alone, values from the seed.
"""
import math
import random

import torch

own = False

PAGE = 16
FP8_MAX = 448.0


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # a handful of chat requests admitted between two steps: latency
        dict(name="tables-few", op="tables", batch=8, lo=20, hi=700, prefix=0, idle=0, spare=0),
        # a large admission behind a system prompt, some batch slots idle
        dict(name="tables-many", op="tables", batch=256, lo=900, hi=32768, prefix=800, idle=9, spare=100),
        # one short prompt's rows into FP8 pages with a scale for each 64 values
        dict(name="write-fp8-short", op="write", tokens=57, hkv=8, d=128, fp8=True, fused=False, holes=3),
        # a long prefill batch into bf16 pages, sliced out of a fused projection
        dict(name="write-long", op="write", tokens=32768, hkv=8, d=128, fp8=False, fused=True, holes=0),
        # a single short prompt of the small multi-head shape: latency
        dict(name="prompt-short", op="prompt", batch=1, lo=37, hi=37, cached_lo=0, cached_hi=0, hq=4, hkv=4, d=64,
             fused=False),
        # ragged multi-head prompts, some of them chunks behind cached tokens
        dict(name="prompt-ragged", op="prompt", batch=11, lo=1, hi=900, cached_lo=0, cached_hi=500, hq=32, hkv=32,
             d=128, fused=True),
        # one long grouped-query prompt
        dict(name="prompt-long", op="prompt", batch=1, lo=8192, hi=8192, cached_lo=0, cached_hi=0, hq=64, hkv=8,
             d=128, fused=False),
        # a few sequences behind a short instruction, single-token decoding
        dict(name="prefix-few", op="prefix", batch=6, lo=1, hi=90, prefix=512, nodes=1, tree=False, hq=32, hkv=8,
             d=128),
        # grouped-query verification of five drafts behind a long document
        dict(name="prefix-long", op="prefix", batch=40, lo=64, hi=1024, prefix=8192, nodes=6, tree=False, hq=64,
             hkv=8, d=128),
        # draft trees behind a shared system prompt, long private histories
        dict(name="prefix-tree", op="prefix", batch=128, lo=1024, hi=8192, prefix=800, nodes=29, tree=True, hq=32,
             hkv=8, d=128),
        # a small batch with a 32K vocabulary: latency
        dict(name="logits-few", op="logits", batch=2, rows=5, vocab=32000, bf16=False, hist=300, bias=4, mask=True,
             tree=False),
        # a full batch of the large vocabulary, bf16 logits, long histories
        dict(name="logits-many", op="logits", batch=64, rows=6, vocab=128256, bf16=True, hist=8192, bias=100,
             mask=True, tree=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("tables", "write", "prompt", "prefix", "logits"))
    if op == "tables":
        pages = rng.choice((0, 0, 1, 7, 50, 128))
        lo = PAGE * pages + _log(rng, 1, 64)
        batch = _log(rng, 2, 256)
        return dict(op=op, batch=batch, lo=lo, hi=lo + _log(rng, 16, 20000), prefix=PAGE * pages,
                    idle=rng.randrange(0, 1 + batch // 2), spare=rng.choice((0, 1, 77)))
    if op == "write":
        fp8 = rng.random() < 0.5
        return dict(op=op, tokens=_log(rng, 1, 32768), hkv=rng.choice((1, 2, 4, 5, 8)),
                    d=rng.choice((64, 128)), fp8=fp8, fused=rng.random() < 0.5, holes=rng.choice((0, 0, 5)))
    if op == "prompt":
        hkv, g = rng.choice(((4, 1), (32, 1), (8, 4), (8, 8), (2, 7), (1, 16)))
        tokens = _log(rng, 16, 7000)
        batch = min(tokens, _log(rng, 1, 40))
        hi = max(1, 2 * tokens // batch - 1) if batch > 1 else tokens
        cached = rng.random() < 0.4
        return dict(op=op, batch=batch, lo=1 if batch > 1 else tokens, hi=hi, cached_lo=0,
                    cached_hi=_log(rng, 1, max(1, 2000 // batch)) if cached else 0, hq=hkv * g, hkv=hkv,
                    d=rng.choice((64, 128, 128)), fused=rng.random() < 0.5)
    if op == "prefix":
        tree = rng.random() < 0.4
        nodes = rng.randrange(2, 30) if tree else rng.randrange(1, 9)
        hkv, g = rng.choice(((8, 4), (8, 8), (32, 1), (2, 7), (1, 4)))
        if g * nodes > 128:
            nodes = 128 // g
        lo = _log(rng, 1, 500)
        return dict(op=op, batch=_log(rng, 2, 64), lo=lo, hi=lo + _log(rng, 1, 1500), prefix=PAGE * _log(rng, 1, 512),
                    nodes=nodes, tree=tree, hq=hkv * g, hkv=hkv, d=rng.choice((64, 128, 128)))
    tree = rng.random() < 0.3
    return dict(op=op, batch=_log(rng, 1, 64), rows=rng.randrange(2, 16) if tree else rng.randrange(1, 9),
                vocab=rng.choice((997, 32000, 50257, 128256)), bf16=rng.random() < 0.5, hist=_log(rng, 1, 8192),
                bias=rng.choice((0, 1, 40, 300)), mask=rng.random() < 0.7, tree=tree)


def _lengths(count, lo, hi, salt):
    """`count` lengths in [lo, hi], the same for every seed."""
    rng = random.Random(salt * 7919 + count)
    return [rng.randint(lo, hi) for _ in range(count)]


def _parents(nodes):
    """A draft tree in breadth-first order: four children of the root, then two of each node."""
    parent = [-1]
    at = 0
    while len(parent) < nodes:
        parent += [at] * min(4 if at == 0 else 2, nodes - len(parent))
        at += 1
    return parent


def _ancestors(nodes, tree):
    """Bit i of entry j: node i is j or an ancestor of j (a chain where there is no tree)."""
    parent = _parents(nodes) if tree else [j - 1 for j in range(nodes)]
    masks = []
    for j in range(nodes):
        masks.append((masks[parent[j]] if j else 0) | 1 << j)
    return masks


def _shape(c):
    """The case's lengths: what every function below derives its sizes from."""
    if c["op"] == "tables":
        lens = _lengths(c["batch"], c["lo"], c["hi"], 1)
        for i in range(c["idle"]):
            lens[(i * 5 + 1) % c["batch"]] = 0  # a batch slot without a request
        return dict(lens=lens, new=[n - c["prefix"] if n else 0 for n in lens],
                    pages=[-(-n // PAGE) for n in lens], width=-(-c["hi"] // PAGE) + 1)
    if c["op"] == "prompt":
        new = _lengths(c["batch"], c["lo"], c["hi"], 2)
        kv = [n + m for n, m in zip(new, _lengths(c["batch"], c["cached_lo"], c["cached_hi"], 3))]
        return dict(new=new, kv=kv, pages=[-(-n // PAGE) for n in kv], width=-(-max(kv) // PAGE))
    if c["op"] == "prefix":
        own_len = _lengths(c["batch"], c["lo"], c["hi"], 4)
        ctx = [c["prefix"] + n for n in own_len]
        pages = [-(-(n + c["nodes"]) // PAGE) for n in ctx]
        return dict(own=own_len, ctx=ctx, pages=pages, width=max(pages), shared=c["prefix"] // PAGE)
    if c["op"] == "logits":
        hist = _lengths(c["batch"], (c["hist"] + 1) // 2, c["hist"], 5)
        prompt = [n * 2 // 3 for n in hist]
        bias = _lengths(c["batch"], (c["bias"] + 1) // 2, c["bias"], 6)
        return dict(hist=hist, prompt=prompt, bias=bias)
    return {}


def work(c):
    s = _shape(c)
    if c["op"] == "tables":
        blocks = sum(s["pages"]) - sum(c["prefix"] // PAGE for n in s["lens"] if n)
        # lengths, blocks popped, counts set, tables, offsets and slots written
        words = c["batch"] + 2 * blocks + c["batch"] * s["width"] + c["batch"] + 1 + sum(s["new"]) + c["spare"]
        return dict(bytes=4 * (words + 2 * c["prefix"] // PAGE), flops=0)
    if c["op"] == "write":
        values = 2 * c["tokens"] * c["hkv"] * c["d"]
        out = values * 1 + values // 64 * 4 if c["fp8"] else values * 2
        return dict(bytes=values * 2 + out + 4 * c["tokens"], flops=0)
    if c["op"] == "prompt":
        pairs = sum(n * m - n * (n - 1) // 2 for n, m in zip(s["new"], s["kv"]))
        t = sum(s["new"])
        return dict(bytes=2 * 2 * t * c["hq"] * c["d"] + 4 * t * c["hq"] + 2 * 2 * sum(s["kv"]) * c["hkv"] * c["d"]
                    + 4 * sum(s["pages"]), flops=4 * c["d"] * c["hq"] * pairs)
    if c["op"] == "prefix":
        seen = sum(bin(m).count("1") for m in _ancestors(c["nodes"], c["tree"]))
        pairs = sum(n * c["nodes"] + seen for n in s["ctx"])
        t = c["batch"] * c["nodes"]
        tokens = c["prefix"] + sum(n + c["nodes"] for n in s["own"])
        return dict(bytes=2 * 2 * t * c["hq"] * c["d"] + 4 * t * c["hq"] + 2 * 2 * tokens * c["hkv"] * c["d"]
                    + 4 * sum(s["pages"]), flops=4 * c["d"] * c["hq"] * pairs)
    n = c["batch"] * c["rows"] * c["vocab"]
    return dict(bytes=n * ((2 if c["bf16"] else 4) + 4) + (n // 8 if c["mask"] else 0) + 4 * sum(s["hist"])
                + 8 * sum(s["bias"]), flops=0)


# ------------------------------------------------------------------ the inputs
def _pages(s, total, gen):
    """A shuffled pool of `total` pages."""
    return torch.randperm(total, generator=gen, device="cuda").to(torch.int32)


def _pool(total, c, gen):
    shape = (total, c["hkv"], PAGE, c["d"])
    return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)


def _table(pages, width, ids, shared):
    """Rows of block ids: the first `shared` pages the same in every row, the others taken in turn, -1 behind."""
    pages = torch.tensor(pages, device="cuda")
    at = torch.arange(width, device="cuda")
    mine = pages - shared
    start = shared + torch.cumsum(mine, 0) - mine
    pick = torch.where(at < shared, at, start[:, None] + at - shared)
    live = at < pages[:, None]
    return torch.where(live, ids[torch.where(live, pick, 0)], -1).to(torch.int32)


def _queries(tokens, c, gen, fused):
    """Query rows; sliced out of a fused Q/K/V projection where `fused`."""
    wide = c["hq"] + (2 * c["hkv"] if fused else 0)
    x = torch.empty((tokens, wide, c["d"]), dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    return x[:, :c["hq"]]


def prepare(c, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s, dev = _shape(c), "cuda"
    state = dict(case=c, shape=s)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    if c["op"] == "tables":
        shared = c["prefix"] // PAGE
        need = sum(s["pages"]) + shared
        total = need + need // 10 + 4
        ids = _pages(s, total, gen)
        # the prefix is held by the cache alone, a tenth of the rest by other requests
        count = torch.zeros(total, dtype=torch.int32, device=dev)
        top = total - shared - need // 20
        count[ids[top:].long()] = 1
        free = torch.full((total,), -1, dtype=torch.int32, device=dev)
        free[:top] = ids[:top]
        state.update(lens=ints(s["lens"]), prefix=ids[total - shared:].clone(), free_stack=free,
                     # [reference counts, free blocks] before and after the call
                     before=torch.cat([count, ints([top])]),
                     after=torch.empty(total + 1, dtype=torch.int32, device=dev),
                     table=torch.empty((c["batch"], s["width"]), dtype=torch.int32, device=dev),
                     offsets=torch.empty(c["batch"] + 1, dtype=torch.int32, device=dev),
                     slots=torch.empty(sum(s["new"]) + c["spare"], dtype=torch.int32, device=dev))
    elif c["op"] == "write":
        total = -(-c["tokens"] // PAGE) + 3
        wide = c["hkv"] * (3 if c["fused"] else 1)
        k = torch.empty((c["tokens"], wide, c["d"]), dtype=torch.bfloat16, device=dev).normal_(generator=gen)
        v = k if c["fused"] else torch.empty_like(k).normal_(generator=gen)
        # the last page stays free
        slots = _pages(s, total - 1, gen)[torch.arange(c["tokens"], device=dev) // PAGE] * PAGE
        slots = (slots + torch.arange(c["tokens"], device=dev) % PAGE).to(torch.int32)
        for i in range(min(c["holes"], c["tokens"] // 2)):  # padding rows of the batch
            slots[2 * i + 1] = -1
        state.update(k=k[:, wide - 2 * c["hkv"]:wide - c["hkv"]] if c["fused"] else k,
                     v=v[:, wide - c["hkv"]:] if c["fused"] else v, slots=slots)
        kind = torch.float8_e4m3fn if c["fp8"] else torch.bfloat16
        for name in ("k_pool", "v_pool"):
            state[name] = torch.zeros((total, c["hkv"], PAGE, c["d"]), dtype=torch.bfloat16, device=dev).to(kind)
        for name in ("k_scale", "v_scale"):
            state[name] = (torch.ones((total, c["hkv"], PAGE, c["d"] // 64), device=dev) if c["fp8"] else None)
    elif c["op"] == "prompt":
        total = sum(s["pages"]) + 5
        ids = _pages(s, total, gen)
        t = sum(s["new"])
        state.update(q=_queries(t, c, gen, c["fused"]), k_pool=_pool(total, c, gen), v_pool=_pool(total, c, gen),
                     table=_table(s["pages"], s["width"], ids, 0), kv_lens=ints(s["kv"]),
                     offsets=ints([sum(s["new"][:i]) for i in range(c["batch"] + 1)]),
                     out=torch.empty((t, c["hq"], c["d"]), dtype=torch.bfloat16, device=dev),
                     lse=torch.empty((t, c["hq"]), device=dev))
    elif c["op"] == "prefix":
        total = sum(s["pages"]) - s["shared"] * (c["batch"] - 1) + 5
        ids = _pages(s, total, gen)
        t = c["batch"] * c["nodes"]
        q = _queries(t, c, gen, False).view(c["batch"], c["nodes"], c["hq"], c["d"])
        state.update(q=q, k_pool=_pool(total, c, gen), v_pool=_pool(total, c, gen), ctx=ints(s["ctx"]),
                     table=_table(s["pages"], s["width"], ids, s["shared"]), prefix=ids[:s["shared"]].clone(),
                     ancestors=_ancestors(c["nodes"], c["tree"]),
                     seen=torch.tensor([[m >> i & 1 for i in range(c["nodes"])]
                                        for m in _ancestors(c["nodes"], c["tree"])], dtype=torch.bool, device=dev),
                     out=torch.empty_like(q), lse=torch.empty(q.shape[:3], device=dev))
    else:
        b, r, v = c["batch"], c["rows"], c["vocab"]
        logits = torch.empty((b, r, v), device=dev).normal_(0.0, 3.0, generator=gen)

        def tokens(*shape):  # a few tokens often, the others seldom, as in text
            u = torch.rand(shape, generator=gen, device=dev)
            return (u ** 4 * v).clamp(max=v - 1).to(torch.int32)

        parent = _parents(r) if c["tree"] else None
        bias_off = ints([sum(s["bias"][:i]) for i in range(b + 1)])
        state.update(logits=logits.bfloat16() if c["bf16"] else logits, history=tokens(b, c["hist"]),
                     hist_lens=ints(s["hist"]), prompt_lens=ints(s["prompt"]), parent=parent,
                     drafts=tokens(b, r if c["tree"] else r - 1),
                     seen=torch.tensor([[m >> i & 1 for i in range(1, r)] for m in _ancestors(r, c["tree"])],
                                       dtype=torch.bool, device=dev),
                     repetition=1.0 + 0.3 * torch.rand(b, generator=gen, device=dev),
                     presence=torch.rand(b, generator=gen, device=dev),
                     frequency=0.5 * torch.rand(b, generator=gen, device=dev),
                     bias_offsets=bias_off if c["bias"] else None,
                     bias_tokens=torch.cat([torch.randperm(v, generator=gen, device=dev)[:n] for n in s["bias"]])
                     .to(torch.int32) if c["bias"] else None,
                     bias_values=torch.empty(sum(s["bias"]), device=dev).normal_(0.0, 2.0, generator=gen)
                     if c["bias"] else None,
                     mask=torch.randint(-2 ** 31, 2 ** 31, (b, r, -(-v // 32)), generator=gen, device=dev)
                     .to(torch.int32) if c["mask"] else None,
                     out=torch.empty((b, r, v), device=dev))
    state["error"] = torch.zeros(1, dtype=torch.int32, device=dev)
    return state


# ------------------------------------------------------------------ the plain forms
def _attend(q, k, v, visible, scale):
    """Softmax attention in 32 bits: q [..., R, D], k and v [..., T, D], visible [..., R, T]."""
    x = torch.matmul(q, k.transpose(-1, -2)).mul_(scale).masked_fill_(~visible, -math.inf)
    top = x.amax(-1, keepdim=True)
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    return torch.matmul(x, v) / total, (top + total.log()).squeeze(-1)


def _plain_tables(s):
    c, shape = s["case"], s["shape"]
    lens, shared = s["lens"].long(), c["prefix"] // PAGE
    s["after"].copy_(s["before"])
    count, top = s["after"][:-1], s["after"][-1:]
    live = lens > 0
    pages = (lens + PAGE - 1) // PAGE
    mine = torch.where(live, pages - shared, 0)
    start = torch.cumsum(mine, 0) - mine
    at = torch.arange(shape["width"], device="cuda")
    nth = start[:, None] + at - shared
    popped = (at >= shared) & (at < pages[:, None])
    table = torch.where(popped, s["free_stack"][torch.where(popped, top - 1 - nth, 0)], -1)
    if shared:
        held = (at < shared) & live[:, None]
        table = torch.where(held, s["prefix"][at.clamp(max=shared - 1)], table)
        count.index_add_(0, s["prefix"].long(), live.sum().expand(shared).to(torch.int32))
    taken = mine.sum()
    n = shape["width"] * c["batch"]
    order = torch.arange(min(n, s["free_stack"].numel()), device="cuda")
    ids = s["free_stack"][(top - 1 - order).clamp(min=0)].long().clamp(min=0)
    count.index_put_((ids,), torch.where(order < taken, 1, 0).to(torch.int32), accumulate=True)
    top.sub_(taken.to(torch.int32))
    new = torch.where(live, lens - c["prefix"], 0)
    offsets = torch.cat([new.new_zeros(1), torch.cumsum(new, 0)])
    token = torch.arange(s["slots"].numel(), device="cuda")
    row = (torch.searchsorted(offsets, token, right=True) - 1).clamp(max=c["batch"] - 1)
    pos = c["prefix"] + token - offsets[row]
    inside = token < offsets[-1]
    block = table[row, torch.where(inside, pos // PAGE, 0)]
    slots = torch.where(inside, block * PAGE + pos % PAGE, -1)
    return dict(table=table.to(torch.int32), offsets=offsets.to(torch.int32), slots=slots.to(torch.int32),
                counts_and_top=s["after"])


def _dequantised(pool, scale):
    p = pool.float()
    return (p.view(*p.shape[:-1], -1, 64) * scale[..., None]).view(p.shape)


def _plain_write(s):
    c = s["case"]
    live = s["slots"] >= 0
    # a padding row writes what the pool's last, free slot holds back to it
    slot = torch.where(live, s["slots"], s["k_pool"].shape[0] * PAGE - 1).long()
    block, at = slot // PAGE, slot % PAGE
    for name in ("k", "v"):
        pool = s[name + "_pool"]
        if c["fp8"]:
            x = s[name].float().reshape(c["tokens"], c["hkv"], c["d"] // 64, 64)
            amax = x.abs().amax(-1)
            # (a quotient of tensors: by a number it would be a product with the reciprocal)
            scale = torch.where(amax > 0, amax / torch.full_like(amax, FP8_MAX), 1.0)
            rows = (x / scale[..., None]).reshape(c["tokens"], c["hkv"], c["d"]).to(torch.float8_e4m3fn)
            rows, raw = rows.view(torch.uint8), pool.view(torch.uint8)
            old = s[name + "_scale"]
            old[block, :, at] = torch.where(live[:, None, None], scale, old[block, :, at])
        else:
            rows, raw = s[name], pool
        raw[block, :, at] = torch.where(live[:, None, None], rows, raw[block, :, at])
    return _written(s)


def _written(s):
    if not s["case"]["fp8"]:
        return dict(k=s["k_pool"], v=s["v_pool"])
    return dict(k=_dequantised(s["k_pool"], s["k_scale"]), v=_dequantised(s["v_pool"], s["v_scale"]),
                k_scale=s["k_scale"], v_scale=s["v_scale"])


def _plain_prompt(s):
    c, t, total = s["case"], s["q"].shape[0], sum(s["shape"]["kv"])
    rows = torch.arange(c["batch"], device="cuda")
    offsets, kv = s["offsets"].long(), s["kv_lens"].long()
    qlens = offsets[1:] - offsets[:-1]
    qrow = torch.repeat_interleave(rows, qlens, output_size=t)
    qpos = torch.arange(t, device="cuda") - offsets[qrow] + (kv - qlens)[qrow]
    krow = torch.repeat_interleave(rows, kv, output_size=total)
    kpos = torch.arange(total, device="cuda") - (torch.cumsum(kv, 0) - kv)[krow]
    block = s["table"][krow, kpos // PAGE].long()
    k = s["k_pool"][block, :, kpos % PAGE].float().transpose(0, 1)
    v = s["v_pool"][block, :, kpos % PAGE].float().transpose(0, 1)
    g = c["hq"] // c["hkv"]
    visible = (qrow[:, None] == krow) & (kpos <= qpos[:, None])
    q = s["q"].float().reshape(t, c["hkv"], g, c["d"]).permute(1, 2, 0, 3)
    out, lse = _attend(q, k[:, None], v[:, None], visible, 1.0 / math.sqrt(c["d"]))
    return dict(out=out.permute(2, 0, 1, 3).reshape(t, c["hq"], c["d"]).bfloat16(),
                lse=lse.permute(2, 0, 1).reshape(t, c["hq"]))


def _plain_prefix(s):
    c = s["case"]
    b, n, g, d = c["batch"], c["nodes"], c["hq"] // c["hkv"], c["d"]
    ctx = s["ctx"].long()
    at = torch.arange(s["shape"]["width"] * PAGE, device="cuda")
    block = s["table"][:, at // PAGE].long().clamp(min=0)
    k = s["k_pool"][block, :, at % PAGE].float().transpose(1, 2)
    v = s["v_pool"][block, :, at % PAGE].float().transpose(1, 2)
    node = at - ctx[:, None]
    draft = s["seen"][:, node.clamp(0, n - 1)].transpose(0, 1) & ((node >= 0) & (node < n))[:, None]
    visible = (node < 0)[:, None] | draft
    q = s["q"].float().view(b, n, c["hkv"], g, d).permute(0, 2, 3, 1, 4).reshape(b, c["hkv"], g * n, d)
    out, lse = _attend(q, k, v, visible[:, None].repeat(1, 1, g, 1), 1.0 / math.sqrt(d))
    return dict(out=out.view(b, c["hkv"], g, n, d).permute(0, 3, 1, 2, 4).reshape(b, n, c["hq"], d).bfloat16(),
                lse=lse.view(b, c["hkv"], g, n).permute(0, 3, 1, 2).reshape(b, n, c["hq"]))


def _plain_logits(s):
    c = s["case"]
    b, r, v = c["batch"], c["rows"], c["vocab"]
    x = s["logits"].float()
    at = torch.arange(c["hist"], device="cuda")
    word = s["history"].long()
    given = (at < s["prompt_lens"][:, None]).float()
    made = ((at >= s["prompt_lens"][:, None]) & (at < s["hist_lens"][:, None])).float()
    prompt = torch.zeros((b, v), device="cuda").scatter_add_(1, word, given)
    count = torch.zeros((b, v), device="cuda").scatter_add_(1, word, made)[:, None].repeat(1, r, 1)
    if r > 1:
        drafts = (s["drafts"][:, 1:] if c["tree"] else s["drafts"]).long()
        count.scatter_add_(2, drafts[:, None].repeat(1, r, 1), s["seen"].float().repeat(b, 1, 1))
    rep = s["repetition"][:, None, None]
    x = torch.where((count > 0) | (prompt > 0)[:, None], torch.where(x > 0, x / rep, x * rep), x)
    x = x - s["frequency"][:, None, None] * count
    x = x - torch.where(count > 0, s["presence"][:, None, None], 0.0)
    if c["bias"]:
        n = s["bias_tokens"].numel()
        row = torch.repeat_interleave(torch.arange(b, device="cuda"), s["bias_offsets"].diff().long(), output_size=n)
        bias = torch.zeros((b, v), device="cuda").index_put_((row, s["bias_tokens"].long()), s["bias_values"])
        x = x + bias[:, None]
    if c["mask"]:
        bit = s["mask"][:, :, :, None] >> torch.arange(32, dtype=torch.int32, device="cuda") & 1
        x = torch.where(bit.view(b, r, -1)[:, :, :v] != 0, x, -math.inf)
    return dict(logits=x)


# ------------------------------------------------------------------ the framework's calls
def _own(s):
    from speculative_verify_paged_attn_gb300 import svpa

    c = s["case"]
    if c["op"] == "tables":
        if "workspace" not in s:
            s["workspace"] = torch.zeros(svpa.block_table_build_workspace_size(c["batch"]), dtype=torch.uint8,
                                         device="cuda")
        s["after"].copy_(s["before"])
        svpa.block_table_build(s["lens"], s["table"], s["offsets"], s["slots"], s["after"][:-1], s["free_stack"],
                               s["after"][-1:], workspace=s["workspace"], error_flag=s["error"],
                               prefix_blocks=s["prefix"] if c["prefix"] else None)
        return dict(table=s["table"], offsets=s["offsets"], slots=s["slots"], counts_and_top=s["after"])
    if c["op"] == "write":
        svpa.kv_write(s["k"], s["v"], s["slots"], s["k_pool"], s["v_pool"], error_flag=s["error"],
                      k_scale=s["k_scale"], v_scale=s["v_scale"], scale_tile=64 if c["fp8"] else 0)
        return _written(s)
    if c["op"] == "prompt":
        if "params" not in s:
            s["params"] = svpa.prompt_params(c["batch"], s["q"].shape[0], c["hq"], c["hkv"], c["d"],
                                             s["table"].shape[1], s["k_pool"].shape[0], q_stride=s["q"].stride(0))
            s["workspace"] = torch.zeros(svpa.paged_prompt_attn_workspace_size(s["params"]), dtype=torch.uint8,
                                         device="cuda")
        svpa.paged_prompt_attn(s["params"], s["q"], s["k_pool"], s["v_pool"], s["table"], s["offsets"], s["kv_lens"],
                               s["out"], workspace=s["workspace"], error_flag=s["error"], lse=s["lse"])
        return dict(out=s["out"], lse=s["lse"])
    if c["op"] == "prefix":
        if "params" not in s:
            s["params"] = svpa.attn_params(c["batch"], c["nodes"], c["hq"], c["hkv"], c["d"], s["table"].shape[1],
                                           s["k_pool"].shape[0])
            s["workspace"] = torch.zeros(svpa.prefix_verify_attn_workspace_size(s["params"], c["prefix"]),
                                         dtype=torch.uint8, device="cuda")
        svpa.prefix_verify_attn(s["params"], s["q"], s["k_pool"], s["v_pool"], s["prefix"], s["table"], s["ctx"],
                                s["out"], workspace=s["workspace"], error_flag=s["error"],
                                ancestor_mask=s["ancestors"] if c["tree"] else None, lse=s["lse"])
        return dict(out=s["out"], lse=s["lse"])
    svpa.logits_process(s["logits"], s["out"], error_flag=s["error"], history=s["history"],
                        prompt_lens=s["prompt_lens"], hist_lens=s["hist_lens"], draft_tokens=s["drafts"],
                        parent=s["parent"], repetition=s["repetition"], presence=s["presence"],
                        frequency=s["frequency"], bias_offsets=s["bias_offsets"], bias_tokens=s["bias_tokens"],
                        bias_values=s["bias_values"], mask=s["mask"])
    return dict(logits=s["out"])


_PLAIN = dict(tables=_plain_tables, write=_plain_write, prompt=_plain_prompt, prefix=_plain_prefix,
              logits=_plain_logits)


def run(state):
    if own:
        return _own(state)
    return _PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------ the definition in 64 bits
def _exact_rows(q, k, v, visible, scale):
    """One sequence and one kv head: q [R, D], k and v [T, D], visible [R, T], a few hundred rows at a time."""
    outs, lses = [], []
    for at in range(0, q.shape[0], 512):
        x = (q[at:at + 512] @ k.T) * scale
        x[~visible[at:at + 512]] = -math.inf
        lse = torch.logsumexp(x, 1)
        outs.append(torch.exp(x - lse[:, None]) @ v)
        lses.append(lse)
    return torch.cat(outs), torch.cat(lses)


def _exact_attention(c, s, firsts, counts, positions, lens, masks=None):
    """Attention of query rows [firsts, firsts + counts) of each sequence over its first `lens` tokens."""
    q, g = s["q"].reshape(-1, c["hq"], c["d"]), c["hq"] // c["hkv"]
    out = torch.zeros((q.shape[0], c["hq"], c["d"]), dtype=torch.float64, device="cuda")
    lse = torch.zeros((q.shape[0], c["hq"]), dtype=torch.float64, device="cuda")
    for b, (first, count, total) in enumerate(zip(firsts, counts, lens)):
        if count == 0:
            continue
        ids = s["table"][b, :-(-total // PAGE)].long()
        pos = torch.arange(total, device="cuda")
        limit = torch.as_tensor(positions[b], device="cuda")
        visible = pos[None] <= limit[:, None] if masks is None else masks(b, pos)
        visible = visible.repeat_interleave(g, 0)
        for h in range(c["hkv"]):
            k = s["k_pool"][ids, h].reshape(-1, c["d"])[:total].double()
            v = s["v_pool"][ids, h].reshape(-1, c["d"])[:total].double()
            mine = q[first:first + count, h * g:(h + 1) * g].reshape(-1, c["d"]).double()
            o, l = _exact_rows(mine, k, v, visible, 1.0 / math.sqrt(c["d"]))
            out[first:first + count, h * g:(h + 1) * g] = o.view(count, g, c["d"])
            lse[first:first + count, h * g:(h + 1) * g] = l.view(count, g)
    return out, lse


def exact(c, seed):
    if c["op"] == "tables":
        return None  # whole numbers only
    s = prepare(c, seed)
    shape = s["shape"]
    if c["op"] == "write":
        done = {}
        slots = s["slots"].tolist()
        live = torch.tensor([i for i, x in enumerate(slots) if x >= 0], device="cuda")
        slot = s["slots"].long()[live]
        for name in ("k", "v"):
            rows = s[name].double()[live]
            pool = torch.zeros(s[name + "_pool"].shape, dtype=torch.float64, device="cuda")
            if c["fp8"]:
                # the stored scale is 32 bits wide, and the quotient is rounded to 32 bits before its 8-bit code
                tiles = rows.view(rows.shape[0], c["hkv"], -1, 64)
                big = tiles.abs().max(-1).values
                scale = torch.where(big == 0, 1.0, (big / torch.full_like(big, FP8_MAX)).float().double())
                codes = (tiles / scale[..., None]).float().to(torch.float8_e4m3fn).double()
                rows = (codes * scale[..., None]).view(rows.shape)
                scales = torch.ones(s[name + "_scale"].shape, dtype=torch.float64, device="cuda")
                flat = scales.transpose(1, 2).contiguous().view(-1, c["hkv"], c["d"] // 64)
                flat[slot] = scale
                done[name + "_scale"] = flat.view(-1, PAGE, c["hkv"], c["d"] // 64).transpose(1, 2)
            flat = pool.transpose(1, 2).contiguous().view(-1, c["hkv"], c["d"])
            flat[slot] = rows
            done[name] = flat.view(-1, PAGE, c["hkv"], c["d"]).transpose(1, 2)
        return done
    if c["op"] == "prompt":
        firsts = s["offsets"].tolist()[:-1]
        spots = [list(range(m - n, m)) for n, m in zip(shape["new"], shape["kv"])]
        out, lse = _exact_attention(c, s, firsts, shape["new"], spots, shape["kv"])
        return dict(out=out, lse=lse)
    if c["op"] == "prefix":
        n = c["nodes"]

        def masks(b, pos):
            rows = [[m >> i & 1 for i in range(n)] for m in s["ancestors"]]
            draft = torch.tensor(rows, dtype=torch.bool, device="cuda")
            return torch.cat([draft.new_ones((n, shape["ctx"][b])), draft], 1)

        out, lse = _exact_attention(c, s, [b * n for b in range(c["batch"])], [n] * c["batch"],
                                    [[0] * n] * c["batch"], [x + n for x in shape["ctx"]], masks)
        return dict(out=out.view(c["batch"], n, c["hq"], c["d"]), lse=lse.view(c["batch"], n, c["hq"]))
    out = s["logits"].double()
    masks = _ancestors(c["rows"], c["tree"])
    for b in range(c["batch"]):
        word = s["history"][b].long()
        prompt, hist = shape["prompt"][b], shape["hist"][b]
        given = torch.bincount(word[:prompt], minlength=c["vocab"]) > 0
        base = torch.bincount(word[prompt:hist], minlength=c["vocab"])
        rep, pres, freq = (s[x][b].double() for x in ("repetition", "presence", "frequency"))
        first = 1 if c["tree"] else 0
        for i in range(c["rows"]):
            path = [n for n in range(1, c["rows"]) if masks[i] >> n & 1]
            made = base + torch.bincount(s["drafts"][b].long()[[n - 1 + first for n in path]],
                                         minlength=c["vocab"]) if path else base
            x = out[b, i]
            seen = given | (made > 0)
            x = torch.where(seen & (x > 0), x / rep, torch.where(seen, x * rep, x))
            x = x - freq * made - pres * (made > 0)
            if c["bias"]:
                lo, hi = s["bias_offsets"][b], s["bias_offsets"][b + 1]
                x[s["bias_tokens"][lo:hi].long()] += s["bias_values"][lo:hi].double()
            if c["mask"]:
                words = s["mask"][b, i].long() & 0xFFFFFFFF
                allowed = (words[:, None] >> torch.arange(32, device="cuda") & 1).reshape(-1)[:c["vocab"]] > 0
                x = torch.where(allowed, x, -math.inf)
            out[b, i] = x
    return dict(logits=out)
