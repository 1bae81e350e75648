"""Cases and plain forms of the operators around a K/V cache held in 4 bits.

Five operators, in the order a serving program uses them:

  rotate  norms of queries and keys for each head, with the position rotation
  write   the same on the way into the pages of a prompt (bf16, FP8, 4 bits)
  append  a step's K/V rows into 4-bit pages behind each sequence's history
  attend  verification attention over 4-bit pages
  read    rows of 4-bit pages back as bf16

A 4-bit page holds, for each kv head, 16 rows of E2M1 codes (two a byte, the
even element low) and behind them one E4M3 scale for each 16 elements; a value
is code * scale * the head's fp32 factor.

``run`` computes an operator in elementary torch operations, or, where ``own``
is true, through the framework's own entry points.  Lengths follow from the
case alone, values from the seed.
"""
import math
import random

import torch

own = False

PAGE = 16
GROUP = 16
FP8_MAX = 448.0
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
EPS = 1e-6


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # the drafts of four sequences, between the projection and the append: latency
        dict(name="rotate-step", op="rotate", tokens=24, hq=64, hkv=8, d=128, rot=128, pairs=False, norm=True,
             fused=True),
        # a long prompt's queries and keys
        dict(name="rotate-prompt", op="rotate", tokens=8192, hq=64, hkv=8, d=128, rot=128, pairs=False, norm=True,
             fused=True),
        # one short prompt into 4-bit pages, some rows of the batch padding
        dict(name="write-fp4-short", op="write", tokens=57, hq=64, hkv=8, d=128, rot=128, pairs=False, norm=True,
             fused=True, pages="fp4", holes=3),
        # a long prefill batch into 4-bit pages
        dict(name="write-fp4-long", op="write", tokens=16384, hq=64, hkv=8, d=128, rot=128, pairs=False, norm=True,
             fused=True, pages="fp4", holes=0),
        # a few chat sequences and their four drafts: latency
        dict(name="append-few", op="append", batch=6, new=5, lo=3, hi=100, hkv=8, d=128),
        # a full batch of multi-head sequences
        dict(name="append-many", op="append", batch=256, new=8, lo=3, hi=200, hkv=32, d=128),
        # single-token decoding of a few short sequences: latency
        dict(name="attend-few", op="attend", batch=4, lo=200, hi=900, nodes=1, tree=False, hq=32, hkv=8, d=128),
        # multi-head verification of four drafts
        dict(name="attend-mha", op="attend", batch=32, lo=512, hi=4096, nodes=5, tree=False, hq=32, hkv=32, d=128),
        # grouped-query verification of five drafts over long histories
        dict(name="attend-long", op="attend", batch=64, lo=8192, hi=32768, nodes=6, tree=False, hq=64, hkv=8, d=128),
        # draft trees
        dict(name="attend-tree", op="attend", batch=64, lo=1024, hi=8192, nodes=29, tree=True, hq=32, hkv=8, d=128),
        # the cached part of a prompt that goes on in bf16 pages
        dict(name="read-short", op="read", tokens=700, hkv=8, d=128),
        # long cached prompts of a batch
        dict(name="read-long", op="read", tokens=65536, hkv=8, d=128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rotate", "write", "append", "attend", "attend", "read"))
    hkv, g = rng.choice(((8, 8), (8, 4), (32, 1), (2, 7), (4, 1), (1, 16)))
    d = rng.choice((64, 128, 128))
    if op in ("rotate", "write"):
        c = dict(op=op, tokens=_log(rng, 1, 8000), hq=hkv * g, hkv=hkv, d=d, rot=rng.choice((d, d, d // 2)),
                 pairs=rng.random() < 0.3, norm=rng.random() < 0.6, fused=rng.random() < 0.6)
        if op == "write":
            c.update(pages=rng.choice(("fp4", "fp4", "fp8", "bf16")), holes=rng.choice((0, 0, 5)))
        return c
    if op == "append":
        lo = rng.randrange(0, 40)
        return dict(op=op, batch=_log(rng, 1, 200), new=rng.randrange(1, 20), lo=lo, hi=lo + _log(rng, 1, 150),
                    hkv=hkv, d=d)
    if op == "read":
        return dict(op=op, tokens=_log(rng, 1, 60000), hkv=rng.choice((1, 2, 4, 8)), d=d)
    tree = rng.random() < 0.3
    nodes = min(128 // g, rng.randrange(2, 30) if tree else rng.choice((1, 1, 2, 3, 5, 6, 8)))
    batch = _log(rng, 1, 64)
    top = min(32768, 400000 // batch // hkv * 4)
    lo = _log(rng, 1, top)
    return dict(op=op, batch=batch, lo=lo, hi=lo + _log(rng, 1, top), nodes=nodes, tree=tree, hq=hkv * g, hkv=hkv, d=d)


def _lengths(count, lo, hi, salt):
    """`count` lengths in [lo, hi], the same for every seed."""
    rng = random.Random(salt * 7919 + count)
    return [rng.randint(lo, hi) for _ in range(count)]


def _ancestors(nodes, tree):
    """Bit i of entry j: node i is j or an ancestor of j.  A chain, or a tree in
    breadth-first order (four children of the root, then two of each node)."""
    parent = [-1] + list(range(nodes - 1))
    if tree:
        parent, at = [-1], 0
        while len(parent) < nodes:
            parent += [at] * min(4 if at == 0 else 2, nodes - len(parent))
            at += 1
    masks = []
    for j in range(nodes):
        masks.append((masks[parent[j]] if j else 0) | 1 << j)
    return masks


def _shape(c):
    """The case's lengths: what every function below derives its sizes from."""
    if c["op"] not in ("append", "attend"):
        return {}
    ctx = _lengths(c["batch"], c["lo"], c["hi"], 11)
    new = c["new"] if c["op"] == "append" else c["nodes"]
    pages = [-(-(n + new) // PAGE) for n in ctx]
    return dict(ctx=ctx, pages=pages, width=max(pages))


def _row_bytes(c, pages="fp4"):
    """Bytes of one token's row of one kv head in the pages."""
    return c["d"] * 9 // 16 if pages == "fp4" else c["d"] + c["d"] // 16 if pages == "fp8" else 2 * c["d"]


def work(c):
    d = c["d"]
    if c["op"] == "rotate":
        return dict(bytes=c["tokens"] * (2 * 2 * d * (c["hq"] + c["hkv"]) + 4 + 4 * c["rot"]), flops=0)
    if c["op"] == "write":
        return dict(bytes=c["tokens"] * (2 * 2 * d * c["hq"] + 2 * c["hkv"] * (2 * d + _row_bytes(c, c["pages"]))
                                         + 8 + 4 * c["rot"]), flops=0)
    if c["op"] == "append":
        rows = c["batch"] * c["new"] * c["hkv"]
        return dict(bytes=2 * rows * (2 * d + _row_bytes(c)) + 4 * c["batch"] * 2, flops=0)
    if c["op"] == "read":
        return dict(bytes=2 * c["tokens"] * c["hkv"] * (2 * d + _row_bytes(c)) + 4 * c["tokens"], flops=0)
    s = _shape(c)
    seen = sum(bin(m).count("1") for m in _ancestors(c["nodes"], c["tree"]))
    pairs = sum(n * c["nodes"] + seen for n in s["ctx"])
    t = c["batch"] * c["nodes"]
    tokens = sum(n + c["nodes"] for n in s["ctx"])
    return dict(bytes=2 * 2 * t * c["hq"] * d + 4 * t * c["hq"] + 2 * tokens * c["hkv"] * _row_bytes(c)
                + 4 * sum(s["pages"]), flops=4 * d * c["hq"] * pairs)


# ------------------------------------------------------------------ 4-bit rows
def _encode(x, factor):
    """Rows x [..., H, D] as packed codes [..., H, D / 2] and E4M3 scale bytes [..., H, D / 16]; factor [H]."""
    x = x.float()
    tiles = x.view(*x.shape[:-1], -1, GROUP)
    f = factor[:, None]
    scale = (tiles.abs().amax(-1) / (6.0 * f)).clamp(max=FP8_MAX).to(torch.float8_e4m3fn)
    step = (scale.float() * f)[..., None]
    y = torch.where(step > 0, tiles / torch.where(step > 0, step, 1.0), 0.0)
    a = y.abs()
    # the borders between neighbouring values; a tie goes to the even code
    code = (a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)
    code = (code | (y < 0).to(torch.uint8) << 3).view(x.shape)
    return code[..., 0::2] | code[..., 1::2] << 4, scale.view(torch.uint8)


def _decode(rows, factor, d):
    """Values [..., H, D] of rows [..., H, 9 D / 16] of codes and scale bytes."""
    codes, scale = rows[..., :d // 2], rows[..., d // 2:]
    code = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    value = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=rows.device)[code.int()]
    step = scale.contiguous().view(torch.float8_e4m3fn).float() * factor[:, None]
    return (value.view(*value.shape[:-1], -1, GROUP) * step[..., None]).view(value.shape)


def _to_pages(rows, d):
    """Rows [P, 16, H, 9 D / 16] as pages [P, H, 16 * 9 D / 16]: a head's codes, then its scales."""
    x = rows.transpose(1, 2)
    return torch.cat((x[..., :d // 2].flatten(2), x[..., d // 2:].flatten(2)), -1).contiguous()


def _from_pages(pages, d):
    """The rows [P, 16, H, 9 D / 16] of pages."""
    codes, scale = pages[..., :PAGE * d // 2], pages[..., PAGE * d // 2:]
    x = torch.cat((codes.unflatten(-1, (PAGE, d // 2)), scale.unflatten(-1, (PAGE, d // 16))), -1)
    return x.transpose(1, 2)


# ------------------------------------------------------------------ the inputs
def _random_pages(total, c, factor, gen):
    """Pages of keys or values as a model makes them: some channels wider than others."""
    out = torch.empty((total, c["hkv"], PAGE * _row_bytes(c)), dtype=torch.uint8, device="cuda")
    width = torch.empty((c["hkv"], c["d"]), device="cuda").normal_(0.0, 0.5, generator=gen).exp_()
    for at in range(0, total, 8192):
        n = min(8192, total - at)
        x = torch.empty((n, PAGE, c["hkv"], c["d"]), device="cuda").normal_(generator=gen) * width
        codes, scale = _encode(x.bfloat16(), factor)
        out[at:at + n] = _to_pages(torch.cat((codes, scale), -1), c["d"])
    return out


def _table(pages, width, ids):
    """Rows of block ids, taken in turn, -1 behind."""
    pages = torch.tensor(pages, device="cuda")
    at = torch.arange(width, device="cuda")
    start = torch.cumsum(pages, 0) - pages
    live = at < pages[:, None]
    return torch.where(live, ids[torch.where(live, start[:, None] + at, 0)], -1).to(torch.int32)


def _projection(c, gen, heads):
    """Rows of several groups of heads; slices of one fused projection where `fused`."""
    t, d = c["tokens"], c["d"]
    if c["fused"]:
        x = torch.empty((t, sum(heads), d), dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
        return x.split(heads, 1)
    return [torch.empty((t, n, d), dtype=torch.bfloat16, device="cuda").normal_(generator=gen) for n in heads]


def prepare(c, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s, dev, d = _shape(c), "cuda", c["d"]
    state = dict(case=c, shape=s, error=torch.zeros(1, dtype=torch.int32, device=dev))

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    for name in ("k_factor", "v_factor"):
        # a head's largest value over 6 * 448, as it is calibrated
        state[name] = (4.0 + 4.0 * torch.rand(c["hkv"], generator=gen, device=dev)) / (6.0 * FP8_MAX)
    if c["op"] in ("rotate", "write"):
        t, far = c["tokens"], 40000
        q, k, v = _projection(c, gen, [c["hq"], c["hkv"], c["hkv"]])
        angle = torch.arange(far, device=dev, dtype=torch.float64)[:, None] * 10000.0 ** (
            -torch.arange(0, c["rot"], 2, device=dev, dtype=torch.float64) / c["rot"])
        state.update(q=q, k=k, v=v, table=torch.cat((angle.cos(), angle.sin()), 1).float(),
                     # two prompts, the second behind cached tokens
                     positions=((torch.arange(t, device=dev) + (torch.arange(t, device=dev) > t // 3) * 20011) % far)
                     .to(torch.int32),
                     q_out=torch.empty((t, c["hq"], d), dtype=torch.bfloat16, device=dev))
        for name in ("q_weight", "k_weight"):
            state[name] = (1.0 + 0.2 * torch.randn(d, generator=gen, device=dev)).bfloat16() if c["norm"] else None
    if c["op"] == "rotate":
        state["k_out"] = torch.empty((c["tokens"], c["hkv"], d), dtype=torch.bfloat16, device=dev)
    elif c["op"] == "write":
        total = -(-c["tokens"] // PAGE) + 2
        ids = torch.randperm(total - 1, generator=gen, device=dev)
        at = torch.arange(c["tokens"], device=dev)
        slots = (ids[at // PAGE] * PAGE + at % PAGE).to(torch.int32)
        for i in range(min(c["holes"], c["tokens"] // 2)):  # padding rows of the batch
            slots[2 * i + 1] = -1
        state.update(slots=slots)
        state["q_out"].zero_()
        _empty_pages(state, total)
    elif c["op"] == "append":
        total = sum(s["pages"]) + 3
        state.update(new_k=torch.empty((c["batch"], c["new"], c["hkv"], d), dtype=torch.bfloat16, device=dev)
                     .normal_(generator=gen),
                     new_v=torch.empty((c["batch"], c["new"], c["hkv"], d), dtype=torch.bfloat16, device=dev)
                     .normal_(generator=gen),
                     ctx=ints(s["ctx"]), blocks=_table(s["pages"], s["width"],
                                                       torch.randperm(total, generator=gen, device=dev)),
                     # every page of the step is mapped already
                     counts=torch.ones(total, dtype=torch.int32, device=dev),
                     free=torch.full((total,), -1, dtype=torch.int32, device=dev), top=ints([0]))
        for name in ("k", "v"):
            state[name + "_pool"] = _random_pages(total, c, state[name + "_factor"], gen)
            state[name + "_rows"] = torch.empty((total * PAGE, c["hkv"], d), dtype=torch.bfloat16, device=dev)
        state["all_slots"] = torch.arange(total * PAGE, dtype=torch.int32, device=dev)
    elif c["op"] == "read":
        total = -(-c["tokens"] // PAGE) + 2
        at = torch.arange(c["tokens"], device=dev)
        ids = torch.randperm(total, generator=gen, device=dev)
        state["slots"] = (ids[at // PAGE] * PAGE + at % PAGE).to(torch.int32)
        for name in ("k", "v"):
            state[name + "_pool"] = _random_pages(total, c, state[name + "_factor"], gen)
            state[name + "_rows"] = torch.empty((c["tokens"], c["hkv"], d), dtype=torch.bfloat16, device=dev)
    elif c["op"] == "attend":
        total = sum(s["pages"]) + 5
        for name in ("k", "v"):
            state[name + "_pool"] = _random_pages(total, c, state[name + "_factor"], gen)
        q = torch.empty((c["batch"], c["nodes"], c["hq"], d), dtype=torch.bfloat16, device=dev).normal_(generator=gen)
        anc = _ancestors(c["nodes"], c["tree"])
        state.update(q=q, ctx=ints(s["ctx"]), ancestors=anc,
                     blocks=_table(s["pages"], s["width"], torch.randperm(total, generator=gen, device=dev)),
                     seen=torch.tensor([[m >> i & 1 for i in range(c["nodes"])] for m in anc], dtype=torch.bool,
                                       device=dev),
                     out=torch.empty_like(q), lse=torch.empty(q.shape[:3], device=dev))
    return state


def _empty_pages(s, total):
    """Zeroed pages of the case's kind, and where their rows are read back to."""
    c, d = s["case"], s["case"]["d"]
    for name in ("k", "v"):
        shape = (total, c["hkv"], PAGE * _row_bytes(c)) if c["pages"] == "fp4" else (total, c["hkv"], PAGE, d)
        kind = torch.bfloat16 if c["pages"] == "bf16" else torch.uint8
        s[name + "_pool"] = torch.zeros(shape, dtype=kind, device="cuda")
        s[name + "_scale"] = torch.ones((total, c["hkv"], PAGE, d // 64), device="cuda") if c["pages"] == "fp8" else None
        s[name + "_rows"] = torch.empty((total * PAGE, c["hkv"], d), dtype=torch.bfloat16, device="cuda")
    s["all_slots"] = torch.arange(total * PAGE, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ the plain forms
def _rotated(x, weight, s):
    """Rows x [T, H, D] normed for each head (with a weight) and rotated at their positions, in 32 bits."""
    c = s["case"]
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.float()
    r = c["rot"]
    at = s["table"][s["positions"].long()][:, None]
    cos, sin = at[..., :r // 2], at[..., r // 2:]
    if c["pairs"]:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((turned, x[..., r:]), -1).bfloat16()


def _plain_rotate(s):
    return dict(q=_rotated(s["q"], s["q_weight"], s), k=_rotated(s["k"], s["k_weight"], s))


def _plain_write(s):
    c, d = s["case"], s["case"]["d"]
    live = s["slots"] >= 0
    out = dict(q=torch.where(live[:, None, None], _rotated(s["q"], s["q_weight"], s), 0.0))
    # a padding row writes what the pool's last, free slot holds back to it
    total = s["k_pool"].shape[0]
    slot = torch.where(live, s["slots"], total * PAGE - 1).long()
    block, at, keep = slot // PAGE, slot % PAGE, live[:, None, None]
    for name, rows in (("k", _rotated(s["k"], s["k_weight"], s)), ("v", s["v"])):
        pool = s[name + "_pool"]
        if c["pages"] == "bf16":
            pool[block, :, at] = torch.where(keep, rows, pool[block, :, at])
            out[name] = pool
        elif c["pages"] == "fp8":
            x = rows.float().reshape(c["tokens"], c["hkv"], d // 64, 64)
            amax = x.abs().amax(-1)
            scale = torch.where(amax > 0, amax / torch.full_like(amax, FP8_MAX), 1.0)
            codes = (x / scale[..., None]).view(rows.shape).to(torch.float8_e4m3fn).view(torch.uint8)
            pool[block, :, at] = torch.where(keep, codes, pool[block, :, at])
            held = s[name + "_scale"]
            held[block, :, at] = torch.where(keep, scale, held[block, :, at])
            value = pool.view(torch.float8_e4m3fn).float().view(*pool.shape[:-1], -1, 64) * held[..., None]
            out[name] = value.view(pool.shape).transpose(1, 2).reshape(total * PAGE, c["hkv"], d).bfloat16()
        else:
            new = torch.cat(_encode(rows, s[name + "_factor"]), -1)
            held = _from_pages(pool, d).contiguous()
            held[block, at] = torch.where(keep, new, held[block, at])
            pool.copy_(_to_pages(held, d))
            out[name] = _decode(held.flatten(0, 1), s[name + "_factor"], d).bfloat16()
    return out


def _plain_append(s):
    c, d = s["case"], s["case"]["d"]
    pos = s["ctx"].long()[:, None] + torch.arange(c["new"], device="cuda")
    block, at = s["blocks"].long().gather(1, pos // PAGE), pos % PAGE
    out = {}
    for name in ("k", "v"):
        held = _from_pages(s[name + "_pool"], d).contiguous()
        held[block, at] = torch.cat(_encode(s["new_" + name], s[name + "_factor"]), -1)
        s[name + "_pool"].copy_(_to_pages(held, d))
        out[name] = _decode(held.flatten(0, 1), s[name + "_factor"], d).bfloat16()
    return out


def _plain_read(s):
    c, d = s["case"], s["case"]["d"]
    slot = s["slots"].long()
    return {name: _decode(_from_pages(s[name + "_pool"], d)[slot // PAGE, slot % PAGE], s[name + "_factor"], d).bfloat16()
            for name in ("k", "v")}


def _plain_attend(s):
    c = s["case"]
    b, n, g, d = c["batch"], c["nodes"], c["hq"] // c["hkv"], c["d"]
    ctx = s["ctx"].long()
    at = torch.arange(s["shape"]["width"] * PAGE, device="cuda")
    pages = s["blocks"].long().clamp(min=0)
    k, v = (_decode(_from_pages(s[x + "_pool"][pages.flatten()], d), s[x + "_factor"], d)
            .view(b, at.numel(), c["hkv"], d).transpose(1, 2) for x in ("k", "v"))
    node = at - ctx[:, None]
    draft = s["seen"][:, node.clamp(0, n - 1)].transpose(0, 1) & ((node >= 0) & (node < n))[:, None]
    visible = ((node < 0)[:, None] | draft)[:, None].repeat(1, 1, g, 1)
    q = s["q"].float().view(b, n, c["hkv"], g, d).permute(0, 2, 3, 1, 4).reshape(b, c["hkv"], g * n, d)
    x = torch.matmul(q, k.transpose(-1, -2)).mul_(1.0 / math.sqrt(d)).masked_fill_(~visible, -math.inf)
    top = x.amax(-1, keepdim=True)
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    out, lse = torch.matmul(x, v) / total, (top + total.log()).squeeze(-1)
    return dict(out=out.view(b, c["hkv"], g, n, d).permute(0, 3, 1, 2, 4).reshape(b, n, c["hq"], d).bfloat16(),
                lse=lse.view(b, c["hkv"], g, n).permute(0, 3, 1, 2).reshape(b, n, c["hq"]))


# ------------------------------------------------------------------ the framework's calls
def _own(s):
    from speculative_verify_paged_attn_gb300 import svpa

    c, err = s["case"], s["error"]
    if c["op"] == "rotate":
        svpa.qk_norm_rope(s["q"], s["k"], s["positions"], s["table"], s["q_out"], s["k_out"], error_flag=err,
                          q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS, interleaved=c["pairs"])
        return dict(q=s["q_out"], k=s["k_out"])
    if c["op"] == "write":
        factors = dict(k_factor=s["k_factor"], v_factor=s["v_factor"]) if c["pages"] == "fp4" else {}
        scales = dict(k_scale=s["k_scale"], v_scale=s["v_scale"], scale_tile=64) if c["pages"] == "fp8" else {}
        svpa.rope_kv_write(s["k"], s["v"], s["positions"], s["slots"], s["table"], s["k_pool"], s["v_pool"],
                           error_flag=err, q=s["q"], q_out=s["q_out"], q_weight=s["q_weight"],
                           k_weight=s["k_weight"], eps=EPS, interleaved=c["pairs"], fp4=c["pages"] == "fp4",
                           **factors, **scales)
        if c["pages"] == "bf16":
            return dict(q=s["q_out"], k=s["k_pool"], v=s["v_pool"])
        svpa.kv_read(s["all_slots"], s["k_pool"], s["v_pool"], s["k_rows"], s["v_rows"], error_flag=err,
                     fp4=c["pages"] == "fp4", **factors, **scales)
        return dict(q=s["q_out"], k=s["k_rows"], v=s["v_rows"])
    if c["op"] == "append":
        svpa.kv_append_fp4(s["new_k"], s["new_v"], s["blocks"], s["ctx"], s["counts"], s["free"], s["top"],
                           s["k_pool"], s["v_pool"], error_flag=err, k_factor=s["k_factor"], v_factor=s["v_factor"])
        svpa.kv_read(s["all_slots"], s["k_pool"], s["v_pool"], s["k_rows"], s["v_rows"], error_flag=err, fp4=True,
                     k_factor=s["k_factor"], v_factor=s["v_factor"])
        return dict(k=s["k_rows"], v=s["v_rows"])
    if c["op"] == "read":
        svpa.kv_read(s["slots"], s["k_pool"], s["v_pool"], s["k_rows"], s["v_rows"], error_flag=err, fp4=True,
                     k_factor=s["k_factor"], v_factor=s["v_factor"])
        return dict(k=s["k_rows"], v=s["v_rows"])
    if "params" not in s:
        s["params"] = svpa.attn_params(c["batch"], c["nodes"], c["hq"], c["hkv"], c["d"], s["blocks"].shape[1],
                                       s["k_pool"].shape[0], kv_fp4=True)
        s["workspace"] = torch.zeros(svpa.paged_verify_attn_fp4_workspace_size(s["params"]), dtype=torch.uint8,
                                     device="cuda")
    svpa.paged_verify_attn_fp4(s["params"], s["q"], s["k_pool"], s["v_pool"], s["blocks"], s["ctx"], s["out"],
                               workspace=s["workspace"], error_flag=err, k_factor=s["k_factor"],
                               v_factor=s["v_factor"], ancestor_mask=s["ancestors"] if c["tree"] else None,
                               lse=s["lse"])
    return dict(out=s["out"], lse=s["lse"])


_PLAIN = dict(rotate=_plain_rotate, write=_plain_write, append=_plain_append, read=_plain_read, attend=_plain_attend)


def run(state):
    if own:
        return _own(state)
    return _PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------ the definition in 64 bits
def _exact_turn(x, weight, c, s):
    """Normed and rotated rows: the pair (a, b) as the complex number a + i b times the position's unit number."""
    x = x.double()
    if weight is not None:
        x = x / ((x ** 2).sum(-1, keepdim=True) / c["d"] + EPS).sqrt() * weight.double()
    r = c["rot"]
    turn = s["table"].double()[s["positions"].long()]
    turn = torch.complex(turn[:, :r // 2], turn[:, r // 2:])[:, None]
    head = x[..., :r]
    pair = head.unflatten(-1, (r // 2, 2)) if c["pairs"] else head.unflatten(-1, (2, r // 2)).transpose(-1, -2)
    z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn)
    z = z if c["pairs"] else z.transpose(-1, -2)
    return torch.cat((z.flatten(-2), x[..., r:]), -1)


def _exact_fp4(rows, factor):
    """The values that 4-bit rows [T, H, D] stand for.  Scales and quotients are
    32 and 8 bits wide by definition; the nearest of the 15 values is searched for."""
    level = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
    done = torch.empty(rows.shape, dtype=torch.float64, device="cuda")
    for h in range(rows.shape[1]):
        f = factor[h]
        x = rows[:, h].double().view(rows.shape[0], -1, GROUP)
        top = (x.abs().max(-1).values.float() / (6.0 * f)).clamp(max=FP8_MAX)
        code = top.to(torch.float8_e4m3fn).float()
        step = (code * f).double()[..., None]
        size = (x.abs() / torch.where(step == 0, 1.0, step)).float().double()
        gap = (size[..., None] - level).abs()
        near = gap.min(-1, keepdim=True).values == gap
        even = torch.tensor([1, 0] * 4, dtype=torch.bool, device="cuda")
        pick = torch.where((near & even).any(-1, keepdim=True), near & even, near).int().argmax(-1)
        value = level[pick] * code.double()[..., None] * f.double() * x.sign()
        done[:, h] = torch.where(step == 0, 0.0, value).view(rows.shape[0], -1)
    return done


def _exact_rows(pool, factor, d, page, at):
    """Rows [R, H, D] in 64 bits out of 4-bit pages, a code at a time by its position in the page."""
    level = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
    el = torch.arange(d, device="cuda")
    byte = pool[page[:, None, None], torch.arange(pool.shape[1], device="cuda")[:, None],
                (at * (d // 2))[:, None, None] + el // 2].int()
    code = byte >> 4 * (el % 2) & 15
    raw = pool[page[:, None, None], torch.arange(pool.shape[1], device="cuda")[:, None],
               (PAGE * d // 2 + at * (d // 16))[:, None, None] + el // GROUP].int()
    # E4M3: 2^(e - 7) (1 + m / 8), below the smallest normal value 2^-6 m / 8
    e, m = raw >> 3, (raw & 7).double()
    scale = torch.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * torch.exp2(e.double() - 7))
    return torch.where(code >= 8, -1.0, 1.0) * level[(code & 7).long()] * scale * factor.double()[:, None]


def exact(c, seed):
    s = prepare(c, seed)
    d = c["d"]
    if c["op"] == "rotate":
        return dict(q=_exact_turn(s["q"], s["q_weight"], c, s), k=_exact_turn(s["k"], s["k_weight"], c, s))
    if c["op"] == "write":
        live = (s["slots"] >= 0).nonzero()[:, 0]
        slot = s["slots"].long()[live]
        q = _exact_turn(s["q"], s["q_weight"], c, s)
        q[s["slots"] < 0] = 0.0
        done = dict(q=q)
        for name, rows in (("k", _exact_turn(s["k"], s["k_weight"], c, s)), ("v", s["v"].double())):
            rows = rows[live].bfloat16().double()  # what a page takes is bf16
            if c["pages"] == "fp4":
                rows = _exact_fp4(rows, s[name + "_factor"])
            elif c["pages"] == "fp8":
                tiles = rows.view(rows.shape[0], c["hkv"], -1, 64)
                big = tiles.abs().max(-1).values
                scale = torch.where(big == 0, 1.0, (big / torch.full_like(big, FP8_MAX)).float().double())[..., None]
                rows = ((tiles / scale).float().to(torch.float8_e4m3fn).double() * scale).view(rows.shape)
            flat = torch.zeros((s["k_pool"].shape[0] * PAGE, c["hkv"], d), dtype=torch.float64, device="cuda")
            flat[slot] = rows
            done[name] = flat.view(-1, PAGE, c["hkv"], d).transpose(1, 2) if c["pages"] == "bf16" else flat
        return done
    if c["op"] == "append":
        done = {}
        every = s["all_slots"].long()
        for name in ("k", "v"):
            rows = torch.cat([_exact_rows(s[name + "_pool"], s[name + "_factor"], d, x // PAGE, x % PAGE)
                              for x in every.split(8192)])
            table = s["blocks"].tolist()
            slot = [table[b][p // PAGE] * PAGE + p % PAGE for b, n in enumerate(s["shape"]["ctx"])
                    for p in range(n, n + c["new"])]
            rows[slot] = _exact_fp4(s["new_" + name].flatten(0, 1), s[name + "_factor"])
            done[name] = rows
        return done
    if c["op"] == "read":
        return {name: torch.cat([_exact_rows(s[name + "_pool"], s[name + "_factor"], d, x // PAGE, x % PAGE)
                                 for x in s["slots"].long().split(8192)]) for name in ("k", "v")}
    n, g = c["nodes"], c["hq"] // c["hkv"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(s["q"].shape[:3], dtype=torch.float64, device="cuda")
    for b, ctx in enumerate(s["shape"]["ctx"]):
        pos = torch.arange(ctx + n, device="cuda")
        page = s["blocks"][b].long()[pos // PAGE]
        k, v = (torch.cat([_exact_rows(s[x + "_pool"], s[x + "_factor"], d, p, a)
                           for p, a in zip(page.split(8192), (pos % PAGE).split(8192))]) for x in ("k", "v"))
        visible = torch.cat([s["seen"].new_ones((n, ctx)), s["seen"]], 1).repeat_interleave(g, 0)
        for h in range(c["hkv"]):
            mine = s["q"][b, :, h * g:(h + 1) * g].reshape(n * g, d).double()
            x = mine @ k[:, h].T / math.sqrt(d)
            x[~visible] = -math.inf
            norm = torch.logsumexp(x, 1)
            out[b, :, h * g:(h + 1) * g] = (torch.exp(x - norm[:, None]) @ v[:, h]).view(n, g, d)
            lse[b, :, h * g:(h + 1) * g] = norm.view(n, g)
    return dict(out=out, lse=lse)
