"""Requests over a 4-bit cache, from admission to the step after the first
commit: block tables and slot maps, the prompts' norms and rotation on the way
into the pages, the prompts' rows read back for their attention, the drafts'
norms, rotation and append, verification, sampler and commit (a chain or a
tree), and a single token over what the commit left; eagerly, on a stream of
its own and as one replayed CUDA graph."""
import math

import pytest
import torch

import fp4_ref as F
import packed_ref as R
from speculative_verify_paged_attn_gb300 import svpa

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BS = 16
BF = torch.bfloat16


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


class Flow:
    def __init__(self, lens, parent, hq=8, hkv=2, d=128, rot=128, interleaved=False, vocab=900, seed=3):
        g = R.gen(seed, DEV)
        self.lens, self.hq, self.hkv, self.d, self.v, self.b = lens, hq, hkv, d, vocab, len(lens)
        self.parent, self.interleaved = parent, interleaved
        self.nq = len(parent)
        depth = [0]
        for p in parent[1:]:
            depth.append(depth[p] + 1)
        self.depth = depth
        self.chain = parent == list(range(-1, self.nq - 1))
        masks = [1]
        for j in range(1, self.nq):
            masks.append(masks[parent[j]] | 1 << j)
        self.masks = masks
        inner = sorted(set(parent[1:]))
        self.t = sum(lens)
        self.width = -(-(max(lens) + self.nq + 1) // BS)
        self.blocks = sum(-(-(n + self.nq + 1) // BS) for n in lens) + 4

        def bf(*s):
            return torch.randn(s, generator=g, device=DEV).to(BF)

        far = max(lens) + self.nq + 2
        angle = torch.arange(far, dtype=torch.float64, device=DEV)[:, None] * 10000.0 ** (
            -torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot)
        self.cs = torch.cat([angle.cos(), angle.sin()], 1).float()
        self.qw, self.kw = (1 + bf(d) / 4).to(BF), (1 + bf(d) / 4).to(BF)
        self.kf, self.vf = [0.5 + torch.rand(hkv, generator=g, device=DEV) for _ in range(2)]
        heads = hq + 2 * hkv
        split = [hq, hkv, hkv]
        # slices of fused projections: the prompts', the drafts' and the next tokens'
        self.prompt = bf(self.t, heads, d).split(split, 1)
        self.drafts = bf(self.b * self.nq, heads, d).split(split, 1)
        self.last = bf(self.b, heads, d).split(split, 1)
        self.pos = ints([i for n in lens for i in range(n)])
        self.dpos = ints([n + x for n in lens for x in depth])
        self.target = torch.randn((self.b, self.nq, vocab), generator=g, device=DEV) * 2
        self.draft = (self.target[:, inner] + 0.3 * torch.randn((self.b, len(inner), vocab), generator=g, device=DEV))
        self.tokens = torch.randint(0, vocab, (self.b, self.nq), generator=g, device=DEV).to(torch.int32)
        for j in range(1, self.nq):  # likely drafts
            self.tokens[:, j] = self.draft[:, inner.index(parent[j])].topk(j, 1).indices[:, -1]
        self.ua = torch.rand((self.b, self.nq), generator=g, device=DEV)
        self.us = torch.rand((self.b,), generator=g, device=DEV)
        self.ctokens, self.cua = self.tokens[:, 1:].contiguous(), self.ua[:, 1:].contiguous()

        self.free0 = torch.randperm(self.blocks, generator=g, device=DEV).to(torch.int32)
        self.table, self.count = ints([[-3] * self.width] * self.b), ints([0] * self.blocks)
        self.free, self.top, self.err = self.free0.clone(), ints([self.blocks]), ints([0])
        self.seq, self.cl = ints(lens), ints(lens)
        # scale bytes that are not numbers where nothing is written
        self.kp = torch.full((self.blocks, hkv, 9 * d), 0xff, dtype=torch.uint8, device=DEV)
        self.vp = self.kp.clone()
        self.kb, self.vb = [torch.full((self.blocks, hkv, BS, d), float("nan"), dtype=BF, device=DEV) for _ in range(2)]
        self.cu, self.slots = ints([0] * (self.b + 1)), ints([0] * self.t)
        self.q0, self.q1, self.q2 = [torch.zeros((x[0].shape[0], hq, d), dtype=BF, device=DEV)
                                     for x in (self.prompt, self.drafts, self.last)]
        self.k1, self.k2 = [torch.zeros((x[1].shape[0], hkv, d), dtype=BF, device=DEV)
                            for x in (self.drafts, self.last)]
        self.kr, self.vr = [torch.zeros((self.t, hkv, d), dtype=BF, device=DEV) for _ in range(2)]
        self.v1, self.v2 = self.drafts[2].contiguous(), self.last[2].contiguous()
        self.o0, self.o1, self.o2 = [torch.zeros_like(x) for x in (self.q0, self.q1, self.q2)]
        self.l0, self.l1, self.l2 = [torch.zeros(x.shape[:2], device=DEV) for x in (self.q0, self.q1, self.q2)]
        self.accepted, self.path = ints([0] * self.b), ints([[-1] * (max(depth) + 1)] * self.b)
        self.emitted = ints([[-1] * (max(depth) + 1)] * self.b)
        self.pp = svpa.prompt_params(self.b, self.t, hq, hkv, d, self.width, self.blocks)
        self.a1 = svpa.attn_params(self.b, self.nq, hq, hkv, d, self.width, self.blocks, kv_fp4=True)
        self.a2 = svpa.attn_params(self.b, 1, hq, hkv, d, self.width, self.blocks, kv_fp4=True)
        # one zeroed buffer for all of them in turn
        self.ws = torch.zeros(max(svpa.block_table_build_workspace_size(self.b),
                                  svpa.paged_prompt_attn_workspace_size(self.pp),
                                  svpa.paged_verify_attn_fp4_workspace_size(self.a1)), dtype=torch.uint8, device=DEV)
        self.sws = torch.zeros(svpa.spec_accept_logits_workspace_size(self.b, max(self.nq - 1, 1), vocab),
                               dtype=torch.uint8, device=DEV)

    def restore(self):
        self.table.fill_(-3)
        self.count.zero_()
        self.free.copy_(self.free0)
        self.top.fill_(self.blocks)
        self.cl.copy_(self.seq)
        for t in (self.kp, self.vp):
            t.fill_(0xff)
        for t in (self.kb, self.vb, self.o0, self.o1, self.o2):
            t.fill_(float("nan"))

    def run(self, stream=None):
        e = dict(error_flag=self.err, stream=stream)
        norm = dict(q_weight=self.qw, k_weight=self.kw, eps=1e-6, interleaved=self.interleaved)
        f = dict(k_factor=self.kf, v_factor=self.vf)
        pages = (self.table, self.cl, self.count, self.free, self.top, self.kp, self.vp)
        svpa.block_table_build(self.seq, self.table, self.cu, self.slots, self.count, self.free, self.top,
                               workspace=self.ws, **e)
        q, k, v = self.prompt
        svpa.rope_kv_write(k, v, self.pos, self.slots, self.cs, self.kp, self.vp, q=q, q_out=self.q0, fp4=True, **norm,
                           **f, **e)
        svpa.kv_read(self.slots, self.kp, self.vp, self.kr, self.vr, fp4=True, **f, **e)
        svpa.kv_write(self.kr, self.vr, self.slots, self.kb, self.vb, **e)
        svpa.paged_prompt_attn(self.pp, self.q0, self.kb, self.vb, self.table, self.cu, self.seq, self.o0,
                               workspace=self.ws, lse=self.l0, **e)
        q, k, v = self.drafts
        svpa.qk_norm_rope(q, k, self.dpos, self.cs, self.q1, self.k1, **norm, **e)
        four = (self.b, self.nq, self.hkv, self.d)
        svpa.kv_append_fp4(self.k1.view(four), self.v1.view(four), *pages, **f, **e)
        svpa.paged_verify_attn_fp4(self.a1, self.q1, self.kp, self.vp, self.table, self.cl, self.o1, workspace=self.ws,
                                   ancestor_mask=None if self.chain else self.masks, lse=self.l1, **f, **e)
        commit = (self.nq, self.table, self.cl, self.accepted, self.count, self.free, self.top)
        if self.chain:
            svpa.spec_accept_logits(self.target, self.draft, self.ctokens, self.cua, self.us, self.accepted,
                                    self.emitted, workspace=self.sws, **e)
            svpa.block_table_commit(*commit, kv_fp4=True, **e)
        else:
            svpa.spec_accept_tree_logits(self.parent, self.target, self.draft, self.tokens, self.ua, self.us,
                                         self.accepted, self.path, self.emitted, **e)
            svpa.block_table_commit(*commit, path_nodes=self.path, k_pool=self.kp, v_pool=self.vp,
                                    num_kv_heads=self.hkv, head_dim=self.d, kv_fp4=True, **e)
        q, k, v = self.last
        svpa.qk_norm_rope(q, k, self.cl, self.cs, self.q2, self.k2, **norm, **e)
        four = (self.b, 1, self.hkv, self.d)
        svpa.kv_append_fp4(self.k2.view(four), self.v2.view(four), *pages, **f, **e)
        svpa.paged_verify_attn_fp4(self.a2, self.q2, self.kp, self.vp, self.table, self.cl, self.o2, workspace=self.ws,
                                   lse=self.l2, **f, **e)

    def results(self):
        return [t.clone() for t in (self.q0, self.o0, self.l0, self.o1, self.l1, self.accepted, self.emitted, self.cl,
                                    self.o2, self.l2, self.top)]

    def held(self, rows, factor):
        """The values that 4-bit rows [T, H, D] hold."""
        return F.values(*F.encode(rows, factor), factor)

    def attend(self, q, keys, values, lens, n, masks):
        """64-bit attention over each sequence's keys and values, in pages of their own."""
        pages = [-(-x.shape[0] // BS) for x in keys]
        table = torch.zeros((self.b, max(pages)), dtype=torch.int32, device=DEV)
        pools, at = torch.zeros((2, sum(pages) * BS, self.hkv, self.d), dtype=torch.float64, device=DEV), 0
        for b in range(self.b):
            table[b, :pages[b]] = torch.arange(at, at + pages[b])
            for pool, rows in zip(pools, (keys[b], values[b])):
                pool[at * BS:at * BS + rows.shape[0]] = rows
            at += pages[b]
        k, v = pools.view(2, sum(pages), BS, self.hkv, self.d)
        return k, v, table, F.attention(q.view(self.b, n, self.hq, self.d), k, v, table, lens, masks,
                                        1 / math.sqrt(self.d))

    def check(self):
        assert svpa.check_error(self.err) == 0
        # the prompts' keys as rows (what the norms and the rotation of rows are held to elsewhere)
        q, k, v = self.prompt
        rows, qs = torch.empty((self.t, self.hkv, self.d), dtype=BF, device=DEV), torch.empty_like(self.q0)
        svpa.qk_norm_rope(q, k, self.pos, self.cs, qs, rows, error_flag=self.err, q_weight=self.qw, k_weight=self.kw,
                          interleaved=self.interleaved)
        assert torch.equal(qs, self.q0)
        first = [sum(self.lens[:b]) for b in range(self.b)]
        kv, vv = self.held(rows, self.kf), self.held(v, self.vf)
        assert torch.equal(self.kr, kv.to(BF)) and torch.equal(self.vr, vv.to(BF))
        keys = [kv[s:s + n] for s, n in zip(first, self.lens)]
        values = [vv[s:s + n] for s, n in zip(first, self.lens)]

        k1, v1 = [x.view(self.b, self.nq, self.hkv, self.d) for x in (self.held(self.k1, self.kf),
                                                                      self.held(self.v1, self.vf))]
        _, _, _, (out, lse, ob, lb) = self.attend(self.q1, [torch.cat(x) for x in zip(keys, k1)],
                                                  [torch.cat(x) for x in zip(values, v1)], self.lens, self.nq,
                                                  self.masks)
        assert ((self.o1.view_as(out).double() - out).abs() <= ob).all()
        assert ((self.l1.view_as(lse).double() - lse).abs() <= lb).all()

        # what the commit kept, and the next token behind it
        taken = self.accepted.tolist()
        k2, v2 = self.held(self.k2, self.kf), self.held(self.v2, self.vf)
        lens = []
        for b, t in enumerate(taken):
            keep = list(range(t + 1)) if self.chain else [0] + self.path[b, 1:t + 1].tolist()
            assert all(self.depth[x] == i for i, x in enumerate(keep))
            lens.append(self.lens[b] + t + 1)
            keys[b] = torch.cat([keys[b], k1[b, keep], k2[b:b + 1]])
            values[b] = torch.cat([values[b], v1[b, keep], v2[b:b + 1]])
        assert self.cl.tolist() == lens
        _, _, _, (out, lse, ob, lb) = self.attend(self.q2, keys, values, lens, 1, None)
        assert ((self.o2.view_as(out).double() - out).abs() <= ob).all()
        assert ((self.l2.view_as(lse).double() - lse).abs() <= lb).all()

        # the prompts over the values rounded to bf16
        pages = [-(-n // BS) for n in self.lens]
        table = torch.zeros((self.b, max(pages)), dtype=torch.int32, device=DEV)
        pools = torch.zeros((2, sum(pages) * BS, self.hkv, self.d), dtype=BF, device=DEV)
        at = 0
        for b, n in enumerate(self.lens):
            table[b, :pages[b]] = torch.arange(at, at + pages[b])
            pools[0, at * BS:at * BS + n], pools[1, at * BS:at * BS + n] = [x[first[b]:first[b] + n] for x in (kv, vv)]
            at += pages[b]
        kb, vb = pools.view(2, at, BS, self.hkv, self.d).transpose(2, 3)
        ref = R.reference(self.q0, kb, vb, table, first, self.lens, self.lens,
                          [list(range(1, n + 1)) for n in self.lens], self.hkv, 1 / math.sqrt(self.d))
        R.check(self.o0, self.l0, ref, "prompts")


TREE = [-1, 0, 0, 1, 1, 2, 3, 3, 4, 6]


@pytest.mark.parametrize("lens,parent,kw", [
    ([150, 97, 1, 129], [-1, 0, 1, 2], {}),
    ([700, 31, 33], TREE, dict(hq=16, hkv=2)),
    ([40 + 7 * i for i in range(30)], [-1, 0, 1, 2, 3], dict(hq=4, hkv=4, d=64, rot=32)),
    ([255, 256, 16, 15], TREE, dict(hq=4, hkv=4, d=64, rot=64, interleaved=True)),
])
def test_from_admission_to_the_next_token(lens, parent, kw):
    f = Flow(lens, parent, **kw)
    f.restore()
    f.run()
    torch.cuda.synchronize()
    f.check()
    assert f.accepted.max() > 0
    eager = f.results()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    f.restore()
    torch.cuda.synchronize()
    f.run(stream=side)
    torch.cuda.synchronize()
    f.check()
    assert all(torch.equal(x, y) for x, y in zip(f.results(), eager))
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        f.run()
    for _ in range(2):
        f.restore()
        graph.replay()
        torch.cuda.synchronize()
        assert svpa.check_error(f.err) == 0
        assert all(torch.equal(x, y) for x, y in zip(f.results(), eager))
    f.check()
