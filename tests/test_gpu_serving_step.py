"""The serving-step operators together, as a serving loop runs them: pages and
slots, QKV append, chunk attention, Lynx planes of the finished pages, draft
decode over the Anchor, verification.  Attention is checked against float64
attention over the whole unpaged sequences."""
import math

import numpy as np
import pytest
import torch

from oracle import serving as sv
from progressive_kv_quantization_gb300 import lynx as L

pytestmark = pytest.mark.gpu
D = 128


class Loop:
    """One layer of a serving loop: requests with their own lengths, one pool of pages."""

    def __init__(self, B, Hq, Hkv, max_pages, n_rows, seed):
        self.B, self.Hq, self.Hkv, self.n_rows = B, Hq, Hkv, n_rows
        g = torch.Generator("cuda").manual_seed(seed)
        n_pool = B * Hkv * max_pages
        self.k = torch.full((n_pool, D, 256), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.v = torch.full((n_pool, D, 256), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.table = torch.zeros(B, Hkv, max_pages, dtype=torch.int32, device="cuda")
        self.free = torch.randperm(n_pool, generator=torch.Generator().manual_seed(seed)).int().cuda()
        self.ctx = torch.zeros(B, dtype=torch.int32, device="cuda")
        ang = torch.arange(max_pages * 256, dtype=torch.float64)[:, None] * 1e4 ** (-torch.arange(64) / 64.0)
        self.cos_sin = torch.cat([ang.cos(), ang.sin()], 1).float().cuda()
        self.wq = 0.5 + torch.rand(D, generator=g, device="cuda")
        self.wk = 0.5 + torch.rand(D, generator=g, device="cuda")
        self.new = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.qkv = torch.zeros(n_rows, (Hq + 2 * Hkv) * D, dtype=torch.bfloat16, device="cuda")
        self.q = torch.empty(n_rows, Hq, D, dtype=torch.bfloat16, device="cuda")
        self.out = torch.full((n_rows, Hq, D), 9.0, device="cuda")
        self.lse = torch.full((n_rows, Hq), 9.0, device="cuda")
        self.ws = torch.empty(L.lynx_chunk_attn_workspace_size(n_rows, B, Hq, Hkv, D), dtype=torch.uint8, device="cuda")
        self.g = g

    def kernels(self):
        """What one step launches (it can be captured)."""
        cu, pos, slots, ctx, taken = L.lynx_assign_pages(self.ctx, self.new, self.table, self.free, self.n_rows)
        L.lynx_qkv_append(self.qkv, self.Hq, self.Hkv, self.cos_sin, pos, slots, self.k, self.v, q_weight=self.wq,
                          k_weight=self.wk, q_out=self.q)
        L.lynx_chunk_attn_bf16(self.q, cu, self.k, self.v, self.table, ctx, self.Hkv, out=self.out, lse=self.lse,
                               workspace=self.ws)
        return cu, ctx, taken

    def fill(self, new):
        rows = sum(new)
        x = torch.randn(rows, self.qkv.shape[1], generator=self.g, device="cuda").bfloat16()
        self.qkv[:rows] = x
        self.new.copy_(torch.tensor(new))
        return x.double().cpu().numpy().reshape(rows, -1, D)


def reference(seqs, Hq, Hkv, wq, wk, table):
    """Attention rows of whole sequences [tokens, heads, 128] in float64: keys and
    queries as the kernels round them (BF16), values as they are."""
    def rot(x, w):
        n = x.shape[0]
        y = sv.norm_rotate(x, w, 1e-6, table[:n, :64].astype(np.float64), table[:n, 64:].astype(np.float64), False)
        return torch.from_numpy(y).bfloat16().double().numpy()
    res = []
    for x in seqs:
        q, k, v = rot(x[:, :Hq], wq), rot(x[:, Hq:Hq + Hkv], wk), x[:, Hq + Hkv:]
        o = np.empty_like(q)
        for h in range(Hq):
            s = q[:, h] @ k[:, h // (Hq // Hkv)].T / math.sqrt(D)
            s = np.where(np.tri(len(s), dtype=bool), s, -np.inf)
            p = np.exp(s - s.max(1, keepdims=True))
            o[:, h] = p @ v[:, h // (Hq // Hkv)] / p.sum(1, keepdims=True)
        res.append(o)
    return res


STEPS = [[300, 1, 40], [200, 256, 0], [1, 700, 217], [1, 1, 1], [0, 65, 1], [1, 1, 1]]


@pytest.mark.parametrize("graph", [False, True])
def test_a_serving_loop_equals_attention_over_the_whole_sequences(cuda_device, graph):
    B, Hq, Hkv, n_rows = 3, 8, 2, 1000
    lp = Loop(B, Hq, Hkv, 6, n_rows, 1)
    lp.kernels()                       # the first call on the device configures the kernels
    torch.cuda.synchronize()
    if graph:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            held = lp.kernels()
    seqs = [np.zeros((0, Hq + 2 * Hkv, D)) for _ in range(B)]
    outs = [np.zeros((0, Hq, D)) for _ in range(B)]
    for new in STEPS:
        x = lp.fill(new)
        lp.out.fill_(9.0)
        cu, ctx, taken = (g.replay(), held)[1] if graph else lp.kernels()
        torch.cuda.synchronize()
        L.lynx_device_status()
        bounds = cu.tolist()
        assert bounds == np.concatenate([[0], np.cumsum(new)]).tolist()
        assert bool((lp.out[sum(new):] == 9).all())           # rows behind the last request stay as they were
        o = lp.out.double().cpu().numpy()
        for b in range(B):
            seqs[b] = np.concatenate([seqs[b], x[bounds[b]:bounds[b + 1]]])
            outs[b] = np.concatenate([outs[b], o[bounds[b]:bounds[b + 1]]])
        lp.ctx.copy_(ctx)
        lp.free = lp.free if graph else lp.free[int(taken):]   # the program keeps its list
        if graph:
            lp.free.copy_(torch.roll(lp.free, -int(taken)))    # a captured list stays where it is
        assert ctx.tolist() == [len(s) for s in seqs]
    ref = reference(seqs, Hq, Hkv, lp.wq.cpu().numpy(), lp.wk.cpu().numpy(), lp.cos_sin.cpu().numpy())
    for b in range(B):
        # P's rounding to BF16 (half a step: 2^-8 of the largest |v|) and scores that differ where float32 and
        # float64 round a query or key to different BF16 neighbours: a step of 2^-8 of one factor of
        # 128, |q k| / sqrt(128) of a few units: together below 2^-6 of the largest |v|
        vm = np.abs(seqs[b][:, Hq + Hkv:]).max()
        assert np.abs(outs[b] - ref[b]).max() <= 2.0 ** -6 * vm
        rel = np.linalg.norm(outs[b] - ref[b]) / np.linalg.norm(ref[b])
        assert rel < 2.0 ** -7


def test_finished_pages_serve_the_packed_cache(cuda_device):
    """The pages that the step writes are what the encoder and the packed decode take:
    chunk attention over the BF16 pages and lynx_decode_attn over their planes agree
    within the quantiser's error, and reconstructed pages feed chunk attention."""
    B, Hq, Hkv = 2, 4, 1
    lp = Loop(B, Hq, Hkv, 4, 1030, 2)
    lp.fill([512, 512])
    _, ctx, taken = lp.kernels()
    lp.ctx.copy_(ctx)
    lp.free = lp.free[int(taken):]
    ids = lp.table[:, :, :2].flatten().long()
    planes_k, planes_v = L.lynx_encode_pages(lp.k[ids].contiguous()), L.lynx_encode_pages(lp.v[ids].contiguous())
    local = torch.arange(B * Hkv * 2, dtype=torch.int32, device="cuda").view(B, Hkv, 2)
    q = torch.randn(B, 1, Hq, D, generator=lp.g, device="cuda").bfloat16()
    cu = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    exact, lse = L.lynx_chunk_attn_bf16(q[:, 0], cu, lp.k, lp.v, lp.table, ctx, Hkv, out_dtype=torch.float32)
    full, lse_full = L.lynx_decode_attn(q, planes_k[0], planes_k[1], planes_k[2], planes_v[0], planes_v[1], planes_v[2],
                                        local, ctx, Hkv)
    rk = L.lynx_reconstruct(*planes_k)
    rv = L.lynx_reconstruct(*planes_v)
    again, lse_again = L.lynx_chunk_attn_bf16(q[:, 0], cu, rk, rv, local, ctx, Hkv, out_dtype=torch.float32)
    torch.cuda.synchronize()
    L.lynx_device_status()
    vm = float(lp.v[ids].float().abs().max())
    # the same dequantised cache, rounded to BF16 for the chunk kernel (half a step, 2^-8, of a value and of a
    # key) and P to BF16 (2^-8)
    assert float((again - full[:, 0]).abs().max()) <= 2.0 ** -6 * vm
    # a full code is within half a step of the 8-bit compander: a few per cent of a chunk's range
    assert float((exact - full[:, 0]).norm() / exact.norm()) < 0.1
    # attention over two disjoint sets of keys, joined: pages 0 and 1 apart
    half = torch.full((B,), 256, dtype=torch.int32, device="cuda")
    a = L.lynx_chunk_attn_bf16(q[:, 0], cu, lp.k, lp.v, lp.table[:, :, :1].contiguous(), half, Hkv, causal=False,
                               out_dtype=torch.float32)
    b = L.lynx_chunk_attn_bf16(q[:, 0], cu, lp.k, lp.v, lp.table[:, :, 1:2].contiguous(), half, Hkv, causal=False,
                               out_dtype=torch.float32)
    o, l = L.lynx_attn_merge(a[0], a[1], b[0], b[1])
    assert float((o - exact).abs().max()) <= 2.0 ** -8 * vm and float((l - lse).abs().max()) <= 2.0 ** -11


def test_speculation_around_the_step(cuda_device):
    """Drafts appended and attended as one chunk, verified, and the rejected ones taken
    back by the context length alone: the next step overwrites them."""
    B, Hq, Hkv, T, V = 2, 4, 2, 4, 1000
    lp = Loop(B, Hq, Hkv, 3, 600, 3)
    lp.fill([250, 300])
    _, ctx, taken = lp.kernels()
    lp.ctx.copy_(ctx)
    lp.free = lp.free[int(taken):]
    x = lp.fill([T, T])
    cu, ctx, taken = lp.kernels()
    proj = torch.randn(Hq * D, V, generator=lp.g, device="cuda") * 0.3
    logits = lp.out[:B * T].reshape(B, T, -1) @ proj
    p = torch.softmax(torch.cat([logits, logits[:, -1:]], 1), -1)
    q = torch.softmax(logits + 0.3 * torch.randn(logits.shape, generator=lp.g, device="cuda"), -1)
    draft = torch.multinomial(q.reshape(B * T, V), 1, generator=lp.g).view(B, T).int()
    u = torch.rand(B, T + 1, generator=lp.g, device="cuda")
    tokens, n = L.lynx_verify_drafts(p, q, draft, u)
    rt, rn = sv.verify_drafts(p.cpu().numpy(), q.cpu().numpy(), draft.cpu().numpy(), None, u.cpu().numpy())
    assert np.array_equal(tokens.cpu().numpy(), rt) and np.array_equal(n.cpu().numpy(), rn)
    # back to the accepted length; the next token's keys go to the first rejected slot
    lp.ctx.copy_(lp.ctx + n)
    lp.free = lp.free[int(taken):]
    lp.fill([1, 1])
    cu2, ctx2, taken2 = lp.kernels()
    torch.cuda.synchronize()
    L.lynx_device_status()
    assert int(taken2) == 0                      # the page is there from the drafts
    assert ctx2.tolist() == [int(250 + rn[0] + 1), int(300 + rn[1] + 1)]
