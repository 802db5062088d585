"""A serving loop over pages in 8 bits: prompts in chunks, then steps of drafted tokens
(pages, append, attention, verification, log probabilities), eager and as one captured graph."""
import math

import numpy as np
import pytest
import torch

from e4m3_testutil import decode_bound
from oracle import e4m3
from oracle import serving as sv
from progressive_kv_quantization_gb300 import lynx as L

pytestmark = pytest.mark.gpu
D, HQ, HKV, B, T, V = 128, 8, 2, 4, 4, 1000
G = HQ // HKV
SCALE = 1 / math.sqrt(D)


class Server:
    def __init__(self, seed, max_pages=4, n_pool=200):
        self.rng = np.random.default_rng(seed)
        angle = np.arange(max_pages * 256)[:, None] * 1e4 ** (-np.arange(0, D, 2) / D)
        self.cs = np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)
        self.w = [self.rng.uniform(0.1, 0.3, D).astype(np.float32), self.rng.uniform(0.5, 1.5, D).astype(np.float32)]
        up = lambda a: torch.from_numpy(a).cuda()
        self.cs_d, self.wq, self.wk = up(self.cs), up(self.w[0]), up(self.w[1])
        self.pools = [torch.randint(0, 255, (n_pool, 256, D), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
                      for _ in range(2)]
        self.scales = torch.randint(0, 255, (n_pool, 2, 8), dtype=torch.uint8, device="cuda")
        self.table = torch.full((B, HKV, max_pages), -1, dtype=torch.int32, device="cuda")
        self.free = torch.from_numpy(self.rng.permutation(n_pool).astype(np.int32)).cuda()
        self.ctx = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.rows = [np.zeros((0, HQ + 2 * HKV, D)) for _ in range(B)]     # each request's projections so far, float64

    def append(self, qkv, new_len, n_rows, free):
        cu, pos, slots, ctx, taken = L.lynx_assign_pages(self.ctx, new_len, self.table, free, n_rows)
        q = L.lynx_qkv_append_e4m3(qkv, HQ, HKV, self.cs_d, pos, slots, *self.pools, self.scales, q_weight=self.wq, k_weight=self.wk)
        return cu, q, ctx, taken

    def values(self, b, h, n):
        """Keys and values as the pages hold them."""
        ids = self.table[b, h, :-(-n // 256)].cpu().numpy()
        s = self.scales.cpu().numpy()
        return [e4m3.dequantise_pages(p.view(torch.uint8).cpu().numpy()[ids], s[ids, i]).reshape(-1, D)[:n]
                for i, p in enumerate(self.pools)]

    def check_pages(self, b, n):
        """Within a block, half an E4M3 step of its largest value's scale; through at most five
        roundings (a block's scale grows by a step of the loop at most) three times that."""
        x = self.rows[b][:n]
        cos, sin = self.cs[:n, :D // 2].astype(float), self.cs[:n, D // 2:].astype(float)
        k = sv.norm_rotate(x[:, HQ:HQ + HKV], self.w[1], 1e-6, cos, sin, False)
        for h in range(HKV):
            for got, want in zip(self.values(b, h, n), (k[:, h], x[:, HQ + HKV + h])):
                for at in range(0, n, 32):
                    g, w = got[at:at + 32], want[at:at + 32]
                    # a normal code's error is 2^-4 of the value, a subnormal one's 2^-10 of a scale that is at most 2^-8 of
                    # the largest value that the block has had (drafts that were taken back among them: 2^3 covers those)
                    assert np.all(np.abs(g - w) <= 2.0 ** -4 * np.abs(w) * (1 + 2.0 ** -10) + 5 * 2.0 ** -15 * np.abs(w).max() + 1e-6)

    def check_attention(self, b, q, out, n, t, tol):
        """q, out [t, Hq, 128] of the last t of n tokens."""
        for h in range(HKV):
            k, v = self.values(b, h, n)
            rows = q[:, h * G:(h + 1) * G].reshape(-1, D)
            ref, _ = e4m3.attention(rows, k, v, SCALE, [n - t + i + 1 for i in range(t) for _ in range(G)])
            assert np.abs(out[:, h * G:(h + 1) * G].reshape(-1, D) - ref).max() <= tol(rows, k, v)


def f64(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("captured", [False, True])
def test_prompts_then_steps_with_drafts(cuda_device, captured):
    srv = Server(3)
    rng = srv.rng
    width = (HQ + 2 * HKV) * D
    make = lambda n: torch.from_numpy(rng.standard_normal((n, width)).astype(np.float32)).cuda().bfloat16()

    # ---- prompts, the longest in two chunks, one request in its own time
    for new in ([300, 37, 0, 1], [211, 0, 64, 0]):
        n = sum(new)
        qkv = make(n + 3)                                   # rows behind the last request
        cu, q, ctx, taken = srv.append(qkv, torch.tensor(new, dtype=torch.int32, device="cuda"), n + 3, srv.free)
        out, _ = L.lynx_chunk_attn_e4m3(q, cu, *srv.pools, srv.scales, srv.table, ctx, HKV)
        srv.free = srv.free[int(taken):].contiguous()
        srv.ctx = ctx
        L.lynx_device_status()
        at = 0
        for b in range(B):
            if not new[b]:
                continue
            srv.rows[b] = np.concatenate([srv.rows[b], f64(qkv[at:at + new[b]]).reshape(new[b], -1, D)])
            total = int(ctx[b])
            srv.check_pages(b, total)
            # P's rounding to BF16 and the output's, 2^-8 each, of values below the largest
            srv.check_attention(b, f64(q[at:at + new[b]]), f64(out[at:at + new[b]]), total, new[b],
                                lambda r, k, v: 2.0 ** -7 * np.abs(v).max())
            at += new[b]

    # ---- steps: T tokens a request, attended and verified; what is refused is taken back
    qkv = torch.empty(B * T, width, dtype=torch.bfloat16, device="cuda")
    logits = torch.empty(B, T, V, device="cuda")
    draft = torch.empty(B, T - 1, dtype=torch.int32, device="cuda")
    u = torch.empty(B, T, device="cuda")
    new_len = torch.full((B,), T, dtype=torch.int32, device="cuda")
    free = srv.free[:2 * B * HKV].clone()
    ws = torch.empty(L.lynx_decode_attn_e4m3_workspace_size(B, T, HQ, HKV, D), dtype=torch.uint8, device="cuda")

    def step():
        _, q, ctx, taken = srv.append(qkv, new_len, B * T, free)
        out, _ = L.lynx_decode_attn_e4m3(q.view(B, T, HQ, D), *srv.pools, srv.scales, srv.table, ctx, HKV, causal=True, workspace=ws)
        tokens, n = L.lynx_verify_drafts(torch.softmax(logits, -1), None, draft, u)
        scores = L.lynx_token_logprobs(logits, tokens, 3)
        return q, out, ctx, taken, tokens, n, scores

    graph = None
    start = srv.ctx.clone()
    for i in range(12):
        qkv.copy_(make(B * T))
        logits.copy_(torch.from_numpy(rng.standard_normal((B, T, V)).astype(np.float32) * 3))
        draft.copy_(logits[:, :T - 1].argmax(-1))           # likely ones
        u.copy_(torch.from_numpy(rng.random((B, T)).astype(np.float32)))
        free.copy_(srv.free[:free.numel()])
        if captured and graph is None:
            kept = [t.clone() for t in (srv.table, srv.scales, *(p.view(torch.uint8) for p in srv.pools))]
            step()                                          # first calls outside the capture; then all as it was
            for t, k in zip((srv.table, srv.scales, *(p.view(torch.uint8) for p in srv.pools)), kept):
                t.copy_(k)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                got = step()
        if graph is not None:
            graph.replay()
        else:
            got = step()
        q, out, ctx, taken, tokens, n, scores = got
        L.lynx_device_status()
        assert ctx.tolist() == (srv.ctx + T).tolist()
        for b in range(B):
            total = int(ctx[b])
            x = f64(qkv[b * T:(b + 1) * T]).reshape(T, -1, D)
            srv.rows[b] = np.concatenate([srv.rows[b], x])
            srv.check_pages(b, total)
            srv.check_attention(b, f64(q[b * T:(b + 1) * T]), f64(out[b]), total, T,
                                lambda r, k, v: decode_bound(r, k, v, SCALE))
            srv.rows[b] = srv.rows[b][:total - T + int(n[b]) + 1]
        # the tokens' log probabilities; -inf behind the last one
        flat = f64(logits).reshape(-1, V)
        lp, h, ids, top = sv.token_logprobs(flat, tokens.cpu().numpy().reshape(-1), 3)
        g = f64(scores[0]).reshape(-1)
        assert np.array_equal(np.isneginf(g), tokens.cpu().numpy().reshape(-1) < 0)
        assert np.all(np.abs(g - lp)[~np.isneginf(lp)] <= 2.0 ** -15)
        assert np.array_equal(scores[2].cpu().numpy().reshape(-1, 3), ids)
        srv.free = srv.free[int(taken):].contiguous()
        srv.ctx.copy_(srv.ctx + n + 1)
    assert torch.all(srv.ctx > start)
