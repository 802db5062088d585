"""Cases that measure the operators of one serving step over the paged cache.

A step takes a ragged batch of requests: it gives their new tokens pages and
slots (``assign``), normalises and rotates the new queries and keys and writes
the new keys and values into the pages (``append``), attends from each chunk
of new tokens to its request's paged cache (``chunk``), and verifies drafted
tokens against the target's probabilities (``verify``).

``run`` computes each operator in its plain form (elementary torch operations
in 32 bits) or, where ``own`` is true, calls the framework's kernels; both take
what ``prepare`` gives.  Pages are channel-major [128 channels][256 tokens]
BF16, one KV head each, addressed through a table [B][KV heads][pages].
"""
import math

import torch

own = False

H, P = 128, 256
DEV = "cuda"
UNIT = 2.0 ** 40      # verify: probabilities are summed as whole multiples of 2^-40
U_STEPS = 1 << 24     # verify: random numbers count in steps of 2^-24


def listed():
    return [
        # one decode step of 64 requests: every request gets one token, few a page
        dict(name="assign decode step", op="assign", B=64, Hkv=8, max_ctx=16384, max_new=1, pad=0),
        # a step that mixes decoding requests with prompts arriving in chunks
        dict(name="assign mixed batch", op="assign", B=96, Hkv=4, max_ctx=131072, max_new=2048, pad=37),
        # a wave of prompts, prefilled at once into a fixed number of rows
        dict(name="assign prompt wave", op="assign", B=256, Hkv=8, max_ctx=300, max_new=1000, pad=512),
        # the new tokens of one decode step of 64 requests (Llama-3-8B-shaped heads)
        dict(name="append decode step", op="append", B=64, Hq=32, Hkv=8, max_new=1, norm=False, rot=128,
             interleaved=False, max_ctx=16384),
        # a 4K chunk with query and key norms (Qwen3-235B-shaped heads), from few requests at odd places
        dict(name="append chunk", op="append", B=5, Hq=16, Hkv=4, max_new=1200, norm=True, rot=128,
             interleaved=False, max_ctx=131072),
        # the prompts of a prefill wave, half of each head rotated in neighbouring pairs
        dict(name="append prompt wave", op="append", B=24, Hq=32, Hkv=8, max_new=2800, norm=True, rot=64,
             interleaved=True, max_ctx=8000),
        # a short follow-up prompt to a short conversation
        dict(name="chunk short prompt", op="chunk", B=1, Hq=32, Hkv=8, max_new=17, max_ctx=983),
        # one decode step over the paged cache, one token a request
        dict(name="chunk decode step", op="chunk", B=16, Hq=32, Hkv=8, max_new=1, max_ctx=16383),
        # chunked prefill of several requests at once, contexts of odd lengths
        dict(name="chunk ragged prefill", op="chunk", B=6, Hq=32, Hkv=8, max_new=1024, max_ctx=7000),
        # a 2K chunk at the end of a 128K context (one Qwen3-235B-shaped layer)
        dict(name="chunk long context", op="chunk", B=1, Hq=16, Hkv=4, max_new=2048, max_ctx=129024),
        # one request with four drafts
        dict(name="verify one request", op="verify", B=1, T=4, V=32000, dtype="float32", drafts=True),
        # a batch of 32 requests with up to eight drafts and a large vocabulary
        dict(name="verify batch", op="verify", B=32, T=8, V=151936, dtype="float32", drafts=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["assign", "append", "chunk", "verify"])
    Hkv = rng.choice([1, 2, 4, 8])
    if op == "assign":
        B = _log_int(rng, 1, 256)
        return dict(op=op, B=B, Hkv=Hkv, max_ctx=_log_int(rng, 200, 131072),
                    max_new=_log_int(rng, 1, max(1, 250000 // B // Hkv)), pad=rng.choice([0, 0, rng.randrange(1, 300)]))
    G = rng.choice([1, 2, 3, 4, 5, 8])
    if op == "append":
        B = _log_int(rng, 1, 128)
        most = max(1, 600000 // B // (Hkv * (G + 2)))
        return dict(op=op, B=B, Hq=G * Hkv, Hkv=Hkv, max_new=_log_int(rng, 1, min(8192, most)), norm=rng.random() < 0.6,
                    rot=rng.choice([128, 128, 64, 32]), interleaved=rng.random() < 0.4, max_ctx=_log_int(rng, 10, 60000))
    if op == "chunk":
        B = _log_int(rng, 1, 24)
        max_ctx = _log_int(rng, 1, 131072 // B)
        most = max(1, int(2.0e9) // (B * G * Hkv * (max_ctx + 2048)))
        return dict(op=op, B=B, Hq=G * Hkv, Hkv=Hkv, max_new=_log_int(rng, 1, min(4096, most)), max_ctx=max_ctx)
    V = _log_int(rng, 500, 200000)
    B = _log_int(rng, 1, max(1, min(256, 4000000 // V)))
    return dict(op=op, B=B, T=rng.randrange(1, 9), V=V, dtype=rng.choice(["float32", "float32", "bfloat16"]),
                drafts=rng.random() < 0.8)


# ----------------------------------------------------------------------------- inputs


def _lengths(case):
    """Cached and new tokens of each request (host lists), the case's own: the
    first request is the longest, the others spread below it, and every third
    one decodes a single token."""
    B, new_hi, ctx_hi = case["B"], case["max_new"], case["max_ctx"]
    rng = torch.Generator().manual_seed(B)
    new, ctx = [new_hi], [ctx_hi]
    for b in range(1, B):
        new.append(1 if b % 3 == 2 else max(1, int(new_hi * (0.25 + 0.75 * float(torch.rand((), generator=rng))))))
        ctx.append(int(ctx_hi * (0.1 + 0.9 * float(torch.rand((), generator=rng)))))
    return new, ctx


def _pages(n):
    return -(-n // P)


def _gens(seed):
    return torch.Generator().manual_seed(seed), torch.Generator(DEV).manual_seed(seed)


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _table(lens, Hkv, max_pages, order):
    """[B][Hkv][max_pages] page ids taken from a shuffled order, -1 past each request's last page."""
    table = torch.full((len(lens), Hkv, max_pages), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(lens):
        k = _pages(n)
        table[b, :, :k] = order[at:at + Hkv * k].view(Hkv, k)
        at += Hkv * k
    return table.to(DEV), at


def prepare(case, seed):
    cpu, gpu = _gens(seed)
    s = {"case": case}
    if case["op"] == "verify":
        B, T, V = case["B"], case["T"], case["V"]
        dt = getattr(torch, case["dtype"])
        # sharp target distributions and drafts from a model near to it
        logits = torch.randn(B, T + 1, V, generator=gpu, device=DEV).mul_(2.5)
        s["p"] = torch.softmax(logits, -1).to(dt)
        near = logits[:, :T] + 0.7 * torch.randn(B, T, V, generator=gpu, device=DEV)
        q = torch.softmax(near, -1)
        s["draft"] = torch.multinomial(q.view(B * T, V), 1, generator=gpu).view(B, T).to(torch.int32)
        s["q"] = q.to(dt) if case["drafts"] else None
        s["n_draft"] = torch.randint(max(0, T - 2), T + 1, (B,), generator=cpu).to(torch.int32).to(DEV)
        s["u"] = torch.rand(B, T + 1, generator=gpu, device=DEV)
        s["tokens"] = torch.empty(B, T + 1, dtype=torch.int32, device=DEV)
        s["n_accept"] = torch.empty(B, dtype=torch.int32, device=DEV)
        return s
    B, Hkv = case["B"], case["Hkv"]
    new, ctx = _lengths(case)
    total = [a + b for a, b in zip(new, ctx)]
    n_rows = sum(new) + case.get("pad", 0)
    max_pages = max(_pages(n) for n in total)
    if case["op"] == "assign":
        held = sum(Hkv * _pages(n) for n in ctx)
        need = sum(Hkv * (_pages(t) - _pages(c)) for t, c in zip(total, ctx))
        order = torch.randperm(held + need + 64, generator=cpu).to(torch.int32)
        s["table"], at = _table(ctx, Hkv, max_pages, order)
        s["free"] = order[at:].contiguous().to(DEV)
        s["new"], s["ctx"], s["n_rows"] = _i32(new), _i32(ctx), n_rows
        s["cu"] = torch.empty(B + 1, dtype=torch.int32, device=DEV)
        s["pos"] = torch.empty(n_rows, dtype=torch.int32, device=DEV)
        s["slots"] = torch.empty(n_rows, Hkv, dtype=torch.int64, device=DEV)
        s["ctx_out"] = torch.empty(B, dtype=torch.int32, device=DEV)
        s["taken"] = torch.empty(1, dtype=torch.int32, device=DEV)
        return s
    Hq = case["Hq"]
    if case["op"] == "append":
        # only the pages that take new tokens, in a shuffled order; every request starts at its own place in a page
        touched = [(c % P) + n for n, c in zip(new, ctx)]
        order = torch.randperm(sum(Hkv * _pages(n) for n in touched) + 3, generator=cpu).to(torch.int32)
        table, _ = _table(touched, Hkv, max(_pages(n) for n in touched), order)
        seq = torch.repeat_interleave(torch.arange(B), torch.tensor(new)).to(DEV)
        first = torch.tensor([sum(new[:b]) for b in range(B)], device=DEV)
        i = torch.arange(n_rows, device=DEV) - first[seq]
        s["pos"] = (torch.tensor(ctx, device=DEV)[seq] + i).to(torch.int32)
        off = torch.tensor([c % P for c in ctx], device=DEV)[seq] + i
        page = table.long()[seq[:, None], torch.arange(Hkv, device=DEV)[None], (off // P)[:, None]]
        s["slots"] = page * P + (off % P)[:, None]
        n_pool = order.numel()
        width = (Hq + 2 * Hkv) * H
        # per-channel scales and offsets as projections give them, rows inside a wider buffer
        wide = torch.randn(n_rows, width + 64, generator=gpu, device=DEV)
        wide[:, :width] *= 0.3 + 2.0 * torch.rand(width, generator=gpu, device=DEV)
        s["qkv"] = wide.to(torch.bfloat16)[:, :width]
        s["wq"] = s["wk"] = None
        if case["norm"]:
            s["wq"] = 0.5 + torch.rand(H, generator=gpu, device=DEV)
            s["wk"] = 0.5 + torch.rand(H, generator=gpu, device=DEV)
        # cosines and sines of the positions, made once in 64 bits
        rot = case["rot"]
        inv = 1e6 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
        angle = torch.arange(max(total), dtype=torch.float64, device=DEV)[:, None] * inv
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        s["k_pages"] = torch.randn(n_pool, H, P, generator=gpu, device=DEV).to(torch.bfloat16)
        s["v_pages"] = torch.randn(n_pool, H, P, generator=gpu, device=DEV).to(torch.bfloat16)
        s["q_out"] = torch.empty(n_rows, Hq, H, dtype=torch.bfloat16, device=DEV)
        return s
    order = torch.randperm(sum(Hkv * _pages(n) for n in total) + 2, generator=cpu).to(torch.int32)
    s["table"], _ = _table(total, Hkv, max_pages, order)
    s["table"].clamp_(min=0)
    n_pool = order.numel()
    # keys and values with an offset for each channel (the caches' structure), queries of unit variance
    offset = torch.randn(2, 1, H, 1, generator=gpu, device=DEV)
    s["k_pages"] = torch.randn(n_pool, H, P, generator=gpu, device=DEV).add_(offset[0]).to(torch.bfloat16)
    s["v_pages"] = torch.randn(n_pool, H, P, generator=gpu, device=DEV).add_(offset[1]).to(torch.bfloat16)
    s["q"] = torch.randn(n_rows, Hq, H, generator=gpu, device=DEV).to(torch.bfloat16)
    s["cu"] = _i32([sum(new[:b]) for b in range(B + 1)])
    s["ctx"] = _i32(total)
    s["max_new"] = max(new)
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty(n_rows, Hq, dtype=torch.float32, device=DEV)
    s["workspace"] = torch.empty(0, dtype=torch.uint8, device=DEV)
    return s


# ----------------------------------------------------------------------------- one pass


def run(s):
    op = s["case"]["op"]
    if own:
        return _own(op, s)
    return {"assign": _assign, "append": _append, "chunk": _chunk, "verify": _verify}[op](s)


def _own(op, s):
    from progressive_kv_quantization_gb300 import lynx as L

    if op == "assign":
        cu, pos, slots, ctx, taken = L.lynx_assign_pages(s["ctx"], s["new"], s["table"], s["free"], s["n_rows"],
                                                         cu_new=s["cu"], positions=s["pos"], slots=s["slots"],
                                                         ctx_out=s["ctx_out"], n_taken=s["taken"])
        return {"table": s["table"], "cu": cu, "pos": pos, "slots": slots, "ctx": ctx, "taken": taken}
    if op == "append":
        c = s["case"]
        q = L.lynx_qkv_append(s["qkv"], c["Hq"], c["Hkv"], s["cos_sin"], s["pos"], s["slots"], s["k_pages"],
                              s["v_pages"], q_weight=s["wq"], k_weight=s["wk"], interleaved=c["interleaved"],
                              q_out=s["q_out"])
        return {"q": q, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    if op == "chunk":
        c = s["case"]
        if s["workspace"].numel() == 0:   # kept by the program from its first call on
            s["workspace"] = torch.empty(L.lynx_chunk_attn_workspace_size(s["q"].shape[0], c["B"], c["Hq"], c["Hkv"], H),
                                         dtype=torch.uint8, device=DEV)
        o, lse = L.lynx_chunk_attn_bf16(s["q"], s["cu"], s["k_pages"], s["v_pages"], s["table"], s["ctx"], c["Hkv"],
                                        causal=True, out=s["out"], lse=s["lse"], workspace=s["workspace"])
        return {"out": o, "lse": lse}
    tokens, n = L.lynx_verify_drafts(s["p"], s["q"], s["draft"], s["u"], n_draft=s["n_draft"], tokens=s["tokens"],
                                     n_accept=s["n_accept"])
    return {"tokens": tokens, "n": n}


def _assign(s):
    """Pages for the tokens that start a new one, from the free list in request
    order, and position and slot of every new token's row (-1 in the rows behind)."""
    table, free = s["table"], s["free"]
    B, Hkv, max_pages = table.shape
    new, ctx = s["new"].long(), s["ctx"].long()
    n_free = free.numel()
    held = (ctx + P - 1) // P
    need = (ctx + new + P - 1) // P - held
    end = (need * Hkv).cumsum(0)
    granted = (end <= n_free) | (need == 0)
    cu = torch.cat([new.new_zeros(1), new.cumsum(0)]).clamp(max=s["n_rows"])
    j = torch.arange(max_pages, device=DEV)
    at = (end - need * Hkv)[:, None, None] + (j - held[:, None])[:, None] * Hkv + torch.arange(Hkv, device=DEV)[:, None]
    fresh = (j >= held[:, None]) & (j < (held + need)[:, None]) & granted[:, None]
    table.copy_(torch.where(fresh[:, None], free[at.clamp(0, n_free - 1)], table))
    r = torch.arange(s["n_rows"], device=DEV)
    seq = torch.searchsorted(cu, r, right=True) - 1
    real = seq < B
    seq = seq.clamp(max=B - 1)
    real &= granted[seq]
    pos = ctx[seq] + r - cu[seq]
    page = table[seq, :, (pos // P).clamp(0, max_pages - 1)].long()
    slots = torch.where(real[:, None], page * P + (pos % P)[:, None], -1)
    taken = torch.where(granted & (need > 0), end, 0).amax().reshape(1)
    return {"table": table, "cu": cu.to(torch.int32), "pos": torch.where(real, pos, -1).to(torch.int32), "slots": slots,
            "ctx": torch.where(granted, ctx + new, ctx).to(torch.int32), "taken": taken.to(torch.int32)}


def _norm_rotate(x, w, cos, sin, interleaved):
    if w is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w
    rot = 2 * cos.shape[-1]
    cos, sin = cos[:, None], sin[:, None]
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _append(s):
    """RMS norm of each query and key head, rotation by the row's position, and the
    keys and values written to their slots."""
    c = s["case"]
    Hq, Hkv = c["Hq"], c["Hkv"]
    x = s["qkv"].view(-1, Hq + 2 * Hkv, H)
    cs = s["cos_sin"][s["pos"].long()]
    cos, sin = cs[:, :c["rot"] // 2], cs[:, c["rot"] // 2:]
    q = _norm_rotate(x[:, :Hq].float(), s["wq"], cos, sin, c["interleaved"]).to(torch.bfloat16)
    k = _norm_rotate(x[:, Hq:Hq + Hkv].float(), s["wk"], cos, sin, c["interleaved"]).to(torch.bfloat16)
    page, off = s["slots"] // P, s["slots"] % P
    s["k_pages"][page, :, off] = k
    s["v_pages"][page, :, off] = x[:, Hq + Hkv:]
    return {"q": q, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _chunk(s):
    """softmax(scale q.k) v of every new token over the keys up to its own position,
    the ragged batch padded to its longest request."""
    q, table = s["q"], s["table"].long()
    N, Hq, _ = q.shape
    B, Hkv, n_pages = table.shape
    G, T, S = Hq // Hkv, s["max_new"], n_pages * P
    cu, ctx = s["cu"].long(), s["ctx"].long()
    i = torch.arange(T, device=DEV)
    rows = (cu[:-1, None] + i).clamp(max=N - 1)
    qp = q[rows].float().view(B, T, Hkv, G, H).transpose(1, 2).reshape(B, Hkv, T * G, H)
    k = s["k_pages"][table].permute(0, 1, 3, 2, 4).reshape(B, Hkv, H, S).float()
    v = s["v_pages"][table].permute(0, 1, 3, 2, 4).reshape(B, Hkv, H, S).float()
    scores = torch.matmul(qp, k).mul_(1 / math.sqrt(H)).view(B, Hkv, T, G, S)
    seen = (ctx - (cu[1:] - cu[:-1]) + 1)[:, None] + i                         # keys that each row sees
    hidden = torch.arange(S, device=DEV) >= seen[:, None, :, None, None]
    scores.masked_fill_(hidden, -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    prob = scores.sub_(top).exp_()
    total = prob.sum(-1, keepdim=True)
    o = torch.matmul(prob.view(B, Hkv, T * G, S), v.transpose(2, 3)).view(B, Hkv, T, G, H)
    o = (o / torch.where(total == 0, 1.0, total)).transpose(1, 2).reshape(B, T, Hq, H)
    lse = (total.log() + top).squeeze(-1).transpose(1, 2).reshape(B, T, Hq)
    r = torch.arange(N, device=DEV)
    seq = torch.searchsorted(cu, r, right=True) - 1
    at = r - cu[seq]
    return {"out": o[seq, at].to(torch.bfloat16), "lse": lse[seq, at]}


def _verify(s):
    """Drafts accepted while u q < p; then a token from max(0, p - q), or from p
    behind the last draft, by the inverse of its running sum."""
    p, q, u = s["p"], s["q"], s["u"]
    B, T = s["draft"].shape
    V = p.shape[-1]
    x = s["draft"].long()[..., None]
    px = p[:, :T].gather(-1, x)[..., 0].float()
    qx = 1.0 if q is None else q.gather(-1, x)[..., 0].float()
    i = torch.arange(T, device=DEV)
    ok = (u[:, :T] * qx < px) & (i < s["n_draft"][:, None])
    n = ok.long().cumprod(1).sum(1)
    b = torch.arange(B, device=DEV)
    row = p[b, n].float()
    at = n.clamp(max=T - 1)
    if q is None:
        drafted = torch.zeros_like(row).scatter_(1, x[b, at], math.inf)
    else:
        drafted = q[b, at].float()
    rejected = (n < s["n_draft"])[:, None]
    left = (torch.where(rejected, row - drafted, row).clamp(0, 1) * UNIT).long()
    whole = (row.clamp(0, 1) * UNIT).long()
    weight = torch.where(left.sum(1, keepdim=True) > 0, left, whole)
    run_sum = weight.cumsum(1)
    total = run_sum[:, -1]
    step = (u[:, T] * U_STEPS).long().clamp(0, U_STEPS - 1)
    limit = (total >> 24) * step + (((total & (U_STEPS - 1)) * step) >> 24)      # floor(total u)
    last = torch.where(total > 0, (run_sum <= limit[:, None]).sum(1), -1)
    i = torch.arange(T + 1, device=DEV)
    padded = torch.cat([s["draft"].long(), last[:, None]], 1)
    tokens = torch.where(i < n[:, None], padded, torch.where(i == n[:, None], last[:, None], -1))
    return {"tokens": tokens.to(torch.int32), "n": n.to(torch.int32)}


# ----------------------------------------------------------------------------- what a pass needs


def work(case):
    """Each input once, each output once; products and sums of the formulas."""
    op, B = case["op"], case["B"]
    if op == "verify":
        size = 4 if case["dtype"] == "float32" else 2
        rows = 2 if case["drafts"] else 1
        return {"bytes": B * (rows * case["V"] * size + case["T"] * 24), "flops": 2 * B * case["V"]}
    new, ctx = _lengths(case)
    n, Hkv = sum(new), case["Hkv"]
    if op == "assign":
        fresh = sum(Hkv * (_pages(a + b) - _pages(b)) for a, b in zip(new, ctx))
        return {"bytes": B * 16 + fresh * 8 + (n + case["pad"]) * (4 + 8 * Hkv), "flops": n * Hkv}
    Hq = case["Hq"]
    if op == "append":
        return {"bytes": n * (2 * H * 2 * (Hq + 2 * Hkv) + 4 * case["rot"] + 4 + 8 * Hkv), "flops": 8 * n * H * (Hq + Hkv)}
    seen = sum(a * b + a * (a + 1) // 2 for a, b in zip(new, ctx))
    held = sum(a + b for a, b in zip(new, ctx))
    return {"bytes": n * Hq * (4 * H + 4) + held * Hkv * 4 * H, "flops": 4 * H * Hq * seen}


# ----------------------------------------------------------------------------- the definition in 64 bits


def exact(case, seed):
    if case["op"] in ("assign", "verify"):
        return None          # whole numbers only
    s = prepare(case, seed)
    return _exact_append(case, s) if case["op"] == "append" else _exact_chunk(case, s)


def _exact_append(case, s):
    Hq, Hkv, rot = case["Hq"], case["Hkv"], case["rot"]
    x = s["qkv"].double().unflatten(1, (Hq + 2 * Hkv, H))
    k_pages, v_pages = s["k_pages"].double(), s["v_pages"].double()
    turn = torch.complex(*s["cos_sin"].double()[s["pos"].long()].chunk(2, 1))
    # where the two parts of each rotated pair stand in a head
    pair = torch.arange(rot, device=DEV)
    pair = pair.view(-1, 2).t() if case["interleaved"] else pair.view(2, -1)
    for h in range(Hq + Hkv):
        y = x[:, h]
        w = s["wq"] if h < Hq else s["wk"]
        if w is not None:
            y = y / ((y ** 2).sum(1, keepdim=True) / H + 1e-6).sqrt() * w.double()
        z = torch.complex(y[:, pair[0]], y[:, pair[1]]) * turn
        y = y.clone()
        y[:, pair[0]], y[:, pair[1]] = z.real, z.imag
        x[:, h] = y
    slots = s["slots"]
    for h in range(Hkv):
        k_pages.permute(0, 2, 1)[slots[:, h] // P, slots[:, h] % P] = x[:, Hq + h]
        v_pages.permute(0, 2, 1)[slots[:, h] // P, slots[:, h] % P] = x[:, Hq + Hkv + h]
    return {"q": x[:, :Hq].contiguous(), "k_pages": k_pages, "v_pages": v_pages}


def _exact_chunk(case, s):
    q, G = s["q"].double(), case["Hq"] // case["Hkv"]
    out = torch.empty_like(q)
    lse = torch.empty(q.shape[:2], dtype=torch.float64, device=DEV)
    cu, ctx = s["cu"].tolist(), s["ctx"].tolist()
    for b in range(case["B"]):
        lo, hi, n = cu[b], cu[b + 1], ctx[b]
        key = torch.arange(n, device=DEV)
        for h in range(case["Hkv"]):
            ids = s["table"][b, h, :_pages(n)].long()
            k = torch.cat(list(s["k_pages"][ids]), 1)[:, :n].double()
            v = torch.cat(list(s["v_pages"][ids]), 1)[:, :n].double()
            for at in range(lo, hi, 512):            # 512 tokens at a time
                end = min(hi, at + 512)
                last = n - (hi - lo) + torch.arange(at - lo, end - lo, device=DEV)
                for g in range(h * G, (h + 1) * G):
                    z = (q[at:end, g] @ k) / H ** 0.5
                    z = z.masked_fill(key[None] > last[:, None], -math.inf)
                    e = torch.logsumexp(z, 1)
                    lse[at:end, g] = e
                    out[at:end, g] = (z - e[:, None]).exp() @ v.t()
    return {"out": out, "lse": lse}
