"""Cases that measure serving over a paged cache held in 8 bits, and the log
probabilities of a step's tokens.

A page holds 256 tokens of one KV head, token-major [256 tokens][128 channels], as
E4M3 codes; each block of 32 tokens has one scale, a power of two 2^(s - 127), s a
byte in scales[page][0: keys, 1: values][8 blocks].  A step normalises and rotates
its new queries and keys and quantises the new keys and values into their blocks
(``append8``), attends from one or a few tokens of every request (``decode8``) or
from ragged chunks of new tokens (``chunk8``) to the paged cache, and gives the log
probabilities of tokens under their logits, the entropies and the most likely
alternatives (``logprobs``).

``run`` computes each operator in its plain form (elementary torch operations
in 32 bits) or, where ``own`` is true, calls the framework's kernels; both take
what ``prepare`` gives.
"""
import math

import torch

own = False

H, P, C = 128, 256, 32
DEV = "cuda"
TOP = 448.0                  # largest E4M3 value
S_LO, S_HI = 74, 198         # scale bytes that a block may have


def listed():
    return [
        # the new tokens of one decode step of 64 requests (Llama-3-8B-shaped heads): one token into a block of each
        dict(name="append8 decode step", op="append8", B=64, Hq=32, Hkv=8, max_new=1, norm=False, rot=128,
             interleaved=False, max_ctx=16384),
        # a 4K chunk with query and key norms (Qwen3-235B-shaped heads), from few requests at odd places
        dict(name="append8 chunk", op="append8", B=5, Hq=16, Hkv=4, max_new=1200, norm=True, rot=128,
             interleaved=False, max_ctx=131072),
        # the prompts of a prefill wave, half of each head rotated in neighbouring pairs
        dict(name="append8 prompt wave", op="append8", B=24, Hq=32, Hkv=8, max_new=2800, norm=True, rot=64,
             interleaved=True, max_ctx=8000),
        # one request's next token after a short prompt
        dict(name="decode8 one request", op="decode8", B=1, T=1, Hq=32, Hkv=8, max_ctx=983),
        # a decode step of a batch with contexts of all lengths
        dict(name="decode8 batch", op="decode8", B=48, T=1, Hq=32, Hkv=8, max_ctx=16383),
        # verification of four drafts a request (Qwen3-235B-shaped heads)
        dict(name="decode8 verification", op="decode8", B=8, T=5, Hq=16, Hkv=4, max_ctx=32000),
        # one token of four requests at the end of 128K contexts (Llama-3-70B-shaped heads)
        dict(name="decode8 long contexts", op="decode8", B=4, T=1, Hq=64, Hkv=8, max_ctx=131071),
        # chunked prefill of several requests at once, contexts of odd lengths
        dict(name="chunk8 ragged prefill", op="chunk8", B=6, Hq=32, Hkv=8, max_new=1024, max_ctx=7000),
        # a 2K chunk at the end of a 128K context (one Qwen3-235B-shaped layer)
        dict(name="chunk8 long context", op="chunk8", B=1, Hq=16, Hkv=4, max_new=2048, max_ctx=129024),
        # the sampled token of one request, with five alternatives
        dict(name="logprobs one token", op="logprobs", N=1, V=32000, dtype="float32", top=5, masked=False),
        # a decode step of 64 requests over a large vocabulary, twenty alternatives
        dict(name="logprobs decode step", op="logprobs", N=64, V=151936, dtype="float32", top=20, masked=False),
        # the log probabilities of a 2K prompt, no alternatives
        dict(name="logprobs prompt", op="logprobs", N=2047, V=128256, dtype="bfloat16", top=0, masked=False),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["append8", "decode8", "decode8", "chunk8", "logprobs"])
    if op == "logprobs":
        V = _log_int(rng, 500, 262144)
        N = _log_int(rng, 1, max(1, min(4096, 250000000 // V)))
        return dict(op=op, N=N, V=V, dtype=rng.choice(["float32", "bfloat16"]), top=rng.choice([0, 1, 5, 8, 20, 32]),
                    masked=rng.random() < 0.2)
    Hkv, G = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 5, 8])
    if op == "append8":
        B = _log_int(rng, 1, 128)
        most = max(1, 600000 // B // (Hkv * (G + 2)))
        return dict(op=op, B=B, Hq=G * Hkv, Hkv=Hkv, max_new=_log_int(rng, 1, min(8192, most)), norm=rng.random() < 0.6,
                    rot=rng.choice([128, 128, 64, 32]), interleaved=rng.random() < 0.4, max_ctx=_log_int(rng, 10, 60000))
    if op == "decode8":
        B = _log_int(rng, 1, 200)
        T = rng.choice([1, 1, 1, rng.randrange(2, 10)])
        max_ctx = _log_int(rng, max(1, T), max(300, min(200000, 3500000 // (B * Hkv))))
        return dict(op=op, B=B, T=T, Hq=G * Hkv, Hkv=Hkv, max_ctx=max_ctx)
    B = _log_int(rng, 1, 24)
    max_ctx = _log_int(rng, 1, 131072 // B)
    most = max(1, int(2.0e9) // (B * G * Hkv * (max_ctx + 2048)))
    return dict(op=op, B=B, Hq=G * Hkv, Hkv=Hkv, max_new=_log_int(rng, 1, min(4096, most)), max_ctx=max_ctx)


# ----------------------------------------------------------------------------- inputs


def _lengths(case):
    """New and earlier tokens of each request (host lists), the case's own: the first
    request is the longest, the others spread below it; in a batch of chunks every
    third one decodes a single token."""
    B, new_hi, ctx_hi = case["B"], case.get("max_new", 1), case["max_ctx"]
    rng = torch.Generator().manual_seed(B)
    new, ctx = [new_hi], [ctx_hi]
    for b in range(1, B):
        new.append(1 if b % 3 == 2 else max(1, int(new_hi * (0.25 + 0.75 * float(torch.rand((), generator=rng))))))
        ctx.append(int(ctx_hi * (0.1 + 0.9 * float(torch.rand((), generator=rng)))))
    return new, ctx


def _pages(n):
    return -(-n // P)


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _table(lens, Hkv, order):
    """[B][Hkv][max_pages] page ids taken from a shuffled order, 0 past each request's last page."""
    table = torch.zeros((len(lens), Hkv, max(_pages(n) for n in lens)), dtype=torch.int32)
    at = 0
    for b, n in enumerate(lens):
        k = _pages(n)
        table[b, :, :k] = order[at:at + Hkv * k].view(Hkv, k)
        at += Hkv * k
    return table.to(DEV)


def _scale_bytes(top):
    """The smallest s with top <= 448 * 2^(s - 127), within the bytes that are allowed."""
    m, e = torch.frexp(top)
    return torch.where(top > 0, e - 9 + (m > 0.875) + 127, S_LO).clamp(S_LO, S_HI)


def _pow2(e):
    return torch.ldexp(torch.ones((), device=DEV), e)


def _pool(n, gpu):
    """Pages of keys or values: an offset for each channel (the caches' structure), tokens of several sizes."""
    offset = torch.randn(H, generator=gpu, device=DEV)
    codes = torch.empty(n, P, H, dtype=torch.float8_e4m3fn, device=DEV)
    scales = torch.empty(n, P // C, dtype=torch.uint8, device=DEV)
    for at in range(0, n, 2048):     # 64 Mi values at a time
        end = min(n, at + 2048)
        x = torch.randn(end - at, P // C, C, H, generator=gpu, device=DEV).add_(offset)
        x.mul_(torch.exp(0.2 * torch.randn(end - at, P // C, C, 1, generator=gpu, device=DEV)))
        s = _scale_bytes(x.abs().amax((2, 3)))
        codes[at:end] = (x * _pow2(127 - s)[..., None, None]).view(end - at, P, H).to(torch.float8_e4m3fn)
        scales[at:end] = s.to(torch.uint8)
    return codes, scales


def prepare(case, seed):
    cpu, gpu = torch.Generator().manual_seed(seed), torch.Generator(DEV).manual_seed(seed)
    s = {"case": case}
    op = case["op"]
    if op == "logprobs":
        N, V = case["N"], case["V"]
        logits = torch.randn(N, V, generator=gpu, device=DEV).mul_(2.5)
        if case["masked"]:           # a grammar that leaves a thousand tokens
            allowed = torch.rand(N, V, generator=gpu, device=DEV).topk(min(V, 1000)).indices
            logits += torch.full_like(logits, -math.inf).scatter_(1, allowed, 0.0)
        # sampled: the largest of the logits with Gumbel noise
        noise = torch.rand(N, V, generator=gpu, device=DEV).clamp_(1e-20, 1 - 1e-7).log_().neg_().log_().neg_()
        s["tokens"] = noise.add_(logits).argmax(1).to(torch.int32)
        s["logits"] = logits.to(getattr(torch, case["dtype"]))
        return s
    B, Hq, Hkv = case["B"], case["Hq"], case["Hkv"]
    new, ctx = _lengths(case)
    total = [a + b for a, b in zip(new, ctx)]
    if op == "append8":
        # only the pages that take new tokens, in a shuffled order; every request starts at its own place in a page
        n_rows = sum(new)
        touched = [(c % P) + n for n, c in zip(new, ctx)]
        n_pool = sum(Hkv * _pages(n) for n in touched) + 3
        table = _table(touched, Hkv, torch.randperm(n_pool, generator=cpu).to(torch.int32))
        seq = torch.repeat_interleave(torch.arange(B), torch.tensor(new)).to(DEV)
        first = torch.tensor([sum(new[:b]) for b in range(B)], device=DEV)
        i = torch.arange(n_rows, device=DEV) - first[seq]
        s["pos"] = (torch.tensor(ctx, device=DEV)[seq] + i).to(torch.int32)
        off = torch.tensor([c % P for c in ctx], device=DEV)[seq] + i
        page = table.long()[seq[:, None], torch.arange(Hkv, device=DEV)[None], (off // P)[:, None]]
        s["slots"] = page * P + (off % P)[:, None]
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
        s["q_out"] = torch.empty(n_rows, Hq, H, dtype=torch.bfloat16, device=DEV)
    else:
        if op == "decode8":          # the context holds the new tokens
            total = [max(case["T"], c) for c in ctx]
            s["q"] = torch.randn(B, case["T"], Hq, H, generator=gpu, device=DEV).to(torch.bfloat16)
            s["out"] = torch.empty(s["q"].shape, dtype=torch.float32, device=DEV)
        else:
            s["q"] = torch.randn(sum(new), Hq, H, generator=gpu, device=DEV).to(torch.bfloat16)
            s["out"] = torch.empty_like(s["q"])
            s["cu"] = _i32([sum(new[:b]) for b in range(B + 1)])
            s["max_new"] = max(new)
        s["ctx"] = _i32(total)
        s["lse"] = torch.empty(s["q"].shape[:-1], dtype=torch.float32, device=DEV)
        s["workspace"] = torch.empty(0, dtype=torch.uint8, device=DEV)
        n_pool = sum(Hkv * _pages(n) for n in total) + 2
        s["table"] = _table(total, Hkv, torch.randperm(n_pool, generator=cpu).to(torch.int32))
    s["k_pages"], k_scales = _pool(n_pool, gpu)
    s["v_pages"], v_scales = _pool(n_pool, gpu)
    s["scales"] = torch.stack([k_scales, v_scales], 1)
    return s


# ----------------------------------------------------------------------------- one pass


def run(s):
    op = s["case"]["op"]
    if own:
        return _own(op, s)
    return {"append8": _append, "decode8": _decode, "chunk8": _chunk, "logprobs": _logprobs}[op](s)


def _own(op, s):
    from progressive_kv_quantization_gb300 import lynx as L

    c = s["case"]
    if op == "append8":
        q = L.lynx_qkv_append_e4m3(s["qkv"], c["Hq"], c["Hkv"], s["cos_sin"], s["pos"], s["slots"], s["k_pages"],
                                   s["v_pages"], s["scales"], q_weight=s["wq"], k_weight=s["wk"],
                                   interleaved=c["interleaved"], q_out=s["q_out"])
        return {"q": q, "k_pages": s["k_pages"], "v_pages": s["v_pages"], "scales": s["scales"]}
    if op == "decode8":
        if s["workspace"].numel() == 0:   # kept by the program from its first call on
            n = L.lynx_decode_attn_e4m3_workspace_size(c["B"], c["T"], c["Hq"], c["Hkv"], H)
            s["workspace"] = torch.empty(n, dtype=torch.uint8, device=DEV)
        o, lse = L.lynx_decode_attn_e4m3(s["q"], s["k_pages"], s["v_pages"], s["scales"], s["table"], s["ctx"], c["Hkv"],
                                         causal=True, out=s["out"], lse=s["lse"], workspace=s["workspace"])
        return {"out": o, "lse": lse}
    if op == "chunk8":
        if s["workspace"].numel() == 0:
            n = L.lynx_chunk_attn_workspace_size(s["q"].shape[0], c["B"], c["Hq"], c["Hkv"], H)
            s["workspace"] = torch.empty(n, dtype=torch.uint8, device=DEV)
        o, lse = L.lynx_chunk_attn_e4m3(s["q"], s["cu"], s["k_pages"], s["v_pages"], s["scales"], s["table"], s["ctx"],
                                        c["Hkv"], causal=True, out=s["out"], lse=s["lse"], workspace=s["workspace"])
        return {"out": o, "lse": lse}
    logprob, entropy, ids, top = L.lynx_token_logprobs(s["logits"], s["tokens"], n_top=c["top"])
    return {"logprob": logprob, "entropy": entropy, "top_ids": ids, "top_logprobs": top}


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


def _write_blocks(x, slots, codes, scales):
    """Rows x [n, Hkv, 128] to their slots: a block's scale covers what it held in front
    of the first new token, rounded to the new scale where that grew, and the new tokens."""
    blocks = scales.numel()
    block = slots // C
    flat = block.flatten()
    top = torch.zeros(blocks, device=DEV).scatter_reduce(0, flat, x.abs().amax(-1).flatten(), "amax")
    first = torch.full((blocks,), C, dtype=torch.int64, device=DEV).scatter_reduce(0, flat, (slots % C).flatten(), "amin")
    old = scales.reshape(-1).to(torch.int32)
    need = _scale_bytes(top)
    new = torch.where(first == 0, need, torch.maximum(old, need))
    new = torch.where(first < C, new, old)
    held = codes.float().view(blocks, C, H)
    kept = (held * _pow2(old - new)[:, None, None]).to(torch.float8_e4m3fn).float()
    earlier = torch.arange(C, device=DEV) < torch.where(first < C, first, 0)[:, None]
    held = torch.where(earlier[..., None], kept, held)
    held.view(-1, H)[slots.flatten()] = (x * _pow2(127 - new[block])[..., None]).clamp(-TOP, TOP).view(-1, H)
    codes.copy_(held.view(codes.shape))
    scales.copy_(new.view(scales.shape))


def _append(s):
    """RMS norm of each query and key head, rotation by the row's position, and the
    keys and values quantised into the blocks of their slots."""
    c = s["case"]
    Hq, Hkv = c["Hq"], c["Hkv"]
    x = s["qkv"].view(-1, Hq + 2 * Hkv, H).float()
    cs = s["cos_sin"][s["pos"].long()]
    cos, sin = cs[:, :c["rot"] // 2], cs[:, c["rot"] // 2:]
    q = _norm_rotate(x[:, :Hq], s["wq"], cos, sin, c["interleaved"]).to(torch.bfloat16)
    k = _norm_rotate(x[:, Hq:Hq + Hkv], s["wk"], cos, sin, c["interleaved"])
    _write_blocks(k, s["slots"], s["k_pages"], s["scales"][:, 0])
    _write_blocks(x[:, Hq + Hkv:], s["slots"], s["v_pages"], s["scales"][:, 1])
    return {"q": q, "k_pages": s["k_pages"], "v_pages": s["v_pages"], "scales": s["scales"]}


def _keys(s, name, which):
    """The cache of every request and head as the values it stands for, [B, Hkv, S, 128]."""
    table = s["table"].long()
    B, Hkv, n = table.shape
    x = s[name][table].float().view(B, Hkv, n * P // C, C, H)
    e = s["scales"][:, which][table].to(torch.int32).view(B, Hkv, n * P // C, 1, 1)
    return x.mul_(_pow2(e - 127)).view(B, Hkv, n * P, H)


def _attend(qp, k, v, seen):
    """qp [B, Hkv, R, 128] over keys and values [B, Hkv, S, 128], row r of request b over
    its first seen[b, r] keys: outputs and log sums of exponentials."""
    scores = torch.matmul(qp, k.transpose(2, 3)).mul_(1 / math.sqrt(H))
    hidden = torch.arange(k.shape[2], device=DEV) >= seen[:, None, :, None]
    scores.masked_fill_(hidden, -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    prob = scores.sub_(top).exp_()
    total = prob.sum(-1, keepdim=True)
    o = torch.matmul(prob, v) / torch.where(total == 0, 1.0, total)
    return o, (total.log() + top).squeeze(-1)


def _decode(s):
    """softmax(scale q.k) v of each request's last T tokens over the keys up to their own."""
    q = s["q"]
    B, T, Hq, _ = q.shape
    Hkv = s["case"]["Hkv"]
    G = Hq // Hkv
    qp = q.float().view(B, T, Hkv, G, H).transpose(1, 2).reshape(B, Hkv, T * G, H)
    seen = s["ctx"].long()[:, None] - T + 1 + torch.arange(T, device=DEV).repeat_interleave(G)
    o, lse = _attend(qp, _keys(s, "k_pages", 0), _keys(s, "v_pages", 1), seen)
    return {"out": o.view(B, Hkv, T, G, H).transpose(1, 2).reshape(B, T, Hq, H),
            "lse": lse.view(B, Hkv, T, G).transpose(1, 2).reshape(B, T, Hq)}


def _chunk(s):
    """softmax(scale q.k) v of every new token over the keys up to its own position,
    the ragged batch padded to its longest request."""
    q = s["q"]
    N, Hq, _ = q.shape
    B, Hkv, T = s["case"]["B"], s["case"]["Hkv"], s["max_new"]
    G = Hq // Hkv
    cu, ctx = s["cu"].long(), s["ctx"].long()
    i = torch.arange(T, device=DEV)
    rows = (cu[:-1, None] + i).clamp(max=N - 1)
    qp = q[rows].float().view(B, T, Hkv, G, H).transpose(1, 2).reshape(B, Hkv, T * G, H)
    seen = (ctx - (cu[1:] - cu[:-1]) + 1)[:, None] + i.repeat_interleave(G)
    o, lse = _attend(qp, _keys(s, "k_pages", 0), _keys(s, "v_pages", 1), seen)
    o = o.view(B, Hkv, T, G, H).transpose(1, 2).reshape(B, T, Hq, H)
    lse = lse.view(B, Hkv, T, G).transpose(1, 2).reshape(B, T, Hq)
    r = torch.arange(N, device=DEV)
    seq = torch.searchsorted(cu, r, right=True) - 1
    at = r - cu[seq]
    return {"out": o[seq, at].to(torch.bfloat16), "lse": lse[seq, at]}


def _logprobs(s):
    """log softmax at the given tokens, its entropy, and its largest values (the lowest
    token first where they are equal)."""
    x, n_top = s["logits"].float(), s["case"]["top"]
    N, V = x.shape
    top = x.amax(1, keepdim=True)
    d = x - top
    p = d.exp()
    total = p.sum(1)
    log_total = total.log()
    entropy = log_total - torch.where(p > 0, p * d, 0.0).sum(1) / total
    logprob = d.gather(1, s["tokens"].long()[:, None])[:, 0] - log_total
    # by value, then by the token from behind: whole numbers in the order of the floats
    bits = (x + 0.0).view(torch.int32)
    order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long() * 2 ** 32 + (2 ** 32 - 1 - torch.arange(V, device=DEV))
    best = order.topk(n_top, dim=1).values
    ids = 2 ** 32 - 1 - (best & (2 ** 32 - 1))
    return {"logprob": logprob, "entropy": entropy, "top_ids": ids.to(torch.int32),
            "top_logprobs": d.gather(1, ids) - log_total[:, None]}


# ----------------------------------------------------------------------------- what a pass needs


def work(case):
    """Each input once, each output once; products and sums of the formulas."""
    if case["op"] == "logprobs":
        size = 4 if case["dtype"] == "float32" else 2
        return {"bytes": case["N"] * (case["V"] * size + 12 + 8 * case["top"]), "flops": 6 * case["N"] * case["V"]}
    new, ctx = _lengths(case)
    n, Hq, Hkv = sum(new), case["Hq"], case["Hkv"]
    page = 2 * H + 2 / C         # bytes of a token's key and value of one head, with their share of the scales
    if case["op"] == "append8":
        # the tokens that stand in front of the first new one in its block are read for the scale only where it
        # grows: the scales alone are counted
        return {"bytes": int(n * (4 * H * Hq + Hkv * (4 * H + page + 8) + 4 * case["rot"] + 4)),
                "flops": 8 * n * H * (Hq + Hkv) + 4 * n * H * Hkv}
    if case["op"] == "decode8":
        T = case["T"]
        held = sum(max(T, c) for c in ctx)
        return {"bytes": int(held * Hkv * page + case["B"] * T * Hq * (6 * H + 4)), "flops": 4 * H * Hq * T * held}
    seen = sum(a * b + a * (a + 1) // 2 for a, b in zip(new, ctx))
    held = sum(a + b for a, b in zip(new, ctx))
    return {"bytes": int(n * Hq * (4 * H + 4) + held * Hkv * page), "flops": 4 * H * Hq * seen}


# ----------------------------------------------------------------------------- the definition in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append8":
        return _exact_append(case, s)
    return _exact_logprobs(case, s) if case["op"] == "logprobs" else _exact_attention(case, s)


def _exact_append(case, s):
    """Queries, and the codes' values before they are rounded; the scales are whole numbers."""
    Hq, Hkv, rot = case["Hq"], case["Hkv"], case["rot"]
    x = s["qkv"].double().unflatten(1, (Hq + 2 * Hkv, H))
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
    grown = {}
    powers = 2.0 ** torch.arange(S_LO - 127, S_HI - 127, dtype=torch.float64, device=DEV)
    for which, name in enumerate(["k_pages", "v_pages"]):
        codes = s[name].double().flatten(0, 1)
        scales = s["scales"][:, which].long().flatten()
        for h in range(Hkv):
            slot, y = s["slots"][:, h], x[:, Hq + which * Hkv + h]
            block, row_of = (slot // C).unique(return_inverse=True)
            # a block's rows side by side, one column for each of its tokens
            peak = torch.zeros(block.numel(), C, dtype=torch.float64, device=DEV)
            new = torch.zeros(block.numel(), C, dtype=torch.bool, device=DEV)
            peak[row_of, slot % C] = y.abs().max(1).values
            new[row_of, slot % C] = True
            need = S_LO + (peak.max(1).values[:, None] / TOP > powers).sum(1)
            was = scales[block]
            now = torch.where(new[:, 0], need, torch.where(need > was, need, was))
            place = torch.arange(C, device=DEV)
            before = place < new.long().argmax(1, keepdim=True)
            at = (block[:, None] * C + place)[before]
            codes[at] *= (2.0 ** (was - now).double())[:, None].expand(-1, C)[before][:, None]
            codes[slot] = (y / (2.0 ** (now[row_of] - 127).double())[:, None]).clamp(-TOP, TOP)
        grown[name] = codes.view(s[name].shape)
    return {"q": x[:, :Hq].contiguous(), "k_pages": grown["k_pages"], "v_pages": grown["v_pages"], "scales": None}


def _exact_attention(case, s):
    q = s["q"].double()
    B, Hq, Hkv = case["B"], case["Hq"], case["Hkv"]
    G = Hq // Hkv
    rows = q.reshape(-1, Hq, H)
    out = torch.empty_like(rows)
    lse = torch.empty(rows.shape[:2], dtype=torch.float64, device=DEV)
    cu = s["cu"].tolist() if case["op"] == "chunk8" else [b * case["T"] for b in range(B + 1)]
    ctx = s["ctx"].tolist()
    size = 2.0 ** (s["scales"].double() - 127)
    for b in range(B):
        lo, hi, n = cu[b], cu[b + 1], ctx[b]
        key = torch.arange(n, device=DEV)
        for h in range(Hkv):
            ids = s["table"][b, h, :_pages(n)].long()
            k = torch.cat(list(s["k_pages"][ids].double()))[:n] * size[ids, 0].repeat_interleave(C)[:n, None]
            v = torch.cat(list(s["v_pages"][ids].double()))[:n] * size[ids, 1].repeat_interleave(C)[:n, None]
            for at in range(lo, hi, 512):            # 512 tokens at a time
                end = min(hi, at + 512)
                last = n - (hi - lo) + torch.arange(at - lo, end - lo, device=DEV)
                for g in range(h * G, (h + 1) * G):
                    z = (rows[at:end, g] @ k.t()) / H ** 0.5
                    z = z.masked_fill(key[None] > last[:, None], -math.inf)
                    e = torch.logsumexp(z, 1)
                    lse[at:end, g] = e
                    out[at:end, g] = (z - e[:, None]).exp() @ v
    return {"out": out.view(q.shape), "lse": lse.view(q.shape[:-1])}


def _exact_logprobs(case, s):
    logprob, entropy, top = [], [], []
    for x, t in zip(s["logits"].split(64), s["tokens"].split(64)):
        y = torch.log_softmax(x.double(), 1)
        logprob.append(y[torch.arange(len(t), device=DEV), t.long()])
        entropy.append(torch.special.entr(y.exp()).sum(1))
        top.append(y.sort(1, descending=True).values[:, :case["top"]])
    return {"logprob": torch.cat(logprob), "entropy": torch.cat(entropy), "top_ids": None, "top_logprobs": torch.cat(top)}
