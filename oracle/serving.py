"""The operators around attention in a serving step, in plain numpy and Python:
page assignment and draft verification in whole numbers, the QKV append in
float64, and attention of ragged chunks over a paged cache in float64."""
from __future__ import annotations

import math

import numpy as np

from . import attention as at

PAGE = 256
UNIT = 1 << 40


def assign_pages(ctx_len, new_len, page_table, free_pages, n_rows):
    """Request after request -> (table, cu_new, positions, slots, ctx_out, n_taken)."""
    table = np.array(page_table, dtype=np.int64)
    B, Hkv, max_pages = table.shape
    cu = [0]
    positions = np.full(n_rows, -1, dtype=np.int64)
    slots = np.full((n_rows, Hkv), -1, dtype=np.int64)
    ctx_out = []
    asked = taken = row = 0
    for b in range(B):
        ctx, new = int(ctx_len[b]), int(new_len[b])
        rows = max(new, 0)
        fits = ctx >= 0 and new >= 0 and ctx + new <= max_pages * PAGE and row + rows <= n_rows
        if fits:
            held = -(-ctx // PAGE)
            need = -(-(ctx + new) // PAGE) - held
            start = asked
            asked += need * Hkv
            if need and asked > len(free_pages):
                fits = False
            elif need:
                taken = asked
                for i in range(need):
                    for h in range(Hkv):
                        table[b, h, held + i] = free_pages[start + i * Hkv + h]
        if fits:
            for i in range(rows):
                pos = ctx + i
                positions[row + i] = pos
                slots[row + i] = table[b, :, pos // PAGE] * PAGE + pos % PAGE
        row += rows
        cu.append(min(row, n_rows))
        ctx_out.append(ctx + new if fits else ctx)
    return table, np.array(cu), positions, slots, np.array(ctx_out), taken


def norm_rotate(x, weight, eps, cos, sin, interleaved):
    """x [rows, heads, 128] float64; cos, sin [rows, rot / 2] (rot 0: no rotation)."""
    y = np.array(x, dtype=np.float64)
    if weight is not None:
        y = y / np.sqrt(np.mean(y * y, axis=-1, keepdims=True) + eps) * weight.astype(np.float64)
    half = cos.shape[1]
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        c, s = cos[:, i, None], sin[:, i, None]
        ya, yb = y[..., a].copy(), y[..., b].copy()
        y[..., a] = ya * c - yb * s
        y[..., b] = yb * c + ya * s
    return y


def verify_drafts(p, q, draft, n_draft, u):
    """p [B, T + 1, V], q [B, T, V] or None, float32 -> (tokens [B, T + 1], accepted [B])."""
    B, T = draft.shape
    V = p.shape[2]
    tokens = np.full((B, T + 1), -1, dtype=np.int64)
    accepted = np.zeros(B, dtype=np.int64)
    f32 = np.float32

    def units(w):
        w = np.where(np.isnan(w), f32(0), w)
        w = np.minimum(np.maximum(w, f32(0)), f32(1)).astype(np.float64)
        return [int(v) for v in np.floor(w * UNIT)]

    with np.errstate(invalid="ignore"):
        for b in range(B):
            nd = T if n_draft is None else min(max(int(n_draft[b]), 0), T)
            n = 0
            while n < nd:
                x = int(draft[b, n])
                if not 0 <= x < V:
                    break
                qx = f32(1) if q is None else f32(q[b, n, x])
                if not f32(u[b, n]) * qx < f32(p[b, n, x]):
                    break
                tokens[b, n] = x
                n += 1
            accepted[b] = n
            w = units(p[b, n])
            if n < nd:
                if q is not None:
                    left = units(p[b, n].astype(f32) - q[b, n].astype(f32))
                else:
                    left = list(w)
                    if 0 <= int(draft[b, n]) < V:
                        left[int(draft[b, n])] = 0
                if sum(left) > 0:
                    w = left
            total = sum(w)
            uf = float(u[b, T])
            step = 0 if math.isnan(uf) else min(max(int(min(max(uf, -1.0), 2.0) * (1 << 24)), 0), (1 << 24) - 1)
            limit = total * step >> 24
            run = 0
            for k, v in enumerate(w):
                run += v
                if run > limit:
                    tokens[b, n] = k
                    break
    return tokens, accepted


def chunk_attention(q, cu_q, k_pages, v_pages, page_table, ctx_len, n_kv_heads, sm_scale, causal):
    """q [rows, Hq, 128] float64 -> (out [rows, Hq, 128], lse [rows, Hq]); rows that
    see no key give 0 and -inf, rows behind the last request NaN."""
    rows, Hq, D = q.shape
    G = Hq // n_kv_heads
    out = np.full(q.shape, np.nan)
    lse = np.full((rows, Hq), np.nan)
    for b in range(len(ctx_len)):
        lo, hi, n = int(cu_q[b]), int(cu_q[b + 1]), int(ctx_len[b])
        T = hi - lo
        if T == 0:
            continue
        seen = np.clip(n - T + 1 + np.arange(T), 0, None) if causal else np.full(T, n)
        for h in range(n_kv_heads):
            ids = page_table[b, h, :-(-n // PAGE)]
            k = at.pages_to_seq(k_pages[ids])[:n] if n else np.zeros((0, D))
            v = at.pages_to_seq(v_pages[ids])[:n] if n else np.zeros((0, D))
            for g in range(G):
                s = q[lo:hi, h * G + g] @ k.T * sm_scale
                s = np.where(np.arange(n) < seen[:, None], s, -np.inf)
                m = np.max(s, axis=1, initial=-np.inf)
                m0 = np.where(np.isneginf(m), 0.0, m)
                e = np.exp(s - m0[:, None])
                l = e.sum(axis=1)
                safe = np.where(l == 0, 1.0, l)
                out[lo:hi, h * G + g] = e @ v / safe[:, None]
                with np.errstate(divide="ignore"):
                    lse[lo:hi, h * G + g] = m0 + np.log(l)
    return out, lse


def token_logprobs(logits, tokens, n_top):
    """logits [N, V] float64 -> (log probability of each token, entropy, ids and log
    probabilities of the n_top largest, the lower id first where they are equal)."""
    N, V = logits.shape
    logprob, entropy = np.full(N, -np.inf), np.zeros(N)
    ids, top = np.zeros((N, n_top), dtype=np.int64), np.zeros((N, n_top))
    for r in range(N):
        x = logits[r]
        ids[r] = np.argsort(-x, kind="stable")[:n_top]
        m = x.max()
        if m == -np.inf:
            top[r] = -np.inf
            continue
        d = x - m
        e = np.exp(d)
        log_s = math.log(e.sum())
        top[r] = d[ids[r]] - log_s
        if 0 <= tokens[r] < V:
            logprob[r] = d[tokens[r]] - log_s
        entropy[r] = log_s - np.sum(e[e > 0] * d[e > 0]) / e.sum()
    return logprob, entropy, ids, top
