"""Closed forms that pin the oracle of the serving-step operators (oracle/serving.py)."""
import math

import numpy as np

from oracle import serving as sv


def test_assign_pages_small_batch_by_hand():
    # request 0: 255 cached + 3 new crosses into a second page; request 1: nothing new;
    # request 2: starts at 0
    table = np.full((3, 2, 2), -1)
    table[0, :, 0] = [7, 8]
    t, cu, pos, slots, ctx, taken = sv.assign_pages([255, 256, 0], [3, 0, 2], table, [20, 21, 22, 23, 24], 7)
    assert list(cu) == [0, 3, 3, 5] and list(pos) == [255, 256, 257, 0, 1, -1, -1]
    assert t[0].tolist() == [[7, 20], [8, 21]] and t[2].tolist() == [[22, -1], [23, -1]]
    assert slots[:, 0].tolist() == [7 * 256 + 255, 20 * 256, 20 * 256 + 1, 22 * 256, 22 * 256 + 1, -1, -1]
    assert slots[2, 1] == 21 * 256 + 1 and list(ctx) == [258, 256, 2] and taken == 4


def test_assign_pages_refuses_by_running_sum():
    table = np.full((4, 1, 4), -1)
    # request 0 takes 1 of 2 pages, request 1 wants 2 and is refused, request 2 wants 1 and
    # is refused too (its running sum is 4), request 3 needs none
    t, cu, pos, slots, ctx, taken = sv.assign_pages([0, 0, 0, 5], [10, 300, 10, 1], table, [3, 4], 400)
    assert taken == 1 and list(ctx) == [10, 0, 0, 6] and t[0, 0, 0] == 3 and (t[1:] == -1).all()
    assert (pos[10:320] == -1).all() and pos[320] == 5


def test_norm_rotate_keeps_lengths_and_turns_by_the_angle():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((3, 2, 128))
    ang = rng.uniform(0, 6, (3, 64))
    y = sv.norm_rotate(x, None, 0.0, np.cos(ang), np.sin(ang), False)
    assert np.allclose(np.linalg.norm(x, axis=-1), np.linalg.norm(y, axis=-1))
    z = (x[..., :64] + 1j * x[..., 64:]) * np.exp(1j * ang)[:, None]
    assert np.allclose(y, np.concatenate([z.real, z.imag], -1))
    n = sv.norm_rotate(x, np.ones(128), 0.0, np.ones((3, 0)), np.ones((3, 0)), False)
    assert np.allclose((n * n).mean(-1), 1)


def test_verify_drafts_follows_the_target_distribution():
    """Speculative sampling returns the target's distribution whatever the draft's is."""
    rng = np.random.default_rng(1)
    V, N = 5, 20000
    p = np.array([0.4, 0.1, 0.2, 0.25, 0.05], np.float32)
    q = np.array([0.1, 0.3, 0.3, 0.2, 0.1], np.float32)
    draft = rng.choice(V, size=(N, 1), p=q.astype(np.float64) / q.sum(dtype=np.float64))
    u = rng.random((N, 2)).astype(np.float32)
    tok, n = sv.verify_drafts(np.broadcast_to(p, (N, 2, V)), np.broadcast_to(q, (N, 1, V)), draft, None, u)
    freq = np.bincount(tok[:, 0], minlength=V) / N
    # five binomial frequencies of N draws: within 5 standard deviations
    assert np.all(np.abs(freq - p) < 5 * np.sqrt(p * (1 - p) / N))
    assert np.isclose(n.mean(), np.minimum(p, q).sum(), atol=5 * math.sqrt(0.25 / N))


def test_verify_drafts_edges():
    p = np.array([[[0.5, 0.5], [0.25, 0.75]]], np.float32)
    # certain draft, rejected: its weight is gone
    tok, n = sv.verify_drafts(p, None, np.array([[0]]), None, np.array([[0.9, 0.0]], np.float32))
    assert tok.tolist() == [[1, -1]] and n[0] == 0
    # accepted: the second row decides, running sum 0.25 <= 0.25 goes to the next
    tok, n = sv.verify_drafts(p, None, np.array([[0]]), None, np.array([[0.1, 0.25]], np.float32))
    assert tok.tolist() == [[0, 1]] and n[0] == 1
    # p == q at the rejection: no residual weight, drawn from p
    tok, n = sv.verify_drafts(p, p[:, :1], np.array([[7]]), None, np.array([[0.1, 0.6]], np.float32))
    assert tok.tolist() == [[1, -1]] and n[0] == 0


def test_chunk_attention_equal_keys_and_empty_rows():
    q = np.ones((3, 2, 128))
    k = np.zeros((1, 128, 256))
    v = np.broadcast_to(np.arange(256.0), (1, 128, 256))
    o, l = sv.chunk_attention(q, [0, 3], k, v, np.zeros((1, 1, 1), int), [2], 1, 0.1, True)
    assert np.allclose(o[0], 0) and np.isneginf(l[0]).all()           # sees 2 - 3 + 1 = 0 keys
    assert np.allclose(o[1], 0) and np.allclose(l[1], 0) and np.allclose(o[2], 0.5) and np.allclose(l[2], math.log(2))
