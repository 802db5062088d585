"""GPU parity of the serving-step operators: page assignment and draft
verification equal the oracle in every value (they compute whole numbers), the
QKV append is within its rounding of the float64 definition."""
import numpy as np
import pytest
import torch

from oracle import serving as sv
from progressive_kv_quantization_gb300 import lynx as L

pytestmark = pytest.mark.gpu


def cu(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t if dtype is None else t.to(dtype)


def status_ok():
    torch.cuda.synchronize()
    L.lynx_device_status()


# --------------------------------------------------------------- page assignment

def assign_case(B, Hkv, max_pages, n_free, seed, new_hi, zero=0.2):
    rng = np.random.default_rng(seed)
    ctx = rng.integers(0, max_pages * 256 + 1, B)
    ctx[rng.random(B) < 0.2] //= 256
    ctx[rng.random(B) < 0.2] = rng.integers(0, max_pages + 1) * 256
    new = rng.integers(1, new_hi + 1, B)
    new[rng.random(B) < zero] = 0
    new = np.minimum(new, max_pages * 256 - ctx)
    ids = rng.permutation(B * Hkv * max_pages + n_free)
    table = ids[:B * Hkv * max_pages].reshape(B, Hkv, max_pages).copy()
    return ctx, new, table, ids[B * Hkv * max_pages:][:n_free]


def check_assign(ctx, new, table, free, n_rows):
    t = cu(table, torch.int32)
    got = L.lynx_assign_pages(cu(ctx, torch.int32), cu(new, torch.int32), t, cu(free, torch.int32), n_rows)
    torch.cuda.synchronize()
    rt, rcu, rpos, rslots, rctx, rtaken = sv.assign_pages(ctx, new, table, list(free), n_rows)
    g = [x.cpu().numpy() for x in got]
    assert np.array_equal(t.cpu().numpy(), rt)
    assert np.array_equal(g[0], rcu) and np.array_equal(g[1], rpos) and np.array_equal(g[2], rslots)
    assert np.array_equal(g[3], rctx) and g[4][0] == rtaken
    return got


@pytest.mark.parametrize("B,Hkv,max_pages,new_hi,pad", [
    (1, 1, 1, 1, 0), (1, 3, 5, 700, 3), (7, 8, 4, 1, 0), (64, 8, 9, 1, 5), (33, 2, 6, 900, 129), (255, 1, 3, 40, 0),
    (256, 5, 2, 300, 1), (257, 4, 3, 2, 0), (700, 1, 2, 90, 1000), (1500, 2, 2, 3, 0)])
def test_assign_pages_equals_the_oracle(cuda_device, B, Hkv, max_pages, new_hi, pad):
    for seed in range(3):
        ctx, new, table, free = assign_case(B, Hkv, max_pages, B * Hkv * max_pages, 10 * B + seed, new_hi)
        check_assign(ctx, new, table, free, int(new.sum()) + pad)
    status_ok()


@pytest.mark.parametrize("n_free", [0, 1, 5, 64])
def test_assign_pages_refuses_requests_that_do_not_fit(cuda_device, n_free):
    ctx, new, table, free = assign_case(90, 2, 4, n_free, n_free, 500)
    check_assign(ctx, new, table, free, int(new.sum()))              # the free list runs out
    ctx, new, table, free = assign_case(90, 2, 4, 720, 5, 500)
    check_assign(ctx, new, table, free, int(new.sum()) // 2)         # the rows run out
    check_assign(ctx, np.zeros_like(new), table, free, 4)            # nothing new: every row behind
    check_assign(ctx, new, table, free, 0)                           # no rows at all
    status_ok()


def test_assign_pages_lengths_outside_the_table_are_refused_and_reported(cuda_device):
    ctx = np.array([-1, 10, 500, 512, 2 ** 31 - 1])
    new = np.array([4, -3, 13, 1, 2 ** 31 - 1])
    table = np.arange(10).reshape(5, 1, 2)
    check_assign(ctx, new, table, np.arange(100, 120), 60)
    torch.cuda.synchronize()
    with pytest.raises(L.LynxError, match="ctx_len"):
        L.lynx_device_status()


def test_assign_pages_takes_the_rest_of_a_list(cuda_device):
    """Two steps in a row: the second takes its ids from the list behind the first's."""
    Hkv, max_pages = 2, 4
    table = np.full((3, Hkv, max_pages), -1)
    free = np.arange(50, 50 + 3 * Hkv * max_pages)
    t, f = cu(table, torch.int32), cu(free, torch.int32)
    ctx, new = np.array([0, 0, 0]), np.array([256, 255, 300])
    out = L.lynx_assign_pages(cu(ctx, torch.int32), cu(new, torch.int32), t, f, 811)
    taken = int(out[4])
    assert taken == 8
    new2 = np.array([1, 1, 212])
    out2 = L.lynx_assign_pages(out[3], cu(new2, torch.int32), t, f[taken:], 214)
    rt, *_ , rctx, rtaken = sv.assign_pages(ctx, new, table, list(free), 811)
    rt, _, _, rslots, rctx, rtaken = sv.assign_pages(rctx, new2, rt, list(free[taken:]), 214)
    assert np.array_equal(t.cpu().numpy(), rt) and np.array_equal(out2[2].cpu().numpy(), rslots)
    assert int(out2[4]) == rtaken == 2
    status_ok()


@pytest.mark.parametrize("huge", [2 ** 30 - 3, 2 ** 30, 2 ** 30 + 1, 2 ** 31 - 1])
@pytest.mark.parametrize("at", [1, 2, 31, 32, 33, 64, 255, 256, 257, 300])
def test_assign_pages_a_huge_request_is_refused_alone(cuda_device, at, huge):
    """Its length passes what the running sums hold; the requests in front of it keep
    their rows and pages, those behind it that ask for nothing their lengths."""
    rng = np.random.default_rng(at)
    Hkv, max_pages, B = 2, 3, at + 6
    ctx = rng.integers(0, 600, B)
    new = rng.integers(0, 4, B)
    new[rng.random(B) < 0.3] = 150                     # some take fresh pages
    new = np.minimum(new, max_pages * 256 - ctx)
    new[0] = 5
    new[at:] = [huge, 0, 3, 0, huge, 0]
    ids = rng.permutation(2 * B * Hkv * max_pages)
    table = ids[:B * Hkv * max_pages].reshape(B, Hkv, max_pages)
    for behind in (0, 3, 200):
        got = check_assign(ctx, new, table, ids[B * Hkv * max_pages:], int(new[:at].sum()) + behind)
        assert int(got[3][0]) == ctx[0] + 5 and int(got[1][0]) == ctx[0]
    torch.cuda.synchronize()
    with pytest.raises(L.LynxError, match="ctx_len"):
        L.lynx_device_status()


def test_assign_pages_a_huge_request_that_its_table_would_hold(cuda_device):
    """The same with a length that is in order: its rows do not fit, the others' do."""
    max_pages = (1 << 22) + 1
    ctx, new = np.array([0, 10, 255, 7]), np.array([4, 3, 2 ** 30, 0])
    check_assign(ctx, new, np.zeros((4, 1, max_pages), dtype=np.int64), np.arange(100, 103), 10)
    status_ok()


# --------------------------------------------------------------- QKV append

def check_append(n_rows, Hq, Hkv, rot, interleaved, norm, seed, pad_cols=0, skip=0.0, run=True):
    rng = np.random.default_rng(seed)
    width = (Hq + 2 * Hkv) * 128
    wide = torch.from_numpy(rng.standard_normal((n_rows, width + pad_cols)).astype(np.float32)
                            * rng.uniform(0.01, 20, (1, width + pad_cols)).astype(np.float32)).bfloat16().cuda()
    qkv = wide[:, :width]
    max_pos = 5000
    wq = wk = None
    if norm:
        wq, wk = rng.uniform(-2, 2, 128).astype(np.float32), rng.uniform(-2, 2, 128).astype(np.float32)
    cos_sin = None
    c = s = np.zeros((n_rows, 0))
    pos = rng.integers(0, max_pos, n_rows)
    if rot:
        ang = rng.uniform(0, 2 * np.pi, (max_pos, rot // 2))
        table = np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)
        cos_sin = cu(table)
        c, s = table[pos, :rot // 2].astype(np.float64), table[pos, rot // 2:].astype(np.float64)
    n_pool = max(2, -(-n_rows * Hkv // 256) + Hkv + 1)
    if run:      # chunks that follow one another, at an odd start
        start = int(rng.integers(0, 200))
        slots = (start + np.arange(n_rows))[:, None] + np.arange(Hkv) * ((n_rows + start) // 256 + 1) * 256
        n_pool = int(slots.max()) // 256 + 1
    else:        # scattered, all different
        slots = rng.permutation(n_pool * 256)[:n_rows * Hkv].reshape(n_rows, Hkv)
    slots = slots.astype(np.int64)
    off = rng.random(n_rows) < skip
    pos_in = np.where(off, -1, pos)
    slots_in = slots.copy()
    if skip and n_rows > 1:
        slots_in[n_rows // 2, Hkv - 1] = -1          # one head of one row is not kept
    k_pages = torch.randn(n_pool, 128, 256, device="cuda").bfloat16()
    v_pages = torch.randn(n_pool, 128, 256, device="cuda").bfloat16()
    k0, v0 = k_pages.clone(), v_pages.clone()
    q_out = torch.full((n_rows, Hq, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    got = L.lynx_qkv_append(qkv, Hq, Hkv, cos_sin, cu(pos_in, torch.int32), cu(slots_in), k_pages, v_pages,
                            q_weight=None if wq is None else cu(wq), k_weight=None if wk is None else cu(wk),
                            norm_eps=1e-5, interleaved=interleaved, q_out=q_out)
    assert got is q_out
    status_ok()
    x = qkv.double().cpu().numpy().reshape(n_rows, Hq + 2 * Hkv, 128)

    def near(g, x, w):
        """float32 work, one rounding to BF16: half a step of the value, and for the
        float32 part at most 32 roundings (a sum of squares over 8 values and four
        exchanges, a reciprocal root of 2 ulp, three products, a rotation) of 2^-24
        relative to the two parts that the rotation joins."""
        ref = sv.norm_rotate(x, w, 1e-5, c, s, interleaved)
        flat = np.abs(sv.norm_rotate(x, w, 1e-5, np.ones_like(c[:, :0]), np.zeros_like(s[:, :0]), interleaved))
        part = flat.copy()
        for i in range(rot // 2):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
            part[..., a] = part[..., b] = flat[..., a] + flat[..., b]
        lim = 2.0 ** -8 * np.abs(ref) + 2 * 32 * 2.0 ** -24 * part + 1e-38
        err = np.abs(g - ref)
        assert np.all(err <= lim), f"largest excess {np.max(err - lim)}"
    on = ~off
    g = q_out.double().cpu().numpy()
    c_all, s_all = c, s
    c, s = c_all[on], s_all[on]
    near(g[on], x[on][:, :Hq], wq)
    assert np.all(g[off] == 7.0)                     # skipped rows stay as they were
    kept = on[:, None] & (slots_in >= 0)
    kg = k_pages.permute(0, 2, 1).reshape(-1, 128)
    vg = v_pages.permute(0, 2, 1).reshape(-1, 128)
    r, h = np.nonzero(kept)
    c, s = c_all[r], s_all[r]
    near(kg[cu(slots[r, h])].double().cpu().numpy()[:, None], x[r, Hq + h][:, None], wk)
    assert np.array_equal(vg[cu(slots[r, h])].double().cpu().numpy(), x[r, Hq + Hkv + h])
    touched = torch.zeros(n_pool * 256, dtype=torch.bool, device="cuda")
    touched[cu(slots[r, h])] = True
    for a, b in ((kg, k0), (vg, v0)):                # nothing else was written
        b = b.permute(0, 2, 1).reshape(-1, 128)
        assert torch.equal(a[~touched].view(torch.int16), b[~touched].view(torch.int16))


@pytest.mark.parametrize("n_rows", [1, 2, 31, 32, 33, 257, 1000])
@pytest.mark.parametrize("Hq,Hkv,rot,interleaved,norm", [
    (4, 1, 128, False, True), (3, 3, 64, True, False), (9, 3, 32, False, True), (8, 2, 128, True, True),
    (2, 2, 96, False, False), (5, 1, 0, False, True), (1, 1, 16, False, False), (2, 1, 112, True, True)])
def test_append_matches_the_definition(cuda_device, n_rows, Hq, Hkv, rot, interleaved, norm):
    check_append(n_rows, Hq, Hkv, rot, interleaved, norm, n_rows + Hq, pad_cols=8 * (n_rows % 3),
                 skip=0.2 if n_rows > 30 else 0.0, run=n_rows % 2 == 1)


def test_append_many_rows(cuda_device):
    check_append(9001, 16, 4, 128, False, True, 3, pad_cols=64, skip=0.01)


def test_append_reports_positions_and_slots_outside(cuda_device):
    qkv = torch.randn(3, 3 * 128, device="cuda").bfloat16()
    table = torch.ones(10, 128, device="cuda")
    k = torch.zeros(1, 128, 256, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    q = torch.full((3, 1, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    pos = torch.tensor([1, 10, 2], dtype=torch.int32, device="cuda")
    slots = torch.tensor([[0], [1], [2]], device="cuda")
    L.lynx_qkv_append(qkv, 1, 1, table, pos, slots, k, v, q_out=q)
    with pytest.raises(L.LynxError, match="= 4"):
        L.lynx_device_status()
    assert (q[1] == 5).all() and (k[0, :, 1] == 0).all() and (k[0, :, 2] != 0).any()
    pos[1] = 9
    slots[1] = 256
    L.lynx_qkv_append(qkv, 1, 1, table, pos, slots, k, v, q_out=q)
    with pytest.raises(L.LynxError, match="= 5"):
        L.lynx_device_status()
    assert (k[0, :, 1] == 0).all()


def test_append_position_offsets_pass_32_bits(cuda_device):
    """A slot beyond 2^31 elements of the pool (70,000 pages, 4.6 GB)."""
    k = torch.zeros(70000, 128, 256, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros(70000, 128, 256, dtype=torch.bfloat16, device="cuda")
    qkv = torch.randn(1, 3 * 128, device="cuda").bfloat16()
    slot = torch.tensor([[69999 * 256 + 255]], device="cuda")
    L.lynx_qkv_append(qkv, 1, 1, None, torch.zeros(1, dtype=torch.int32, device="cuda"), slot, k, v)
    status_ok()
    assert torch.equal(k[69999, :, 255], qkv[0, 128:256]) and torch.equal(v[69999, :, 255], qkv[0, 256:])
    assert int((k != 0).any(2).any(1).sum()) == 1


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("rot,interleaved", [(0, False), (0, True), (64, False), (64, True), (112, False), (16, True)])
def test_append_keeps_infinities_and_nan_to_their_channels(cuda_device, rot, interleaved, norm):
    """A channel that is not finite reaches the other one of its rotated pair, and under a
    norm what the formula says; channels that are neither rotated nor normalised are
    copied, every bit."""
    Hq, Hkv, n_rows = 2, 1, 128 * 3
    rng = np.random.default_rng(rot)
    x = torch.from_numpy(rng.standard_normal((n_rows, Hq + 2 * Hkv, 128)).astype(np.float32)).bfloat16()
    x[1::7, :, 5::9] = -0.0
    odd = torch.tensor([float("inf"), float("-inf"), float("nan")]).bfloat16()
    for r in range(n_rows):                                  # one channel a row
        x[r, :, r // 3] = odd[r % 3]
    x = x.cuda()
    max_pos = 50
    ang = rng.uniform(0.1, 1.4, (max_pos, rot // 2))
    table = np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)
    pos = rng.integers(0, max_pos, n_rows)
    w = rng.uniform(0.5, 2, 128).astype(np.float32) if norm else None
    k = torch.zeros(2, 128, 256, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    slots = torch.arange(n_rows, device="cuda").view(-1, 1)
    q = L.lynx_qkv_append(x.view(n_rows, -1), Hq, Hkv, cu(table) if rot else None, cu(pos, torch.int32), slots, k, v,
                          q_weight=None if w is None else cu(w), k_weight=None if w is None else cu(w), norm_eps=0.0,
                          interleaved=interleaved)
    status_ok()
    with np.errstate(invalid="ignore"):
        ref = sv.norm_rotate(x[:, :Hq + Hkv].double().cpu().numpy(), w, 0.0, table[pos, :rot // 2].astype(np.float64),
                             table[pos, rot // 2:].astype(np.float64), interleaved)
    kg = k.permute(0, 2, 1).reshape(-1, 1, 128)[:n_rows]
    vg = v.permute(0, 2, 1).reshape(-1, 1, 128)[:n_rows]
    bits = lambda t: t.contiguous().view(torch.int16)
    got = torch.cat([q, kg], 1)
    g = got.double().cpu().numpy()
    assert np.array_equal(np.isnan(g), np.isnan(ref))
    inf = np.isinf(ref)
    assert np.array_equal(np.isinf(g), inf) and np.array_equal(g[inf], ref[inf])
    fin = np.isfinite(ref)
    # half a BF16 step of the value, and the float32 part as in near(): |x| is below 6, times 2
    # for a weight, twice for a pair; a mean over values that are not finite leaves zeros
    assert np.all(np.abs(g[fin] - ref[fin]) <= 2.0 ** -8 * np.abs(ref[fin]) + 64 * 2.0 ** -24 * 24)
    if not norm:
        assert torch.equal(bits(got[..., rot:]), bits(x[:, :Hq + Hkv, rot:]))
    assert torch.equal(bits(vg), bits(x[:, Hq + Hkv:]))


# --------------------------------------------------------------- draft verification

def probs(rng, shape, sharp):
    x = rng.standard_normal(shape) * sharp
    e = np.exp(x - x.max(-1, keepdims=True))
    return (e / e.sum(-1, keepdims=True)).astype(np.float32)


def check_verify(p, q, draft, n_draft, u, dtype=torch.float32, pad=0):
    def up(x):
        t = cu(x).to(dtype)
        if pad:
            wide = torch.full((*t.shape[:-1], t.shape[-1] + pad), float("nan"), dtype=dtype, device="cuda")
            wide[..., :t.shape[-1]] = t
            t = wide[..., :t.shape[-1]]
        return t
    tp, tq = up(p), None if q is None else up(q)
    tok, n = L.lynx_verify_drafts(tp, tq, cu(draft, torch.int32), cu(u),
                                  n_draft=None if n_draft is None else cu(n_draft, torch.int32))
    rt, rn = sv.verify_drafts(tp.float().cpu().numpy(), None if q is None else tq.float().cpu().numpy(), draft, n_draft,
                              u)
    assert np.array_equal(n.cpu().numpy(), rn)
    assert np.array_equal(tok.cpu().numpy(), rt)
    return rn


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,T,V,pad", [(1, 1, 1, 0), (3, 2, 7, 0), (2, 5, 511, 1), (5, 4, 513, 3), (40, 3, 1000, 0),
                                       (2, 64, 2049, 0), (1, 3, 32001, 7), (300, 2, 600, 0), (90, 1, 5003, 1)])
def test_verify_equals_the_oracle(cuda_device, B, T, V, pad, dtype):
    rng = np.random.default_rng(B * T + V)
    p = probs(rng, (B, T + 1, V), 2.0)
    near = np.log(p[:, :T] + 1e-12) + 0.5 * rng.standard_normal((B, T, V))
    q = np.exp(near - near.max(-1, keepdims=True))
    q = (q / q.sum(-1, keepdims=True)).astype(np.float32)
    draft = np.array([[rng.choice(V, p=q[b, t].astype(np.float64) / q[b, t].sum(dtype=np.float64)) for t in range(T)]
                      for b in range(B)])
    u = rng.random((B, T + 1)).astype(np.float32)
    n_draft = rng.integers(-1, T + 2, B)
    check_verify(p, q, draft, None, u, dtype, pad)
    check_verify(p, q, draft, n_draft, u, dtype, pad)
    check_verify(p, None, draft, n_draft, u, dtype, pad)
    status_ok()


def test_verify_accepts_and_rejects_every_count(cuda_device):
    """Drafts that are certain up to the n-th: n = 0..64 accepted, ends of the random range."""
    T, V = 64, 300
    rng = np.random.default_rng(4)
    B = T + 1
    draft = rng.integers(0, V, (B, T))
    p = probs(rng, (B, T + 1, V), 1.0)
    q = probs(rng, (B, T, V), 1.0)
    for b in range(B):
        for t in range(T):
            p[b, t, draft[b, t]] = 0.9 if t < b else 0.0
            q[b, t, draft[b, t]] = 0.5
    for last in (0.0, 0.5, 1.0 - 2.0 ** -24, 1.0, -1.0, np.nan):
        u = rng.random((B, T + 1)).astype(np.float32)
        u[:, T] = last
        n = check_verify(p, q, draft, None, u)
        assert np.array_equal(n, np.arange(B))


def test_verify_rows_without_weight_and_odd_values(cuda_device):
    V, T = 1500, 2
    rng = np.random.default_rng(5)
    p = probs(rng, (8, T + 1, V), 1.0)
    q = p[:, :T].copy()                      # 0: the same row, no residual weight
    draft = rng.integers(0, V, (8, T))
    u = np.full((8, T + 1), 0.7, np.float32)
    u[:, 0] = 1.0                            # u q < p is false where q = p
    p[1] = 0.0                               # 1: no weight at all: token -1
    p[2] = np.nan
    p[3, 0, :] = -1.0                        # 3: negative counts as none
    p[3, 0, 77] = 0.25
    p[4, 0] = 0.0
    p[4, 0, V - 1] = 1.0                     # 4: all weight on the last id
    q[4, 0] = 0.0
    p[5, 0] = np.inf                         # 5: at most 1 each
    p[6, 0] = 1e-13                          # 6: below 2^-40: none
    draft[7] = [-1, V]                       # 7: ids outside the vocabulary
    check_verify(p, q, draft, None, u)
    check_verify(p, None, draft, None, u)
    status_ok()


def test_verify_large_vocabulary_limit(cuda_device):
    V = 1 << 20
    p = torch.zeros(2, 2, V, device="cuda")
    p[0, 0, V - 1] = 1e-6
    p[1, :, ::2] = 2.0 / V
    tok, n = L.lynx_verify_drafts(p, None, torch.zeros(2, 1, dtype=torch.int32, device="cuda"),
                                  torch.tensor([[0.5, 0.3], [0.9, 0.5]], device="cuda"))
    rt, rn = sv.verify_drafts(p.cpu().numpy(), None, np.zeros((2, 1), int),
                              None, np.array([[0.5, 0.3], [0.9, 0.5]], np.float32))
    assert np.array_equal(tok.cpu().numpy(), rt) and np.array_equal(n.cpu().numpy(), rn)
    with pytest.raises(L.LynxError, match="V="):
        L.lynx_verify_drafts(torch.zeros(1, 2, V + 1, device="cuda"), None,
                             torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.zeros(1, 2, device="cuda"))


def test_verify_many_requests_of_the_largest_vocabulary(cuda_device):
    """One CTA a request with all 4,096 of its runs: uniform rows, whose tokens follow
    from u alone (each weight is 2^20 units of a sum of 2^40)."""
    B, V = 200, 1 << 20
    p = torch.full((1, 2, V), 2.0 ** -20, dtype=torch.bfloat16, device="cuda").expand(B, 2, V)
    u = torch.rand(B, 2, generator=torch.Generator("cuda").manual_seed(4), device="cuda")
    u[0, 1], u[1, 1] = 0.0, 1.0 - 2.0 ** -24
    draft = torch.full((B, 1), -1, dtype=torch.int32, device="cuda")
    tok, n = L.lynx_verify_drafts(p, None, draft, u)
    want = (u[:, 1].double() * 2.0 ** 24).floor().long() >> 4
    assert torch.equal(tok[:, 0].long(), want) and (tok[:, 1] == -1).all() and (n == 0).all()


# --------------------------------------------------------------- graphs and streams

def test_operators_in_a_captured_graph(cuda_device):
    """The three operators captured and replayed with other lengths, rows and numbers."""
    B, Hkv, Hq, max_pages, n_rows = 4, 2, 4, 3, 40
    ctx, new = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    table = torch.zeros(B, Hkv, max_pages, dtype=torch.int32, device="cuda")
    free = torch.arange(B * Hkv * max_pages, 2 * B * Hkv * max_pages, dtype=torch.int32, device="cuda")
    k = torch.zeros(2 * B * Hkv * max_pages, 128, 256, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    qkv = torch.zeros(n_rows, (Hq + 2 * Hkv) * 128, dtype=torch.bfloat16, device="cuda")
    p = torch.zeros(B, 3, 900, device="cuda")
    u = torch.zeros(B, 3, device="cuda")
    draft = torch.zeros(B, 2, dtype=torch.int32, device="cuda")

    def step():
        a = L.lynx_assign_pages(ctx, new, table, free, n_rows)
        q = L.lynx_qkv_append(qkv, Hq, Hkv, None, a[1], a[2], k, v, q_out=torch.zeros(n_rows, Hq, 128,
                              dtype=torch.bfloat16, device="cuda"))
        return (*a, q, *L.lynx_verify_drafts(p, None, draft, u))
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = step()
    for seed in range(3):
        torch.manual_seed(seed)
        ctx.copy_(torch.randint(0, 500, (B,)))
        new.copy_(torch.randint(0, 10, (B,)))
        table.copy_(torch.arange(B * Hkv * max_pages).view(B, Hkv, max_pages))
        qkv.copy_(torch.randn(n_rows, (Hq + 2 * Hkv) * 128))
        p.copy_(torch.softmax(torch.randn(B, 3, 900), -1))
        u.copy_(torch.rand(B, 3))
        draft.copy_(torch.randint(0, 900, (B, 2)))
        t0 = table.clone()
        g.replay()
        replayed = [x.clone() for x in held] + [k.clone(), v.clone(), table.clone()]
        table.copy_(t0)
        k.zero_(); v.zero_()
        eager = step()
        # pages not of this step hold what earlier replays wrote: compare this step's slots only
        for a, b in zip(replayed, eager):
            assert torch.equal(a, b)
        rows = eager[2][eager[2] >= 0]
        for a, b in ((replayed[-3], k), (replayed[-2], v)):
            assert torch.equal(a.permute(0, 2, 1).reshape(-1, 128)[rows], b.permute(0, 2, 1).reshape(-1, 128)[rows])
        assert torch.equal(replayed[-1], table)
    status_ok()


# --------------------------------------------------------------- the binding

def test_binding_refuses_what_does_not_fit(cuda_device):
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")
    table = i32(2, 1, 3)
    for args, text in (
            ((i32(3), i32(2), table, i32(4), 5), "ctx_len"), ((i32(2), i32(2).long(), table, i32(4), 5), "new_len"),
            ((i32(2), i32(2), i32(2, 3), i32(4), 5), "page_table"), ((i32(2), i32(2), table, i32(4), -1), "n_rows"),
            ((i32(2), i32(2), table, i32(2, 2), 5), "free_pages"), ((i32(2).cpu(), i32(2), table, i32(4), 5), "ctx_len"),
            ((i32(2), i32(2), i32(2, 1, 6)[:, :, ::2], i32(4), 5), "page_table")):
        with pytest.raises(L.LynxError, match=text):
            L.lynx_assign_pages(*args)
    with pytest.raises(L.LynxError, match="slots"):
        L.lynx_assign_pages(i32(2), i32(2), table, i32(4), 5, slots=i32(5, 1))
    with pytest.raises(TypeError):
        L.lynx_assign_pages(i32(2), i32(2), table, i32(4), "5")
    slots = torch.zeros(2, 1, dtype=torch.int64, device="cuda")
    good = dict(qkv=bf(2, 384), n_q_heads=1, n_kv_heads=1, cos_sin=None, positions=i32(2), slots=slots, k_pages=bf(1, 128, 256),
                v_pages=bf(1, 128, 256))
    for kw, text in ((dict(qkv=bf(2, 383)), "qkv"), (dict(qkv=bf(2, 768)[:, ::2]), "qkv"), (dict(n_kv_heads=0), "qkv"),
                     (dict(positions=i32(3)), "positions"), (dict(k_pages=bf(1, 128, 128)), "k_pages"),
                     (dict(v_pages=bf(2, 128, 256)), "v_pages"), (dict(cos_sin=torch.zeros(4, 24, device="cuda")), "rot_dim"),
                     (dict(q_weight=torch.zeros(64, device="cuda")), "q_weight"), (dict(q_out=bf(2, 2, 128)), "q_out")):
        with pytest.raises(L.LynxError, match=text):
            L.lynx_qkv_append(**{**good, **kw})
    good = dict(q=bf(2, 2, 128), cu_q=i32(2), k_pages=bf(1, 128, 256), v_pages=bf(1, 128, 256), page_table=i32(1, 1, 1),
                ctx_len=i32(1), n_kv_heads=1)
    for kw, text in ((dict(q=bf(2, 2, 64)), "q must"), (dict(cu_q=i32(3)), "cu_q"), (dict(n_kv_heads=2), "page_table"),
                     (dict(out=bf(2, 2, 128).half()), "out"), (dict(out_dtype=torch.float16), "out_dtype"),
                     (dict(lse=bf(2, 2)), "lse"), (dict(workspace=torch.zeros(4, device="cuda")), "workspace"),
                     (dict(sm_scale=-1.0), "sm_scale"), (dict(ctx_len=i32(1).cpu()), "ctx_len")):
        with pytest.raises(L.LynxError, match=text):
            L.lynx_chunk_attn_bf16(**{**good, **kw})
    p = torch.zeros(1, 3, 8, device="cuda")
    good = dict(p=p, q=p[:, :2], draft=i32(1, 2), u=torch.zeros(1, 3, device="cuda"))
    for kw, text in ((dict(p=p.double()), "p must"), (dict(p=p[:, :1]), "p must"), (dict(q=p), "q must"),
                     (dict(q=p[:, :2].bfloat16()), "q must"), (dict(draft=i32(1, 3)), "draft"),
                     (dict(u=torch.zeros(1, 2, device="cuda")), "u must"), (dict(n_draft=i32(2)), "n_draft"),
                     (dict(p=p.transpose(1, 2)), "p must")):
        with pytest.raises(L.LynxError, match=text):
            L.lynx_verify_drafts(**{**good, **kw})
    status_ok()


def test_outputs_that_are_passed_come_back_and_streams_are_used(cuda_device):
    s = torch.cuda.Stream()
    tok, n = torch.empty(1, 2, dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
    p = torch.zeros(1, 2, 50, device="cuda")
    p[0, :, 3] = 1.0
    torch.cuda.synchronize()
    a, b = L.lynx_verify_drafts(p, None, torch.full((1, 1), 3, dtype=torch.int32, device="cuda"),
                                torch.zeros(1, 2, device="cuda"), tokens=tok, n_accept=n, stream=s)
    assert a is tok and b is n
    s.synchronize()
    assert tok.tolist() == [[3, 3]] and n.tolist() == [1]
    with torch.cuda.stream(s):               # torch's current stream
        t2, _ = L.lynx_verify_drafts(p, None, torch.full((1, 1), 4, dtype=torch.int32, device="cuda"),
                                     torch.full((1, 2), 0.5, device="cuda"))
    s.synchronize()
    assert t2.tolist() == [[3, -1]]
