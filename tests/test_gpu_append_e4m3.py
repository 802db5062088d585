"""lynx_qkv_append_e4m3 against the float64 oracle: blocks begun, gone on with and grown,
ragged batches, rows left out, and everything else in the pools as it was."""
import numpy as np
import pytest
import torch

from oracle import e4m3
from oracle import serving as sv
from progressive_kv_quantization_gb300 import lynx as L

pytestmark = pytest.mark.gpu
D = 128
# the norm's sum, root, division and the rotation's two products: some twelve roundings of
# 2^-24 of terms that a rotation may cancel to a fraction of; relative to a row's largest value
F32 = 2.0 ** -19


def case(reqs, Hq, Hkv, seed, norm=True, rot=128, interleaved=False, extra=0, sizes=3, pad=0):
    """reqs: (tokens held, new tokens) of each request.  Pools of random codes and scales."""
    rng = np.random.default_rng(seed)
    n_rows = sum(n for _, n in reqs) + pad
    pages = [-(-(c + n) // 256) for c, n in reqs]
    order = rng.permutation(sum(pages) * Hkv + 2)
    positions = np.full(n_rows, -1, dtype=np.int32)
    slots = np.full((n_rows, Hkv), -1, dtype=np.int64)
    row = at = 0
    for (c, n), p in zip(reqs, pages):
        ids = order[at:at + p * Hkv].reshape(Hkv, p)
        at += p * Hkv
        for i in range(n):
            positions[row] = c + i
            slots[row] = ids[:, (c + i) // 256] * 256 + (c + i) % 256
            row += 1
    n_pool = order.size
    codes = rng.integers(0, 256, (2, n_pool, 256, D), dtype=np.uint8)
    codes[codes % 128 == 127] = 3
    scales = rng.integers(115, 130, (2, n_pool, 8)).astype(np.uint8)
    width = (Hq + 2 * Hkv) * D
    x = rng.standard_normal((n_rows, width + extra)).astype(np.float32)
    x *= np.exp2(rng.integers(-sizes, sizes + 1, (n_rows, 1)))
    qkv = torch.from_numpy(x).cuda().bfloat16()[:, :width]
    w = [rng.uniform(0.5, 1.5, D).astype(np.float32) for _ in range(2)] if norm else [None, None]
    angle = np.arange(max(c + n for c, n in reqs) + 1)[:, None] * 1e4 ** (-np.arange(0, max(rot, 2), 2) / max(rot, 2))
    cs = np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32) if rot else None
    return dict(qkv=qkv, Hq=Hq, Hkv=Hkv, positions=positions, slots=slots, codes=codes, scales=scales, w=w, cs=cs, rot=rot,
                interleaved=interleaved)


def call(c, pools, **kw):
    up = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return L.lynx_qkv_append_e4m3(c["qkv"], c["Hq"], c["Hkv"], up(c["cs"]), up(c["positions"]), up(c["slots"]), *pools,
                                  q_weight=up(c["w"][0]), k_weight=up(c["w"][1]), interleaved=c["interleaved"], **kw)


def pools_of(c):
    k, v = (torch.from_numpy(x.copy()).cuda().view(torch.float8_e4m3fn) for x in c["codes"])
    return k, v, torch.from_numpy(np.ascontiguousarray(c["scales"].transpose(1, 0, 2))).cuda()


def check(c, q, pools):
    torch.cuda.synchronize()
    L.lynx_device_status()
    Hq, Hkv = c["Hq"], c["Hkv"]
    x = c["qkv"].double().cpu().numpy().reshape(-1, Hq + 2 * Hkv, D)
    pos = np.maximum(c["positions"], 0)
    half = c["rot"] // 2
    cos, sin = (c["cs"][pos, :half].astype(float), c["cs"][pos, half:].astype(float)) if half else (np.zeros((len(pos), 0)),) * 2
    qr = sv.norm_rotate(x[:, :Hq], c["w"][0], 1e-6, cos, sin, c["interleaved"])
    kr = sv.norm_rotate(x[:, Hq:Hq + Hkv], c["w"][1], 1e-6, cos, sin, c["interleaved"])
    real = c["positions"] >= 0
    g = q.double().cpu().numpy()
    big = np.abs(qr).max(-1, keepdims=True)
    assert np.all(np.abs(g - qr)[real] <= (2.0 ** -8 * np.abs(qr) + F32 * big)[real])
    slots = np.where(real[:, None], c["slots"], -1)
    got_scales = pools[2].cpu().numpy()
    exact_k = c["w"][1] is None and not half          # keys are copied
    for which, rows in ((0, kr), (1, x[:, Hq + Hkv:])):
        codes, scales, wanted = e4m3.append(rows, slots, c["codes"][which], c["scales"][which])
        assert np.array_equal(got_scales[:, which], scales)
        got = pools[which].view(torch.uint8).cpu().numpy()
        if which == 1 or exact_k:
            assert np.array_equal(got, codes)
            continue
        off = got != codes
        assert off.mean() < 1e-3
        # a code may be the other one only where its value lies within float32's error of the middle
        a, b = e4m3.decode(got[off]), e4m3.decode(codes[off])
        near = np.abs((a + b) / 2 - wanted[off])
        assert np.all(near <= F32 * e4m3.TOP) and np.all(np.abs(a - b) <= 2.0 ** -3 * np.maximum(np.abs(a), np.abs(b)) + 2.0 ** -9)
        untouched = np.ones(codes.shape[:2], dtype=bool)
        for s in slots[slots >= 0]:
            untouched[s // 256, s % 256] = False
        assert not off[untouched].any()


STARTS = [(0, 1), (1, 1), (31, 1), (32, 1), (255, 1), (256, 1), (5, 1), (40, 3), (30, 4), (250, 9), (0, 33), (17, 100)]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm,rot", [(True, 128), (False, 64), (True, 0), (False, 0), (False, 128), (True, 16)])
def test_blocks_at_every_edge(cuda_device, norm, rot, interleaved):
    c = case(STARTS, 6, 2, 1, norm=norm, rot=rot, interleaved=interleaved)
    pools = pools_of(c)
    check(c, call(c, pools), pools)


@pytest.mark.parametrize("reqs,Hq,Hkv", [
    ([(0, 1)], 1, 1), ([(7, 1)], 8, 8), ([(13, 2500)], 4, 1), ([(200, 300), (3, 700), (31, 1)], 16, 4),
    ([(i * 37, 1) for i in range(130)], 32, 8), ([(i, 1 + 5 * i) for i in range(40)], 3, 1), ([(0, 32)] * 9 + [(31, 33)] * 9, 2, 2)])
def test_ragged_batches(cuda_device, reqs, Hq, Hkv):
    c = case(reqs, Hq, Hkv, len(reqs), extra=64)
    pools = pools_of(c)
    q = torch.empty(c["qkv"].shape[0], Hq, D, dtype=torch.bfloat16, device="cuda")
    assert call(c, pools, q_out=q) is q
    check(c, q, pools)


def test_rows_left_out_stay_as_they_are(cuda_device):
    """Rows without a position and rows behind the last request; a head without a slot."""
    c = case([(20, 50), (3, 40), (100, 7)], 4, 2, 3, pad=9)
    c["positions"][50:90] = -1                # a refused request
    c["slots"][95, 1] = -1                    # one head's key is not kept: its block's rows behind are a run of their own
    c["slots"][95:, 1] = -1
    pools = pools_of(c)
    q = torch.full((106, 4, D), 5.0, dtype=torch.bfloat16, device="cuda")
    call(c, pools, q_out=q)
    check(c, q, pools)
    assert (q[50:90] == 5).all() and (q[97:] == 5).all()


def test_a_scale_that_grows_token_by_token(cuda_device):
    """Forty steps of one token each, four times as large every fifth; then small ones in the next block."""
    c = case([(3, 1)], 2, 2, 5, norm=False, rot=0)
    pools = pools_of(c)
    rng = np.random.default_rng(6)
    for step in range(40):
        c["positions"][:] = 3 + step
        page = c["slots"][0] // 256
        c["slots"] = (page * 256 + 3 + step)[None]
        size = 4.0 ** (step // 5) if step < 29 else 1e-3
        c["qkv"] = torch.from_numpy(rng.standard_normal((1, 6 * D)).astype(np.float32) * size).cuda().bfloat16()
        c["codes"] = np.stack([p.view(torch.uint8).cpu().numpy() for p in pools[:2]])
        c["scales"] = pools[2].cpu().numpy().transpose(1, 0, 2)
        check(c, call(c, pools), pools)


def test_sizes_past_the_scales(cuda_device):
    """Zeros, values below the smallest scale's codes, and values that only saturate."""
    c = case([(0, 3), (10, 2), (0, 1)], 1, 1, 7, norm=False, rot=0, sizes=0)
    x = c["qkv"].clone()
    x[0:3] = 0
    x[3] *= 2.0 ** -70
    x[4] *= 2.0 ** -60
    x[5] *= 2.0 ** 85
    c["qkv"] = x
    c["scales"][:] = 90
    pools = pools_of(c)
    check(c, call(c, pools), pools)
    s = pools[2].cpu().numpy()
    assert s[c["slots"][0, 0] // 256, 0, 0] == 74 and s[c["slots"][5, 0] // 256, 1, 0] == 198
    # scales outside the range count as its bounds
    for byte in (0, 255):
        c["scales"][:] = byte
        pools = pools_of(c)
        check(c, call(c, pools), pools)


def test_far_slots(cuda_device):
    c = case([(70, 20)], 2, 1, 8)
    far = 140000
    big = [torch.zeros(far, 256, D, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = torch.zeros(far, 2, 8, dtype=torch.uint8, device="cuda")
    small = pools_of(c)
    n = small[0].shape[0]
    for pool, part in zip(big, small):
        pool[far - n:] = part.view(torch.uint8)
    scales[far - n:] = small[2]
    near = c["slots"]
    c["slots"] = near + (far - n) * 256
    q = call(c, [big[0].view(torch.float8_e4m3fn), big[1].view(torch.float8_e4m3fn), scales])
    c["slots"] = near
    check(c, q, [big[0][far - n:].view(torch.float8_e4m3fn), big[1][far - n:].view(torch.float8_e4m3fn), scales[far - n:]])


def test_words_of_bad_slots_and_positions(cuda_device):
    c = case([(0, 40)], 2, 1, 9)
    pools = pools_of(c)
    c["slots"][7] = pools[0].shape[0] * 256
    call(c, pools)
    with pytest.raises(L.LynxError, match="= 5 "):
        L.lynx_device_status()
    c = case([(0, 40)], 2, 1, 9)
    pools = pools_of(c)
    c["positions"][39] = 1000
    call(c, pools)
    with pytest.raises(L.LynxError, match="= 4 "):
        L.lynx_device_status()
    c["positions"][39] = -1                   # the row was left out
    check(c, call(c, pools), pools)


def test_empty_stream_and_graph(cuda_device):
    c = case([(5, 30), (100, 3)], 4, 2, 10)
    pools = pools_of(c)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):           # the inputs are made on it
        q = call(c, pools)
    torch.cuda.current_stream().wait_stream(stream)
    check(c, q, pools)
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    pools = pools_of(c)
    fresh = [p.clone() for p in pools]
    args = (c["qkv"], 4, 2, up(c["cs"]), up(c["positions"]), up(c["slots"]), *pools)
    kw = dict(q_weight=up(c["w"][0]), k_weight=up(c["w"][1]), q_out=q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.lynx_qkv_append_e4m3(*args, **kw)
    for _ in range(2):
        for p, f in zip(pools, fresh):
            p.view(torch.uint8).copy_(f.view(torch.uint8))
        q.zero_()
        graph.replay()
        check(c, q, pools)
    none = torch.empty(0, 8 * D, dtype=torch.bfloat16, device="cuda")
    out = L.lynx_qkv_append_e4m3(none, 4, 2, args[3], args[4][:0], args[5][:0], *pools)
    assert out.shape == (0, 4, D)


def test_refusals(cuda_device):
    c = case([(5, 4)], 4, 2, 11)
    k, v, s = pools_of(c)
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    good = dict(qkv=c["qkv"], n_q_heads=4, n_kv_heads=2, cos_sin=up(c["cs"]), positions=up(c["positions"]), slots=up(c["slots"]),
                k_pages=k, v_pages=v, scales=s)
    L.lynx_qkv_append_e4m3(**good)
    for change, word in [
            (dict(qkv=c["qkv"].float()), "qkv"), (dict(n_kv_heads=3), "channels"), (dict(k_pages=k.view(torch.uint8)), "k_pages"),
            (dict(v_pages=v[:1]), "v_pages"), (dict(scales=s.int()), "scales"), (dict(scales=s[:, :1]), "scales"),
            (dict(positions=up(c["positions"]).long()), "positions"), (dict(slots=up(c["slots"]).int()), "slots"),
            (dict(cos_sin=up(c["cs"])[:, :24].contiguous()), "rot_dim"), (dict(q_weight=torch.ones(64, device="cuda")), "q_weight"),
            (dict(k_weight=torch.ones(D, device="cuda"), norm_eps=2.0), "norm_eps"),
            (dict(q_out=c["qkv"].as_strided((4, 4, D), (4 * D, D, 1))), "overlaps")]:
        with pytest.raises(L.LynxError, match=word):
            L.lynx_qkv_append_e4m3(**{**good, **change})
    L.lynx_device_status()
