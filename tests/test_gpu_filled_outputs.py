"""Outputs that a call makes itself, where torch fills what it allocates
(torch.use_deterministic_algorithms): what a kernel leaves out holds the fill."""
import pytest
import torch

from progressive_kv_quantization_gb300 import lynx as L

pytestmark = pytest.mark.gpu


@pytest.fixture
def filling():
    was = torch.are_deterministic_algorithms_enabled()
    torch.use_deterministic_algorithms(True)
    yield
    torch.use_deterministic_algorithms(was)


def append_args(positions, e4m3):
    n = len(positions)
    qkv = torch.ones(n, 4 * 128, dtype=torch.bfloat16, device="cuda")
    slots = torch.arange(n, device="cuda")[:, None].contiguous()
    if e4m3:
        pools = [torch.zeros(1, 256, 128, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2)]
        pools.append(torch.zeros(1, 2, 8, dtype=torch.uint8, device="cuda"))
    else:
        pools = [torch.zeros(1, 128, 256, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    return qkv, 2, 1, None, torch.tensor(positions, dtype=torch.int32, device="cuda"), slots, *pools


@pytest.mark.parametrize("e4m3", [False, True])
def test_rows_that_are_left_out_read_nan(cuda_device, filling, e4m3):
    call = L.lynx_qkv_append_e4m3 if e4m3 else L.lynx_qkv_append
    for _ in range(3):      # memory that held numbers before
        q = call(*append_args([0, -1, 2, -1], e4m3))
        assert (q[[0, 2]] == 1).all() and q[[1, 3]].isnan().all()
        q.fill_(5)
        del q


def test_rows_behind_the_last_request_read_the_fill(cuda_device, filling):
    pages = [torch.zeros(1, 128, 256, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    q = torch.ones(5, 2, 128, dtype=torch.bfloat16, device="cuda")
    out, lse = L.lynx_chunk_attn_bf16(q, i32(0, 3), *pages, i32(0).view(1, 1, 1), i32(3), 1)
    assert not out[:3].isnan().any() and out[3:].isnan().all() and lse[3:].isnan().all()
    # every output is made this way, whole numbers among them
    out = L.lynx_token_logprobs(torch.zeros(0, 9, device="cuda"), i32(), 2)
    assert out[2].shape == (0, 2) and out[2].dtype == torch.int32 and out[2].device.type == "cuda"


def test_the_fill_can_be_switched_off(cuda_device, filling):
    was = torch.utils.deterministic.fill_uninitialized_memory
    torch.utils.deterministic.fill_uninitialized_memory = False
    try:
        q = L.lynx_qkv_append(*append_args([0, 1], False))
        assert (q == 1).all()
    finally:
        torch.utils.deterministic.fill_uninitialized_memory = was
