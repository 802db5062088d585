"""lynx_token_logprobs where one CTA sums a whole row of a large vocabulary, and all
roundings of a running float32 sum would go one way."""
import numpy as np
import pytest
import torch

from progressive_kv_quantization_gb300 import lynx as L

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n_top", [0, 4])
@pytest.mark.parametrize("N,V,dtype", [(320, 1 << 20, torch.float32), (320, 1 << 20, torch.bfloat16), (306, (1 << 22) + 3, torch.float32),
                                       (306, 1 << 24, torch.bfloat16)])
def test_flat_rows_of_large_vocabularies(cuda_device, N, V, dtype, n_top):
    """Every thread's first piece is 0 and the others one value below it, which differs from row to row.

    A log probability is off by 2^-17 at most: the exponential's 2^-21, twice 2^-22 for the difference in
    powers of two (up to 2^3, each rounding half a step of 2^-21), at most 32 additions of a batch (2^-24
    each of the sum so far, half of that over all: 2^-20) and one lost rounding of the running sum,
    log2's 2^-22 of up to 24; two roundings of its own.  The entropy the same, of a range of 7."""
    x = torch.empty(N, V, dtype=dtype, device="cuda")
    c = (-torch.linspace(0.01, 5.9, N)).to(dtype)
    x[:] = c.cuda()[:, None]
    first = 256 * 16 // x.element_size()
    x[:, :first] = 0
    tokens = torch.zeros(N, dtype=torch.int32, device="cuda")
    tokens[::2] = V - 1
    logprob, entropy, ids, top = L.lynx_token_logprobs(x, tokens, n_top)
    torch.cuda.synchronize()
    d = c.double().numpy()
    s = first + (V - first) * np.exp(d)
    want = np.where(np.arange(N) % 2 == 0, d, 0.0) - np.log(s)
    assert np.abs(logprob.double().cpu().numpy() - want).max() <= 2.0 ** -17 + 2.0 ** -22 * np.abs(want).max()
    h = np.log(s) - (V - first) * np.exp(d) * d / s
    assert np.abs(entropy.double().cpu().numpy() - h).max() <= 2.0 ** -17 * 7
    if n_top:
        assert torch.equal(ids.cpu(), torch.arange(n_top, dtype=torch.int32).expand(N, n_top))
        assert np.abs(top.double().cpu().numpy() + np.log(s)[:, None]).max() <= 2.0 ** -17 + 2.0 ** -22 * 17
