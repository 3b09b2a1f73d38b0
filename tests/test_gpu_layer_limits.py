"""The convolution on more rows of a wide layer than 2^32 threads of a row and a vector each
(marked gpu; 34 GB a tensor)."""
import gc

import pytest
import torch

import gated_deltanet_chunked_gdn_amd as gdn

pytestmark = pytest.mark.gpu
DEV = "cuda"
T, C, TAIL = 4200000, 4096, 37


@pytest.fixture(autouse=True)
def _free():
    yield
    gc.collect()
    torch.cuda.empty_cache()


def test_conv_of_4200000_rows():
    """Every output is formed by the same operations in the same order wherever its row
    stands, so the last rows are those of a call on them alone."""
    gen = torch.Generator(device=DEV).manual_seed(0)
    x = torch.zeros(1, T, C, device=DEV, dtype=torch.bfloat16)
    assert x.numel() // 4 > 1 << 32
    for at in (0, 1 << 20, T - 1000):  # zeros between: the sums of dweight stay those of few rows
        x[:, at:at + 1000] = torch.randn(1, 1000, C, generator=gen, device=DEV).bfloat16()
    w, b = torch.randn(C, 4, generator=gen, device=DEV), torch.randn(C, generator=gen, device=DEV)
    tail = x[:, T - TAIL:].contiguous()
    rows = x[:, T - TAIL - 3:T - TAIL].contiguous()
    y, last = gdn.conv_fwd(x, w, bias=b)
    want, want_last = gdn.conv_fwd(tail, w, bias=b, state0=rows)
    assert torch.equal(y[:, T - TAIL:], want) and torch.equal(last, want_last)
    del y
    got = gdn.conv_bwd(x, w, x, bias=b)
    want = gdn.conv_bwd(tail, w, tail, bias=b, state0=rows)
    assert torch.equal(got["dx"][:, T - TAIL:], want["dx"])
    alone = [gdn.conv_bwd(p, w, p, bias=b) for p in (x[:, at:at + 1016].contiguous() for at in (0, (1 << 20) - 8, T - 1008))]
    for key in ("dweight", "dbias"):
        # rows of zeros add nothing.  Each value is a sum of about 3000 terms of about 1, in
        # another order here: at most 3000 roundings of sums below 3000 on either side
        total = sum(g[key].double() for g in alone)
        assert float((got[key].double() - total).abs().max()) <= 2 * 3000 * 2.0 ** -24 * 3000
