"""The selective scan of few channels over more than 100 segments of the time axis, against
its float64 definition (marked gpu).  Roundings counted as in test_gpu_scan.py: three per
token for a state, twice that for a gradient, and the sums."""
import pytest
import torch

import gated_deltanet_chunked_gdn_amd as gdn
import _layer_oracle as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("T,cu", [(16401, None), (16900, [0, 3, 3, 16590, 16900])])
def test_more_than_100_segments(T, cu):
    D, N = 8, 8
    gen = torch.Generator(device=DEV).manual_seed(0)
    r = lambda *s: torch.randn(*s, generator=gen, device=DEV)  # noqa: E731
    n = 1 if cu is None else len(cu) - 1
    # slow and fast decays: exp(-0.0003) to exp(-0.3) a token
    a = dict(u=r(1, T, D), dt=0.1 + 0.1 * torch.rand(1, T, D, generator=gen, device=DEV), A=-torch.logspace(-2.5, 0.2, D * N).reshape(N, D).t().contiguous().to(DEV),
             Bm=r(1, T, 1, N), Cm=r(1, T, 1, N), D=r(D), z=r(1, T, D))
    h0, dy, dl = r(n, D, N), r(1, T, D), r(n, D, N)
    sizes = gdn.scan_buffers(a["u"], a["Bm"], cu_seqlens=cu)
    assert sizes["forward"] > 100 * D * N * 4  # end states of more than 100 segments
    want, size = (ref.scan(a["u"], a["dt"], a["A"], a["Bm"], a["Cm"], a["D"], a["z"], None, h0, cu, False, dy, dl, s) for s in (False, True))
    y, h, saved = gdn.scan_fwd_save(**a, h0=h0, cu_seqlens=cu, dt_softplus=False)
    got = gdn.scan_bwd_saved(**a, dy=dy, saved=saved, dh_final=dl, cu_seqlens=cu, dt_softplus=False)
    ref.check("y", y, want["y"], size["y"], 3 * T + N + 64)
    ref.check("state", h, want["state"], size["state"], 3 * T + 64)
    for key in ("du", "ddt", "dA", "dB", "dC", "dD", "dz", "dh0"):
        ref.check(key, got[key], want[key], size[key], 7 * T + N + D + 128)
