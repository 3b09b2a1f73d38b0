"""Selective scan on the GPU against its float64 definition: forward (serial and split
over the time axis), backward from the kept states, single-token step (marked gpu).

Roundings counted per term of T tokens: three per token for the decays and the state
(the exponential's two and the multiply-add), twice for the gradient's chain, the sums
over N states and, for dB and dC, over the channels, and 64 for the softplus, the gate
and the composed segment starts."""
import pytest
import torch

import gated_deltanet_chunked_gdn_amd as gdn
import _layer_oracle as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def _inputs(B, T, D, N, G, io, z=True, skip=True, bias=True, state=True, cu=None, seed=0):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, device=DEV)  # noqa: E731
    n = B if cu is None else len(cu) - 1
    a = dict(u=r(B, T, D).to(io), dt=r(B, T, D).to(io), A=-(0.1 + 3 * torch.rand(D, N, generator=gen, device=DEV)),
             Bm=r(B, T, G, N).to(io), Cm=r(B, T, G, N).to(io), D=r(D) if skip else None, z=r(B, T, D).to(io) if z else None,
             dt_bias=r(D) - 2 if bias else None)
    return a, (r(n, D, N) if state else None), r(B, T, D).to(io), (r(n, D, N) if state else None)


def _ref(a, h0, cu, softplus, dy=None, dlast=None, size=False):
    return ref.scan(a["u"], a["dt"], a["A"], a["Bm"], a["Cm"], a["D"], a["z"], a["dt_bias"], h0, cu, softplus, dy, dlast, size)


CASES = [  # B, T, D, N, G, cu, z, skip, bias, state
    (2, 33, 64, 16, 1, None, True, True, True, True),
    (1, 1, 8, 8, 1, None, True, True, True, True),
    (2, 50, 72, 16, 1, None, False, True, False, False),
    (1, 17, 80, 32, 2, None, True, False, True, True),
    (1, 40, 144, 64, 2, None, True, True, True, True),
    (3, 16, 24, 8, 3, None, False, False, True, False),
    (1, 97, 64, 16, 1, [0, 0, 1, 16, 33, 33, 96, 97, 97], True, True, True, True),
    (1, 60, 40, 64, 1, [0, 31, 60], True, True, True, True),
    (1, 66, 136, 8, 1, [0, 2, 66], False, True, True, True),
    (1, 150, 72, 16, 3, [0, 40, 40, 150], True, True, True, True),
    (2, 129, 24, 8, 1, None, True, True, False, False),
]


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("B,T,D,N,G,cu,z,skip,bias,state", CASES)
def test_scan(B, T, D, N, G, cu, z, skip, bias, state, io):
    a, h0, dy, dl = _inputs(B, T, D, N, G, io, z, skip, bias, state, cu)
    want = _ref(a, h0, cu, True, dy, dl)
    size = _ref(a, h0, cu, True, dy, dl, size=True)
    room = torch.full((1, T + 2, D), 7.0, device=DEV, dtype=io) if B == 1 else None
    y, h = gdn.scan_fwd(**a, h0=h0, cu_seqlens=cu, out=room[:, 1:T + 1] if room is not None else None)
    y2, h2, saved = gdn.scan_fwd_save(**a, h0=h0, cu_seqlens=cu)
    got = gdn.scan_bwd_saved(**a, dy=dy, saved=saved, dh_final=dl, cu_seqlens=cu)
    again = gdn.scan_bwd_saved(**a, dy=dy, saved=saved, dh_final=dl, cu_seqlens=cu)
    torch.cuda.synchronize()
    if room is not None:
        assert bool((room[:, 0] == 7).all()) and bool((room[:, T + 1] == 7).all())
    assert torch.equal(y, y2) and torch.equal(h, h2)
    ref.check("y", y, want["y"], size["y"], 3 * T + N + 64)
    ref.check("state", h, want["state"], size["state"], 3 * T + 64)
    for key in ("du", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dh0"):
        if got[key] is None:
            assert key == "dD" and not skip or key == "dz" and not z or key == "ddt_bias" and not bias
            continue
        assert torch.equal(got[key], again[key]), key
        ref.check(key, got[key], want[key], size[key], 6 * T + N + D + T + 128)


@pytest.mark.parametrize("T,D,N,cu", [(1100, 8, 16, None), (2050, 64, 8, None), (1500, 16, 64, [0, 1000, 1003, 1003, 1500])])
def test_split_over_time(T, D, N, cu):
    """Few channels and many tokens: several segments, whose starts are composed."""
    a, h0, dy, dl = _inputs(1, T, D, N, 1, F32, cu=cu)
    sizes = gdn.scan_buffers(a["u"], a["Bm"], cu_seqlens=cu)
    assert sizes["forward"] > 0  # segment states: the split is taken
    want = _ref(a, h0, cu, True, dy, dl)
    size = _ref(a, h0, cu, True, dy, dl, size=True)
    y, h, saved = gdn.scan_fwd_save(**a, h0=h0, cu_seqlens=cu)
    got = gdn.scan_bwd_saved(**a, dy=dy, saved=saved, dh_final=dl, cu_seqlens=cu)
    torch.cuda.synchronize()
    ref.check("y", y, want["y"], size["y"], 3 * T + N + 64)
    ref.check("state", h, want["state"], size["state"], 3 * T + 64)
    for key in ("du", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dh0"):
        ref.check(key, got[key], want[key], size[key], 6 * T + N + D + T + 128)


def test_many_short_sequences_and_a_long_one():
    """Slots of segments that no sequence has, between those that have one."""
    cu = [0, 0]
    for n in range(60):
        cu.append(cu[-1] + (1, 0, 17, 5, 63, 2)[n % 6])
    cu += [cu[-1] + 700, cu[-1] + 701, cu[-1] + 701]
    T, D, N = cu[-1], 40, 32
    a, h0, dy, dl = _inputs(1, T, D, N, 1, F32, cu=cu)
    want, size = _ref(a, h0, cu, True, dy, dl), _ref(a, h0, cu, True, dy, dl, size=True)
    y, h, saved = gdn.scan_fwd_save(**a, h0=h0, cu_seqlens=cu)
    ws = torch.full((gdn.scan_buffers(a["u"], a["Bm"], cu_seqlens=cu)["backward"],), 255, dtype=torch.uint8, device=DEV)  # NaN
    got = gdn.scan_bwd_saved(**a, dy=dy, saved=saved, dh_final=dl, cu_seqlens=cu, workspace=ws)
    ref.check("y", y, want["y"], size["y"], 3 * 700 + N + 64)
    ref.check("state", h, want["state"], size["state"], 3 * 700 + 64)
    for key in ("du", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dh0"):
        ref.check(key, got[key], want[key], size[key], 6 * 700 + N + D + T + 128)


def test_optional_outputs_of_the_c_abi():
    """dDskip without Dskip and ddt_bias without dt_bias may be asked for; dDskip, dz,
    ddt_bias and dh0 need not be."""
    import ctypes

    from gated_deltanet_chunked_gdn_amd import _native as nat

    B, T, D, N = 2, 40, 72, 16
    a, _, dy, _ = _inputs(B, T, D, N, 1, F32, skip=False, bias=False, state=False)
    _, _, saved = gdn.scan_fwd_save(**a)
    full = gdn.scan_bwd_saved(**a, dy=dy, saved=saved)
    want = _ref(a, None, None, True, dy)
    size = _ref(a, None, None, True, dy, size=True)
    lib, prob = nat.load(), nat.ScanProblem(B, T, D, N, 1, B, None, None, nat.GDN_FP32, 1)
    ws = torch.empty(gdn.scan_buffers(a["u"], a["Bm"])["backward"], dtype=torch.uint8, device=DEV)

    def call(**asked):
        out = {k: torch.empty_like(full[k]) for k in ("du", "ddt", "dA", "dB", "dC")}
        out.update(asked)
        names = ("du", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dh0")
        ins = [a[k] for k in ("u", "dt", "A", "Bm", "Cm", "D", "z", "dt_bias")] + [dy, None, saved]
        p = lambda t: None if t is None else t.data_ptr()  # noqa: E731
        st = lib.gdn_scan_bwd_saved(ctypes.byref(prob), *map(p, ins), saved.numel(), *(p(out.get(k)) for k in names), p(ws), ws.numel(),
                                    torch.cuda.current_stream().cuda_stream)
        assert st == nat.GDN_OK
        return out

    none = call()
    for k in ("du", "ddt", "dA", "dB", "dC"):
        assert torch.equal(none[k], full[k]), k
    more = call(dD=torch.empty(D, device=DEV), ddt_bias=torch.empty(D, device=DEV))
    for k in ("dD", "ddt_bias"):
        ref.check(k, more[k], want[k], size[k], 7 * T + N + D + 128)


@pytest.mark.parametrize("io", [BF, F32])
def test_raw_steps_and_extremes(io):
    """No softplus; steps of zero (the state stays), large steps (it is forgotten), and
    softplus arguments from -40 to 40."""
    a, h0, dy, dl = _inputs(1, 24, 64, 16, 1, io, bias=False)
    a["dt"] = a["dt"].abs()
    a["dt"][:, 3] = 0
    a["dt"][:, 9] = 300
    for softplus in (False, True):
        if softplus:
            a["dt"] = torch.linspace(-40, 40, 24, device=DEV).reshape(1, 24, 1).expand(1, 24, 64).to(io).contiguous()
        want = _ref(a, h0, None, softplus, dy, dl)
        size = _ref(a, h0, None, softplus, dy, dl, size=True)
        y, h, saved = gdn.scan_fwd_save(**a, h0=h0, dt_softplus=softplus)
        got = gdn.scan_bwd_saved(**a, dy=dy, saved=saved, dh_final=dl, dt_softplus=softplus)
        ref.check("y", y, want["y"], size["y"], 3 * 24 + 80)
        ref.check("state", h, want["state"], size["state"], 3 * 24 + 64)
        for key in ("du", "ddt", "dA", "dB", "dC", "dD", "dz", "dh0"):
            ref.check(key, got[key], want[key], size[key], 7 * 24 + 16 + 64 + 128)


def test_a_sequence_of_nan_stays_alone():
    cu = [0, 10, 30, 41]
    a, h0, dy, dl = _inputs(1, 41, 64, 16, 1, F32, cu=cu)
    clean_y, clean_h, saved = gdn.scan_fwd_save(**a, h0=h0, cu_seqlens=cu)
    clean = gdn.scan_bwd_saved(**a, dy=dy, saved=saved, dh_final=dl, cu_seqlens=cu)
    for key in ("u", "Bm", "z"):
        a[key][:, 10:30] = float("nan")
    y, h, saved = gdn.scan_fwd_save(**a, h0=h0, cu_seqlens=cu)
    got = gdn.scan_bwd_saved(**a, dy=dy, saved=saved, dh_final=dl, cu_seqlens=cu)
    for rows in (slice(0, 10), slice(30, 41)):
        assert torch.equal(y[:, rows], clean_y[:, rows])
        for key in ("du", "ddt", "dB", "dC", "dz"):
            assert torch.equal(got[key][:, rows], clean[key][:, rows]), key
    assert torch.equal(h[[0, 2]], clean_h[[0, 2]]) and torch.equal(got["dh0"][[0, 2]], clean["dh0"][[0, 2]])
    assert bool(y[:, 10:30].isnan().all())


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("B,D,N,G,z", [(1, 8, 8, 1, True), (3, 72, 16, 1, True), (2, 144, 32, 2, False), (5, 64, 64, 4, True)])
def test_step(B, D, N, G, z, io):
    a, h0, _, _ = _inputs(B, 1, D, N, G, io, z)
    want, size = _ref(a, h0, None, True), _ref(a, h0, None, True, size=True)
    state = h0.clone()
    y = gdn.scan_step(**a, state=state)
    torch.cuda.synchronize()
    ref.check("y", y, want["y"], size["y"], N + 80)
    ref.check("state", state, want["state"], size["state"], 80)


def test_no_tokens_and_no_sequences():
    a, h0, dy, dl = _inputs(2, 0, 16, 16, 1, F32)
    y, h, saved = gdn.scan_fwd_save(**a, h0=h0)
    got = gdn.scan_bwd_saved(**a, dy=dy, saved=saved, dh_final=dl)
    assert y.shape == (2, 0, 16) and torch.equal(h, h0) and torch.equal(got["dh0"], dl)
    assert float(got["dA"].abs().max()) == 0 and float(got["ddt_bias"].abs().max()) == 0
    a, h0, dy, dl = _inputs(0, 4, 16, 16, 1, F32)
    y, h, saved = gdn.scan_fwd_save(**a, h0=h0)
    got = gdn.scan_bwd_saved(**a, dy=dy, saved=saved, dh_final=dl)
    assert y.shape == (0, 4, 16) and float(got["dA"].abs().max()) == 0


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("B,T,D,N,G,cu,split", [
    (1, 1100, 24, 8, 1, None, True),
    (1, 1100, 72, 16, 3, None, True),
    (2, 1030, 40, 32, 1, None, True),
    (1, 1500, 80, 32, 2, [0, 1000, 1003, 1003, 1500], True),
    (1, 1100, 72, 64, 1, None, True),
    (1, 1700, 16, 64, 2, [0, 0, 990, 1000, 1700], True),
    (2, 16, 136, 32, 1, None, False),
    (1, 45, 48, 64, 2, [0, 16, 16, 29, 45], False),
    (1, 77, 24, 32, 1, [0, 77], False),
    (1, 200, 12 * 8, 64, 3, [0, 64, 129, 200], False),
])
def test_every_form_and_width(B, T, D, N, G, cu, split, io):
    """The forms over segments, over the time axis inside a workgroup, and serial, with
    every number of states and both types."""
    a, h0, dy, dl = _inputs(B, T, D, N, G, io, cu=cu, seed=5)
    sizes = gdn.scan_buffers(a["u"], a["Bm"], cu_seqlens=cu)
    assert (sizes["forward"] > 0) == split
    want, size = _ref(a, h0, cu, True, dy, dl), _ref(a, h0, cu, True, dy, dl, size=True)
    y, h, saved = gdn.scan_fwd_save(**a, h0=h0, cu_seqlens=cu)
    got = gdn.scan_bwd_saved(**a, dy=dy, saved=saved, dh_final=dl, cu_seqlens=cu)
    ref.check("y", y, want["y"], size["y"], 3 * T + N + 64)
    ref.check("state", h, want["state"], size["state"], 3 * T + 64)
    for key in ("du", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dh0"):
        ref.check(key, got[key], want[key], size[key], 6 * T + N + D + T + 128)


@pytest.mark.parametrize("T,D,N", [(16, 4112, 32), (13, 2064, 64)])
def test_many_channels_and_few_tokens(T, D, N):
    """Wide states in the serial form."""
    a, h0, dy, dl = _inputs(1, T, D, N, 1, BF, seed=6)
    want, size = _ref(a, h0, None, True), _ref(a, h0, None, True, size=True)
    y, h = gdn.scan_fwd(**a, h0=h0)
    ref.check("y", y, want["y"], size["y"], 3 * T + N + 64)
    ref.check("state", h, want["state"], size["state"], 3 * T + 64)


@pytest.mark.parametrize("N", [8, 32, 64])
def test_no_tokens_of_other_widths(N):
    a, h0, dy, dl = _inputs(3, 0, 16, N, 1, BF)
    y, h, saved = gdn.scan_fwd_save(**a, h0=h0)
    got = gdn.scan_bwd_saved(**a, dy=dy, saved=saved, dh_final=dl)
    assert y.shape == (3, 0, 16) and torch.equal(h, h0) and torch.equal(got["dh0"], dl)
    a, h0, dy, dl = _inputs(1, 3, 16, N, 1, BF, cu=[0, 0, 3, 3])
    y, h = gdn.scan_fwd(**a, h0=h0, cu_seqlens=[0, 0, 3, 3])
    alone = gdn.scan_fwd(**a, h0=h0[1:2].contiguous())
    assert torch.equal(h[[0, 2]], h0[[0, 2]]) and torch.equal(y, alone[0]) and torch.equal(h[1:2], alone[1])
