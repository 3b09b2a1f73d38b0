"""Host-side checks of the layer operators' C ABI and of their Python calls (CPU only:
no kernel is launched; pointers passed here are never dereferenced)."""
import ctypes

import numpy as np
import pytest
import torch

from gated_deltanet_chunked_gdn_amd import _native as nat
from gated_deltanet_chunked_gdn_amd import layer

P = 0x10000000  # an address that is 16-byte aligned and never read
BIG = 1 << 26   # distance between the addresses of different tensors


@pytest.fixture(scope="module")
def lib():
    return nat.load()


def at(i, off=0):
    return P + i * BIG + off


_keep = []


def offsets(cu):
    a = np.asarray(cu, dtype=np.int32)
    _keep.append(a)
    return a.ctypes.data


# --------------------------------------------------------------------------- step

def step_problem(**kw):
    d = dict(B=2, T=1, H=3, Dk=64, Dv=48, num_seqs=2, io_dtype=nat.GDN_BF16, scale=1.0, chunk=64, num_segments=1)
    return nat.Problem(**(d | kw))


def call_step(lib, p, ptrs=None, name="gdn_step"):
    q = [at(i) for i in range(7)] if ptrs is None else ptrs
    return getattr(lib, name)(p, *q, None)


@pytest.mark.parametrize("name", ["gdn_step", "gdn_kda_step"])
@pytest.mark.parametrize("kw,status", [
    (dict(T=2), nat.GDN_ERR_SHAPE), (dict(T=0), nat.GDN_ERR_SHAPE), (dict(Dk=96), nat.GDN_ERR_UNSUPPORTED),
    (dict(Dv=40), nat.GDN_ERR_UNSUPPORTED), (dict(io_dtype=5), nat.GDN_ERR_DTYPE), (dict(num_seqs=1), nat.GDN_ERR_SHAPE),
    (dict(H=0), nat.GDN_ERR_SHAPE), (dict(B=65535, num_seqs=65535, H=600, Dv=16), nat.GDN_ERR_UNSUPPORTED),
])
def test_step_problem(lib, name, kw, status):
    assert call_step(lib, step_problem(**kw), name=name) == status


def test_step_packed_is_refused(lib):
    p = step_problem(B=1, num_seqs=1, cu_seqlens_host=offsets([0, 1]), cu_seqlens_dev=P)
    assert call_step(lib, p) == nat.GDN_ERR_SHAPE


@pytest.mark.parametrize("slot", range(7))
def test_step_pointers(lib, slot):
    ptrs = [at(i) for i in range(7)]
    ptrs[slot] = None
    assert call_step(lib, step_problem(), ptrs) == nat.GDN_ERR_NULL
    ptrs[slot] = at(slot, 2)
    assert call_step(lib, step_problem(), ptrs) == nat.GDN_ERR_ALIGN
    if slot != 6:  # o over another tensor
        ptrs[slot] = at(6)
        assert call_step(lib, step_problem(), ptrs) == nat.GDN_ERR_ALIAS


# --------------------------------------------------------------------------- convolution

def conv_problem(**kw):
    d = dict(B=2, T=5, C=16, W=4, num_seqs=2, io_dtype=nat.GDN_BF16, activation=nat.GDN_ACT_SILU)
    return nat.ConvProblem(**(d | kw))


CONV_BAD = [
    (dict(io_dtype=3), nat.GDN_ERR_DTYPE), (dict(C=0), nat.GDN_ERR_SHAPE), (dict(C=12), nat.GDN_ERR_UNSUPPORTED),
    (dict(C=(1 << 20) + 8), nat.GDN_ERR_UNSUPPORTED), (dict(W=0), nat.GDN_ERR_SHAPE), (dict(W=1), nat.GDN_ERR_UNSUPPORTED),
    (dict(W=5), nat.GDN_ERR_UNSUPPORTED), (dict(T=-1), nat.GDN_ERR_SHAPE), (dict(num_seqs=3), nat.GDN_ERR_SHAPE),
    (dict(activation=2), nat.GDN_ERR_UNSUPPORTED), (dict(B=70000, num_seqs=70000), nat.GDN_ERR_UNSUPPORTED),
    (dict(B=60000, num_seqs=60000, T=60000), nat.GDN_ERR_UNSUPPORTED),
]


@pytest.mark.parametrize("kw,status", CONV_BAD)
def test_conv_problem(lib, kw, status):
    p, n = conv_problem(**kw), ctypes.c_size_t(7)
    assert lib.gdn_conv_workspace_size(p, n) == status and n.value == 7
    assert lib.gdn_conv_fwd(p, *[at(i) for i in range(6)], None) == status
    assert lib.gdn_conv_bwd(p, *[at(i) for i in range(11)], BIG, None) == status
    assert lib.gdn_conv_step(p, *[at(i) for i in range(5)], None) == status


def test_conv_offsets(lib):
    for cu, T, status in (([0, 3, 2, 5], 5, nat.GDN_ERR_SEQLENS), ([1, 5], 5, nat.GDN_ERR_SEQLENS), ([0, 4], 5, nat.GDN_ERR_SEQLENS)):
        p = conv_problem(B=1, T=T, num_seqs=len(cu) - 1, cu_seqlens_host=offsets(cu), cu_seqlens_dev=P)
        assert lib.gdn_conv_fwd(p, *[at(i) for i in range(6)], None) == status
    p = conv_problem(B=1, T=5, num_seqs=1, cu_seqlens_host=offsets([0, 5]))
    assert lib.gdn_conv_fwd(p, *[at(i) for i in range(6)], None) == nat.GDN_ERR_NULL
    p = conv_problem(B=2, T=5, num_seqs=1, cu_seqlens_host=offsets([0, 5]), cu_seqlens_dev=P)
    assert lib.gdn_conv_fwd(p, *[at(i) for i in range(6)], None) == nat.GDN_ERR_SHAPE
    p = conv_problem(B=1, T=1, num_seqs=1, cu_seqlens_host=offsets([0, 1]), cu_seqlens_dev=P)
    assert lib.gdn_conv_step(p, *[at(i) for i in range(5)], None) == nat.GDN_ERR_SHAPE


def test_conv_pointers(lib):
    p = conv_problem()
    need = ctypes.c_size_t(0)
    assert lib.gdn_conv_workspace_size(p, need) == nat.GDN_OK
    assert need.value == 16 * 5 * 4  # one block of rows: (W + 1) C sums
    assert lib.gdn_conv_workspace_size(p, None) == nat.GDN_ERR_NULL
    optional_fwd, optional_bwd = {2, 3, 5}, {2, 3, 5, 8, 9}
    for slot in range(6):
        ptrs = [at(i) for i in range(6)]
        if slot not in optional_fwd:
            ptrs[slot] = None
            assert lib.gdn_conv_fwd(p, *ptrs, None) == nat.GDN_ERR_NULL, slot
        ptrs[slot] = at(slot, 8)
        assert lib.gdn_conv_fwd(p, *ptrs, None) == nat.GDN_ERR_ALIGN, slot
        if slot != 4:
            ptrs[slot] = at(4)
            assert lib.gdn_conv_fwd(p, *ptrs, None) == nat.GDN_ERR_ALIAS, slot
    for slot in range(10):
        ptrs = [at(i) for i in range(11)]
        if slot not in optional_bwd:
            ptrs[slot] = None
            assert lib.gdn_conv_bwd(p, *ptrs, need.value, None) == nat.GDN_ERR_NULL, slot
        if slot != 6:
            ptrs[slot] = at(6)
            assert lib.gdn_conv_bwd(p, *ptrs, need.value, None) == nat.GDN_ERR_ALIAS, slot
    ptrs = [at(i) for i in range(11)]
    assert lib.gdn_conv_bwd(p, *ptrs, need.value - 1, None) == nat.GDN_ERR_WORKSPACE
    assert lib.gdn_conv_bwd(p, *ptrs[:10], None, need.value, None) == nat.GDN_ERR_WORKSPACE
    assert lib.gdn_conv_step(conv_problem(), *ptrs[:5], None) == nat.GDN_ERR_SHAPE  # T != 1


# --------------------------------------------------------------------------- scan

def scan_problem(**kw):
    d = dict(B=2, T=40, D=64, N=16, G=1, num_seqs=2, io_dtype=nat.GDN_BF16, dt_softplus=1)
    return nat.ScanProblem(**(d | kw))


def scan_size(p, pass_):
    n = ctypes.c_size_t(0)
    st = nat.load().gdn_scan_workspace_size(p, pass_, n)
    return st, n.value


@pytest.mark.parametrize("kw,status", [
    (dict(io_dtype=2), nat.GDN_ERR_DTYPE), (dict(N=0), nat.GDN_ERR_SHAPE), (dict(N=24), nat.GDN_ERR_UNSUPPORTED),
    (dict(N=128), nat.GDN_ERR_UNSUPPORTED), (dict(G=3), nat.GDN_ERR_SHAPE), (dict(D=72, G=2), nat.GDN_ERR_UNSUPPORTED),
    (dict(D=60), nat.GDN_ERR_UNSUPPORTED), (dict(D=(1 << 20) + 8), nat.GDN_ERR_UNSUPPORTED), (dict(T=-1), nat.GDN_ERR_SHAPE),
    (dict(num_seqs=1), nat.GDN_ERR_SHAPE), (dict(B=70000, num_seqs=70000, T=1), nat.GDN_ERR_UNSUPPORTED),
    (dict(B=50000, num_seqs=50000, T=50000), nat.GDN_ERR_UNSUPPORTED),
    (dict(B=40000, num_seqs=40000, T=40000, D=64, G=8), nat.GDN_ERR_UNSUPPORTED),
    (dict(B=4000, num_seqs=4000, T=100000), nat.GDN_ERR_UNSUPPORTED),
])
def test_scan_problem(lib, kw, status):
    p = scan_problem(**kw)
    for pass_ in (nat.GDN_SCAN_FWD, nat.GDN_SCAN_SAVED, nat.GDN_SCAN_BWD):
        assert scan_size(p, pass_)[0] == status
    assert lib.gdn_scan_fwd(p, *[at(i) for i in range(12)], BIG, None) == status
    assert lib.gdn_scan_fwd_save(p, *[at(i) for i in range(12)], BIG, at(12), BIG, None) == status
    assert lib.gdn_scan_bwd_saved(p, *[at(i) for i in range(11)], BIG, *[at(i) for i in range(11, 21)], BIG, None) == status
    assert lib.gdn_scan_step(p, *[at(i) for i in range(10)], None) == status


def test_scan_sizes():
    p = scan_problem()
    # short sequences: no split; a kept state every 16 tokens, 80 / 16 + 2 + 1 slots
    assert scan_size(p, nat.GDN_SCAN_FWD) == (nat.GDN_OK, 0)
    assert scan_size(p, nat.GDN_SCAN_SAVED) == (nat.GDN_OK, 8 * 64 * 16 * 4)
    st, n = scan_size(p, nat.GDN_SCAN_BWD)
    assert st == nat.GDN_OK and n >= 80 * 2 * 16 * 4 + 2 * 64 * 18 * 4
    assert scan_size(p, 3)[0] == nat.GDN_ERR_UNSUPPORTED
    # one long sequence of few channels: segment states and sums
    st, n = scan_size(scan_problem(B=1, num_seqs=1, T=4096), nat.GDN_SCAN_FWD)
    assert st == nat.GDN_OK and n >= 64 * 17 * 4 * 2
    # no sequences and no tokens need next to nothing
    assert scan_size(scan_problem(B=0, num_seqs=0), nat.GDN_SCAN_BWD) == (nat.GDN_OK, 0)
    # a large batch stays within 64-bit sizes
    st, n = scan_size(scan_problem(B=2000, num_seqs=2000, T=100000, D=8192), nat.GDN_SCAN_BWD)
    assert st == nat.GDN_OK and n > 1 << 40
    # many short packed sequences beside a long one: slots by tokens, not by the longest
    cu = [0] + list(range(8192, 8192 + 5001))
    p = scan_problem(B=1, T=cu[-1], num_seqs=len(cu) - 1, D=1024, cu_seqlens_host=offsets(cu), cu_seqlens_dev=P)
    st, n = scan_size(p, nat.GDN_SCAN_FWD)
    assert st == nat.GDN_OK and n < 5600 * 1024 * 17 * 4


def test_scan_pointers(lib):
    p = scan_problem()
    need = {k: scan_size(p, v)[1] for k, v in dict(fwd=0, saved=1, bwd=2).items()}
    base = [at(i) for i in range(12)]
    optional = {5, 6, 7, 8, 10, 11}
    for slot in range(11):
        ptrs = list(base)
        if slot not in optional:
            ptrs[slot] = None
            assert lib.gdn_scan_fwd(p, *ptrs, 0, None) == nat.GDN_ERR_NULL, slot
        ptrs[slot] = at(slot, 4)
        assert lib.gdn_scan_fwd(p, *ptrs, 0, None) == nat.GDN_ERR_ALIGN, slot
        if slot != 9:
            ptrs[slot] = at(9)
            assert lib.gdn_scan_fwd(p, *ptrs, 0, None) == nat.GDN_ERR_ALIAS, slot
    assert lib.gdn_scan_fwd_save(p, *base[:11], None, need["saved"], None, 0, None) == nat.GDN_ERR_WORKSPACE
    assert lib.gdn_scan_fwd_save(p, *base, need["saved"] - 1, None, 0, None) == nat.GDN_ERR_WORKSPACE
    # the split's workspace
    long = scan_problem(B=1, num_seqs=1, T=4096)
    n = scan_size(long, nat.GDN_SCAN_FWD)[1]
    assert lib.gdn_scan_fwd(long, *base, n - 1, None) == nat.GDN_ERR_WORKSPACE
    assert lib.gdn_scan_fwd(long, *base[:11], None, n, None) == nat.GDN_ERR_WORKSPACE
    bwd = [at(i) for i in range(21)]

    def call(ptrs, nsaved=need["saved"], nws=need["bwd"]):
        return lib.gdn_scan_bwd_saved(p, *ptrs[:11], nsaved, *ptrs[11:], nws, None)

    optional = {5, 6, 7, 9, 16, 17, 18, 19}
    for slot in range(20):
        ptrs = list(bwd)
        if slot not in optional:
            ptrs[slot] = None
            want = nat.GDN_ERR_WORKSPACE if slot == 10 else nat.GDN_ERR_NULL
            assert call(ptrs) == want, slot
        if slot != 11:
            ptrs[slot] = at(11)
            assert call(ptrs) == nat.GDN_ERR_ALIAS, slot
    ptrs = list(bwd)
    ptrs[6] = None  # dz without z
    assert call(ptrs) == nat.GDN_ERR_NULL
    assert call(bwd, nsaved=need["saved"] - 1) == nat.GDN_ERR_WORKSPACE
    assert call(bwd, nws=need["bwd"] - 1) == nat.GDN_ERR_WORKSPACE


# --------------------------------------------------------------------------- Python calls

class _NoCalls:
    def __getattr__(self, name):
        if name.startswith("gdn_"):
            raise AssertionError(f"library entry point {name} reached before the checks")
        raise AttributeError(name)


def test_host_tensors_are_refused(monkeypatch):
    monkeypatch.setattr(nat, "load", lambda: _NoCalls())
    f = torch.zeros
    q, S = f(1, 1, 2, 64), f(1, 2, 64, 64)
    with pytest.raises(ValueError, match="q must be on a GPU"):
        layer.step(q, q, q, f(1, 1, 2), f(1, 1, 2), S)
    with pytest.raises(ValueError, match="q must be on a GPU"):
        layer.kda_step(q, q, q, q, f(1, 1, 2), S)
    x, w = f(1, 5, 16), f(16, 4)
    with pytest.raises(ValueError, match="x must be on a GPU"):
        layer.conv_fwd(x, w)
    with pytest.raises(ValueError, match="x must be on a GPU"):
        layer.conv_bwd(x, w, x)
    with pytest.raises(ValueError, match="x must be on a GPU"):
        layer.conv_step(x, w, f(1, 3, 16))
    u, A, B = f(1, 5, 16), f(16, 16), f(1, 5, 1, 16)
    for call in (lambda: layer.scan_fwd(u, u, A, B, B), lambda: layer.scan_fwd_save(u, u, A, B, B),
                 lambda: layer.scan_bwd_saved(u, u, A, B, B, u, f(4)), lambda: layer.scan_step(u, u, A, B, B, f(1, 16, 16)),
                 lambda: layer.scan_buffers(u, B)):
        with pytest.raises(ValueError, match="u must be on a GPU"):
            call()
    with pytest.raises(TypeError):
        layer.conv_fwd([1.0], w)


def test_want_names_what_is_wrong():
    dev = -1  # what get_device() gives for host tensors
    t = torch.zeros(3, 4)
    assert layer._want(t, (3, 4), torch.float32, dev, "t") == t.data_ptr()
    with pytest.raises(ValueError, match="shape"):
        layer._want(t, (4, 3), torch.float32, dev, "t")
    with pytest.raises(TypeError, match="bfloat16"):
        layer._want(t, (3, 4), torch.bfloat16, dev, "t")
    with pytest.raises(ValueError, match="contiguous"):
        layer._want(t.t(), (4, 3), torch.float32, dev, "t")
    with pytest.raises(ValueError, match="must be on"):
        layer._want(t, (3, 4), torch.float32, 0, "t")
    for bad in (None, [1.0]):
        with pytest.raises(TypeError):
            layer._want(bad, (3, 4), torch.float32, dev, "t")
    assert layer._may(None, (3, 4), torch.float32, dev, "t") is None
