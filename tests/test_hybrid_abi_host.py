"""Host-side checks of the C ABI of gdn_glr_*, gdn_rope_* and gdn_swa_*, and of their Python
calls (CPU only: no kernel is launched; pointers passed here are never dereferenced)."""
import ctypes

import numpy as np
import pytest
import torch

from gated_deltanet_chunked_gdn_amd import _native as nat
from gated_deltanet_chunked_gdn_amd import hybrid

P = 0x10000000  # an address that is 16-byte aligned and never read
BIG = 1 << 40   # distance between the addresses of different tensors
OK, NULL, SHAPE, DTYPE = nat.GDN_OK, nat.GDN_ERR_NULL, nat.GDN_ERR_SHAPE, nat.GDN_ERR_DTYPE
ALIGN, ALIAS, SEQS, UNSUP, WS = (nat.GDN_ERR_ALIGN, nat.GDN_ERR_ALIAS, nat.GDN_ERR_SEQLENS, nat.GDN_ERR_UNSUPPORTED,
                                 nat.GDN_ERR_WORKSPACE)


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


class Call:
    """One entry point: the problem that passes every check, and its pointers as 'i' (an input),
    'o' (an output; capitals may be NULL) or 'w' (a buffer that has to be there, with its bytes)."""

    def __init__(self, name, make, slots, align=None):
        self.name, self.make, self.slots, self.align = name, make, slots, align or {}

    def args(self, change=None):
        out = []
        for n, kind in enumerate(self.slots):
            ptr = at(n) if not change or n not in change else change[n]
            out += [ptr, BIG // 2] if kind in "wr" else [ptr]
        return out

    def __call__(self, lib, p=None, change=None):
        return getattr(lib, self.name)(self.make() if p is None else p, *self.args(change), None)


def glr(**kw):
    d = dict(B=2, T=300, C=64, num_seqs=2, io_dtype=nat.GDN_BF16, c=8.0)
    return nat.GlrProblem(**(d | kw))


def rope(**kw):
    d = dict(B=2, T=5, Hq=4, Hk=2, D=64, R=32, norm=nat.GDN_ROPE_RMS, interleaved=0, io_dtype=nat.GDN_BF16, eps=1e-6)
    return nat.RopeProblem(**(d | kw))


def swa(**kw):
    d = dict(B=2, T=300, Hq=4, Hk=2, D=64, window=100, sinks=4, num_seqs=2, io_dtype=nat.GDN_BF16, scale=1.0)
    return nat.SwaProblem(**(d | kw))


def one(**kw):
    return swa(**(dict(T=1, window=1000) | kw))


# lam, floats and positions: in the order of the header; w: workspace, r: a read buffer
CALLS = {
    "gdn_glr_fwd": Call("gdn_glr_fwd", glr, "iiiiIIoOw"),
    "gdn_glr_fwd_save": Call("gdn_glr_fwd_save", glr, "iiiiIIoOww"),
    "gdn_glr_bwd_saved": Call("gdn_glr_bwd_saved", glr, "iiiiIiIroooo" + "OOw"),
    "gdn_glr_step": Call("gdn_glr_step", lambda **kw: glr(**(dict(T=1) | kw)), "iiiiIoo"),
    "gdn_rope_fwd": Call("gdn_rope_fwd", rope, "iiiIIIoo", {2: 4, 3: 4}),
    "gdn_rope_bwd": Call("gdn_rope_bwd", rope, "iiiIIIiiooOOw", {2: 4, 3: 4}),
    "gdn_swa_fwd": Call("gdn_swa_fwd", swa, "iiioO", {4: 4}),
    "gdn_swa_bwd": Call("gdn_swa_bwd", swa, "iiiiiiooow", {4: 4}),
    "gdn_swa_fill": Call("gdn_swa_fill", swa, "iioo"),
    "gdn_swa_step": Call("gdn_swa_step", one, "iiiooiow", {5: 4}),
}
SIZES = [("gdn_glr_workspace_size", glr, range(3)), ("gdn_rope_workspace_size", rope, None), ("gdn_swa_workspace_size", swa, range(2))]


def kinds(prefix):
    return [c for n, c in CALLS.items() if n.startswith(prefix)]


@pytest.mark.parametrize("name", CALLS)
def test_pointers(lib, name):
    call = CALLS[name]
    first_out = next(n for n, k in enumerate(call.slots) if k in "oO")
    assert call(lib, change={0: None}) == NULL and getattr(lib, name)(None, *call.args(), None) == NULL
    for n, kind in enumerate(call.slots):
        align = call.align.get(n, 16)
        assert call(lib, change={n: at(n, align // 2)}) == ALIGN, n
        if kind in "io":
            assert call(lib, change={n: None}) == NULL, n
        if kind == "w" or kind == "r":
            assert call(lib, change={n: None}) == WS, n
        if n != first_out:
            assert call(lib, change={n: at(first_out)}) == ALIAS, n


@pytest.mark.parametrize("name", CALLS)
def test_no_gpu_is_an_error(lib, name):
    """Arguments that pass every check reach the launch, which fails where there is no GPU."""
    if torch.cuda.is_available():
        pytest.skip("would launch on addresses that are not memory")
    assert CALLS[name](lib) == nat.GDN_ERR_HIP


@pytest.mark.parametrize("kw,status", [
    (dict(io_dtype=2), DTYPE), (dict(B=-1, num_seqs=-1), SHAPE), (dict(T=-1), SHAPE), (dict(C=0), SHAPE), (dict(C=12), UNSUP),
    (dict(C=(1 << 20) + 8), UNSUP), (dict(c=-1.0), UNSUP), (dict(c=float("nan")), UNSUP), (dict(num_seqs=1), SHAPE),
    (dict(B=70000, num_seqs=70000), UNSUP), (dict(B=60000, num_seqs=60000, T=60000), UNSUP), (dict(T=1 << 20, C=1 << 18), UNSUP)])
def test_glr_problem(lib, kw, status):
    for call in kinds("gdn_glr"):
        assert call(lib, call.make(**kw)) == status, call.name
    n = ctypes.c_size_t(7)
    for pass_ in range(3):
        assert lib.gdn_glr_workspace_size(glr(**kw), pass_, n) == status and n.value == 7


@pytest.mark.parametrize("kw,status", [
    (dict(io_dtype=2), DTYPE), (dict(B=-1), SHAPE), (dict(T=-1), SHAPE), (dict(Hq=0), SHAPE), (dict(Hk=0), SHAPE), (dict(D=0), SHAPE),
    (dict(R=80), SHAPE), (dict(R=-16), SHAPE), (dict(R=24), UNSUP), (dict(D=96), UNSUP), (dict(Hq=4097), UNSUP), (dict(norm=3), UNSUP),
    (dict(B=1 << 20, T=1 << 11), UNSUP), (dict(q_stride=255), SHAPE), (dict(q_stride=260), ALIGN), (dict(k_stride=(1 << 21) + 8), UNSUP)])
def test_rope_problem(lib, kw, status):
    for call in kinds("gdn_rope"):
        assert call(lib, call.make(**kw)) == status, call.name
    n = ctypes.c_size_t(7)
    assert lib.gdn_rope_workspace_size(rope(**kw), n) == status and n.value == 7


def test_rope_weights_need_their_norm(lib):
    for norm in (nat.GDN_ROPE_NONE, nat.GDN_ROPE_L2):
        for name, slots in (("gdn_rope_fwd", (4, 5)), ("gdn_rope_bwd", (4, 5, 10, 11))):
            for n in slots:
                others = {m: None for m in slots if m != n}
                assert CALLS[name](lib, rope(norm=norm), others) == UNSUP
    assert CALLS["gdn_rope_fwd"](lib, rope(R=0, B=0), {2: None}) == OK


@pytest.mark.parametrize("kw,status", [
    (dict(io_dtype=2), DTYPE), (dict(B=-1, num_seqs=-1), SHAPE), (dict(T=-1), SHAPE), (dict(Hq=3), SHAPE), (dict(Hk=0), SHAPE),
    (dict(window=0), SHAPE), (dict(window=-5), SHAPE), (dict(sinks=-1), SHAPE), (dict(sinks=1025), UNSUP), (dict(D=96), UNSUP),
    (dict(Hq=8192, Hk=1), UNSUP), (dict(num_seqs=3), SHAPE), (dict(B=70000, num_seqs=70000), UNSUP), (dict(q_stride=128), SHAPE),
    (dict(k_stride=132), ALIGN), (dict(v_stride=(1 << 21) + 8), UNSUP)])
def test_swa_problem(lib, kw, status):
    for call in kinds("gdn_swa"):
        assert call(lib, call.make(**kw)) == status, call.name
    n = ctypes.c_size_t(7)
    for pass_ in range(2):
        assert lib.gdn_swa_workspace_size(swa(**kw), pass_, n) == status and n.value == 7


def test_swa_limits(lib):
    fwd, fill, step = (CALLS["gdn_swa_" + n] for n in ("fwd", "fill", "step"))
    assert fwd(lib, swa(B=1 << 16, num_seqs=1 << 16, T=1)) == UNSUP
    assert fwd(lib, swa(B=2, T=(1 << 29) + 64)) == UNSUP
    assert fwd(lib, swa(B=60000, num_seqs=60000, T=2305)) == UNSUP  # workgroups
    for call in (fill, step):
        assert call(lib, call.make(window=(1 << 30) + 1)) == UNSUP
        assert call(lib, call.make(window=1 << 29, B=512, num_seqs=512)) == UNSUP  # pieces to fill
    assert step(lib, one(T=2)) == SHAPE
    assert step(lib, one(B=1, num_seqs=1, cu_seqlens_host=offsets([0, 1]), cu_seqlens_dev=P)) == SHAPE
    assert CALLS["gdn_glr_step"](lib, glr(T=2)) == SHAPE


@pytest.mark.parametrize("name", ["gdn_glr_fwd", "gdn_glr_fwd_save", "gdn_glr_bwd_saved", "gdn_swa_fwd", "gdn_swa_bwd", "gdn_swa_fill"])
def test_offsets(lib, name):
    call = CALLS[name]
    for cu in ([0, 3, 2, 5], [1, 5], [0, 4], [0, 6]):
        p = call.make(B=1, T=5, num_seqs=len(cu) - 1, cu_seqlens_host=offsets(cu), cu_seqlens_dev=P)
        assert call(lib, p) == SEQS, cu
    assert call(lib, call.make(B=1, T=5, num_seqs=1, cu_seqlens_host=offsets([0, 5]))) == NULL
    assert call(lib, call.make(B=1, T=5, num_seqs=1, cu_seqlens_dev=P)) == NULL
    assert call(lib, call.make(B=2, T=5, num_seqs=1, cu_seqlens_host=offsets([0, 5]), cu_seqlens_dev=P)) == SHAPE


def test_sizes(lib):
    n = ctypes.c_size_t(7)
    for name, make, passes in SIZES:
        f = getattr(lib, name)
        for a in ([()] if passes is None else [(i,) for i in passes]):
            assert f(make(), *a, None) == NULL and f(None, *a, n) == NULL and n.value == 7
        if passes is not None:
            for bad in (-1, len(passes)):
                assert f(make(), bad, n) == UNSUP and n.value == 7
    # short buffers
    for name, make, pass_, slot in (("gdn_glr_fwd", glr, nat.GDN_GLR_FWD, 8), ("gdn_glr_fwd_save", glr, nat.GDN_GLR_SAVED, 8),
                                    ("gdn_glr_fwd_save", glr, nat.GDN_GLR_FWD, 9), ("gdn_glr_bwd_saved", glr, nat.GDN_GLR_SAVED, 7),
                                    ("gdn_glr_bwd_saved", glr, nat.GDN_GLR_BWD, 14), ("gdn_swa_bwd", swa, nat.GDN_SWA_BWD, 9),
                                    ("gdn_swa_step", one, nat.GDN_SWA_STEP, 7)):
        size = getattr(lib, "gdn_glr_workspace_size" if make is glr else "gdn_swa_workspace_size")
        assert size(make(), pass_, n) == OK and n.value > 0, (name, pass_)
        call, args = CALLS[name], CALLS[name].args()
        args[slot + sum(k in "wr" for k in call.slots[:slot]) + 1] = n.value - 1
        assert getattr(lib, name)(make(), *args, None) == WS, name
    # one segment passes nothing on
    assert lib.gdn_glr_workspace_size(glr(T=128), nat.GDN_GLR_FWD, n) == OK and n.value == 0


def test_nothing_to_do(lib):
    """No sequences and no tokens: no tensor is needed and nothing is launched."""
    for name in CALLS:
        call = CALLS[name]
        if name == "gdn_glr_bwd_saved" or name == "gdn_rope_bwd":
            continue  # write the parameters' gradients, zero
        p = call.make(B=0) if name.startswith("gdn_rope") else call.make(B=0, num_seqs=0)
        optional = {n: None for n, k in enumerate(call.slots) if name.startswith("gdn_swa") or (name.startswith("gdn_glr") and n != 3 and k not in "w")}
        assert call(lib, p, optional) == OK, name


# --------------------------------------------------------------------------- Python calls

def test_host_tensors_are_refused():
    x, lam = torch.zeros(1, 4, 64), torch.zeros(64)
    q, k = torch.zeros(1, 4, 2, 64), torch.zeros(1, 4, 1, 64)
    f, cache, lens = torch.zeros(16), torch.zeros(1, 8, 1, 64), torch.zeros(1, dtype=torch.int32)
    for call in (lambda: hybrid.glr_fwd(x, x, x, lam), lambda: hybrid.glr_fwd_save(x, x, x, lam), lambda: hybrid.glr_buffers(x),
                 lambda: hybrid.glr_bwd_saved(x, x, x, lam, x, lam), lambda: hybrid.glr_step(x, x, x, lam, lam),
                 lambda: hybrid.rope_fwd(q, k, f), lambda: hybrid.rope_bwd(q, k, f, q, k), lambda: hybrid.swa_fwd(q, k, k, 4),
                 lambda: hybrid.swa_bwd(q, k, k, q, lam, q, 4), lambda: hybrid.swa_fill(k, k, cache, cache),
                 lambda: hybrid.swa_step(q, k, k, cache, cache, lens)):
        with pytest.raises(ValueError, match="GPU device"):
            call()
    for call in (lambda: hybrid.glr_fwd([1], x, x, lam), lambda: hybrid.rope_fwd(1, k, f), lambda: hybrid.swa_fwd(None, k, k, 4)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(ValueError, match="kcache"):
        hybrid.swa_step(q, k, k, cache, cache, lens, sinks=8)  # no window left


def test_sizes_beyond_32_bits_are_refused():
    with pytest.raises(ValueError, match="32 bits"):
        hybrid._problem(nat.SwaProblem, (1, 2, 2, 1, 64, 1 << 31, 0, 1), None, None, 0, 1.0, 0, 0, 0)


class _Rows(torch.Tensor):
    """A host tensor that says it is on device 0, for the checks of strides alone."""
    def get_device(self):
        return 0


@pytest.mark.parametrize("T", [1, 6])
def test_rows(T):
    base = torch.zeros(2, T, 5 * 64).as_subclass(_Rows)
    q, k = (t.unflatten(-1, (-1, 64)) for t in base.split([3 * 64, 2 * 64], dim=-1))
    assert hybrid._rows(q, q.shape, torch.float32, 0, "q") == (base.data_ptr(), 320)
    assert hybrid._rows(k, k.shape, torch.float32, 0, "k") == (base.data_ptr() + 3 * 256, 320)
    for bad in (*([q.transpose(0, 1)] if T > 1 else []), q.flip(1)[:, :, ::2], q[..., ::2], q[:1].expand(2, T, 3, 64)):
        if not bad.is_contiguous():
            with pytest.raises(ValueError, match="contiguous"):
                hybrid._rows(bad, bad.shape, torch.float32, 0, "q")


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_factors_that_are_not_finite(lib, bad):
    """An infinite c has no gradient (a la is zero times infinity), and the running maximum has no
    base with a scale that is not finite."""
    n = ctypes.c_size_t(7)
    for call in kinds("gdn_glr"):
        assert call(lib, call.make(c=bad)) == UNSUP, call.name
    for call in kinds("gdn_swa"):
        assert call(lib, call.make(scale=bad)) == UNSUP, call.name
    for pass_ in range(3):
        assert lib.gdn_glr_workspace_size(glr(c=bad), pass_, n) == UNSUP and n.value == 7
    for pass_ in range(2):
        assert lib.gdn_swa_workspace_size(swa(scale=bad), pass_, n) == UNSUP and n.value == 7


def test_one_long_sequence_beside_many_short_ones(lib):
    """Blocks are counted by what the sequences hold, not by the longest one's length."""
    n = ctypes.c_size_t(7)
    for long, many, each in ((32768, 1100, 8), (16384, 2100, 16), (4096, 60000, 1), (128, 65000, 0)):
        cu = np.concatenate([[0], long + each * np.arange(many + 1)])
        p = swa(B=1, T=int(cu[-1]), Hq=16, Hk=4, D=128, window=1024, sinks=4, num_seqs=len(cu) - 1, cu_seqlens_host=offsets(cu), cu_seqlens_dev=P)
        assert lib.gdn_swa_workspace_size(p, nat.GDN_SWA_BWD, n) == OK and n.value > 0
        if not torch.cuda.is_available():  # they reach the launch
            for name in ("gdn_swa_fwd", "gdn_swa_bwd", "gdn_swa_fill"):
                assert CALLS[name](lib, p) == nat.GDN_ERR_HIP, name
    # too many blocks for the attention, which filling the cache has none of
    cu = np.arange(0, 33 * 65535 + 1, 33)
    p = swa(B=1, T=int(cu[-1]), Hq=132, Hk=1, num_seqs=65535, cu_seqlens_host=offsets(cu), cu_seqlens_dev=P)
    assert CALLS["gdn_swa_fwd"](lib, p) == UNSUP and lib.gdn_swa_workspace_size(p, nat.GDN_SWA_BWD, n) == UNSUP
    if not torch.cuda.is_available():
        assert CALLS["gdn_swa_fill"](lib, p) == nat.GDN_ERR_HIP
