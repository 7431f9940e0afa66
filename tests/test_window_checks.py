"""Refusals of the windowed attention, the paged cache and the attention over it: by the C ABI
(fake pointers, never dereferenced: the checks come first) and by the binding. CPU only."""
import ctypes
import os
import re

import pytest

torch = pytest.importorskip("torch")

import block_sparse_attention_pisa_b200 as P  # noqa: E402
from block_sparse_attention_pisa_b200 import build as B  # noqa: E402

OK, INVALID, UNSUPPORTED = 0, 1, 2
FAKE = 0x7f0000100000
BF, F32, I32, E4M3 = torch.bfloat16, torch.float32, torch.int32, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def L():
    B.build()
    return P.lib()


def vp(x):
    return ctypes.c_void_p(x)


def shape(B=1, Hq=4, Hkv=2, N=256, d=64):
    return P.WindowShape(B, Hq, Hkv, N, d)


def win(left=-1, right=0, sinks=0):
    return P.Window(left, right, sinks)


def fwd(L, s=None, w=None, scale=0.1, **p):
    a = {k: FAKE for k in ("Q", "K", "V", "O", "lse")} | p
    return L.pisa_window_attention(vp(a["Q"]), vp(a["K"]), vp(a["V"]), s or shape(), w or win(), scale, vp(a["O"]),
                                   vp(a["lse"]), None)


def bwd(L, s=None, w=None, scale=0.1, ws=FAKE, nbytes=1 << 40, **p):
    a = {k: FAKE for k in ("dO", "Q", "K", "V", "O", "lse", "dQ", "dK", "dV")} | p
    return L.pisa_window_attention_backward(*[vp(a[k]) for k in ("dO", "Q", "K", "V", "O", "lse")], s or shape(),
                                            w or win(), scale, vp(a["dQ"]), vp(a["dK"]), vp(a["dV"]), vp(ws), nbytes, None)


def cache(K=FAKE, V=FAKE, ks=FAKE, vs=FAKE, num_pages=9, Hkv=2, page=16, d=64, type=1):
    return P.CacheArgs(K, V, ks, vs, num_pages, Hkv, page, d, type)


def seqs(table=FAKE, kv=FAKE, q=None, B=2, N=3, max_pages=4):
    return P.Sequences(table, kv, q, B, N, max_pages)


def paged(L, c=None, s=None, Hq=4, w=None, scale=0.1, Q=FAKE, O=FAKE, lse=FAKE, ws=FAKE, nbytes=1 << 40):
    return L.pisa_paged_attention(vp(Q), c or cache(), s or seqs(), Hq, w or win(), scale, vp(O), vp(lse), vp(ws),
                                  nbytes, None)


def test_window_pointers(L):
    for name in ("Q", "K", "V", "O"):
        assert fwd(L, **{name: 0}) == INVALID and name.encode() in L.pisa_last_error()
        assert fwd(L, **{name: FAKE + 8}) == INVALID and b"16-byte" in L.pisa_last_error()
    assert fwd(L, lse=FAKE + 2) == INVALID
    for name in ("dO", "Q", "K", "V", "O", "lse", "dQ", "dK", "dV"):
        assert bwd(L, **{name: 0}) == INVALID and name.encode() in L.pisa_last_error()
    assert bwd(L, ws=0) == INVALID and bwd(L, ws=FAKE + 16) == INVALID
    assert bwd(L, nbytes=16) == INVALID and b"workspace" in L.pisa_last_error()


@pytest.mark.parametrize("bad,status", [
    (dict(B=-1), INVALID), (dict(Hq=3), INVALID), (dict(Hkv=0), INVALID), (dict(d=0), INVALID),
    (dict(d=96), UNSUPPORTED), (dict(N=(1 << 30) + 1), UNSUPPORTED), (dict(B=1 << 15, Hq=1 << 10, N=1 << 10), UNSUPPORTED),
    (dict(B=2 ** 31 - 1, Hq=2 ** 31 - 1, Hkv=1), UNSUPPORTED),
])
def test_window_shapes(L, bad, status):
    n = ctypes.c_size_t()
    assert fwd(L, shape(**bad)) == status and bwd(L, shape(**bad)) == status
    assert L.pisa_window_attention_backward_workspace(shape(**bad), win(), ctypes.byref(n)) == status


@pytest.mark.parametrize("w", [win(left=-2), win(right=-7), win(sinks=-1)])
def test_windows(L, w):
    n = ctypes.c_size_t()
    assert fwd(L, w=w) == INVALID and bwd(L, w=w) == INVALID and paged(L, w=w) == INVALID
    assert L.pisa_window_attention_backward_workspace(shape(), w, ctypes.byref(n)) == INVALID
    assert L.pisa_paged_attention_workspace(cache(), seqs(), 4, w, ctypes.byref(n)) == INVALID


@pytest.mark.parametrize("scale", [0.0, -1.0, float("nan"), float("inf")])
def test_scales(L, scale):
    assert fwd(L, scale=scale) == INVALID and bwd(L, scale=scale) == INVALID and paged(L, scale=scale) == INVALID


def test_nothing_to_do_touches_nothing(L):
    for s in (shape(B=0), shape(N=0), shape(Hq=0)):
        assert fwd(L, s, Q=0, K=0, V=0, O=0, lse=0) == OK
        assert bwd(L, s, ws=0, nbytes=0, dO=0, Q=0, dQ=0) == OK
    assert paged(L, s=seqs(B=0, table=None, kv=None), Q=0, O=0, ws=0, nbytes=0) == OK
    assert L.pisa_cache_write(vp(0), vp(0), cache(K=None), seqs(N=0), None) == OK
    assert L.pisa_cache_read(cache(K=None), seqs(B=0), vp(0), vp(0), None) == OK


@pytest.mark.parametrize("c,s,status", [
    (dict(K=None), {}, INVALID), (dict(V=FAKE + 4), {}, INVALID), (dict(ks=None), {}, INVALID), (dict(vs=None), {}, INVALID),
    (dict(num_pages=0), {}, INVALID), (dict(page=0), {}, INVALID), (dict(page=-16), {}, INVALID), (dict(page=48), {}, UNSUPPORTED),
    (dict(page=256), {}, UNSUPPORTED), (dict(d=32), {}, UNSUPPORTED), (dict(type=2), {}, INVALID),
    (dict(num_pages=2 ** 31 - 1), {}, UNSUPPORTED), ({}, dict(table=None), INVALID), ({}, dict(kv=None), INVALID),
    ({}, dict(kv=FAKE + 1), INVALID), ({}, dict(q=FAKE + 2), INVALID), ({}, dict(max_pages=0), INVALID),
    ({}, dict(max_pages=2 ** 30), UNSUPPORTED), ({}, dict(B=-1), INVALID),
])
def test_caches(L, c, s, status):
    n = ctypes.c_size_t()
    assert paged(L, cache(**c), seqs(**s)) == status
    assert L.pisa_paged_attention_workspace(cache(**c), seqs(**s), 4, win(), ctypes.byref(n)) == status
    assert L.pisa_cache_write(vp(FAKE), vp(FAKE), cache(**c), seqs(**s), None) == status
    if "q" not in s:  # not used by the reading call
        assert L.pisa_cache_read(cache(**c), seqs(**s), vp(FAKE), vp(FAKE), None) == status


def test_paged_operands(L):
    assert paged(L, Q=0) == INVALID and paged(L, O=FAKE + 4) == INVALID and paged(L, lse=FAKE + 1) == INVALID
    assert paged(L, Hq=3) == INVALID
    assert L.pisa_cache_write(vp(0), vp(FAKE), cache(), seqs(), None) == INVALID
    assert L.pisa_cache_read(cache(), seqs(), vp(FAKE), vp(FAKE + 2), None) == INVALID
    assert L.pisa_paged_attention_workspace(cache(), seqs(), 4, win(), None) == INVALID
    assert L.pisa_window_attention_backward_workspace(shape(), win(), None) == INVALID


# ------------------------------------------------------------------ the binding

def q(h=4, N=8, d=64, dtype=BF):
    return torch.zeros(1, h, N, d, dtype=dtype)


def test_binding_refuses_wrong_tensors(L):
    lse = torch.zeros(1, 4, 8)
    with pytest.raises(ValueError, match="CUDA"):
        P.window_attention(q(), q(2), q(2))
    for bad in ((q(dtype=F32), q(2), q(2)), (q(), q(2, N=9), q(2)), (q(), q(2), q(4)), (q(), q(2, d=128), q(2)),
                (q()[0], q(2), q(2)), (q(d=128)[..., ::2], q(2), q(2))):
        with pytest.raises(ValueError):
            P.window_attention(*bad)
    with pytest.raises(ValueError, match="lse"):
        P.window_attention(q(), q(2), q(2), lse=lse.double())
    with pytest.raises(ValueError, match="O"):
        P.window_attention(q(), q(2), q(2), out=q(2))
    with pytest.raises(ValueError, match="dO"):
        P.window_attention_backward(q(2), q(), q(2), q(2), q(), lse)
    with pytest.raises(ValueError, match="dK"):
        P.window_attention_backward(q(), q(), q(2), q(2), q(), lse, out=(q(), q(), q(2)))
    with pytest.raises(ValueError, match="32 bits"):
        P.window_attention_backward_workspace(1, 4, 2, 8, 64, left=2 ** 31)


def test_binding_refuses_wrong_caches(L):
    c = P.paged_cache(4, 2, 16, 64, E4M3, device="cpu")
    table, lens = torch.zeros(1, 3, dtype=I32), torch.zeros(1, dtype=I32)

    def args(cache=c, table=table, lens=lens, news=None):
        with pytest.raises(ValueError, match="CUDA"):  # host tensors: refused last
            P._check_operands(P._cache_checks(cache, table, lens, news, 1))
        return P._cache_args(cache, table, lens, news, 1, 8)

    a, s = args()
    assert (a.num_pages, a.Hkv, a.page, a.d, a.type, s.B, s.N, s.max_pages) == (4, 2, 16, 64, 1, 1, 8, 3)
    bad = [dict(cache=c._replace(k_scale=None)), dict(cache=c._replace(v_scale=c.v_scale.double())),
           dict(cache=c._replace(V=c.V[:3])), dict(cache=c._replace(K=c.K.float())), dict(cache=c._replace(K=c.K[0])),
           dict(table=table.long()), dict(table=table[0]), dict(table=torch.zeros(2, 3, dtype=I32)),
           dict(lens=lens.long()), dict(lens=torch.zeros(2, dtype=I32)), dict(news=torch.zeros(1)),
           dict(table=torch.zeros(1, 6, dtype=I32)[:, ::2])]
    for kw in bad:
        a = dict(cache=c, table=table, lens=lens, news=None) | kw
        with pytest.raises(ValueError) as e:
            P._check_operands(P._cache_checks(a["cache"], a["table"], a["lens"], a["news"], 1))
        assert "CUDA" not in str(e.value), kw
    with pytest.raises(ValueError, match="dtype"):
        P.paged_cache(4, 2, 16, 64, torch.float16, device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        P.paged_attention(q(), c, table, lens)
    with pytest.raises(ValueError, match="CUDA"):
        P.cache_write(q(2), q(2), c, table, lens)
    with pytest.raises(ValueError, match="CUDA"):
        P.cache_read(c, table, lens, 8)
    with pytest.raises(ValueError, match="V"):
        P.cache_write(q(2), q(2, N=9), c, table, lens)


def test_binding_refuses_wrong_workspaces():
    cpu = torch.device("cpu")
    for bad in (torch.zeros(8), torch.zeros(4, dtype=torch.uint8), torch.zeros(32, dtype=torch.uint8)[::2], "no"):
        with pytest.raises(ValueError, match="workspace"):
            P._workspace(bad, 16, cpu)
    assert P._workspace(torch.zeros(16, dtype=torch.uint8), 16, cpu)[1] == 16
    assert P._workspace(None, 0, cpu) == (None, 0, None)


def test_outputs_cannot_be_given_while_autograd_records(L):
    for kw in (dict(out=q()), dict(lse=torch.zeros(1, 4, 8))):
        for need in range(3):
            ops = [q(), q(2), q(2)]
            ops[need].requires_grad_()
            with pytest.raises(ValueError, match="autograd"):
                P.window_attention(*ops, **kw)
            with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):  # host tensors: refused last
                P.window_attention(*ops, **kw)
            with pytest.raises(ValueError, match="CUDA"):
                P.window_attention(*ops)


def test_sizes_past_32_bits_are_refused(L):
    """ctypes would take them modulo 2^32."""
    good = dict(B=1, Hq=4, Hkv=2, N=8, d=64)
    assert P.window_attention_backward_workspace(**good) > 0
    for name in good:
        for x in (good[name] + 2 ** 32, -2 ** 31 - 1):
            with pytest.raises(ValueError, match=name):
                P.window_attention_backward_workspace(**(good | {name: x}))


# ------------------------------------------------------------------ the sources

def test_kernels_that_start_early_read_no_results_as_constants():
    """A kernel that starts beside the one before it (and waits) may not load through the read-only
    path: what it reads may still have been written when it started."""
    early = 0
    for name in sorted(os.listdir(B.CSRC)):
        with open(os.path.join(B.CSRC, name)) as f:
            text = f.read()
        for part in re.split(r"(?=__global__ )", text)[1:]:
            body = part[:part.index("\n}\n")]
            if "griddepcontrol.wait" in body:
                early += 1
                assert not re.search(r"__ldg\b|ldg_stream|ldg16|ld\.global\.nc|__restrict__", body), (name, body[:80])
    assert early == 4
