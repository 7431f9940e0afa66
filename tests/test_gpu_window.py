"""Windowed attention and its gradient on the GPU against the fp64 oracle."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import block_sparse_attention_pisa_b200 as P  # noqa: E402
from oracle import window as W  # noqa: E402
from tests import window_bounds as T  # noqa: E402

pytestmark = pytest.mark.gpu

# (B, Hq, Hkv, N, d, left, right, sinks)
SHAPES = [
    (1, 1, 1, 1, 64, -1, 0, 0),            # one token
    (1, 2, 1, 2, 128, 0, 0, 0),            # every token sees itself only
    (1, 3, 1, 127, 64, -1, -1, 0),         # whole sequence, three heads per key head, odd length
    (2, 4, 2, 128, 128, -1, 0, 0),         # causal, one tile
    (1, 4, 4, 129, 64, 16, 0, 0),          # one token over a tile
    (1, 2, 2, 257, 128, 5, 7, 3),          # both sides, odd reaches, sinks
    (1, 8, 2, 300, 64, 31, 0, 1),          # sinks of one token
    (1, 2, 1, 520, 128, 40, 0, 130),       # sinks over a tile's edge
    (1, 5, 1, 401, 64, 64, 64, 0),         # group of five
    (1, 7, 1, 200, 128, 20, 0, 4),         # group of seven: rows of a tile end inside a token
    (2, 2, 2, 700, 64, 100, 0, 600),       # sinks longer than the window
    (1, 2, 2, 384, 128, -1, 5, 0),         # no limit to the left, a few to the right
    (1, 2, 1, 390, 64, 0, -1, 2),          # none before its own, all behind it
    (3, 6, 3, 65, 128, 1000000000, 2000000000, 2000000000),  # reaches far past the end
    (1, 16, 1, 150, 64, 33, 0, 8),         # sixteen heads on one key head
    (1, 130, 1, 12, 64, 4, 0, 1),          # more heads of a group than rows of a tile
]


def make(B, Hq, Hkv, N, d, seed=0, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    new = lambda h, s=1.0: (torch.randn(B, h, N, d, generator=g) * s).to(torch.bfloat16).cuda()  # noqa: E731
    return new(Hq, spread), new(Hkv, spread), new(Hkv), new(Hq)


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def check_forward(O, lse, Q, K, V, left, right, sinks, scale, heads=None):
    q, k, v, o, l = (f64(t) for t in (Q, K, V, O, lse))
    B, Hq, N, _ = q.shape
    G = Hq // k.shape[1]
    see = W.visible(np.arange(N), N, left, right, sinks)
    want = np.zeros_like(q)
    for b in range(B):
        for h in range(Hq) if heads is None else heads:
            want[b, h], wl, to, tl = T.forward(q[b, h], k[b, h // G], v[b, h // G], see, scale)
            T.check(o[b, h], want[b, h], to, f"O[{b},{h}]")
            T.check(l[b, h], wl, tl, f"lse[{b},{h}]")
    if heads is None:
        T.check_norm(o, want, "O")


def check_backward(grads, dO, Q, K, V, left, right, sinks, scale, norms=True):
    do, q, k, v = (f64(t) for t in (dO, Q, K, V))
    dQ, dK, dV = (f64(t) for t in grads)
    B, Hq, N, _ = q.shape
    G = Hq // k.shape[1]
    see = W.visible(np.arange(N), N, left, right, sinks)
    wq, tq = np.zeros_like(q), np.zeros_like(q)
    wk, wv, tk, tv = (np.zeros_like(k) for _ in range(4))
    for b in range(B):
        for h in range(Hq):
            dq, dk, dv, a, c, e = T.backward(do[b, h], q[b, h], k[b, h // G], v[b, h // G], see, scale)
            wq[b, h], tq[b, h] = dq, a
            wk[b, h // G] += dk
            wv[b, h // G] += dv
            tk[b, h // G] += c
            tv[b, h // G] += e
    T.check(dQ, wq, tq, "dQ")
    T.check(dK, wk, tk + T.U * np.abs(wk) * T.SLACK, "dK")
    T.check(dV, wv, tv + T.U * np.abs(wv) * T.SLACK, "dV")
    if norms:
        for got, want, name in ((dQ, wq, "dQ"), (dK, wk, "dK"), (dV, wv, "dV")):
            T.check_norm(got, want, name)


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward_and_gradient(shape):
    B, Hq, Hkv, N, d, left, right, sinks = shape
    Q, K, V, dO = make(B, Hq, Hkv, N, d, seed=N)
    mask = dict(left=left, right=right, sinks=sinks)
    O, lse = P.window_attention(Q, K, V, **mask)
    P.device_error()
    check_forward(O, lse, Q, K, V, left, right, sinks, d ** -0.5)
    grads = P.window_attention_backward(dO, Q, K, V, O, lse, **mask)
    P.device_error()
    # with few keys per row ds cancels: dQ, dK are small beside what their roundings are relative to
    check_backward(grads, dO, Q, K, V, left, right, sinks, d ** -0.5, norms=N > 100)


@pytest.mark.parametrize("d", [64, 128])
def test_scale_and_large_scores(d):
    """Scores of several hundred: the running maximum moves by much more than one rescale step."""
    Q, K, V, dO = make(1, 2, 1, 333, d, seed=5, spread=6.0)
    mask = dict(left=150, right=0, sinks=10, scale=0.5)
    O, lse = P.window_attention(Q, K, V, **mask)
    check_forward(O, lse, Q, K, V, 150, 0, 10, 0.5)
    check_backward(P.window_attention_backward(dO, Q, K, V, O, lse, **mask), dO, Q, K, V, 150, 0, 10, 0.5, norms=False)


def test_growing_scores_rescale():
    """Keys grow along the sequence, so every tile raises the maximum."""
    Q, K, V, dO = make(1, 1, 1, 600, 64, seed=6)
    ramp = torch.linspace(0, 20, 600, device="cuda")[None, None, :, None]
    K = (K.float() * 0.1 + ramp * 0.2).to(torch.bfloat16)
    Q = (Q.float() * 0.1 + 1).to(torch.bfloat16)
    O, lse = P.window_attention(Q, K, V)
    check_forward(O, lse, Q, K, V, -1, -1, 0, 64 ** -0.5)
    check_backward(P.window_attention_backward(dO, Q, K, V, O, lse), dO, Q, K, V, -1, -1, 0, 64 ** -0.5, norms=False)


def test_long_sequence_last_rows():
    """A long sequence: the last rows against the oracle on the keys they see."""
    N, left, sinks = 20011, 300, 40
    Q, K, V, _ = make(1, 2, 1, N, 128, seed=7)
    O, lse = P.window_attention(Q, K, V, left=left, right=0, sinks=sinks)
    q, k, v = f64(Q), f64(K), f64(V)
    rows = np.arange(N - 200, N)
    see = W.visible(rows, N, left, 0, sinks)
    for h in range(2):
        o, l, to, tl = T.forward(q[0, h, rows], k[0, 0], v[0, 0], see, 128 ** -0.5)
        T.check(f64(O)[0, h, rows], o, to, "O")
        T.check(f64(lse)[0, h, rows], l, tl, "lse")


def test_gradient_against_differences():
    """<dX, direction> against the change of the loss along it, both from the kernel's own forward
    call on a smooth problem: forward differences in O of size eps, O to bf16."""
    N, d = 260, 64
    Q, K, V, dO = make(1, 2, 1, N, d, seed=8)
    mask = dict(left=90, right=0, sinks=5)
    O, lse = P.window_attention(Q, K, V, **mask)
    grads = P.window_attention_backward(dO, Q, K, V, O, lse, **mask)
    see = W.visible(np.arange(N), N, 90, 0, 5)
    do = f64(dO)

    def loss(q, k, v):
        return sum((W.attend(q[0, h], k[0, 0], v[0, 0], see, d ** -0.5)[0] * do[0, h]).sum() for h in range(2))

    rng = np.random.default_rng(9)
    base = [f64(Q), f64(K), f64(V)]
    for i, g in enumerate(grads):
        # along the gradient's own direction the product is its norm: no cancellation
        way = f64(g) + 0.1 * np.abs(f64(g)).mean() * rng.normal(size=base[i].shape)
        way /= np.linalg.norm(way)
        eps = 1e-4
        up, down = ([x + s * eps * way if k == i else x for k, x in enumerate(base)] for s in (1, -1))
        want = (loss(*up) - loss(*down)) / (2 * eps)
        got = float((f64(g) * way).sum())
        assert abs(got - want) <= T.U * abs(want)


def test_same_bits_and_head_alone():
    """The same call gives the same bits, and a head alone gives the bits it has in a batch."""
    shape = (2, 6, 2, 777, 128)
    Q, K, V, dO = make(*shape, seed=11)
    mask = dict(left=200, right=0, sinks=30)
    first = [*P.window_attention(Q, K, V, **mask)]
    first += P.window_attention_backward(dO, Q, K, V, *first, **mask)
    for _ in range(3):
        again = [*P.window_attention(Q, K, V, **mask)]
        again += P.window_attention_backward(dO, Q, K, V, *again, **mask)
        assert all(torch.equal(a, b) for a, b in zip(first, again))
    q, k, v, do = Q[1:, 3:], K[1:, 1:], V[1:, 1:], dO[1:, 3:]
    q, k, v, do = (t.contiguous() for t in (q, k, v, do))
    alone = [*P.window_attention(q, k, v, **mask)]
    assert torch.equal(alone[0], first[0][1:, 3:]) and torch.equal(alone[1], first[1][1:, 3:])
    alone += P.window_attention_backward(do, q, k, v, *alone, **mask)
    for a, b, h in zip(alone[2:], first[2:], (3, 1, 1)):
        assert torch.equal(a, b[1:, h:])


def test_outputs_given_streams_and_graph():
    """Preallocated outputs and workspace, a stream of its own, and a captured step replayed on
    new inputs give the bits of plain calls."""
    B, Hq, Hkv, N, d = 1, 4, 2, 333, 64
    Q, K, V, dO = make(B, Hq, Hkv, N, d, seed=12)
    mask = dict(left=70, right=3, sinks=9)
    outs = [torch.empty_like(Q), torch.empty(B, Hq, N, device="cuda"), torch.empty_like(Q), torch.empty_like(K),
            torch.empty_like(V)]
    ws = torch.empty(P.window_attention_backward_workspace(B, Hq, Hkv, N, d, **mask), dtype=torch.uint8, device="cuda")

    def step():
        P.window_attention(Q, K, V, out=outs[0], lse=outs[1], **mask)
        P.window_attention_backward(dO, Q, K, V, outs[0], outs[1], out=outs[2:], workspace=ws, **mask)

    want = [*P.window_attention(Q, K, V, **mask)]
    want += P.window_attention_backward(dO, Q, K, V, *want, **mask)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    new = make(B, Hq, Hkv, N, d, seed=13)
    for t, x in zip((Q, K, V, dO), new):
        t.copy_(x)
    ws.fill_(255)  # nothing of an earlier call is needed: the bytes read as NaN
    g.replay()
    torch.cuda.synchronize()
    want = [*P.window_attention(*new[:3], **mask)]
    want += P.window_attention_backward(new[3], *new[:3], *want, **mask)
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    P.device_error()


def test_infinities_and_nan_stay_in_their_sequence_and_head():
    """A NaN in one head's keys reaches that key head's rows only; the other heads keep their bits."""
    Q, K, V, _ = make(2, 4, 2, 200, 64, seed=14)
    want, _ = P.window_attention(Q, K, V, left=50, right=0)
    bad = K.clone()
    bad[1, 0, 120] = float("nan")
    O, lse = P.window_attention(Q, bad, V, left=50, right=0)
    assert torch.equal(O[0], want[0]) and torch.equal(O[1, 2:], want[1, 2:])
    assert torch.equal(O[1, :2, :120], want[1, :2, :120])
    assert torch.isnan(O[1, :2, 120:171].float()).all() and torch.isnan(lse[1, :2, 120:171]).all()
    assert torch.equal(O[1, :2, 171:], want[1, :2, 171:])


def test_empty_problem():
    Q = torch.empty(0, 2, 5, 64, dtype=torch.bfloat16, device="cuda")
    O, lse = P.window_attention(Q, Q, Q)
    assert O.shape == Q.shape and lse.shape == (0, 2, 5)
    assert [g.shape for g in P.window_attention_backward(Q, Q, Q, Q, O, lse)] == [Q.shape] * 3


def test_key_tiles_cut_into_many_runs():
    """A causal sequence with many heads on one key head: its first key tiles are cut into runs."""
    B, Hq, Hkv, N, d = 1, 6, 1, 1300, 64
    Q, K, V, dO = make(B, Hq, Hkv, N, d, seed=21)
    for mask in (dict(left=-1, right=0, sinks=0), dict(left=100, right=0, sinks=200)):
        O, lse = P.window_attention(Q, K, V, **mask)
        grads = P.window_attention_backward(dO, Q, K, V, O, lse, **mask)
        P.device_error()
        check_backward(grads, dO, Q, K, V, mask["left"], 0, mask["sinks"], d ** -0.5)


def test_two_streams_at_once():
    """Calls in flight on two streams, each with its own workspace, give the bits of calls alone."""
    args = [make(1, 4, 2, 900 + 100 * i, 128, seed=30 + i) for i in range(2)]
    mask = dict(left=300, right=0, sinks=16)

    def step(Q, K, V, dO):
        O, lse = P.window_attention(Q, K, V, **mask)
        return O, lse, *P.window_attention_backward(dO, Q, K, V, O, lse, **mask)

    want = [step(*a) for a in args]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in args]
    got = [None, None]
    for _ in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = step(*args[i])
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("what", [float("nan"), float("inf"), float("-inf")], ids=["nan", "inf", "-inf"])
def test_a_value_that_is_not_finite_reaches_the_rows_that_see_it(d, what):
    """One element of one value changes its column alone: there the rows that see it hold it, the
    others what they held (a row that shares a tile with it sums the column again, with weights that
    are not rounded: off by a rounding of p and one of either O, 3 u max|v|). A key changes no bit of
    the rows that do not see it. Tiles that every row sees whole and partly seen ones."""
    B, Hq, Hkv, N = 2, 6, 2, 700
    Q, K, V, _ = make(B, Hq, Hkv, N, d, seed=51)
    p, j = np.arange(N)[:, None], np.arange(N)[None]
    for left, right, sinks in ((-1, 0, 0), (90, 0, 5), (-1, -1, 0), (20, 200, 0)):
        mask = dict(left=left, right=right, sinks=sinks)
        see = (j <= p + (N if right < 0 else right)) & ((j >= p - (N if left < 0 else left)) | (j < sinks))
        O, lse = P.window_attention(Q, K, V, **mask)
        for at in (3, 130, 255, 256, 500, 699):
            c = at % d
            rows = torch.from_numpy(see[:, at]).cuda()
            bad = V.clone()
            bad[1, 1, at, c] = what
            got, glse = P.window_attention(Q, K, bad, **mask)
            assert torch.equal(glse, lse)
            want = O.clone()
            want[1, 3:, rows, c] = what
            assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.isinf(), want.isinf())
            off = (got.float() - O.float())[1, 3:, ~rows, c].abs()
            assert not off.numel() or float(off.max()) <= T.SLACK * 3 * T.U * float(V[1, 1, :, c].abs().max())
            got[1, 3:, :, c] = want[1, 3:, :, c]
            assert torch.equal(got.nan_to_num(), want.nan_to_num())
            bad = K.clone()
            bad[1, 1, at] = what
            got, glse = P.window_attention(Q, bad, V, **mask)
            want = O.clone()
            assert torch.equal(got[:, :, ~rows], O[:, :, ~rows]) and torch.equal(glse[:, :, ~rows], lse[:, :, ~rows])
            assert torch.equal(got[:, :3], O[:, :3]) and torch.equal(got[0], O[0])


@pytest.mark.parametrize("d", [64, 128])
def test_a_sequence_that_is_lost_from_a_token_on(d):
    """Keys and values are NaN (values: NaN and infinities in turn) from token 2900 on: rows before it
    hold what they held, to the roundings of the rows that share a tile with it; the others are NaN."""
    B, Hq, Hkv, N, at = 1, 4, 2, 4000, 2900
    Q, K, V, _ = make(B, Hq, Hkv, N, d, seed=52)
    for mask in (dict(left=-1, right=0), dict(left=700, right=0, sinks=9)):
        O, _ = P.window_attention(Q, K, V, **mask)
        for lose_keys in (False, True):
            bad_k, bad_v = K.clone(), V.clone()
            bad_v[:, :, at:] = float("nan")
            bad_v[:, :, at::3, ::2] = float("inf")
            if lose_keys:
                bad_k[:, :, at:] = float("nan")
            got, lse = P.window_attention(Q, bad_k, bad_v, **mask)
            off = (got - O)[:, :, :at].float().abs()
            assert float(off.max()) <= T.SLACK * 3 * T.U * float(V.abs().max())
            assert not torch.isfinite(got[:, :, at:].float()).any()
            assert torch.isfinite(lse[:, :, :at]).all()
            assert bool(torch.isnan(lse[:, :, at:]).all()) == lose_keys
    P.device_error()


@pytest.mark.parametrize("what", [float("inf"), float("nan")], ids=["inf", "nan"])
def test_a_value_that_is_not_finite_at_the_end_of_a_long_sequence(what):
    """A million keys: the rows beside the value hold what they held however long they are, every other
    row keeps its bits, and nothing runs out of time."""
    N, d, at, c = 2 ** 20 + 37, 64, 2 ** 20 + 30, 5
    g = torch.Generator(device="cuda").manual_seed(53)
    Q, K, V = (torch.randn(1, h, N, d, device="cuda", generator=g).to(torch.bfloat16) for h in (2, 1, 1))
    O, lse = P.window_attention(Q, K, V, right=0)
    bad = V.clone()
    bad[0, 0, at, c] = what
    got, glse = P.window_attention(Q, K, bad, right=0)
    P.device_error()
    assert torch.equal(glse, lse) and torch.isfinite(O.float()).all()
    col = got[:, :, :, c].clone()
    assert (col[:, :, at:].isnan() if what != what else col[:, :, at:] == what).all()
    # p rounded in either sum, and either O
    off = (col.float() - O[:, :, :, c].float())[:, :, :at].abs()
    assert float(off.max()) <= T.SLACK * 4 * T.U * float(V[0, 0, :, c].abs().max())
    got[:, :, :, c] = O[:, :, :, c]
    assert torch.equal(got, O)


@pytest.mark.parametrize("d", [64, 128])
def test_values_near_the_end_of_the_range(d):
    """Values of one sign up to 2^126.3, beside columns of 2^-90: sums of exp(s - m) v leave fp32, the
    averages do not. An infinity in between reaches the rows that see it, and no others."""
    N = 1500
    Q, K, V, _ = make(1, 4, 2, N, d, seed=54)
    V = (V.float().abs().clamp_max(4) + 0.5) * 2.0 ** 124
    V[..., ::3] *= 2.0 ** -214
    V = V.to(torch.bfloat16)
    for left, right in ((-1, -1), (700, 0)):
        O, lse = P.window_attention(Q, K, V, left=left, right=right)
        check_forward(O, lse, Q, K, V, left, right, 0, d ** -0.5)
        bad = V.clone()
        bad[0, 1, 1000, 1] = float("inf")
        got, glse = P.window_attention(Q, K, bad, left=left, right=right)
        see = torch.from_numpy(W.visible(np.arange(N), N, left, right, 0)[:, 1000]).cuda()
        assert torch.equal(glse, lse) and (got[0, 2:, see, 1] == float("inf")).all()
        got[0, 2:, see, 1] = O[0, 2:, see, 1]
        check_forward(got, glse, Q, K, V, left, right, 0, d ** -0.5)
    P.device_error()


def test_autograd_records_the_call():
    """O carries the gradient that window_attention_backward gives, bit for bit, for the operands that
    ask for one; nothing is recorded without a need, and a second derivative is refused."""
    mask = dict(left=70, right=3, sinks=9)
    Q, K, V, dO = make(1, 4, 2, 333, 64, seed=55)
    O, lse = P.window_attention(Q, K, V, **mask)
    assert not O.requires_grad
    want = P.window_attention_backward(dO, Q, K, V, O, lse, **mask)
    for need in ((1, 1, 1), (0, 0, 1), (1, 0, 0)):
        leaves = [torch.nn.Parameter(t.clone(), requires_grad=bool(n)) for t, n in zip((Q, K, V), need)]
        got, glse = P.window_attention(*leaves, **mask)
        assert got.requires_grad and not glse.requires_grad
        assert torch.equal(got, O) and torch.equal(glse, lse)
        got.backward(dO)
        for leaf, w, n in zip(leaves, want, need):
            assert torch.equal(leaf.grad, w) if n else leaf.grad is None
        with torch.no_grad():
            assert not P.window_attention(*leaves, **mask)[0].requires_grad
    # through other operations, scale given, on another stream, and a gradient that is a broadcast scalar
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        leaves = [t.clone().requires_grad_() for t in (Q, K, V)]
        got, _ = P.window_attention(leaves[0] * 1, leaves[1] * 1, leaves[2] * 1, scale=0.2, **mask)
        got.sum().backward()
    torch.cuda.current_stream().wait_stream(s)
    O, lse = P.window_attention(Q, K, V, scale=0.2, **mask)
    want = P.window_attention_backward(torch.ones_like(O), Q, K, V, O, lse, scale=0.2, **mask)
    assert all(torch.equal(x.grad, w) for x, w in zip(leaves, want))
    leaves = [t.clone().requires_grad_() for t in (Q, K, V)]
    got, _ = P.window_attention(*leaves, **mask)
    (g,) = torch.autograd.grad(got, leaves[0], dO, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()
    P.device_error()


def test_keys_without_query_heads_have_no_gradient():
    """No query head at all: the gradients of the keys and values are zero, preallocated or not."""
    Q, K = torch.empty(2, 0, 9, 64, dtype=torch.bfloat16, device="cuda"), torch.ones(2, 3, 9, 64, dtype=torch.bfloat16, device="cuda")
    O, lse = P.window_attention(Q, K, K)
    out = torch.empty_like(Q), torch.full_like(K, 3.0), torch.full_like(K, 3.0)
    for grads in (P.window_attention_backward(Q, Q, K, K, O, lse), P.window_attention_backward(Q, Q, K, K, O, lse, out=out)):
        assert grads[0].shape == Q.shape and all(g.shape == K.shape and (g == 0).all() for g in grads[1:])


def gradient64(do, q, k, v, see, scale):
    """(dq, dk, dv, tol_dq, tol_dk, tol_dv) of one head in 64 bits on the device: the formulas and the
    bounds of window_bounds.backward."""
    u, f, d = T.U, 2.0 ** -24, q.shape[1]
    n, top = k.shape[0], scale * float((q.abs() @ k.abs().mT).max())
    e = 2 * (d + 8) * f * top + 2.0 ** -19
    p = torch.softmax((scale * q @ k.mT).masked_fill_(~see, float("-inf")), 1)
    o, dp = p @ v, do @ v.mT
    delta = (p * dp).sum(1, keepdim=True)
    tol_o = T.SLACK * ((u + e + n * f) * (p @ v.abs()) + u * o.abs())
    t_delta = (do.abs() * tol_o).sum(1, keepdim=True)
    ds = p * (dp - delta)
    t_ds = p * (t_delta + e * (dp.abs() + delta.abs()) + d * f * (do.abs() @ v.abs().mT)) + (u + n * f) * ds.abs()
    dq = scale * ds @ k
    return (dq, scale * ds.mT @ q, p.mT @ do, T.SLACK * (scale * t_ds @ k.abs() + u * dq.abs()),
            T.SLACK * scale * t_ds.mT @ q.abs(), T.SLACK * ((u + e + n * f) * p).mT @ do.abs())


@pytest.mark.parametrize("shape", [
    (1, 4, 1, 6000, 64, -1, 0, 0),       # 44 of 47 key tiles cut, 315 runs on 148 SMs
    (2, 8, 2, 5003, 64, -1, 0, 0),       # 29 of 40, 376 runs
    (1, 6, 2, 8200, 128, 700, 0, 300),   # 61 of 65, 338 runs
    (1, 4, 2, 4100, 128, -1, -1, 0),     # all 33, 330 runs
    (1, 16, 4, 9000, 128, 2047, 0, 64),  # 56 of 71, 520 runs
], ids=str)
def test_gradient_in_several_waves(shape):
    """Gradients whose runs of query tiles take more than one wave of the SMs, with many cut key tiles."""
    B, Hq, Hkv, N, d, left, right, sinks = shape
    Q, K, V, dO = make(B, Hq, Hkv, N, d, seed=56)
    mask = dict(left=left, right=right, sinks=sinks)
    O, lse = P.window_attention(Q, K, V, **mask)
    grads = P.window_attention_backward(dO, Q, K, V, O, lse, **mask)
    P.device_error()
    see = torch.from_numpy(W.visible(np.arange(N), N, left, right, sinks)).cuda()
    G = Hq // Hkv
    for b in range(B):
        for hk in range(Hkv):
            sums = [0.0] * 4
            for h in range(hk * G, (hk + 1) * G):
                dq, dk, dv, tq, tk, tv = gradient64(dO[b, h].double(), Q[b, h].double(), K[b, hk].double(), V[b, hk].double(), see, d ** -0.5)
                assert bool(((grads[0][b, h].double() - dq).abs() <= tq + T.LOST).all()), f"dQ[{b},{h}]"
                assert float((grads[0][b, h].double() - dq).norm() / dq.norm()) <= T.U
                sums = [x + y for x, y in zip(sums, (dk, dv, tk, tv))]
            for got, want, tol, name in ((grads[1], sums[0], sums[2], "dK"), (grads[2], sums[1], sums[3], "dV")):
                off = (got[b, hk].double() - want).abs()
                assert bool((off <= tol + T.SLACK * T.U * want.abs() + T.LOST).all()), f"{name}[{b},{hk}]"
                assert float(off.norm() / want.norm()) <= T.U
