"""The paged cache and the attention over it on the GPU against the fp64 oracle, alone and
together as a program uses them: write, attend, write, attend."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import block_sparse_attention_pisa_b200 as P  # noqa: E402
from oracle import window as W  # noqa: E402
from tests import window_bounds as T  # noqa: E402

pytestmark = pytest.mark.gpu

E4M3, BF16 = torch.float8_e4m3fn, torch.bfloat16


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def randn(*shape, seed=0, spread=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * spread).to(BF16).cuda()


def table_of(lens, page, spare=3, seed=0, slack=0):
    """A shuffled page table (-1 where nothing is held), the number of pages."""
    held = [-(-n // page) for n in lens]
    total = sum(held) + spare
    order = np.random.default_rng(seed).permutation(total)
    t = np.full((len(lens), max(max(held), 1) + slack), -1, np.int32)
    at = 0
    for b, n in enumerate(held):
        t[b, :n] = order[at:at + n]
        at += n
    return torch.from_numpy(t).cuda(), total


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def values(cache):
    """The cache's K and V as the values they stand for, fp64 [pages, Hkv, page, d]."""
    if cache.k_scale is None:
        return f64(cache.K), f64(cache.V)
    return [f64(c) * f64(s)[..., None] for c, s in ((cache.K, cache.k_scale), (cache.V, cache.v_scale))]


def filled(lens, Hkv, page, d, dtype, seed=0, spread=1.0, slack=0):
    """A cache holding random rows of `lens` tokens each; what no sequence holds is NaN."""
    table, total = table_of(lens, page, seed=seed, slack=slack)
    cache = P.paged_cache(total, Hkv, page, d, dtype)
    if dtype == BF16:
        cache.K.fill_(float("nan"))
        cache.V.fill_(float("nan"))
    else:
        for t in (cache.K, cache.V):
            t.view(torch.uint8).fill_(0x7e)
        cache.k_scale.fill_(float("nan"))
        cache.v_scale.fill_(float("nan"))
    most = max(lens)
    if most:
        K, V = (randn(len(lens), Hkv, most, d, seed=seed + 1 + i, spread=spread) for i in range(2))
        P.cache_write(K, V, cache, table, ints(lens), ints(lens))
    return cache, table


# ------------------------------------------------------------------ write and read

@pytest.mark.parametrize("dtype", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("page,d,Hkv,N,lens,news", [
    (16, 64, 1, 1, [1], [1]),
    (16, 128, 3, 5, [5, 17, 40], [5, 1, 4]),
    (32, 64, 2, 33, [33, 64, 100, 7], [33, 0, 20, 7]),
    (64, 128, 2, 70, [65, 300], [65, 70]),
    (128, 64, 5, 129, [129, 128, 1000], [129, 100, 129]),
])
def test_write_then_read(dtype, page, d, Hkv, N, lens, news):
    table, total = table_of(lens, page, seed=page)
    cache = P.paged_cache(total, Hkv, page, d, dtype)
    before = [t.clone() for t in cache if t is not None]
    K, V = randn(len(lens), Hkv, N, d, seed=1), randn(len(lens), Hkv, N, d, seed=2, spread=3.0)
    K[0, 0, 0] = 0  # a row of zeros
    P.cache_write(K, V, cache, table, ints(lens), ints(news))
    P.device_error()
    at = table.cpu().numpy()
    written = np.zeros((total, page), bool)
    for x, c, s in ((f64(K), cache.K, cache.k_scale), (f64(V), cache.V, cache.v_scale)):
        got = f64(c)
        for b, (n, m) in enumerate(zip(lens, news)):
            for t in range(m):
                pos = n - m + t
                i, r = at[b, pos // page], pos % page
                written[i, r] = True
                if dtype == BF16:
                    assert np.array_equal(got[i, :, r], x[b, :, t])
                else:
                    code, scale = W.quantise_rows(x[b, :, t])
                    assert np.array_equal(s[i, :, r].cpu().numpy(), scale)
                    assert np.array_equal(got[i, :, r], code)
    # rows that no new token belongs to keep their bits
    keep = torch.from_numpy(~written).cuda()
    for t, old in zip([t for t in cache if t is not None], before):
        t, old = (x.view(torch.uint8) if x.dtype == E4M3 else x for x in (t, old))
        assert torch.equal(t.transpose(1, 2)[keep], old.transpose(1, 2)[keep])
    # read back: values to half a bf16 step, rows behind a sequence's last untouched
    rd = max(lens) + 3
    out = [torch.full((len(lens), Hkv, rd, d), 7.0, dtype=BF16, device="cuda") for _ in "KV"]
    P.cache_read(cache, table, ints(lens), rd, out=out)
    P.device_error()
    for got, pages in zip(out, values(cache)):
        got = f64(got)
        for b, n in enumerate(lens):
            want = W.gather(pages, at[b], n)
            # fp32 product, then bf16: half a bf16 step and half an fp32 step
            assert np.all(np.abs(got[b, :, :n] - want) <= np.abs(want) * (2.0 ** -8 + 2.0 ** -23) + 2.0 ** -133)
            assert np.all(got[b, :, n:] == 7)
    assert (P.cache_read(cache, table, ints(lens), rd)[0][0, :, lens[0]:] == 0).all()


def test_quantised_rows_at_the_edges():
    """Zero, subnormal, huge, infinite and NaN rows, ties of the rounding."""
    d, page = 64, 16
    cache, (table, _) = P.paged_cache(1, 1, page, d, E4M3), (ints([[0]]), 1)
    x = torch.zeros(1, 1, 8, d)
    x[0, 0, 1] = 1e-39 * torch.arange(d)
    x[0, 0, 2] = torch.linspace(-1.5e38, 1.5e38, d)
    x[0, 0, 3] = torch.arange(d).float() * 7       # amax 441
    x[0, 0, 4] = torch.linspace(0, 448, d)
    x[0, 0, 5, 3] = float("nan")
    x[0, 0, 6, 5] = float("-inf")
    x[0, 0, 7, :16] = torch.tensor([448.0, 17, 19, 21, 33, 35, 1.0625, 1.1875, 2 ** -9, 2 ** -10, 3 * 2 ** -10, 2 ** -11, -17, -19, 416, 432])
    x = x.to(BF16).cuda()
    P.cache_write(x, x, cache, table, ints([8]))
    P.device_error()
    ok = [0, 1, 2, 3, 4, 7]
    code, scale = W.quantise_rows(f64(x)[0, 0, ok])
    assert np.array_equal(f64(cache.K)[0, 0, ok], code) and np.array_equal(cache.k_scale[0, 0, ok].cpu().numpy(), scale)
    back = f64(P.cache_read(cache, table, ints([8]), 8)[0])[0, 0]
    assert np.isnan(back[5]).all() and np.isnan(back[6]).all() and np.isfinite(back[ok]).all()


def test_lengths_and_pages_out_of_range_are_flagged_and_skipped():
    """A bad page entry or length is reported and nothing outside the cache is touched."""
    d, page, Hkv = 64, 16, 2
    for dtype in (BF16, E4M3):
        lens = [40, 40]
        table, total = table_of(lens, page)
        cache = P.paged_cache(total, Hkv, page, d, dtype)
        K = randn(2, Hkv, 40, d, seed=3)
        bad = table.clone()
        bad[0, 1] = total  # one past the last page
        P.cache_write(K, K, cache, bad, ints(lens))
        with pytest.raises(P.PisaError, match="out of range"):
            P.device_error()
        P.device_error()  # taken
        full = P.paged_cache(total, Hkv, page, d, dtype)
        P.cache_write(K, K, full, table, ints(lens))
        hole = int(table[0, 1])
        assert (cache.K.view(torch.uint8)[hole] == 0).all()
        same = [i for i in range(total) if i != hole]
        assert torch.equal(cache.K.view(torch.uint8)[same], full.K.view(torch.uint8)[same])
        out = [torch.full((2, Hkv, 40, d), 7.0, dtype=BF16, device="cuda") for _ in "KV"]
        P.cache_read(full, bad, ints(lens), 40, out=out)
        with pytest.raises(P.PisaError, match="out of range"):
            P.device_error()
        want = P.cache_read(full, table, ints(lens), 40)
        assert (out[0][0, :, 16:32] == 7).all() and torch.equal(out[0][1], want[0][1])
        # attention leaves the hole out
        Q = randn(2, 4, 3, d, seed=4)
        O, lse = P.paged_attention(Q, full, bad, ints(lens))
        with pytest.raises(P.PisaError, match="out of range"):
            P.device_error()
        k, v = values(full)
        row = table.cpu().numpy()
        for h in range(4):
            see = W.visible(37 + np.arange(3), 40, -1, 0, 0)
            see[:, 16:32] = False
            o, l, to, tl = T.forward(f64(Q)[0, h], W.gather(k, row[0], 40)[h // 2], W.gather(v, row[0], 40)[h // 2], see, d ** -0.5)
            T.check(f64(O)[0, h], o, to, "O")
            T.check(f64(lse)[0, h], l, tl, "lse")
        # a length past the table's end is taken as its end
        long = P.paged_attention(Q, full, table, ints([100000, -5]), right=-1)
        with pytest.raises(P.PisaError, match="out of range"):
            P.device_error()
        cap = table.shape[1] * page
        want = P.paged_attention(Q, full, table, ints([cap, 0]), right=-1)
        P.device_error()
        assert torch.equal(long[0], want[0]) and torch.equal(long[1], want[1])


# ------------------------------------------------------------------ attention

def check_attention(O, lse, Q, cache, table, lens, news, left, right, sinks, scale):
    k, v = values(cache)
    q, o, l, at = f64(Q), f64(O), f64(lse), table.cpu().numpy()
    G = Q.shape[1] // k.shape[1]
    for b, (n, m) in enumerate(zip(lens, news)):
        K, V = W.gather(k, at[b], n), W.gather(v, at[b], n)
        see = W.visible(n - m + np.arange(m), n, left, right, sinks)
        for h in range(Q.shape[1]):
            wo, wl, to, tl = T.forward(q[b, h, :m], K[h // G], V[h // G], see, scale)
            T.check(o[b, h, :m], wo, to, f"O[{b},{h}]")
            T.check(l[b, h, :m], wl, tl, f"lse[{b},{h}]")


# (page, d, Hq, Hkv, N, lens, news, left, right, sinks)
CASES = [
    (16, 64, 1, 1, 1, [1], None, -1, 0, 0),                         # one token that sees itself
    (16, 64, 4, 2, 1, [17, 0, 5], [1, 0, 1], -1, 0, 0),             # an empty sequence in the batch
    (64, 128, 8, 1, 1, [500, 64, 63, 65], None, -1, 0, 0),          # a group of eight, pages that end at the length
    (32, 128, 5, 5, 1, [1000, 3], None, 100, 0, 7),                 # window and sinks, single tokens
    (128, 64, 40, 8, 1, [700, 129], None, -1, -1, 0),
    (16, 128, 32, 1, 1, [333], None, 50, 0, 0),                     # more heads than a 16-row tile
    (16, 64, 6, 2, 4, [40, 4, 3], [4, 4, 1], -1, 0, 0),             # a few tokens each
    (64, 128, 4, 4, 16, [16, 200, 129], [16, 16, 9], 64, 0, 4),
    (32, 64, 8, 2, 33, [33, 400], [33, 20], -1, 0, 0),
    (128, 128, 2, 1, 128, [128, 513], None, -1, 0, 0),
    (64, 64, 3, 1, 150, [150, 1000], [150, 111], 200, 0, 64),       # rows of a tile end inside a token
    (16, 128, 4, 2, 130, [700, 140], [130, 130], 300, 5, 33),       # a little to the right
    (32, 128, 2, 2, 40, [520], None, -1, -1, 0),                    # the chunk sees all of itself
    (16, 64, 2, 1, 20, [10, 0], [20, 20], -1, 0, 0),                # more new tokens than held: rows that see nothing
    (64, 64, 2, 2, 7, [300], None, 0, 0, 0),                        # each sees itself only
    (128, 128, 2, 1, 9, [260], None, 3, 0, 1000),                   # sinks past the end
]


@pytest.mark.parametrize("dtype", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_paged_attention(case, dtype):
    page, d, Hq, Hkv, N, lens, news, left, right, sinks = case
    cache, table = filled(lens, Hkv, page, d, dtype, seed=N, slack=2)
    Q = randn(len(lens), Hq, N, d, seed=50 + N)
    O, lse = torch.full_like(Q, 5.0), torch.full(Q.shape[:3], 5.0, device="cuda")
    q_lens = None if news is None else ints(news)
    P.paged_attention(Q, cache, table, ints(lens), q_lens, left=left, right=right, sinks=sinks, out=O, lse=lse)
    P.device_error()
    news = [N] * len(lens) if news is None else news
    check_attention(O, lse, Q, cache, table, lens, news, left, right, sinks, d ** -0.5)
    for b, m in enumerate(news):  # rows behind the last new token are left as they were
        assert (O[b, :, m:] == 5).all() and (lse[b, :, m:] == 5).all()


@pytest.mark.parametrize("dtype", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("N", [1, 3, 70])
def test_long_and_short_sequences_together(dtype, N):
    """One long sequence among short ones: its keys are split over many blocks."""
    lens = [9000, N, 130, 2048]
    cache, table = filled(lens, 2, 64, 128, dtype, seed=3)
    Q = randn(4, 6, N, 128, seed=60)
    for mask in (dict(left=-1, right=0, sinks=0), dict(left=1500, right=0, sinks=100)):
        O, lse = P.paged_attention(Q, cache, table, ints(lens), **mask)
        P.device_error()
        check_attention(O, lse, Q, cache, table, lens, [N] * 4, mask["left"], mask["right"], mask["sinks"], 128 ** -0.5)


def test_large_scores():
    lens = [700, 90]
    for N in (1, 40):
        cache, table = filled(lens, 1, 32, 64, E4M3, seed=4, spread=20.0)
        Q = randn(2, 2, N, 64, seed=61, spread=4.0)
        O, lse = P.paged_attention(Q, cache, table, ints(lens), scale=0.3)
        check_attention(O, lse, Q, cache, table, lens, [N] * 2, -1, 0, 0, 0.3)


def test_pages_out_of_the_window_need_not_be_held():
    """Entries of pages that no query sees may hold anything, for every tile of the chunk."""
    for dtype in (BF16, E4M3):
        for N in (1, 20):
            lens, page = [1000], 16
            cache, table = filled(lens, 2, page, 64, dtype, seed=5)
            mask = dict(left=130, right=0, sinks=20)
            Q = randn(1, 4, N, 64, seed=62)
            want = P.paged_attention(Q, cache, table, ints(lens), **mask)
            first, last = 2, (1000 - N - 130) // page  # pages [first, last) hold nothing visible
            freed = table.clone()
            freed[0, first:last] = -7
            for i in range(first, last):
                for t in cache:
                    if t is not None and t.dtype != E4M3:
                        t[int(table[0, i])] = float("nan")
            got = P.paged_attention(Q, cache, freed, ints(lens), **mask)
            P.device_error()
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_sequences_share_pages():
    """Two sequences with a common prefix held once."""
    cache, table = filled([256, 256], 2, 64, 128, BF16, seed=6)
    table[1, :2] = table[0, :2]
    for N in (1, 30):
        Q = randn(2, 4, N, 128, seed=63)
        O, lse = P.paged_attention(Q, cache, table, ints([256, 200]))
        check_attention(O, lse, Q, cache, table, [256, 200], [N] * 2, -1, 0, 0, 128 ** -0.5)


@pytest.mark.parametrize("dtype", [BF16, E4M3], ids=["bf16", "e4m3"])
def test_a_sequence_grows(dtype):
    """Prompt, a chunk, then single tokens: at every step the cache's attention agrees with the
    oracle, and in bf16 the whole agrees with windowed attention over the plain sequence."""
    Hq, Hkv, d, page, total = 4, 2, 64, 32, 150
    mask = dict(left=60, right=0, sinks=6)
    Q, K, V = randn(2, Hq, total, d, seed=70), randn(2, Hkv, total, d, seed=71), randn(2, Hkv, total, d, seed=72)
    table, pages = table_of([total, total], page)
    cache = P.paged_cache(pages, Hkv, page, d, dtype)
    at, outs = 0, []
    for step in (100, 40, *[1] * 10):
        new = [t[:, :, at:at + step].contiguous() for t in (Q, K, V)]
        at += step
        lens = ints([at, at])
        P.cache_write(new[1], new[2], cache, table, lens)
        O, lse = P.paged_attention(new[0], cache, table, lens, **mask)
        check_attention(O, lse, new[0], cache, table, [at, at], [step] * 2, 60, 0, 6, d ** -0.5)
        outs.append(O)
    P.device_error()
    if dtype == BF16:
        whole, _ = P.window_attention(Q, K, V, **mask)
        got = f64(torch.cat(outs, 2))
        # both sides are within the forward bound of the exact rows: p and O rounded, twice
        assert np.linalg.norm(got - f64(whole)) <= 2 * T.U * np.linalg.norm(got)


def test_same_bits_stream_and_graph():
    """The same call gives the same bits; a captured token step, replayed with new lengths and
    inputs and a workspace full of NaN, gives the bits of a plain call. Two graphs share the
    workspace, replayed one after the other."""
    lens, page, d = [900, 40], 64, 128
    for N in (1, 24):
        cache, table = filled(lens, 2, page, d, BF16, seed=8)
        Q, n = randn(2, 8, N, d, seed=80), ints(lens)
        O, lse = torch.empty_like(Q), torch.empty(2, 8, N, device="cuda")
        ws = torch.empty(max(1, P.paged_attention_workspace(Q, cache, table, n)), dtype=torch.uint8, device="cuda")
        call = lambda **k: P.paged_attention(Q, cache, table, n, out=O, lse=lse, workspace=ws, **k)  # noqa: E731
        want = P.paged_attention(Q, cache, table, n)
        for _ in range(3):
            call()
            assert torch.equal(O, want[0]) and torch.equal(lse, want[1])
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            call()
        torch.cuda.current_stream().wait_stream(s)
        graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
        masks = [dict(left=-1), dict(left=30, sinks=3)]
        for g, mask in zip(graphs, masks):
            with torch.cuda.graph(g):
                call(**mask)
        n.copy_(ints([333, 39]))
        Q.copy_(randn(*Q.shape, seed=81))
        for g, mask in [*zip(graphs, masks)] * 2:
            ws.fill_(255)
            O.zero_()
            g.replay()
            torch.cuda.synchronize()
            want = P.paged_attention(Q, cache, table, n, **mask)
            assert torch.equal(O, want[0]) and torch.equal(lse, want[1])
        P.device_error()


def test_table_rows_and_lengths_at_odd_offsets():
    """int32 operands that start at an odd element, and a table wider than what is held."""
    cache, table = filled([100, 200, 50], 1, 16, 64, BF16, seed=9, slack=3)
    big = torch.cat([ints([0]), table.flatten()])[1:].view(table.shape)
    n = torch.cat([ints([0]), ints([100, 200, 50])])[1:]
    Q = randn(3, 2, 1, 64, seed=90)
    a, b = P.paged_attention(Q, cache, big, n), P.paged_attention(Q, cache, table, n.clone())
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_codes_near_every_tie():
    """Rows whose quotients fall on and beside ties of the rounding, over many scales: the codes
    are those of the fp32 quotient."""
    d, page = 128, 128
    rng = np.random.default_rng(21)
    x = np.zeros((128, d), np.float32)
    for r in range(128):
        amax = np.float32(rng.choice([448, 7, 1, 3.5, 0.21875, 1000, 2.0 ** -120, 57]) * (1 if r % 3 else rng.uniform(1, 2)))
        scale = amax / 448
        ties = rng.integers(0, 16, d) * 2.0 ** rng.integers(-10, 5, d) + 2.0 ** rng.integers(-10, 5, d)
        x[r] = np.clip(ties, 0, 448) * scale * rng.choice([-1, 1], d)
        x[r, 0] = amax
    x = torch.from_numpy(x).to(BF16).cuda().view(1, 1, 128, d)
    cache = P.paged_cache(1, 1, page, d, E4M3)
    P.cache_write(x, x, cache, ints([[0]]), ints([128]))
    code, scale = W.quantise_rows(f64(x)[0, 0])
    assert np.array_equal(f64(cache.K)[0, 0], code) and np.array_equal(cache.k_scale[0, 0].cpu().numpy(), scale)


@pytest.mark.parametrize("N", [1, 40])
def test_scales_of_every_size(N):
    """Value rows whose scales differ by up to 2^60, key rows with codes down to the smallest, and
    queries whose dimensions differ by 2^12: the weights keep their precision beside them."""
    lens, d, page = [600, 77], 128, 32
    rng = np.random.default_rng(31)
    table, total = table_of(lens, page, seed=31)
    cache = P.paged_cache(total, 2, page, d, E4M3)
    x = torch.randn(2, 2, 600, d, generator=torch.Generator().manual_seed(31))
    K = x.flip(2) * torch.from_numpy(rng.choice([1.0, 2.0 ** -7, 2.0 ** -12], (2, 2, 600, d))).float()
    V = x * torch.from_numpy(2.0 ** rng.integers(-30, 31, (2, 2, 600, 1))).float()
    P.cache_write(K.to(BF16).cuda(), V.to(BF16).cuda(), cache, table, ints(lens), ints(lens))
    Q = torch.randn(2, 8, N, d, generator=torch.Generator().manual_seed(32)) * torch.from_numpy(
        2.0 ** rng.integers(-12, 1, (2, 8, N, d))).float()
    Q = (Q * 4).to(BF16).cuda()
    O, lse = P.paged_attention(Q, cache, table, ints(lens))
    P.device_error()
    check_attention(O, lse, Q, cache, table, lens, [N] * 2, -1, 0, 0, d ** -0.5)


def test_offsets_past_32_bits():
    """A cache of more than 2^31 elements whose sequences lie in its last pages."""
    Hkv, page, d = 8, 128, 128
    num = 2 ** 31 // (Hkv * page * d) + 12
    cache = P.PagedCache(*(torch.empty(num, Hkv, page, d, dtype=BF16, device="cuda") for _ in "KV"))
    lens = [300, 130]
    table = ints([[num - 1, num - 3, num - 2], [num - 7, num - 4, -1]])
    K, V = randn(2, Hkv, 300, d, seed=41), randn(2, Hkv, 300, d, seed=42)
    P.cache_write(K, V, cache, table, ints(lens), ints(lens))
    back = P.cache_read(cache, table, ints(lens), 300)
    for b, n in enumerate(lens):
        assert torch.equal(back[0][b, :, :n], K[b, :, :n]) and torch.equal(back[1][b, :, :n], V[b, :, :n])
    for N in (1, 24):
        Q = randn(2, 16, N, d, seed=43)
        O, lse = P.paged_attention(Q, cache, table, ints(lens))
        P.device_error()
        for b, n in enumerate(lens):
            see = W.visible(n - N + np.arange(N), n, -1, 0, 0)
            for h in (0, 15):
                wo, wl, to, tl = T.forward(f64(Q)[b, h], f64(K)[b, h // 2, :n], f64(V)[b, h // 2, :n], see, d ** -0.5)
                T.check(f64(O)[b, h], wo, to, "O")
                T.check(f64(lse)[b, h], wl, tl, "lse")


@pytest.mark.parametrize("N", [1, 20])
def test_many_sequences(N):
    """More sequences than a block has threads, of all lengths, some empty, some without new tokens."""
    rng = np.random.default_rng(51)
    lens = [int(x) for x in rng.integers(0, 70, 300)]
    news = [min(int(x), n) for x, n in zip(rng.integers(0, N + 1, 300), lens)]
    cache, table = filled(lens, 1, 16, 64, E4M3, seed=51)
    Q = randn(300, 2, N, 64, seed=52)
    O, lse = P.paged_attention(Q, cache, table, ints(lens), ints(news))
    P.device_error()
    check_attention(O, lse, Q, cache, table, lens, news, -1, 0, 0, 64 ** -0.5)
    for b, m in enumerate(news):
        assert (O[b, :, m:] == 0).all() and (lse[b, :, m:] == 0).all()


def test_two_streams_at_once():
    """Calls in flight on two streams over one cache, each with its own workspace."""
    lens = [3000, 40]
    cache, table = filled(lens, 2, 64, 128, BF16, seed=53)
    Q = [randn(2, 8, n, 128, seed=54) for n in (1, 1, 30)]
    want = [P.paged_attention(q, cache, table, ints(lens)) for q in Q]
    n = ints(lens)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in Q]
    for _ in range(5):
        got = []
        for q, s in zip(Q, streams):
            with torch.cuda.stream(s):
                got.append(P.paged_attention(q, cache, table, n))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for x, y in zip(want, got) for a, b in zip(x, y))


@pytest.mark.parametrize("dtype", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("what", [float("nan"), float("inf")], ids=["nan", "inf"])
@pytest.mark.parametrize("N,Hq,d,mask", [
    (2, 4, 64, dict(left=-1, right=0, sinks=0)),
    (8, 4, 128, dict(left=40, right=0, sinks=7)),
    (5, 6, 64, dict(left=3, right=1, sinks=0)),
    (90, 2, 128, dict(left=-1, right=0, sinks=0)),
    (90, 6, 64, dict(left=33, right=10, sinks=50)),
])
def test_a_token_that_is_not_finite_reaches_the_rows_that_see_it(dtype, what, N, Hq, d, mask):
    """A value (in 8 bits its whole row) reaches the rows that see it; the others hold what they held
    (rows that share a tile with it sum again, without rounding the weights: 3 u max|v|). A key
    changes no bit of a row that does not see it. Tokens of the chunk, and older ones."""
    Hkv, page, lens = 2, 16, [400, 210]
    cache, table = filled(lens, Hkv, page, d, dtype, seed=8)
    Q = randn(2, Hq, N, d, seed=80)
    O, lse = P.paged_attention(Q, cache, table, ints(lens), **mask)
    top = float(np.nanmax(np.abs(values(cache)[1])))
    G, b, hk = Hq // Hkv, 1, 1
    left, right, sinks = (lens[b] if v < 0 else v for v in mask.values())
    p = np.arange(N) + lens[b] - N
    for at in (lens[b] - 1, lens[b] - 2, lens[b] - N, lens[b] - N - 2, 4):
        see = torch.from_numpy((at <= p + right) & ((at >= p - left) | (at < sinks))).cuda()
        i, r = int(table[b, at // page]), at % page
        for key in (False, True):
            t = cache.K if key else cache.V
            if dtype == E4M3:
                t = cache.k_scale if key else cache.v_scale
            old = t[i, hk, r].clone()
            if dtype == E4M3:
                t[i, hk, r] = float("nan")
            else:
                t[i, hk, r, 5] = what
            got, glse = P.paged_attention(Q, cache, table, ints(lens), **mask)
            t[i, hk, r] = old
            want = O.clone()
            mine = want[b, hk * G:(hk + 1) * G]
            if key:
                assert torch.equal(got[b, :, ~see], O[b, :, ~see]) and torch.equal(glse[b, :, ~see], lse[b, :, ~see])
                assert torch.equal(got[b, :hk * G], O[b, :hk * G]) and torch.equal(got[0], O[0])
                continue
            assert torch.equal(glse, lse)
            cols = slice(None) if dtype == E4M3 else slice(5, 6)
            mine[:, see, cols] = float("nan") if dtype == E4M3 else what
            assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.isinf(), want.isinf())
            have = got[b, hk * G:(hk + 1) * G]
            off = (have.float() - mine.float())[:, ~see, cols].abs()
            assert not off.numel() or float(off.max()) <= T.SLACK * 3 * T.U * top
            have[..., cols] = mine[..., cols]
            assert torch.equal(got.nan_to_num(), want.nan_to_num())
    P.device_error()


@pytest.mark.parametrize("dtype", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("N,Hq", [(7, 2), (90, 2), (90, 6)])
def test_rows_that_see_nothing_beside_rows_that_see_a_nan(dtype, N, Hq):
    """More new tokens than the sequence holds: the first ones have negative positions and see
    nothing, whatever the values that the others of their tile see."""
    Hkv, page, d = 2, 16, 64
    lens = [N - 4, 300]
    cache, table = filled(lens, Hkv, page, d, dtype, seed=9)
    Q = randn(2, Hq, N, d, seed=81)
    (cache.V if dtype == BF16 else cache.v_scale)[int(table[0, 0]), :, 1] = float("nan")
    O, lse = P.paged_attention(Q, cache, table, ints(lens))
    assert (O[0, :, :4] == 0).all() and (lse[0, :, :4] == float("-inf")).all()
    assert torch.isfinite(O[0, :, 4].float()).all() and torch.isnan(O[0, :, 5:].float()).all()
    assert torch.isfinite(O[1].float()).all() and torch.isfinite(lse[0, :, 4:]).all() and torch.isfinite(lse[1]).all()


@pytest.mark.parametrize("what", [float("nan"), float("inf")], ids=["nan", "inf"])
@pytest.mark.parametrize("N,Hq,d,mask", [
    (2, 4, 64, dict(left=-1, right=0, sinks=0)),
    (3, 8, 128, dict(left=-1, right=0, sinks=0)),
    (8, 4, 128, dict(left=40, right=0, sinks=7)),
    (5, 6, 64, dict(left=3, right=1, sinks=0)),
    (90, 2, 128, dict(left=-1, right=0, sinks=0)),
    (90, 6, 64, dict(left=33, right=10, sinks=50)),
])
def test_a_lost_token_as_the_cache_holds_it(what, N, Hq, d, mask):
    """8 bits: the row of a token that is not finite, written by cache_write (codes and scale are
    both NaN then), reaches the rows that see it and no others. An element of the value, or of the key."""
    Hkv, page, lens = 2, 16, [400, 210]
    cache, table = filled(lens, Hkv, page, d, E4M3, seed=8)
    Q = randn(2, Hq, N, d, seed=80)
    O, lse = P.paged_attention(Q, cache, table, ints(lens), **mask)
    top = float(np.nanmax(np.abs(values(cache)[1])))
    G, b = Hq // Hkv, 1
    left, right, sinks = (lens[b] if v < 0 else v for v in mask.values())
    p = np.arange(N) + lens[b] - N
    for at in (lens[b] - 1, lens[b] - 2, lens[b] - N, lens[b] - N - 2, 4):
        see = torch.from_numpy((at <= p + right) & ((at >= p - left) | (at < sinks))).cuda()
        i, r = int(table[b, at // page]), at % page
        for key in (False, True):
            written, lost = (P.PagedCache(*(t.clone() for t in cache)) for _ in range(2))
            new = [randn(1, Hkv, 1, d, seed=82 + k) for k in range(2)]
            new[0 if key else 1][0, 1, 0, 7] = what
            P.cache_write(*new, written, table[b:b + 1].contiguous(), ints([at + 1]))
            for t, w in ((lost.K, written.K), (lost.k_scale, written.k_scale)) if key else ((lost.V, written.V), (lost.v_scale, written.v_scale)):
                assert w[i, 1, r].float().isnan().all()
                t[i, 1, r] = w[i, 1, r]
            got, glse = P.paged_attention(Q, lost, table, ints(lens), **mask)
            assert torch.equal(got[0], O[0]) and torch.equal(got[b, :G], O[b, :G])
            assert got[b, G:, see].isnan().all()
            if key:
                assert glse[b, G:, see].isnan().all() and torch.equal(glse[b, :, ~see], lse[b, :, ~see])
                assert torch.equal(got[b, :, ~see], O[b, :, ~see])
            else:
                assert torch.equal(glse, lse)
                off = (got[b].float() - O[b].float())[:, ~see].abs()
                # p rounded once or not at all, either O rounded
                assert not off.numel() or float(off.max()) <= T.SLACK * 3 * T.U * top
    P.device_error()


def test_a_hundred_million_keys():
    """Sequences whose walk over the keys takes seconds: a role that waits for the next one's scores or
    queries does not give up. Keys of zero: lse = log of the keys seen. The sequences share their pages;
    only one of either tile has rows."""
    B, N, d, page, n = 300, 17, 64, 128, 110_000_000
    num = -(-n // page)
    cache = P.PagedCache(torch.zeros(num, 1, page, d, dtype=BF16, device="cuda"), torch.ones(num, 1, page, d, dtype=BF16, device="cuda"))
    table = torch.arange(num, dtype=torch.int32, device="cuda").repeat(B, 1)
    lens = torch.arange(n - B, n, dtype=torch.int32, device="cuda")
    Q = randn(B, 1, N, d, seed=61)
    O, lse = torch.full_like(Q, 5.0), torch.full((B, 1, N), 5.0, device="cuda")
    P.paged_attention(Q, cache, table, lens, out=O, lse=lse)
    P.device_error()
    seen = (lens[:, None].double() - N + 1 + torch.arange(N, device="cuda"))[:, None]
    assert float((lse.double() - seen.log()).abs().max()) <= 2.0 ** -19 + 2.0 ** -22 * 19
    # a sum of n terms in fp32 is off by up to n 2^-24 of sum p|v| = 1, here 6.6: that the rows were
    # written is all that can be said of O (the tensor core drops a product below 2^-26 of its sum)
    assert torch.isfinite(O.float()).all() and not (O == 5).any()


@pytest.mark.parametrize("dtype", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("N,lens,left", [(1, [5000, 70], -1), (4, [3000, 900], 2000), (70, [1500, 300], -1), (20, [9000], -1)])
@pytest.mark.parametrize("d", [64, 128])
def test_values_near_the_end_of_the_range(dtype, N, lens, left, d):
    """Values of one sign up to 2^126.3 (bf16: beside columns of 2^-90): the sums of exp(s - m) v leave
    fp32, the averages do not. Single tokens, chunks, sequences cut into runs."""
    Hkv, page = 2, 32
    table, total = table_of(lens, page, seed=62)
    cache = P.paged_cache(total, Hkv, page, d, dtype)
    K, V = (randn(len(lens), Hkv, max(lens), d, seed=62 + i) for i in range(2))
    V = (V.float().abs().clamp_max(4) + 0.5) * 2.0 ** 124
    if dtype == BF16:
        V[..., ::3] *= 2.0 ** -214
    P.cache_write(K, V.to(BF16), cache, table, ints(lens), ints(lens))
    Q = randn(len(lens), 4, N, d, seed=64)
    O, lse = P.paged_attention(Q, cache, table, ints(lens), left=left)
    P.device_error()
    check_attention(O, lse, Q, cache, table, lens, [N] * len(lens), left, 0, 0, d ** -0.5)
