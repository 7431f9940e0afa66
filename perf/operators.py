"""Cases of the windowed attention, its gradient, the paged key/value cache and the attention over it.

Every case is one call (or a forward with its backward) as a program makes it. The plain form
computes the same from elementary torch operations in 32 bits, rounded once at the end.

Mask of the attentions: a query at position p sees key j if j <= p + right and (j >= p - left or
j < sinks); a negative left or right sets no limit on that side. Query head h reads key head
h // (Hq / Hkv). A cache holds pages of tokens; new tokens are the last ones of their sequence.
"""
import math

import numpy as np
import torch

own = False

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
TINY = 2.0 ** -126  # smallest scale of a quantised cache row


def listed():
    return [
        # one small map, window on both sides: the call's latency
        dict(name="window_small", op="window", B=1, Hq=8, Hkv=8, N=256, d=64, left=64, right=64, sinks=4),
        # image latents 64 x 64, eight image rows to either side
        dict(name="window_image", op="window", B=2, Hq=24, Hkv=24, N=4096, d=128, left=512, right=512, sinks=0),
        # a training step on a short odd sequence, shared key heads
        dict(name="train_odd", op="train", B=1, Hq=12, Hkv=4, N=2049, d=64, left=511, right=0, sinks=5),
        # a training step on a long causal sequence with first tokens that stay visible
        dict(name="train_long", op="train", B=1, Hq=16, Hkv=4, N=16384, d=128, left=2047, right=0, sinks=64),
        # every sequence of a batch appends its newest token
        dict(name="write_token", op="write", B=64, Hkv=8, N=1, d=128, page=64, kv=4096, kind="e4m3"),
        # a frame's worth of latents is appended
        dict(name="write_chunk", op="write", B=2, Hkv=24, N=4096, d=128, page=128, kv=8192, kind="e4m3"),
        # whole sequences of different lengths are read back
        dict(name="read_ragged", op="read", B=8, Hkv=8, N=16384, d=128, page=64, kv=16384, kind="e4m3"),
        # one sequence, one token, short cache: the call's latency
        dict(name="token_small", op="paged", B=1, Hq=8, Hkv=2, N=1, d=64, page=16, kv=300, kind="bf16",
             left=-1, right=0, sinks=0),
        # one token for each sequence of a batch of different lengths
        dict(name="token_batch", op="paged", B=32, Hq=32, Hkv=8, N=1, d=128, page=64, kv=8192, kind="bf16",
             left=-1, right=0, sinks=0),
        # one token each over long quantised caches
        dict(name="token_long", op="paged", B=4, Hq=40, Hkv=8, N=1, d=128, page=128, kv=75600, kind="e4m3",
             left=-1, right=0, sinks=0),
        # a chunk of new tokens over a longer cache, window and first tokens
        dict(name="chunk", op="paged", B=2, Hq=24, Hkv=8, N=1024, d=128, page=64, kv=16384, kind="bf16",
             left=8191, right=0, sinks=64),
        # an odd chunk over a quantised cache of small pages
        dict(name="chunk_odd", op="paged", B=3, Hq=12, Hkv=4, N=333, d=64, page=16, kv=5003, kind="e4m3",
             left=-1, right=0, sinks=0),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    d = rng.choice([64, 128])
    op = rng.choice(["window", "train", "write", "read", "paged", "paged", "paged"])
    if op in ("window", "train"):
        Hkv = rng.choice([1, 2, 3, 4, 8])
        Hq = Hkv * rng.choice([1, 2, 3, 4])
        N = log(100, 12000)
        while Hq * N * N > 2 * 10 ** 9:
            N = N * 2 // 3
        left = rng.choice([-1, log(16, 4096), log(16, 4096)])
        right = rng.choice([0, 0, left, log(16, 1024)])
        return dict(op=op, B=rng.choice([1, 1, 2]), Hq=Hq, Hkv=Hkv, N=N, d=d, left=left, right=right,
                    sinks=rng.choice([0, rng.randint(1, 200)]))
    c = dict(op=op, d=d, page=rng.choice([16, 32, 64, 128]), kind=rng.choice(["bf16", "e4m3"]))
    Hkv = rng.choice([1, 2, 4, 5, 8, 24])
    if op in ("write", "read"):
        B = rng.choice([1, 2, 5, 16, 48])
        kv = log(64, 20000)
        while B * Hkv * kv > 2 * 10 ** 6:
            kv = kv * 2 // 3 + 1
        return dict(c, B=B, Hkv=Hkv, N=kv if op == "read" else min(kv, rng.choice([1, log(2, 4096)])), kv=kv)
    N = rng.choice([1, 1, log(2, 16), log(16, 1500)])
    Hq = Hkv * rng.choice([1, 2, 3, 4, 5, 8])
    B = rng.choice([1, 2, 3, 8, 20])
    kv = max(N, log(100, 60000))
    while B * Hkv * kv > 3 * 10 ** 6 or B * Hq * N * kv > 4 * 10 ** 8:
        kv = kv * 2 // 3 + 1
        N = min(N, kv)
        B = max(1, B - 1)
    return dict(c, B=B, Hq=Hq, Hkv=Hkv, N=N, kv=kv, left=rng.choice([-1, -1, log(64, 8192)]),
                right=rng.choice([0, 0, 0, -1]), sinks=rng.choice([0, 0, rng.randint(1, 200)]))


def _lens(c):
    """Tokens held by each sequence: the longest has kv, the others between half of it and all."""
    B, kv, N = c["B"], c["kv"], c["N"] if c["op"] != "read" else 1
    return [max(N, kv - (kv // 2) * ((b * 37) % B) // B) for b in range(B)]


def _randn(g, *shape):
    return torch.randn(*shape, device="cuda", generator=g)


def _quantised(x):
    """(codes, scale) of rows of x (32 bits)."""
    scale = (x.abs().amax(-1) / 448).clamp_min(TINY)
    return (x / scale[..., None]).to(E4M3), scale


def _pages(c, g):
    """A filled cache, its page table (-1 where no page is held) and the sequences' lengths."""
    lens = _lens(c)
    held = [-(-n // c["page"]) for n in lens]
    total = sum(held)
    order = torch.randperm(total, device="cuda", generator=g).to(torch.int32)
    at = np.full((c["B"], max(held)), -1, np.int64)
    used = 0
    for b, n in enumerate(held):
        at[b, :n] = np.arange(used, used + n)
        used += n
    at = torch.from_numpy(at).to("cuda")
    table = torch.where(at >= 0, order[at.clamp_min(0)], -1).to(torch.int32).contiguous()
    s = dict(c, table=table, lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    shape = (total, c["Hkv"], c["page"], c["d"])
    for name in ("K", "V"):
        x = _randn(g, *shape)
        if c["kind"] == "bf16":
            s["c" + name], s["s" + name] = x.to(BF16), None
        else:
            s["c" + name], s["s" + name] = _quantised(x)
    return s


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if c["op"] in ("window", "train"):
        s = dict(c, Q=_randn(g, c["B"], c["Hq"], c["N"], c["d"]).to(BF16))
        for name in ("K", "V"):
            s[name] = _randn(g, c["B"], c["Hkv"], c["N"], c["d"]).to(BF16)
        if c["op"] == "train":
            s["dO"] = _randn(g, c["B"], c["Hq"], c["N"], c["d"]).to(BF16)
        return s
    s = _pages(c, g)
    if c["op"] == "write":
        for name in ("K", "V"):
            s[name] = _randn(g, c["B"], c["Hkv"], c["N"], c["d"]).to(BF16)
    elif c["op"] == "paged":
        s["Q"] = _randn(g, c["B"], c["Hq"], c["N"], c["d"]).to(BF16)
    else:
        s["out"] = [torch.zeros(c["B"], c["Hkv"], c["N"], c["d"], device="cuda", dtype=BF16) for _ in "KV"]
    return s


# ------------------------------------------------------------------ plain forms

def _visible(s, p, n):
    """Truth values [..., rows, n]: which keys the queries at positions p see."""
    j = torch.arange(n, device=p.device)
    p = p[..., None]
    see = (j >= p - s["left"]) | (j < s["sinks"]) if s["left"] >= 0 else torch.ones_like(j >= p)
    return see & (j <= p + s["right"]) if s["right"] >= 0 else see


def _attend(q, K, V, see):
    """Softmax attention of q [.., rows, d] (scaled) over K, V [.., n, d]; (o, lse, p). No key: o = 0, lse = -inf."""
    p = q @ K.mT
    p.masked_fill_(~see, -math.inf)
    m = p.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    lse = m + l.log()
    p.div_(torch.where(l == 0, 1.0, l))
    return p @ V, lse[..., 0], p


def _plain_window(s):
    B, Hq, Hkv, N, d = (s[k] for k in ("B", "Hq", "Hkv", "N", "d"))
    G = Hq // Hkv
    scale = d ** -0.5
    grouped = (B, Hkv, G * N, d)
    q, K, V = s["Q"].float().view(grouped) * scale, s["K"].float(), s["V"].float()
    see = _visible(s, torch.arange(N, device=q.device), N).repeat(G, 1)
    o, lse, p = _attend(q, K, V, see)
    out = dict(O=o.view(B, Hq, N, d).to(BF16), lse=lse.reshape(B, Hq, N))
    if s["op"] == "window":
        return out
    do = s["dO"].float().view(grouped)
    dv = p.mT @ do
    dp = do @ V.mT
    dp.sub_((do * o).sum(-1, keepdim=True)).mul_(p)
    dq = dp @ K * scale
    dk = dp.mT @ q
    return dict(out, dQ=dq.view(B, Hq, N, d).to(BF16), dK=dk.to(BF16), dV=dv.to(BF16))


def _slots(s):
    """Page and row of the new tokens [B, N]."""
    pos = s["lens"][:, None].long() - s["N"] + torch.arange(s["N"], device="cuda")
    return s["table"].gather(1, pos // s["page"]).long(), pos % s["page"]


def _plain_write(s):
    page, row = _slots(s)
    for name in ("K", "V"):
        x = s[name].transpose(1, 2)  # [B, N, Hkv, d]
        if s["kind"] == "bf16":
            s["c" + name][page, :, row] = x
        else:
            code, scale = _quantised(x.float())
            s["c" + name].view(torch.uint8)[page, :, row] = code.view(torch.uint8)
            s["s" + name][page, :, row] = scale
    return {k: s[k] for k in ("cK", "cV", "sK", "sV") if s[k] is not None}


def _gathered(s, name):
    """The sequences' rows [B, Hkv, tokens, d] in 32 bits; rows behind a sequence's last are zero."""
    at = s["table"].clamp_min(0).long()
    x = s["c" + name].view(torch.uint8)[at].view(s["c" + name].dtype).float()  # [B, pages, Hkv, page, d]
    if s["kind"] != "bf16":
        x = x * s["s" + name][at][..., None]
    x = x.transpose(1, 2).flatten(2, 3)
    held = torch.arange(x.shape[2], device=x.device) < s["lens"][:, None]
    return x.masked_fill_(~held[:, None, :, None], 0.0), held


def _plain_read(s):
    for out, name in zip(s["out"], ("K", "V")):
        x, held = _gathered(s, name)
        n = min(s["N"], x.shape[2])
        out[:, :, :n] = torch.where(held[:, None, :n, None], x[:, :, :n].to(BF16), out[:, :, :n])
    return dict(K=s["out"][0], V=s["out"][1])


def _plain_paged(s):
    B, Hq, Hkv, N, d = (s[k] for k in ("B", "Hq", "Hkv", "N", "d"))
    G = Hq // Hkv
    K, held = _gathered(s, "K")
    V, _ = _gathered(s, "V")
    pos = s["lens"][:, None] - N + torch.arange(N, device="cuda")
    see = _visible(s, pos, K.shape[2]) & held[:, None]
    q = s["Q"].float().view(B, Hkv, G * N, d) * d ** -0.5
    o, lse, _ = _attend(q, K, V, see.repeat(1, G, 1)[:, None])
    return dict(O=o.view(B, Hq, N, d).to(BF16), lse=lse.reshape(B, Hq, N))


# ------------------------------------------------------------------ one pass

def _cache(s):
    import block_sparse_attention_pisa_b200 as P

    return P.PagedCache(s["cK"], s["cV"], s["sK"], s["sV"])


def run(state):
    s = state
    if not own:
        return {"window": _plain_window, "train": _plain_window, "write": _plain_write, "read": _plain_read,
                "paged": _plain_paged}[s["op"]](s)
    import block_sparse_attention_pisa_b200 as P

    if s["op"] in ("window", "train"):
        mask = dict(left=s["left"], right=s["right"], sinks=s["sinks"])
        O, lse = P.window_attention(s["Q"], s["K"], s["V"], **mask)
        if s["op"] == "window":
            return dict(O=O, lse=lse)
        dQ, dK, dV = P.window_attention_backward(s["dO"], s["Q"], s["K"], s["V"], O, lse, **mask)
        return dict(O=O, lse=lse, dQ=dQ, dK=dK, dV=dV)
    if s["op"] == "write":
        P.cache_write(s["K"], s["V"], _cache(s), s["table"], s["lens"])
        return {k: s[k] for k in ("cK", "cV", "sK", "sV") if s[k] is not None}
    if s["op"] == "read":
        K, V = P.cache_read(_cache(s), s["table"], s["lens"], s["N"], out=s["out"])
        return dict(K=K, V=V)
    O, lse = P.paged_attention(s["Q"], _cache(s), s["table"], s["lens"], left=s["left"], right=s["right"],
                               sinks=s["sinks"])
    return dict(O=O, lse=lse)


# ------------------------------------------------------------------ what a pass cannot do without

def _pairs(c, p, n):
    """(visible pairs, keys that some row sees) for queries at positions p over n keys."""
    left = c["left"] if c["left"] >= 0 else n + len(p)
    right = c["right"] if c["right"] >= 0 else n + len(p)
    lo, hi = np.clip(p - left, 0, n), np.clip(p + right + 1, 0, n)
    first = np.minimum(np.minimum(c["sinks"], lo), hi)
    seen = max(0, int(hi.max() - lo.min())) + int(min(c["sinks"], lo.min()))
    return int((np.maximum(hi - lo, 0) + np.maximum(first, 0)).sum()), seen


def work(case):
    c = case
    if c["op"] in ("window", "train"):
        B, Hq, Hkv, N, d = (c[k] for k in ("B", "Hq", "Hkv", "N", "d"))
        pairs, _ = _pairs(c, np.arange(N), N)
        q, k, row = 2 * B * Hq * N * d, 2 * B * Hkv * N * d, 4 * B * Hq * N
        if c["op"] == "window":
            return dict(bytes=2 * q + 2 * k + row, flops=4 * d * pairs * B * Hq)
        return dict(bytes=4 * q + 4 * k + row, flops=14 * d * pairs * B * Hq)
    B, Hkv, N, d = (c[k] for k in ("B", "Hkv", "N", "d"))
    per = 2 * d if c["kind"] == "bf16" else d + 4
    lens = _lens(c)
    if c["op"] == "write":
        return dict(bytes=2 * B * Hkv * N * (2 * d + per) + 4 * B * (N // c["page"] + 1), flops=2 * 2 * B * Hkv * N * d)
    if c["op"] == "read":
        tokens = sum(min(n, N) for n in lens)
        return dict(bytes=2 * Hkv * tokens * (2 * d + per) + 4 * tokens // c["page"], flops=2 * Hkv * tokens * d)
    both = [_pairs(c, np.arange(n - N, n), n) for n in lens]
    return dict(bytes=sum(2 * Hkv * seen * per for _, seen in both) + 4 * B * c["Hq"] * N * (d + 1),
                flops=sum(4 * d * pairs * c["Hq"] for pairs, _ in both))


# ------------------------------------------------------------------ from the definitions, in 64 bits

def _exact_rows(q, K, V, see, do=None):
    """One head: q, do [rows, d], K, V [n, d], see [rows, n]."""
    s = torch.where(see, torch.einsum("rd,nd->rn", q, K), -math.inf)
    lse = torch.logsumexp(s, 1)
    p = torch.where(see, torch.exp(s - torch.where(torch.isfinite(lse), lse, 0.0)[:, None]), 0.0)
    o = torch.einsum("rn,nd->rd", p, V)
    if do is None:
        return o, lse
    w = torch.einsum("rd,nd->rn", do, V)
    ds = p * (w - (p * w).sum(1, keepdim=True))
    return o, lse, torch.einsum("rn,nd->rd", ds, K), torch.einsum("rn,rd->nd", ds, q), torch.einsum("rn,rd->nd", p, do)


def _exact_see(c, pos, n):
    see = torch.zeros(len(pos), n, dtype=torch.bool, device="cuda")
    key = torch.arange(n, device="cuda").expand(len(pos), n)
    at = torch.tensor(pos, device="cuda")[:, None]
    near = key >= at - c["left"] if c["left"] >= 0 else key >= 0
    see |= near | (key < c["sinks"])
    if c["right"] >= 0:
        see &= key <= at + c["right"]
    return see


def _exact_cache(s, name, b, h, n):
    rows = []
    for i in range(-(-n // s["page"])):
        at = int(s["table"][b, i])
        x = s["c" + name][at, h].double()
        rows.append(x if s["s" + name] is None else x * s["s" + name][at, h].double()[:, None])
    return torch.cat(rows)[:n]


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    scale = c["d"] ** -0.5
    if c["op"] in ("window", "train"):
        G = c["Hq"] // c["Hkv"]
        see = _exact_see(c, list(range(c["N"])), c["N"])
        out = {k: torch.zeros(*s[n].shape, dtype=torch.float64, device="cuda")
               for k, n in (("O", "Q"), ("dQ", "Q"), ("dK", "K"), ("dV", "V"))}
        out["lse"] = torch.zeros(*s["Q"].shape[:3], dtype=torch.float64, device="cuda")
        for b in range(c["B"]):
            for h in range(c["Hq"]):
                q, K, V = s["Q"][b, h].double() * scale, s["K"][b, h // G].double(), s["V"][b, h // G].double()
                r = _exact_rows(q, K, V, see, s["dO"][b, h].double() if c["op"] == "train" else None)
                out["O"][b, h], out["lse"][b, h] = r[0], r[1]
                if c["op"] == "train":
                    out["dQ"][b, h] = r[2] * scale
                    out["dK"][b, h // G] += r[3]
                    out["dV"][b, h // G] += r[4]
        return out if c["op"] == "train" else {k: out[k] for k in ("O", "lse")}
    if c["op"] == "write":
        out = {}
        for name in ("K", "V"):
            codes = s["c" + name].double()
            scales = None if s["s" + name] is None else s["s" + name].double()
            for b in range(c["B"]):
                pos = torch.arange(c["N"], device="cuda") + int(s["lens"][b]) - c["N"]
                page, row = s["table"][b][pos // c["page"]].long(), pos % c["page"]
                x = s[name][b].double()  # [Hkv, N, d]
                if scales is None:
                    codes[page, :, row] = x.transpose(0, 1)
                    continue
                step = (x.abs().amax(2) / 448).clamp_min(TINY)
                # three mantissa bits: the step of a value in [2^e, 2^(e+1)) is 2^(e-3), at least 2^-9
                y = x / step[..., None]
                e = torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6)))
                unit = torch.exp2(e - 3)
                codes[page, :, row] = (torch.round(y / unit) * unit).clamp(-448, 448).transpose(0, 1)
                scales[page, :, row] = step.transpose(0, 1)
            out["c" + name] = codes
            if scales is not None:
                out["s" + name] = scales
        return out
    if c["op"] == "read":
        out = dict(K=s["out"][0].double(), V=s["out"][1].double())
        for b, n in enumerate(_lens(c)):
            for h in range(c["Hkv"]):
                for name in ("K", "V"):
                    m = min(n, c["N"])
                    out[name][b, h, :m] = _exact_cache(s, name, b, h, n)[:m]
        return out
    G = c["Hq"] // c["Hkv"]
    O = torch.zeros(*s["Q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(*s["Q"].shape[:3], dtype=torch.float64, device="cuda")
    for b, n in enumerate(_lens(c)):
        see = _exact_see(c, list(range(n - c["N"], n)), n)
        for h in range(c["Hkv"]):
            K, V = _exact_cache(s, "K", b, h, n), _exact_cache(s, "V", b, h, n)
            for i in range(h * G, h * G + G):
                O[b, i], lse[b, i] = _exact_rows(s["Q"][b, i].double() * scale, K, V, see)
    return dict(O=O, lse=lse)
