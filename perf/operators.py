"""Cases for the operators that stand around differential attention: the rotary
positions with several axes that q and k get, the attention's forward, a
training pass through it, and its form for a few query rows over a key/value
cache.

``run`` computes them in plain 32-bit torch operations, or through this
package's entry points where ``own`` is set; ``exact`` says what they are in 64
bits. Layouts: q [B, Sq, H, 2, D], k [B, Sk, Hk, 2, D], v [B, Sk, Hk, Dv], the
weights of the second map broadcast over [B, Sq, H]; rotary tensors
[B, S, heads, D] with positions [axes, B, S].
"""
import math

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # One new token of 32 sequences: latency of the smallest call.
        dict(name="rotary_token", op="rotary", dtype="bf16", B=32, S=1, H=16, Hk=4, D=64, t=8, h=12, w=12,
             interleaved=False, inverse=False, packed=False, far=200000),
        # The gradient of a video clip's q and k, heads of both maps in a row, an odd token count.
        dict(name="rotary_video_gradient", op="rotary", dtype="fp16", B=2, S=4095, H=24, Hk=24, D=64, t=8, h=12, w=12,
             interleaved=True, inverse=True, packed=False, far=0),
        # A long batch, q and k as views of the packed projection, part of the head dim rotated.
        dict(name="rotary_packed_long", op="rotary", dtype="bf16", B=8, S=8192, H=16, Hk=16, D=128, t=16, h=16, w=16,
             interleaved=False, inverse=False, packed=True, far=0),
        # The forward on the smallest workload.
        dict(name="attend_small", op="attend", dtype="fp16", B=1, H=2, Hk=2, Sq=128, Sk=128, D=64, Dv=128, causal=False,
             lam="head"),
        # Narrow heads that share keys, ragged lengths, more keys than queries.
        dict(name="attend_ragged_shared", op="attend", dtype="bf16", B=2, H=12, Hk=4, Sq=1777, Sk=2000, D=40, Dv=80,
             causal=True, lam="token"),
        # The long context forward.
        dict(name="attend_long", op="attend", dtype="bf16", B=1, H=8, Hk=8, Sq=8192, Sk=8192, D=64, Dv=128, causal=True,
             lam="token"),
        # Training passes (forward and all gradients): an encoder's short sequences,
        dict(name="train_short", op="train", dtype="fp16", B=2, H=12, Hk=12, Sq=512, Sk=512, D=64, Dv=128, causal=False,
             lam="token"),
        # ragged lengths with shared key heads,
        dict(name="train_ragged_shared", op="train", dtype="bf16", B=2, H=12, Hk=4, Sq=2000, Sk=2000, D=64, Dv=64,
             causal=True, lam="token"),
        # and the long context.
        dict(name="train_long", op="train", dtype="bf16", B=1, H=8, Hk=8, Sq=8192, Sk=8192, D=64, Dv=128, causal=True,
             lam="token"),
        # Serving: one token of one sequence over a short cache,
        dict(name="token_short", op="token", dtype="fp16", B=1, H=8, Hk=8, Sq=1, Sk=1000, D=64, Dv=128, lam="head"),
        # a batch of sequences of mixed lengths with shared key heads,
        dict(name="token_batch", op="token", dtype="bf16", B=32, H=16, Hk=4, Sq=1, Sk=8192, D=64, Dv=128, lam="head"),
        # and four drafted tokens at the end of one very long sequence.
        dict(name="token_long", op="token", dtype="bf16", B=1, H=16, Hk=8, Sq=4, Sk=131000, D=64, Dv=128, lam="head"),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(("rotary", "attend", "train", "token"))
    c = dict(op=op, dtype=rng.choice(("fp16", "bf16")))
    if op == "rotary":
        D = 8 * rng.randint(2, 16)
        pairs = D // 2 if rng.random() < 0.7 else rng.randint(3, D // 2)
        t = rng.randint(1, pairs - 2)
        h = rng.randint(1, pairs - t - 1)
        Hk = rng.randint(1, 16)
        H = Hk * rng.choice((1, 1, 2, 4))
        B = rng.randint(1, 8)
        tokens = _log(rng, 1, max(2, 8192 * 8 * 32 * 128 // (D * (H + Hk)) // B))
        c.update(B=B, S=min(tokens, 20000), H=H, Hk=Hk, D=D, t=t, h=h, w=pairs - t - h, interleaved=rng.random() < 0.5,
                 inverse=rng.random() < 0.5, packed=rng.random() < 0.5, far=rng.choice((0, 0, 200000)))
        return c
    D, Dv = 8 * rng.randint(1, 8), 8 * rng.randint(1, 16)
    if rng.random() < 0.5:
        D, Dv = 64, 128
    Hk = rng.randint(1, 8)
    H = Hk * rng.choice((1, 1, 2, 3, 4))
    c.update(H=H, Hk=Hk, D=D, Dv=Dv, lam=rng.choice(("token", "head")) if op == "attend" else "head")
    if op == "token":
        B = _log(rng, 1, 32)
        c.update(B=B, Sq=rng.choice((1, 1, 1, 2, 4, 5)), Sk=_log(rng, 5, min(131000, 8192 * 32 * 4 // (B * Hk))))
        return c
    B = rng.randint(1, 3)
    most = 8 * 8192 * 8192 / (B * H)
    Sq = _log(rng, 32, min(8192, int(math.sqrt(most))))
    Sk = Sq if rng.random() < 0.5 else _log(rng, 32, min(8192, int(most / Sq)))
    c.update(B=B, Sq=Sq, Sk=Sk, causal=rng.random() < 0.6)
    if op == "train":
        c["lam"] = "token"
    return c


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dt)

    c = case
    s = dict(case=case)
    if c["op"] == "rotary":
        B, S, H, Hk, D = c["B"], c["S"], c["H"], c["Hk"], c["D"]
        if c["packed"]:  # the projection's output: q, k and v heads in one tensor
            x = normal(B, S, H + 2 * Hk, D)
            s["q"], s["k"] = x[:, :, :H], x[:, :, H:H + Hk]
        else:
            s["q"], s["k"] = normal(B, S, H, D), normal(B, S, Hk, D)
        # Patches of a clip in time, height, width order, each sequence from a start of its own.
        side = max(1, int(S ** (1 / 3)))
        at = torch.arange(S, device="cuda")
        start = torch.randint(0, c["far"] + 64, (B, 1), generator=g, device="cuda")
        grid = torch.stack((at // (side * side), at // side % side, at % side))
        s["positions"] = (grid[:, None, :] + start).to(torch.int32)
        s["sections"] = (c["t"], c["h"], c["w"])
        pairs = c["t"] + c["h"] + c["w"]
        s["inv_freq"] = 10000.0 ** (-torch.arange(pairs, device="cuda", dtype=torch.float64) / pairs)
        return s
    B, H, Hk, Sq, Sk, D, Dv = (c[n] for n in ("B", "H", "Hk", "Sq", "Sk", "D", "Dv"))
    s["q"], s["k"], s["v"] = normal(B, Sq, H, 2, D), normal(B, Sk, Hk, 2, D), normal(B, Sk, Hk, Dv)
    if c["lam"] == "head":  # one learned weight a head
        s["lam"] = torch.rand(H, generator=g, device="cuda") * 0.6 + 0.2
    else:  # a gate of every token and head, from a projection
        s["lam"] = torch.sigmoid(torch.randn((B, Sq, H), generator=g, device="cuda")).to(dt)
    if c["op"] == "train":
        s["do"] = normal(B, Sq, H, Dv)
        for n in ("q", "k", "v", "lam"):
            s[n].requires_grad_()
    if c["op"] == "token":
        low = max(min(Sq, Sk), Sk // 2)
        s["lens"] = torch.randint(low, Sk + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    return s


# ------------------------------------------------------------------ plain forms
def _rotate(x, cos, sin, pairs, interleaved):
    y = x.float()
    rot, rest = y[..., :2 * pairs], y[..., 2 * pairs:]
    if interleaved:
        a, b = rot[..., 0::2], rot[..., 1::2]
        out = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = rot[..., :pairs], rot[..., pairs:]
        out = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((out, rest), -1).to(x.dtype)


def _plain_rotary(s):
    c = s["case"]
    counts = torch.tensor(s["sections"], device="cuda")
    axis = torch.repeat_interleave(torch.arange(3, device="cuda"), counts)
    pairs = sum(s["sections"])
    angle = s["positions"].double()[axis].permute(1, 2, 0) * s["inv_freq"]  # [B, S, pairs]
    angle = -angle if c["inverse"] else angle
    cos, sin = angle.cos().float()[:, :, None], angle.sin().float()[:, :, None]
    return tuple(_rotate(s[n], cos, sin, pairs, c["interleaved"]) for n in ("q", "k"))


def _grouped(x, Hk):
    """[B, S, H, ...] -> [B, Hk, H/Hk * S, ...]: the rows that share a key head."""
    B, S, H = x.shape[:3]
    x = x.reshape(B, S, Hk, H // Hk, *x.shape[3:])
    return x.transpose(1, 2).transpose(2, 3).reshape(B, Hk, (H // Hk) * S, *x.shape[4:])


def _ungrouped(x, H, S):
    """The inverse of _grouped."""
    B, Hk = x.shape[:2]
    x = x.reshape(B, Hk, H // Hk, S, *x.shape[3:])
    return x.transpose(2, 3).transpose(1, 2).reshape(B, S, H, *x.shape[4:])


def _plain_maps(s, causal):
    """Both maps' probabilities [B, Hk, rows, Sk] and LSE [B, Hk, rows], in 32 bits."""
    c = s["case"]
    Hk, Sq, Sk = c["Hk"], c["Sq"], c["Sk"]
    G = c["H"] // Hk
    q = _grouped(s["q"].detach().float(), Hk)
    k = s["k"].detach().float().transpose(1, 2)
    cols = torch.arange(Sk, device="cuda")
    lens = s["lens"].long() if "lens" in s else torch.full((c["B"],), Sk, device="cuda")
    hide = (cols >= lens[:, None])[:, None, :]
    if causal:
        rows = torch.arange(Sq, device="cuda").repeat(G)
        hide = hide | (cols > rows[:, None] + (lens - Sq)[:, None, None])
    ps, lses = [], []
    for i in (0, 1):
        x = torch.matmul(q[..., i, :], k[..., i, :].transpose(-1, -2)) * c["D"] ** -0.5
        x = x.masked_fill(hide[:, None], -math.inf)
        top = x.amax(-1, keepdim=True)
        top = torch.where(top == -math.inf, torch.zeros_like(top), top)
        e = torch.exp(x - top)
        total = e.sum(-1, keepdim=True)
        ps.append(e / torch.where(total == 0, torch.ones_like(total), total))
        lses.append((top + torch.log(total))[..., 0])
    return q, k, ps, lses, hide


def _plain_values(s):
    """V [B, Hk, Sk, Dv] in 32 bits; rows behind a sequence's end hold nothing that counts."""
    v = s["v"].detach().float().transpose(1, 2)
    if "lens" in s:
        gone = torch.arange(s["case"]["Sk"], device="cuda") >= s["lens"][:, None]
        v = v.masked_fill(gone[:, None, :, None], 0.0)
    return v


def _plain_attend(s, causal):
    c = s["case"]
    H, Hk, Sq = c["H"], c["Hk"], c["Sq"]
    q, k, (p1, p2), lses, _ = _plain_maps(s, causal)
    v = _plain_values(s)
    lam = s["lam"].detach().float().expand(c["B"], Sq, H)
    lam = _grouped(lam, Hk)[..., None]
    o = torch.matmul(p1 - lam * p2, v)
    lse = torch.stack([_ungrouped(x, H, Sq).transpose(1, 2) for x in lses])
    return q, k, v, p1, p2, lam, o, lse


def _plain_train(s):
    c = s["case"]
    H, Hk, Sq = c["H"], c["Hk"], c["Sq"]
    scale = c["D"] ** -0.5
    q, k, v, p1, p2, lam, o, _ = _plain_attend(s, c["causal"])
    do = _grouped(s["do"].float(), Hk)
    dv = torch.matmul((p1 - lam * p2).transpose(-1, -2), do)
    dp = torch.matmul(do, v.transpose(-1, -2))
    d1, d2 = (p1 * dp).sum(-1, keepdim=True), (p2 * dp).sum(-1, keepdim=True)
    ds = (p1 * (dp - d1), -lam * p2 * (dp - d2))
    dq = torch.stack([torch.matmul(ds[i], k[..., i, :]) * scale for i in (0, 1)], -2)
    dk = torch.stack([torch.matmul(ds[i].transpose(-1, -2), q[..., i, :]) * scale for i in (0, 1)], -2)
    dt = s["q"].dtype
    return dict(o=_ungrouped(o, H, Sq).to(dt), dq=_ungrouped(dq, H, Sq).to(dt), dk=dk.transpose(1, 2).to(dt),
                dv=dv.transpose(1, 2).to(dt), dlam=_ungrouped(-d2[..., 0], H, Sq).to(s["lam"].dtype))


def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        from exact_io_aware_96_b200 import fa
        from exact_io_aware_96_b200.autograd import diff_attn_func
        if op == "rotary":
            return fa.rotary(s["q"], s["k"], s["positions"], s["inv_freq"], s["sections"],
                             interleaved=c["interleaved"], inverse=c["inverse"])
        if op == "train":
            o = diff_attn_func(s["q"], s["k"], s["v"], s["lam"], causal=c["causal"])
            dq, dk, dv, dlam = torch.autograd.grad(o, (s["q"], s["k"], s["v"], s["lam"]), s["do"])
            return dict(o=o, dq=dq, dk=dk, dv=dv, dlam=dlam)
        if op == "token":
            o, lse, _ = fa.diff_forward(s["q"], s["k"], s["v"], s["lam"], causal=True, k_lens=s["lens"])
        else:
            o, lse, _ = fa.diff_forward(s["q"], s["k"], s["v"], s["lam"], causal=c["causal"])
        return dict(o=o, lse=lse)
    if op == "rotary":
        return _plain_rotary(s)
    if op == "train":
        return _plain_train(s)
    *_, o, lse = _plain_attend(s, True if op == "token" else c["causal"])
    return dict(o=_ungrouped(o, c["H"], c["Sq"]).to(s["q"].dtype), lse=lse)


# ------------------------------------------------------------------ what counts
def _pairs(c):
    """(query, key) pairs of one head that the mask leaves."""
    if c["op"] == "token" or not c["causal"]:
        return c["Sq"] * c["Sk"]
    first = c["Sk"] - c["Sq"] + 1  # keys of the first row
    if first >= 1:
        return c["Sq"] * first + c["Sq"] * (c["Sq"] - 1) // 2
    return c["Sk"] * (c["Sk"] + 1) // 2


def work(case):
    c = case
    if c["op"] == "rotary":
        n = c["B"] * c["S"] * (c["H"] + c["Hk"]) * c["D"]
        return dict(bytes=4 * n + 12 * c["B"] * c["S"], flops=3 * n)
    B, H, Hk, Sq, Sk, D, Dv = (c[n] for n in ("B", "H", "Hk", "Sq", "Sk", "D", "Dv"))
    q, kv, o, rows = 2 * B * Sq * H * 2 * D, 2 * B * Sk * Hk * (2 * D + Dv), 2 * B * Sq * H * Dv, B * Sq * H
    pairs = B * H * _pairs(c)
    share = 0.75 if c["op"] == "token" else 1.0  # lengths are spread over the upper half of Sk
    if c["op"] == "train":  # q, k, v, lam, do in; o and four gradients out
        return dict(bytes=2 * (q + kv + o + 2 * rows), flops=2 * pairs * ((2 * D + 2 * Dv) + (6 * D + 2 * Dv)))
    return dict(bytes=q + share * kv + o + 8 * rows, flops=2 * share * pairs * (2 * D + 2 * Dv))


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "rotary":
        axis = [a for a, n in enumerate(s["sections"]) for _ in range(n)]
        pairs = len(axis)
        out = []
        for n in ("q", "k"):
            x = s[n].double()
            y = x.clone()
            for j, a in enumerate(axis):
                th = s["positions"][a].double() * s["inv_freq"][j]
                co, si = torch.cos(th)[..., None], torch.sin(th)[..., None]
                si = -si if c["inverse"] else si
                i0, i1 = (2 * j, 2 * j + 1) if c["interleaved"] else (j, j + pairs)
                y[..., i0] = x[..., i0] * co - x[..., i1] * si
                y[..., i1] = x[..., i0] * si + x[..., i1] * co
            out.append(y)
        return tuple(out)
    B, H, Hk, Sq, Sk, D, Dv = (c[n] for n in ("B", "H", "Hk", "Sq", "Sk", "D", "Dv"))
    train = c["op"] == "train"
    causal = True if c["op"] == "token" else c["causal"]
    q, k, v, lam = (s[n].detach().double() for n in ("q", "k", "v", "lam"))
    lam = lam.expand(B, Sq, H)
    o = torch.zeros(B, Sq, H, Dv, device="cuda", dtype=torch.float64)
    lse = torch.full((2, B, H, Sq), -math.inf, device="cuda", dtype=torch.float64)
    if train:
        do = s["do"].double()
        dq, dk, dv, dlam = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v), torch.zeros_like(lam)
    for b in range(B):
        n = int(s["lens"][b]) if "lens" in s else Sk
        see = torch.ones(Sq, n, device="cuda", dtype=torch.bool)
        if causal:
            see = see.tril(n - Sq)
        some = see.any(1)
        for h in range(H):
            kh = h // (H // Hk)
            vals = v[b, :n, kh]
            maps = []
            for i in (0, 1):
                x = (q[b, :, h, i] @ k[b, :n, kh, i].T / math.sqrt(D)).masked_fill(~see, -math.inf)
                lse[i, b, h] = torch.logsumexp(x, 1)
                maps.append(torch.where(see, torch.exp(x - torch.where(some, lse[i, b, h], 0.0)[:, None]), 0.0))
            o2 = maps[1] @ vals
            o[b, :, h] = maps[0] @ vals - lam[b, :, h, None] * o2
            if train:
                g = do[b, :, h]
                dlam[b, :, h] = -(g * o2).sum(1)
                dp = g @ vals.T
                weights = (torch.ones_like(lam[b, :, h]), -lam[b, :, h])
                for i in (0, 1):
                    inner = (maps[i] * dp).sum(1, keepdim=True)
                    ds = weights[i][:, None] * maps[i] * (dp - inner) / math.sqrt(D)
                    dq[b, :, h, i] = ds @ k[b, :, kh, i]
                    dk[b, :, kh, i] += ds.T @ q[b, :, h, i]
                    dv[b, :, kh] += weights[i][:, None].mul(maps[i]).T @ g
    if train:
        return dict(o=o, dq=dq, dk=dk, dv=dv, dlam=dlam)
    return dict(o=o, lse=lse)
