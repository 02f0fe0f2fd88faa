"""Cases for the operators of a hybrid transformer block around the frame scan:
layer norm, rotary positions over several axes, and softmax attention.

``run`` computes each in plain torch operations, or, where ``own`` is true,
through the library's entry points.  The sizes are the library's workloads: a
22 x 40 = 880-token latent frame, a 21-frame clip, a 121-frame minute, 16 heads
of 128 and a model width of 2048, beside generic ragged ones.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one streamed latent frame through a block's norm (serving; a call of a few microseconds)
        dict(name="norm_frame", op="norm", rows=880, C=2048, dtype="bf16", wdtype="bf16", train=False),
        # a minute's training step through a block's norm
        dict(name="norm_minute_train", op="norm", rows=121 * 880, C=2048, dtype="bf16", wdtype="f32", train=True),
        # fp32 training on a short odd batch: a width that fills no vector width evenly
        dict(name="norm_odd_f32_train", op="norm", rows=1777, C=1001, dtype="f32", wdtype="f32", train=True),
        # queries and keys of one streamed frame, far into the rollout
        dict(name="rotary_frame", op="rotary", B=1, F=1, Hg=22, Wg=40, Hq=16, Hk=16, D=128, axes="44,42,42",
             offset=1210, halves=False, dtype="bf16", train=False),
        # queries and keys of a whole minute
        dict(name="rotary_minute", op="rotary", B=1, F=121, Hg=22, Wg=40, Hq=16, Hk=16, D=128, axes="44,42,42",
             offset=0, halves=False, dtype="bf16", train=False),
        # fp32 training: forward and gradient, grouped heads, half-split pairs, part of the head rotated
        dict(name="rotary_grouped_f32_train", op="rotary", B=2, F=5, Hg=17, Wg=23, Hq=12, Hk=4, D=64, axes="16,20,20",
             offset=3, halves=True, dtype="f32", train=True),
        # serving single tokens: eight requests, each one query against a cache filled in part
        dict(name="attn_token", op="attn", lens_q="1,1,1,1,1,1,1,1", lens_k="40,511,1000,3777,8191,12000,30001,32768",
             room=32768, Hq=32, Hk=8, D=128, causal=True, block=1, dtype="bf16", train=False),
        # streaming: the 22nd frame's queries against the cache of all frames so far
        dict(name="attn_frame", op="attn", lens_q="880", lens_k="19360", room=20000, Hq=16, Hk=16, D=128, causal=True,
             block=880, dtype="bf16", train=False),
        # a softmax block over a short clip, frame-causal
        dict(name="attn_clip", op="attn", lens_q="18480", lens_k="18480", room=0, Hq=16, Hk=16, D=128, causal=True,
             block=880, dtype="bf16", train=False),
        # training on packed sequences of different lengths, token-causal, grouped heads
        dict(name="attn_packed_train", op="attn", lens_q="4096,1,2309,880,64,777,17,32",
             lens_k="4096,1,2309,880,64,777,17,32", room=0, Hq=16, Hk=4, D=128, causal=True, block=1, dtype="bf16",
             train=True),
        # training on eight frames, every token sees every token (the bidirectional weights)
        dict(name="attn_full_train", op="attn", lens_q="7040", lens_k="7040", room=0, Hq=16, Hk=16, D=64,
             causal=False, block=1, dtype="bf16", train=True),
        # fp32 training on short odd sequences, one of them with fewer keys than queries (rows that see nothing)
        dict(name="attn_odd_f32_train", op="attn", lens_q="333,100,7,65", lens_k="333,37,200,65", room=0, Hq=6, Hk=2,
             D=64, causal=True, block=1, dtype="f32", train=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw_norm(rng):
    train = rng.random() < 0.5
    C = rng.choice([_log(rng, 16, 8192), 8 * _log(rng, 8, 1024), 64 * rng.randint(4, 64)])
    rows = _log(rng, 1, min(121 * 880, (121 * 880 * 2048) // C // 2))
    dtype = rng.choice(["bf16", "bf16", "f32"])
    return dict(op="norm", rows=rows, C=C, dtype=dtype, wdtype="f32" if dtype == "f32" else rng.choice(["bf16", "f32"]),
                train=train)


def _draw_rotary(rng):
    D = rng.choice([32, 64, 64, 128, 128])
    kind = rng.randrange(3)
    if kind == 0:
        a = 2 * (D // 6)
        axes = [D - 2 * a, a, a]
    elif kind == 1:
        axes = [D // 4, D // 4, D // 4]
    else:
        axes = [D // 2, D // 2]
    Hk = rng.choice([1, 2, 4, 8, 16])
    Hq = Hk * rng.choice([1, 1, 2, 4])
    Hg, Wg = rng.randint(1, 24), rng.randint(1, 40)
    B = rng.choice([1, 1, 2, 3])
    dtype, train = rng.choice(["bf16", "bf16", "f32"]), rng.random() < 0.4
    cost = (1 if dtype == "bf16" else 2) * (2 if train else 1)
    most = (121 * 880 * 32 * 128) // (B * Hg * Wg * (Hq + Hk) * D * cost)
    return dict(op="rotary", B=B, F=_log(rng, 1, max(1, min(121, most))), Hg=Hg, Wg=Wg, Hq=Hq, Hk=Hk, D=D,
                axes=",".join(map(str, axes)), offset=_log(rng, 1, 100000) - 1, halves=rng.random() < 0.5,
                dtype=dtype, train=train)


def _draw_attn(rng):
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    D = rng.choice([32, 64, 128, 128])
    Hk = rng.choice([1, 2, 4, 8])
    Hq = Hk * rng.choice([1, 2, 4, 8])
    kind = rng.choice(["token", "stream", "prompt", "packed", "packed"])
    room, train = 0, False
    if kind == "token":
        n = _log(rng, 1, 32)
        lq = [rng.choice([1, 1, 1, rng.randint(2, 5)])] * n
        most = min(32768, 1500000000 // (n * Hk * D * (4 if dtype == "bf16" else 8)))
        lk = [max(lq[0], _log(rng, 1, most)) for _ in range(n)]
        room, causal, block = max(lk) + rng.randint(0, 100), True, 1
    elif kind == "stream":
        N = _log(rng, 32, 880)
        lq, lk = [N], [N * rng.randint(1, 16)]
        room, causal, block = lk[0] + rng.randint(0, 500), True, N
    elif kind == "prompt":
        n, length = rng.randint(1, 3), _log(rng, 16, 4096 if dtype == "bf16" else 1024)
        lq = [length] * n
        lk, train = list(lq), rng.random() < 0.5
        causal, block = rng.random() < 0.7, rng.choice([1, 1, _log(rng, 2, 880)])
    else:
        n = rng.randint(2, 12)
        lq = [_log(rng, 1, 2048 if dtype == "bf16" else 512) for _ in range(n)]
        lk = [x if rng.random() < 0.7 else _log(rng, 1, 1024) for x in lq]
        train, causal, block = rng.random() < 0.6, rng.random() < 0.7, 1
    # no more than the listed clip: its scores, and its products
    while Hq * sum(lq) * max(room * len(lk), sum(lk)) > 16 * 18480 ** 2 or \
            sum(map(lambda a, b: a * b, lq, lk)) * Hq * D * (14 if train else 4) > 1.4e12:
        Hq, Hk = (Hq // 2, Hk) if Hq > Hk else (Hq // 2, Hk // 2)
    return dict(op="attn", lens_q=",".join(map(str, lq)), lens_k=",".join(map(str, lk)), room=room, Hq=Hq, Hk=Hk, D=D,
                causal=causal, block=block, dtype=dtype, train=train)


def draw(rng):
    return rng.choice([_draw_norm, _draw_rotary, _draw_attn, _draw_attn])(rng)


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, shape, dtype, std=1.0, mean=0.0):
    return (torch.randn(shape, generator=g, device="cuda") * std + mean).to(dtype)


def _lens(case):
    return [[int(x) for x in case[n].split(",")] for n in ("lens_q", "lens_k")]


def _starts(lens, room=0):
    at = [0]
    for n in lens:
        at.append(at[-1] + (room or n))
    return at


def prepare(case, seed):
    g = _gen(seed)
    dt = DTYPES[case["dtype"]]
    s = dict(case)
    if case["op"] == "norm":
        rows, C, wt = case["rows"], case["C"], DTYPES[case["wdtype"]]
        # hidden states: a channel profile shared by all tokens, plus each token's own part
        s["x"] = (torch.randn((rows, C), generator=g, device="cuda") +
                  0.5 * torch.randn((1, C), generator=g, device="cuda")).to(dt)
        s["weight"], s["bias"] = _randn(g, (C,), wt, 0.2, 1.0), _randn(g, (C,), wt, 0.2)
        if case["train"]:
            s["dy"] = _randn(g, (rows, C), dt)
    elif case["op"] == "rotary":
        B, F, Hg, Wg, Hq, Hk, D = (case[n] for n in ("B", "F", "Hg", "Wg", "Hq", "Hk", "D"))
        s["axes"] = tuple(int(x) for x in case["axes"].split(","))
        grid = torch.meshgrid(torch.arange(F, device="cuda") + case["offset"], torch.arange(Hg, device="cuda"),
                              torch.arange(Wg, device="cuda"), indexing="ij")
        pos = torch.stack(grid, dim=-1).reshape(F, Hg * Wg, 3)
        if len(s["axes"]) == 2:
            pos = pos[..., 1:]
        s["pos"] = pos.to(torch.int32).contiguous()
        s["q"], s["k"] = _randn(g, (B, F, Hg * Wg, Hq, D), dt), _randn(g, (B, F, Hg * Wg, Hk, D), dt)
        if case["train"]:
            s["dq"], s["dk"] = _randn(g, s["q"].shape, dt), _randn(g, s["k"].shape, dt)
    else:
        lq, lk = _lens(case)
        Hq, Hk, D, room = case["Hq"], case["Hk"], case["D"], case["room"]
        cu_q, cu_k = _starts(lq), _starts(lk, room)
        s["lq"], s["lk"] = lq, lk
        s["q"] = _randn(g, (cu_q[-1], Hq, D), dt)
        s["k"], s["v"] = _randn(g, (cu_k[-1], Hk, D), dt), _randn(g, (cu_k[-1], Hk, D), dt)
        s["cu_q"], s["cu_k"] = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (cu_q, cu_k))
        s["k_len"] = torch.tensor(lk, dtype=torch.int32, device="cuda")
        if case["train"]:
            s["do"] = _randn(g, (cu_q[-1], Hq, D), dt)
    return s


# ------------------------------------------------------------------ plain forms
def _norm_plain(s):
    x = s["x"].float()
    w, b = s["weight"].float(), s["bias"].float()
    mean = x.sum(-1, keepdim=True) / x.shape[-1]
    xc = x - mean
    rstd = 1.0 / torch.sqrt((xc * xc).sum(-1, keepdim=True) / x.shape[-1] + 1e-6)
    xh = xc * rstd
    out = {"y": (xh * w + b).to(s["x"].dtype)}
    if s["train"]:
        dy = s["dy"].float()
        gw = dy * w
        c1 = gw.sum(-1, keepdim=True) / x.shape[-1]
        c2 = (gw * xh).sum(-1, keepdim=True) / x.shape[-1]
        out["dx"] = ((gw - c1 - xh * c2) * rstd).to(s["x"].dtype)
        # the weight's gradients are sums over all tokens: 64 bits
        out["dweight"] = (dy * xh).sum(0, dtype=torch.float64).to(s["weight"].dtype)
        out["dbias"] = dy.sum(0, dtype=torch.float64).to(s["bias"].dtype)
    return out


def _angles(pos, axes, theta=10000.0):
    """Angles of every (token, pair) in 64 bits: pair i of an axis of d features turns by position * theta^(-2i/d)."""
    at = torch.cat([torch.full((d // 2,), a, device=pos.device) for a, d in enumerate(axes)])
    expo = torch.cat([torch.arange(d // 2, device=pos.device, dtype=torch.float64) * 2 / d for d in axes])
    return pos.double()[..., at] * torch.exp(expo * -math.log(theta))


def _turn(x, cos, sin, halves):
    """Rotates the first 2 * pairs features of x [B, F, N, H, D] in 32 bits."""
    R = 2 * cos.shape[-1]
    x32 = x.float()
    out = x32.clone()
    c, n = cos.unsqueeze(-2), sin.unsqueeze(-2)
    if halves:
        a, b = x32[..., :R // 2], x32[..., R // 2:R]
        out[..., :R // 2], out[..., R // 2:R] = a * c - b * n, a * n + b * c
    else:
        a, b = x32[..., 0:R:2], x32[..., 1:R:2]
        out[..., 0:R:2], out[..., 1:R:2] = a * c - b * n, a * n + b * c
    return out.to(x.dtype)


def _rotary_plain(s):
    ang = _angles(s["pos"], s["axes"])
    cos, sin = ang.cos().float(), ang.sin().float()
    out = {"q": _turn(s["q"], cos, sin, s["halves"]), "k": _turn(s["k"], cos, sin, s["halves"])}
    if s["train"]:
        out["dq"], out["dk"] = _turn(s["dq"], cos, -sin, s["halves"]), _turn(s["dk"], cos, -sin, s["halves"])
    return out


def _seq_of(cu, rows):
    """Sequence number of each row (n_seq for rows behind the last)."""
    return torch.bucketize(torch.arange(rows, device=cu.device, dtype=torch.int32), cu[1:], right=True)


def _visible(s):
    """[Tq, Tk]: key j of the same sequence lies in the query's block of positions or before it; the queries are the
    last positions of their sequence."""
    Tq, Tk = s["q"].shape[0], s["k"].shape[0]
    sq, sk = _seq_of(s["cu_q"], Tq), _seq_of(s["cu_k"], Tk)
    jk = torch.arange(Tk, device=sk.device) - s["cu_k"][sk].long()
    iq = torch.arange(Tq, device=sq.device) - s["cu_q"][sq].long()
    lk, lq = s["k_len"].long(), (s["cu_q"][1:] - s["cu_q"][:-1]).long()
    see = (sq[:, None] == sk[None, :]) & (jk < lk[sk])[None, :]
    if s["causal"]:
        p = iq + lk[sq] - lq[sq]
        last = torch.div(p, s["block"], rounding_mode="floor") * s["block"] + s["block"]
        see &= (jk[None, :] < last[:, None]) & (p >= 0)[:, None]
    return see


def _attn_plain(s):
    Tq, Hq, D = s["q"].shape
    Tk, Hk, _ = s["k"].shape
    G, scale = Hq // Hk, 1.0 / math.sqrt(D)
    q = s["q"].float().reshape(Tq, Hk, G, D).permute(1, 2, 0, 3).reshape(Hk, G * Tq, D)
    k, v = s["k"].float().transpose(0, 1).contiguous(), s["v"].float().transpose(0, 1).contiguous()
    see = _visible(s)
    sc = (q @ k.transpose(1, 2)).mul_(scale).reshape(Hk, G, Tq, Tk)
    sc.masked_fill_(~see, -math.inf)
    m = sc.amax(-1, keepdim=True)
    m0 = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = sc.sub_(m0).exp_()
    total = p.sum(-1, keepdim=True)
    lse = (m0 + total.log())[..., 0]
    p = p.div_(torch.where(total == 0, torch.ones_like(total), total)).reshape(Hk, G * Tq, Tk)
    o = p @ v

    def rows(x):
        return x.reshape(Hk, G, Tq, D).permute(2, 0, 1, 3).reshape(Tq, Hq, D).to(s["q"].dtype)

    out = {"o": rows(o), "lse": lse.permute(2, 0, 1).reshape(Tq, Hq).contiguous()}
    if s["train"]:
        do = s["do"].float().reshape(Tq, Hk, G, D).permute(1, 2, 0, 3).reshape(Hk, G * Tq, D)
        dp = do @ v.transpose(1, 2)
        dv = p.transpose(1, 2) @ do
        ds = dp.sub_((do * o).sum(-1, keepdim=True)).mul_(p).mul_(scale)
        out["dq"] = rows(ds @ k)
        out["dk"] = (ds.transpose(1, 2) @ q).transpose(0, 1).contiguous().to(s["k"].dtype)
        out["dv"] = dv.transpose(0, 1).contiguous().to(s["v"].dtype)
    return out


# ------------------------------------------------------------------ the library's calls
def _norm_own(s):
    from gated_deltanet_scan_amd import api
    if not s["train"]:
        return {"y": api.layer_norm_fwd(s["x"], s["weight"], s["bias"], eps=1e-6, return_stats=False)[0]}
    y, mean, rstd = api.layer_norm_fwd(s["x"], s["weight"], s["bias"], eps=1e-6)
    dx, dw, db = api.layer_norm_bwd(s["dy"], s["x"], mean, rstd, s["weight"], s["bias"])
    return {"y": y, "dx": dx, "dweight": dw, "dbias": db}


def _rotary_own(s):
    from gated_deltanet_scan_amd import api
    kw = dict(axes=s["axes"], halves=s["halves"])
    q, k = api.rotary(s["q"], s["k"], s["pos"], **kw)
    out = {"q": q, "k": k}
    if s["train"]:
        out["dq"], out["dk"] = api.rotary(s["dq"], s["dk"], s["pos"], inverse=True, **kw)
    return out


def _attn_own(s):
    from gated_deltanet_scan_amd import api
    kw = dict(causal=s["causal"], causal_block=s["block"], cu_q=s["cu_q"], cu_k=s["cu_k"], max_q=max(s["lq"]),
              max_k=max(s["lk"]))
    if not s["train"]:
        o, lse = api.attention_fwd(s["q"], s["k"], s["v"], k_len=s["k_len"], **kw)
        return {"o": o, "lse": lse}
    o, lse = api.attention_fwd(s["q"], s["k"], s["v"], **kw)
    dq, dk, dv = api.attention_bwd(s["q"], s["k"], s["v"], o, lse, s["do"], **kw)
    return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


def run(state):
    op = state["op"]
    if own:
        return {"norm": _norm_own, "rotary": _rotary_own, "attn": _attn_own}[op](state)
    return {"norm": _norm_plain, "rotary": _rotary_plain, "attn": _attn_plain}[op](state)


# ------------------------------------------------------------------ work
def _pairs(lq, lk, causal, block):
    """(query, key) pairs that the mask leaves."""
    if not causal:
        return lq * lk
    n, p = 0, lk - lq
    at = max(p, 0)
    while at < lk:  # one block of positions at a time
        end = min(lk, (at // block + 1) * block)
        n += (end - at) * end
        at = end
    return n


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "norm":
        n, C = case["rows"] * case["C"], case["C"]
        w = 2 if case["wdtype"] == "bf16" else 4
        if not case["train"]:
            return {"bytes": 2 * n * e + 2 * C * w, "flops": 8 * n}
        return {"bytes": 4 * n * e + 4 * C * w, "flops": 22 * n}
    if case["op"] == "rotary":
        tok = case["F"] * case["Hg"] * case["Wg"]
        n = case["B"] * tok * (case["Hq"] + case["Hk"]) * case["D"]
        times = 2 if case["train"] else 1
        return {"bytes": times * 2 * n * e + 12 * tok, "flops": times * 3 * n}
    lq, lk = _lens(case)
    Hq, Hk, D = case["Hq"], case["Hk"], case["D"]
    pairs = sum(_pairs(a, b, case["causal"], case["block"]) for a, b in zip(lq, lk))
    tq, tk = sum(lq), sum(lk)
    moved = tq * Hq * D * e * 2 + tq * Hq * 4 + tk * Hk * D * e * 2
    flops = 4 * pairs * Hq * D
    if case["train"]:
        moved += tq * Hq * D * e * 2 + tk * Hk * D * e * 2
        flops += 10 * pairs * Hq * D
    return {"bytes": moved, "flops": flops}


# ------------------------------------------------------------------ 64 bits
def _exact_norm(s):
    x, w, b = s["x"].double(), s["weight"].double(), s["bias"].double()
    var, mean = torch.var_mean(x, -1, unbiased=False, keepdim=True)
    inv = (var + 1e-6) ** -0.5
    h = (x - mean) * inv
    out = {"y": torch.addcmul(b, h, w)}
    if s["train"]:
        g = s["dy"].double()
        out["dweight"], out["dbias"] = (g * h).sum(0), g.sum(0)
        g = g * w
        out["dx"] = inv * (g - g.mean(-1, keepdim=True) - h * (g * h).mean(-1, keepdim=True))
    return out


def _exact_rotary(s):
    p = s["pos"].double()
    turn, col = [], 0
    for a, d in enumerate(s["axes"]):
        turn += [p[..., a] / 10000.0 ** (2.0 * i / d) for i in range(d // 2)]
    z = torch.polar(torch.ones_like(turn[0]), turn[0])
    pairs = len(turn)
    out = {}
    for name, back in (("q", False), ("k", False), ("dq", True), ("dk", True)):
        if name not in s:
            continue
        y = s[name].double().clone()
        for j in range(pairs):
            lo, hi = (j, j + pairs) if s["halves"] else (2 * j, 2 * j + 1)
            z = torch.polar(torch.ones_like(turn[j]), -turn[j] if back else turn[j])[..., None]
            w = torch.complex(y[..., lo], y[..., hi]) * z
            y[..., lo], y[..., hi] = w.real, w.imag
        out[name] = y
    return out


def _exact_attn(s):
    q, k, v = s["q"], s["k"], s["v"]
    Hq, Hk, D = q.shape[1], k.shape[1], q.shape[2]
    o = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=q.device)
    dq = torch.zeros_like(o) if s["train"] else None
    dk = torch.zeros(k.shape, dtype=torch.float64, device=q.device) if s["train"] else None
    dv = torch.zeros_like(dk) if s["train"] else None
    q0, k0 = 0, 0
    for lq, lk in zip(s["lq"], s["lk"]):
        first = lk - lq if s["causal"] else lk  # position of the first query
        at = torch.arange(lq, device=q.device) + first
        ends = ((at // s["block"] + 1) * s["block"]).clamp(max=lk) if s["causal"] else torch.full_like(at, lk)
        ends = torch.where(at < 0, torch.zeros_like(ends), ends)
        hide = torch.arange(lk, device=q.device)[None, :] >= ends[:, None]
        some = ends > 0
        for h in range(Hq):
            kk, vv = k[k0:k0 + lk, h // (Hq // Hk)].double(), v[k0:k0 + lk, h // (Hq // Hk)].double()
            for a in range(0, lq, 4096):
                z = slice(a, min(lq, a + 4096))
                sl = slice(q0 + z.start, q0 + z.stop)
                qq = q[sl, h].double()
                logit = (qq @ kk.T / D ** 0.5).masked_fill(hide[z], -math.inf)
                top = torch.logsumexp(logit, -1)
                lse[sl, h] = top
                p = torch.where(some[z, None], torch.exp(logit - top[:, None]), torch.zeros_like(logit))
                o[sl, h] = p @ vv
                if s["train"]:
                    g = s["do"][sl, h].double()
                    w = p * (g @ vv.T - (g * o[sl, h]).sum(-1, keepdim=True)) / D ** 0.5
                    dq[sl, h] = w @ kk
                    dk[k0:k0 + lk, h // (Hq // Hk)] += w.T @ qq
                    dv[k0:k0 + lk, h // (Hq // Hk)] += p.T @ g
        q0, k0 = q0 + lq, k0 + (s["room"] or lk)
    out = {"o": o, "lse": lse}
    return dict(out, dq=dq, dk=dk, dv=dv) if s["train"] else out


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "rotary": _exact_rotary, "attn": _exact_attn}[case["op"]](s)
