"""Cases for the operators that serve a hybrid block in low precision: a
root-mean-square norm with the residual's addition and an 8-bit output, the same
quantisation alone, matrix products of 8-bit floats with a scale for each block
of 128, key/value caches in MXFP8 and MXFP4 (written token by token and read
back), and softmax attention over such a cache.

``run`` computes each in plain torch operations, or, where ``own`` is true,
through the library's entry points.  The sizes are the library's workloads: a
22 x 40 = 880-token latent frame, a 21-frame clip, a 121-frame minute, 16 heads
of 128 and a model width of 2048, beside generic ragged ones.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
GROUP = 128   # columns (and weight rows) of an fp32 scale of the 8-bit products
MX = 32       # features of an E8M0 scale of the caches


def listed():
    return [
        # the norm in front of a projection, eight requests a token each (a call of a few microseconds)
        dict(name="norm_tokens", op="norm", rows=8, C=2048, residual=True, dtype="bf16", wdtype="bf16"),
        # a whole minute through a block's norm
        dict(name="norm_minute", op="norm", rows=121 * 880, C=2048, residual=True, dtype="bf16", wdtype="f32"),
        # a streamed frame's attention output on its way to the output projection
        dict(name="quant_frame", op="quant", rows=880, C=2048, dtype="bf16"),
        # fp32 activations of a width that fills neither groups nor vectors
        dict(name="quant_odd_f32", op="quant", rows=1777, C=1001, dtype="f32"),
        # query, key and value projections of seven requests, a token each
        dict(name="matmul_tokens", op="matmul", M=7, K=2048, N=6144, parts=3),
        # the output projection of a streamed frame
        dict(name="matmul_frame", op="matmul", M=880, K=2048, N=2048, parts=1),
        # query, key and value projections of a minute
        dict(name="matmul_minute", op="matmul", M=121 * 880, K=2048, N=6144, parts=3),
        # one token for each of eight requests into 4-bit caches, and the caches read back
        dict(name="cache_tokens_fp4", op="cache", lens_new="1,1,1,1,1,1,1,1", lens_k="40,511,1,1000,64,129,777,2",
             room=1024, H=8, D=128, fmt="fp4", dtype="bf16"),
        # a frame into an 8-bit cache of the frames so far, and the cache read back
        dict(name="cache_frame_fp8", op="cache", lens_new="880", lens_k="19360", room=20000, H=16, D=128, fmt="fp8",
             dtype="bf16"),
        # serving single tokens: eight requests, each one query against a 4-bit cache filled in part
        dict(name="attn_tokens_fp4", op="attn", lens_q="1,1,1,1,1,1,1,1", lens_k="40,511,1000,3777,8191,12000,30001,32768",
             room=32768, Hq=32, Hk=8, D=128, block=1, fmt="fp4"),
        # streaming: a frame's queries against the 4-bit cache of all frames so far
        dict(name="attn_frame_fp4", op="attn", lens_q="880", lens_k="19360", room=20000, Hq=16, Hk=16, D=128, block=880,
             fmt="fp4"),
        # a few queries a request against ragged 8-bit caches: an empty one, and one with fewer keys than queries
        dict(name="attn_odd_fp8", op="attn", lens_q="3,1,64,5,1", lens_k="700,0,40,2049,333", room=2100, Hq=12, Hk=4,
             D=64, block=1, fmt="fp8"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw_rows(rng):
    C = rng.choice([_log(rng, 16, 8192), 16 * _log(rng, 4, 512), 128 * rng.randint(1, 64)])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    rows = _log(rng, 1, (121 * 880 * 2048) // C // (1 if dtype == "bf16" else 2))
    rows = min(rows, 121 * 880)
    if rng.random() < 0.4:
        return dict(op="quant", rows=rows, C=C, dtype=dtype)
    return dict(op="norm", rows=rows, C=C, residual=rng.random() < 0.7, dtype=dtype,
                wdtype="f32" if dtype == "f32" else rng.choice(["bf16", "f32"]))


def _draw_matmul(rng):
    K = rng.choice([16 * _log(rng, 1, 512), 128 * rng.randint(1, 64)])
    parts = rng.choice([1, 1, 2, 3])
    N = parts * rng.choice([_log(rng, 1, 8192) if parts == 1 else 16 * _log(rng, 1, 256), 128 * rng.randint(1, 32)])
    # no more than the listed minute: its products, and its output
    most = min((121 * 880 * 2048 * 6144) // (K * N), (121 * 880 * 6144) // N)
    M = _log(rng, 1, max(1, min(121 * 880, most)))
    return dict(op="matmul", M=M, K=K, N=N, parts=parts)


def _draw_cache(rng):
    D, H, fmt = rng.choice([32, 64, 128, 128]), rng.choice([1, 2, 3, 4, 8, 16]), rng.choice(["fp4", "fp8"])
    n = _log(rng, 1, 32)
    new = [rng.choice([1, 1, _log(rng, 1, 880)])] * n if rng.random() < 0.5 else [_log(rng, 1, 400) for _ in range(n)]
    most = max(1024, 20000 * 16 * 128 // (n * H * D))
    lk = [max(a, min(most, _log(rng, 1, 20000))) for a in new]
    return dict(op="cache", lens_new=",".join(map(str, new)), lens_k=",".join(map(str, lk)),
                room=max(lk) + rng.randint(0, 100), H=H, D=D, fmt=fmt, dtype=rng.choice(["bf16", "bf16", "f32"]))


def _draw_attn(rng):
    D, Hk, fmt = rng.choice([32, 64, 128, 128]), rng.choice([1, 2, 4, 8]), rng.choice(["fp4", "fp4", "fp8"])
    Hq = Hk * rng.choice([1, 2, 4, 8])
    kind = rng.choice(["token", "token", "stream", "ragged"])
    block = 1
    if kind == "token":
        n = _log(rng, 1, 32)
        lq = [rng.choice([1, 1, 1, rng.randint(2, 5)])] * n
        most = min(32768, 268435456 // (n * Hk * D))
        lk = [max(lq[0], _log(rng, 1, most)) for _ in range(n)]
    elif kind == "stream":
        block = _log(rng, 32, 880)
        lq, lk = [block], [block * rng.randint(1, 22)]
    else:
        n = rng.randint(2, 8)
        lq = [_log(rng, 1, 400) for _ in range(n)]
        lk = [_log(rng, 1, 8000) - 1 for _ in range(n)]
    room = max(lk) + rng.randint(1, 100)
    # no more than the listed frame against its cache
    while Hq > 1 and (Hq * sum(lq) * room * len(lk) > 16 * 880 * 20000 or
                      sum(map(lambda a, b: a * b, lq, lk)) * Hq * D > 880 * 19360 * 16 * 128):
        Hq, Hk = (Hq // 2, Hk) if Hq > Hk else (Hq // 2, Hk // 2)
    return dict(op="attn", lens_q=",".join(map(str, lq)), lens_k=",".join(map(str, lk)), room=room, Hq=Hq, Hk=Hk, D=D,
                block=block, fmt=fmt)


def draw(rng):
    return rng.choice([_draw_rows, _draw_matmul, _draw_cache, _draw_attn, _draw_attn])(rng)


# ------------------------------------------------------------------ inputs
def _randn(g, shape, dtype, std=1.0, mean=0.0):
    return (torch.randn(shape, generator=g, device="cuda") * std + mean).to(dtype)


def _hidden(g, rows, C, dtype):
    """Hidden states: a channel profile shared by all tokens, plus each token's own part."""
    return (torch.randn((rows, C), generator=g, device="cuda") * 0.9 +
            0.5 * torch.randn((1, C), generator=g, device="cuda")).to(dtype)


def _ints(text):
    return [int(x) for x in text.split(",")]


def _starts(lens, room=0):
    at = [0]
    for n in lens:
        at.append(at[-1] + (room or n))
    return at


def _offsets(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _heads(case):
    return case["H"] if case["op"] == "cache" else case["Hk"]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    s = dict(case)
    op = case["op"]
    if op in ("norm", "quant"):
        rows, C, dt = case["rows"], case["C"], DTYPES[case["dtype"]]
        s["x"] = _hidden(g, rows, C, dt)
        if op == "norm":
            if case["residual"]:
                s["r"] = _hidden(g, rows, C, dt)
            s["weight"] = _randn(g, (C,), DTYPES[case["wdtype"]], 0.2, 1.0)
    elif op == "matmul":
        M, K, N = case["M"], case["K"], case["N"]
        s["x"], s["xs"] = _quant_rows(_hidden(g, M, K, torch.float32))
        s["w"], s["ws"] = _quant_weight(_randn(g, (N, K), torch.float32, K ** -0.5))
    else:
        fp4 = case["fmt"] == "fp4"
        H, D, room = _heads(case), case["D"], case["room"]
        lk = _ints(case["lens_k"])
        cu_k = _starts(lk, room)
        for name in ("k", "v"):
            s[name + "c"], s[name + "s"] = _mx_pieces(_randn(g, (cu_k[-1], H, D), torch.bfloat16), fp4)
        s["cu_k"], s["k_len"], s["max_k"] = _offsets(cu_k), _offsets(lk), max(lk)
        new = _ints(case["lens_new" if op == "cache" else "lens_q"])
        s["cu_q"], s["max_q"] = _offsets(_starts(new)), max(new)
        if op == "cache":
            dt = DTYPES[case["dtype"]]
            s["k"], s["v"] = _randn(g, (sum(new), H, D), dt), _randn(g, (sum(new), H, D), dt)
            s["ko"], s["vo"] = (torch.zeros((cu_k[-1], H, D), dtype=dt, device="cuda") for _ in range(2))
        else:
            s["q"] = _randn(g, (sum(new), case["Hq"], D), torch.bfloat16)
    return s


# ------------------------------------------------------------------ plain forms
def _groups(x):
    """x [..., C] as [..., groups, 128], zeros behind the last column."""
    C = x.shape[-1]
    n = (C + GROUP - 1) // GROUP
    if n * GROUP != C:
        x = torch.cat([x, x.new_zeros(x.shape[:-1] + (n * GROUP - C,))], -1)
    return x.reshape(x.shape[:-1] + (n, GROUP))


def _quant_rows(y):
    """Each group of 128 columns of y [rows, C] (32 bits) by its largest magnitude: (e4m3 codes, scales)."""
    g = _groups(y)
    top = g.abs().amax(-1).clamp_min(2.0 ** -100)
    codes = (g * (448.0 / top).unsqueeze(-1)).to(torch.float8_e4m3fn)
    return codes.reshape(y.shape[0], -1)[:, :y.shape[1]].contiguous(), top / 448.0


def _quant_weight(w):
    """Each 128 x 128 block of w [N, K]: (e4m3 codes, scales [N / 128, K / 128])."""
    N = w.shape[0]
    n = (N + GROUP - 1) // GROUP
    g = _groups(torch.cat([w, w.new_zeros((n * GROUP - N, w.shape[1]))]))
    g = g.reshape(n, GROUP, g.shape[1], GROUP)
    top = g.abs().amax((1, 3)).clamp_min(2.0 ** -100)
    codes = (g * (448.0 / top)[:, None, :, None]).to(torch.float8_e4m3fn)
    return codes.reshape(n * GROUP, -1)[:N, :w.shape[1]].contiguous(), top / 448.0


def _norm_plain(s):
    t = s["x"].float()
    out = {}
    if s["op"] == "norm":
        if s["residual"]:
            t = t + s["r"].float()
            out["sum"] = t.to(s["x"].dtype)
        inv = 1.0 / torch.sqrt((t * t).sum(-1, keepdim=True) / t.shape[-1] + 1e-6)
        t = t * inv * s["weight"].float()
    out["y"], out["scale"] = _quant_rows(t)
    return out


def _matmul_plain(s):
    K, N = s["K"], s["N"]
    x = (s["x"].float() * s["xs"].repeat_interleave(GROUP, 1)[:, :K])
    w = s["w"].float() * s["ws"].repeat_interleave(GROUP, 0)[:N].repeat_interleave(GROUP, 1)[:, :K]
    y = (x @ w.t()).to(torch.bfloat16)
    if s["parts"] > 1:
        y = y.reshape(s["M"], s["parts"], N // s["parts"]).transpose(0, 1).contiguous()
    return {"y": y}


def _mx_encode(x, fp4):
    """x [T, H, D] in blocks of 32 features: (codes, scale bytes e + 127), the largest magnitude m of a block giving
    e = floor(log2 m) less the format's largest exponent."""
    b = x.float().reshape(x.shape[:-1] + (x.shape[-1] // MX, MX))
    top = b.abs().amax(-1)
    e = torch.where(top > 0, torch.frexp(top)[1] - 1 - (2 if fp4 else 8), torch.zeros_like(top, dtype=torch.int32))
    e = e.clamp(-127, 127)
    y = b / torch.exp2(e.float()).unsqueeze(-1)
    if not fp4:
        codes = y.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).reshape(x.shape)
    else:
        a = y.abs()
        # magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6: the midpoints passed, ties to the even code
        m = ((a > 0.25).byte() + (a >= 0.75).byte() + (a > 1.25).byte() + (a >= 1.75).byte() + (a > 2.5).byte() +
             (a >= 3.5).byte() + (a > 5.0).byte())
        m = (m + ((y < 0) & (m > 0)).byte() * 8).reshape(x.shape)
        codes = m[..., 0::2] + m[..., 1::2] * 16
    return codes, (e + 127).byte()


def _mx_pieces(x, fp4):
    """_mx_encode in pieces, for large caches."""
    got = [_mx_encode(p, fp4) for p in x.split(1 << 15)]
    return torch.cat([c.view(torch.uint8) for c, _ in got]).view(got[0][0].dtype), torch.cat([e for _, e in got])


def _mx_decode(codes, scale, fp4):
    """The values that the codes stand for, in 32 bits."""
    if fp4:
        table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0],
                             device=codes.device)
        pair = torch.stack((codes & 15, codes >> 4), -1).reshape(codes.shape[:-1] + (-1,))
        x = table[pair.int()]
    else:
        x = codes.float()
    b = x.reshape(x.shape[:-1] + (x.shape[-1] // MX, MX))
    return (b * torch.exp2(scale.float() - 127.0).unsqueeze(-1)).reshape(x.shape)


def _seq_of(cu, rows):
    """Sequence number of each row."""
    return torch.bucketize(torch.arange(rows, device=cu.device, dtype=torch.int32), cu[1:], right=True)


def _cache_plain(s):
    fp4, new, room = s["fmt"] == "fp4", s["k"].shape[0], s["kc"].shape[0]
    sq = _seq_of(s["cu_q"], new)
    i = torch.arange(new, device=sq.device) - s["cu_q"][sq]
    # the new tokens are the last of their sequence
    at = s["cu_k"][sq].long() + s["k_len"][sq] - (s["cu_q"][1:] - s["cu_q"][:-1])[sq] + i
    sk = _seq_of(s["cu_k"], room)
    used = (torch.arange(room, device=sk.device) - s["cu_k"][sk] < s["k_len"][sk])[:, None, None]
    out = {}
    for n in ("k", "v"):
        codes, scale = _mx_encode(s[n], fp4)
        s[n + "c"].view(torch.uint8)[at] = codes.view(torch.uint8)
        s[n + "s"][at] = scale
        s[n + "o"].copy_(torch.where(used, _mx_decode(s[n + "c"], s[n + "s"], fp4).to(s[n + "o"].dtype), s[n + "o"]))
        out[n] = s[n + "o"]
    return out


def _visible(s):
    """[Tq, Tk]: key j of the same sequence lies in the query's block of positions or before it; the queries are the
    last positions of their sequence."""
    Tq, Tk = s["q"].shape[0], s["kc"].shape[0]
    sq, sk = _seq_of(s["cu_q"], Tq), _seq_of(s["cu_k"], Tk)
    jk = torch.arange(Tk, device=sk.device) - s["cu_k"][sk].long()
    iq = torch.arange(Tq, device=sq.device) - s["cu_q"][sq].long()
    lk, lq = s["k_len"].long(), (s["cu_q"][1:] - s["cu_q"][:-1]).long()
    p = iq + lk[sq] - lq[sq]
    last = torch.div(p, s["block"], rounding_mode="floor") * s["block"] + s["block"]
    see = (sq[:, None] == sk[None, :]) & (jk < lk[sk])[None, :]
    return see & (jk[None, :] < last[:, None]) & (p >= 0)[:, None]


def _attn_plain(s):
    Tq, Hq, D = s["q"].shape
    Tk, Hk = s["kc"].shape[:2]
    G, fp4 = Hq // Hk, s["fmt"] == "fp4"
    q = s["q"].float().reshape(Tq, Hk, G, D).permute(1, 2, 0, 3).reshape(Hk, G * Tq, D)
    k, v = (_mx_decode(s[n + "c"], s[n + "s"], fp4).transpose(0, 1).contiguous() for n in ("k", "v"))
    see = _visible(s)
    sc = (q @ k.transpose(1, 2)).mul_(1.0 / math.sqrt(D)).reshape(Hk, G, Tq, Tk)
    sc.masked_fill_(~see, -math.inf)
    m = sc.amax(-1, keepdim=True)
    m0 = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = sc.sub_(m0).exp_()
    total = p.sum(-1, keepdim=True)
    lse = (m0 + total.log())[..., 0]
    p = p.div_(torch.where(total == 0, torch.ones_like(total), total)).reshape(Hk, G * Tq, Tk)
    o = (p @ v).reshape(Hk, G, Tq, D).permute(2, 0, 1, 3).reshape(Tq, Hq, D)
    return {"o": o.to(s["q"].dtype), "lse": lse.permute(2, 0, 1).reshape(Tq, Hq).contiguous()}


# ------------------------------------------------------------------ the library's calls
def _norm_own(s):
    from gated_deltanet_scan_amd import api
    if s["op"] == "quant":
        y, scale = api.quantize_fp8(s["x"])
        return {"y": y, "scale": scale}
    y, scale, total = api.rms_norm_fwd_fp8(s["x"], s["weight"], s["r"] if s["residual"] else None, eps=1e-6)
    return {"y": y, "scale": scale, "sum": total} if s["residual"] else {"y": y, "scale": scale}


def _matmul_own(s):
    from gated_deltanet_scan_amd import api
    return {"y": api.matmul_fp8(s["x"], s["xs"], s["w"], s["ws"], parts=s["parts"])}


def _cache_own(s):
    from gated_deltanet_scan_amd import api
    cache = s["kc"], s["ks"], s["vc"], s["vs"]
    api.cache_write(s["k"], s["v"], *cache, k_len=s["k_len"], cu_new=s["cu_q"], cu_k=s["cu_k"], max_new=s["max_q"],
                    max_k=s["max_k"])
    k, v = api.cache_read(*cache, k_len=s["k_len"], cu_k=s["cu_k"], max_k=s["max_k"], k=s["ko"], v=s["vo"])
    return {"k": k, "v": v}


def _attn_own(s):
    from gated_deltanet_scan_amd import api
    fwd = api.attention_fwd_fp4 if s["fmt"] == "fp4" else api.attention_fwd_fp8
    o, lse = fwd(s["q"], s["kc"], s["ks"], s["vc"], s["vs"], causal=True, causal_block=s["block"], cu_q=s["cu_q"],
                 cu_k=s["cu_k"], max_q=s["max_q"], max_k=s["max_k"], k_len=s["k_len"])
    return {"o": o, "lse": lse}


def run(state):
    op = state["op"]
    if own:
        return {"norm": _norm_own, "quant": _norm_own, "matmul": _matmul_own, "cache": _cache_own,
                "attn": _attn_own}[op](state)
    return {"norm": _norm_plain, "quant": _norm_plain, "matmul": _matmul_plain, "cache": _cache_plain,
            "attn": _attn_plain}[op](state)


# ------------------------------------------------------------------ work
def _pairs(lq, lk, block):
    """(query, key) pairs that the mask leaves."""
    n, p = 0, lk - lq
    at = max(p, 0)
    while at < lk:  # one block of positions at a time
        end = min(lk, (at // block + 1) * block)
        n += (end - at) * end
        at = end
    return n


def work(case):
    op = case["op"]
    e = 4 if case.get("dtype") == "f32" else 2
    if op in ("norm", "quant"):
        n, rows, C = case["rows"] * case["C"], case["rows"], case["C"]
        out = n + 4 * rows * ((C + GROUP - 1) // GROUP)
        if op == "quant":
            return {"bytes": n * e + out, "flops": 3 * n}
        extra = 2 * n * e if case["residual"] else 0
        return {"bytes": n * e + extra + out + C * (4 if case["wdtype"] == "f32" else 2), "flops": 8 * n}
    if op == "matmul":
        M, K, N = case["M"], case["K"], case["N"]
        kb, nb = (K + GROUP - 1) // GROUP, (N + GROUP - 1) // GROUP
        return {"bytes": M * K + N * K + 4 * kb * (M + nb) + M * N * 2, "flops": 2 * M * N * K}
    H, D = _heads(case), case["D"]
    token = H * (D // (2 if case["fmt"] == "fp4" else 1) + D // MX)       # bytes of a token's codes and scales
    lk = _ints(case["lens_k"])
    if op == "cache":
        new = sum(_ints(case["lens_new"]))
        return {"bytes": 2 * (new * (H * D * e + token) + sum(lk) * (H * D * e + token)), "flops": 4 * H * D * (new + sum(lk))}
    lq, Hq = _ints(case["lens_q"]), case["Hq"]
    pairs = sum(_pairs(a, b, case["block"]) for a, b in zip(lq, lk))
    return {"bytes": sum(lq) * Hq * (D * 4 + 4) + 2 * sum(lk) * token, "flops": 4 * pairs * Hq * D}


# ------------------------------------------------------------------ 64 bits
def _nearest(v, bits, low, top):
    """v rounded to `bits` fraction bits (ties to even) from 2^low on, with that value's step below it, at most top."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** low))) - bits)
    return (torch.round(v / step) * step).clamp(-top, top)


def _exact_rows(s):
    t = s["x"].double()
    out = {}
    if s["op"] == "norm":
        if s["residual"]:
            t = t + s["r"].double()
            out["sum"] = t
        t = t * (t.square().mean(-1, keepdim=True) + 1e-6) ** -0.5 * s["weight"].double()
    rows, C = t.shape
    scale = torch.empty((rows, -(-C // GROUP)), dtype=torch.float64, device=t.device)
    y = torch.empty_like(t)
    for j in range(scale.shape[1]):
        part = t[:, GROUP * j:GROUP * (j + 1)]
        scale[:, j] = part.abs().amax(-1) / 448.0
        y[:, GROUP * j:GROUP * (j + 1)] = _nearest(part / scale[:, j:j + 1], 3, -6, 448.0)
    return dict(out, y=y, scale=scale)


def _exact_matmul(s):
    M, K, N, parts = s["M"], s["K"], s["N"], s["parts"]
    y = torch.zeros((M, N), dtype=torch.float64, device=s["x"].device)
    for n in range(0, N, GROUP):
        for k in range(0, K, GROUP):
            w = s["w"][n:n + GROUP, k:k + GROUP].double() * s["ws"][n // GROUP, k // GROUP].double()
            y[:, n:n + GROUP] += (s["x"][:, k:k + GROUP].double() * s["xs"][:, k // GROUP, None].double()) @ w.T
    if parts > 1:
        y = torch.stack(y.chunk(parts, -1))
    return {"y": y}


def _exact_values(codes, scale, fp4):
    """What a cache's codes stand for: sign, exponent and fraction bits."""
    if fp4:
        c = torch.stack((codes % 16, codes // 16), -1).flatten(-2).long()
        mag, exp, frac = c % 8, (c % 8) // 2, c % 2
        x = torch.where(exp > 0, (2 + frac).double() * 2.0 ** (exp - 2).double(), mag.double() / 2)
        x = torch.where(c >= 8, -x, x)
    else:
        c = codes.view(torch.uint8).long()
        exp, frac = (c // 8) % 16, c % 8
        x = torch.where(exp > 0, (8 + frac).double() * 2.0 ** (exp - 10).double(), frac.double() * 2.0 ** -9)
        x = torch.where(c >= 128, -x, x)
    return x * (2.0 ** (scale.double() - 127)).repeat_interleave(MX, -1)


def _exact_cache(s):
    fp4 = s["fmt"] == "fp4"
    new, lk, room = _ints(s["lens_new"]), _ints(s["lens_k"]), s["room"]
    out = {}
    for n in ("k", "v"):
        old = _exact_values(s[n + "c"], s[n + "s"], fp4)
        got = torch.zeros_like(old)
        q0 = 0
        for i, (a, b) in enumerate(zip(new, lk)):
            got[i * room:i * room + b] = old[i * room:i * room + b]
            x = s[n][q0:q0 + a].double().unflatten(-1, (-1, MX))
            unit = torch.exp2(torch.floor(torch.log2(x.abs().amax(-1, keepdim=True))) - (2 if fp4 else 8))
            x = _nearest(x / unit, 1 if fp4 else 3, 0 if fp4 else -6, 6.0 if fp4 else 448.0) * unit
            got[i * room + b - a:i * room + b] = x.flatten(-2)
            q0 += a
        out[n] = got
    return out


def _exact_attn(s):
    q = s["q"]
    Hq, D, G = q.shape[1], q.shape[2], q.shape[1] // s["kc"].shape[1]
    o = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=q.device)
    q0, k0 = 0, 0
    for lq, lk in zip(_ints(s["lens_q"]), _ints(s["lens_k"])):
        at = torch.arange(lq, device=q.device) + (lk - lq)
        ends = ((at // s["block"] + 1) * s["block"]).clamp(max=lk)
        rows = (at >= 0).nonzero()[:, 0]
        k, v = (_exact_values(s[n + "c"][k0:k0 + lk], s[n + "s"][k0:k0 + lk], s["fmt"] == "fp4") for n in ("k", "v"))
        for h in range(Hq if len(rows) else 0):
            logit = q[q0 + rows, h].double() @ k[:, h // G].T / D ** 0.5
            hide = torch.arange(lk, device=q.device)[None, :] >= ends[rows, None]
            logit = logit.masked_fill(hide, -math.inf)
            top = torch.logsumexp(logit, -1)
            lse[q0 + rows, h] = top
            o[q0 + rows, h] = torch.exp(logit - top[:, None]) @ v[:, h // G]
        q0, k0 = q0 + lq, k0 + s["room"]
    return {"o": o, "lse": lse}


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_rows, "quant": _exact_rows, "matmul": _exact_matmul, "cache": _exact_cache,
            "attn": _exact_attn}[case["op"]](s)
