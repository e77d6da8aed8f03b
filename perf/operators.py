"""Cases for timing the operators around the attention of a transformer block: root-mean-square
norm with the residual's addition, rotary positions with the norm of queries and keys, and
attention with capped scores, a distance bias and causal, prefix and document masks.

`run` computes an operator in plain torch arithmetic (fp32, angles in 64 bits), or, where
`own` is true, through the library's calls.  `exact` states each operator once more in 64 bits.
Shapes follow this repository's workloads: heads 24 x 64 (sd3_1024, S = 4429), 24 x 128
(flux, S = 4608 and 16896), 40 x 128 (video, S = 32760), text of 333 and 512 tokens.
"""

import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------------------- the cases

def listed():
    return [
        # one token of a wide block: the norm between two layers of a step that generates
        # frames or tokens one at a time; latency is all that counts
        dict(name="norm_token", op="norm", rows=1, C=5120, dtype="bf16", residual=True, out="bf16", group=0),
        # text tokens of an odd width with an fp32 residual stream and no addition
        dict(name="norm_odd_fp32", op="norm", rows=333, C=1001, dtype="fp32", residual=False, out="bf16", group=0),
        # the video block's tokens ahead of an FP8 layer, one scale per 128 columns
        dict(name="norm_video_e4m3", op="norm", rows=32760, C=5120, dtype="bf16", residual=True, out="e4m3", group=128),
        # one new token per sequence, half layout on half of the head, long-context frequencies
        dict(name="rope_token", op="rope", B=8, S=1, H=24, H_kv=24, D=128, rot=64, axes=1, interleaved=False,
             norm=False, out="bf16", packed=False, far=1000000, scaling="by_parts"),
        # two stacked batches (guidance) of image and text tokens, E4M3 blocks for FP8 attention
        dict(name="rope_flux_e4m3", op="rope", B=2, S=4429, H=24, H_kv=24, D=128, rot=128, axes=2, interleaved=True,
             norm=True, out="e4m3", packed=True, far=0, scaling="none"),
        # the video block: (t, y, x) positions, normed queries and keys read out of packed QKV
        dict(name="rope_video", op="rope", B=1, S=32760, H=40, H_kv=40, D=128, rot=128, axes=3, interleaved=True,
             norm=True, out="bf16", packed=True, far=0, scaling="none"),
        # self-attention of one short prompt: the smallest call
        dict(name="attn_text", op="attn", B=1, H=24, H_kv=24, S_q=77, S_kv=77, D=64, cap=0.0, bias=False, causal=True,
             prefix=0, docs=0, pad=0, lens=False),
        # one new token per sequence against caches of different lengths, shared heads
        dict(name="attn_token_cache", op="attn", B=4, H=40, H_kv=8, S_q=1, S_kv=32760, D=128, cap=0.0, bias=False,
             causal=True, prefix=0, docs=0, pad=0, lens=True),
        # images of several sizes and their padding packed into one sequence, two batches
        dict(name="attn_docs", op="attn", B=2, H=24, H_kv=24, S_q=4429, S_kv=4429, D=64, cap=0.0, bias=False,
             causal=False, prefix=0, docs=7, pad=77, lens=False),
        # image and text tokens with capped scores and no mask
        dict(name="attn_cap", op="attn", B=1, H=24, H_kv=24, S_q=4608, S_kv=4608, D=128, cap=30.0, bias=False,
             causal=False, prefix=0, docs=0, pad=0, lens=False),
        # causal generation with a distance bias and shared heads
        dict(name="attn_bias", op="attn", B=1, H=24, H_kv=6, S_q=4608, S_kv=4608, D=128, cap=0.0, bias=True,
             causal=True, prefix=0, docs=0, pad=0, lens=False),
        # a long sequence generated after a fully visible text prefix
        dict(name="attn_prefix", op="attn", B=1, H=8, H_kv=4, S_q=16896, S_kv=16896, D=128, cap=0.0, bias=False,
             causal=True, prefix=512, docs=0, pad=0, lens=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw_once(rng):
    op = rng.choice(["norm", "rope", "attn"])
    if op == "norm":
        out = rng.choice(["bf16", "fp32", "e4m3", "e4m3"])
        return dict(op=op, rows=_log_int(rng, 1, 32760), C=_log_int(rng, 64, 8192) if rng.random() < 0.4
                    else 8 * _log_int(rng, 8, 1024), dtype=rng.choice(["bf16", "bf16", "fp32"]),
                    residual=rng.random() < 0.7, out=out, group=rng.choice([0, 128]) if out == "e4m3" else 0)
    if op == "rope":
        D = rng.choice([64, 128])
        H_kv = rng.choice([1, 2, 6, 8, 24])
        return dict(op=op, B=rng.choice([1, 2, 3, 8]), S=_log_int(rng, 1, 16896), H=H_kv * rng.choice([1, 2, 4]),
                    H_kv=H_kv, D=D, rot=rng.choice([D, D, D // 2, 48]), axes=rng.choice([1, 1, 2, 3]),
                    interleaved=rng.random() < 0.5, norm=rng.random() < 0.5, out=rng.choice(["bf16", "bf16", "e4m3"]),
                    packed=rng.random() < 0.5, far=rng.choice([0, 100000, 1000000]),
                    scaling=rng.choice(["none", "linear", "ntk", "by_parts"]))
    form = rng.choice(["token", "few", "self", "self"])
    S_kv = _log_int(rng, 512 if form == "token" else 1, 32760 if form == "token" else 8192)
    S_q = 1 if form == "token" else (_log_int(rng, 2, 64) if form == "few" else S_kv)
    H_kv = rng.choice([1, 2, 4, 8, 24] if form != "self" else [1, 2, 6])
    causal = form == "token" or rng.random() < 0.6
    docs = rng.choice([0, 0, 2, 9]) if form == "self" else 0
    return dict(op=op, B=rng.choice([1, 2, 3]), H=H_kv * rng.choice([1, 2, 4, 5]), H_kv=H_kv, S_q=S_q, S_kv=S_kv,
                D=rng.choice([64, 128]), cap=rng.choice([0.0, 0.0, 15.0, 50.0]), bias=rng.random() < 0.3, causal=causal,
                prefix=rng.choice([0, max(1, S_kv // 7)]) if causal and form == "self" else 0, docs=docs,
                pad=rng.choice([0, S_kv // 9]) if docs else 0, lens=form != "self" and causal and rng.random() < 0.7)


def draw(rng):
    # no more work than the largest listed case of its operator
    most = {}
    for c in listed():
        w = work(c)
        m = most.setdefault(c["op"], {"bytes": 0, "flops": 0})
        for k in m:
            m[k] = max(m[k], w[k])
    while True:
        c = _draw_once(rng)
        w = work(c)
        scores = c["B"] * c["H"] * c["S_q"] * c["S_kv"] if c["op"] == "attn" else 0   # the plain form holds them
        if w["bytes"] <= most[c["op"]]["bytes"] and w["flops"] <= most[c["op"]]["flops"] and scores < 2.5e9:
            return c


# ----------------------------------------------------------------- what a case's inputs look like

def _doc_ids(case):
    """Document of each key: `docs` runs of ragged lengths, then `pad` keys of none (-1)."""
    S, n = case["S_kv"], case["docs"]
    ids = np.full(S, -1, np.int32)
    w = np.array([1 + (i * 7) % 5 for i in range(n)], np.float64)
    ends = np.floor(np.cumsum(w) / w.sum() * (S - case["pad"])).astype(np.int64)
    ids[:ends[-1]] = np.searchsorted(ends, np.arange(ends[-1]), side="right")
    return ids


def _starts(case):
    """Position of the first query in each sequence: caches of different lengths."""
    last = case["S_kv"] - case["S_q"]
    if not case["lens"]:
        return [last] * case["B"]
    return [max(0, last - (b * 997) % (last // 4 + 1)) for b in range(case["B"])]


def _pairs(case):
    """(query, key) pairs that the masks leave, and keys that any query sees, over the batches."""
    S_kv, pairs, seen = case["S_kv"], 0, 0
    i = np.arange(case["S_q"], dtype=np.int64)
    for start in _starts(case):
        lim = np.minimum(np.maximum(start + i + 1, case["prefix"]), S_kv) if case["causal"] else np.full_like(i, S_kv)
        lim = np.maximum(lim, 0)
        if case["docs"]:
            ids = _doc_ids(case)
            on = ids >= 0
            first = np.searchsorted(np.where(on, ids, 1 << 30), ids, side="left")
            end = np.searchsorted(np.where(on, ids, 1 << 30), ids, side="right")
            pairs += int(np.where(on, np.maximum(np.minimum(end, lim) - first, 0), 0).sum())
            seen += int(on.sum())
        else:
            pairs += int(lim.sum())
            seen += int(lim.max())
    return pairs, seen


def work(case):
    if case["op"] == "norm":
        n, e = case["rows"] * case["C"], 2 if case["dtype"] == "bf16" else 4
        out = {"bf16": 2, "fp32": 4, "e4m3": 1}[case["out"]]
        groups = 0 if case["out"] != "e4m3" else (1 if not case["group"] else -(-case["C"] // case["group"]))
        return {"bytes": n * (e * (3 if case["residual"] else 1) + out) + case["C"] * e + case["rows"] * groups * 4,
                "flops": n * 5}
    if case["op"] == "rope":
        n = case["B"] * case["S"] * (case["H"] + case["H_kv"]) * case["D"]
        return {"bytes": n * (2 + (2 if case["out"] == "bf16" else 1)) + case["B"] * case["S"] * case["axes"] * 4,
                "flops": n * (7 if case["norm"] else 3)}
    pairs, seen = _pairs(case)
    rows = case["B"] * case["H"] * case["S_q"]
    return {"bytes": rows * (case["D"] * 4 + 4)
            + 4 * seen * case["H_kv"] * case["D"], "flops": 4 * pairs * case["H"] * case["D"]}


def _freqs(case):
    """Radians per position of each rotated pair, theta = 10000, stretched 8-fold from 8192 positions."""
    rot = case["rot"]
    pairs = rot // 2
    per = _axis_pairs(case)
    i = np.concatenate([np.arange(p) / p for p in per])
    f = 10000.0 ** -i
    if case["scaling"] == "linear":
        f = f / 8.0
    elif case["scaling"] == "ntk":
        f = (10000.0 * 8.0 ** (rot / (rot - 2))) ** -i
    elif case["scaling"] == "by_parts":
        turns = 8192 * f / (2 * math.pi)                 # whole turns within the original length
        keep = np.clip((turns - 1.0) / (32.0 - 1.0), 0.0, 1.0)
        f = f * keep + f / 8.0 * (1.0 - keep)
    assert f.shape == (pairs,)
    return f


def _axis_pairs(case):
    pairs, n = case["rot"] // 2, case["axes"]
    rest = [pairs * 3 // 8] * (n - 1)
    return [pairs - sum(rest)] + rest


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed * 7919 + 13)

    def normal(*shape, dtype=torch.bfloat16, scale=1.0):
        return (torch.randn(*shape, generator=g, device=DEV) * scale).to(dtype)

    st = dict(case)
    if case["op"] == "norm":
        t = TYPES[case["dtype"]]
        # a residual stream: channels of different loudness, as after many layers
        loud = torch.exp(torch.randn(case["C"], generator=g, device=DEV) * 0.7)
        st["x"] = (normal(case["rows"], case["C"], dtype=torch.float32) * loud).to(t)
        st["r"] = (normal(case["rows"], case["C"], dtype=torch.float32, scale=2.0) * loud).to(t) if case["residual"] else None
        st["w"] = (1.0 + 0.2 * torch.randn(case["C"], generator=g, device=DEV)).to(t)
        return st
    if case["op"] == "rope":
        B, S, H, Hk, D = (case[k] for k in ("B", "S", "H", "H_kv", "D"))
        if case["packed"]:                       # one projection's output: [B, S, heads of q | k | v, D]
            qkv = normal(B, S, H + 2 * Hk, D)
            st["q"], st["k"] = qkv[:, :, :H], qkv[:, :, H:H + Hk]
        else:
            st["q"], st["k"] = normal(B, S, H, D), normal(B, S, Hk, D)
        st["wq"] = (1.0 + 0.2 * torch.randn(D, generator=g, device=DEV)).to(torch.bfloat16) if case["norm"] else None
        st["wk"] = (1.0 + 0.2 * torch.randn(D, generator=g, device=DEV)).to(torch.bfloat16) if case["norm"] else None
        s = torch.arange(S, device=DEV)
        if case["axes"] == 1:
            pos = s[None, :, None].expand(B, S, 1)
        else:                                    # a grid of tokens in rows of 52, 30 rows a frame
            pos = torch.stack([s // 1560, s // 52 % 30, s % 52][-case["axes"]:], -1)[None].expand(B, S, case["axes"])
        far = torch.randint(0, case["far"] + 1, (B, 1, 1), generator=g, device=DEV)
        st["pos"] = (pos + far).to(torch.int32).contiguous()
        st["freqs"] = torch.from_numpy(_freqs(case)).to(DEV)
        st["mag"] = 0.1 * math.log(8.0) + 1.0 if case["scaling"] == "by_parts" else 1.0
        st["axis_pairs"] = _axis_pairs(case)
        st["axis"] = torch.repeat_interleave(torch.arange(case["axes"]), torch.tensor(st["axis_pairs"])).to(DEV)
        return st
    B, H, Hk, D = (case[k] for k in ("B", "H", "H_kv", "D"))
    # capped scores are worth capping: queries louder than the normed ones
    st["q"] = normal(B, H, case["S_q"], D, scale=3.0 if case["cap"] else 1.0)
    st["k"] = normal(B, Hk, case["S_kv"], D)
    st["v"] = normal(B, Hk, case["S_kv"], D)
    st["scale"] = 1.0 / math.sqrt(D)
    st["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)], device=DEV) if case["bias"] else None
    st["start"] = torch.tensor(_starts(case), dtype=torch.int32, device=DEV) if case["lens"] else None
    st["prefix"] = torch.full((B,), case["prefix"], dtype=torch.int32, device=DEV) if case["prefix"] else None
    st["docs"] = torch.from_numpy(_doc_ids(case)).to(DEV)[None].repeat(B, 1) if case["docs"] else None
    return st


# ------------------------------------------------------------------------------- one pass

def run(st):
    if own:
        return _run_own(st)
    return {"norm": _norm, "rope": _rope, "attn": _attn}[st["op"]](st)


def _run_own(st):
    import long_sequence_attention_b200 as lsa
    code = {"bf16": torch.bfloat16, "fp32": torch.float32, "e4m3": torch.uint8}.get(st.get("out"))
    if st["op"] == "norm":
        y, h, d = lsa.rms_norm(st["x"], st["w"], residual=st["r"], eps=1e-6, out_dtype=code, group=st["group"])
        return (y if d is None else y.view(torch.float8_e4m3fn)), h, d
    if st["op"] == "rope":
        q, k, dq, dk = lsa.rope_qk(st["q"], st["k"], st["pos"], st["freqs"], q_weight=st["wq"], k_weight=st["wk"],
                                   eps=1e-6, axis_pairs=st["axis_pairs"], interleaved=st["interleaved"],
                                   magnitude=st["mag"], out_dtype=code)
        return (q, k) if dq is None else (q.view(torch.float8_e4m3fn), k.view(torch.float8_e4m3fn), dq, dk)
    return lsa.masked_attention(st["q"], st["k"], st["v"], scale=st["scale"], softcap=st["cap"], slopes=st["slopes"],
                                causal=st["causal"], q_start=st["start"], prefix=st["prefix"], q_doc=st["docs"],
                                kv_doc=st["docs"])


def _e4m3(y, amax, empty):
    """Codes of y and their scale amax / 448 (`empty` where there is nothing but zeros)."""
    d = torch.where(amax > 0, amax / 448.0, torch.full_like(amax, empty))
    return (y / torch.where(d > 0, d, torch.ones_like(d))).clamp(-448.0, 448.0).to(torch.float8_e4m3fn), d


def _norm(st):
    h = st["x"].float()
    if st["r"] is not None:
        h = h + st["r"].float()
    y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + 1e-6) * st["w"].float()
    stream = h.to(st["x"].dtype) if st["r"] is not None else None
    if st["out"] != "e4m3":
        return y.to(TYPES[st["out"]]), stream, None
    rows, C = y.shape
    g = st["group"] or C
    n = -(-C // g)
    z = torch.nn.functional.pad(y, (0, n * g - C)).view(rows, n, g)
    q, d = _e4m3(z, z.abs().amax(-1, keepdim=True), 1.0)
    return q.view(rows, n * g)[:, :C].contiguous(), stream, d.view(rows, n)


def _rope(st):
    angle = st["pos"].double()[..., st["axis"]] * st["freqs"]                 # [B, S, pairs]
    cos = (torch.cos(angle) * st["mag"]).float()[:, None]
    sin = (torch.sin(angle) * st["mag"]).float()[:, None]

    def one(x, w):
        x = x.float().transpose(1, 2)                                        # [B, H, S, D]
        if w is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w.float()
        r, rest = x[..., :st["rot"]], x[..., st["rot"]:]
        if st["interleaved"]:
            a, b = r[..., 0::2], r[..., 1::2]
            r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = r.chunk(2, -1)
            r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        y = torch.cat([r, rest], -1)
        if st["out"] != "e4m3":
            return y.to(TYPES[st["out"]]), None
        B, H, S, D = y.shape
        n = -(-S // 128)
        z = torch.nn.functional.pad(y, (0, 0, 0, n * 128 - S)).view(B, H, n, 128, D)
        c, d = _e4m3(z, z.abs().amax((-1, -2), keepdim=True), 0.0)
        return c.view(B, H, n * 128, D)[:, :, :S].contiguous(), d.view(B, H, n)

    (q, dq), (k, dk) = one(st["q"], st["wq"]), one(st["k"], st["wk"])
    return (q, k) if dq is None else (q, k, dq, dk)


def _allowed(st):
    """[B, 1, S_q, S_kv] (or None): which keys each query attends to, and the queries' positions [B, S_q]."""
    B, S_q, S_kv = st["B"], st["S_q"], st["S_kv"]
    start = st["start"] if st["start"] is not None else torch.full((B,), S_kv - S_q, device=DEV, dtype=torch.int32)
    pos = start[:, None] + torch.arange(S_q, device=DEV)
    j = torch.arange(S_kv, device=DEV)
    ok = None
    if st["causal"]:
        ok = j <= pos[:, :, None]
        if st["prefix"] is not None:
            ok = ok | (j < st["prefix"][:, None, None])
    if st["docs"] is not None:
        same = (st["docs"][:, :, None] == st["docs"][:, None, :]) & (st["docs"] >= 0)[:, :, None]
        ok = same if ok is None else ok & same
    return (None if ok is None else ok[:, None]), pos


def _attn(st):
    G = st["H"] // st["H_kv"]
    k = st["k"].float().repeat_interleave(G, 1)
    v = st["v"].float().repeat_interleave(G, 1)
    s = torch.matmul(st["q"].float(), k.transpose(-1, -2)).mul_(st["scale"])
    if st["cap"]:
        s = s.div_(st["cap"]).tanh_().mul_(st["cap"])
    ok, pos = _allowed(st)
    if st["slopes"] is not None:
        far = (pos[:, None, :, None] - torch.arange(st["S_kv"], device=DEV)).abs().float()
        s = s - st["slopes"][:, None, None] * far
    if ok is not None:
        s = s.masked_fill_(~ok, -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    p = s.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v) / torch.where(l > 0, l, torch.ones_like(l))
    return out.to(torch.bfloat16), (m + torch.log(l)).squeeze(-1)


# ------------------------------------------------------------------------ the same in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    return {"norm": _exact_norm, "rope": _exact_rope, "attn": _exact_attn}[case["op"]](st)


def _grid_e4m3(x):
    """x on E4M3's grid, to the nearest, ties to even: 3 bits after the leading one, least exponent -6."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))).clamp(-6, 8)
    ulp = torch.exp2(e - 3)
    return (torch.round(x / ulp) * ulp).clamp(-448.0, 448.0)


def _exact_norm(st):
    x, w = st["x"].double(), st["w"].double()
    if st["r"] is not None:
        x = x + st["r"].double()
    y = x / torch.sqrt(x.square().sum(1, keepdim=True) / x.shape[1] + 1e-6) * w
    h = x if st["r"] is not None else None
    if st["out"] != "e4m3":
        return y, h, None
    out, ds = torch.empty_like(y), []
    g = st["group"] or st["C"]
    for c in range(0, st["C"], g):
        part = y[:, c:c + g]
        d = part.abs().max(1, keepdim=True).values / 448.0
        d[d == 0] = 1.0
        out[:, c:c + g] = _grid_e4m3(part / d)
        ds.append(d)
    return out, h, torch.cat(ds, 1)


def _exact_rope(st):
    rot, pairs = st["rot"], st["rot"] // 2
    turn = torch.empty(st["B"], st["S"], pairs, dtype=torch.complex128, device=DEV)
    c = 0
    for a, n in enumerate(st["axis_pairs"]):
        ang = st["pos"][:, :, a:a + 1].double() * st["freqs"][c:c + n]
        turn[:, :, c:c + n] = torch.polar(torch.full_like(ang, st["mag"]), ang)
        c += n
    outs, scales = [], []
    for x, w in ((st["q"], st["wq"]), (st["k"], st["wk"])):
        B, S, H, D = x.shape
        y = torch.empty(B, H, S, D, dtype=torch.float64, device=DEV)
        for h in range(H):
            z = x[:, :, h].double()
            if w is not None:
                z = z / torch.sqrt(z.square().sum(-1, keepdim=True) / D + 1e-6) * w.double()
            lo, hi = (slice(0, rot, 2), slice(1, rot, 2)) if st["interleaved"] else (slice(0, pairs), slice(pairs, rot))
            t = torch.complex(z[..., lo], z[..., hi]) * turn
            z[..., lo], z[..., hi] = t.real, t.imag
            y[:, h] = z
        if st["out"] == "e4m3":
            d = torch.empty(B, H, -(-S // 128), dtype=torch.float64, device=DEV)
            for i in range(d.shape[2]):
                blk = y[:, :, i * 128:(i + 1) * 128]
                d[:, :, i] = blk.abs().amax((-1, -2)) / 448.0
                s = d[:, :, i, None, None]
                y[:, :, i * 128:(i + 1) * 128] = _grid_e4m3(blk / torch.where(s > 0, s, torch.ones_like(s)))
            scales.append(d)
        outs.append(y)
    return tuple(outs + scales)


def _exact_attn(st):
    B, H, S_q, S_kv, D = (st[k] for k in ("B", "H", "S_q", "S_kv", "D"))
    out = torch.zeros(B, H, S_q, D, dtype=torch.float64, device=DEV)
    lse = torch.full((B, H, S_q), -math.inf, dtype=torch.float64, device=DEV)
    key = torch.arange(S_kv, device=DEV)
    for b in range(B):
        start = int(st["start"][b]) if st["start"] is not None else S_kv - S_q
        for r0 in range(0, S_q, 8192):
            row = start + torch.arange(r0, min(r0 + 8192, S_q), device=DEV)[:, None]
            hidden = torch.zeros(row.shape[0], S_kv, dtype=torch.bool, device=DEV)
            if st["causal"]:
                hidden |= (key > row) & (key >= (int(st["prefix"][b]) if st["prefix"] is not None else 0))
            if st["docs"] is not None:
                mine = st["docs"][b, r0:r0 + 8192, None]
                hidden |= (mine != st["docs"][b]) | (mine < 0)
            for h in range(H):
                hk = h * st["H_kv"] // H
                z = st["q"][b, h, r0:r0 + 8192].double() @ st["k"][b, hk].double().T * st["scale"]
                if st["cap"]:
                    z = st["cap"] * torch.tanh(z / st["cap"])
                if st["slopes"] is not None:
                    z = z - st["slopes"][h].double() * (row - key).abs()
                z[hidden] = -math.inf
                lse[b, h, r0:r0 + 8192] = torch.logsumexp(z, 1)
                z = torch.exp(z - lse[b, h, r0:r0 + 8192, None])
                out[b, h, r0:r0 + 8192] = torch.nan_to_num(z) @ st["v"][b, hk].double()
    return out, lse
