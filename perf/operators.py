"""What is measured of the operators around grouped-head attention: the cases, their
inputs, the operators' plain forms and the library's calls.

Operators (include/rec_attn.h):
  attn        masked time-RoPE attention over a packed ragged batch in which groups of
              query heads share a key/value head (rec_attn_plan_grouped + rec_attn_fwd)
  attn_train  the same with its backward pass: out, dq, dk, dv (rec_attn_fwd + rec_attn_bwd)
  score       candidates of a request against its cached history, read once for all
              candidates and all heads of a group (rec_attn_cache_create_grouped +
              rec_attn_cache_score)
  norm        layer norm with one gain and bias for each token type, or one for all
              (rec_attn_layernorm_fwd)
  norm_train  its backward pass: dx, dweight, dbias (rec_attn_layernorm_bwd)

`own` selects the library's calls; otherwise `run` computes the operators in elementary
torch operations, in 32 bits, rounded once.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
GLOBAL, HIST, RT, CAND = 0, 1, 2, 3
EPOCH = 1_700_000_000
PHI_MIN, DT_MAX, BASE = 1e-4, 365.0 * 86400.0, 6e5
EPS = 1e-5
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases
def attn_case(kind, batch, longest, shortest, heads, kv_heads, head_dim, special=0, cand=0, window=0, bidir=False,
              rope=True, dtype="bf16"):
    return {"kind": kind, "batch": batch, "longest": longest, "shortest": shortest, "heads": heads,
            "kv_heads": kv_heads, "head_dim": head_dim, "special": special, "cand": cand, "window": window,
            "bidir": bidir, "rope": rope, "dtype": dtype}


def score_case(batch, longest, shortest, cands, fewest, heads, kv_heads, head_dim, rt=0, dtype="bf16"):
    return {"kind": "score", "batch": batch, "longest": longest, "shortest": shortest, "cands": cands,
            "fewest": fewest, "heads": heads, "kv_heads": kv_heads, "head_dim": head_dim, "rt": rt, "dtype": dtype}


def norm_case(kind, rows, width, by_type, dtype="bf16"):
    return {"kind": kind, "rows": rows, "width": width, "by_type": by_type, "dtype": dtype}


def listed():
    cases = {
        # one user's short history, one request: latency
        "attn_one_request": attn_case("attn", 1, 301, 301, 8, 2, 64),
        # a serving batch of request-centric samples: special tokens, a windowed history, candidates
        "attn_requests": attn_case("attn", 32, 2264, 1133, 8, 2, 64, special=16, cand=200, window=256),
        # a 20K-token history with its target, causal: the longest prompts
        "attn_long_history": attn_case("attn", 1, 20001, 20001, 8, 2, 64, cand=1),
        # a training step on ragged samples whose profile and history see each other; wide heads
        "train_requests": attn_case("attn_train", 16, 1850, 603, 8, 2, 128, special=32, cand=60, bidir=True),
        # a training step on long causal histories without the rotation
        "train_long_history": attn_case("attn_train", 2, 8192, 7000, 8, 1, 64, rope=False),
        # one candidate of one request against its history: the smallest call, latency
        "score_one": score_case(1, 1023, 1023, 1, 1, 8, 2, 64),
        # a batch of requests with a single new token each: the cache's bytes
        "score_single_tokens": score_case(64, 8192, 4100, 1, 1, 8, 2, 128),
        # hundreds of candidates per request against a long history with real-time events
        "score_candidates": score_case(16, 4096, 3500, 500, 420, 8, 2, 64, rt=100),
        # layer norm of one request's tokens, one gain for all: latency
        "norm_one_request": norm_case("norm", 301, 512, False),
        # layer norm of a training batch of 20K-token histories, a gain for each token type
        "norm_histories": norm_case("norm", 320016, 512, True),
        # its backward pass in fp32 on a ragged batch with a wider hidden state
        "norm_train_wide": norm_case("norm_train", 50001, 1408, False, "fp32"),
        # the backward pass of the training batch, a gain for each token type
        "norm_train_histories": norm_case("norm_train", 320016, 512, True),
    }
    return [{"name": n, **c} for n, c in cases.items()]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["attn", "attn_train", "score", "norm", "norm_train"])
    if kind in ("norm", "norm_train"):
        width = 8 * _spread(rng, 8, 1024)
        rows = min(_spread(rng, 1, 320016), 320016 * 512 // width)
        return norm_case(kind, rows, width, rng.random() < 0.6, "bf16" if rng.random() < 0.75 else "fp32")
    kv = rng.choice([1, 2, 4])
    heads = kv * rng.choice([1, 2, 3, 4, 8])
    d = rng.choice([64, 128])
    if kind == "score":
        longest = _spread(rng, 1, 20000)
        cands = _spread(rng, 1, 500)
        batch = max(1, min(_spread(rng, 1, 64), int(16 * 8 * 500 * 4096 * 64 / (heads * cands * longest * d)),
                           int(64 * 8192 * 2 * 128 / (longest * kv * d))))
        return score_case(batch, longest, rng.randint(longest // 2, longest), cands, rng.randint(0, cands), heads,
                          kv, d, rng.choice([0, 0, rng.randint(0, longest // 4)]))
    fp32 = rng.random() < 0.15
    d = rng.choice([32, 64]) if fp32 else d
    # (a training batch in which no query sees a second key would have zero dq and dk)
    fewest = 1 if kind == "attn" else 16
    longest = _spread(rng, fewest, 700 if fp32 else 20001 if kind == "attn" else 8192)
    pairs = 4e7 if fp32 else 8 * 20001**2 if kind == "attn" else 16 * 8192**2
    batch = max(1, min(_spread(rng, 1, 64), int(pairs * 64 / (heads * longest**2 * d))))
    while heads * longest**2 * d > pairs * 64:
        longest = longest * 2 // 3
    bidir = rng.random() < 0.25
    return attn_case(kind, batch, longest, rng.randint((longest + 1) // 2, longest), heads, kv, d,
                     special=rng.choice([0, 16, 64]), cand=rng.choice([0, 1, rng.randint(0, longest // 8 + 1)]),
                     window=0 if bidir or rng.random() < 0.6 else _spread(rng, 1 if kind == "attn" else 4, 512), bidir=bidir,
                     rope=rng.random() < 0.7, dtype="fp32" if fp32 else "bf16")


# ------------------------------------------------------------------ shapes
def _lengths(case, most, least):
    """Lengths of the batch's requests, from `most` down to `least`."""
    n = case["batch"]
    return [most - (most - least) * b // max(1, n - 1) for b in range(n)]


def _parts(case, length):
    """(special, history, candidate) tokens of a request of `length` tokens."""
    g = min(case["special"], length)
    c = min(case["cand"], length - g)
    return g, length - g - c, c


def _pairs(case):
    """Visible (query, key) pairs of the batch for one head."""
    total = 0
    for length in _lengths(case, case["longest"], case["shortest"]):
        g, h, c = _parts(case, length)
        u = g + h
        i = np.arange(u, dtype=np.int64)
        if case["bidir"]:
            total += u * u
        elif case["window"]:
            w = case["window"]
            seen = np.where(i < g, i + 1, np.minimum(i + 1, w) + np.clip(i - w + 1, 0, g))
            total += int(seen.sum())
        else:
            total += u * (u + 1) // 2
        total += c * (u + 1)
    return total


def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    if case["kind"] in ("norm", "norm_train"):
        n = case["rows"] * case["width"]
        gains = (4 if case["by_type"] else 1) * case["width"] * 4
        types = case["rows"] if case["by_type"] else 0
        if case["kind"] == "norm":
            return {"bytes": 2 * n * size + 2 * gains + types, "flops": 8 * n}
        return {"bytes": 3 * n * size + 3 * gains + types, "flops": 16 * n}
    h, hk, d = case["heads"], case["kv_heads"], case["head_dim"]
    if case["kind"] == "score":
        hist = _lengths(case, case["longest"], case["shortest"])
        cands = _lengths(case, case["cands"], case["fewest"])
        pairs = sum(c * (n + 1) for n, c in zip(hist, cands))
        rows = sum(n for n, c in zip(hist, cands) if c > 0)
        return {"bytes": 2 * rows * hk * d * size + 9 * rows + sum(cands) * ((2 * h + 2 * hk) * d * size + 8),
                "flops": 4 * d * h * pairs}
    tokens = sum(_lengths(case, case["longest"], case["shortest"]))
    if case["kind"] == "attn":
        return {"bytes": tokens * ((2 * h + 2 * hk) * d * size + 9), "flops": 4 * d * h * _pairs(case)}
    # q, k, v and dout read; out, dq, dk, dv written; two products forward, five backward
    return {"bytes": tokens * ((4 * h + 4 * hk) * d * size + 9), "flops": 14 * d * h * _pairs(case)}


# ------------------------------------------------------------------ inputs
class _Kept:
    """A plan or cache that a program keeps, released with the state that holds it."""

    def __init__(self, handle, free):
        self.handle, self.free = handle, free

    def __del__(self):
        self.free(self.handle)


def _offsets(lengths):
    return np.concatenate([[0], np.cumsum(np.asarray(lengths, dtype=np.int64))]).astype(np.int64)


def _stamps(gen, n):
    """n increasing times, half an hour apart on average."""
    gaps = torch.randint(1, 3000, (n,), generator=gen, device=DEV)
    return EPOCH + torch.cumsum(gaps, 0)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    dtype = DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=DEV).to(dtype)

    if case["kind"] in ("norm", "norm_train"):
        rows, width = case["rows"], case["width"]
        s = {"case": case, "x": normal(rows, width) * 1.5 + 0.25, "groups": 4 if case["by_type"] else 1}
        s["weight"] = 1 + 0.1 * torch.randn(s["groups"], width, generator=gen, device=DEV)
        s["bias"] = 0.1 * torch.randn(s["groups"], width, generator=gen, device=DEV)
        s["types"] = None
        if case["by_type"]:
            # requests of a few hundred tokens: special tokens, a history, real-time events, candidates
            place = (torch.arange(rows, device=DEV) * 7 + int(torch.randint(0, 700, (1,), generator=gen, device=DEV))) % 4900
            s["types"] = ((place >= 112).int() + (place >= 4000).int() + (place >= 4600).int()).to(torch.int8)
        if case["kind"] == "norm_train":
            s["dy"] = normal(rows, width)
        return s
    h, hk, d = case["heads"], case["kv_heads"], case["head_dim"]
    if case["kind"] == "score":
        hist = _lengths(case, case["longest"], case["shortest"])
        cands = _lengths(case, case["cands"], case["fewest"])
        s = {"case": case, "hoff": _offsets(hist), "coff": _offsets(cands)}
        t, ty, tc = [], [], []
        for n, c in zip(hist, cands):
            times = _stamps(gen, n + 1)
            rt = min(case["rt"], n)
            t.append(times[:n])
            ty.append(torch.tensor([HIST] * (n - rt) + [RT] * rt, dtype=torch.int8, device=DEV))
            # candidates stand among the real-time events, or at the request's time
            back = torch.randint(0, 1500 * rt + 1, (c,), generator=gen, device=DEV)
            tc.append(times[n] - back)
        s["t"], s["ty"], s["tc"] = torch.cat(t), torch.cat(ty), torch.cat(tc)
        s["k"], s["v"] = normal(sum(hist), hk, d), normal(sum(hist), hk, d)
        s["qc"], s["kc"], s["vc"] = normal(sum(cands), h, d), normal(sum(cands), hk, d), normal(sum(cands), hk, d)
        s["hoff_d"], s["coff_d"] = torch.from_numpy(s["hoff"]).to(DEV), torch.from_numpy(s["coff"]).to(DEV)
        ref = _padded(s["hoff_d"], s["t"], case["longest"])[0][:, :1]
        s["ref"] = ref  # each request's reference time
        row_ref = torch.repeat_interleave(ref[:, 0], s["hoff_d"].diff())
        s["kr"] = _rotate(s["k"].float(), s["t"] - row_ref)  # the history's rotated keys, kept
        if own:
            from generative_recommender_ranking_gb300 import binding as bd
            params = bd.make_params(h, d, dtype=case["dtype"], phi_min=PHI_MIN, dt_max_s=DT_MAX, rope_base=BASE)
            cache = bd.rec_attn_cache_create_grouped(params, hk, s["hoff"], s["t"], s["ty"], s["k"], s["v"],
                                                     max(1, case["cands"]))
            s["kept"] = _Kept(cache, bd.rec_attn_cache_free)
        return s
    lengths = _lengths(case, case["longest"], case["shortest"])
    tokens = sum(lengths)
    s = {"case": case, "off": _offsets(lengths)}
    t, ty = [], []
    for n in lengths:
        g, u, c = _parts(case, n)
        times = _stamps(gen, u + 1)
        t += [times[-1:].expand(g), times[:u], times[-1:].expand(c)]
        ty += [GLOBAL] * g + [HIST] * u + [CAND] * c
    s["t"], s["ty"] = torch.cat(t), torch.tensor(ty, dtype=torch.int8, device=DEV)
    s["off_d"] = torch.from_numpy(s["off"]).to(DEV)
    s["q"], s["k"], s["v"] = normal(tokens, h, d), normal(tokens, hk, d), normal(tokens, hk, d)
    if case["kind"] == "attn_train":
        s["dout"] = normal(tokens, h, d)
    if own:
        from generative_recommender_ranking_gb300 import binding as bd
        params = bd.make_params(h, d, dtype=case["dtype"], window=case["window"], hist_bidirectional=case["bidir"],
                                use_rope=case["rope"], phi_min=PHI_MIN, dt_max_s=DT_MAX, rope_base=BASE)
        plan = bd.rec_attn_plan_grouped(params, hk, s["off"], s["off_d"], s["t"], s["ty"])
        s["kept"] = _Kept(plan, bd.rec_attn_free)
    return s


# ------------------------------------------------------------------ plain forms
def _padded(off, rows, longest):
    """Packed rows as [batch, longest, ...] (request b's rows first), and which are rows."""
    i = torch.arange(longest, device=rows.device)
    valid = i < off.diff()[:, None]
    at = (off[:-1, None] + i).clamp_max(max(rows.shape[0] - 1, 0))
    if rows.shape[0] == 0:
        return rows.new_zeros((off.shape[0] - 1, longest) + rows.shape[1:]), valid
    return rows[at], valid


def _rotate(x, dt, back=False):
    """The time-RoPE of rows x [..., heads, d] at dt [...] seconds: angles in 64 bits."""
    d = x.shape[-1]
    i = torch.arange(d // 2, device=x.device, dtype=torch.float64)
    angle = dt[..., None, None].double() * (PHI_MIN / DT_MAX * BASE ** (2 * i / d))
    cos, sin = angle.cos().to(x.dtype), angle.sin().to(x.dtype)
    if back:
        sin = -sin
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)


def _visible(case, ty, valid):
    """[batch, L, L]: which keys each query sees."""
    p = torch.arange(ty.shape[1], device=ty.device)
    gap = p[:, None] - p[None, :]
    user = ty != CAND
    near = gap >= 0
    if case["window"]:
        is_g = ty == GLOBAL
        near = near & ((gap < case["window"]) | is_g[:, :, None] | is_g[:, None, :])
    if case["bidir"]:
        near = torch.ones_like(near)
    seen = user[:, None, :] & (~user[:, :, None] | near) | (gap == 0)
    return seen & valid[:, None, :] & valid[:, :, None]


def _weights(scores, seen):
    """Softmax over the seen keys; a row that sees none is all zero.  In place on scores."""
    scores.masked_fill_(~seen, -math.inf)
    top = scores.amax(-1, keepdim=True)
    scores.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = scores.sum(-1, keepdim=True)
    return scores.div_(torch.where(total == 0, 1.0, total))


def _plain_attn(s):
    c = s["case"]
    h, hk, d, n = c["heads"], c["kv_heads"], c["head_dim"], c["longest"]
    scale = 1 / math.sqrt(d)
    t, valid = _padded(s["off_d"], s["t"], n)
    dt = t - t[:, :1]
    turn = _rotate if c["rope"] else lambda x, *a: x

    def split(rows, turned):  # [B, kv heads, heads of the group, L, d] in 32 bits
        x = _padded(s["off_d"], rows, n)[0].float()
        x = turn(x, dt) if turned else x
        return x.unflatten(2, (hk, -1)).permute(0, 2, 3, 1, 4)

    def packed(x, turned):  # back to [T, heads, d] in the inputs' type
        x = x.permute(0, 3, 1, 2, 4).flatten(2, 3)
        x = turn(x, dt, True) if turned else x
        return x[valid].to(DTYPES[c["dtype"]])

    q, k, v = split(s["q"], True), split(s["k"], True), split(s["v"], False)
    seen = _visible(c, _padded(s["off_d"], s["ty"], n)[0], valid)[:, None, None]
    p = _weights((q * scale) @ k.transpose(-1, -2), seen)
    o = p @ v
    if c["kind"] == "attn":
        return {"out": packed(o, False)}
    g = split(s["dout"], False) * valid[:, None, None, :, None]
    dv = (p.transpose(-1, -2) @ g).sum(2, keepdim=True)
    ds = g @ v.transpose(-1, -2)
    ds.sub_((g * o).sum(-1, keepdim=True)).mul_(p).mul_(scale)
    dq = ds @ k
    dk = (ds.transpose(-1, -2) @ q).sum(2, keepdim=True)
    return {"out": packed(o, False), "dq": packed(dq, True), "dk": packed(dk, True), "dv": packed(dv, False)}


def _plain_score(s):
    c = s["case"]
    h, hk, d = c["heads"], c["kv_heads"], c["head_dim"]
    n, m = c["longest"], c["cands"]
    t, old = _padded(s["hoff_d"], s["t"], n)
    ty = _padded(s["hoff_d"], s["ty"], n)[0]
    k, v = (_padded(s["hoff_d"], x, n)[0].float().permute(0, 2, 1, 3)[:, :, None] for x in (s["kr"], s["v"]))
    tc, valid = _padded(s["coff_d"], s["tc"], m)
    dt = tc - s["ref"]
    q, kc, vc = (_padded(s["coff_d"], s[x], m)[0].float() for x in ("qc", "kc", "vc"))
    q = _rotate(q, dt).unflatten(2, (hk, -1)).permute(0, 2, 3, 1, 4) / math.sqrt(d)
    kc = _rotate(kc, dt).permute(0, 2, 1, 3)[:, :, None]
    vc = vc.permute(0, 2, 1, 3)[:, :, None]
    seen = old[:, None, :] & ((ty[:, None, :] != RT) | (t[:, None, :] < tc[:, :, None]))
    past = (q @ k.transpose(-1, -2)).masked_fill_(~seen[:, None, None], -math.inf)
    itself = (q * kc).sum(-1, keepdim=True)
    top = torch.maximum(past.amax(-1, keepdim=True), itself)
    past.sub_(top).exp_()
    itself = (itself - top).exp()
    o = (past @ v + itself * vc) / (past.sum(-1, keepdim=True) + itself)
    return {"out": o.permute(0, 3, 1, 2, 4).flatten(2, 3)[valid].to(DTYPES[c["dtype"]])}


def _plain_norm(s):
    x = s["x"].float()
    mean = x.mean(-1, keepdim=True)
    x = x - mean
    rstd = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    x = x * rstd
    ty = s["types"]
    by_type = ty is not None
    w = s["weight"][ty.long()] if by_type else s["weight"]
    if s["case"]["kind"] == "norm":
        b = s["bias"][ty.long()] if by_type else s["bias"]
        return {"y": (x * w + b).to(s["x"].dtype)}
    dy = s["dy"].float()
    g = dy * w
    dx = rstd * (g - g.mean(-1, keepdim=True) - x * (g * x).mean(-1, keepdim=True))
    if by_type:
        group = (ty == torch.arange(s["groups"], device=ty.device)[:, None]).float()
        dw, db = group @ (dy * x), group @ dy
    else:
        dw, db = (dy * x).sum(0, keepdim=True), dy.sum(0, keepdim=True)
    return {"dx": dx.to(s["x"].dtype), "dweight": dw, "dbias": db}


def run(s):
    c = s["case"]
    if not own:
        if c["kind"] in ("norm", "norm_train"):
            return _plain_norm(s)
        return _plain_score(s) if c["kind"] == "score" else _plain_attn(s)
    from generative_recommender_ranking_gb300 import binding as bd
    if c["kind"] == "norm":
        y = torch.empty_like(s["x"])
        bd.rec_attn_layernorm_fwd(s["x"], s["weight"], s["bias"], y, types=s["types"], eps=EPS)
        return {"y": y}
    if c["kind"] == "norm_train":
        dx, dw, db = torch.empty_like(s["x"]), torch.empty_like(s["weight"]), torch.empty_like(s["bias"])
        bd.rec_attn_layernorm_bwd(s["x"], s["weight"], s["dy"], dx, dw, db, types=s["types"], eps=EPS)
        return {"dx": dx, "dweight": dw, "dbias": db}
    if c["kind"] == "score":
        out = torch.empty_like(s["qc"])
        bd.rec_attn_cache_score(s["kept"].handle, s["coff"], s["tc"], s["qc"], s["kc"], s["vc"], out)
        return {"out": out}
    plan, q, k, v = s["kept"].handle, s["q"], s["k"], s["v"]
    out = torch.empty_like(q)
    if c["kind"] == "attn":
        bd.rec_attn_fwd(plan, q, k, v, out)
        return {"out": out}
    lse = torch.empty(q.shape[:2], dtype=torch.float32, device=DEV)
    bd.rec_attn_fwd(plan, q, k, v, out, lse)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    bd.rec_attn_bwd(plan, q, k, v, out, lse, s["dout"], dq, dk, dv)
    return {"out": out, "dq": dq, "dk": dk, "dv": dv}


# ------------------------------------------------------------------ in 64 bits
def _turned(x, seconds):
    """Adjacent pairs of rows x [n, d] as complex numbers, turned by the time's angle."""
    d = x.shape[-1]
    speed = torch.tensor([PHI_MIN / DT_MAX * BASE ** (2.0 * i / d) for i in range(d // 2)], dtype=torch.float64, device=DEV)
    z = torch.view_as_complex(x.reshape(x.shape[0], d // 2, 2).contiguous())
    z = z * torch.polar(torch.ones_like(speed), speed * seconds.double()[:, None])
    return torch.view_as_real(z).reshape(x.shape[0], d)


def _exact_head(q, k, v, seen):
    """Definition of one head: exp of the seen scores over their sum, times the values."""
    s = (q @ k.T) / math.sqrt(q.shape[1])
    s = torch.where(seen, s, torch.full((), -math.inf, dtype=s.dtype, device=DEV))
    lse = torch.logsumexp(s, 1, keepdim=True)
    return torch.where(seen, (s - torch.where(lse.isinf(), torch.zeros_like(lse), lse)).exp(), torch.zeros((), dtype=s.dtype, device=DEV)) @ v


def _exact_seen(case, length):
    g, u, _ = _parts(case, length)
    u += g
    seen = torch.eye(length, dtype=torch.bool, device=DEV)
    seen[u:, :u] = True
    if case["bidir"]:
        seen[:u, :u] = True
    else:
        causal = torch.ones(u, u, dtype=torch.bool, device=DEV).tril_()
        if case["window"]:
            band = causal & ~torch.ones(u, u, dtype=torch.bool, device=DEV).tril_(-case["window"])
            band[:, :g] = causal[:, :g]
            band[:g] = causal[:g]
            causal = band
        seen[:u, :u] = causal
    return seen


def _exact_attn(case, s):
    h, hk = case["heads"], case["kv_heads"]
    train = case["kind"] == "attn_train"
    outs = {x: torch.zeros_like(s[y], dtype=torch.float64)
            for x, y in (("out", "q"), ("dq", "q"), ("dk", "k"), ("dv", "v"))}
    for lo, hi in zip(s["off"][:-1], s["off"][1:]):
        seen = _exact_seen(case, int(hi - lo))
        dt = s["t"][lo:hi] - s["t"][lo:hi][:1]
        for j in range(h):
            kv = j * hk // h
            q, k, v = (s[x][lo:hi, i].double().requires_grad_(train) for x, i in (("q", j), ("k", kv), ("v", kv)))
            o = _exact_head(_turned(q, dt) if case["rope"] else q, _turned(k, dt) if case["rope"] else k, v, seen)
            outs["out"][lo:hi, j] = o.detach()
            if train:
                o.backward(s["dout"][lo:hi, j].double())
                outs["dq"][lo:hi, j] = q.grad
                outs["dk"][lo:hi, kv] += k.grad
                outs["dv"][lo:hi, kv] += v.grad
            del o
    return outs if train else {"out": outs["out"]}


def _exact_score(case, s):
    h, hk = case["heads"], case["kv_heads"]
    out = torch.zeros_like(s["qc"], dtype=torch.float64)
    for b in range(case["batch"]):
        lo, hi = s["hoff"][b], s["hoff"][b + 1]
        c0, c1 = s["coff"][b], s["coff"][b + 1]
        n, m = int(hi - lo), int(c1 - c0)
        if m == 0:
            continue
        time = torch.cat([s["t"][lo:hi], s["tc"][c0:c1]])
        dt = time - time[0]
        seen = torch.cat([torch.ones(m, n, dtype=torch.bool, device=DEV), torch.eye(m, dtype=torch.bool, device=DEV)], 1)
        late = (s["ty"][lo:hi] == RT)[None, :] & (time[None, :n] >= time[n:, None])
        seen[:, :n] &= ~late
        for j in range(h):
            kv = j * hk // h
            q = _turned(s["qc"][c0:c1, j].double(), dt[n:])
            k = _turned(torch.cat([s["k"][lo:hi, kv], s["kc"][c0:c1, kv]]).double(), dt)
            v = torch.cat([s["v"][lo:hi, kv], s["vc"][c0:c1, kv]]).double()
            out[c0:c1, j] = _exact_head(q, k, v, seen)
    return {"out": out}


def _exact_norm(case, s):
    x = s["x"].double()
    n = x.shape[1]
    centre = x - x.sum(1, keepdim=True) / n
    root = ((centre**2).sum(1, keepdim=True) / n + EPS).sqrt()
    unit = centre / root
    ty = s["types"].tolist() if s["types"] is not None else [0] * x.shape[0]
    group = torch.tensor(ty, device=DEV)
    w, b = s["weight"].double()[group], s["bias"].double()[group]
    if case["kind"] == "norm":
        return {"y": unit * w + b}
    dy = s["dy"].double()
    g = dy * w
    dx = (n * g - g.sum(1, keepdim=True) - unit * (g * unit).sum(1, keepdim=True)) / (n * root)
    zero = torch.zeros(s["groups"], n, dtype=torch.float64, device=DEV)
    return {"dx": dx, "dweight": zero.index_add(0, group, dy * unit), "dbias": zero.index_add(0, group, dy)}


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] in ("norm", "norm_train"):
        return _exact_norm(case, s)
    return _exact_score(case, s) if case["kind"] == "score" else _exact_attn(case, s)
