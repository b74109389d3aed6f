"""Cases and plain forms of the operators around the mixers of a decode step: the norm with the
residual's addition, 4-bit projections of few rows, attention of sequences that share a prefix, and
sampling.

``run`` computes an operator in elementary torch operations (32 bits; sampling, whose borders are
exact, in 64), or, where ``own`` is true, calls the framework's operator.  Sizes and sequence lengths
follow from the case alone; values, page numbers and parameters from the seed.
"""

import math
import random

import torch

own = False

DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
# sizes of the largest listed cases, which drawn ones stay below
MAX_NORM = 8192 * 2048
MAX_WEIGHTS = 131072 * 2048
MAX_LOGITS = 256 * 131072
MAX_KEYS = 64 * 16900 * 2 * 256


# ------------------------------------------------------------------------------- cases

def listed():
    return [
        # the stream of one decode step of 4 sequences (latency)
        {"name": "norm_decode", "op": "norm", "tokens": 4, "heads": 1, "of": 1, "width": 2048, "dtype": "bf16",
         "residual": True, "out": "same", "group": 0, "offset": 0.0},
        # queries of 1531 tokens normalised by head, out of the fused projection of 16 + 2 + 2 heads
        {"name": "norm_heads", "op": "norm", "tokens": 1531, "heads": 16, "of": 20, "width": 256, "dtype": "fp16",
         "residual": False, "out": "same", "group": 0, "offset": 1.0},
        # a chunk of 8192 tokens on its way into an 8-bit projection, a scale for each 128 elements
        {"name": "norm_int8", "op": "norm", "tokens": 8192, "heads": 1, "of": 1, "width": 2048, "dtype": "bf16",
         "residual": True, "out": "int8", "group": 128, "offset": 0.0},
        # the fused query/key/value projection of one token, 16 + 2 + 2 heads of 256 (latency)
        {"name": "proj_one", "op": "proj", "tokens": 1, "k": 2048, "n": 5120, "x": "bf16", "group": 0, "out": "bf16"},
        # an output projection of 37 rows in 8 bits, of an odd number of outputs
        {"name": "proj_int8", "op": "proj", "tokens": 37, "k": 4096, "n": 2047, "x": "int8", "group": 128, "out": "bf16"},
        # logits of 8 tokens over a vocabulary of 131072 (weight bandwidth)
        {"name": "proj_head", "op": "proj", "tokens": 8, "k": 2048, "n": 131072, "x": "bf16", "group": 0, "out": "fp32"},
        # one token, nucleus sampling (latency: one row over the whole chip)
        {"name": "sample_one", "op": "sample", "rows": 1, "vocab": 131072, "dtype": "fp32", "kind": "top_p"},
        # 61 rows of an odd vocabulary, every row with its own parameters, some greedy; ties among bf16 logits
        {"name": "sample_mixed", "op": "sample", "rows": 61, "vocab": 100003, "dtype": "bf16", "kind": "mixed"},
        # 256 rows (logit bandwidth)
        {"name": "sample_batch", "op": "sample", "rows": 256, "vocab": 131072, "dtype": "fp32", "kind": "mixed"},
        # 4 samples of one prompt of 1K (latency)
        {"name": "prefix_small", "op": "prefix", "groups": 1, "seqs": 4, "prefix": 1024, "suffix": 60, "q": 1, "heads": 16,
         "kv_heads": 2, "dim": 256, "dtype": "bf16", "page": 32, "lse": False},
        # 64 samples of one prompt of 16K, the answers up to 512 tokens long
        {"name": "prefix_batch", "op": "prefix", "groups": 1, "seqs": 64, "prefix": 16384, "suffix": 512, "q": 1, "heads": 16,
         "kv_heads": 2, "dim": 256, "dtype": "bf16", "page": 32, "lse": False},
        # 23 samples of 5 prompts of uneven lengths, drafts of up to 4 tokens to verify, log-sum-exp returned
        {"name": "prefix_ragged", "op": "prefix", "groups": 5, "seqs": 23, "prefix": 5000, "suffix": 333, "q": 4, "heads": 32,
         "kv_heads": 8, "dim": 128, "dtype": "fp16", "page": 16, "lse": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "proj", "sample", "prefix"))
    if op == "norm":
        out = rng.choice(("same", "same", "int8"))
        group = rng.choice((0, 64, 128)) if out == "int8" else 0
        heads = rng.choice((1, 1, 1, 16, 5))
        width = rng.choice((64, 128, 256)) if heads > 1 else _log(rng, 1, 8192)
        if group:
            width = -(-width // group) * group
        return {"op": op, "tokens": _log(rng, 1, min(8192, max(1, MAX_NORM // (heads * width)))), "heads": heads,
                "of": heads + rng.choice((0, 4)) if heads > 1 else 1, "width": width, "dtype": rng.choice(("bf16", "bf16", "fp16")),
                "residual": rng.random() < 0.6, "out": out, "group": group, "offset": rng.choice((0.0, 1.0))}
    if op == "proj":
        k = 64 * _log(rng, 1, 128)
        x = rng.choice(("bf16", "bf16", "fp16", "int8"))
        return {"op": op, "tokens": _log(rng, 1, 64), "k": k, "n": _log(rng, 1, min(131072, MAX_WEIGHTS // k)), "x": x,
                "group": rng.choice([0, 64] + ([128] if k % 128 == 0 else [])) if x == "int8" else 0,
                "out": rng.choice(("fp32", "bf16" if x == "int8" else x))}
    if op == "sample":
        vocab = _log(rng, 1, 131072)
        return {"op": op, "rows": _log(rng, 1, 256), "vocab": vocab, "dtype": rng.choice(("fp32", "bf16", "fp16")),
                "kind": rng.choice(("top_p", "mixed", "mixed", "whole"))}
    heads, kv = rng.choice(((16, 2), (16, 2), (32, 8), (8, 8), (15, 3), (7, 1)))
    dim = rng.choice((64, 128, 256, 256))
    seqs = _log(rng, 1, 64)
    suffix = _log(rng, 1, 512)
    return {"op": op, "groups": rng.randint(1, min(6, seqs)), "seqs": seqs,
            "prefix": min(_log(rng, 16, 16384), MAX_KEYS // (seqs * kv * dim) - 2 * suffix), "suffix": suffix,
            "q": rng.choice((1, 1, rng.randint(1, 5))), "heads": heads, "kv_heads": kv, "dim": dim,
            "dtype": rng.choice(("bf16", "bf16", "fp16")), "page": rng.choice((16, 32, 64)), "lse": rng.random() < 0.3}


def _sequences(case):
    """Of a prefix case: group bounds, prefix lengths, new tokens and lengths, from the case alone."""
    rng = random.Random(case["seqs"] * 1000003 + case["prefix"] * 31 + case["suffix"] * 7 + case["q"])
    n, g = case["seqs"], case["groups"]
    bounds = [0] + sorted(rng.sample(range(1, n), g - 1)) + [n]
    prefix = [case["prefix"] if i == 0 else _log(rng, max(1, case["prefix"] // 4), case["prefix"]) for i in range(g)]
    new = [case["q"] if i == 0 or case["q"] == 1 else rng.randint(0, case["q"]) for i in range(n)]
    length = []
    for i in range(g):
        for b in range(bounds[i], bounds[i + 1]):
            length.append(prefix[i] + new[b] + rng.randint(0, max(0, case["suffix"] - new[b])))
    return bounds, prefix, new, length


def work(case):
    op = case["op"]
    if op == "norm":
        rows = case["tokens"] * case["heads"]
        el = rows * case["width"]
        out = 1 if case["out"] == "int8" else 2
        scales = 4 * rows * (case["width"] // case["group"] if case["group"] else 1) if case["out"] == "int8" else 0
        return {"bytes": el * (2 + out + (4 if case["residual"] else 0)) + scales + 2 * case["width"], "flops": 4 * el}
    if op == "proj":
        t, k, n = case["tokens"], case["k"], case["n"]
        x = t * k * (1 if case["x"] == "int8" else 2) + (4 * t * (k // case["group"] if case["group"] else 1) if case["x"] == "int8" else 0)
        return {"bytes": n * k // 2 + n * (k // 64) * 4 + x + t * n * (4 if case["out"] == "fp32" else 2), "flops": 2 * t * k * n}
    if op == "sample":
        return {"bytes": case["rows"] * (case["vocab"] * (4 if case["dtype"] == "fp32" else 2) + 28), "flops": 4 * case["rows"] * case["vocab"]}
    bounds, prefix, new, length = _sequences(case)
    keys = seen = 0
    for i, p in enumerate(prefix):
        mine = range(bounds[i], bounds[i + 1])
        if any(new[b] for b in mine):
            keys += p
        for b in mine:
            if new[b]:
                keys += length[b] - p
                seen += new[b] * (length[b] - new[b]) + new[b] * (new[b] + 1) // 2
    el = 2 * sum(new) * case["heads"] * case["dim"] + 2 * keys * case["kv_heads"] * case["dim"]
    return {"bytes": 2 * el, "flops": 4 * seen * case["heads"] * case["dim"]}


# ------------------------------------------------------------------------------ inputs

def _normal(gen, *shape, dtype=torch.float32):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32).to(dtype)


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    op = case["op"]
    s = {"case": case, "op": op}
    if op == "norm":
        t, h, w, dt = case["tokens"], case["heads"], case["width"], TYPES[case["dtype"]]
        # rows of uneven size, and a few channels far larger than the others
        x = _normal(gen, t, case["of"], w) * torch.exp(0.5 * _normal(gen, t, 1, 1)) * torch.exp(_normal(gen, 1, 1, w))
        s["x"] = x.to(dt)[:, :h]
        s["residual"] = (4.0 * _normal(gen, t, h, w)).to(dt) if case["residual"] else None
        s["weight"] = (1.0 - case["offset"] + 0.2 * _normal(gen, w)).to(dt)
        return s
    if op == "proj":
        t, k, n = case["tokens"], case["k"], case["n"]
        s["codes"] = torch.randint(-2 ** 31, 2 ** 31, (n, k // 8), generator=gen, device=DEV, dtype=torch.int64).int()
        s["scale"] = (0.005 + 0.015 * torch.rand((n, k // 64), generator=gen, device=DEV)).half()
        s["bias"] = (s["scale"].float() * (-8.0 + 0.5 * _normal(gen, n, k // 64))).half()
        x = _normal(gen, t, k) * torch.exp(_normal(gen, 1, k))
        if case["x"] == "int8":
            g = case["group"] or k
            top = x.view(t, k // g, g).abs().amax(-1) / 127.0
            s["x"] = torch.round(x.view(t, k // g, g) / top[..., None]).to(torch.int8).view(t, k)
            s["x_scale"] = top
        else:
            s["x"], s["x_scale"] = x.to(TYPES[case["x"]]), None
        if own:  # the weights in the framework's layout, as a server keeps them
            from sparse_moe_02_amd.linear import QLinear

            s["linear"] = QLinear(s["codes"], s["scale"], s["bias"], device=DEV)
        return s
    if op == "sample":
        r, v = case["rows"], case["vocab"]
        pick = random.Random(seed)
        # rows from flat to sharp; a tenth of the tokens ruled out, as by a grammar
        sharp = torch.tensor([pick.uniform(1.0, 4.0) for _ in range(r)], device=DEV)
        logits = _normal(gen, r, v) * sharp[:, None]
        banned = torch.rand((1, v), generator=gen, device=DEV) < 0.1
        banned[:, 0] = False
        s["logits"] = logits.masked_fill(banned, float("-inf")).to(TYPES[case["dtype"]])
        s["u"] = torch.rand(r, generator=gen, device=DEV)
        kind = case["kind"]
        temperature, top_k, top_p, min_p = [], [], [], []
        for _ in range(r):
            how = pick.choice(("greedy", "top_k", "top_p", "min_p", "all", "whole")) if kind == "mixed" else kind
            temperature.append(0.0 if how == "greedy" else pick.uniform(0.5, 1.3))
            top_k.append(pick.randint(1, 100) if how in ("top_k", "all") else 0)
            top_p.append(pick.uniform(0.5, 0.98) if how in ("top_p", "all") else 1.0)
            min_p.append(pick.uniform(0.01, 0.2) if how in ("min_p", "all") else 0.0)
        s["top_k"] = _ints(top_k)
        s["temperature"], s["top_p"], s["min_p"] = (torch.tensor(x, device=DEV) for x in (temperature, top_p, min_p))
        return s
    dt, hk, d, page = TYPES[case["dtype"]], case["kv_heads"], case["dim"], case["page"]
    bounds, prefix, new, length = _sequences(case)
    # the prefix's full pages belong to all sequences of a group, the others to one each
    counts, own_pages = 0, []
    cols = -(-max(length) // page) + 1
    for i, p in enumerate(prefix):
        shared = list(range(counts, counts + p // page))
        counts += len(shared)
        for b in range(bounds[i], bounds[i + 1]):
            more = -(-length[b] // page) - len(shared)
            own_pages.append(shared + list(range(counts, counts + more)) + [-1] * (cols - len(shared) - more))
            counts += more
    order = list(range(counts + 3))
    random.Random(seed).shuffle(order)
    s["table"] = _ints([[order[c] if c >= 0 else -1 for c in row] for row in own_pages])
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    s["q_start"], s["kv_len"], s["group_start"], s["prefix_len"] = map(_ints, (starts, length, bounds, prefix))
    s["max_q"], s["max_prefix"] = max(new), max(prefix)
    s["max_suffix"] = max(length[b] - prefix[i] for i in range(len(prefix)) for b in range(bounds[i], bounds[i + 1]))
    s["max_kv"], s["seq_group"] = max(length), [i for i in range(len(prefix)) for _ in range(bounds[i], bounds[i + 1])]
    s["q"] = 2.0 * _normal(gen, starts[-1], case["heads"], d)
    s["q"] = s["q"].to(dt)
    s["k_cache"], s["v_cache"] = (_normal(gen, counts + 3, page, hk, d, dtype=dt) for _ in range(2))
    # the part of a prefix behind its last full page: in each sequence's own page, alike
    for i, p in enumerate(prefix):
        if p % page and bounds[i + 1] - bounds[i] > 1:
            at = s["table"][bounds[i]:bounds[i + 1], p // page].long()
            for c in (s["k_cache"], s["v_cache"]):
                c[at, :p % page] = c[at[0], :p % page]
    return s


# --------------------------------------------------------------------------------- run

def run(s):
    if own:
        return _own(s)
    return {"norm": _norm, "proj": _proj, "sample": _sample, "prefix": _prefix}[s["op"]](s)


def _values(codes, scale, dtype):
    """The numbers that 8-bit codes and their scales stand for."""
    groups = codes.view(*scale.shape, -1)
    out = torch.empty(groups.shape, dtype=dtype, device=codes.device)
    return torch.mul(groups, scale[..., None], out=out).view(codes.shape)


def _own(s):
    case, op = s["case"], s["op"]
    if op == "norm":
        from sparse_moe_02_amd.norm import rms_norm

        if case["out"] == "int8":
            y, scale, *h = rms_norm(s["x"], s["weight"], residual=s["residual"], out_dtype=torch.int8, group=case["group"],
                                    offset=case["offset"])
            y = _values(y, scale, s["x"].dtype)
        elif case["residual"]:
            y, *h = rms_norm(s["x"], s["weight"], residual=s["residual"], offset=case["offset"])
        else:
            y, h = rms_norm(s["x"], s["weight"], offset=case["offset"]), []
        return {"y": y, "h": h[0]} if h else {"y": y}
    if op == "proj":
        return {"out": s["linear"](s["x"], s["x_scale"], out_dtype=TYPES[case["out"]])}
    if op == "sample":
        from sparse_moe_02_amd.sample import sample

        token, prob = sample(s["logits"], s["u"], s["temperature"], s["top_k"], s["top_p"], s["min_p"], return_prob=True)
        return {"token": token, "prob": prob}
    from sparse_moe_02_amd.attn import prefix_attn

    out = prefix_attn(s["q"], s["k_cache"], s["v_cache"], s["table"], s["q_start"], s["kv_len"], s["group_start"],
                      s["prefix_len"], s["max_q"], s["max_prefix"], s["max_suffix"], return_lse=case["lse"])
    return {"out": out[0], "lse": out[1]} if case["lse"] else {"out": out}


def _norm(s):
    case, dt = s["case"], s["x"].dtype
    h = s["x"].float()
    if case["residual"]:
        h = h + s["residual"].float()
    y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + 1e-6) * (case["offset"] + s["weight"].float())
    if case["out"] == "int8":
        groups = y.view(case["tokens"], case["heads"], -1, case["group"] or case["width"])
        scale = groups.abs().amax(-1) / 127.0
        codes = torch.round(groups / torch.where(scale == 0, 1.0, scale)[..., None])
        y = _values(codes.view(y.shape), scale, dt)
    out = {"y": y.to(dt)}
    if case["residual"]:
        out["h"] = h.to(dt)
    return out


def _proj(s):
    case, codes = s["case"], s["codes"]
    n, k = case["n"], case["k"]
    q = (codes[:, :, None] >> torch.arange(0, 32, 4, device=DEV, dtype=torch.int32)) & 15
    w = q.view(n, k // 64, 64).float() * s["scale"].float()[..., None] + s["bias"].float()[..., None]
    x = s["x"].float()
    if s["x_scale"] is not None:
        x = (x.view(*s["x_scale"].shape, -1) * s["x_scale"][..., None]).view(x.shape)
    return {"out": torch.matmul(x, w.view(n, k).t()).to(TYPES[case["out"]])}


def _sample(s):
    x = s["logits"].double()
    v = x.shape[1]
    x, order = torch.sort(x, dim=1, descending=True, stable=True)  # ties: the lowest index first
    t = s["temperature"].double()[:, None]
    w = torch.exp((x - x[:, :1]) / torch.where(t > 0, t, 1.0))
    rank = torch.arange(v, device=DEV)
    k = torch.where(s["top_k"] > 0, s["top_k"], v)[:, None]
    w = torch.where((rank < k) & ((t > 0) | (rank == 0)), w, 0.0)
    before = w.cumsum(1) - w
    p = s["top_p"].double()[:, None]
    keep = (p >= 1) | (before < p * w.sum(1, keepdim=True))
    keep &= w >= s["min_p"].double()[:, None]
    w = torch.where(keep | (rank == 0), w, 0.0)
    w = torch.zeros_like(w).scatter_(1, order, w)  # back in the tokens' order
    upto = w.cumsum(1)
    token = (upto <= s["u"].double()[:, None] * upto[:, -1:]).sum(1, keepdim=True).clamp(max=v - 1)
    prob = w.gather(1, token) / upto[:, -1:]
    return {"token": token[:, 0].int(), "prob": prob[:, 0].float()}


def _prefix(s):
    case = s["case"]
    n, h, hk, d, nq, nk = case["seqs"], case["heads"], case["kv_heads"], case["dim"], s["max_q"], s["max_kv"]
    g, t = h // hk, s["q"].shape[0]
    cols = -(-nk // case["page"])
    pages = s["table"][:, :cols].long().clamp(min=0)

    def rows(cache):
        return cache[pages].reshape(n, cols * case["page"], hk, d)[:, :nk].float()

    # queries padded to [sequence][kv head][group x token]
    start, length = s["q_start"].long(), s["kv_len"].long()
    at = (start[:-1, None] + torch.arange(nq, device=DEV)).clamp(max=max(t - 1, 0))
    q = s["q"][at].float().view(n, nq, hk, g, d).permute(0, 2, 3, 1, 4).reshape(n, hk, g * nq, d)
    p = torch.matmul(q, rows(s["k_cache"]).permute(0, 2, 3, 1).contiguous()).view(n, hk, g, nq, nk)
    p *= 1.0 / math.sqrt(d)
    pos = (length - (start[1:] - start[:-1]))[:, None] + torch.arange(nq, device=DEV)
    hidden = torch.arange(nk, device=DEV) > pos[..., None]
    p.masked_fill_(hidden[:, None, None], float("-inf"))
    top = p.amax(-1, keepdim=True)
    p.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p.view(n, hk, g * nq, nk), rows(s["v_cache"]).permute(0, 2, 1, 3).contiguous())
    out = out.view(n, hk, g, nq, d) / total
    # back to the tokens' order
    i = torch.arange(t, device=DEV)
    b = torch.searchsorted(start[1:], i, right=True)
    i = i - start[b]
    y = out.permute(0, 3, 1, 2, 4)[b, i].reshape(t, h, d).to(s["q"].dtype)
    if not case["lse"]:
        return {"out": y}
    lse = (top + total.log()).squeeze(-1).permute(0, 3, 1, 2)[b, i].reshape(t, h)
    return {"out": y, "lse": lse}


# ------------------------------------------------------------------------------- exact

def exact(case, seed):
    """The definitions in binary64, row by row or sequence by sequence."""
    s = prepare(case, seed)
    return {"norm": _exact_norm, "proj": _exact_proj, "sample": _exact_sample, "prefix": _exact_prefix}[case["op"]](case, s)


def _exact_norm(case, s):
    h = s["x"].double()
    if case["residual"]:
        h += s["residual"].double()
    size = torch.linalg.vector_norm(h, dim=-1, keepdim=True)
    y = h / torch.sqrt(size ** 2 / case["width"] + 1e-6) * (s["weight"].double() + case["offset"])
    out = {"y": y}
    if case["out"] == "int8":
        g = case["group"] or case["width"]
        parts = []
        for part in torch.split(y, g, dim=-1):
            step = torch.linalg.vector_norm(part, ord=float("inf"), dim=-1, keepdim=True) / 127
            parts.append(torch.round(part / step.clamp(min=1e-300)) * step)
        out["y"] = torch.cat(parts, -1)
    if case["residual"]:
        out["h"] = h
    return out


def _exact_proj(case, s):
    k, n = case["k"], case["n"]
    x = s["x"].double()
    if s["x_scale"] is not None:
        x = x * s["x_scale"].double().repeat_interleave(k // s["x_scale"].shape[1], 1)
    out = torch.empty((case["tokens"], n), dtype=torch.float64, device=DEV)
    for a in range(0, n, 8192):
        code = s["codes"][a:a + 8192]
        q = torch.stack([torch.bitwise_and(torch.bitwise_right_shift(code, 4 * j), 15) for j in range(8)], -1).flatten(1).double()
        scale, bias = (s[name][a:a + 8192].double().repeat_interleave(64, 1) for name in ("scale", "bias"))
        out[:, a:a + 8192] = x @ (q * scale + bias).t().contiguous()
    return {"out": out}


def _exact_sample(case, s):
    tokens, probs = [], []
    params = zip(s["u"].tolist(), s["temperature"].tolist(), s["top_k"].tolist(), s["top_p"].tolist(), s["min_p"].tolist())
    for row, (u, t, k, p, m) in zip(s["logits"].double(), params):
        if t <= 0:
            tokens.append(int(torch.nonzero(row == row.max())[0, 0]))
            probs.append(1.0)
            continue
        # the tokens by logit and, of equal ones, by index; then cut three times
        order = torch.argsort(row, descending=True, stable=True)
        if k > 0:
            order = order[:k]
        w = torch.softmax(row[order] / t, 0)
        if p < 1:
            whole = w.cumsum(0)
            order = order[:max(1, int((whole < p * whole[-1]).sum()) + 1)]
            w = w[:order.shape[0]]
        kept = order[w >= m * w[0]].sort().values
        w = torch.softmax(row[kept] / t, 0)
        i = min(int(torch.searchsorted(w.cumsum(0), u * float(w.sum()), right=True)), kept.shape[0] - 1)
        tokens.append(int(kept[i]))
        probs.append(float(w[i]))
    return {"token": torch.tensor(tokens, dtype=torch.int32, device=DEV), "prob": torch.tensor(probs, dtype=torch.float64, device=DEV)}


def _exact_prefix(case, s):
    _, _, new, length = _sequences(case)
    g, page, at = case["heads"] // case["kv_heads"], case["page"], 0
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full(s["q"].shape[:2], float("-inf"), dtype=torch.float64, device=DEV)
    for b, (n, t) in enumerate(zip(new, length)):
        if n:
            pages = s["table"][b, :-(-t // page)].long()
            seen = torch.arange(t, device=DEV) <= torch.arange(t - n, t, device=DEV)[:, None]
            for j in range(case["kv_heads"]):
                k = s["k_cache"][pages, :, j].reshape(-1, case["dim"])[:t].double()
                v = s["v_cache"][pages, :, j].reshape(-1, case["dim"])[:t].double()
                mine = slice(j * g, (j + 1) * g)
                x = s["q"][at:at + n, mine].double().reshape(n * g, -1) @ k.t().contiguous() / math.sqrt(case["dim"])
                x = torch.where(seen.repeat_interleave(g, 0), x, torch.full_like(x, float("-inf")))
                lse[at:at + n, mine] = torch.logsumexp(x, -1).view(n, g)
                out[at:at + n, mine] = (torch.softmax(x, -1) @ v).view(n, g, -1)
        at += n
    return {"out": out, "lse": lse} if case["lse"] else {"out": out}
