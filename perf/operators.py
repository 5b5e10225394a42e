"""Cases of the decode-step operators: filling a paged key-value cache
(qkv_rope_store), one new token's attention over it (attn_paged) and sampling
from sharded logits (sample_merge).

`run` computes a case in its plain form (elementary torch operations) where
`own` is false, and through the package where it is true; `exact` is the
definition in 64 bits."""
import math
import random

import numpy as np
import torch

own = False

E4M3_MAX = 448.0


# ------------------------------------------------------------------- cases

def _attn(name, rows, max_len, ragged, q_heads, kv_heads, head_dim, page_tokens, kind, order, window=0, sinks=0,
          out="bf16"):
    return {"name": name, "op": "attn", "rows": rows, "max_len": max_len, "ragged": ragged, "q_heads": q_heads,
            "kv_heads": kv_heads, "head_dim": head_dim, "page_tokens": page_tokens, "kind": kind, "order": order,
            "window": window, "sinks": sinks, "out": out}


def _store(name, tokens, q_heads, kv_heads, head_dim, page_tokens, kind, order, norm, rot_dim, interleaved):
    return {"name": name, "op": "store", "tokens": tokens, "q_heads": q_heads, "kv_heads": kv_heads,
            "head_dim": head_dim, "page_tokens": page_tokens, "kind": kind, "order": order, "norm": norm,
            "rot_dim": rot_dim, "interleaved": interleaved}


def _sample(name, rows, ncols0, ncols1, filters, masked):
    return {"name": name, "op": "sample", "rows": rows, "ncols0": ncols0, "ncols1": ncols1, "filters": filters,
            "masked": masked}


def listed():
    return [
        # one request early in its answer: nothing but latency
        _attn("attn one short row", 1, 41, False, 8, 1, 128, 16, "bf16", "tokens"),
        # a serving batch, every request at another length; a head's page is one 4 KiB segment
        _attn("attn ragged batch", 48, 8192, True, 32, 8, 128, 16, "bf16", "heads"),
        # two requests over long documents, hidden size 5120 (40 heads of 128), partials for the all-reduce in F32
        _attn("attn two long rows", 2, 131071, False, 40, 8, 128, 16, "bf16", "heads", out="f32"),
        # layers that see a window and four first tokens, 8-bit cache, heads of 64
        _attn("attn window and sinks e4m3", 96, 16000, True, 64, 8, 64, 32, "e4m3", "tokens", window=1024, sinks=4),
        # many queries for few wide key heads, 8-bit cache
        _attn("attn wide heads e4m3", 8, 20001, True, 64, 2, 256, 64, "e4m3", "heads"),
        # one new token of one request
        _store("store one token", 1, 40, 8, 128, 16, "bf16", "heads", True, 128, False),
        # a decode batch into an 8-bit cache, a part of each head rotated in pairs of neighbours, no norms
        _store("store decode batch e4m3", 77, 64, 8, 64, 32, "e4m3", "tokens", False, 32, True),
        # a prompt batch of 16384 tokens at hidden size 5120
        _store("store prompt 16384", 16384, 40, 8, 128, 16, "bf16", "heads", True, 128, False),
        # one request over the drafter's vocabulary, the usual filters together
        _sample("sample one row", 1, 64768, 64512, "all", False),
        # 4 requests x 4 drafted positions, each with settings of its own
        _sample("sample 16 rows mixed", 16, 64768, 64512, "mixed", False),
        # a large batch over a larger vocabulary, temperature and min-p alone
        _sample("sample 256 rows", 256, 75968, 75968, "minp", False),
        # many rows of a narrow ragged vocabulary under a grammar's mask
        _sample("sample narrow masked rows", 333, 2304, 1695, "mixed", True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "store", "sample"])
    if op == "attn":
        head_dim = rng.choice([64, 128, 256])
        kind = rng.choice(["bf16", "e4m3"])
        kv_heads = rng.choice([1, 2, 4, 8])
        q_heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 7, 8, 16, 20])
        window = rng.choice([0, 0, _log(rng, 100, 5000)])
        rows = _log(rng, 1, 128)
        # no more cache than the largest listed case reads
        most = 131071 * 2 * 8 * 128 // (rows * kv_heads * head_dim)
        return {k: v for k, v in _attn("", rows, _log(rng, 1, max(1, min(131071, most))), rng.choice([True, False]),
                                       q_heads, kv_heads, head_dim, rng.choice([1, 8, 16, 32, 64, 128]), kind,
                                       rng.choice(["tokens", "heads"]), window, rng.choice([0, 1, 4]) if window else 0,
                                       rng.choice(["bf16", "f32"])).items() if k != "name"}
    if op == "store":
        head_dim = rng.choice([64, 128, 256])
        kv_heads = rng.choice([1, 2, 4, 8])
        q_heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 7, 8])
        most = 16384 * 56 * 128 // ((q_heads + 2 * kv_heads) * head_dim)
        return {k: v for k, v in _store("", _log(rng, 1, max(1, min(16384, most))), q_heads, kv_heads, head_dim,
                                        rng.choice([1, 8, 16, 32, 64, 128]), rng.choice(["bf16", "e4m3"]),
                                        rng.choice(["tokens", "heads"]), rng.choice([True, False]),
                                        rng.choice([head_dim, head_dim, head_dim // 2]),
                                        rng.choice([True, False])).items() if k != "name"}
    rows = _log(rng, 1, 512)
    most = 256 * 151936 // rows
    cols = _log(rng, 1000, min(262144, most))
    n0 = rng.randrange(1, cols)
    return {k: v for k, v in _sample("", rows, n0, cols - n0, rng.choice(["all", "mixed", "minp", "topk", "topp"]),
                                     rng.choice([True, False])).items() if k != "name"}


# ------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) & 0x7FFFFFFF)
    return g


def _normal(shape, g, dtype=torch.bfloat16, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _lens(case):
    """The rows' lengths, the same for every seed: all of max_len, or spread over the range up to it."""
    rows, m = case["rows"], case["max_len"]
    return [max(1, int(m * ((i + 1) / rows) ** 2)) if case["ragged"] else m for i in range(rows)]


def _visible(case):
    w, s = case["window"], case["sinks"]
    return [n if w == 0 else min(n, w + s) for n in _lens(case)]


def _cache(case, n_pages, g):
    """K and V of a paged cache as [page, token, head, dim] views, and their scales (8-bit caches)."""
    p, h, d = case["page_tokens"], case["kv_heads"], case["head_dim"]
    shape = (n_pages, p, h, d) if case["order"] == "tokens" else (n_pages, h, p, d)
    dt = torch.bfloat16 if case["kind"] == "bf16" else torch.float8_e4m3fn
    k, v = _normal(shape, g, dt), _normal(shape, g, dt)
    if case["order"] == "heads":
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    if case["kind"] == "bf16":
        return k, v, None, None
    # powers of two and others, as a calibration leaves them
    ks = torch.rand(h, generator=g, device="cuda") * 1.5 + 0.25
    vs = torch.rand(h, generator=g, device="cuda") * 1.5 + 0.25
    return k, v, ks, vs


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    if case["op"] == "attn":
        rows, p = case["rows"], case["page_tokens"]
        lens = _lens(case)
        random.Random(int(seed)).shuffle(lens)
        width = -(-case["max_len"] // p)
        used = [-(-n // p) for n in lens]
        n_pages = sum(used) + 3
        s["k"], s["v"], s["ks"], s["vs"] = _cache(case, n_pages, g)
        order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
        table = torch.zeros((rows, width), dtype=torch.int32, device="cuda")
        col = torch.arange(width, device="cuda")[None, :]
        n = torch.tensor(used, device="cuda")[:, None]
        at = torch.cumsum(n, 0) - n + col
        s["table"] = torch.where(col < n, order[at.clamp(max=n_pages - 1)], table)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["q"] = _normal((rows, case["q_heads"], case["head_dim"]), g, scale=1.5)
        s["scale"] = case["head_dim"] ** -0.5
        s["out"] = torch.empty((rows, case["q_heads"], case["head_dim"]), device="cuda",
                               dtype=torch.bfloat16 if case["out"] == "bf16" else torch.float32)
    elif case["op"] == "store":
        t, d, hq, hkv = case["tokens"], case["head_dim"], case["q_heads"], case["kv_heads"]
        p = case["page_tokens"]
        n_pages = -(-t // p) + 5
        s["k"], s["v"], s["ks"], s["vs"] = _cache(case, n_pages, g)
        # one fused projection's output, as the model's product leaves it: q, k and v are slices of its rows
        qkv = _normal((t, (hq + 2 * hkv) * d), g, scale=2.0)
        s["q"] = qkv[:, :hq * d].view(t, hq, d)
        s["new_k"] = qkv[:, hq * d:(hq + hkv) * d].view(t, hkv, d)
        s["new_v"] = qkv[:, (hq + hkv) * d:].view(t, hkv, d)
        s["wq"] = _normal((d,), g, scale=0.2) + 1 if case["norm"] else None
        s["wk"] = _normal((d,), g, scale=0.2) + 1 if case["norm"] else None
        s["eps"] = 1e-6
        max_pos, r = 32768, case["rot_dim"]
        s["positions"] = torch.randint(0, max_pos, (t,), generator=g, device="cuda").to(torch.int32)
        a = (torch.arange(max_pos, dtype=torch.float64, device="cuda")[:, None]
             * 1e6 ** (-torch.arange(0, r, 2, dtype=torch.float64, device="cuda") / r)[None, :])
        s["cos_sin"] = torch.cat([a.cos(), a.sin()], 1).float()
        slots = torch.randperm(n_pages * p, generator=g, device="cuda")[:t]
        if t > 8:
            slots[::97] = -1  # tokens that another rank keeps
        s["slots"] = slots
        s["q_out"] = torch.empty((t, hq, d), dtype=torch.bfloat16, device="cuda")
    else:
        rows, n0, n1 = case["rows"], case["ncols0"], case["ncols1"]
        shards = []
        for n in (n0, n1):
            x = torch.randn((rows, -(-n // 8) * 8), generator=g, device="cuda") * 2.5
            x = x + 8.0 * (torch.rand(x.shape, generator=g, device="cuda") < 2e-4)
            if case["masked"]:
                x = x.masked_fill(torch.rand(x.shape, generator=g, device="cuda") < 0.7, -math.inf)
            shards.append(x.to(torch.bfloat16))
        s["l0"], s["l1"] = shards
        presets = {"all": [(0.8, 50, 0.95, 0.02)], "minp": [(1.0, 0, 1.0, 0.05)], "topk": [(0.7, 40, 1.0, 0.0)],
                   "topp": [(1.0, 0, 0.9, 0.0)],
                   "mixed": [(0.8, 50, 0.95, 0.0), (1.0, 0, 1.0, 0.0), (0.0, 0, 1.0, 0.0), (1.3, 0, 0.9, 0.0),
                             (0.6, 1000, 1.0, 0.1), (1.0, 1, 0.5, 0.0), (2.0, 0, 0.99, 0.001)]}[case["filters"]]
        rng = random.Random(int(seed))
        rows_p = [presets[rng.randrange(len(presets))] for _ in range(rows)]
        s["params"] = torch.from_numpy(np.array(rows_p, dtype=np.dtype(
            [("temperature", "<f4"), ("top_k", "<u4"), ("top_p", "<f4"), ("min_p", "<f4")])).view(np.uint8)).cuda()
        s["u"] = torch.rand(rows, generator=g, device="cuda")
        s["out"] = torch.empty((rows, 2), dtype=torch.int32, device="cuda")
    if own:
        from bf16_wire_all_amd import decode
        if case["op"] == "sample":
            s["s0"] = decode.shard(s["l0"], case["ncols0"], 0)
            s["s1"] = decode.shard(s["l1"], case["ncols1"], case["ncols0"])
            need = decode.sample_workspace_bytes(case["rows"], case["ncols0"], case["ncols1"])
        else:
            s["cache"] = decode.kv_cache(s["k"], s["v"], s["ks"], s["vs"])
            need = 0
            if case["op"] == "attn":
                need = decode.attn_workspace_bytes(s["cache"], case["rows"], case["q_heads"], case["max_len"],
                                                   case["window"], case["sinks"])
        s["workspace"] = torch.empty(max(16, need), dtype=torch.uint8, device="cuda")
    return s


# -------------------------------------------------------------- plain forms

def _plain_attn(s):
    c = s["case"]
    rows, kv, d, p = c["rows"], c["kv_heads"], c["head_dim"], c["page_tokens"]
    lens = s["lens"].long()[:, None]
    vis = c["max_len"] if c["window"] == 0 else min(c["max_len"], c["window"] + c["sinks"])
    i = torch.arange(vis, device="cuda")[None, :].expand(rows, vis)
    # the i-th visible token of a row: its first ones, then the window's
    n_vis = lens if c["window"] == 0 else lens.clamp(max=c["window"] + c["sinks"])
    token = torch.where(i < c["sinks"], i, i + (lens - n_vis))
    there = i < n_vis
    token = torch.where(there, token, 0)
    page = torch.gather(s["table"].long(), 1, token // p)
    k = s["k"].view(torch.uint8 if c["kind"] == "e4m3" else torch.bfloat16)[page, token % p].view(s["k"].dtype).float()
    v = s["v"].view(torch.uint8 if c["kind"] == "e4m3" else torch.bfloat16)[page, token % p].view(s["v"].dtype).float()
    if s["ks"] is not None:
        k, v = k * s["ks"][:, None], v * s["vs"][:, None]
    q = s["q"].float().view(rows, kv, c["q_heads"] // kv, d)
    score = torch.matmul(q, k.permute(0, 2, 3, 1)) * s["scale"]
    score = score.masked_fill(~there[:, None, None, :], -math.inf)
    w = torch.exp(score - score.amax(-1, keepdim=True))
    o = torch.matmul(w, v.permute(0, 2, 1, 3)) / w.sum(-1, keepdim=True)
    s["out"].copy_(o.view(rows, c["q_heads"], d))
    return s["out"]


def _plain_rotated(x, w, s):
    c = s["case"]
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * w.float()
    r = c["rot_dim"]
    cs = s["cos_sin"][s["positions"].long()][:, None, :]
    cos, sin = cs[..., :r // 2], cs[..., r // 2:]
    if c["interleaved"]:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., r:]], -1)


def _plain_put(cache, scale, x, s):
    """x into the cache slots of the tokens that have one."""
    c = s["case"]
    kept = s["slots"] >= 0
    page, at = s["slots"][kept] // c["page_tokens"], s["slots"][kept] % c["page_tokens"]
    if scale is None:
        cache[page, at] = x[kept].to(torch.bfloat16)
    else:
        y = (x.float()[kept] / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX)
        cache.view(torch.uint8)[page, at] = y.to(torch.float8_e4m3fn).view(torch.uint8)


def _plain_store(s):
    s["q_out"].copy_(_plain_rotated(s["q"], s["wq"], s))
    _plain_put(s["k"], s["ks"], _plain_rotated(s["new_k"], s["wk"], s), s)
    _plain_put(s["v"], s["vs"], s["new_v"], s)
    return {"q": s["q_out"], "k": s["k"], "v": s["v"]}


def _plain_sample(s):
    c = s["case"]
    p = s["params"].view(torch.float32).view(-1, 4)
    top_k = s["params"].view(torch.int32).view(-1, 4)[:, 1:2].long()
    temperature, top_p, min_p = p[:, 0:1].double(), p[:, 2:3].double(), p[:, 3:4].double()
    x = torch.cat([s["l0"][:, :c["ncols0"]], s["l1"][:, :c["ncols1"]]], 1).float()
    # the row's order: larger first, then the lower id
    x, ids = torch.sort(x, dim=1, descending=True, stable=True)
    x = x.double()
    top = x[:, :1]
    greedy = temperature <= 0
    w = torch.exp((x - top) / torch.where(greedy, 1.0, temperature))
    n = torch.arange(w.shape[1], device="cuda")[None, :]
    keep = (x > -math.inf) & ((top_k == 0) | (n < top_k)) & (~greedy | (n == 0))
    w = torch.where(keep, w, 0.0)
    run_sum = torch.cumsum(w, 1)
    keep = keep & ((top_p >= 1) | (run_sum - w < top_p * run_sum[:, -1:]))
    keep = keep & (w >= min_p)
    w = torch.where(keep, w, 0.0)
    run_sum = torch.cumsum(w, 1)
    total = run_sum[:, -1:]
    at = (run_sum <= s["u"].double()[:, None] * total).sum(1, keepdim=True)
    at = torch.minimum(at, keep.sum(1, keepdim=True) - 1).clamp(min=0)
    got = keep.any(1)
    idx = torch.where(got, torch.gather(ids, 1, at)[:, 0], -1)
    prob = torch.where(got, (torch.gather(w, 1, at) / total)[:, 0], 0.0)
    return {"idx": idx.to(torch.int32), "prob": prob.float()}


def run(state):
    s = state
    c = s["case"]
    if not own:
        return {"attn": _plain_attn, "store": _plain_store, "sample": _plain_sample}[c["op"]](s)
    from bf16_wire_all_amd import decode
    if c["op"] == "attn":
        decode.attn_paged(s["cache"], s["q"], s["table"], s["lens"], c["max_len"], s["scale"], s["out"],
                          s["workspace"], window=c["window"], sinks=c["sinks"])
        return s["out"]
    if c["op"] == "store":
        decode.qkv_rope_store(s["cache"], s["q"], s["new_k"], s["new_v"], s["positions"], s["cos_sin"], s["slots"],
                              s["q_out"], q_weight=s["wq"], k_weight=s["wk"], eps=s["eps"],
                              interleaved=c["interleaved"])
        return {"q": s["q_out"], "k": s["k"], "v": s["v"]}
    decode.sample_merge(s["s0"], s["s1"], s["params"], s["u"], s["out"], s["workspace"])
    return {"idx": s["out"][:, 1], "prob": s["out"].view(torch.float32)[:, 0]}


# --------------------------------------------------------------------- work

def work(case):
    if case["op"] == "attn":
        d, hq, hkv = case["head_dim"], case["q_heads"], case["kv_heads"]
        tokens = sum(_visible(case))
        cb = 2 if case["kind"] == "bf16" else 1
        pages = sum(-(-n // case["page_tokens"]) for n in _visible(case))
        return {"bytes": tokens * hkv * 2 * d * cb + pages * 4
                + case["rows"] * (hq * d * (2 + (2 if case["out"] == "bf16" else 4)) + 4),
                "flops": 4 * tokens * hq * d}
    if case["op"] == "store":
        t, d, hq, hkv = case["tokens"], case["head_dim"], case["q_heads"], case["kv_heads"]
        cb = 2 if case["kind"] == "bf16" else 1
        elements = t * (hq + 2 * hkv) * d
        return {"bytes": elements * 2 + t * hq * d * 2 + t * 2 * hkv * d * cb + t * (case["rot_dim"] * 4 + 12),
                "flops": 7 * t * (hq + hkv) * d}
    cells = case["rows"] * (case["ncols0"] + case["ncols1"])
    return {"bytes": cells * 2 + case["rows"] * 28, "flops": cells}


# ------------------------------------------------- the definition in 64 bits

def _exact_attn(s):
    c = s["case"]
    d, hkv, p = c["head_dim"], c["kv_heads"], c["page_tokens"]
    group = c["q_heads"] // hkv
    out = torch.zeros((c["rows"], c["q_heads"], d), dtype=torch.float64)
    for r in range(c["rows"]):
        n = int(s["lens"][r])
        tokens = [j for j in range(n) if c["window"] == 0 or j < c["sinks"] or n - j <= c["window"]]
        j = torch.tensor(tokens, device="cuda")
        pages = s["table"][r][torch.div(j, p, rounding_mode="floor")].long()
        for h in range(hkv):
            head = {}
            for name, scale in (("k", s["ks"]), ("v", s["vs"])):
                a = s[name][:, :, h, :]
                a = (a.view(torch.uint8)[pages, j % p].view(torch.float8_e4m3fn) if c["kind"] == "e4m3"
                     else a[pages, j % p])
                head[name] = a.to(torch.float64) * (1.0 if scale is None else float(scale[h]))
            q = s["q"][r, h * group:(h + 1) * group].to(torch.float64)
            z = (q @ head["k"].t().contiguous()) * s["scale"]
            out[r, h * group:(h + 1) * group] = (torch.softmax(z, 1) @ head["v"]).cpu()
    return out


def _exact_store(s):
    c = s["case"]
    d, r, p = c["head_dim"], c["rot_dim"], c["page_tokens"]
    table = s["cos_sin"][s["positions"].long()].to(torch.float64)
    # the rotation as a complex product of each pair
    turn = torch.complex(table[:, :r // 2], table[:, r // 2:])[:, None, :]

    def heads(x, w):
        x = x.to(torch.float64)
        if w is not None:
            norm = torch.sqrt(x.square().sum(-1, keepdim=True) / d + s["eps"])
            x = x / norm * w.to(torch.float64)
        pairs = (x[..., :r].unflatten(-1, (r // 2, 2)) if c["interleaved"]
                 else x[..., :r].unflatten(-1, (2, r // 2)).transpose(-1, -2))
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
        z = z if c["interleaved"] else z.transpose(-1, -2)
        return torch.cat([z.reshape(*x.shape[:-1], r), x[..., r:]], -1)

    def put(cache, scale, x):
        whole = cache.to(torch.float64).reshape(-1, p, c["kv_heads"], d)
        if scale is not None:
            x = torch.clamp(x / scale.to(torch.float64)[None, :, None], -E4M3_MAX, E4M3_MAX)
        flat = whole.contiguous().view(-1, c["kv_heads"], d)
        there = torch.nonzero(s["slots"] >= 0)[:, 0]
        flat[s["slots"][there]] = x[there]
        return flat.view(whole.shape)

    return {"q": heads(s["q"], s["wq"]), "k": put(s["k"], s["ks"], heads(s["new_k"], s["wk"])),
            "v": put(s["v"], s["vs"], s["new_v"].to(torch.float64))}


def _exact_sample(s):
    c = s["case"]
    params = s["params"].cpu().numpy().view(
        [("temperature", "<f4"), ("top_k", "<u4"), ("top_p", "<f4"), ("min_p", "<f4")])
    rows = torch.cat([s["l0"][:, :c["ncols0"]], s["l1"][:, :c["ncols1"]]], 1).float().cpu().numpy().astype(np.float64)
    u = s["u"].cpu().numpy().astype(np.float64)
    idx, prob = np.full(c["rows"], -1, np.int32), np.zeros(c["rows"])
    for r in range(c["rows"]):
        x = rows[r]
        t, k, tp, mp = (float(params[r][f]) for f in ("temperature", "top_k", "top_p", "min_p"))
        order = np.argsort(-x, kind="stable")
        order = order[x[order] > -np.inf]
        if not order.size:
            continue
        if t <= 0:
            order = order[:1]
        w = np.exp((x[order] - x[order[0]]) / (t if t > 0 else 1.0))
        if k > 0:
            w = w[:int(k)]
        if tp < 1:
            sums = np.cumsum(w)
            w = w[:1 + int(np.searchsorted(sums, tp * sums[-1], side="left"))]
        w = w[w >= mp * w[0]]
        sums = np.cumsum(w)
        at = min(int(np.searchsorted(sums, u[r] * sums[-1], side="right")), w.size - 1)
        idx[r], prob[r] = order[at], w[at] / sums[-1]
    return {"idx": idx, "prob": prob}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "sample":
        if case["rows"] * (case["ncols0"] + case["ncols1"]) > 45_000_000:
            return None
        return _exact_sample(s)
    return _exact_attn(s) if case["op"] == "attn" else _exact_store(s)
