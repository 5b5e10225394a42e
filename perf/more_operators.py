"""Cases of the operators for several answers of one prompt: attention over a
shared prefix (attn_shared), a cache's slots in 8 or 4 bits on the wire
(kv_quantize, kv_restore), and the tokens' log probabilities from sharded
logits (logprobs_merge).

`run` computes a case in its plain form (elementary torch operations) where
`own` is false, and through the package where it is true; `exact` is the
definition in 64 bits."""
import math
import random

import numpy as np
import torch

own = False

LARGEST = {8: 448.0, 4: 6.0}   # of an element of so many bits
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------- cases

def _shared(name, mode, rows, groups, prefix, ragged, suffix, q_heads, kv_heads, head_dim, page_tokens, kind, order,
            out="bf16"):
    return {"name": name, "op": "shared", "mode": mode, "rows": rows, "groups": groups, "prefix": prefix,
            "ragged": ragged, "suffix": suffix, "q_heads": q_heads, "kv_heads": kv_heads, "head_dim": head_dim,
            "page_tokens": page_tokens, "kind": kind, "order": order, "out": out}


def _wire(name, mode, tokens, kv_heads, head_dim, page_tokens, kind, order, bits, to_kind="bf16", to_order="heads"):
    return {"name": name, "op": "wire", "mode": mode, "tokens": tokens, "kv_heads": kv_heads, "head_dim": head_dim,
            "page_tokens": page_tokens, "kind": kind, "order": order, "bits": bits, "to_kind": to_kind,
            "to_order": to_order}


def _logprobs(name, rows, ncols0, ncols1, n_tokens, n_top, temperature, masked):
    return {"name": name, "op": "logprobs", "rows": rows, "ncols0": ncols0, "ncols1": ncols1, "n_tokens": n_tokens,
            "n_top": n_top, "temperature": temperature, "masked": masked}


def listed():
    return [
        # two answers to one short prompt: nothing but latency
        _shared("shared two short answers", "answers", 2, 1, 32, False, 9, 8, 1, 128, 16, "bf16", "heads"),
        # 4 requests x 4 drafted positions: rows of one request see its tokens up to their own
        _shared("shared drafted positions", "drafted", 16, 4, 6000, True, 0, 40, 8, 128, 16, "bf16", "heads"),
        # 64 answers sampled for one prompt of 8192 tokens, each at another length
        _shared("shared 64 answers", "answers", 64, 1, 8192, False, 1000, 32, 8, 128, 16, "bf16", "heads"),
        # 24 questions about one long document, hidden size 5120 (40 heads of 128), partials for the all-reduce in F32
        _shared("shared long document f32", "answers", 24, 1, 131056, False, 300, 40, 8, 128, 16, "bf16", "heads",
                out="f32"),
        # a serving batch with three system prompts, 8-bit cache, heads of 64
        _shared("shared system prompts e4m3", "answers", 99, 3, 6016, True, 1500, 64, 8, 64, 32, "e4m3", "tokens"),
        # one page of new tokens for the wire
        _wire("quantize one page", "quantize", 16, 8, 128, 16, "bf16", "heads", 8),
        # a prompt batch of 16384 tokens at 8 heads of 128 leaves for its decode worker
        _wire("quantize prompt 16384", "quantize", 16384, 8, 128, 16, "bf16", "heads", 8),
        # and arrives there, in a cache of whole tokens in 8 bits
        _wire("restore prompt 65521 e4m3", "restore", 65521, 8, 128, 16, "bf16", "heads", 8, "e4m3", "tokens"),
        # a ragged set of an 8-bit cache through a wire of 4 bits into a BF16 one
        _wire("4 bit wire 24001", "both", 24001, 8, 64, 32, "e4m3", "tokens", 4, "bf16", "heads"),
        # 4 requests x 4 drafted positions, the drawn tokens and five alternatives
        _logprobs("logprobs 16 rows", 16, 64768, 64512, 1, 5, "mixed", False),
        # a prompt's tokens scored, no alternatives
        _logprobs("logprobs 2048 prompt rows", 2048, 75968, 75968, 1, 0, "one", False),
        # many rows of a narrow ragged vocabulary under a grammar's mask, the most alternatives
        _logprobs("logprobs narrow masked rows", 333, 2304, 1695, 3, 20, "mixed", True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["shared", "shared", "wire", "logprobs"])
    if op == "shared":
        head_dim = rng.choice([64, 128, 256])
        kv_heads = rng.choice([1, 2, 4, 8])
        q_heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 7, 8, 16, 20])
        page = rng.choice([1, 8, 16, 32, 64, 128])
        mode = rng.choice(["answers", "answers", "drafted"])
        rows = _log(rng, 1, 128)
        groups = min(rows, _log(rng, 1, 16))
        # no more products and no more cache than the largest listed case has
        most = min(24 * 40 * 131056 * 128 // (rows * q_heads * head_dim),
                   131056 * 8 * 128 // (groups * kv_heads * head_dim))
        prefix = _log(rng, 1, max(1, min(131056, most)))
        suffix = _log(rng, 1, max(1, min(4000, 131056 * 8 * 128 // (rows * kv_heads * head_dim))))
        if mode == "answers":
            prefix = max(1, prefix // page) * page
        c = _shared("", mode, rows, groups, prefix, rng.choice([True, False]), suffix if mode == "answers" else 0,
                    q_heads, kv_heads, head_dim, page, rng.choice(["bf16", "e4m3"]), rng.choice(["tokens", "heads"]),
                    rng.choice(["bf16", "bf16", "f32"]))
    elif op == "wire":
        head_dim, kv_heads = rng.choice([64, 128, 256]), rng.choice([1, 2, 4, 8])
        most = 65521 * 8 * 128 // (kv_heads * head_dim)
        mode = rng.choice(["quantize", "restore", "both"])
        tokens = _log(rng, 1, max(1, min(65521, most // (2 if mode == "both" else 1))))
        c = _wire("", mode, tokens, kv_heads, head_dim, rng.choice([1, 8, 16, 32, 64, 128]),
                  rng.choice(["bf16", "e4m3"]), rng.choice(["tokens", "heads"]),
                  8 if mode == "quantize" else rng.choice([4, 8]), rng.choice(["bf16", "e4m3"]),
                  rng.choice(["tokens", "heads"]))
    else:
        n_top = rng.choice([0, 1, 5, 20, 32])
        rows = _log(rng, 1, 512 if n_top else 2048)
        cols = _log(rng, 1000, min(262144, (256 if n_top else 2048) * 151936 // rows))
        n0 = rng.randrange(1, cols)
        c = _logprobs("", rows, n0, cols - n0, rng.choice([0, 1, 1, 2, 4]) if n_top else rng.choice([1, 1, 2]), n_top,
                      rng.choice(["one", "mixed"]), rng.choice([True, False]))
    del c["name"]
    return c


# ------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) & 0x7FFFFFFF)
    return g


def _normal(shape, g, dtype=torch.bfloat16, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _cache(kv_heads, head_dim, page_tokens, kind, order, n_pages, g):
    """K and V of a paged cache as [page, token, head, dim] views, and their scales (8-bit caches)."""
    shape = ((n_pages, page_tokens, kv_heads, head_dim) if order == "tokens" else
             (n_pages, kv_heads, page_tokens, head_dim))
    dt = torch.bfloat16 if kind == "bf16" else torch.float8_e4m3fn
    k, v = _normal(shape, g, dt), _normal(shape, g, dt)
    if order == "heads":
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    if kind == "bf16":
        return k, v, None, None
    ks = torch.rand(kv_heads, generator=g, device="cuda") * 1.5 + 0.25
    vs = torch.rand(kv_heads, generator=g, device="cuda") * 1.5 + 0.25
    return k, v, ks, vs


def _group_sizes(case):
    """Rows of each group: the first groups are larger."""
    rows, n = case["rows"], case["groups"]
    cut = [int(rows * (1 - (1 - i / n) ** 1.3)) if case["ragged"] else rows * i // n for i in range(n + 1)]
    cut = [min(max(c, i), rows - (n - i)) for i, c in enumerate(cut)]
    return [cut[i + 1] - cut[i] for i in range(n)]


def _prefixes(case):
    """Shared tokens of each group, whole pages of them where rows go on in pages of their own."""
    n, top = case["groups"], case["prefix"]
    p = [max(1, int(top * ((i + 1) / n) ** 1.5)) if case["ragged"] else top for i in range(n)]
    if case["mode"] == "answers":
        p = [max(1, x // case["page_tokens"]) * case["page_tokens"] for x in p]
    return p


def _lens(case):
    """Each row's length, the same for every seed but for the order of the answers within the batch."""
    lens, i = [], 0
    for size, p in zip(_group_sizes(case), _prefixes(case)):
        for j in range(size):
            lens.append(p + (j if case["mode"] == "drafted" else
                             max(1, int(case["suffix"] * ((i + 1) / case["rows"]) ** 2))))
            i += 1
    return lens


def _prepare_shared(s, case, seed, g):
    rows, p = case["rows"], case["page_tokens"]
    sizes, prefixes = _group_sizes(case), _prefixes(case)
    own_len = [n - q for n, q in zip(_lens(case), [q for q, size in zip(prefixes, sizes) for _ in range(size)])]
    if case["mode"] == "answers":
        random.Random(int(seed)).shuffle(own_len)
    lens, table, n_pages, r = [], [], 0, 0
    for size, q in zip(sizes, prefixes):
        common = list(range(n_pages, n_pages + -(-(q + (size - 1 if case["mode"] == "drafted" else 0)) // p)))
        n_pages += len(common)
        for _ in range(size):
            lens.append(q + own_len[r])
            mine = -(-lens[-1] // p) - len(common) if case["mode"] == "answers" else 0
            table.append(common + list(range(n_pages, n_pages + mine)))
            n_pages += mine
            r += 1
    n_pages += 3
    width = max(map(len, table))
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    at = np.zeros((rows, width), np.int64)
    for i, t in enumerate(table):
        at[i, :len(t)] = t
    s["table"] = order[torch.from_numpy(at).cuda()]
    s["k"], s["v"], s["ks"], s["vs"] = _cache(case["kv_heads"], case["head_dim"], p, case["kind"], case["order"],
                                              n_pages, g)
    s["sizes"], s["prefixes"], s["host_lens"], s["max_len"] = sizes, prefixes, lens, max(lens)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["starts"] = torch.tensor([sum(sizes[:i]) for i in range(len(sizes) + 1)], dtype=torch.int32, device="cuda")
    s["shared"] = torch.tensor(prefixes, dtype=torch.int32, device="cuda")
    s["q"] = _normal((rows, case["q_heads"], case["head_dim"]), g, scale=1.5)
    s["scale"] = case["head_dim"] ** -0.5
    s["out"] = torch.empty((rows, case["q_heads"], case["head_dim"]), device="cuda",
                           dtype=torch.bfloat16 if case["out"] == "bf16" else torch.float32)
    if own:
        from bf16_wire_all_amd import decode
        s["cache"] = decode.kv_cache(s["k"], s["v"], s["ks"], s["vs"])
        need = decode.attn_shared_workspace_bytes(s["cache"], rows, len(sizes), case["q_heads"], s["max_len"])
        s["workspace"] = torch.empty(max(16, need), dtype=torch.uint8, device="cuda")


def _record_bytes(case):
    n = 2 * case["kv_heads"] * case["head_dim"]
    return -(-(n * case["bits"] // 8 + n // 32) // 16) * 16


def _prepare_wire(s, case, seed, g):
    t, p, bits = case["tokens"], case["page_tokens"], case["bits"]
    n_pages = -(-t // p) + 5

    def slots():
        # whole pages, in any order of them
        pages = torch.randperm(n_pages, generator=g, device="cuda")[:-(-t // p)]
        return (pages[:, None] * p + torch.arange(p, device="cuda")[None, :]).flatten()[:t].contiguous()

    s["records"] = torch.zeros((t, _record_bytes(case)), dtype=torch.uint8, device="cuda")
    if case["mode"] != "restore":
        s["k"], s["v"], s["ks"], s["vs"] = _cache(case["kv_heads"], case["head_dim"], p, case["kind"], case["order"],
                                                  n_pages, g)
        # a few channels far larger than the rest, as keys have them
        wide = 1.0 + 15.0 * (torch.rand(case["head_dim"], generator=g, device="cuda") < 0.05)
        for x in (s["k"], s["v"]):
            x.copy_((x.float() * wide).clamp(-448.0, 448.0).to(x.dtype))
        s["slots"] = slots()
    else:
        n = 2 * case["kv_heads"] * case["head_dim"]
        data = torch.randint(0, 256, (t, n * bits // 8), generator=g, device="cuda", dtype=torch.uint8)
        if bits == 8:
            data = torch.where((data & 0x7F) == 0x7F, 0x38, data)   # no NaN
        s["records"][:, :n * bits // 8] = data
        s["records"][:, n * bits // 8:n * bits // 8 + n // 32] = torch.randint(
            110, 122, (t, n // 32), generator=g, device="cuda").to(torch.uint8)
    if case["mode"] != "quantize":
        s["tk"], s["tv"], s["tks"], s["tvs"] = _cache(case["kv_heads"], case["head_dim"], p, case["to_kind"],
                                                      case["to_order"], n_pages, g)
        s["to_slots"] = slots()
        if t > 8:
            s["to_slots"][::97] = -1   # tokens that another rank keeps
    if own:
        from bf16_wire_all_amd import decode
        if "k" in s:
            s["cache"] = decode.kv_cache(s["k"], s["v"], s["ks"], s["vs"])
        if "tk" in s:
            s["to_cache"] = decode.kv_cache(s["tk"], s["tv"], s["tks"], s["tvs"])


def _prepare_logprobs(s, case, seed, g):
    rows, n0, n1 = case["rows"], case["ncols0"], case["ncols1"]
    shards = []
    for n in (n0, n1):
        x = torch.randn((rows, -(-n // 8) * 8), generator=g, device="cuda")
        x.mul_(2.5).add_(8.0 * (torch.rand(x.shape, generator=g, device="cuda") < 2e-4))
        if case["masked"]:
            x.masked_fill_(torch.rand(x.shape, generator=g, device="cuda") < 0.7, -math.inf)
        shards.append(x.to(torch.bfloat16))
    s["l0"], s["l1"] = shards
    s["temperature"] = None
    if case["temperature"] == "mixed":
        s["temperature"] = torch.rand(rows, generator=g, device="cuda") * 1.5 + 0.5
    s["tokens"] = torch.randint(0, n0 + n1, (rows, case["n_tokens"]), generator=g, device="cuda").to(torch.int32)
    s["token_out"] = torch.zeros((rows, case["n_tokens"], 2), dtype=torch.int32, device="cuda")
    s["top_out"] = torch.zeros((rows, case["n_top"], 2), dtype=torch.int32, device="cuda")
    s["entropy"] = torch.zeros(rows, device="cuda")
    if own:
        from bf16_wire_all_amd import decode
        s["s0"] = decode.shard(s["l0"], n0, 0)
        s["s1"] = decode.shard(s["l1"], n1, n0)
        need = decode.logprobs_workspace_bytes(rows, n0, n1, case["n_tokens"], case["n_top"])
        s["workspace"] = torch.empty(max(16, need), dtype=torch.uint8, device="cuda")


def prepare(case, seed):
    s = {"case": case}
    {"shared": _prepare_shared, "wire": _prepare_wire, "logprobs": _prepare_logprobs}[case["op"]](s, case, seed,
                                                                                                  _gen(seed))
    return s


# -------------------------------------------------------------- plain forms

def _read(s, which, page, slot):
    """Keys or values of slots in 32 bits."""
    x = s[which]
    x = x[page, slot] if s["case"]["kind"] == "bf16" else x.view(torch.uint8)[page, slot].view(torch.float8_e4m3fn)
    x = x.float()
    scale = s[which + "s"]
    return x if scale is None else x * scale[:, None]


def _part(q, k, v, there, scale):
    """(max, sum, weighted sum) of q [n, kv, m, d] over k, v [n, t, kv, d]; there [n, t] or None."""
    score = torch.matmul(q, k.permute(0, 2, 3, 1)) * scale
    if there is not None:
        score = score.masked_fill(~there[:, None, None, :], -math.inf)
    m = score.amax(-1, keepdim=True)
    w = torch.exp(score - m.clamp(min=-3e38))
    return m, w.sum(-1, keepdim=True), torch.matmul(w, v.permute(0, 2, 1, 3))


def _plain_shared(s):
    c = s["case"]
    kv, d, p = c["kv_heads"], c["head_dim"], c["page_tokens"]
    group = c["q_heads"] // kv
    r = 0
    for size, q_len in zip(s["sizes"], s["prefixes"]):
        q = s["q"][r:r + size].float().view(size, kv, group, d)
        # the shared tokens once, for all of the group's heads
        j = torch.arange(q_len, device="cuda")
        page = s["table"][r, j // p].long()
        k, v = _read(s, "k", page, j % p), _read(s, "v", page, j % p)
        all_q = q.permute(1, 0, 2, 3).reshape(1, kv, size * group, d)
        m0, l0, o0 = (x.view(kv, size, group, -1).permute(1, 0, 2, 3) for x in _part(all_q, k[None], v[None], None,
                                                                                     s["scale"]))
        # each row's own tokens
        rest = [n - q_len for n in s["host_lens"][r:r + size]]
        if max(rest) > 0:
            i = torch.arange(max(rest), device="cuda")[None, :]
            there = i < s["lens"][r:r + size, None] - q_len
            token = torch.where(there, i + q_len, 0)
            page = torch.gather(s["table"][r:r + size].long(), 1, token // p)
            m1, l1, o1 = _part(q, _read(s, "k", page, token % p), _read(s, "v", page, token % p), there, s["scale"])
            m = torch.maximum(m0, m1)
            f0, f1 = torch.exp(m0 - m), torch.exp(m1 - m)
            l0, o0 = l0 * f0 + l1 * f1, o0 * f0 + o1 * f1
        s["out"][r:r + size] = (o0 / l0).reshape(size, c["q_heads"], d)
        r += size
    return s["out"]


def _plain_quantize(s):
    c = s["case"]
    t, p, bits = c["tokens"], c["page_tokens"], c["bits"]
    page, slot = s["slots"] // p, s["slots"] % p
    x = torch.stack([_read(s, "k", page, slot), _read(s, "v", page, slot)], 1).view(t, -1, 32)
    # the smallest power of two that brings the largest element to LARGEST at most
    man, e = torch.frexp(x.abs().amax(-1))
    e = e - (9 if bits == 8 else 3) + (man > (0.875 if bits == 8 else 0.75))
    e = torch.where(man == 0, -127, e.clamp(min=-127))
    y = torch.ldexp(torch.ldexp(x, -(e // 2)[..., None]), -(e - e // 2)[..., None])
    if bits == 8:
        data = y.to(torch.float8_e4m3fn).view(torch.uint8).view(t, -1)
    else:
        a = y.abs()
        step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
        a = torch.round(a / step) * step
        code = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
        code = code | (torch.signbit(y).to(torch.uint8) << 3)
        data = (code[..., 0::2] | (code[..., 1::2] << 4)).view(t, -1)
    n = data.shape[1]
    s["records"][:, :n] = data
    s["records"][:, n:n + e.shape[1]] = (e + 127).to(torch.uint8)


def _plain_restore(s):
    c = s["case"]
    t, p, bits, h, d = c["tokens"], c["page_tokens"], c["bits"], c["kv_heads"], c["head_dim"]
    n = 2 * h * d
    data = s["records"][:, :n * bits // 8].contiguous()
    e = s["records"][:, n * bits // 8:n * bits // 8 + n // 32].to(torch.int32) - 127
    if bits == 8:
        x = data.view(torch.float8_e4m3fn).float()
    else:
        table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device="cuda")
        x = table[torch.stack([data & 15, data >> 4], -1).view(t, n).int()]
    x = x.view(t, -1, 32)
    x = torch.ldexp(torch.ldexp(x, (e // 2)[..., None]), (e - e // 2)[..., None]).view(t, 2, h, d)
    kept = s["to_slots"] >= 0
    page, slot = s["to_slots"][kept] // p, s["to_slots"][kept] % p
    for i, which in enumerate(("tk", "tv")):
        y = x[kept, i]
        if c["to_kind"] == "bf16":
            s[which][page, slot] = y.to(torch.bfloat16)
        else:
            y = (y / s[which + "s"][:, None]).clamp(-448.0, 448.0)
            s[which].view(torch.uint8)[page, slot] = y.to(torch.float8_e4m3fn).view(torch.uint8)


def _wire_out(s):
    c = s["case"]
    if c["mode"] != "quantize":
        return {"k": s["tk"], "v": s["tv"]}
    n = 2 * c["kv_heads"] * c["head_dim"]
    return {"data": s["records"][:, :n].view(torch.float8_e4m3fn), "exponents": s["records"][:, n:n + n // 32]}


def _plain_wire(s):
    if s["case"]["mode"] != "restore":
        _plain_quantize(s)
    if s["case"]["mode"] != "quantize":
        _plain_restore(s)
    return _wire_out(s)


def _plain_logprobs(s):
    c = s["case"]
    x = torch.cat([s["l0"][:, :c["ncols0"]], s["l1"][:, :c["ncols1"]]], 1).float()
    top = x.amax(1, keepdim=True)
    z = x - top
    if s["temperature"] is not None:
        z = z / s["temperature"][:, None]
    w = torch.exp(z)
    total = w.sum(1, keepdim=True)
    log_total = torch.log(total)
    entropy = log_total[:, 0] - (w * z.clamp(min=-1e30)).sum(1) / total[:, 0]
    out = {"entropy": entropy}
    if c["n_tokens"]:
        ids = s["tokens"].long()
        mine = torch.gather(x, 1, ids)
        before, n = [], torch.arange(x.shape[1], device="cuda")[None, :]
        for i in range(c["n_tokens"]):
            before.append(((x > mine[:, i:i + 1]) | ((x == mine[:, i:i + 1]) & (n < ids[:, i:i + 1]))).sum(1))
        there = mine > -math.inf
        out["logprob"] = torch.gather(z, 1, ids) - log_total
        out["rank"] = torch.where(there, torch.stack(before, 1), -1).to(torch.int32)
    if c["n_top"]:
        # the row's order: larger first, then the lower id
        values, ids = torch.sort(x, dim=1, descending=True, stable=True)
        values, ids = values[:, :c["n_top"]], ids[:, :c["n_top"]]
        z = values - top
        if s["temperature"] is not None:
            z = z / s["temperature"][:, None]
        out["top_id"] = torch.where(values > -math.inf, ids, -1).to(torch.int32)
        out["top_logprob"] = z - log_total
    return out


def run(state):
    s = state
    c = s["case"]
    if not own:
        return {"shared": _plain_shared, "wire": _plain_wire, "logprobs": _plain_logprobs}[c["op"]](s)
    from bf16_wire_all_amd import decode
    if c["op"] == "shared":
        decode.attn_shared(s["cache"], s["q"], s["table"], s["lens"], s["max_len"], s["starts"], s["shared"],
                           s["scale"], s["out"], s["workspace"])
        return s["out"]
    if c["op"] == "wire":
        if c["mode"] != "restore":
            decode.kv_quantize(s["cache"], s["slots"], s["records"], c["bits"])
        if c["mode"] != "quantize":
            decode.kv_restore(s["records"], c["bits"], s["to_cache"], s["to_slots"])
        return _wire_out(s)
    decode.logprobs_merge(s["s0"], s["s1"], s["tokens"], s["token_out"], s["top_out"], s["entropy"], s["workspace"],
                          temperature=s["temperature"])
    out = {"entropy": s["entropy"]}
    if c["n_tokens"]:
        out["logprob"], out["rank"] = s["token_out"].view(torch.float32)[..., 0], s["token_out"][..., 1]
    if c["n_top"]:
        out["top_id"], out["top_logprob"] = s["top_out"][..., 1], s["top_out"].view(torch.float32)[..., 0]
    return out


# --------------------------------------------------------------------- work

def work(case):
    if case["op"] == "shared":
        d, hq, hkv, p = case["head_dim"], case["q_heads"], case["kv_heads"], case["page_tokens"]
        sizes, prefixes, lens = _group_sizes(case), _prefixes(case), _lens(case)
        cb = 2 if case["kind"] == "bf16" else 1
        if case["mode"] == "drafted":
            # the rows of a request read the same pages to the end
            once = sum(q + size - 1 for q, size in zip(prefixes, sizes))
        else:
            once = sum(prefixes) + sum(lens) - sum(q * size for q, size in zip(prefixes, sizes))
        return {"bytes": once * hkv * 2 * d * cb + -(-once // p) * 4
                + case["rows"] * (hq * d * (2 + (2 if case["out"] == "bf16" else 4)) + 4),
                "flops": 4 * sum(lens) * hq * d}
    if case["op"] == "wire":
        t, n = case["tokens"], 2 * case["kv_heads"] * case["head_dim"]
        size = {"bf16": 2, "e4m3": 1}
        record = n * case["bits"] // 8 + n // 32
        moved = 0
        if case["mode"] != "restore":
            moved += t * (n * size[case["kind"]] + 8)
        if case["mode"] != "quantize":
            moved += t * (n * size[case["to_kind"]] + 8)
        return {"bytes": moved + t * record * (2 if case["mode"] == "both" else 1),
                "flops": 2 * t * n * (2 if case["mode"] == "both" else 1)}
    cells = case["rows"] * (case["ncols0"] + case["ncols1"])
    return {"bytes": cells * 2 + case["rows"] * (8 + 12 * case["n_tokens"] + 8 * case["n_top"]), "flops": 5 * cells}


# ------------------------------------------------- the definition in 64 bits

def _exact_shared(s):
    c = s["case"]
    d, hkv, p = c["head_dim"], c["kv_heads"], c["page_tokens"]
    group = c["q_heads"] // hkv
    out = torch.zeros((c["rows"], c["q_heads"], d), dtype=torch.float64)
    for r in range(c["rows"]):
        # every row by itself, over its own page table
        j = torch.arange(int(s["lens"][r]), device="cuda")
        pages = s["table"][r][torch.div(j, p, rounding_mode="floor")].long()
        for h in range(hkv):
            head = {}
            for name in ("k", "v"):
                a = s[name][:, :, h, :]
                a = (a.view(torch.uint8)[pages, j % p].view(torch.float8_e4m3fn) if c["kind"] == "e4m3"
                     else a[pages, j % p])
                head[name] = a.to(torch.float64) * (1.0 if s[name + "s"] is None else float(s[name + "s"][h]))
            q = s["q"][r, h * group:(h + 1) * group].to(torch.float64)
            z = (q @ head["k"].t().contiguous()) * s["scale"]
            out[r, h * group:(h + 1) * group] = (torch.softmax(z, 1) @ head["v"]).cpu()
    return out


def _exact_code(y, bits):
    """The nearest element (of even code where two are as near) of each y, as its number in the order of magnitudes."""
    if bits == 8:
        table = [(m / 8) * 2.0 ** -6 for m in range(8)] + [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16)
                                                           for m in range(8)]
        table = table[:-1]
    else:
        table = list(E2M1)
    t = torch.tensor(table, dtype=torch.float64, device=y.device)
    a = y.abs()
    hi = torch.bucketize(a, t).clamp(1, len(table) - 1)
    to_lo, to_hi = a - t[hi - 1], t[hi] - a
    up = (to_hi < to_lo) | ((to_hi == to_lo) & (hi % 2 == 0))
    return torch.where(up, hi, hi - 1), t


def _exact_wire(s):
    c = s["case"]
    t, p, bits, h, d = c["tokens"], c["page_tokens"], c["bits"], c["kv_heads"], c["head_dim"]
    if c["mode"] != "restore":
        parts = []
        for which in ("k", "v"):
            x = s[which].to(torch.float64).reshape(-1, p, h, d).contiguous().view(-1, h, d)[s["slots"]]
            if s[which + "s"] is not None:   # a product in binary32, as the definition has it
                x = (x * s[which + "s"].to(torch.float64)[None, :, None]).to(torch.float32).to(torch.float64)
            parts.append(x)
        x = torch.stack(parts, 1).view(t, -1, 32)
        ratio = x.abs().amax(-1) / LARGEST[bits]
        e = torch.where(ratio > 0, torch.ceil(torch.log2(ratio)), -127.0)
        e = torch.where(ratio > torch.exp2(e), e + 1, e)     # where the logarithm's rounding
        e = torch.where(ratio <= torch.exp2(e - 1), e - 1, e).clamp(min=-127)   # crossed a whole number
        y = x / torch.exp2(e)[..., None]
        code, table = _exact_code(y, bits)
        value = torch.copysign(table[code], y)
        if c["mode"] == "quantize":
            return {"data": value.view(t, -1), "exponents": (e + 127).to(torch.uint8)}
        x = value * torch.exp2(e)[..., None]
    else:
        n = 2 * h * d
        raw = s["records"].cpu().numpy().astype(np.int64)
        data, e = raw[:, :n * bits // 8], raw[:, n * bits // 8:n * bits // 8 + n // 32] - 127
        if bits == 8:
            man, ex = data & 7, (data >> 3) & 15
            value = np.where(ex == 0, man * 2.0 ** -9, (8 + man) * 2.0 ** (ex - 10))
            value = np.where(data & 128, -value, value)
        else:
            code = np.stack([data & 15, data >> 4], -1).reshape(t, n)
            value = np.array(E2M1)[code & 7] * np.where(code & 8, -1.0, 1.0)
        x = torch.from_numpy(value.reshape(t, -1, 32) * 2.0 ** e[..., None]).cuda()
    x = x.view(t, 2, h, d)
    out = {}
    kept = torch.nonzero(s["to_slots"] >= 0)[:, 0]
    for i, which in enumerate(("tk", "tv")):
        whole = s[which].to(torch.float64).reshape(-1, p, h, d).contiguous()
        y = x[:, i]
        if s[which + "s"] is not None:
            y = torch.clamp(y / s[which + "s"].to(torch.float64)[None, :, None], -448.0, 448.0)
        whole.view(-1, h, d)[s["to_slots"][kept]] = y[kept]
        out[which[1:]] = whole
    return out


def _exact_logprobs(s):
    c = s["case"]
    x = torch.cat([s["l0"][:, :c["ncols0"]], s["l1"][:, :c["ncols1"]]], 1)
    names = ["entropy"] + ["logprob", "rank"] * (c["n_tokens"] > 0) + ["top_id", "top_logprob"] * (c["n_top"] > 0)
    out = {name: [] for name in names}
    for r in range(c["rows"]):
        z = x[r].to(torch.float64)
        if s["temperature"] is not None:
            z = z / float(s["temperature"][r])
        lse = torch.logsumexp(z, 0)
        lp = z - lse
        p = torch.exp(lp)
        out["entropy"].append(-(p * torch.where(p > 0, lp, 0.0)).sum())
        if c["n_tokens"]:
            ids = s["tokens"][r].long()
            out["logprob"].append(lp[ids])
            raw = x[r].float()
            rank = []
            for i in ids.tolist():
                rank.append(int((raw > raw[i]).sum() + (raw[:i] == raw[i]).sum()) if raw[i] > -math.inf else -1)
            out["rank"].append(torch.tensor(rank, dtype=torch.int32))
        if c["n_top"]:
            # the order as one whole number each: the value's, then the id's
            bits = x[r].view(torch.int16).long() & 0xFFFF
            bits = torch.where(bits == 0x8000, 0, bits)
            key = torch.where(bits >= 0x8000, 0x8000 - bits, bits) * (1 << 32) - torch.arange(len(bits), device="cuda")
            ids = torch.topk(key, c["n_top"])[1]
            out["top_logprob"].append(lp[ids])
            out["top_id"].append(torch.where(x[r][ids].float() > -math.inf, ids, -1).to(torch.int32))
    return {name: torch.stack(v).cpu() for name, v in out.items()}


def exact(case, seed):
    if case["op"] == "logprobs" and case["rows"] * (case["ncols0"] + case["ncols1"]) > 350_000_000:
        return None
    s = prepare(case, seed)
    return {"shared": _exact_shared, "wire": _exact_wire, "logprobs": _exact_logprobs}[case["op"]](s)
