"""GPU: the decode-step operators one after the other, as a decode worker runs
them.  A prompt worker stores its prompts' keys and values, xfer_paged_copy
moves the pages to other page numbers of a second cache, and every step then
stores one token of each request, attends, multiplies by a head and samples
the token that the next step takes.  Each operator's result is compared with
its formulas in 64 bits, from what it read on the device; the step captured
in a graph and replayed has to give the eager run's bits."""
from concurrent.futures import ThreadPoolExecutor

import numpy as np
import pytest
import torch

import bf16_wire_all_amd as x
from bf16_wire_all_amd import decode
from tests import decode_reference as ref
from tests.gpu_util import say

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
HQ, HKV, PAGE, VOCAB, SPLIT = 8, 2, 16, 1000, 603
EPS = 1e-6
PARAMS = [(0.8, 50, 0.95, 0.02), (1.0, 0, 1.0, 0.0), (0.0, 0, 1.0, 0.0), (1.3, 0, 0.9, 0.01)]


def wide(t):
    return t.cpu().float().numpy().astype(np.float64)


class Worker:
    """A cache whose pages hold [keys, values][head][slot][dim], so that a page is one copy."""

    def __init__(self, n_pages, d, kind, scales):
        dtype = torch.bfloat16 if kind == "bf16" else torch.float8_e4m3fn
        size = 2 if kind == "bf16" else 1
        self.bytes = torch.zeros((n_pages, 2, HKV, PAGE, d * size), dtype=torch.uint8, device=DEV)
        self.pages = self.bytes.view(dtype)
        self.page_bytes = 2 * HKV * PAGE * d * size
        self.cache = decode.kv_cache(self.pages[:, 0].transpose(1, 2), self.pages[:, 1].transpose(1, 2), *scales)

    def region(self):
        return self.pages.data_ptr(), self.pages.shape[0] * self.page_bytes


class Step:
    """One decode step of all requests, on buffers that stay where they are."""

    def __init__(self, worker, table, lens, embed, head, table_cs, weights, d, window, sinks):
        rows = lens.numel()
        self.w, self.table, self.embed, self.head, self.cs, self.weights = worker, table, embed, head, table_cs, weights
        self.d, self.window, self.sinks, self.rows = d, window, sinks, rows
        self.lens, self.tok = lens.clone(), torch.arange(rows, dtype=torch.int32, device=DEV)
        self.positions = torch.zeros(rows, dtype=torch.int32, device=DEV)
        self.slots = torch.zeros(rows, dtype=torch.int64, device=DEV)
        self.fused = torch.zeros((rows, (HQ + 2 * HKV) * d), dtype=torch.bfloat16, device=DEV)
        self.q_out = torch.zeros((rows, HQ, d), dtype=torch.bfloat16, device=DEV)
        self.out = torch.zeros((rows, HQ, d), dtype=torch.bfloat16, device=DEV)
        self.logits = torch.zeros((rows, VOCAB + 16), dtype=torch.bfloat16, device=DEV)
        self.u = torch.zeros(rows, dtype=torch.float32, device=DEV)
        params = np.array([PARAMS[r % len(PARAMS)] for r in range(rows)], dtype=decode.SAMPLE_PARAMS)
        self.params = params
        self.dparams = torch.from_numpy(params.view(np.uint8).copy()).to(DEV)
        self.sampled = torch.zeros((rows, 2), dtype=torch.int32, device=DEV)
        self.max_len = table.shape[1] * PAGE
        self.attn_ws = torch.zeros(max(16, decode.attn_workspace_bytes(worker.cache, rows, HQ, self.max_len, window,
                                                                       sinks)), dtype=torch.uint8, device=DEV)
        self.sample_ws = torch.zeros(decode.sample_workspace_bytes(rows, SPLIT, VOCAB - SPLIT), dtype=torch.uint8,
                                     device=DEV)
        self.shards = decode.shard(self.logits[:, :SPLIT + 5], SPLIT, 0), decode.shard(
            self.logits[:, 608:], VOCAB - SPLIT, SPLIT)

    def split(self):
        f, d = self.fused, self.d
        return (f[:, :HQ * d].view(-1, HQ, d), f[:, HQ * d:(HQ + HKV) * d].view(-1, HKV, d),
                f[:, (HQ + HKV) * d:].view(-1, HKV, d))

    def run(self):
        torch.index_select(self.embed, 0, self.tok, out=self.fused)
        self.positions.copy_(self.lens)
        page = self.table.gather(1, (self.lens // PAGE).long()[:, None])[:, 0]
        self.slots.copy_(page.long() * PAGE + self.lens % PAGE)
        self.lens.add_(1)
        q, k, v = self.split()
        decode.qkv_rope_store(self.w.cache, q, k, v, self.positions, self.cs, self.slots, self.q_out, *self.weights,
                              eps=EPS)
        decode.attn_paged(self.w.cache, self.q_out, self.table, self.lens, self.max_len, self.d ** -0.5, self.out,
                          self.attn_ws, window=self.window, sinks=self.sinks)
        product = torch.matmul(self.out.view(self.rows, -1), self.head)
        # the second shard begins at a multiple of 8 elements
        self.logits[:, :SPLIT].copy_(product[:, :SPLIT])
        self.logits[:, 608:608 + VOCAB - SPLIT].copy_(product[:, SPLIT:])
        decode.sample_merge(*self.shards, self.dparams, self.u, self.sampled, self.sample_ws)
        self.tok.copy_(self.sampled[:, 1])

    def state(self):
        return [t.clone() for t in (self.w.bytes, self.lens, self.tok)]

    def restore(self, s):
        self.w.bytes.copy_(s[0])
        self.lens.copy_(s[1])
        self.tok.copy_(s[2])

    def results(self):
        return [t.clone() for t in (self.q_out.view(torch.int16), self.out.view(torch.int16),
                                    self.logits.view(torch.int16), self.sampled, self.lens,
                                    self.w.bytes)]

    def row_of_cache(self, r, which, scale):
        """Row r's keys (0) or values (1) in the values they stand for, [tokens, heads, D]."""
        n = int(self.lens[r])
        pages = self.table[r, :-(-n // PAGE)].long()
        held = self.w.bytes[pages, which].cpu().view(self.w.pages.dtype)
        a = wide(held.transpose(1, 2).reshape(-1, HKV, self.d)[:n])
        return a if scale is None else a * wide(scale)[:, None]


@pytest.mark.parametrize("d,kind,window,sinks", [(128, "bf16", 0, 0), (64, "e4m3", 24, 3), (256, "bf16", 0, 0)])
def test_prompts_moved_and_continued(d, kind, window, sinks):
    say("decode step", d, kind, window, sinks)
    g = torch.Generator().manual_seed(d)
    prompts = [37, 1, 16, 63]
    steps, rows = 5, len(prompts)
    scales = (None, None)
    if kind == "e4m3":
        scales = tuple((torch.rand(HKV, generator=g) * 0.02 + 0.03).to(DEV) for _ in range(2))
    embed = torch.randn((VOCAB, (HQ + 2 * HKV) * d), generator=g).to(torch.bfloat16).to(DEV)
    head = (torch.randn((HQ * d, VOCAB), generator=g) * 0.2).to(torch.bfloat16).to(DEV)
    angle = torch.arange(256)[:, None] * 10000.0 ** (-torch.arange(d // 2) / (d // 2))
    cs = torch.cat([angle.cos(), angle.sin()], 1).float().contiguous().to(DEV)
    weights = tuple((torch.rand(d, generator=g) + 0.5).to(torch.bfloat16).to(DEV) for _ in range(2))

    # the prompts' keys and values, all tokens in one call
    used = [-(-n // PAGE) for n in prompts]
    prompt = Worker(sum(used) + 3, d, kind, scales)
    src = torch.randperm(sum(used) + 3, generator=g)[:sum(used)]
    tokens = torch.randint(0, VOCAB, (sum(prompts),), generator=g).to(DEV)
    fused = embed[tokens]
    pos, slots, first = [], [], 0
    for n, pages in zip(prompts, used):
        j = torch.arange(n)
        pos.append(j)
        slots.append(src[first + j // PAGE] * PAGE + j % PAGE)
        first += pages
    pos, slots = torch.cat(pos).int().to(DEV), torch.cat(slots).to(DEV)
    q, k, v = (fused[:, a * d:b * d].view(-1, b - a, d) for a, b in ((0, HQ), (HQ, HQ + HKV), (HQ + HKV, HQ + 2 * HKV)))
    decode.qkv_rope_store(prompt.cache, q, k, v, pos, cs, slots, torch.empty_like(q).contiguous(), *weights, eps=EPS)

    # their pages at other numbers of the decode worker's cache
    width = -(-(max(prompts) + steps) // PAGE)
    decoder = Worker(rows * width + 5, d, kind, scales)
    numbers = torch.randperm(rows * width + 5, generator=g)[:rows * width].view(rows, width)
    dst = torch.cat([numbers[r, :used[r]] for r in range(rows)])
    plan = x.pages_prepare(prompt.page_bytes, prompt.region(), src.numpy(), prompt.page_bytes, 0, decoder.region(),
                           dst.numpy(), decoder.page_bytes, 0,
                           torch.zeros(x.pages_plan_bytes(len(src)), dtype=torch.uint8, device=DEV))
    x.paged_copy(plan)

    step = Step(decoder, numbers.int().to(DEV), torch.tensor(prompts, dtype=torch.int32, device=DEV), embed, head, cs,
                weights, d, window, sinks)
    us = torch.rand((steps, rows), generator=g).to(DEV)
    begin = step.state()
    inputs = [list(part) for part in torch.split(fused, prompts)]   # each row's projections, token by token
    ids = np.arange(VOCAB)
    eager = []
    for i in range(steps):
        step.u.copy_(us[i])
        step.run()
        torch.cuda.synchronize()
        eager.append(step.results())
        for r in range(rows):
            inputs[r].append(step.fused[r].clone())
            n = len(inputs[r])
            assert int(step.lens[r]) == n
            rowin = wide(torch.stack(inputs[r]))
            at = np.arange(n)
            # the queries of the new token, the keys and values of all
            y, mag = ref.rope_heads(rowin[-1:, :HQ * d].reshape(1, HQ, d), wide(weights[0]), EPS, cs.cpu().numpy(),
                                    at[-1:], d, False)
            got_q = wide(step.q_out[r])
            assert np.all(np.abs(got_q - y[0]) <= ref.rope_tolerance(y[0], mag[0], "bf16")), ("queries", i, r)
            keys, values = (step.row_of_cache(r, w, scales[w]) for w in range(2))
            y, mag = ref.rope_heads(rowin[:, HQ * d:(HQ + HKV) * d].reshape(n, HKV, d), wide(weights[1]), EPS,
                                    cs.cpu().numpy(), at, d, False)
            vals = rowin[:, (HQ + HKV) * d:].reshape(n, HKV, d)
            ks, vs = (1.0 if s is None else wide(s)[:, None] for s in scales)
            assert np.all(np.abs(keys - y) <= ks * ref.rope_tolerance(y / ks, mag / ks, kind)), ("keys", i, r)
            assert np.all(np.abs(values - vals) <= vs * ref.rope_tolerance(vals / vs, np.abs(vals / vs), kind))
            # attention over what the cache holds
            seen = ref.visible(n, window, sinks)
            o, tol = ref.attention(got_q, keys[seen], values[seen], d ** -0.5)
            tol = tol * (1 + ref.HALF["bf16"]) + ref.HALF["bf16"] * np.abs(o)
            assert np.all(np.abs(wide(step.out[r]) - o) <= tol), ("attention", i, r)
            # the draw from the logits that there are
            row = wide(step.logits[r])
            p = [float(f) for f in step.params[r]]
            idx, prob, margin = ref.sample(np.concatenate([row[:SPLIT], row[608:608 + VOCAB - SPLIT]]), ids, p[0],
                                           int(p[1]), p[2], p[3], float(us[i, r]))
            got = step.sampled[r].cpu().numpy().view(decode.SAMPLED)[0]
            assert margin > 1e-12 and got["idx"] == idx, ("sample", i, r, got, idx)
            assert abs(got["prob"] - prob) <= 2.0 ** -23 * prob
            assert int(step.tok[r]) == idx

    # the same steps from a graph, with other work between the replays
    stream = torch.cuda.Stream()
    step.restore(begin)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step.run()
    step.restore(begin)
    for i in range(steps):
        step.u.copy_(us[i])
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(step.results(), eager[i]):
            assert torch.equal(a, b), ("replay", i)
        step.attn_ws.fill_(0xFF)
        step.sample_ws.fill_(0xFF)


def test_two_workers_at_once():
    """Two threads with streams, caches and workspaces of their own: each gets the bits that it gets alone."""
    say("decode step, two workers")
    d, rows, steps = 128, 3, 12
    g = torch.Generator().manual_seed(9)
    embed = torch.randn((VOCAB, (HQ + 2 * HKV) * d), generator=g).to(torch.bfloat16).to(DEV)
    head = (torch.randn((HQ * d, VOCAB), generator=g) * 0.2).to(torch.bfloat16).to(DEV)
    angle = torch.arange(4096)[:, None] * 10000.0 ** (-torch.arange(d // 2) / (d // 2))
    cs = torch.cat([angle.cos(), angle.sin()], 1).float().contiguous().to(DEV)
    workers = []
    for w in range(2):
        decoder = Worker(rows * 200 + 3, d, "bf16", (None, None))
        fill = torch.randn(decoder.pages.shape, generator=g).to(torch.bfloat16)
        decoder.pages.copy_(fill)
        numbers = torch.randperm(rows * 200 + 3, generator=g)[:rows * 200].view(rows, 200).int().to(DEV)
        lens = torch.tensor([2900 - 7 * w, 5 + w, 900], dtype=torch.int32, device=DEV)
        workers.append(Step(decoder, numbers, lens, embed, head, cs, (None, None), d, 0, 0))
    us = torch.rand((steps, rows), generator=g).to(DEV)

    def go(step, stream):
        with torch.cuda.stream(stream):
            got = []
            for i in range(steps):
                step.u.copy_(us[i])
                step.run()
                got.append(step.results())
            stream.synchronize()
        return got

    begins = [s.state() for s in workers]
    streams = [torch.cuda.Stream() for _ in workers]
    torch.cuda.synchronize()
    alone = []
    for s, stream in zip(workers, streams):
        alone.append(go(s, stream))
    for s, b in zip(workers, begins):
        s.restore(b)
    torch.cuda.synchronize()
    with ThreadPoolExecutor(2) as ex:
        both = list(ex.map(go, workers, streams))
    for a, b in zip(alone, both):
        for i in range(steps):
            assert all(torch.equal(p, q) for p, q in zip(a[i], b[i])), ("step", i)
