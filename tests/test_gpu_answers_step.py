"""GPU: the operators of many answers to one prompt, one after the other, as
they are used.  A prompt worker stores its prompts' keys and values, sends them
as records of 8 or 4 bits, a decode worker restores them into its cache once
for all answers to a prompt, and every step stores one token of each answer,
attends with the prompt's tokens shared, draws a token and gives its log
probability and the best alternatives.  Each result is compared with its
formula in 64 bits, from what the operator read on the device; the step
captured in a graph and replayed has to give the eager run's bits."""
import numpy as np
import pytest
import torch

from bf16_wire_all_amd import decode
from tests import decode_reference as ref
from tests import wire_reference as wire
from tests.gpu_util import say
from tests.test_gpu_attn_shared import SPLIT
from tests.test_gpu_decode_step import DEV, EPS, HKV, HQ, PAGE, VOCAB, Step, Worker, wide
from tests.test_gpu_decode_step import SPLIT as COLS
from tests.test_gpu_logprobs import near, reference

pytestmark = pytest.mark.gpu

N_TOP = 5


class Answers(Step):
    """A step of all answers; groups: (first row, rows, prompt's tokens)."""

    def __init__(self, worker, table, lens, embed, head, table_cs, d, groups):
        super().__init__(worker, table, lens, embed, head, table_cs, (None, None), d, 0, 0)
        self.groups = groups
        self.starts = torch.tensor([g[0] for g in groups] + [self.rows], dtype=torch.int32, device=DEV)
        self.shared = torch.tensor([g[2] for g in groups], dtype=torch.int32, device=DEV)
        self.attn_ws = torch.zeros(decode.attn_shared_workspace_bytes(worker.cache, self.rows, len(groups), HQ, self.max_len),
                                   dtype=torch.uint8, device=DEV)
        self.temperature = torch.from_numpy(self.params["temperature"].copy()).to(DEV)
        self.token_out = torch.zeros((self.rows, 1, 2), dtype=torch.int32, device=DEV)
        self.top_out = torch.zeros((self.rows, N_TOP, 2), dtype=torch.int32, device=DEV)
        self.entropy = torch.zeros(self.rows, dtype=torch.float32, device=DEV)
        self.logprob_ws = torch.zeros(decode.logprobs_workspace_bytes(self.rows, COLS, VOCAB - COLS, 1, N_TOP) or 16,
                                      dtype=torch.uint8, device=DEV)

    def run(self):
        torch.index_select(self.embed, 0, self.tok, out=self.fused)
        self.positions.copy_(self.lens)
        page = self.table.gather(1, (self.lens // PAGE).long()[:, None])[:, 0]
        self.slots.copy_(page.long() * PAGE + self.lens % PAGE)
        self.lens.add_(1)
        q, k, v = self.split()
        decode.qkv_rope_store(self.w.cache, q, k, v, self.positions, self.cs, self.slots, self.q_out, eps=EPS)
        decode.attn_shared(self.w.cache, self.q_out, self.table, self.lens, self.max_len, self.starts, self.shared,
                           self.d ** -0.5, self.out, self.attn_ws)
        product = torch.matmul(self.out.view(self.rows, -1), self.head)
        self.logits[:, :COLS].copy_(product[:, :COLS])
        self.logits[:, 608:608 + VOCAB - COLS].copy_(product[:, COLS:])
        decode.sample_merge(*self.shards, self.dparams, self.u, self.sampled, self.sample_ws)
        self.tok.copy_(self.sampled[:, 1])
        decode.logprobs_merge(*self.shards, self.tok.view(-1, 1), self.token_out, self.top_out, self.entropy, self.logprob_ws,
                              temperature=self.temperature)

    def results(self):
        return super().results() + [t.clone() for t in (self.token_out, self.top_out, self.entropy.view(torch.int32))]

    def seen(self, r, which, scale):
        """Keys (0) or values (1) that row r sees: the prompt's from its group's first row's pages."""
        lead, _, p = next(g for g in self.groups if g[0] <= r < g[0] + g[1])
        j = torch.arange(int(self.lens[r]))
        t = self.table.cpu().long()
        pages = torch.where(j < p, t[lead, j // PAGE], t[r, j // PAGE])
        a = wide(self.w.bytes.cpu()[pages, which, :, j % PAGE].contiguous().view(self.w.pages.dtype))
        return a if scale is None else a * wide(scale)[:, None]


@pytest.mark.parametrize("d,kind,bits,to_kind", [(128, "bf16", 8, "bf16"), (64, "bf16", 8, "e4m3"), (256, "e4m3", 4, "bf16"),
                                                 (128, "e4m3", 8, "e4m3")])
def test_prompts_sent_and_answered(d, kind, bits, to_kind):
    say("answers", d, kind, bits, to_kind)
    g = torch.Generator().manual_seed(d + bits)
    prompts, answers, steps = [37, 64, 9], [3, 14, 1], 4
    rows = sum(answers)
    made = lambda k: tuple((torch.rand(HKV, generator=g) * 0.02 + 0.03).to(DEV) for _ in range(2)) if k == "e4m3" else (None, None)
    embed = torch.randn((VOCAB, (HQ + 2 * HKV) * d), generator=g).to(torch.bfloat16).to(DEV)
    head = (torch.randn((HQ * d, VOCAB), generator=g) * 0.2).to(torch.bfloat16).to(DEV)
    angle = torch.arange(256)[:, None] * 10000.0 ** (-torch.arange(d // 2) / (d // 2))
    cs = torch.cat([angle.cos(), angle.sin()], 1).float().contiguous().to(DEV)

    # the prompts' keys and values in the prompt worker's cache
    used = [-(-n // PAGE) for n in prompts]
    from_scales, to_scales = made(kind), made(to_kind)
    prompt = Worker(sum(used) + 3, d, kind, from_scales)
    src = torch.randperm(sum(used) + 3, generator=g)[:sum(used)]
    fused = embed[torch.randint(0, VOCAB, (sum(prompts),), generator=g).to(DEV)]
    q, k, v = (fused[:, a * d:b * d].view(-1, b - a, d) for a, b in ((0, HQ), (HQ, HQ + HKV), (HQ + HKV, HQ + 2 * HKV)))
    # the answers' rows in the decode worker's: the full pages of a prompt are all its rows', its last tokens the first row's
    width = -(-(max(prompts) + steps) // PAGE)
    decoder = Worker(rows * width + 5, d, to_kind, to_scales)
    numbers = torch.randperm(rows * width + 5, generator=g)[:rows * width].view(rows, width)
    pos, slots, to_slots, groups, first, row = [], [], [], [], 0, 0
    for n, pages, count in zip(prompts, used, answers):
        j = torch.arange(n)
        pos.append(j)
        slots.append(src[first + j // PAGE] * PAGE + j % PAGE)
        to_slots.append(numbers[row, j // PAGE] * PAGE + j % PAGE)
        numbers[row:row + count, :n // PAGE] = numbers[row, :n // PAGE].clone()
        groups.append((row, count, n))
        first, row = first + pages, row + count
    pos, slots, to_slots = torch.cat(pos).int().to(DEV), torch.cat(slots).to(DEV), torch.cat(to_slots).to(DEV)
    decode.qkv_rope_store(prompt.cache, q, k, v, pos, cs, slots, torch.empty_like(q).contiguous(), eps=EPS)

    # their records, and what the decode worker makes of them
    need = decode.kv_record_bytes(prompt.cache, bits)
    sent = torch.zeros((len(slots), need), dtype=torch.uint8, device=DEV)
    decode.kv_quantize(prompt.cache, slots, sent, bits)
    received = torch.empty_like(sent).copy_(sent)
    decode.kv_restore(received, bits, decoder.cache, to_slots)
    torch.cuda.synchronize()
    at = slots.cpu()
    held = prompt.bytes.cpu()[at // PAGE, :, :, at % PAGE].contiguous().view(prompt.pages.dtype).float()
    if from_scales[0] is not None:
        held = held * torch.stack(from_scales).cpu()[None, :, :, None]
    records = wire.records(held.numpy().astype(np.float64).reshape(len(slots), -1), bits)
    assert np.array_equal(sent.cpu().numpy(), records), "records"
    values = wire.values(records, 2 * HKV * d, bits).reshape(-1, 2, HKV, d)
    at = to_slots.cpu()
    got = decoder.bytes.cpu()[at // PAGE, :, :, at % PAGE].contiguous()
    if to_kind == "bf16":
        assert np.array_equal(got.view(torch.int16).numpy().view(np.uint16), wire.bf16_bits(values)), "restored"
    else:
        quotient = values.astype(np.float32) / torch.stack(to_scales).cpu().numpy()[None, :, :, None]
        assert np.array_equal(got.view(torch.uint8).numpy(), wire.nearest(np.clip(quotient, -448, 448).astype(np.float64), 8))

    lens = torch.cat([torch.full((count,), n) for n, count in zip(prompts, answers)]).int().to(DEV)
    step = Answers(decoder, numbers.int().to(DEV), lens, embed, head, cs, d, groups)
    us = torch.rand((steps, rows), generator=g).to(DEV)
    begin = step.state()
    ids = np.arange(VOCAB)
    eager = []
    for i in range(steps):
        step.u.copy_(us[i])
        step.run()
        torch.cuda.synchronize()
        eager.append(step.results())
        for r in range(rows):
            got_q = wide(step.q_out[r])
            keys, vals = (step.seen(r, w, to_scales[w]) for w in range(2))
            o, tol = ref.attention(got_q, keys, vals, d ** -0.5)
            for h in range(HQ):
                s = keys[:, h // (HQ // HKV)] @ got_q[h] * d ** -0.5
                p = np.exp(s - s.max())
                tol[h] += (SPLIT["bf16"] - 2.0 ** -18) * (2 * (p / p.sum() @ np.abs(vals[:, h // (HQ // HKV)])) + np.abs(o[h]))
            tol = tol * (1 + ref.HALF["bf16"]) + ref.HALF["bf16"] * np.abs(o)
            assert np.all(np.abs(wide(step.out[r]) - o) <= tol), ("attention", i, r)
            row = wide(step.logits[r])
            row = np.concatenate([row[:COLS], row[608:608 + VOCAB - COLS]])
            p = [float(f) for f in step.params[r]]
            idx, _, margin = ref.sample(row, ids, p[0], int(p[1]), p[2], p[3], float(us[i, r]))
            assert margin > 1e-12 and int(step.tok[r]) == idx, ("sample", i, r)
            want = reference(row, ids, p[0], [idx], N_TOP)
            tok = step.token_out[r].cpu().numpy().view(decode.TOKEN_LOGPROB)[:, 0]
            top = step.top_out[r].cpu().numpy().view(decode.TOP_LOGPROB)[:, 0]
            assert list(tok["rank"]) == want["rank"] and list(top["idx"]) == want["top_idx"], ("ranks", i, r)
            for x, w, t in (*zip(tok["logprob"], want["logprob"], want["tol"]),
                            *zip(top["logprob"], want["top_logprob"], want["top_tol"]),
                            (float(step.entropy[r]), want["entropy"], want["entropy_tol"])):
                assert near(float(x), w, t), ("log probabilities", i, r, x, w, t)

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
        for ws in (step.attn_ws, step.sample_ws, step.logprob_ws):
            ws.fill_(0xFF)
