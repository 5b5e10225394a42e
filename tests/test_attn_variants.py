"""Every variant of the attention kernel that the library holds has a case here:
`choice` says which one a call's sizes lead to, a test on the CPU compares the
cases' variants with the library's own list, and one on the GPU runs each case
against the formula in 64 bits."""
import os
import re
import shutil
import subprocess

import numpy as np
import pytest

import bf16_wire_all_amd as x
from tests import decode_reference as ref

UNIT, CACHED, COMPUTE_UNITS = 128, 96 << 20, 256
# of a softmax weight in the product: two BF16 numbers are off by up to 2^-17 of it, three hold it whole
SPLIT = {"bf16": 2.0 ** -17, "f32": 0.0}
LENS = [700, 0, 1, 33, 300, 129]


def choice(rows, kv_heads, group, d, kind, vis_max, heads_adjacent, out):
    """(head_dim, kind, 16-head tiles, weight parts, waves, past the caches, heads side by side), and whether rows are cut up."""
    size = 2 if kind == "bf16" else 1
    row, tiles, steps = d * size, 1 if group <= 16 else 2, -(-vis_max // UNIT)
    inner = kv_heads * -(-group // (16 * tiles))
    two = not (d == 256 and (kind == "bf16" or tiles == 2))      # waves that share a SIMD
    most = COMPUTE_UNITS * (2 if two else 1)
    stream = vis_max > CACHED // (2 * row) // (rows * kv_heads)
    heads = 4 if kv_heads % 4 == 0 else 2
    beside = (stream and two and kv_heads % 2 == 0 and heads_adjacent
              and row <= (256 if heads == 4 and tiles == 1 else 128))
    whole = (24 if row <= 64 else 16 if row <= 128 else 8) if beside else 32 if row <= 64 else 16
    share = rows * inner * steps // most
    joined = steps > whole or steps > share + 3
    wait = 10 if row <= 64 else 6 if row <= 128 else 3
    waves = 4
    if (two and rows * inner <= COMPUTE_UNITS and steps > 1 and steps * row <= 2048
            and steps <= 2 * rows * inner * steps // most + wait):
        waves, joined = 8, False
    heads = heads if beside and joined else 1
    if heads > 1:
        waves = 4 // heads
    past = row >= 128 and (heads > 1 or (waves == 4 and stream))
    return (d, 0 if kind == "bf16" else 1, tiles, 2 if out == "bf16" else 3, waves, past, heads), joined


def cases():
    """One call for each variant, and for one head with four waves both cut up and whole."""
    found = {}
    for d in (64, 128, 256):
        for kind in ("bf16", "e4m3"):
            for group in (3, 20):
                for out in ("bf16", "f32"):
                    for kv_heads, order in ((2, "heads"), (2, "tokens"), (4, "tokens"), (1, "heads"), (12, "heads")):
                        for max_len in (700, 1500, 2500, 6000, 25000, 60000, 120000, 260000):
                            for lens in (LENS, LENS * 12, [min(n, 150) for n in LENS] * 12):
                                top = max(lens) if max_len == 700 else max_len
                                v, cut = choice(len(lens), kv_heads, group, d, kind, top, order == "tokens", out)
                                if len(lens) > 6 and (cut or max_len > 700):
                                    continue
                                found.setdefault((v, cut), (lens, kv_heads * group, kv_heads, order, top))
    return sorted(found.items(), key=str)


CASES = cases()


def test_the_cases_reach_every_variant_of_the_library():
    nm = shutil.which("nm")
    if not nm:
        pytest.skip("no nm to list the library's kernels with")
    names = subprocess.run([nm, "-C", x.LIB_PATH], capture_output=True, text=True).stdout
    built = set()
    for line in re.findall(r"__device_stub__attn_kernel<([^>]*)>", names):
        built.add(tuple({"true": True, "false": False}.get(a) if a in ("true", "false") else int(a)
                        for a in line.replace(" ", "").split(",")))
    assert len(built) > 50, "the library's kernels are not listed"
    assert {v for (v, _), _ in CASES} == built


def exact(w):
    """The formula in 64 bits and how far binary32 with one rounding may be from it, with the split of the weights as it is."""
    o, t = [], []
    for r in range(w.rows):
        pages, slots = w.at[r]
        kv = []
        for bits, scale in ((w.k, w.ks), (w.v, w.vs)):
            a = w.float_of(bits[pages, slots])
            kv.append(a if scale is None else a * scale.numpy().astype(np.float64)[:, None])
        q, group = w.q[r].float().numpy().astype(np.float64), w.hq // w.hkv
        out, tol = ref.attention(q, kv[0], kv[1], w.scale)
        for h in range(w.hq if len(pages) else 0):
            s = kv[0][:, h // group] @ q[h] * w.scale
            p = np.exp(s - s.max())
            p /= p.sum()
            # ref.attention counts 2^-18 for the split, in the numerator twice and in the quotient once
            tol[h] += (SPLIT[w.out_kind] - 2.0 ** -18) * (2 * (p @ np.abs(kv[1][:, h // group])) + np.abs(out[h]))
        o.append(out)
        t.append(tol)
    o, t = np.stack(o), np.stack(t)
    return o, t * (1 + ref.HALF[w.out_kind]) + ref.HALF[w.out_kind] * np.abs(o)


def name(case):
    (v, cut), _ = case
    d, kind, tiles, parts, waves, past, heads = v
    return (f"{d}-{('bf16', 'e4m3')[kind]}-{16 * tiles}-{('bf16', 'f32')[parts - 2]}-{waves}waves-{heads}heads"
            f"{'-past' if past else ''}-{'cut' if cut else 'whole'}")


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=name)
def test_variant(case):
    import torch
    from tests.test_gpu_attn_paged import World, run

    (v, cut), (lens, hq, hkv, order, max_len) = case
    kind, out = ("bf16", "e4m3")[v[1]], ("bf16", "f32")[v[3] - 2]
    d = v[0]

    class Exact(World):
        def float_of(self, bits):
            t = torch.bfloat16 if self.kind == "bf16" else torch.float8_e4m3fn
            return bits.contiguous().view(t).float().numpy().astype(np.float64)

        def want(self):
            return exact(self)

    w = Exact(lens, hq, hkv, d, 16, kind, order, out=out, seed=41 + d, max_len=max_len)
    assert (w.workspace()[1] > 0) == cut
    run(w, calls=2)
