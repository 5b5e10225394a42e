"""The decode-step calls on the CPU: the header's declarations against the
library and the binding, struct layouts as a C compiler sees them, and every
documented refusal.  No call here reaches a launch: each either fails a host
check or is empty work."""
import ctypes
import os
import re
import shutil
import subprocess

import numpy as np
import pytest

import bf16_wire_all_amd as x
from bf16_wire_all_amd import decode

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
S0 = 0  # NULL stream: nothing here is enqueued
K, V, Q, KN, VN, QO = (0x10_0000_0000 * (i + 1) for i in range(6))

STRUCTS = {"xfer_kv_cache": decode.KVCacheC, "xfer_rope": decode.RopeC, "xfer_qkv": decode.QKVC,
           "xfer_paged_batch": decode.PagedBatchC}
RECORDS = {"xfer_sample_params": decode.SAMPLE_PARAMS, "xfer_sampled": decode.SAMPLED}
C_TYPES = {"int": ctypes.c_int, "uint32_t": ctypes.c_uint32, "uint64_t": ctypes.c_uint64, "size_t": ctypes.c_size_t,
           "float": ctypes.c_float}


def _declared():
    src = open(os.path.join(ROOT, "include", "xfer_decode.h")).read()
    return re.findall(r"XFER_API\s+(\w+)\s+(xfer_\w+)\s*\(([^)]*)\)\s*;", src, re.S)


def test_every_declared_call_is_exported_with_the_binding_s_signature():
    L = decode.lib()
    decls = _declared()
    assert sorted(d[1] for d in decls) == sorted(decode.EXPORTED)
    pointers = {"xfer_shard": x.Shard, **STRUCTS}
    for ret, name, params in decls:
        fn = getattr(L, name)
        assert fn.restype is C_TYPES[ret], name
        params = [re.sub(r"\bconst\b", "", p).split() for p in " ".join(params.split()).split(",")]
        assert len(fn.argtypes) == len(params), name
        for p, py in zip(params, fn.argtypes):
            if "*" in "".join(p):
                base = p[0].rstrip("*")
                assert py is ctypes.c_void_p or py is ctypes.POINTER(pointers.get(base)), (name, p, py)
            elif p[0] == "hipStream_t":
                assert py is ctypes.c_void_p
            else:
                assert py is C_TYPES[p[0]], (name, p, py)


@pytest.mark.skipif(shutil.which("gcc") is None, reason="needs gcc")
def test_struct_layouts_match_c(tmp_path):
    lines = [f'printf("{n} . %zu\\n", sizeof({n}));' for n in STRUCTS]
    lines += [f'printf("{n} {f[0]} %zu\\n", offsetof({n}, {f[0]}));' for n, s in STRUCTS.items() for f in s._fields_]
    lines += [f'printf("{n} . %zu\\n", sizeof({n}));' for n in RECORDS]
    lines += [f'printf("{n} {f} %zu\\n", offsetof({n}, {f}));' for n, r in RECORDS.items() for f in r.names]
    src = tmp_path / "layout.c"
    src.write_text("#include <stddef.h>\n#include <stdio.h>\n#include \"xfer_decode.h\"\nint main(void) {\n"
                   + "\n".join(lines) + "\nreturn 0;\n}\n")
    exe = str(tmp_path / "layout")
    inc = os.environ.get("ROCM_PATH", "/opt/rocm") + "/include"
    r = subprocess.run(["gcc", "-std=c11", "-Wall", "-Wextra", "-Werror", "-D__HIP_PLATFORM_AMD__", "-I", inc, "-I",
                        os.path.join(ROOT, "include"), str(src), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    for line in subprocess.run([exe], capture_output=True, text=True, timeout=60).stdout.splitlines():
        name, field, value = line.split()
        if name in RECORDS:
            r = RECORDS[name]
            assert (r.itemsize if field == "." else r.fields[field][1]) == int(value), line
            continue
        s = STRUCTS[name]
        assert (ctypes.sizeof(s) if field == "." else getattr(s, field).offset) == int(value), line


# ------------------------------------------------------------------ caches

def cache(**kw):
    c = decode.KVCacheC(K, V, None, None, 16 * 2 * 256, 2 * 256, 256, 100, 16, 2, 128, decode.KV_BF16, 0)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


BAD_CACHES = [
    (dict(k=0), x.E_INVAL), (dict(v=0), x.E_INVAL), (dict(k=K + 8), x.E_INVAL), (dict(v=V + 4), x.E_INVAL),
    (dict(kind=2), x.E_INVAL), (dict(kind=-1), x.E_INVAL), (dict(page_stride=8200), x.E_INVAL),
    (dict(token_stride=520), x.E_INVAL), (dict(head_stride=8), x.E_INVAL), (dict(n_pages=0), x.E_INVAL),
    (dict(page_tokens=0), x.E_INVAL), (dict(page_tokens=12), x.E_INVAL), (dict(kv_heads=0), x.E_INVAL),
    (dict(k_scale=64), x.E_INVAL), (dict(v_scale=64), x.E_INVAL), (dict(reserved=1), x.E_INVAL),
    (dict(head_dim=96), x.E_UNSUPPORTED), (dict(head_dim=0), x.E_UNSUPPORTED),
    (dict(page_tokens=1 << 17), x.E_UNSUPPORTED), (dict(page_stride=1 << 46), x.E_INVAL),
    (dict(page_stride=(1 << 64) - 16), x.E_INVAL),
]


# -------------------------------------------------------------- rope store

def qkv(**kw):
    q = decode.QKVC(Q, KN, VN, 1024, 256, 256, 64, 64, 10, 8, 1e-6, 0)
    for k, v in kw.items():
        setattr(q, k, v)
    return q


def rope(**kw):
    r = decode.RopeC(128, 64, 1000, 128, decode.ROPE_HALVES, 0)
    for k, v in kw.items():
        setattr(r, k, v)
    return r


def store(c=None, q=None, r=None, slots=64, out=QO, out_ld=1024):
    return decode.qkv_rope_store_raw(c or cache(), q or qkv(), r or rope(), slots, out, out_ld, stream=S0)


@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_store_refuses_bad_caches(kw, status):
    assert store(cache(**kw)) == status


def test_store_refuses_overlapping_slots():
    assert store(cache(head_stride=128)) == x.E_OVERLAP          # heads of 256 bytes, 128 apart
    assert store(cache(token_stride=256)) == x.E_OVERLAP         # a token's second head is the next token's first
    assert store(cache(page_stride=4096)) == x.E_OVERLAP
    assert store(cache(page_stride=0)) == x.E_OVERLAP
    assert store(cache(v=K)) == x.E_OVERLAP
    # heads first, and keys and values in turn, are fine (empty work: nothing is enqueued)
    empty = qkv(tokens=0)
    assert store(cache(head_stride=4096, token_stride=256), empty) == x.OK
    assert store(cache(page_stride=2 * 8192, v=K + 8192), empty) == x.OK
    assert store(cache(n_pages=1, page_stride=0), empty) == x.OK  # one page: its stride is never walked


def test_store_refuses_values_over_keys():
    """Every way of laying small caches of keys and values into one another, against their bytes."""
    rng = np.random.default_rng(4)
    seen = {x.OK: 0, x.E_OVERLAP: 0}
    for _ in range(3000):
        counts = [int(n) for n in rng.integers(1, 4, 2)] + [int(2 ** rng.integers(0, 3))]   # pages, heads, slots
        # nested strides in any order, with room for the other half somewhere, or a little too small
        strides, extent = [0, 0, 0], 64
        for i in rng.permutation(3):
            strides[i] = extent + 16 * int(rng.integers(-1 if rng.random() < 0.1 else 0, 2)) + extent * int(
                rng.integers(0, 2))
            extent = strides[i] * counts[i] if rng.random() < 0.5 else extent + strides[i] * (counts[i] - 1)
        by = 16 * int(rng.integers(-2 * extent // 16, 2 * extent // 16))
        if rng.random() < 0.5:                                     # a likely place: a multiple of a part
            by = int(rng.choice([64, -64, *strides, *[-s for s in strides]])) * int(rng.integers(1, 3))
        c = cache(k=K, v=K + by, page_stride=strides[0], head_stride=strides[1], token_stride=strides[2],
                  n_pages=counts[0], kv_heads=counts[1], page_tokens=counts[2], head_dim=64, kind=decode.KV_E4M3)
        at = [p * strides[0] + h * strides[1] + t * strides[2] for p in range(counts[0]) for h in range(counts[1])
              for t in range(counts[2])]
        starts = sorted(at + [a + by for a in at])
        touch = any(b - a < 64 for a, b in zip(starts, starts[1:]))
        got = store(c, qkv(tokens=0), rope(rot_dim=64))
        seen[got] += 1
        if touch:
            assert got == x.E_OVERLAP, (counts, strides, by)
        else:
            # slots that are disjoint without being nested are refused too
            nested, e = True, 64
            for st, n in sorted(zip(strides, counts)):
                nested &= n == 1 or st >= e
                e += st * (n - 1) if n > 1 else 0
            assert got == (x.OK if nested else x.E_OVERLAP), (counts, strides, by)
    assert min(seen.values()) > 500, seen


@pytest.mark.parametrize("q,r,more,status", [
    (dict(reserved=1), {}, {}, x.E_INVAL), ({}, dict(reserved=1), {}, x.E_INVAL), ({}, dict(style=2), {}, x.E_INVAL),
    (dict(eps=-1e-6), {}, {}, x.E_INVAL), (dict(eps=float("nan")), {}, {}, x.E_INVAL),
    (dict(eps=float("inf")), {}, {}, x.E_INVAL), ({}, dict(rot_dim=12), {}, x.E_INVAL),
    ({}, dict(rot_dim=136), {}, x.E_INVAL), ({}, dict(cos_sin=0), {}, x.E_INVAL), ({}, dict(cos_sin=72), {}, x.E_INVAL),
    ({}, dict(positions=0), {}, x.E_INVAL), ({}, dict(max_pos=0), {}, x.E_INVAL), ({}, {}, dict(slots=0), x.E_INVAL),
    (dict(k=0), {}, {}, x.E_INVAL), (dict(v=0), {}, {}, x.E_INVAL), (dict(q=0), {}, {}, x.E_INVAL),
    ({}, {}, dict(out=0), x.E_INVAL), (dict(k=KN + 2), {}, {}, x.E_INVAL), (dict(q=Q + 8), {}, {}, x.E_INVAL),
    ({}, {}, dict(out=QO + 8), x.E_INVAL), (dict(q_weight=8), {}, {}, x.E_INVAL), (dict(k_weight=24), {}, {}, x.E_INVAL),
    (dict(q_ld=1028), {}, {}, x.E_INVAL), (dict(k_ld=248), {}, {}, x.E_INVAL), (dict(v_ld=0), {}, {}, x.E_INVAL),
    ({}, {}, dict(out_ld=1016), x.E_INVAL), (dict(q_ld=(1 << 64) - 8), {}, {}, x.E_INVAL),
    ({}, {}, dict(out=KN), x.E_INVAL),                              # q_out over k
    ({}, {}, dict(out=Q + 16), x.E_INVAL),                          # over q, not exactly in place
    ({}, {}, dict(out=Q, out_ld=1032), x.E_INVAL),                  # in place needs the same ld
    ({}, {}, dict(out=K + 4096), x.E_INVAL), ({}, {}, dict(out=V), x.E_INVAL),
    (dict(k=K + 16), {}, {}, x.E_INVAL), (dict(q=V + 16), {}, {}, x.E_INVAL),
    (dict(tokens=1 << 31, q=Q, q_ld=1024), {}, {}, x.E_INVAL),      # so many rows reach the next buffer
    (dict(tokens=(1 << 24), q_heads=0, q=0), {}, dict(out=0), x.E_UNSUPPORTED),
])
def test_store_refusals(q, r, more, status):
    assert store(q=qkv(**q), r=rope(**r), **more) == status


@pytest.mark.parametrize("q,r,c,more", [
    ({}, dict(positions=66), {}, {}), ({}, {}, {}, dict(slots=68)),                 # misaligned
    ({}, {}, dict(kind=decode.KV_E4M3, k_scale=66), {}), ({}, {}, dict(kind=decode.KV_E4M3, v_scale=65), {}),
    ({}, {}, {}, dict(slots=QO + 64)), ({}, dict(positions=QO), {}, {}),            # q_out over what is read
    ({}, dict(cos_sin=QO + 4096), {}, {}), (dict(q_weight=QO), {}, {}, {}), (dict(k_weight=QO + 16), {}, {}, {}),
    ({}, {}, dict(kind=decode.KV_E4M3, k_scale=QO + 4), {}), ({}, {}, {}, dict(slots=K + 64)),   # the cache over it
    ({}, dict(positions=V + 8), {}, {}), ({}, dict(cos_sin=K), {}, {}), (dict(q_weight=V), {}, {}, {}),
    ({}, {}, dict(kind=decode.KV_E4M3, v_scale=K + 4), {}),
])
def test_store_refuses_misaligned_and_overlapping_inputs(q, r, c, more):
    assert store(cache(**c), qkv(**q), rope(**r), **more) == x.E_INVAL


@pytest.mark.parametrize("c,more", [
    (dict(k_scale=66), {}), (dict(v_scale=67), {}), (dict(k_scale=QO), {}), (dict(v_scale=QO + 2048), {}),
    (dict(k_scale=0xC0_0000), {}), (dict(v_scale=0xC0_0010), {}),
])
def test_attn_refuses_misaligned_scales_and_an_output_over_them(c, more):
    assert attn(cache(kind=decode.KV_E4M3, **c), **more) == x.E_INVAL


def test_store_in_a_fused_buffer():
    """q, k and v as slices of rows of 1536 elements; q_out may not touch k's slice."""
    f = qkv(q=Q, k=Q + 2 * 1024, v=Q + 2 * 1280, q_ld=1536, k_ld=1536, v_ld=1536)
    assert store(q=f, out=Q + 2 * 512, out_ld=1536) == x.E_INVAL
    f.tokens = 0
    assert store(q=f, out=Q, out_ld=1536) == x.OK


def test_store_empty_work_needs_no_buffers():
    e = decode.QKVC(0, 0, 0, 0, 0, 0, 0, 0, 0, 8, 1e-6, 0)
    assert store(q=e, slots=0, out=0, out_ld=0) == x.OK
    assert decode.lib().xfer_qkv_rope_store(None, None, None, None, None, 0, None) == x.E_INVAL


# --------------------------------------------------------------- attention

TABLE, LENS, WS = 0x40_0000, 0x80_0000, 0xC0_0000


def batch(**kw):
    b = decode.PagedBatchC(TABLE, LENS, 64, 3, 1000, 0, 0)
    for k, v in kw.items():
        setattr(b, k, v)
    return b


def attn(c=None, b=None, q=Q, q_ld=1024, heads=8, scale=0.1, out=QO, out_ld=1024, mode=x.OUT_BF16, ws=WS, ws_bytes=1 << 20):
    return decode.attn_paged_raw(c or cache(), b or batch(), q, q_ld, heads, scale, out, out_ld, mode, ws, ws_bytes,
                                 stream=S0)


@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_attn_refuses_bad_caches(kw, status):
    assert attn(cache(**kw)) == status


def _need(c, b, heads):
    return decode.lib().xfer_attn_workspace_bytes(ctypes.byref(c), ctypes.byref(b), heads)


@pytest.mark.parametrize("b,more", [
    (dict(page_table=0), {}), (dict(page_table=TABLE + 2), {}), (dict(lens=0), {}), (dict(lens=LENS + 1), {}),
    (dict(max_len=0), {}), (dict(max_len=1 << 31), {}), (dict(sinks=4), {}), (dict(table_ld=62), {}),
    (dict(table_ld=1 << 62), {}), ({}, dict(q=0)), ({}, dict(q=Q + 8)), ({}, dict(out=0)), ({}, dict(out=QO + 4)),
    ({}, dict(q_ld=1016)), ({}, dict(q_ld=1025)), ({}, dict(out_ld=1020)), ({}, dict(out_ld=1 << 63)),
    ({}, dict(heads=0)), ({}, dict(heads=7)), ({}, dict(mode=2)), ({}, dict(scale=float("nan"))),
    ({}, dict(scale=float("inf"))), ({}, dict(ws=0)), ({}, dict(ws=WS + 4)), ({}, dict(ws_bytes=100)),
    ({}, dict(out=Q)), ({}, dict(out=Q + 2048)), ({}, dict(out=K + 64)), ({}, dict(out=V)), ({}, dict(out=TABLE + 64)),
    ({}, dict(out=LENS)), ({}, dict(out=WS)), ({}, dict(ws=Q)), ({}, dict(ws=K)), ({}, dict(ws=TABLE)),
    ({}, dict(ws=LENS)), ({}, dict(ws=QO, mode=x.OUT_F32)),
])
def test_attn_refusals(b, more):
    assert attn(b=batch(**b), **more) == x.E_INVAL


def test_attn_launch_size_limit():
    b = batch(rows=1 << 24, max_len=16, table_ld=1)
    far = 1 << 44
    b.page_table, b.lens = 3 * far, 4 * far
    assert attn(b=b, q=far, out=2 * far, ws=0, ws_bytes=0, heads=2, q_ld=256, out_ld=256) == x.E_UNSUPPORTED


def test_attn_empty_work_and_workspace_sizes():
    assert attn(b=batch(rows=0, page_table=0, lens=0), q=0, out=0, ws=0, ws_bytes=0) == x.OK
    c = cache()
    assert _need(c, batch(rows=0), 8) == 0
    assert _need(c, batch(max_len=128), 8) == 0                    # one piece: nothing to join
    assert _need(c, batch(max_len=100000, window=100, sinks=4), 8) == 0
    assert _need(c, batch(max_len=100000), 8) > 0
    assert _need(c, batch(max_len=100000), 7) == 0                 # refused sizes
    assert _need(cache(head_dim=80), batch(max_len=100000), 8) == 0
    # a piece's partial results are far smaller than the keys and values it reads
    for rows in (1, 7, 64, 500):
        for n in (300, 5000, 131071, 1 << 20):
            need = _need(c, batch(rows=rows, max_len=n, table_ld=1 << 17), 8)
            assert need <= max(1 << 20, rows * n * 2 * 2 * 128 * 2 // 16), (rows, n, need)


def test_attn_workspace_of_batches_past_the_launch_limit():
    """A batch that the call refuses for its size needs no workspace."""
    far = 1 << 44
    b = batch(rows=1 << 22, max_len=100000, table_ld=6250, page_table=3 * far, lens=4 * far)
    assert attn(b=b, q=far, out=2 * far, heads=8, ws=6 * far, ws_bytes=1 << 40) == x.E_UNSUPPORTED
    assert _need(cache(), b, 8) == 0
    b.rows = 1 << 20
    assert _need(cache(), b, 8) > 0


# ---------------------------------------------------------------- sampling

def shards(n0=1000, n1=900, ld0=1000, ld1=904, rows=3, off0=0, off1=1000, p0=K, p1=V):
    return x.Shard(p0, ld0, rows, n0, off0), x.Shard(p1, ld1, rows, n1, off1)


def samp(s=None, params=Q, u=KN, out=QO, ws=VN, ws_bytes=1 << 24):
    s0, s1 = s or shards()
    return decode.sample_merge_raw(s0, s1, params, u, out, ws, ws_bytes, stream=S0)


@pytest.mark.parametrize("s,more,status", [
    (dict(n0=0), {}, x.E_INVAL), (dict(n1=0), {}, x.E_INVAL), (dict(off1=999), {}, x.E_INVAL),
    (dict(off0=500, off1=0), {}, x.E_INVAL), (dict(off1=(1 << 31) - 899), {}, x.E_INVAL),
    (dict(p0=0), {}, x.E_INVAL), (dict(p1=V + 8), {}, x.E_INVAL), (dict(ld0=1004), {}, x.E_INVAL),
    (dict(ld1=896), {}, x.E_INVAL), (dict(ld0=1 << 62), {}, x.E_INVAL),
    (dict(n0=2097153, ld0=2097160, off1=3000000), {}, x.E_UNSUPPORTED),
    (dict(rows=1 << 24), {}, x.E_UNSUPPORTED),
    (dict(rows=1 << 22, n0=100000, ld0=100000, off1=100000), {}, x.E_UNSUPPORTED),
    ({}, dict(params=0), x.E_INVAL), ({}, dict(params=Q + 8), x.E_INVAL), ({}, dict(u=0), x.E_INVAL),
    ({}, dict(u=KN + 2), x.E_INVAL), ({}, dict(out=0), x.E_INVAL), ({}, dict(out=QO + 8), x.E_INVAL),
    ({}, dict(ws=0), x.E_INVAL), ({}, dict(ws=VN + 4), x.E_INVAL), ({}, dict(ws_bytes=1000), x.E_INVAL),
    ({}, dict(out=K + 16), x.E_INVAL), ({}, dict(out=V), x.E_INVAL), ({}, dict(out=Q + 32), x.E_INVAL),
    ({}, dict(out=KN), x.E_INVAL), ({}, dict(out=VN + 64), x.E_INVAL), ({}, dict(ws=K), x.E_INVAL),
    ({}, dict(ws=V + 32), x.E_INVAL), ({}, dict(ws=Q), x.E_INVAL), ({}, dict(ws=KN), x.E_INVAL),
])
def test_sample_refusals(s, more, status):
    assert samp(shards(**s), **more) == status


def test_sample_empty_work_and_workspace_sizes():
    assert samp(shards(rows=0, p0=0, p1=0, n0=0), params=0, u=0, out=0, ws=0, ws_bytes=0) == x.OK
    s0, s1 = shards()
    s1.rows = 4
    assert samp((s0, s1)) == x.E_INVAL
    assert decode.lib().xfer_sample_merge(None, None, None, None, None, None, 0, None) == x.E_INVAL
    need = decode.sample_workspace_bytes
    assert need(0, 10, 10) == 0 and need(5, 0, 10) == 0 and need(5, 10, 2097153) == 0
    for n0, n1 in ((1, 1), (16384, 16384), (16384, 16392), (64768, 64512), (2097152, 2097152)):
        assert 0 < need(1, n0, n1) <= 8 * 65280 + 4 * (n0 + n1 + 128 * 8) + 1024
        assert need(7, n0, n1) >= 7 * (need(1, n0, n1) - 1024)
