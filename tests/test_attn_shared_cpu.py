"""xfer_attn_shared on the CPU: every documented refusal, the workspace's size
and the struct's layout.  No call here reaches a launch: each either fails a
host check or is empty work."""
import ctypes
import os
import re

import pytest

import bf16_wire_all_amd as x
from bf16_wire_all_amd import decode
from tests.test_decode_cpu import BAD_CACHES, K, KN, Q, QO, V, VN, cache

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TABLE, LENS, STARTS, SHARED = KN, KN + (1 << 30), KN + (2 << 30), KN + (3 << 30)


def batch(**kw):
    b = decode.PagedBatchC(TABLE, LENS, 7, 6, 100, 0, 0)
    for k, v in kw.items():
        setattr(b, k, v)
    return b


def groups(**kw):
    g = decode.PrefixGroupsC(STARTS, SHARED, 2, 0)
    for k, v in kw.items():
        setattr(g, k, v)
    return g


def attn(c=None, b=None, g=None, q=Q, q_ld=1024, q_heads=8, scale=0.1, out=QO, out_ld=1024, mode=x.OUT_BF16, ws=VN,
         ws_bytes=1 << 34):
    return decode.attn_shared_raw(c or cache(), b or batch(), g or groups(), q, q_ld, q_heads, scale, out, out_ld, mode, ws,
                                  ws_bytes, stream=0)


def need(c=None, b=None, g=None, q_heads=8):
    f = decode.lib().xfer_attn_shared_workspace_bytes
    return f(ctypes.byref(c or cache()), ctypes.byref(b or batch()), ctypes.byref(g or groups()), q_heads)


@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_bad_caches_are_refused(kw, status):
    assert attn(cache(**kw)) == status
    assert need(cache(**kw)) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(page_table=0), x.E_INVAL), (dict(page_table=TABLE + 2), x.E_INVAL), (dict(lens=0), x.E_INVAL),
    (dict(lens=LENS + 1), x.E_INVAL), (dict(table_ld=6), x.E_INVAL), (dict(table_ld=1 << 60), x.E_INVAL),
    (dict(max_len=0), x.E_INVAL), (dict(max_len=1 << 31), x.E_INVAL), (dict(sinks=1), x.E_INVAL),
    (dict(window=8), x.E_UNSUPPORTED), (dict(window=8, sinks=1), x.E_UNSUPPORTED), (dict(rows=1 << 22), x.E_UNSUPPORTED)])
def test_bad_batches_are_refused(kw, status):
    assert attn(b=batch(**kw)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(starts=0), x.E_INVAL), (dict(shared=0), x.E_INVAL), (dict(starts=STARTS + 2), x.E_INVAL),
    (dict(shared=SHARED + 1), x.E_INVAL), (dict(reserved=1), x.E_INVAL), (dict(groups=4097), x.E_UNSUPPORTED)])
def test_bad_groups_are_refused(kw, status):
    assert attn(g=groups(**kw)) == status


@pytest.mark.parametrize("kw", [
    dict(q=0), dict(q=Q + 8), dict(out=0), dict(out=QO + 8), dict(q_ld=1020), dict(q_ld=1016), dict(out_ld=1020), dict(out_ld=512),
    dict(q_heads=0), dict(q_heads=3), dict(scale=float("nan")), dict(scale=float("inf")), dict(mode=2), dict(ws=0),
    dict(ws=VN + 8), dict(ws_bytes=1000),
    # an output or the workspace over an input or another
    dict(out=Q), dict(out=K + 4096), dict(out=V), dict(out=TABLE), dict(out=LENS - 1024), dict(out=STARTS - 64),
    dict(out=SHARED), dict(ws=Q - 64), dict(ws=K), dict(ws=V + 160), dict(ws=TABLE + 32), dict(ws=STARTS), dict(ws=SHARED - 1024),
    dict(ws=LENS - 1024), dict(out=VN + 64)])
def test_bad_arguments_are_refused(kw):
    assert attn(**kw) == x.E_INVAL


def test_scales_under_an_output_are_refused():
    for bad in (dict(k_scale=QO + 64), dict(v_scale=VN + 64)):
        assert attn(cache(kind=decode.KV_E4M3, **bad)) == x.E_INVAL


def test_empty_work_and_no_groups():
    assert attn(b=batch(rows=0), q=0, out=0, ws=0) == x.OK
    assert need(b=batch(rows=0)) == 0
    # without groups their pointers are not looked at: the first refusal is the workspace's
    assert attn(g=groups(groups=0, starts=0, shared=0), ws=0) == x.E_INVAL
    assert need(g=groups(groups=0)) > 0


def test_workspace_bytes():
    assert need() > 0 and need() % 16 == 0
    assert need(b=batch(window=5)) == 0 and need(b=batch(max_len=0)) == 0 and need(q_heads=3) == 0
    assert need(g=groups(groups=4097)) == 0 and need(g=groups(reserved=2)) == 0
    assert need(b=batch(page_table=0, lens=0, table_ld=0), g=groups(starts=0, shared=0)) == need()
    assert need(b=batch(max_len=1 << 30)) == need()
    assert need(b=batch(rows=600)) > need()
    assert attn(ws_bytes=need() - 1) == x.E_INVAL


def test_the_struct_matches_the_header():
    text = open(os.path.join(ROOT, "include", "xfer_decode.h")).read()
    body = re.search(r"typedef struct \{((?:(?!typedef)[\s\S])*?)\} xfer_prefix_groups;", text).group(1)
    fields = re.findall(r"^\s*(const uint32_t \*|uint32_t )\s*(\w+);", body, re.M)
    assert [f for _, f in fields] == [f for f, _ in decode.PrefixGroupsC._fields_]
    want = {"const uint32_t *": ctypes.c_void_p, "uint32_t ": ctypes.c_uint32}
    assert [want[t] for t, _ in fields] == [t for _, t in decode.PrefixGroupsC._fields_]
    assert ctypes.sizeof(decode.PrefixGroupsC) == 24
