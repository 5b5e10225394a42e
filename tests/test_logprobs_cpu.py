"""xfer_logprobs_merge on the CPU: every documented refusal, the workspace's
size and the records' layout.  No call here reaches a launch: each either
fails a host check or is empty work."""
import os
import re

import numpy as np
import pytest

import bf16_wire_all_amd as x
from bf16_wire_all_amd import decode
from tests.test_decode_cpu import K, KN, Q, QO, V, VN, shards

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TOP, ENT, TEMP, IDS = QO + (1 << 30), QO + (2 << 30), Q + (1 << 30), Q + (2 << 30)


def call(s=None, temperature=TEMP, tokens=IDS, n_tokens=2, n_top=5, token_out=QO, top_out=TOP, entropy=ENT, ws=VN,
         ws_bytes=1 << 24):
    s0, s1 = s or shards()
    return decode.logprobs_merge_raw(s0, s1, temperature, tokens, n_tokens, n_top, token_out, top_out, entropy, ws, ws_bytes,
                                     stream=0)


@pytest.mark.parametrize("s,status", [
    (dict(n0=0), x.E_INVAL), (dict(n1=0), x.E_INVAL), (dict(off1=999), x.E_INVAL), (dict(off0=500, off1=0), x.E_INVAL),
    (dict(off1=(1 << 31) - 899), x.E_INVAL), (dict(p0=0), x.E_INVAL), (dict(p1=V + 8), x.E_INVAL),
    (dict(ld0=1004), x.E_INVAL), (dict(ld1=896), x.E_INVAL), (dict(ld0=1 << 62), x.E_INVAL),
    (dict(n0=2097153, ld0=2097160, off1=3000000), x.E_UNSUPPORTED), (dict(rows=1 << 24), x.E_UNSUPPORTED)])
def test_bad_shards_are_refused(s, status):
    assert call(shards(**s)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(n_tokens=17), x.E_UNSUPPORTED), (dict(n_top=33), x.E_UNSUPPORTED), (dict(n_top=1 << 31), x.E_UNSUPPORTED),
    (dict(tokens=0), x.E_INVAL), (dict(tokens=IDS + 2), x.E_INVAL), (dict(token_out=0), x.E_INVAL),
    (dict(token_out=QO + 4), x.E_INVAL), (dict(top_out=0), x.E_INVAL), (dict(top_out=TOP + 4), x.E_INVAL),
    (dict(entropy=ENT + 2), x.E_INVAL), (dict(temperature=TEMP + 1), x.E_INVAL), (dict(ws_bytes=100), x.E_INVAL),
    (dict(ws=0), x.E_INVAL), (dict(ws=VN + 8), x.E_INVAL),
    # an output or the workspace over an input or another
    (dict(token_out=K + 8), x.E_INVAL), (dict(top_out=V), x.E_INVAL), (dict(entropy=K + 2 * 1000), x.E_INVAL),
    (dict(token_out=IDS + 16), x.E_INVAL), (dict(entropy=TEMP + 8), x.E_INVAL), (dict(top_out=QO + 40), x.E_INVAL),
    (dict(entropy=QO + 44), x.E_INVAL), (dict(entropy=TOP + 116), x.E_INVAL), (dict(ws=K), x.E_INVAL),
    (dict(ws=QO - 64), x.E_INVAL), (dict(temperature=VN + 64), x.E_INVAL)])
def test_bad_arguments_are_refused(kw, status):
    assert call(**kw) == status


def test_different_rows_and_empty_work():
    s0, s1 = shards()
    s1.rows = 4
    assert call((s0, s1)) == x.E_INVAL
    assert call(shards(rows=0), temperature=0, tokens=0, token_out=0, top_out=0, entropy=0, ws=0) == x.OK


def test_workspace_bytes():
    need = decode.logprobs_workspace_bytes
    for bad in ((0, 10, 10, 1, 1), (5, 0, 10, 1, 1), (5, 10, 0, 1, 1), (5, 2097153, 10, 1, 1), (5, 10, 10, 17, 1),
                (5, 10, 10, 1, 33), (1 << 24, 10, 10, 1, 1)):
        assert need(*bad) == 0, bad
    assert need(5000, 64768, 64512, 16, 32) == 0                  # a workgroup for each row
    sizes = [need(r, 64768, 64512, 1, 5) for r in (1, 16, 300)]
    assert all(s > 0 and s % 16 == 0 for s in sizes) and sizes == sorted(sizes)
    assert need(16, 64768, 64512, 0, 0) < need(16, 64768, 64512, 0, 32)


def test_records_match_the_header():
    text = open(os.path.join(ROOT, "include", "xfer_decode.h")).read()
    for name, dt in (("xfer_token_logprob", decode.TOKEN_LOGPROB), ("xfer_top_logprob", decode.TOP_LOGPROB)):
        body = re.search(r"typedef struct \{((?:(?!typedef)[\s\S])*?)\} %s;" % name, text).group(1)
        fields = re.findall(r"^\s*(float|int32_t) (\w+);", body, re.M)
        assert [(f, {"float": "<f4", "int32_t": "<i4"}[t]) for t, f in fields] == [(n, dt.fields[n][0].str) for n in dt.names]
        assert np.dtype(dt).itemsize == 8
