"""How far a binary32 weight is from the sum of two or three BF16 numbers, each
the nearest to what the ones before leave (attention's weights in the matrix
product): for every mantissa, and as the header states it."""
import os
import re

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_two_parts_hold_a_weight_to_2_17_and_three_hold_it_whole():
    w = (torch.arange(1 << 23, dtype=torch.int32) + 0x3F800000).view(torch.float32)   # [1, 2)
    left, off = w.clone(), []
    for _ in range(3):
        left = left - left.to(torch.bfloat16).float()          # exact: both have few bits in common
        off.append(float((left.double().abs() / w.double()).max()))
    assert 2.0 ** -9 < off[0] <= 2.0 ** -8
    assert 2.0 ** -18 < off[1] <= 2.0 ** -17
    assert off[2] == 0


def test_weights_from_2_100_on_need_no_subnormal_part():
    w = (torch.arange(1 << 23, dtype=torch.int32) + 0x3F800000).view(torch.float32) * 2.0 ** -100
    for _ in range(3):
        part = w.to(torch.bfloat16).float()
        assert float(part[part != 0].abs().min()) >= 2.0 ** -126
        w = w - part
    assert float(w.abs().max()) == 0


def test_the_header_states_these_figures():
    text = open(os.path.join(ROOT, "include", "xfer_decode.h")).read()
    text = " ".join(re.sub(r"^ \* ?", "", text, flags=re.M).split())
    assert "keep it to 2^-17 of itself (two numbers, for XFER_OUT_BF16) or, from 2^-100 on, exactly (three" in text
