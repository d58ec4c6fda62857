"""The README's Python examples run as they stand, and its 8-bit weight keeps
the weight's values."""

from __future__ import annotations

import re
from pathlib import Path

import pytest
import torch

import sublayer_ref as R

README = Path(__file__).resolve().parent.parent / "README.md"


@pytest.mark.gpu
def test_examples(device):
    names: dict = {}
    torch.manual_seed(0)
    for block in re.findall(r"^```python\n(.*?)^```", README.read_text(), flags=re.M | re.S):
        exec(compile(block, str(README), "exec"), names)
    torch.cuda.synchronize()
    T, H, w1 = names["T"], names["H"], names["w1"]
    assert names["streams"].shape == (T, 4, H) and names["z"].shape == (T, H)
    # codes and scales stand for the weight: half a step of e4m3 off, or half of its smallest value in the scale of
    # the smallest power of two that holds the block (twice that: the power's logarithm is rounded)
    want = w1.cpu().double()
    got = R.dequantise(names["qw"], names["sw"])
    unit = (2.0 ** R.mx_power(R.block_amax(want)).double()).repeat_interleave(32, 1)
    tol = want.abs() * R.HALF_STEP[torch.float8_e4m3fn] + 2 * unit * R.HALF_TINY[torch.float8_e4m3fn]
    R.assert_within(got, want, tol, "weight")
    # and so does the product: the roundings to 8 bits of both sides and the outputs' to bf16, by the norm
    exact = R.dequantise(names["q"].y, names["q"].scales).to(device) @ w1.double().t()
    off = float((names["z"].double() - exact).norm() / exact.norm())
    assert off <= 2.0 ** -4 + 2.0 ** -8, off
