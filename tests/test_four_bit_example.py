"""The example of a 4-bit layer runs and its two paths agree with the formula
on the packed weights' values: decode (bf16 activations, one bf16 rounding of the
result) within that rounding, prefill within what E2M1 activations allow.

An E2M1 value is off by at most 1/4 of its block's largest magnitude's power of two
(2 of 8 units at the top, half a step elsewhere), about 1/10 of the norm of Gaussian
rows (step 1/2 .. 2 around |x| <= 6 units, one unit about 0.6 sigma); two products in
a row and SiLU's slope (at most 1.1) put the layer's error below 3 x 0.15.  A wrong
row, expert or weight order gives a relative error of about 1.4."""
import os
import sys

import pytest
import torch

from conftest import ROOT

sys.path.insert(0, os.path.join(ROOT, "examples"))


@pytest.mark.gpu
@pytest.mark.parametrize("args", [[], ["--tokens", "7", "--experts", "3", "--topk", "2", "--hidden", "288", "--inter", "96"]])
def test_example_runs(args):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import four_bit_layer
    r = four_bit_layer.main(args)
    assert r["decode"] <= 2.0 ** -8
    assert r["prefill"] <= 0.45 and r["weights"] <= 0.45
