"""The example that runs the cache's write, read and attention together, small."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "paged_decode.py")

# Relative to the largest value: 2^-9 is the output's rounding to bfloat16, 2^-10 the weights' and the
# values' to binary16.  A score moves by at most 2^-11 of scale * sum |q||k| <= scale * |q||k|, and the
# output by twice that; the projections of normalised rows have unit variance, so 128 of them have a norm
# of about 11.3, and scale * |q||k| stays under 16.
BOUND = 2.0 ** -9 + 2.0 ** -10 + 16 * 2.0 ** -10


def example():
    spec = importlib.util.spec_from_file_location("paged_decode", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("bits,seqs,page", [(4, 3, 16), (8, 6, 32)])
def test_graph_steps_equal_eager_steps(bits, seqs, page):
    argv = ["--seqs", str(seqs), "--prompt", "75", "--steps", "7", "--layers", "2", "--vocab", "256",
            "--bits", str(bits), "--page-size", str(page)]
    tokens, error = example().main(argv)
    again, error2 = example().main(argv + ["--eager"])
    assert tokens.shape == (seqs, 7)
    assert torch.equal(tokens, again)
    assert error < BOUND and error2 < BOUND
