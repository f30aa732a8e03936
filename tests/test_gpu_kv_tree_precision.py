"""How exact bq_kv_tree_attention is as a whole: the 2-norm of its error against binary64 sums, in units of what rounding the exact
result to the type costs.  A bound on each element (draft_helpers.reference) has to allow for roundings that all go one way; they
do not, and the norm tells a part that is missing.

bfloat16, whose unit is 8 times binary16's: keys (or the table's entries: times scores of a few, 5/8), values, weights and the table's entries
(1/8 each) are rounded to binary16 once: 1.2 units.

binary16, kernel for few rows: entries in two parts (2^-22), weights too where the form's registers hold their rests, so that the result's
own rounding is nearly all: 1.2 units; where they do not, weights are rounded once, independently of the result and as much:
sqrt(2), 1.5.  Kernel for many rows: the same of values, sqrt(2); of its keys and weights a rest remains below 2^-4 of a rounding,
times scores of a few: 1.5."""
import numpy as np
import pytest
import torch

from draft_helpers import reference, run_tree
from gpu_helpers import TORCH_DT
from test_gpu_kv_tree_rows import BOUND, dev, make

pytestmark = pytest.mark.gpu

LENS = {"drafts": [(40, 1200), (24, 900), (64, 3000)], "one": [(60, 3000)], "short": [(20, 1500), (32, 900)], "from the start": [(120, 500), (64, 300)]}


def check(dev, name, dim, block, bits, dtype, bound, limit, heads=8):
    lens = LENS[name]
    rng = np.random.default_rng(dim + block + bits)
    pool, batch, parents, q = make(dev, rng, lens, heads, 2, dim, block, bits, 32, dtype, bound=bound)
    for _ in range(2):  # scores that spread little, where weights' roundings show most, and twice as much, where keys' do
        want = torch.from_numpy(reference(pool, batch, parents, q, dtype, dim ** -0.5)[0])
        rounding = want.to(TORCH_DT[dtype]).double() - want
        out, _ = run_tree(dev, pool, batch, parents, q, dtype, dim ** -0.5)
        error = out.double().cpu() - want
        for s, (n, _) in enumerate(lens):  # each sequence by itself
            rows = slice(batch.starts[s], batch.starts[s] + n)
            assert error[rows].norm() <= limit * rounding[rows].norm(), (s, float(error[rows].norm() / rounding[rows].norm()))
        q *= 2.0


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("block", [32, 64, 128])
@pytest.mark.parametrize("name", ["drafts", "one", "from the start"])
def test_many_rows(dev, name, block, bits, dtype):
    check(dev, name, 128, block, bits, dtype, BOUND, 1.5 if dtype == "float16" else 1.2)


# Lengths, head_dim, block, bits, bound, query heads of each key/value head, and what binary16 is held to.  few_rows (k_tree_few.hip) gives a
# workgroup 16 rows up to a work of 2^17 (128 wide) or 2^21 (64 wide), tiles of 16 rows x 2 heads x sequences x keys, and to 256 wide
# heads always: "drafts" are 16 x 2 x 3 x 3000 = 2^18.1, so 32 rows where heads are 128 wide, "one" is 15 x 2 x 3000 = 2^16.5.  The forms
# that hold the weights' rests (Occupancy::kRests, bq_attend.h): 64 wide all; 128 wide with 16 rows all but two blocks of 4-bit codes, with
# 32 rows those of one or two blocks; 256 wide those of one or two blocks.
FEW = [*(("drafts", 64, block, bits, bound, 4, 1.2) for block in (32, 64) for bits in (4, 8) for bound in (None, BOUND)),  # 16, 64 rows
       *(("short", 64, block, bits, BOUND, 1, 1.2) for block in (32, 64) for bits in (4, 8)),  # 32 rows
       *(("drafts", 128, block, bits, None, 4, 1.5 if block == 32 else 1.2) for block in (32, 64, 128) for bits in (4, 8)),
       *(("one", 128, block, bits, None, 4, 1.5 if (block, bits) == (64, 4) else 1.2) for block in (32, 64, 128) for bits in (4, 8)),
       *(("drafts", 256, block, bits, None, 4, 1.2 if block >= 128 else 1.5) for block in (32, 64, 128, 256) for bits in (4, 8))]


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("name,dim,block,bits,bound,group,limit", FEW)
def test_few_rows(dev, name, dim, block, bits, bound, group, limit, dtype):
    check(dev, name, dim, block, bits, dtype, bound, limit if dtype == "float16" else 1.2, 2 * group)
