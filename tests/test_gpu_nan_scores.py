"""Rows whose visible scores hold a NaN or an infinity, in the forward with the
learned relative position bias: o and lse say so (NaN, as the formula gives), and
do not read like a row that sees nothing (0 and -inf). Rows that do not see the
key in question keep their bits. One to four rows, the keys split or not."""
import numpy as np
import pytest
import torch

import masked_attention_fa_b200 as fa
from masked_attention_fa_b200.workloads import random_inputs

pytestmark = pytest.mark.gpu

B, N, REACH = 2, 3, 20


@pytest.fixture(scope="module", autouse=True)
def _built():
    from masked_attention_fa_b200 import build
    build.build()
    fa.load_library()


def setup(rows, keys, D, seed=8100):
    inp = random_inputs("BSND", B, N, rows, keys, D, seed=seed)
    g = torch.Generator().manual_seed(seed)
    m = np.arange(2 * REACH + 1, dtype=np.int32)  # a bucket a distance
    return inp, torch.randn(2 * REACH + 1, N, generator=g), m


def run(inp, table, m, rows, keys, D):
    attn = fa.MaskedAttention("BSND", B, N, rows, keys, D, 3)
    o, lse = attn(*(inp[x].cuda() for x in "qkv"), rel_bias=table.cuda(), rel_buckets=m)
    torch.cuda.synchronize()
    attn.sync_status()
    attn.close()
    return o.cpu(), lse.cpu()


def check(got, want, hit):
    """hit: [B, N, rows], the rows that must be NaN; the others keep their bits."""
    o, lse = got
    at = hit.transpose(1, 2)  # [B, rows, N]
    assert torch.isnan(o[at]).all() and torch.isnan(lse[hit]).all()
    assert torch.equal(o[~at], want[0][~at]) and torch.equal(lse[~hit], want[1][~hit])


# 130 keys are one share, 2,000 several.
SHAPES = [(1, 130), (1, 2000), (4, 130), (4, 2000)]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rows,keys", SHAPES)
def test_nan_in_a_query_row(rows, keys, D):
    inp, table, m = setup(rows, keys, D)
    want = run(inp, table, m, rows, keys, D)
    inp["q"][1, rows - 1, 2, 5] = float("nan")
    hit = torch.zeros(B, N, rows, dtype=torch.bool)
    hit[1, 2, rows - 1] = True
    check(run(inp, table, m, rows, keys, D), want, hit)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rows,keys", SHAPES)
def test_nan_in_a_visible_key(rows, keys, D):
    inp, table, m = setup(rows, keys, D)
    want = run(inp, table, m, rows, keys, D)
    inp["k"][0, keys - 1, 1, 0] = float("nan")  # only the last row sees it
    inp["k"][1, 7, 0, D - 1] = float("nan")     # every row sees it
    hit = torch.zeros(B, N, rows, dtype=torch.bool)
    hit[0, 1, rows - 1] = True
    hit[1, 0] = True
    check(run(inp, table, m, rows, keys, D), want, hit)


@pytest.mark.parametrize("rows,keys", SHAPES)
def test_nan_in_the_table(rows, keys):
    inp, table, m = setup(rows, keys, 64)
    want = run(inp, table, m, rows, keys, 64)
    table[REACH - 3, 1] = float("nan")  # the key three before the diagonal
    hit = torch.zeros(B, N, rows, dtype=torch.bool)
    hit[:, 1] = True
    check(run(inp, table, m, rows, keys, 64), want, hit)


@pytest.mark.parametrize("rows,keys", SHAPES)
def test_infinite_score(rows, keys):
    """exp(inf - inf): o is NaN, lse anything but finite or -inf."""
    inp, table, m = setup(rows, keys, 64)
    want = run(inp, table, m, rows, keys, 64)
    inp["q"][0, 0, 0, 3] = 2.0
    inp["k"][0, 11, 0, 3] = float("inf")
    inp["k"][0, 11, 0, :3] = inp["k"][0, 11, 0, 4:] = 0.0
    o, lse = run(inp, table, m, rows, keys, 64)
    assert torch.isnan(o[0, 0, 0]).all()
    assert torch.isnan(lse[0, 0, 0]) or lse[0, 0, 0] == float("inf")
    assert torch.equal(o[1], want[0][1]) and torch.equal(lse[1], want[1][1])
    assert torch.equal(o[:, :, 1:], want[0][:, :, 1:]) and torch.equal(lse[:, 1:], want[1][:, 1:])
