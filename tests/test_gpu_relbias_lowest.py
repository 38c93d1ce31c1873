"""Bias tables that hold the lowest fp32 number or -inf, as a mask would: pairs of
such buckets get no weight, like hidden ones, in the forward of few and of many rows
and in the backward, and rows that see nothing else read as rows that see nothing
(o = 0, lse = -inf, no gradient). Bounds as in the tests of the operators, against
the formulas with the bucket at -1e4, whose weights are 0 in 64 bits too."""
import numpy as np
import pytest
import torch

import masked_attention_fa_b200 as fa
import training_reference as ref
from gpu_helpers import problem_of
from masked_attention_fa_b200.workloads import random_inputs

pytestmark = pytest.mark.gpu

REACH, N = 150, 2


@pytest.fixture(scope="module", autouse=True)
def _built():
    from masked_attention_fa_b200 import build
    build.build()
    fa.load_library()


def case(rows, keys, D):
    """Bucket 1 (masked) takes the distances 4 and more left of the diagonal of
    even distance, and everything past the reach; bucket 2 the others."""
    c = dict(layout="BNSD", sparse_mode=3, B=1, N=N, Sq=rows, Skv=keys, D=D)
    rel = np.arange(-REACH, REACH + 1)
    m = np.where((rel <= -4) & (rel % 2 == 0), 1, np.where(np.abs(rel) == REACH, 1, 2))
    inp = random_inputs("BNSD", 1, N, rows, keys, D, seed=9300)
    table = torch.randn(3, N, generator=torch.Generator().manual_seed(8))
    return c, m.astype(np.int32), inp, table


def run(c, m, inp, table):
    attn = fa.MaskedAttention(**c)
    dev = [inp[x].cuda() for x in "qkv"]
    o, lse = attn(*dev, rel_bias=table.cuda(), rel_buckets=m)
    do = torch.randn(o.shape, generator=torch.Generator().manual_seed(9)).to(torch.bfloat16)
    grads = attn.backward(do.cuda(), *dev, o, lse, rel_bias=table.cuda(), rel_buckets=m)
    torch.cuda.synchronize()
    attn.sync_status()
    attn.close()
    return o, lse, do, grads


LOWEST = [torch.finfo(torch.float32).min, -float("inf")]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rows,keys", [(1, 500), (4, 500), (200, 700)])
@pytest.mark.parametrize("low", LOWEST, ids=["lowest", "inf"])
def test_a_masked_bucket(low, rows, keys, D):
    c, m, inp, table = case(rows, keys, D)
    table[1] = low
    o, lse, do, grads = run(c, m, inp, table)
    table[1] = -1e4
    kw = dict(table=ref.f64(table), bucket_of=m)
    pb = problem_of(c)
    q, k, v = (ref.f64(inp[x]) for x in "qkv")
    want_o, want_lse = ref.forward(pb, q, k, v, **kw)
    spread, _ = ref.forward(pb, q, k, np.abs(v), **kw)
    w = ref.W if rows <= 4 else ref.U / 2 + ref.W  # P in bf16 for the tensor cores
    assert (np.abs(ref.f64(o) - want_o) <= 1.02 * (ref.U * np.abs(want_o) + 2 * w * spread)).all()
    assert (np.abs(ref.f64(lse) - want_lse) <= ref.W + 2.0 ** -22 * np.abs(want_lse)).all()
    ref.check(grads, ref.backward(pb, q, k, v, ref.f64(o), ref.f64(lse), ref.f64(do), **kw))


@pytest.mark.parametrize("rows,keys", [(1, 500), (4, 500), (200, 700)])
@pytest.mark.parametrize("low", LOWEST, ids=["lowest", "inf"])
def test_a_masked_head(low, rows, keys):
    c, m, inp, table = case(rows, keys, 64)
    table[:, 1] = low
    o, lse, do, grads = run(c, m, inp, table)
    assert (o[:, 1] == 0).all() and torch.isneginf(lse[:, 1]).all()
    assert torch.isfinite(lse[:, 0]).all()
    for x in grads[:3]:
        assert (x[:, 1] == 0).all() and torch.isfinite(x).all() and (x[:, 0] != 0).any()
    assert (grads[3][:, 1] == 0).all() and torch.isfinite(grads[3]).all()
