"""The log-sum-exp of rows whose visible scores hold a NaN: NaN, as o is, and not
the -inf of a row that sees nothing (the backward takes -inf for a row without
weights and would give it a zero gradient). Every bias and mask kind of the
tensor-core forward and the paged forward. Rows that do not see the key keep
their bits."""
import numpy as np
import pytest
import torch

import masked_attention_fa_b200 as fa
from masked_attention_fa_b200.workloads import random_inputs

pytestmark = pytest.mark.gpu

B, N, S = 2, 2, 300
KINDS = ["none", "right", "sqrt", "left", "learned", "mask"]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from masked_attention_fa_b200 import build
    build.build()
    fa.load_library()


def arguments(kind):
    """(descriptor arguments, call arguments) of one kind; every one causal."""
    g = torch.Generator().manual_seed(3)
    if kind == "learned":
        return {}, dict(rel_bias=torch.randn(8, N, generator=g).cuda(),
                        rel_buckets=fa.relative_buckets(8, 30))
    if kind == "mask":
        mask = torch.triu(torch.ones(S, S, dtype=torch.uint8), diagonal=1)
        return dict(sparse_mode=1, mask_kind="SS"), dict(atten_mask=mask.cuda())
    if kind == "none":
        return {}, {}
    return dict(alibi=kind), dict(slopes=torch.tensor([0.25, 0.01], device="cuda"))


def run(kind, inp, D):
    desc, call = arguments(kind)
    attn = fa.MaskedAttention(**dict(dict(layout="BNSD", B=B, N=N, Sq=S, Skv=S, D=D, sparse_mode=2),
                                     **desc))
    o, lse = attn(*(inp[x].cuda() for x in "qkv"), **call)
    torch.cuda.synchronize()
    attn.sync_status()
    attn.close()
    return o.cpu(), lse.cpu()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kind", KINDS)
def test_forward(kind, D):
    inp = random_inputs("BNSD", B, N, S, S, D, seed=8200)
    want = run(kind, inp, D)
    inp["q"][0, 1, 140, 3] = float("nan")
    inp["k"][1, 0, 200, 0] = float("nan")  # rows 200 and on see it
    hit = torch.zeros(B, N, S, dtype=torch.bool)
    hit[0, 1, 140] = True
    hit[1, 0, 200:] = True
    o, lse = run(kind, inp, D)
    assert torch.isnan(o[hit]).all() and torch.isnan(lse[hit]).all()
    assert torch.equal(o[~hit], want[0][~hit]) and torch.equal(lse[~hit], want[1][~hit])


@pytest.mark.parametrize("D", [64, 128])
def test_paged(D):
    lens, bs = [700, 65], 64
    blocks = [(n + bs - 1) // bs for n in lens]
    g = torch.Generator().manual_seed(8300)
    q = torch.randn(2, N, D, generator=g).to(torch.bfloat16)
    kc, vc = (torch.randn(sum(blocks), bs, N, D, generator=g).to(torch.bfloat16) for _ in range(2))
    table = torch.zeros(2, max(blocks), dtype=torch.int32)
    table[0, :blocks[0]] = torch.arange(blocks[0])
    table[1, :blocks[1]] = torch.arange(blocks[0], sum(blocks))
    attn = fa.MaskedAttention("TND", 2, N, 2, sum(lens), D, 3)

    def call(kc):
        o, lse = attn.paged(q.cuda(), kc.cuda(), vc.cuda(), table.cuda(), [1, 2],
                            np.cumsum(lens).tolist())
        torch.cuda.synchronize()
        attn.sync_status()
        return o.cpu(), lse.cpu()

    want = call(kc)
    kc[4, 9, 1, 2] = float("nan")  # sequence 0, key 265, head 1
    o, lse = call(kc)
    attn.close()
    assert torch.isnan(o[0, 1]).all() and torch.isnan(lse[1, 0])
    assert torch.equal(o[1], want[0][1]) and torch.equal(o[0, 0], want[0][0, 0])
    assert torch.equal(lse[0], want[1][0]) and lse[1, 1] == want[1][1, 1]
