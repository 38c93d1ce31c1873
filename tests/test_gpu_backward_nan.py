"""NaN in operands of the backward: every gradient that the formula makes NaN is
NaN, in every column of a tile (the exponentials of a tile are shared out between
two units), and not an infinity or a finite value."""
import pytest
import torch

import masked_attention_fa_b200 as fa
from masked_attention_fa_b200.workloads import random_inputs

pytestmark = pytest.mark.gpu

B, N, S = 1, 2, 400


@pytest.fixture(scope="module", autouse=True)
def _built():
    from masked_attention_fa_b200 import build
    build.build()
    fa.load_library()


# Which rows of a tile take which unit repeats after eight.
@pytest.mark.parametrize("row", [288, 289, 290, 295])
@pytest.mark.parametrize("bias", [None, "right", "learned"])
@pytest.mark.parametrize("D", [64, 128])
def test_nan_in_a_query_row(D, bias, row):
    g = torch.Generator().manual_seed(8400)
    inp = random_inputs("BNSD", B, N, S, S, D, seed=8400)
    q, k, v = (inp[x].cuda() for x in "qkv")
    do = torch.randn(B, N, S, D, generator=g).to(torch.bfloat16).cuda()
    call = {}
    if bias == "right":
        call = dict(slopes=torch.tensor([0.25, 0.01], device="cuda"))
    elif bias == "learned":
        call = dict(rel_bias=torch.randn(8, N, generator=g).cuda(),
                    rel_buckets=fa.relative_buckets(8, 30))
    attn = fa.MaskedAttention("BNSD", B, N, S, S, D, 2, alibi="right" if bias == "right" else None)
    o, lse = attn(q, k, v, **call)
    clean = attn.backward(do, q, k, v, o, lse, **call)
    q[0, 1, row, 3] = float("nan")  # o and lse stay those of the forward before
    got = attn.backward(do, q, k, v, o, lse, **call)
    torch.cuda.synchronize()
    attn.sync_status()
    attn.close()
    dq, dk, dv = got[:3]
    assert torch.isnan(dq[0, 1, row]).all()
    assert torch.isnan(dv[0, 1, :row + 1]).all()
    assert torch.isnan(dk[0, 1, :row + 1]).all()  # dS NaN, or a finite dS times the NaN of q
    if bias == "learned":
        assert torch.isnan(got[3][:, 1]).any() and torch.isfinite(got[3][:, 0]).all()
    # The other head and the other rows do not see it.
    for a, b in zip(got[:3], clean[:3]):
        assert torch.equal(a[:, 0], b[:, 0])
    assert torch.equal(dq[0, 1, :row], clean[0][0, 1, :row])
    assert torch.equal(dq[0, 1, row + 1:], clean[0][0, 1, row + 1:])


@pytest.mark.parametrize("D", [64, 128])
def test_nan_rows_of_a_chain(D):
    """Forward and backward of inputs with a NaN key: the rows that see it get a NaN
    dq, not the zeros of a row that sees nothing."""
    inp = random_inputs("BNSD", B, N, S, S, D, seed=8500)
    q, k, v = (inp[x].cuda() for x in "qkv")
    k[0, 0, 250, 1] = float("nan")
    attn = fa.MaskedAttention("BNSD", B, N, S, S, D, 2)
    o, lse = attn(q, k, v)
    dq, dk, dv = attn.backward(torch.ones_like(o), q, k, v, o, lse)
    torch.cuda.synchronize()
    attn.sync_status()
    attn.close()
    assert torch.isnan(dq[0, 0, 250:]).all() and torch.isnan(dv[0, 0]).all()
    assert torch.isfinite(dq[0, 1]).all() and torch.isfinite(dk[0, 1]).all()
    assert torch.isfinite(dv[0, 1]).all()
