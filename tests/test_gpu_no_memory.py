"""A call that finds no memory for a larger workspace leaves the handle usable:
later calls of the earlier lengths (on the forward, the learned bias, the paged
path) make their work list again, also behind a backward that has meanwhile
brought in a small workspace for its error word. The hook fails the allocation
where cudaMalloc would, with the old workspace already given back."""
import numpy as np
import pytest
import torch

import masked_attention_fa_b200 as fa
from gpu_helpers import TOL_LSE, TOL_MAX_O

pytestmark = pytest.mark.gpu

N, T, B, D = 8, 4096, 64, 64
ONE = [T] * B                                # one sequence has every token
MANY = (np.arange(B) * 64 + 64).tolist()     # 64 of 64 tokens: four times the items


@pytest.fixture(scope="module", autouse=True)
def _built():
    from masked_attention_fa_b200 import build
    build.build()
    fa.load_library()


@pytest.fixture
def case():
    g = torch.Generator().manual_seed(8700)
    q, k, v = (torch.randn(T, N, D, generator=g).to(torch.bfloat16).cuda() for _ in range(3))
    attn = fa.MaskedAttention("TND", B, N, T, T, D, 3)
    yield attn, q, k, v
    attn.close()


def forward(attn, q, k, v, lens, **kw):
    o, lse = attn(q, k, v, actual_seq_qlen=lens, actual_seq_kvlen=lens, **kw)
    torch.cuda.synchronize()
    attn.sync_status()
    return o, lse


def failing(call, monkeypatch):
    monkeypatch.setenv("FA_TEST_FAIL_ALLOC", "1")
    with pytest.raises(fa.FaError) as e:
        call()
    assert e.value.name == "FA_ERR_ALLOC"
    monkeypatch.delenv("FA_TEST_FAIL_ALLOC")


@pytest.mark.parametrize("between", ["nothing", "status", "backward"])
@pytest.mark.parametrize("bias", [False, True])
def test_forward(case, bias, between, monkeypatch):
    attn, q, k, v = case
    kw = {}
    if bias:
        kw = dict(rel_bias=torch.randn(8, N, generator=torch.Generator().manual_seed(5)).cuda(),
                  rel_buckets=fa.relative_buckets(8, 40))
    fresh = fa.MaskedAttention("TND", B, N, T, T, D, 3)
    want_many = forward(fresh, q, k, v, MANY, **kw)
    fresh.close()
    want = forward(attn, q, k, v, ONE, **kw)
    failing(lambda: forward(attn, q, k, v, MANY, **kw), monkeypatch)
    if between == "status":
        attn.sync_status()
    elif between == "backward":
        o, lse = want
        attn.backward(torch.ones_like(o), q, k, v, o, lse, actual_seq_qlen=ONE,
                      actual_seq_kvlen=ONE, **kw)
    for x, y in zip(forward(attn, q, k, v, ONE, **kw), want):
        assert torch.equal(x, y)
    for x, y in zip(forward(attn, q, k, v, MANY, **kw), want_many):
        assert torch.equal(x, y)


def test_paged(monkeypatch):
    """A paged plan behind a forward whose workspace is too small for it."""
    bs = 64
    g = torch.Generator().manual_seed(8800)
    q, k, v = (torch.randn(T, N, D, generator=g).to(torch.bfloat16).cuda() for _ in range(3))
    table = torch.zeros(B, T // bs, dtype=torch.int32)
    table[:, 0] = torch.arange(B)
    pages = [x.view(T // bs, bs, N, D) for x in (k, v)]
    attn = fa.MaskedAttention("TND", B, N, T, T, D, 3)

    def paged():
        o, lse = attn.paged(q, *pages, table.cuda(), MANY, MANY)
        torch.cuda.synchronize()
        attn.sync_status()
        return o, lse

    want = forward(attn, q, k, v, ONE)
    failing(paged, monkeypatch)
    for x, y in zip(forward(attn, q, k, v, ONE), want):
        assert torch.equal(x, y)
    first = paged()
    packed = forward(attn, q, k, v, MANY)  # fits where the paged plan did
    for x, y in zip(paged(), first):
        assert torch.equal(x, y)
    # Block b holds the keys of sequence b: the packed forward's sums in another order.
    assert (first[0].float() - packed[0].float()).abs().max() <= TOL_MAX_O
    assert (first[1] - packed[1]).abs().max() <= TOL_LSE
    attn.close()
