"""Backward of sequences of 2^20 tokens: offsets past 2^31 elements (4 GiB an
operand), dS in more than one share. A band sees 130 keys back, so the gradients
of the last tokens are those of a short call over them. The short call has more
than four items per SM too, so that it also writes dS: the same products in the
same order, equal bits."""
import pytest
import torch

import masked_attention_fa_b200 as fa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from masked_attention_fa_b200 import build
    build.build()
    fa.load_library()


@pytest.mark.parametrize("layout", ["BSND", "BNSD"])
def test_last_tokens_of_a_million(layout):
    S, N, D, short = 1 << 20, 17, 128, 2560
    assert 2 * (short // 128) * N > 4 * 148
    axis = 1 if layout == "BSND" else 2
    band = dict(sparse_mode=4, pre_tokens=130, next_tokens=0)
    shape = lambda s: (1, s, N, D) if layout == "BSND" else (1, N, s, D)
    g = torch.Generator(device="cuda").manual_seed(81)
    q, k, v, do = (torch.empty(shape(S), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
                   for _ in range(4))
    attn = fa.MaskedAttention(layout, 1, N, S, S, D, **band)
    o, lse = attn(q, k, v)
    got = attn.backward(do, q, k, v, o, lse)
    torch.cuda.synchronize()
    attn.sync_status()
    attn.close()
    last = lambda t: t.narrow(axis, S - short, short).contiguous()
    small = fa.MaskedAttention(layout, 1, N, short, short, D, **band)
    want = small.backward(*(last(t) for t in (do, q, k, v, o)), lse[..., S - short:].contiguous())
    torch.cuda.synchronize()
    small.sync_status()
    small.close()
    # (The first rows of the short call lack keys.)
    for a, b in zip(got, want):
        assert torch.equal(a.narrow(axis, S - 512, 512), b.narrow(axis, short - 512, 512))
        assert torch.isfinite(a.narrow(axis, 0, 512)).all() and a.narrow(axis, 0, 512).any()
