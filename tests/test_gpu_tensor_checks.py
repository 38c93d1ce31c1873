"""Tensors that are too small, or not on the GPU of q, are refused by the forward,
paged and occupancy calls before anything is launched; larger buffers are taken as
before (the library reads as many elements as the problem has)."""
import pytest
import torch

import masked_attention_fa_b200 as fa
from masked_attention_fa_b200.workloads import random_inputs

pytestmark = pytest.mark.gpu

B, N, S, D = 2, 2, 130, 64


@pytest.fixture(scope="module", autouse=True)
def _built():
    from masked_attention_fa_b200 import build
    build.build()
    fa.load_library()


def tensors():
    inp = random_inputs("BNSD", B, N, S, S, D, seed=9400)
    t = {x: inp[x].cuda() for x in "qkv"}
    t["out"] = torch.empty_like(t["q"])
    t["lse"] = torch.empty(B, N, S, device="cuda")
    return t


def smaller(x):
    return x.flatten()[:-1].clone()


def refused(call, t, names):
    """call(**t) with each of the tensors cut short, and on the host."""
    for name in names:
        for bad in (smaller(t[name]), t[name].cpu()):
            with pytest.raises(ValueError):
                call(**dict(t, **{name: bad}))


def test_forward():
    t = tensors()
    attn = fa.MaskedAttention("BNSD", B, N, S, S, D, 2)
    refused(attn, t, ("q", "k", "v", "out", "lse"))
    attn(**t)
    want = [t["out"].clone(), t["lse"].clone()]
    more = {x: torch.cat([y.flatten(), torch.zeros(64, dtype=y.dtype, device="cuda")])
            for x, y in t.items()}
    o, lse = attn(**more)
    torch.cuda.synchronize()
    attn.sync_status()
    attn.close()
    assert torch.equal(o[:-64].view_as(want[0]), want[0])
    assert torch.equal(lse[:-64].view_as(want[1]), want[1])


def test_alibi():
    t = dict(tensors(), slopes=torch.rand(N, device="cuda"))
    attn = fa.MaskedAttention("BNSD", B, N, S, S, D, 2, alibi="right")
    refused(attn, t, ("q", "k", "v", "out", "lse", "slopes"))
    attn(**t)
    torch.cuda.synchronize()
    attn.sync_status()
    attn.close()


@pytest.mark.parametrize("kind,shape", [("SS", (S, S)), ("B1SS", (B, 1, S, S)),
                                        ("BNSS", (B, N, S, S))])
def test_masks_and_ranges(kind, shape):
    mask = torch.triu(torch.ones(S, S, dtype=torch.uint8), 1).expand(shape).contiguous().cuda()
    t = dict(tensors(), atten_mask=mask)
    attn = fa.MaskedAttention("BNSD", B, N, S, S, D, 1, mask_kind=kind)
    refused(attn, t, ("q", "k", "v", "out", "lse", "atten_mask"))
    _, ranges = attn.occupancy(mask)
    refused(attn, dict(t, ranges=ranges), ("atten_mask", "ranges"))
    with pytest.raises(ValueError):
        attn(**dict(t, ranges=ranges.long()))
    refused(attn.occupancy, dict(atten_mask=mask), ("atten_mask",))
    attn(**t)
    want = t["out"].clone()
    attn(**dict(t, ranges=ranges))
    torch.cuda.synchronize()
    attn.sync_status()
    attn.close()
    assert torch.equal(t["out"], want)


def test_paged():
    bs, lens = 64, [100, 130]
    g = torch.Generator().manual_seed(9500)
    rnd = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).cuda()
    t = dict(q=rnd(2, N, D), k_cache=rnd(5, bs, N, D), v_cache=rnd(5, bs, N, D),
             block_table=torch.tensor([[0, 1, 0], [2, 3, 4]], dtype=torch.int32, device="cuda"),
             out=rnd(2, N, D), lse=torch.empty(N, 2, device="cuda"))
    attn = fa.MaskedAttention("TND", 2, N, 2, sum(lens), D, 3)

    def call(**t):
        return attn.paged(actual_seq_qlen=[1, 2], actual_seq_kvlen=[100, 230], **t)

    refused(call, t, ("q", "k_cache", "v_cache", "block_table", "out", "lse"))
    call(**t)
    torch.cuda.synchronize()
    attn.sync_status()
    attn.close()
