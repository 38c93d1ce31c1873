"""A bucket map in pinned host memory: it is read during the call, so the caller
may rewrite it as soon as the call has returned, while the stream is still busy
with other work; and a later call with the first map uses the first map."""
import pytest
import torch

import masked_attention_fa_b200 as fa
from masked_attention_fa_b200.workloads import random_inputs

pytestmark = pytest.mark.gpu

B, N, S, D = 1, 2, 200, 64


@pytest.fixture(scope="module", autouse=True)
def _built():
    from masked_attention_fa_b200 import build
    build.build()
    fa.load_library()


def make_calls(table):
    """(forward, backward) of one handle, each call(map, stream)."""
    inp = random_inputs("BNSD", B, N, S, S, D, seed=8600)
    q, k, v = (inp[x].cuda() for x in "qkv")
    attn = fa.MaskedAttention("BNSD", B, N, S, S, D, 2)
    o, lse = attn(q, k, v, rel_bias=table, rel_buckets=fa.relative_buckets(8, 40))
    torch.cuda.synchronize()

    def forward(m, stream=None):
        return attn(q, k, v, rel_bias=table, rel_buckets=m, stream=stream)

    def backward(m, stream=None):
        return attn.backward(torch.ones_like(o), q, k, v, o, lse, rel_bias=table, rel_buckets=m,
                             stream=stream)

    return attn, dict(forward=forward, backward=backward)


@pytest.mark.parametrize("op", ["forward", "backward"])
def test_map_rewritten_after_the_call(op):
    table = torch.randn(8, N, generator=torch.Generator().manual_seed(4)).cuda()
    first = torch.from_numpy(fa.relative_buckets(8, 40))
    other = first.flip(0).contiguous()
    attn, calls = make_calls(table)
    want = calls[op](first.numpy())
    calls[op](fa.relative_buckets(8, 35))  # so that the next call uploads its map
    torch.cuda.synchronize()
    pinned = first.clone().pin_memory()
    busy = torch.cuda.Stream()
    with torch.cuda.stream(busy):
        torch.cuda._sleep(200_000_000)
    got = calls[op](pinned, busy)
    pinned.copy_(other)
    torch.cuda.synchronize()
    attn.sync_status()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    again = calls[op](first.numpy())
    torch.cuda.synchronize()
    attn.close()
    assert all(torch.equal(a, b) for a, b in zip(again, want))
