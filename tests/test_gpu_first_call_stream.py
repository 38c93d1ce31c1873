"""A handle's first call on a stream that does not wait for the default stream,
while the default stream is busy: the workspace's header (error word, claim
counters) is cleared on the call's own stream. The workspace is made from memory
that held other values before."""
import ctypes

import pytest
import torch

import masked_attention_fa_b200 as fa
from masked_attention_fa_b200.workloads import random_inputs

pytestmark = pytest.mark.gpu

B, N, S, D = 1, 160, 2048, 64  # 8 items per SM: claimed at run time


@pytest.fixture(scope="module", autouse=True)
def _built():
    from masked_attention_fa_b200 import build
    build.build()
    fa.load_library()


def used_memory():
    """Leaves freed device memory of the workspace's size with every bit set."""
    rt = ctypes.CDLL("libcudart.so.12")
    size, blocks = 1 << 20, []
    for _ in range(4):
        p = ctypes.c_void_p()
        assert rt.cudaMalloc(ctypes.byref(p), ctypes.c_size_t(size)) == 0
        assert rt.cudaMemset(p, 0xff, ctypes.c_size_t(size)) == 0
        blocks.append(p)
    assert rt.cudaDeviceSynchronize() == 0
    for p in blocks:
        assert rt.cudaFree(p) == 0


@pytest.mark.parametrize("bias", [False, True])
def test_first_call_beside_a_busy_default_stream(bias):
    inp = random_inputs("BNSD", B, N, S, S, D, seed=8900)
    q, k, v = (inp[x].cuda() for x in "qkv")
    kw = {}
    if bias:
        kw = dict(rel_bias=torch.randn(8, N, generator=torch.Generator().manual_seed(6)).cuda(),
                  rel_buckets=fa.relative_buckets(8, 40))
    first = fa.MaskedAttention("BNSD", B, N, S, S, D, 2)
    want = first(q, k, v, **kw)
    out, lse = (torch.full_like(x, float("nan")) for x in want)
    torch.cuda.synchronize()
    first.close()
    used_memory()
    side = torch.cuda.Stream()
    attn = fa.MaskedAttention("BNSD", B, N, S, S, D, 2)
    torch.cuda._sleep(100_000_000)  # the default stream
    attn(q, k, v, out=out, lse=lse, stream=side, **kw)
    side.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    torch.cuda.synchronize()
    attn.sync_status()
    attn.close()
