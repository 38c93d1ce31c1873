"""Backward calls whose lengths change while the stream is busy: the work lists
(6 MB) are uploaded without the host waiting for the stream, as the forward's are
(from pageable memory, 1.5 MB did not wait and 6 MB did); and lists that are replaced before they were used by the GPU."""
import numpy as np
import pytest
import torch

import masked_attention_fa_b200 as fa

pytestmark = pytest.mark.gpu

N, T, B, D = 32, 8192, 2048, 64


@pytest.fixture(scope="module", autouse=True)
def _built():
    from masked_attention_fa_b200 import build
    build.build()
    fa.load_library()


def lengths(seed):
    cuts = np.random.default_rng(seed).integers(0, T + 1, B - 1)
    return np.concatenate([np.sort(cuts), [T]]).tolist()


def test_new_lengths_on_a_busy_stream():
    g = torch.Generator().manual_seed(9100)
    q, k, v, do = (torch.randn(T, N, D, generator=g).to(torch.bfloat16).cuda() for _ in range(4))
    all_lens = [lengths(s) for s in range(4)]
    fresh = fa.MaskedAttention("TND", B, N, T, T, D, 3)
    fwd = [fresh(q, k, v, actual_seq_qlen=x, actual_seq_kvlen=x) for x in all_lens]

    def backward(attn, n):
        return attn.backward(do, q, k, v, *fwd[n], actual_seq_qlen=all_lens[n],
                             actual_seq_kvlen=all_lens[n])

    want = [[x.clone() for x in backward(fresh, n)] for n in range(4)]
    attn = fa.MaskedAttention("TND", B, N, T, T, D, 3)
    # Buffers as large as they can get: B - 1 sequences of one token and one of the
    # rest have (T - B) / 128 + B tiles, which bounds what any lengths have.
    most = list(range(1, B)) + [T]
    attn.backward(do, q, k, v, *fwd[0], actual_seq_qlen=most, actual_seq_kvlen=most)
    backward(attn, 0)
    out = [torch.empty_like(x) for x in want[0]]
    torch.cuda.synchronize()
    done = torch.cuda.Event()
    torch.cuda._sleep(1_000_000_000)
    done.record()
    attn.backward(do, q, k, v, *fwd[1], actual_seq_qlen=all_lens[1], actual_seq_kvlen=all_lens[1],
                  dq=out[0], dk=out[1], dv=out[2])
    assert not done.query(), "the call waited for the stream"
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want[1]))
    # Several lists in a row, the stream still busy with other work at the first.
    torch.cuda._sleep(200_000_000)
    got = [backward(attn, n) for n in (2, 3, 0, 2)]
    torch.cuda.synchronize()
    attn.sync_status()
    for n, x in zip((2, 3, 0, 2), got):
        assert all(torch.equal(a, b) for a, b in zip(x, want[n]))
    attn.close()
    fresh.close()
