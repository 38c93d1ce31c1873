"""The sums behind the bias table's gradient, where they cancel: dS that is exact
(d_o = 0 and q = 0, so that P = exp(0 - 0) = 1 and dS = d_lse), in sequences of
one row and one or two keys. Bucket 0 takes both distances, so that its sum is the
difference of two sums of 2^24 + 1 and -2^24: exact in 64 bits, 0 where one of them
is first rounded to 32."""
import numpy as np
import pytest
import torch

import masked_attention_fa_b200 as fa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from masked_attention_fa_b200 import build
    build.build()
    fa.load_library()


@pytest.mark.parametrize("reach", [1, 40, 1024])
@pytest.mark.parametrize("D", [64, 128])
def test_sums_that_cancel(D, reach):
    # Two-key sequences add d_lse to the distances -1 and 0, one-key ones to 0.
    two, one = [2.0 ** 24, 1.0], [-2.0 ** 25, -1.0]
    lens_q, lens_kv = [1] * 4, [2, 2, 1, 1]
    cu_q, cu_kv = np.cumsum(lens_q).tolist(), np.cumsum(lens_kv).tolist()
    N = 2
    dlse = torch.tensor([two + one, [0.0, 3.0, 0.0, -1.0]], device="cuda")
    zq = torch.zeros(4, N, D, dtype=torch.bfloat16, device="cuda")
    zk = torch.zeros(6, N, D, dtype=torch.bfloat16, device="cuda")
    table = torch.zeros(2, N, device="cuda")
    m = np.zeros(2 * reach + 1, dtype=np.int32)
    m[reach + 1:] = 1  # keys right of the diagonal: there are none
    attn = fa.MaskedAttention("TND", 4, N, 4, 6, D, 3)
    got = attn.backward(torch.zeros_like(zq), zq, zk, zk, zq, torch.zeros(N, 4, device="cuda"),
                        d_lse=dlse, rel_bias=table, rel_buckets=m, actual_seq_qlen=cu_q,
                        actual_seq_kvlen=cu_kv)
    torch.cuda.synchronize()
    attn.sync_status()
    attn.close()
    # Head 0: (2^24 + 1) - (2^25 + 1) = -2^24 at distance 0, 2^24 + 1 at -1.
    assert got[3].tolist() == [[1.0, 5.0], [0.0, 0.0]]
