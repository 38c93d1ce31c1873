"""Single tokens against a growing key axis, forward and backward in a chain: the
gradients of each step, from the o and lse that the few-row forward gave, against
the formulas in 64 bits of those same o and lse, inside the bounds derived in
training_reference. One and four rows a step, both head dims."""
import pytest
import torch

import masked_attention_fa_b200 as fa
import training_reference as ref
from gpu_helpers import problem_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from masked_attention_fa_b200 import build
    build.build()
    fa.load_library()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rows", [1, 4])
def test_gradients_of_decoding_steps(rows, D):
    N, S, first = 3, 400, 380
    g = torch.Generator().manual_seed(9200)
    q, k, v, do = (torch.randn(1, S, N, D, generator=g).to(torch.bfloat16) for _ in range(4))
    m = fa.relative_buckets(16, 60, bidirectional=False)
    table = torch.randn(16, N, generator=g)
    for t in list(range(first, S - rows, 7)):
        c = dict(layout="BSND", sparse_mode=3, B=1, N=N, Sq=rows, Skv=t + rows, D=D)
        a = [x[:, y:t + rows].contiguous() for x, y in ((q, t), (k, 0), (v, 0), (do, t))]
        dev = [x.cuda() for x in a]
        attn = fa.MaskedAttention(**c)
        bias = dict(rel_bias=table.cuda(), rel_buckets=m)
        o, lse = attn(*dev[:3], **bias)
        got = attn.backward(dev[3], *dev[:3], o, lse, **bias)
        torch.cuda.synchronize()
        attn.sync_status()
        attn.close()
        want = ref.backward(problem_of(c), *(ref.f64(x) for x in a[:3]), ref.f64(o), ref.f64(lse),
                            ref.f64(a[3]), table=ref.f64(table), bucket_of=m)
        ref.check(got, want, f"{rows} rows at {t}")
