"""Forward calls captured into CUDA graphs, beside eager calls of the same handle:
a backward, a status query and calls of other lengths after the capture, then
replays, which still use the captured call's work list; and the refusal to
capture a call whose list is not there yet."""
import numpy as np
import pytest
import torch

import masked_attention_fa_b200 as fa

pytestmark = pytest.mark.gpu

N, T, B, D = 8, 4096, 64, 64
ONE = [T] * B                                 # one sequence has every token
MANY = (np.arange(B) * 64 + 64).tolist()      # 64 of 64 tokens: four times the items


@pytest.fixture(scope="module", autouse=True)
def _built():
    from masked_attention_fa_b200 import build
    build.build()
    fa.load_library()


def tensors(*shapes, seed=9000):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(s, generator=g).to(torch.bfloat16).cuda() for s in shapes]


def capture(call):
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    return graph, out


def replay(graph, out):
    for x in out:
        x.fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    return [x.clone() for x in out]


def equal(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("alibi", [None, "right"])
def test_eager_calls_after_a_capture(alibi):
    q, k, v, do = tensors(*[(1, N, 700, D)] * 4)
    kw = dict(slopes=torch.linspace(0.01, 0.3, N).cuda()) if alibi else {}
    attn = fa.MaskedAttention("BNSD", 1, N, 700, 700, D, 2, alibi=alibi)
    want = attn(q, k, v, **kw)
    grads = attn.backward(do, q, k, v, *want, **kw)
    graph, out = capture(lambda: attn(q, k, v, **kw))
    attn.sync_status()
    assert equal(attn.backward(do, q, k, v, *want, **kw), grads)
    assert equal(attn(q, k, v, **kw), want)
    torch.cuda.synchronize()
    attn.sync_status()
    assert equal(replay(graph, out), want)
    attn.sync_status()
    del graph
    attn.close()


def test_learned_bias_after_a_capture():
    q, k, v = tensors(*[(1, N, 700, D)] * 3)
    bias = dict(rel_bias=torch.randn(8, N, generator=torch.Generator().manual_seed(7)).cuda(),
                rel_buckets=fa.relative_buckets(8, 40))
    attn = fa.MaskedAttention("BNSD", 1, N, 700, 700, D, 2)
    want, want_bias = attn(q, k, v), attn(q, k, v, **bias)
    graph, out = capture(lambda: attn(q, k, v))
    assert equal(attn(q, k, v, **bias), want_bias)
    assert equal(replay(graph, out), want)
    attn.sync_status()
    del graph
    attn.close()


@pytest.mark.parametrize("first,then", [(ONE, MANY), (MANY, ONE)])
def test_replay_after_calls_of_other_lengths(first, then):
    q, k, v = tensors(*[(T, N, D)] * 3)
    attn = fa.MaskedAttention("TND", B, N, T, T, D, 3)

    def call(lens):
        return attn(q, k, v, actual_seq_qlen=lens, actual_seq_kvlen=lens)

    want_then, want = call(then), call(first)
    graph, out = capture(lambda: call(first))
    assert equal(replay(graph, out), want)
    assert equal(call(then), want_then)
    assert equal(replay(graph, out), want)
    graph2, out2 = capture(lambda: call(then))
    assert equal(call(first), want)
    assert equal(replay(graph, out), want) and equal(replay(graph2, out2), want_then)
    attn.sync_status()
    del graph, graph2
    attn.close()


def test_dense_mask():
    S = 515
    q, k, v = tensors(*[(2, N, S, D)] * 3)
    attn = fa.MaskedAttention("BNSD", 2, N, S, S, D, 1, mask_kind="SS")
    mask = torch.triu(torch.ones(S, S, dtype=torch.uint8), diagonal=1).cuda()
    other = torch.tril(torch.ones(S, S, dtype=torch.uint8), diagonal=-200).cuda()
    want, want_other = attn(q, k, v, atten_mask=mask), attn(q, k, v, atten_mask=other)
    graph, out = capture(lambda: attn(q, k, v, atten_mask=mask))
    assert equal(replay(graph, out), want)
    assert equal(attn(q, k, v, atten_mask=other), want_other)
    assert equal(replay(graph, out), want)
    mask.copy_(other)
    assert equal(replay(graph, out), want_other)
    attn.sync_status()
    del graph
    attn.close()


def test_paged():
    bs = 64
    q, k, v = tensors((B, N, D), (T // bs, bs, N, D), (T // bs, bs, N, D))
    table = torch.zeros(B, T // bs, dtype=torch.int32)
    table[:, 0] = torch.arange(B)
    table = table.cuda()
    attn = fa.MaskedAttention("TND", B, N, B, T, D, 3)
    rows = list(range(1, B + 1))

    def call(lens):
        return attn.paged(q, k, v, table, rows, lens)

    want = call(MANY)
    graph, out = capture(lambda: call(MANY))
    assert equal(replay(graph, out), want)
    lens = MANY[:]
    lens[0] = 1  # sequence 0 has one key, sequence 1 the rest of its share
    table[1, 1] = 0
    call(lens)
    torch.cuda.synchronize()
    assert equal(replay(graph, out), want)
    attn.sync_status()
    del graph
    attn.close()


def test_a_capture_needs_the_list():
    q, k, v = tensors(*[(T, N, D)] * 3)
    attn = fa.MaskedAttention("TND", B, N, T, T, D, 3)

    def call(lens):
        return attn(q, k, v, actual_seq_qlen=lens, actual_seq_kvlen=lens)

    want = call(ONE)
    torch.cuda.synchronize()
    with pytest.raises(fa.FaError) as e:
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            call(MANY)
    assert e.value.name == "FA_ERR_UNSUPPORTED"
    assert equal(call(ONE), want)
    torch.cuda.synchronize()
    attn.sync_status()
    attn.close()
