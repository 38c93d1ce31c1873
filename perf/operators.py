"""Measured cases of the attention training operators.

Three operators over the sparseMode geometry of the masked attention forward:

  "backward"       dq, dk, dv of O = softmax(scale q k^T + bias) v over the visible keys,
                   from q, k, v, the forward's o and lse, and the gradient do of o.  With
                   P = exp(score - lse) and delta_i = sum_d do_id o_id:
                     dV = P^T dO,  dS = P * (dO V^T - delta),  dQ = scale dS K,
                     dK = scale dS^T Q
                   (bias: none, or the right-aligned ALiBi bias slopes[h] * rel)
  "bias"           the forward with a learned relative position bias: the score of row i and
                   key j is scale q.k + table[bucket(rel), h], rel = j - (i + Skv - Sq),
                   bucket(rel) = bucket_of[clip(rel, -R, R) + R]
  "bias_backward"  the backward with that bias, and the table's gradient
                     dtable[c, h] = sum of dS over the pairs in bucket c

Every case is a dict of plain values; list-valued arguments are comma-separated texts.
With `own` false, `run` computes the plain form in elementary torch operations; with `own`
true it calls the framework's entry points.
"""
import math

import numpy as np
import torch

own = False

CHUNK = 1 << 27  # score elements a plain form holds at once


# ---------------------------------------------------------------- cases

def _case(name, op, layout, B, N, Sq, Skv, D, mode, pre=0, nxt=0, mask="", lens_q="", lens_kv="",
          prefix="", alibi=False, buckets=0, reach=0, two_sided=True):
    return {"name": name, "op": op, "layout": layout, "B": B, "N": N, "Sq": Sq, "Skv": Skv, "D": D,
            "mode": mode, "pre": pre, "next": nxt, "mask": mask, "lens_q": lens_q,
            "lens_kv": lens_kv, "prefix": prefix, "alibi": alibi, "buckets": buckets,
            "reach": reach, "two_sided": two_sided}


def listed():
    ragged_q = "513,1,2047,700,0,3001,1024,129,64,1999,2500,333"
    ragged_kv = "600,1,2047,1400,5,3100,1024,512,64,2500,2500,1000"
    packed = "130,1,257,64,5,0,399,31"
    return [
        # one short sequence per head: latency of a fine-tuning step on tiny batches
        _case("backward_causal_256", "backward", "BNSD", 1, 2, 256, 256, 64, 2),
        # an ordinary decoder training step
        _case("backward_causal_4k", "backward", "BNSD", 2, 16, 4096, 4096, 128, 2),
        # long-context training with a bidirectional prefix per batch entry (the largest)
        _case("backward_prefix_8k", "backward", "BNSD", 4, 16, 8192, 8192, 128, 5,
              prefix="512,1024,2048,4096"),
        # a sliding window over a long key axis, token-major layout
        _case("backward_band_2k_8k", "backward", "BSND", 1, 32, 2048, 8192, 128, 4, pre=1024),
        # packed sequences of unequal lengths, one empty and one of a single token
        _case("backward_varlen_12seq", "backward", "TND", 12, 16, _total(ragged_q),
              _total(ragged_kv), 128, 3, lens_q=ragged_q, lens_kv=ragged_kv),
        # documents packed into padded rows, given as an explicit mask; padding rows see nothing
        _case("backward_documents_2049", "backward", "BSND", 2, 12, 2049, 2049, 64, 1,
              mask="documents"),
        # a decoder trained with fixed ALiBi slopes
        _case("backward_alibi_2k", "backward", "BNSD", 2, 16, 2048, 2048, 128, 2, alibi=True),
        # an encoder's forward on a short odd batch
        _case("bias_encoder_200", "bias", "BNSD", 2, 8, 200, 200, 64, 0, buckets=32, reach=128),
        # an encoder's forward at length
        _case("bias_encoder_4k", "bias", "BNSD", 2, 16, 4096, 4096, 128, 0, buckets=32, reach=128),
        # one query token against a long key axis, one-sided buckets
        _case("bias_one_token_8k", "bias", "BSND", 8, 16, 1, 8191, 128, 3, buckets=32, reach=128,
              two_sided=False),
        # training on short packed sequences, one-sided buckets
        _case("bias_backward_packed", "bias_backward", "TND", 8, 6, _total(packed), _total(packed),
              64, 3, lens_q=packed, lens_kv=packed, buckets=32, reach=128, two_sided=False),
        # an encoder's training step at length
        _case("bias_backward_encoder_4k", "bias_backward", "BNSD", 2, 16, 4096, 4096, 64, 0,
              buckets=32, reach=128),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["backward", "backward", "bias", "bias_backward"])
    layout = rng.choice(["BNSD", "BSND", "TND"])
    D = rng.choice([64, 128])
    N = rng.randint(1, 16)
    buckets = reach = 0
    two_sided, alibi, mask = True, False, ""
    if op != "backward":
        buckets, reach = rng.choice([(8, 20), (32, 128), (64, 256), (10, 33)])
        two_sided = rng.random() < 0.5
    if layout == "TND":
        B = rng.randint(1, 12)
        ql, kl = [], []
        mode = rng.choice([0, 2, 3, 3, 4])
        for _ in range(B):
            n = 0 if rng.random() < 0.05 else _log_int(rng, 1, 2500)
            ql.append(n)
            kl.append(n if rng.random() < 0.5 else n + rng.randint(0, 700))
        if sum(ql) == 0:
            ql[0], kl[0] = 77, 90
        lens_q, lens_kv = ",".join(map(str, ql)), ",".join(map(str, kl))
        Sq, Skv = sum(ql), sum(kl)
    else:
        B = rng.randint(1, 4)
        lens_q = lens_kv = ""
        Sq = _log_int(rng, 33, 4096)
        Skv = Sq if rng.random() < 0.5 else _log_int(rng, 33, 4096)
        mode = rng.choice([0, 2, 3, 4, 5])
        if op == "bias" and rng.random() < 0.25:
            Sq, Skv, mode = rng.randint(1, 3), _log_int(rng, 500, 16000), 3
        if op == "backward" and rng.random() < 0.25:
            mode, mask, Skv = 1, "documents", Sq
    if op == "backward" and not mask and rng.random() < 0.2:
        alibi = True
    pre = rng.randint(0, 1500) if mode == 4 else 0
    nxt = rng.randint(-min(pre, 40), 300) if mode == 4 else 0
    prefix = ",".join(str(rng.randint(0, Skv)) for _ in range(B)) if mode == 5 else ""
    c = _case("", op, layout, B, N, Sq, Skv, D, mode, pre, nxt, mask, lens_q, lens_kv, prefix,
              alibi, buckets, reach, two_sided)
    del c["name"]
    return c


# ---------------------------------------------------------------- geometry

def _ints(text):
    return [int(x) for x in text.split(",")] if text else []


def _total(text):
    return sum(_ints(text))


def _sequences(case):
    """(b, first query token, first key token, query rows, keys) of every sequence."""
    if case["layout"] != "TND":
        return [(b, 0, 0, case["Sq"], case["Skv"]) for b in range(case["B"])]
    out, q0, k0 = [], 0, 0
    for b, (sq, skv) in enumerate(zip(_ints(case["lens_q"]), _ints(case["lens_kv"]))):
        out.append((b, q0, k0, sq, skv))
        q0, k0 = q0 + sq, k0 + skv
    return out


def _interval(case, b, i, sq, skv):
    """First and last visible key of query rows i (an integer array); empty when first > last."""
    delta, mode = skv - sq, case["mode"]
    lo, hi = i * 0, i * 0 + (skv - 1)
    if mode == 2:
        hi = i + 0
    elif mode in (3, 5):
        hi = i + delta
        if mode == 5:
            hi = hi.clip(_ints(case["prefix"])[b] - 1, None)
    elif mode == 4:
        lo, hi = i + delta - case["pre"], i + delta + case["next"]
    return lo.clip(0, None), hi.clip(None, skv - 1)


def _documents(S, b):
    """Document number of each of S tokens (-1 for padding at the end of the row)."""
    pad = (S // 16) * (b % 4) + b % 3
    doc, start, n, x = np.full(S, -1, np.int64), 0, 0, 12345 + 777 * b
    while start < S - pad:
        x = (1103515245 * x + 12345) % (1 << 31)
        end = min(S - pad, start + 1 + x % max(1, S // 3))
        doc[start:end] = n
        start, n = end, n + 1
    return doc


def _pairs(case):
    """Visible (row, key) pairs of one head over all sequences."""
    total = 0
    for b, _, _, sq, skv in _sequences(case):
        if case["mask"]:
            doc = _documents(sq, b)
            sizes = np.bincount(doc[doc >= 0], minlength=1)
            total += int((sizes * (sizes + 1) // 2).sum())
        else:
            lo, hi = _interval(case, b, np.arange(sq, dtype=np.int64), sq, skv)
            total += int((hi - lo + 1).clip(0, None).sum())
    return total


def _bucket_map(case):
    """bucket_of[rel + R] of the usual logarithmic buckets: half of a side's buckets are single
    distances, the rest grow with the logarithm up to R."""
    R, n = case["reach"], case["buckets"]
    side = n // 2 if case["two_sided"] else n
    exact_ = side // 2
    out = np.zeros(2 * R + 1, np.int32)
    for rel in range(-R, R + 1):
        base, d = 0, max(-rel, 0)
        if case["two_sided"]:
            base, d = (side if rel > 0 else 0), abs(rel)
        if d >= exact_:
            grow = math.log(d / exact_) / math.log(R / exact_) * (side - exact_)
            d = min(exact_ + int(math.floor(grow + 1e-9)), side - 1)
        out[rel + R] = base + d
    return out


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)

    def normal(shape, dtype=torch.bfloat16):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32).to(dtype)

    def shape(S):
        return {"BNSD": (case["B"], case["N"], S, case["D"]),
                "BSND": (case["B"], S, case["N"], case["D"]),
                "TND": (S, case["N"], case["D"])}[case["layout"]]

    st = {"case": case, "q": normal(shape(case["Sq"])), "k": normal(shape(case["Skv"])),
          "v": normal(shape(case["Skv"])), "mask": None, "slopes": None, "table": None,
          "bucket_of": None, "lens": {}}
    if case["mask"]:
        doc = torch.stack([torch.from_numpy(_documents(case["Sq"], b)) for b in range(case["B"])])
        doc = doc.to(dev)
        seen = (doc[:, :, None] == doc[:, None, :]) & (doc[:, :, None] >= 0)
        st["mask"] = (~seen.tril()).to(torch.uint8)[:, None].contiguous()
    if case["alibi"]:
        st["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / case["N"]) for h in range(case["N"])],
                                    device=dev, dtype=torch.float32)
    if case["buckets"]:
        st["table"] = normal((case["buckets"], case["N"]), torch.float32)
        st["bucket_of"] = _bucket_map(case)
    if case["layout"] == "TND":
        st["lens"] = {"actual_seq_qlen": np.cumsum(_ints(case["lens_q"])).tolist(),
                      "actual_seq_kvlen": np.cumsum(_ints(case["lens_kv"])).tolist()}
    if case["prefix"]:
        st["lens"]["prefix"] = _ints(case["prefix"])
    if case["op"] != "bias":
        st["o"], st["lse"] = _forward(st)
        st["do"] = normal(shape(case["Sq"]))
    if own:
        st["attention"] = _attention(case)
    return st


def _attention(case):
    import masked_attention_fa_b200 as fa
    return fa.MaskedAttention(case["layout"], case["B"], case["N"], case["Sq"], case["Skv"],
                              case["D"], case["mode"], case["pre"], case["next"],
                              mask_kind="B1SS" if case["mask"] else None,
                              alibi="right" if case["alibi"] else None)


# ---------------------------------------------------------------- the plain form, 32 bits

def _heads(x, case, b, first, n):
    """[N, n, D] view of n tokens of sequence b."""
    if case["layout"] == "BNSD":
        return x[b]
    if case["layout"] == "BSND":
        return x[b].transpose(0, 1)
    return x[first:first + n].transpose(0, 1)


def _rows(x, case, b, first, n):
    """[N, n] view of a per-row statistic of sequence b."""
    return x[:, first:first + n] if case["layout"] == "TND" else x[b]


def _chunks(case, sq, skv):
    step = max(1, CHUNK // max(1, case["N"] * skv))
    return [(r, min(sq, r + step)) for r in range(0, sq, step)]


def _scores(st, b, q, k, r0, r1, sq, skv):
    """Masked scores [N, r1 - r0, skv] of rows r0..r1, the hidden pairs and the bucket of each."""
    case, dev = st["case"], q.device
    i = torch.arange(r0, r1, device=dev)
    j = torch.arange(skv, device=dev)
    lo, hi = _interval(case, b, i, sq, skv)
    hidden = (j[None, :] < lo[:, None]) | (j[None, :] > hi[:, None])
    if st["mask"] is not None:
        hidden = hidden | (st["mask"][b, 0, r0:r1] != 0)
    s = (q[:, r0:r1] @ k.transpose(1, 2)) * (1.0 / math.sqrt(case["D"]))
    rel = j[None, :] - (i[:, None] + (skv - sq))
    bucket = None
    if st["slopes"] is not None:
        s += st["slopes"][:, None, None] * rel
    if st["table"] is not None:
        R = case["reach"]
        bucket = torch.from_numpy(st["bucket_of"]).to(dev).long()[rel.clip(-R, R) + R]
        s += st["table"].t()[:, bucket]
    return s.masked_fill_(hidden, -math.inf), bucket


def _forward(st):
    case = st["case"]
    o = torch.zeros_like(st["q"])
    rows = (case["N"], case["Sq"]) if case["layout"] == "TND" else (case["B"], case["N"], case["Sq"])
    lse = torch.full(rows, -math.inf, device=o.device, dtype=torch.float32)
    for b, q0, k0, sq, skv in _sequences(case):
        if sq == 0 or skv == 0:
            continue
        q = _heads(st["q"], case, b, q0, sq).float()
        k = _heads(st["k"], case, b, k0, skv).float()
        v = _heads(st["v"], case, b, k0, skv).float()
        for r0, r1 in _chunks(case, sq, skv):
            s, _ = _scores(st, b, q, k, r0, r1, sq, skv)
            top = s.amax(-1, keepdim=True)
            top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
            e = torch.exp_(s.sub_(top))
            den = e.sum(-1, keepdim=True)
            out = (e @ v) / torch.where(den > 0, den, torch.ones_like(den))
            _heads(o, case, b, q0, sq)[:, r0:r1] = out.to(o.dtype)
            _rows(lse, case, b, q0, sq)[:, r0:r1] = (torch.log(den) + top)[..., 0]
    return o, lse


def _backward(st):
    case = st["case"]
    scale = 1.0 / math.sqrt(case["D"])
    dq, dk, dv = (torch.zeros_like(st[x]) for x in ("q", "k", "v"))
    dtable = None
    if st["table"] is not None:
        dtable = torch.zeros(st["table"].shape, device=dq.device, dtype=torch.float64)
    for b, q0, k0, sq, skv in _sequences(case):
        if sq == 0 or skv == 0:
            continue
        q, o, do = (_heads(st[x], case, b, q0, sq).float() for x in ("q", "o", "do"))
        k, v = (_heads(st[x], case, b, k0, skv).float() for x in ("k", "v"))
        lse = _rows(st["lse"], case, b, q0, sq)
        lse = torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)  # rows that see nothing
        delta = (do * o).sum(-1)
        gk, gv = torch.zeros_like(k), torch.zeros_like(v)
        for r0, r1 in _chunks(case, sq, skv):
            s, bucket = _scores(st, b, q, k, r0, r1, sq, skv)
            p = torch.exp_(s.sub_(lse[:, r0:r1, None]))
            gv += p.transpose(1, 2) @ do[:, r0:r1]
            ds = (do[:, r0:r1] @ v.transpose(1, 2)).sub_(delta[:, r0:r1, None]).mul_(p)
            gk += ds.transpose(1, 2) @ q[:, r0:r1]
            _heads(dq, case, b, q0, sq)[:, r0:r1] = ((ds @ k) * scale).to(dq.dtype)
            if dtable is not None:
                for c in range(case["buckets"]):
                    dtable[c] += (ds * (bucket == c)).sum((1, 2), dtype=torch.float64)
        _heads(dk, case, b, k0, skv)[:] = (gk * scale).to(dk.dtype)
        _heads(dv, case, b, k0, skv)[:] = gv.to(dv.dtype)
    return (dq, dk, dv) if dtable is None else (dq, dk, dv, dtable.float())


# ---------------------------------------------------------------- one pass

def run(state):
    case = state["case"]
    if not own:
        return _forward(state) if case["op"] == "bias" else _backward(state)
    if "attention" not in state:
        state["attention"] = _attention(case)
    bias = {}
    if state["table"] is not None:
        bias = {"rel_bias": state["table"], "rel_buckets": state["bucket_of"]}
    if case["op"] == "bias":
        return state["attention"](state["q"], state["k"], state["v"], **state["lens"], **bias)
    return state["attention"].backward(state["do"], state["q"], state["k"], state["v"], state["o"],
                                       state["lse"], atten_mask=state["mask"],
                                       slopes=state["slopes"], **state["lens"], **bias)


def work(case):
    pairs, N, D = _pairs(case) * case["N"], case["N"], case["D"]
    rows_q = case["Sq"] * (1 if case["layout"] == "TND" else case["B"]) * N
    rows_k = case["Skv"] * (1 if case["layout"] == "TND" else case["B"]) * N
    table = 4 * case["buckets"] * N
    if case["op"] == "bias":
        return {"bytes": 2 * D * (2 * rows_q + 2 * rows_k) + 4 * rows_q + table, "flops": 4 * D * pairs}
    mask = case["B"] * case["Sq"] * case["Skv"] if case["mask"] else 0
    return {"bytes": 2 * D * (4 * rows_q + 4 * rows_k) + 4 * rows_q + mask + 2 * table,
            "flops": 10 * D * pairs}


# ---------------------------------------------------------------- 64 bits

def exact(case, seed):
    """The formulas of the module's docstring head by head in 64 bits."""
    st = prepare(case, seed)
    dev, f64 = st["q"].device, torch.float64
    N, scale = case["N"], 1.0 / math.sqrt(case["D"])
    backward = case["op"] != "bias"
    names = ("q", "k", "v") if backward else ("q",)
    out = [torch.zeros(st[x].shape, device=dev, dtype=f64) for x in names]
    rows = (N, case["Sq"]) if case["layout"] == "TND" else (case["B"], N, case["Sq"])
    lse_out = torch.full(rows, -math.inf, device=dev, dtype=f64)
    grad = torch.zeros((case["buckets"], N), device=dev, dtype=f64)

    def pick(x, b, h, first, n):
        if case["layout"] == "BNSD":
            return x[b, h]
        return x[b, :, h] if case["layout"] == "BSND" else x[first:first + n, h]

    for b, q0, k0, sq, skv in _sequences(case):
        if min(sq, skv) == 0:
            continue
        at = np.arange(sq)[:, None]
        key = np.arange(skv)[None, :]
        lo, hi = _interval(case, b, at, sq, skv)
        see = torch.from_numpy((key >= lo) & (key <= hi)).to(dev)
        if st["mask"] is not None:
            see &= st["mask"][b, 0] == 0
        rel = torch.arange(skv, device=dev)[None] - torch.arange(skv - sq, skv, device=dev)[:, None]
        if case["buckets"]:
            R = case["reach"]
            to = torch.from_numpy(st["bucket_of"]).to(dev).long()
            cell = to[(rel + R).clamp(0, 2 * R)]
        for h in range(N):
            q, k, v = (pick(st[x], b, h, f, n).to(f64) for x, f, n in
                       (("q", q0, sq), ("k", k0, skv), ("v", k0, skv)))
            z = torch.einsum("id,jd->ij", q, k) * scale
            if case["alibi"]:
                z = z + st["slopes"][h].to(f64) * rel
            if case["buckets"]:
                z = z + st["table"][:, h].to(f64)[cell]
            if not backward:
                z = z.masked_fill(~see, -math.inf)
                den = torch.logsumexp(z, 1)
                w = torch.exp(z - den[:, None]).masked_fill(~see, 0.0)
                pick(out[0], b, h, q0, sq).copy_(torch.einsum("ij,jd->id", w, v))
                (lse_out[h, q0:q0 + sq] if case["layout"] == "TND" else lse_out[b, h]).copy_(den)
                continue
            den = st["lse"][h, q0:q0 + sq] if case["layout"] == "TND" else st["lse"][b, h]
            o, do = (pick(st[x], b, h, q0, sq).to(f64) for x in ("o", "do"))
            w = torch.where(see, torch.exp(z - den.to(f64)[:, None]), torch.zeros((), device=dev, dtype=f64))
            pick(out[2], b, h, k0, skv).copy_(torch.einsum("ij,id->jd", w, do))
            w = w * (torch.einsum("id,jd->ij", do, v) - torch.einsum("id,id->i", do, o)[:, None])
            pick(out[0], b, h, q0, sq).copy_(torch.einsum("ij,jd->id", w, k) * scale)
            pick(out[1], b, h, k0, skv).copy_(torch.einsum("ij,id->jd", w, q) * scale)
            if case["buckets"]:
                # row i of `diag` is row i of w shifted so that equal distances share a column
                wide = torch.zeros((sq, sq + skv), device=dev, dtype=f64)
                wide[:, sq:] = w
                diag = torch.cat([wide.flatten(), wide.new_zeros(sq)]).view(sq, sq + skv + 1)
                dist = torch.arange(sq + skv + 1, device=dev) - sq - (skv - sq)
                grad[:, h].index_add_(0, to[(dist + R).clamp(0, 2 * R)], diag.sum(0))
    if not backward:
        return out[0], lse_out
    return (*out, grad) if case["buckets"] else tuple(out)
