"""The serving operators over a paged key-value cache: cases, inputs, plain forms.

paged_append   rotate packed queries and keys, write keys and values into cache pages
paged_decode   attention of one new token per sequence over the pages
packed_prefill causal attention of packed prompts of different lengths
paged_prefill  the same with keys and values read from the pages (chunks after a prefix)

``run`` computes them in elementary torch operations in 32 bits, or, where
``own`` is true, by the package's entry points.
"""
import math

import numpy as np
import torch

own = False

D = 128                 # head size
SCRATCH = 64 << 20      # bytes of scratch that a serving program keeps for these calls


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token of one conversation: what the append costs when nothing hides its latency
        dict(name="append_step_b1", op="append", heads=32, kv_heads=8, page=16, seqs=1, new=1, prefix=1000, ragged=False),
        # a decode step of a batch of conversations of every length
        dict(name="append_step_b64", op="append", heads=32, kv_heads=8, page=16, seqs=64, new=1, prefix=8191,
             ragged=True),
        # a batch of fresh prompts, odd lengths: the cache fill of a prefill step
        dict(name="append_prompts_b7", op="append", heads=32, kv_heads=8, page=64, seqs=7, new=4095, prefix=0,
             ragged=True),
        # the first tokens of one conversation
        dict(name="decode_b1_p15", op="decode", heads=32, kv_heads=8, page=16, seqs=1, prefix=15, ragged=False),
        # the benchmark's batch: 16 sequences of 1,000 cached rows
        dict(name="decode_b16_p1000", op="decode", heads=32, kv_heads=8, page=16, seqs=16, prefix=1000, ragged=False),
        # the multi-head variant of the same batch: four times the cache
        dict(name="decode_mha_b16_p1000", op="decode", heads=32, kv_heads=32, page=32, seqs=16, prefix=1000,
             ragged=False),
        # a full server: conversations from one row to 8,192
        dict(name="decode_b64_ragged", op="decode", heads=32, kv_heads=8, page=64, seqs=64, prefix=8191, ragged=True),
        # one conversation at the end of its context window
        dict(name="decode_b1_p131071", op="decode", heads=32, kv_heads=8, page=128, seqs=1, prefix=131071,
             ragged=False),
        # a short question, pages as fresh as the prompt
        dict(name="prefill_paged_17", op="paged_prefill", heads=32, kv_heads=8, page=16, seqs=1, new=17, prefix=0,
             ragged=False),
        # the benchmark's prompt
        dict(name="prefill_packed_2048", op="packed_prefill", heads=32, kv_heads=8, seqs=1, new=2048, prefix=0,
             ragged=False),
        # a batch of prompts of odd lengths, one of them empty
        dict(name="prefill_packed_b9", op="packed_prefill", heads=32, kv_heads=8, seqs=9, new=4095, prefix=0,
             ragged=True),
        # the last chunk of an 8,192-token prompt, its prefix in the cache
        dict(name="prefill_chunk_p7168", op="paged_prefill", heads=32, kv_heads=8, page=64, seqs=1, new=1024,
             prefix=7168, ragged=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    """One more case: head layouts from a multi-head model to a slice with one KV head, sizes over their logarithm."""
    heads, kv_heads = rng.choice([(32, 8), (32, 8), (32, 32), (16, 4), (8, 2), (4, 1), (28, 4), (64, 4)])
    page = rng.choice([16, 32, 64, 128, 256])
    op = rng.choice(["append", "decode", "decode", "paged_prefill", "packed_prefill"])
    ragged = rng.random() < 0.7
    c = dict(op=op, heads=heads, kv_heads=kv_heads, page=page, ragged=ragged)
    if op == "append":
        new = _log(rng, 1, 4096)
        c.update(seqs=_log(rng, 1, max(1, 16384 // new)) if new > 64 else _log(rng, 1, 256), new=new,
                 prefix=rng.choice([0, _log(rng, 1, 8192)]))
    elif op == "decode":
        seqs = _log(rng, 1, 128)
        c.update(seqs=seqs, prefix=_log(rng, 1, max(16, min(131072, (1 << 22) // (seqs * kv_heads)))))
    else:
        seqs = _log(rng, 1, 8)
        new = _log(rng, 1, 4096 // seqs)
        c.update(seqs=seqs, new=new, prefix=rng.choice([0, _log(rng, 1, 8192 // seqs)]) if op == "paged_prefill" else 0)
        if op == "packed_prefill":
            del c["page"]
    return c


def _lengths(case, longest, salt):
    """One length per sequence: all `longest`, or, ragged, from the longest down to almost none, in no order."""
    n = case["seqs"]
    if not case["ragged"] or n == 1:
        return [longest] * n
    return [longest if i == n // 2 else int(longest * ((0.6180339887498949 * (i + salt)) % 1.0)) for i in range(n)]


def _shape(case):
    """(new tokens of each sequence, cached rows before them)."""
    new = [1] * case["seqs"] if case["op"] == "decode" or case["new"] == 1 else _lengths(case, case["new"], 1)
    return new, _lengths(case, case["prefix"], 3)


def work(case):
    new, start = _shape(case)
    heads, kv, n = case["heads"], case["kv_heads"], sum(new)
    rows = sum(s + t for s, t in zip(start, new) if t)
    index = 8 * len(new)
    if case["op"] == "append":
        positions = max((s + t for s, t in zip(start, new) if t), default=0)
        return {"bytes": n * (heads + 2 * kv) * D * 4 + min(n, positions) * D * 4 + index, "flops": 3 * n * (heads + kv) * D}
    pairs = sum(t * s + t * (t + 1) // 2 for s, t in zip(start, new))
    if "page" in case:
        index += 4 * sum(-(-(s + t) // case["page"]) for s, t in zip(start, new) if t)
    return {"bytes": n * heads * D * 4 + rows * kv * D * 4 + index, "flops": 4 * heads * D * pairs}


# ------------------------------------------------------------------ inputs

def _rope(rows):
    """(cos, sin) of position x theta^(-2i/128), theta 500000."""
    f = 500000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64, device="cuda") / D)
    a = torch.arange(rows, dtype=torch.float64, device="cuda")[:, None] * f
    return torch.stack([a.cos(), a.sin()], -1).float()


def _normal(g, *shape, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * scale).bfloat16()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    new, start = _shape(case)
    heads, kv, n, op = case["heads"], case["kv_heads"], sum(new), case["op"]
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    s = dict(op=op, heads=heads, kv=kv, longest=max(new), deepest=max(a + t for a, t in zip(start, new)),
             cu=torch.from_numpy(cu).cuda(), start=torch.tensor(start, dtype=torch.int32, device="cuda"),
             workspace=torch.zeros(SCRATCH, dtype=torch.uint8, device="cuda"))
    if op in ("append", "packed_prefill"):
        # one projection's output rows, q | k | v: the three are views of it
        qkv = _normal(g, n, heads + 2 * kv, D, scale=1.5)
        s["q"], s["k"], s["v"] = qkv[:, :heads], qkv[:, heads:heads + kv], qkv[:, heads + kv:]
    else:
        s["q"] = _normal(g, n, heads, D, scale=1.5)
    if op != "packed_prefill":
        page = case["page"]
        columns = -(-s["deepest"] // page)
        pages = len(new) * columns + 1
        s["page"] = page
        # pages are handed out in no order
        s["table"] = torch.randperm(pages, generator=g, device="cuda")[:len(new) * columns].view(len(new), columns).int()
        s["k_pages"] = _normal(g, pages, page, kv, D)
        s["v_pages"] = _normal(g, pages, page, kv, D)
    if op == "append":
        s["rope"] = _rope(s["deepest"])
        s["q_out"] = torch.empty(n, heads, D, dtype=torch.bfloat16, device="cuda")
    else:
        s["out"] = torch.empty(n, heads, D, dtype=torch.bfloat16, device="cuda")
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    return _run_own(s) if own else _PLAIN[s["op"]](s)


def _run_own(s):
    import grouped_query_attention_gemv_gb300 as G
    if s["op"] == "append":
        G.paged_append(s["q"], s["k"], s["v"], s["start"], s["rope"], s["k_pages"], s["v_pages"], s["table"],
                       cu_tokens=s["cu"], q_out=s["q_out"], workspace=s["workspace"])
        return s["q_out"], s["k_pages"], s["v_pages"]
    if s["op"] == "decode":
        return G.paged_decode(s["q"], s["start"], s["k_pages"], s["v_pages"], s["table"], out=s["out"],
                              workspace=s["workspace"])
    if s["op"] == "paged_prefill":
        return G.paged_prefill(s["q"], s["cu"], s["start"], s["k_pages"], s["v_pages"], s["table"], out=s["out"],
                               workspace=s["workspace"])
    return G.packed_prefill(s["q"], s["k"], s["v"], s["cu"], out=s["out"], workspace=s["workspace"])


def _tokens(s):
    """Sequence of each packed token, and its place in it."""
    m = torch.arange(s["q"].shape[0], device="cuda")
    b = torch.searchsorted(s["cu"][1:].long(), m, right=True)
    return b, m - s["cu"].long()[b]


def _rotated(x, cs):
    x = x.float().unflatten(-1, (D // 2, 2))
    a, b, c, d = x[..., 0], x[..., 1], cs[:, None, :, 0], cs[:, None, :, 1]
    return torch.stack([a * c - b * d, a * d + b * c], -1).flatten(-2).bfloat16()


def _plain_append(s):
    b, i = _tokens(s)
    p = s["start"].long()[b] + i
    cs = s["rope"][p]
    page, row = s["table"].long()[b, p // s["page"]], p % s["page"]
    s["q_out"].copy_(_rotated(s["q"], cs))
    s["k_pages"][page, row] = _rotated(s["k"], cs)
    s["v_pages"][page, row] = s["v"]
    return s["q_out"], s["k_pages"], s["v_pages"]


def _attend(q, k, v, last):
    """q [b, t, h, d], k, v [b, s, g, d] in 32 bits; query (b, t) sees keys 0..last[b, t], none where that is -1."""
    q = q.unflatten(2, (k.shape[2], -1))
    key = torch.arange(k.shape[1], device="cuda")
    v = v * (key <= last.amax(1, keepdim=True))[:, :, None, None]
    x = torch.einsum("btgrd,bsgd->bgrts", q, k) * D ** -0.5
    x.masked_fill_((key > last[:, :, None])[:, None, None], -math.inf)
    x -= x.amax(-1, keepdim=True).clamp_min(-1e30)
    x.exp_()
    total = x.sum(-1, keepdim=True)
    x /= total.clamp_min(1e-30)
    return torch.einsum("bgrts,bsgd->btgrd", x, v).flatten(2, 3)


def _plain_decode(s):
    k = s["k_pages"][s["table"].long()].flatten(1, 2).float()
    v = s["v_pages"][s["table"].long()].flatten(1, 2).float()
    s["out"].copy_(_attend(s["q"].float()[:, None], k, v, s["start"].long()[:, None])[:, 0])
    return s["out"]


def _plain_prefill(s):
    b, i = _tokens(s)
    n = s["cu"].numel() - 1
    q = torch.zeros(n, s["longest"], s["heads"], D, device="cuda")
    q[b, i] = s["q"].float()
    t = torch.arange(s["longest"], device="cuda")
    if s["op"] == "packed_prefill":
        k, v = (torch.zeros(n, s["longest"], s["kv"], D, device="cuda") for _ in range(2))
        k[b, i], v[b, i] = s["k"].float(), s["v"].float()
        last = t.expand(n, -1)
    else:
        k = s["k_pages"][s["table"].long()].flatten(1, 2).float()
        v = s["v_pages"][s["table"].long()].flatten(1, 2).float()
        last = s["start"].long()[:, None] + t
    s["out"].copy_(_attend(q, k, v, last)[b, i])
    return s["out"]


_PLAIN = {"append": _plain_append, "decode": _plain_decode, "paged_prefill": _plain_prefill,
          "packed_prefill": _plain_prefill}


# ------------------------------------------------------------------ from the definition, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    new, start = _shape(case)
    heads, kv, op = case["heads"], case["kv_heads"], case["op"]
    first = np.concatenate([[0], np.cumsum(new)])
    out = torch.zeros(sum(new), heads, D, dtype=torch.float64, device="cuda")
    if op == "append":
        kp, vp = s["k_pages"].double(), s["v_pages"].double()
        # the table's angles, as complex numbers
        turn = torch.view_as_complex(s["rope"].double())
        for b, (t, a) in enumerate(zip(new, start)):
            if not t:
                continue
            rows = slice(int(first[b]), int(first[b]) + t)
            at = torch.arange(a, a + t, device="cuda")
            spot = s["table"][b].long()[at // case["page"]] * case["page"] + at % case["page"]
            z = torch.view_as_complex(s["q"][rows].double().reshape(t, heads, D // 2, 2).contiguous()) * turn[at][:, None]
            out[rows] = torch.view_as_real(z).reshape(t, heads, D)
            z = torch.view_as_complex(s["k"][rows].double().reshape(t, kv, D // 2, 2).contiguous()) * turn[at][:, None]
            kp.view(-1, kv, D)[spot] = torch.view_as_real(z).reshape(t, kv, D)
            vp.view(-1, kv, D)[spot] = s["v"][rows].double()
        return out, kp, vp
    for b, (t, a) in enumerate(zip(new, start)):
        if not t:
            continue
        rows = slice(int(first[b]), int(first[b]) + t)
        if op == "packed_prefill":
            ks, vs = s["k"][rows].double(), s["v"][rows].double()
        else:
            at = torch.arange(a + t, device="cuda")
            spot = s["table"][b].long()[at // case["page"]] * case["page"] + at % case["page"]
            ks, vs = (x.view(-1, kv, D)[spot].double() for x in (s["k_pages"], s["v_pages"]))
            # a decode step's own row is in the cache: start rows before it, and itself
        hidden = torch.ones(t, a + t, dtype=torch.bool, device="cuda").triu(a + 1)
        for h in range(heads):
            g = h * kv // heads
            x = (s["q"][rows, h].double() @ ks[:, g].T) / math.sqrt(D)
            out[rows, h] = torch.softmax(x.masked_fill(hidden, -math.inf), -1) @ vs[:, g]
    return out
