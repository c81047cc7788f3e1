"""More serving operators over a paged key-value cache: cases, inputs, plain forms.

append   rotate packed queries and keys, write keys and values into cache pages: rotary layouts that pair dim i with
         i + half, or rotate a part of the head; pages in bf16, or in 8 bits, quantised as they are written
read     rows of an 8-bit cache back into bf16 pages
decode   attention of one new token per sequence over an 8-bit cache
shared   attention of one new token per sequence over a bf16 cache, groups of sequences sharing their first rows

An 8-bit row (128 values of one token and head) is held as e4m3 times 2^e, e in [-100, 120] the least with
|row| <= 448 x 2^e; its byte e + 127 lies beside the pages.

``run`` computes them in elementary torch operations in 32 bits, or, where ``own`` is true, by the package's entry
points.
"""
import math

import numpy as np
import torch

own = False

D = 128                 # head size
SCRATCH = 64 << 20      # bytes of scratch that a serving program keeps for these calls
LEAST_E, MOST_E = -100, 120


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token of one conversation into an 8-bit cache: what the call costs when nothing hides its latency
        dict(name="append8_step_b1", op="append", bits=8, heads=32, kv_heads=8, page=16, rotary=128, halves=False, seqs=1,
             new=1, prefix=1000, ragged=False),
        # a batch of fresh prompts, odd lengths: the 8-bit cache's fill of a prefill step
        dict(name="append8_prompts_b7", op="append", bits=8, heads=32, kv_heads=8, page=64, rotary=128, halves=True,
             seqs=7, new=4095, prefix=0, ragged=True),
        # a decode step of a batch, weights in the layout that pairs the two halves of a head
        dict(name="append_halves_b64", op="append", bits=16, heads=32, kv_heads=8, page=16, rotary=128, halves=True,
             seqs=64, new=1, prefix=8191, ragged=True),
        # prompts of a model that rotates half of each head, pairs side by side
        dict(name="append_part_b5", op="append", bits=16, heads=32, kv_heads=8, page=64, rotary=64, halves=False,
             seqs=5, new=4095, prefix=0, ragged=True),
        # the prefix of one prompt's last chunk, for the prefill attention
        dict(name="read8_p7168", op="read", heads=32, kv_heads=8, page=64, to_page=64, seqs=1, prefix=7168, ragged=False),
        # many conversations moved to a bf16 cache of another page size
        dict(name="read8_b48_ragged", op="read", heads=32, kv_heads=8, page=16, to_page=128, seqs=48, prefix=8191,
             ragged=True),
        # the first tokens of one conversation
        dict(name="decode8_b1_p15", op="decode", heads=32, kv_heads=8, page=16, seqs=1, prefix=15, ragged=False),
        # the benchmark's batch: 16 sequences of 1,000 cached rows
        dict(name="decode8_b16_p1000", op="decode", heads=32, kv_heads=8, page=16, seqs=16, prefix=1000, ragged=False),
        # a full server: conversations from one row to 8,192
        dict(name="decode8_b64_ragged", op="decode", heads=32, kv_heads=8, page=64, seqs=64, prefix=8191, ragged=True),
        # four samples of one prompt, a few tokens in
        dict(name="shared_b4_p511", op="shared", heads=32, kv_heads=8, page=16, seqs=4, groups=1, prefix=511, own_rows=8,
             ragged=True),
        # one system prompt under a batch of conversations
        dict(name="shared_b64_p8000", op="shared", heads=32, kv_heads=8, page=64, seqs=64, groups=1, prefix=8000,
             own_rows=512, ragged=True),
        # three system prompts of different lengths
        dict(name="shared_b96_g3", op="shared", heads=32, kv_heads=8, page=16, seqs=96, groups=3, prefix=4095,
             own_rows=900, ragged=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    """One more case: head layouts from a multi-head model to a slice with one KV head, sizes over their logarithm."""
    heads, kv_heads = rng.choice([(32, 8), (32, 8), (32, 32), (16, 4), (8, 2), (4, 1), (28, 4), (64, 4)])
    page = rng.choice([16, 32, 64, 128, 256])
    op = rng.choice(["append", "append", "read", "decode", "decode", "shared", "shared"])
    c = dict(op=op, heads=heads, kv_heads=kv_heads, page=page, ragged=rng.random() < 0.7)
    if op == "append":
        new = _log(rng, 1, 4096)
        c.update(bits=rng.choice([8, 8, 16]), rotary=rng.choice([128, 128, 64, 32, 96]), halves=rng.random() < 0.5,
                 seqs=_log(rng, 1, max(1, 12288 // new)) if new > 64 else _log(rng, 1, 256), new=new,
                 prefix=rng.choice([0, _log(rng, 1, 8192)]))
        if c["bits"] == 16 and c["rotary"] == 128:
            c["halves"] = True
    elif op in ("read", "decode"):
        seqs = _log(rng, 1, 128)
        most = 1 << (20 if op == "read" else 21)
        c.update(seqs=seqs, prefix=_log(rng, 1, max(16, min(131072, most // (seqs * kv_heads)))))
        if op == "read":
            c["to_page"] = rng.choice([16, 64, 128, 1024])
    else:
        seqs = _log(rng, 2, 128)
        rows = max(32, (1 << 22) // (seqs * kv_heads))
        c.update(seqs=seqs, groups=rng.randint(1, min(4, seqs)), prefix=_log(rng, 1, min(32768, rows * 7 // 8)),
                 own_rows=_log(rng, 1, min(2048, max(2, rows // 8))))
    return c


def _lengths(case, n, longest, salt):
    """One length for each of n: all `longest`, or, ragged, from the longest down to almost none, in no order."""
    if not case["ragged"] or n == 1:
        return [longest] * n
    return [longest if i == n // 2 else int(longest * ((0.6180339887498949 * (i + salt)) % 1.0)) for i in range(n)]


def _shape(case):
    """(new tokens of each sequence, cached rows before them)."""
    n = case["seqs"]
    if case["op"] == "append":
        new = [1] * n if case["new"] == 1 else _lengths(case, n, case["new"], 1)
        return new, _lengths(case, n, case["prefix"], 3)
    if case["op"] == "shared":
        prefix, group = _groups(case)
        own_rows = [max(1, x) for x in _lengths(case, n, case["own_rows"], 3)]
        return [1] * n, [prefix[g] + x - 1 for g, x in zip(group, own_rows)]
    return [1] * n, _lengths(case, n, case["prefix"], 3)


def _groups(case):
    """(shared rows of each group, group of each sequence): groups of like sizes, one after the other."""
    n, g = case["seqs"], case["groups"]
    return _lengths(case, g, case["prefix"], 2), [i * g // n for i in range(n)]


def work(case):
    new, start = _shape(case)
    heads, kv, n, op = case["heads"], case["kv_heads"], sum(new), case["op"]
    index = 8 * len(new)
    if op == "append":
        positions = max((s + t for s, t in zip(start, new) if t), default=0)
        row = D * 2 + (D * 2 if case["bits"] == 16 else D + 1)
        return {"bytes": n * heads * D * 4 + n * 2 * kv * row + min(n, positions) * case["rotary"] * 4 + index,
                "flops": 3 * n * (heads + kv) * case["rotary"]}
    if op == "read":
        rows = sum(start)
        index += 4 * sum(-(-s // case["page"]) + -(-s // case["to_page"]) for s in start)
        return {"bytes": rows * 2 * kv * (D + 1 + 2 * D) + index, "flops": rows * 2 * kv * D}
    rows = sum(s + 1 for s in start)
    pages = sum(-(-(s + 1) // case["page"]) for s in start)
    flops = 4 * heads * D * rows
    if op == "decode":
        return {"bytes": n * heads * D * 4 + rows * 2 * kv * (D + 1) + index + 4 * pages, "flops": flops}
    prefix, group = _groups(case)
    rows = sum(s + 1 - prefix[g] for s, g in zip(start, group)) + sum(prefix)
    pages = sum(-(-(s + 1) // case["page"]) - prefix[g] // case["page"] for s, g in zip(start, group))
    pages += sum(p // case["page"] for p in prefix)
    return {"bytes": n * heads * D * 4 + rows * 2 * kv * D * 2 + index + 4 * pages + 8 * len(prefix), "flops": flops}


# ------------------------------------------------------------------ inputs

def _rope(rows, rotary):
    """(cos, sin) of position x theta^(-2i/rotary), theta 500000."""
    f = 500000.0 ** (-torch.arange(0, rotary, 2, dtype=torch.float64, device="cuda") / rotary)
    a = torch.arange(rows, dtype=torch.float64, device="cuda")[:, None] * f
    return torch.stack([a.cos(), a.sin()], -1).float()


def _normal(g, *shape, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * scale).bfloat16()


def _quantised(g, pages, page, kv):
    """Pages of rows as an append leaves them: the largest value of a row between 224 and 448 units."""
    x = torch.randn(pages, page, kv, D, generator=g, device="cuda")
    x *= 2.0 ** torch.randint(-3, 4, (pages, page, kv, 1), generator=g, device="cuda")
    e = _exponent(x)
    return (x * _power(-e)).to(torch.float8_e4m3fn), (e[..., 0] + 127).to(torch.uint8)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    new, start = _shape(case)
    heads, kv, n, op, page = case["heads"], case["kv_heads"], sum(new), case["op"], case["page"]
    s = dict(op=op, heads=heads, kv=kv, page=page, start=torch.tensor(start, dtype=torch.int32, device="cuda"),
             workspace=torch.zeros(SCRATCH, dtype=torch.uint8, device="cuda"))
    # cached rows of each sequence, its new ones among them
    rows = start if op == "read" else [a + t for a, t in zip(start, new)]
    columns = max(1, -(-max(rows) // page))
    pages = len(new) * columns + 1
    # pages are handed out in no order
    table = torch.randperm(pages, generator=g, device="cuda")[:len(new) * columns].view(len(new), columns).int()
    bits = case.get("bits", 16 if op == "shared" else 8)
    if bits == 16:
        s["k_pages"], s["v_pages"] = _normal(g, pages, page, kv, D), _normal(g, pages, page, kv, D)
    else:
        s["k_pages"], s["k_scales"] = _quantised(g, pages, page, kv)
        s["v_pages"], s["v_scales"] = _quantised(g, pages, page, kv)
    if op == "append":
        cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        # one projection's output rows, q | k | v: the three are views of it
        qkv = _normal(g, n, heads + 2 * kv, D, scale=1.5)
        s.update(bits=bits, rotary=case["rotary"], halves=case["halves"], cu=torch.from_numpy(cu).cuda(),
                 rope=_rope(max(rows), case["rotary"]), q=qkv[:, :heads], k=qkv[:, heads:heads + kv],
                 v=qkv[:, heads + kv:], q_out=torch.empty(n, heads, D, dtype=torch.bfloat16, device="cuda"))
    elif op == "read":
        to = case["to_page"]
        columns = max(1, -(-max(rows) // to))
        s["to_page"] = to
        s["to_table"] = torch.randperm(len(new) * columns, generator=g, device="cuda").view(len(new), columns).int()
        s["k_out"], s["v_out"] = (torch.zeros(len(new) * columns, to, kv, D, dtype=torch.bfloat16, device="cuda")
                                  for _ in range(2))
    else:
        s["q"] = _normal(g, n, heads, D, scale=1.5)
        s["out"] = torch.empty(n, heads, D, dtype=torch.bfloat16, device="cuda")
    if op == "shared":
        prefix, group = _groups(case)
        cu = [0]
        for i, p in enumerate(prefix):
            a, b = group.index(i), len(group) - group[::-1].index(i)
            cu.append(b)
            # whole pages of the prefix are one copy, the page that it ends in each sequence has to itself
            full = p // page
            table[a:b, :full] = table[a, :full].clone()
            if p % page:
                to = table[a:b, full].long()
                for x in (s["k_pages"], s["v_pages"]):
                    x[to, :p % page] = x[to[0], :p % page].clone()
        s["cu_groups"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        s["prefix"] = torch.tensor(prefix, dtype=torch.int32, device="cuda")
    s["table"] = table
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    return _run_own(s) if own else _PLAIN[s["op"]](s)


def _run_own(s):
    import grouped_query_attention_gemv_gb300 as G
    if s["op"] == "append" and s["bits"] == 8:
        G.paged_append_fp8(s["q"], s["k"], s["v"], s["start"], s["rope"], s["k_pages"], s["v_pages"], s["k_scales"],
                           s["v_scales"], s["table"], cu_tokens=s["cu"], q_out=s["q_out"], rotary_dim=s["rotary"],
                           halves=s["halves"], workspace=s["workspace"])
        return s["q_out"], s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"]
    if s["op"] == "append":
        G.paged_append(s["q"], s["k"], s["v"], s["start"], s["rope"], s["k_pages"], s["v_pages"], s["table"],
                       cu_tokens=s["cu"], q_out=s["q_out"], rotary_dim=s["rotary"], halves=s["halves"],
                       workspace=s["workspace"])
        return s["q_out"], s["k_pages"], s["v_pages"]
    if s["op"] == "read":
        G.paged_read_fp8(s["start"], s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"], s["table"], s["k_out"],
                         s["v_out"], s["to_table"], workspace=s["workspace"])
        return s["k_out"], s["v_out"]
    if s["op"] == "decode":
        return G.paged_decode_fp8(s["q"], s["start"], s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"],
                                  s["table"], out=s["out"], workspace=s["workspace"])
    return G.paged_decode_shared(s["q"], s["start"], s["cu_groups"], s["prefix"], s["k_pages"], s["v_pages"],
                                 s["table"], out=s["out"], workspace=s["workspace"])


def _rotated(x, cs, halves):
    """x [n, h, 128], its first dims turned by cs [n, pairs, 2]."""
    x = x.float()
    r = 2 * cs.shape[1]
    y = x[..., :r].unflatten(-1, (2, -1)).transpose(-1, -2) if halves else x[..., :r].unflatten(-1, (-1, 2))
    a, b, c, d = y[..., 0], y[..., 1], cs[:, None, :, 0], cs[:, None, :, 1]
    y = torch.stack([a * c - b * d, a * d + b * c], -1)
    y = (y.transpose(-1, -2) if halves else y).flatten(-2)
    return torch.cat([y, x[..., r:]], -1)


def _exponent(x):
    """e of rows [..., 128], [..., 1]: the least with |row| <= 448 x 2^e. 448 is 0.875 x 2^9."""
    m, e = torch.frexp(x.abs().amax(-1, keepdim=True))
    return (e - 9 + (m > 0.875).int()).clamp(LEAST_E, MOST_E)


def _power(e):
    """2^e for whole e in [-126, 127], by its bits: a rounded power would break ties."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _plain_append(s):
    m = torch.arange(s["q"].shape[0], device="cuda")
    b = torch.searchsorted(s["cu"][1:].long(), m, right=True)
    p = s["start"].long()[b] + m - s["cu"].long()[b]
    cs = s["rope"][p]
    page, row = s["table"].long()[b, p // s["page"]], p % s["page"]
    s["q_out"].copy_(_rotated(s["q"], cs, s["halves"]))
    k, v = _rotated(s["k"], cs, s["halves"]), s["v"].float()
    if s["bits"] == 16:
        s["k_pages"][page, row] = k.bfloat16()
        s["v_pages"][page, row] = v.bfloat16()
        return s["q_out"], s["k_pages"], s["v_pages"]
    ke, ve = _exponent(k), _exponent(v)
    s["k_pages"].view(torch.uint8)[page, row] = (k * _power(-ke)).to(torch.float8_e4m3fn).view(torch.uint8)
    s["v_pages"].view(torch.uint8)[page, row] = (v * _power(-ve)).to(torch.float8_e4m3fn).view(torch.uint8)
    s["k_scales"][page, row] = (ke[..., 0] + 127).to(torch.uint8)
    s["v_scales"][page, row] = (ve[..., 0] + 127).to(torch.uint8)
    return s["q_out"], s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"]


def _values(pages, scales, table):
    """Rows of the sequences as the values that they stand for: [b, rows, kv, 128]."""
    t = table.long()
    e = scales[t].flatten(1, 2).int() - 127
    return pages.view(torch.uint8)[t].view(torch.float8_e4m3fn).flatten(1, 2).float() * _power(e)[..., None]


def _plain_read(s):
    b, p = (torch.arange(s["table"].shape[1] * s["page"], device="cuda")[None] < s["start"][:, None]).nonzero(as_tuple=True)
    at = s["to_table"].long()[b, p // s["to_page"]], p % s["to_page"]
    s["k_out"][at] = _values(s["k_pages"], s["k_scales"], s["table"])[b, p].bfloat16()
    s["v_out"][at] = _values(s["v_pages"], s["v_scales"], s["table"])[b, p].bfloat16()
    return s["k_out"], s["v_out"]


def _attend(q, k, v, last):
    """q [b, h, d], k, v [b, s, g, d] in 32 bits; query b sees keys 0..last[b]."""
    q = q.unflatten(1, (k.shape[2], -1))
    hidden = torch.arange(k.shape[1], device="cuda") > last[:, None]
    v = v * ~hidden[:, :, None, None]
    x = torch.einsum("bgrd,bsgd->bgrs", q, k) * D ** -0.5
    x.masked_fill_(hidden[:, None, None], -math.inf)
    x = (x - x.amax(-1, keepdim=True)).exp()
    return (torch.einsum("bgrs,bsgd->bgrd", x, v) / x.sum(-1, keepdim=True)).flatten(1, 2)


def _plain_decode(s):
    k = _values(s["k_pages"], s["k_scales"], s["table"])
    v = _values(s["v_pages"], s["v_scales"], s["table"])
    s["out"].copy_(_attend(s["q"].float(), k, v, s["start"].long()))
    return s["out"]


def _plain_shared(s):
    k = s["k_pages"][s["table"].long()].flatten(1, 2).float()
    v = s["v_pages"][s["table"].long()].flatten(1, 2).float()
    s["out"].copy_(_attend(s["q"].float(), k, v, s["start"].long()))
    return s["out"]


_PLAIN = {"append": _plain_append, "read": _plain_read, "decode": _plain_decode, "shared": _plain_shared}


# ------------------------------------------------------------------ from the definition, in 64 bits

def _two_to(e):
    """2^e in 64 bits, by its bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _e4m3(x, e):
    """x / 2^e to the nearest multiple of an eighth of its leading power of two, at least of 2^-9; ties to even."""
    y = x * _two_to(-e)
    step = _two_to(torch.frexp(y)[1].clamp_min(-5) - 4)
    return torch.round(y / step) * step


def _row_exponent(x):
    a = x.abs().amax(-1, keepdim=True)
    near = torch.log2(a.clamp_min(1e-100) / 448).round().int() - 1
    return (near + sum((a > 448 * _two_to(near + i)).int() for i in range(2))).clamp(LEAST_E, MOST_E)


def _turned(x, cs, halves):
    """Rows [t, h, 128] in 64 bits, pairs of dims as complex numbers times cos + i sin."""
    turn = torch.view_as_complex(cs.double().contiguous())[:, None]
    n = turn.shape[-1]
    at = torch.arange(n, device="cuda")
    first, second = (at, at + n) if halves else (2 * at, 2 * at + 1)
    x = x.double()
    z = torch.complex(x[..., first], x[..., second]) * turn
    y = x.clone()
    y[..., first], y[..., second] = z.real, z.imag
    return y


def exact(case, seed):
    s = prepare(case, seed)
    new, start = _shape(case)
    heads, kv, op, page = case["heads"], case["kv_heads"], case["op"], case["page"]

    def spots(table, size, b, first, n):
        at = torch.arange(first, first + n, device="cuda")
        return table[b].long()[at // size] * size + at % size

    def rows(name, b, n):
        spot = spots(s["table"], page, b, 0, n)
        x = s[name + "_pages"].view(-1, kv, D)[spot] if op == "shared" else \
            s[name + "_pages"].view(torch.uint8).view(-1, kv, D)[spot].view(torch.float8_e4m3fn).float()
        if op == "shared":
            return x.double()
        return x.double() * _two_to(s[name + "_scales"].view(-1, kv)[spot].int() - 127)[..., None]

    if op == "append":
        out = torch.zeros(sum(new), heads, D, dtype=torch.float64, device="cuda")
        kp, vp = s["k_pages"].float().double(), s["v_pages"].float().double()
        first = 0
        for b, (t, a) in enumerate(zip(new, start)):
            if not t:
                continue
            r = slice(first, first + t)
            first += t
            cs, spot = s["rope"][a:a + t], spots(s["table"], page, b, a, t)
            out[r] = _turned(s["q"][r], cs, case["halves"])
            k, v = _turned(s["k"][r], cs, case["halves"]), s["v"][r].double()
            if case["bits"] == 8:
                k, v = _e4m3(k, _row_exponent(k)), _e4m3(v, _row_exponent(v))
            kp.view(-1, kv, D)[spot], vp.view(-1, kv, D)[spot] = k, v
        return (out, kp, vp, None, None) if case["bits"] == 8 else (out, kp, vp)
    if op == "read":
        ko, vo = s["k_out"].double(), s["v_out"].double()
        for b, n in enumerate(start):
            spot = spots(s["to_table"], case["to_page"], b, 0, n)
            ko.view(-1, kv, D)[spot], vo.view(-1, kv, D)[spot] = rows("k", b, n), rows("v", b, n)
        return ko, vo
    out = torch.zeros(len(new), heads, D, dtype=torch.float64, device="cuda")
    for b, a in enumerate(start):
        ks, vs = rows("k", b, a + 1), rows("v", b, a + 1)
        for h in range(heads):
            g = h * kv // heads
            out[b, h] = torch.softmax(ks[:, g] @ s["q"][b, h].double() / math.sqrt(D), -1) @ vs[:, g]
    return out
