"""What is measured of the operators around packed prompts and a cache in 4 bits:
the attention over packed prompts of different lengths whose query heads share
key heads, its gradients, and the step that appends new tokens to a paged cache
held in 4 bits and attends over it.

`run` computes a case through the framework's own calls where `own` is true
and in elementary torch operations otherwise; `exact` evaluates the
definition in 64 bits.
"""
import math
import random

import torch

own = False

BLOCK = 16  # entries of a cached row that share one scale


def listed():
    return [
        # a few short questions that arrive together: latency
        fwd_case("packed_fwd_short", n=12, most=90, Hq=32, Hk=8, d=128),
        # a serving prefill: prompts from a few tokens to 2000 in one launch
        fwd_case("packed_fwd_mixed", n=14, most=2000, Hq=32, Hk=8, d=128),
        # an encoder's batch: no causal mask, three heads to a key head, odd lengths
        fwd_case("packed_fwd_odd_64", n=9, most=1537, Hq=12, Hk=4, d=64, causal=False),
        # one long document
        fwd_case("packed_fwd_32k", n=1, most=32768, Hq=8, Hk=2, d=128),
        # a fine-tuning step on a handful of short samples
        bwd_case("packed_bwd_short", n=6, most=200, Hq=16, Hk=4, d=128),
        # a training step on samples packed to about 7000 tokens
        bwd_case("packed_bwd_mixed", n=10, most=2000, Hq=32, Hk=8, d=128),
        # seven heads to a key head, odd lengths
        bwd_case("packed_bwd_odd_64", n=5, most=1111, Hq=14, Hk=2, d=64),
        # a long-document training step
        bwd_case("packed_bwd_16k", n=1, most=16384, Hq=16, Hk=4, d=128),
        # one conversation's next token: latency
        step_case("step4_short", B=1, nq=1, Hq=32, Hk=8, d=128, page=16, held=700),
        # a running batch, from a few tokens to 16K
        step_case("step4_ragged", B=32, nq=1, Hq=32, Hk=8, d=128, page=16, held=16384),
        # three tokens of each sequence checked at once, odd page and lengths
        step_case("step4_odd_64", B=7, nq=3, Hq=15, Hk=5, d=64, page=48, held=5001),
        # long conversations, as a cache in 4 bits holds them: up to 128K tokens
        step_case("step4_long", B=16, nq=1, Hq=32, Hk=8, d=128, page=64, held=131072),
    ]


def fwd_case(name, *, n, most, Hq, Hk, d, causal=True):
    return {"name": name, "op": "fwd", "n": n, "most": most, "Hq": Hq, "Hk": Hk, "d": d,
            "causal": causal}


def bwd_case(name, *, n, most, Hq, Hk, d, causal=True):
    return {**fwd_case(name, n=n, most=most, Hq=Hq, Hk=Hk, d=d, causal=causal), "op": "bwd"}


def step_case(name, *, B, nq, Hq, Hk, d, page, held):
    return {"name": name, "op": "step", "B": B, "nq": nq, "Hq": Hq, "Hk": Hk, "d": d,
            "page": page, "held": held}


def spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["fwd", "bwd", "step"])
    d = rng.choice([64, 128])
    Hk = rng.choice([1, 2, 4, 5, 8])
    Hq = Hk * rng.choice([1, 2, 3, 4, 7, 8] if Hk <= 4 else [1, 2, 3, 4])
    if op == "step":
        nq = rng.choice([1, 1, 1, 2, 4])
        B = spread(rng, 1, 64)
        return {k: v for k, v in step_case(
            "", B=B, nq=nq, Hq=Hq, Hk=Hk, d=d, page=rng.choice([16, 32, 48, 64, 128]),
            held=spread(rng, 1, 1000000 // B)).items() if k != "name"}
    n = spread(rng, 1, 24)
    causal = rng.random() < 0.75
    # pairs of a query head and a key, with the longest length for all
    pairs = (8e9 if op == "fwd" else 4e9) / (1 if causal else 2)
    most = spread(rng, 1, min(32768, int(math.sqrt(pairs / (n * Hq)))))
    case = fwd_case("", n=n, most=most, Hq=Hq, Hk=Hk, d=d, causal=causal)
    return {k: v for k, v in {**case, "op": op}.items() if k != "name"}


# ------------------------------------------------------------------- inputs
def lengths(n, most):
    """n lengths from short to long, the longest included; six or more have an empty one."""
    return [0 if n >= 6 and i == 0 else 1 + round((most - 1) * ((i + 1) / n) ** 2)
            for i in range(n)]


def held_lengths(case):
    """Tokens that each sequence holds before the step; -1: an unused row of the batch, which
    batches of eight or more have."""
    B, most = case["B"], case["held"]
    used = B - (B >= 8)
    return [-1] * (B - used) + [round(most * ((i + 1) / used) ** 2) for i in range(used)]


def padding(case):
    """Rows behind the last sequence."""
    return sum(lengths(case["n"], case["most"])) % 37


def generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * seed + 29)
    return g


def normal(g, shape, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


def prepare(case, seed):
    g, rng = generator(seed), random.Random(seed)
    return prepare_step(case, g, rng) if case["op"] == "step" else prepare_packed(case, g, rng)


def prepare_packed(case, g, rng):
    Hq, Hk, d = case["Hq"], case["Hk"], case["d"]
    lens = lengths(case["n"], case["most"])
    rng.shuffle(lens)
    total, T = sum(lens), sum(lens) + padding(case)
    offsets = [sum(lens[:i]) for i in range(len(lens) + 1)]
    # views of one projection's output, as a layer has them
    qkv = normal(g, (T, Hq + 2 * Hk, d), 1.5)
    st = {"case": case, "total": total, "longest": max(lens),
          "q": qkv[:, :Hq], "k": qkv[:, Hq:Hq + Hk], "v": qkv[:, Hq + Hk:],
          "seq_offsets": torch.tensor(offsets, dtype=torch.int32, device="cuda"),
          "out": torch.zeros((T, Hq, d), dtype=torch.bfloat16, device="cuda"),
          "lse": torch.zeros((Hq, T), dtype=torch.float32, device="cuda")}
    if case["op"] == "bwd":
        plain_fwd(st)
        st["dout"] = normal(g, (T, Hq, d))
        for x in "qkv":
            st["d" + x] = torch.zeros_like(st[x], memory_format=torch.contiguous_format)
    return st


def by_heads(rows, page):
    """Rows [pages * page, Hk, n] as [pages, page, Hk, n], a head's tokens of a page side by side."""
    return rows.unflatten(0, (-1, page)).transpose(1, 2).contiguous().transpose(1, 2)


def prepare_step(case, g, rng):
    B, nq, Hq, Hk, d, page = (case[x] for x in ("B", "nq", "Hq", "Hk", "d", "page"))
    held = held_lengths(case)
    rng.shuffle(held)
    counts = [0 if h < 0 else (h + nq + page - 1) // page for h in held]
    order = list(range(sum(counts) + 1))
    rng.shuffle(order)
    table, at = torch.full((B, max(counts)), -1, dtype=torch.int32), 0
    for b, c in enumerate(counts):
        table[b, :c] = torch.tensor(order[at:at + c], dtype=torch.int32)
        at += c
    st = {"case": case, "page_table": table.cuda()}
    for x in "kv":
        st[x + "_descale"] = 0.5 + torch.rand(Hk, generator=g, device="cuda")
        rows = torch.randn(((sum(counts) + 1) * page, Hk, d), generator=g, device="cuda")
        st[x + "_cache"], st[x + "_scale"] = (
            by_heads(t, page) for t in quantised(rows, st[x + "_descale"]))
    st["cache_lens"] = torch.tensor([max(h, 0) for h in held], dtype=torch.int32, device="cuda")
    st["new_lens"] = torch.tensor([0 if h < 0 else nq for h in held], dtype=torch.int32,
                                  device="cuda")
    st["seq_lens"] = st["cache_lens"] + st["new_lens"]
    # the step's queries and keys, normed and turned already; views of one buffer
    qkv = normal(g, (B, nq, Hq + 2 * Hk, d), 1.5)
    st["q"], st["k"], st["v"] = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hk], qkv[:, :, Hq + Hk:]
    return st


# --------------------------------------------------------------- plain forms
def padded(x, st):
    """Packed rows [T, H, d] as [n, longest, H, d] in 32 bits; rows behind a sequence are zeros."""
    offsets, L = st["seq_offsets"].long(), st["longest"]
    at = offsets[:-1, None] + torch.arange(L, device="cuda")
    there = at < offsets[1:, None]
    return x[at.clamp(max=x.shape[0] - 1)].float().masked_fill(~there[..., None, None], 0.0)


def packed_rows(st):
    """The sequence and the place in it of each of the packed rows."""
    rows = torch.arange(st["total"], device="cuda")
    offsets = st["seq_offsets"].long()
    seq = torch.searchsorted(offsets, rows, right=True) - 1
    return seq, rows - offsets[seq]


def hidden(st):
    """[n, 1, 1, longest, longest]: pairs of a query and a key that it does not see."""
    offsets, at = st["seq_offsets"], torch.arange(st["longest"], device="cuda")
    lens = (offsets[1:] - offsets[:-1])[:, None, None]
    seen = (at < lens).expand(-1, st["longest"], -1)
    if st["case"]["causal"]:
        seen = seen & (at <= at[:, None])
    return ~seen[:, None, None]


def heads(x, Hk):
    """[n, L, Hq, d] as [n, L, Hk, Hq / Hk, d]."""
    return x.unflatten(2, (Hk, -1))


def plain_scores(st):
    q, k = heads(padded(st["q"], st), st["case"]["Hk"]), padded(st["k"], st)
    s = torch.einsum("nqhgd,nkhd->nhgqk", q, k).mul_(1 / math.sqrt(st["case"]["d"]))
    return s.masked_fill_(hidden(st), -math.inf)


def plain_fwd(st):
    s = plain_scores(st)
    top = s.amax(-1, keepdim=True)
    top = top.masked_fill(top == -math.inf, 0.0)
    e = s.sub_(top).exp_()
    sums = e.sum(-1, keepdim=True)
    lse = (top + sums.log())[..., 0].flatten(1, 2)
    out = torch.einsum("nhgqk,nkhd->nqhgd", e, padded(st["v"], st)).flatten(2, 3)
    out = out / sums.flatten(1, 2).permute(0, 2, 1, 3)
    seq, at = packed_rows(st)
    st["out"][:st["total"]] = out[seq, at].to(torch.bfloat16)
    st["lse"][:, :st["total"]] = lse[seq, :, at].T
    return st["out"], st["lse"]


def plain_bwd(st):
    case, scale = st["case"], 1 / math.sqrt(st["case"]["d"])
    Hk = case["Hk"]
    seq, at = packed_rows(st)
    q, k, v, g = (padded(st[x], st) for x in ("q", "k", "v", "dout"))
    delta = (g * padded(st["out"], st)).sum(-1).transpose(1, 2).unflatten(1, (Hk, -1))
    lse = padded(st["lse"].T[..., None], st)[..., 0].transpose(1, 2).unflatten(1, (Hk, -1))
    q, g = heads(q, Hk), heads(g, Hk)
    p = plain_scores(st).sub_(lse[..., None]).exp_()
    dv = torch.einsum("nhgqk,nqhgd->nkhd", p, g)
    ds = torch.einsum("nqhgd,nkhd->nhgqk", g, v).sub_(delta[..., None]).mul_(p)
    dq = torch.einsum("nhgqk,nkhd->nqhgd", ds, k).flatten(2, 3) * scale
    dk = torch.einsum("nhgqk,nqhgd->nkhd", ds, q) * scale
    for x, grad in (("dq", dq), ("dk", dk), ("dv", dv)):
        st[x][:st["total"]] = grad[seq, at].to(torch.bfloat16)
    return st["dq"], st["dk"], st["dv"]


def quantised(x, descale):
    """Rows x [n, Hk, d] in 32 bits as codes [n, Hk, d / 2] and scales [n, Hk, d / 16]: entry
    i of a block of 16 is (code - 8) * scale * descale[head]."""
    y = (x * (1 / descale)[:, None]).unflatten(-1, (-1, BLOCK))
    scale = (y.abs().amax(-1) * (1 / 7)).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = scale.float()[..., None]
    n = torch.where(s > 0, (y / s).round().clamp(-7, 7), 0.0).add(8).to(torch.uint8).flatten(-2)
    return n[..., ::2] | n[..., 1::2] << 4, scale


def plain_append(st):
    case, page = st["case"], st["case"]["page"]
    B, nq = case["B"], case["nq"]
    i = torch.arange(nq, device="cuda")
    at = (st["cache_lens"][:, None] + i).long()
    pages = st["page_table"].long().gather(1, (at // page).clamp(max=st["page_table"].shape[1] - 1))
    live = i < st["new_lens"][:, None]
    # tokens that are not there go to the last page, which no sequence has
    spare = st["k_cache"].shape[0] - 1
    for x in "kv":
        codes, scale = quantised(st[x].float().flatten(0, 1), st[x + "_descale"])
        where = torch.where(live, pages, spare).flatten(), (at % page).flatten()
        keep = live.flatten()[:, None, None]
        cache, scales = st[x + "_cache"], st[x + "_scale"].view(torch.uint8)
        cache[where] = torch.where(keep, codes, cache[where])
        scales[where] = torch.where(keep, scale.view(torch.uint8), scales[where])


def widened(st, x):
    """The table's tokens in 32 bits: [B, max_pages * page, Hk, d]."""
    pages = st["page_table"].clamp(min=0).long()
    codes = st[x + "_cache"][pages].flatten(1, 2)
    n = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float().sub_(8.0)
    scale = st[x + "_scale"].view(torch.uint8)[pages].view(torch.float8_e4m3fn).flatten(1, 2).float()
    scale = scale * st[x + "_descale"][:, None]
    return n.unflatten(-1, (-1, BLOCK)).mul_(scale[..., None]).flatten(-2)


def plain_step(st):
    plain_append(st)
    case = st["case"]
    B, nq, Hk, d = case["B"], case["nq"], case["Hk"], case["d"]
    k = widened(st, "k")
    at = torch.arange(k.shape[1], device="cuda")
    last = st["seq_lens"][:, None] - nq + torch.arange(nq, device="cuda")
    seen = (at <= last[..., None]) & (st["seq_lens"] > 0)[:, None, None]
    score = torch.einsum("bnhgd,bkhd->bnhgk", heads(st["q"].float(), Hk) / math.sqrt(d), k)
    score = score.masked_fill_(~seen[:, :, None, None], -math.inf)
    del k
    top = score.amax(-1, keepdim=True)
    top = top.masked_fill(top == -math.inf, 0.0)
    e = (score - top).exp()
    total = e.sum(-1, keepdim=True)
    v = widened(st, "v").masked_fill_(~seen.any(1)[..., None, None], 0.0)
    out = torch.einsum("bnhgk,bkhd->bnhgd", e, v) / total
    out = out.masked_fill(total == 0, 0.0).reshape(B, nq, -1, d).to(torch.bfloat16)
    lse = (top + total.log())[..., 0].reshape(B, nq, -1).transpose(1, 2).contiguous()
    return out, lse, st["k_scale"], st["v_scale"]


def run(st):
    case = st["case"]
    if own:
        import context_ring_attention_fwd_gb300 as pkg
        if case["op"] == "fwd":
            return pkg.packed_attn_fwd(st["q"], st["k"], st["v"], st["seq_offsets"],
                                       case["causal"], out=st["out"], lse=st["lse"])
        if case["op"] == "bwd":
            return pkg.packed_attn_bwd(st["q"], st["k"], st["v"], st["out"], st["lse"],
                                       st["dout"], st["seq_offsets"], case["causal"],
                                       dq=st["dq"], dk=st["dk"], dv=st["dv"])
        cache = {x: st[x] for x in ("k_descale", "v_descale", "k_scale", "v_scale")}
        pkg.paged_append(None, st["k"], st["v"], st["k_cache"], st["v_cache"], st["page_table"],
                         st["cache_lens"], st["new_lens"], **cache)
        out, lse = pkg.paged_attn_decode(st["q"], st["k_cache"], st["v_cache"], st["page_table"],
                                         st["seq_lens"], **cache)
        return out, lse, st["k_scale"], st["v_scale"]
    return {"fwd": plain_fwd, "bwd": plain_bwd, "step": plain_step}[case["op"]](st)


# ---------------------------------------------------------------------- work
def work(case):
    Hq, Hk, d = case["Hq"], case["Hk"], case["d"]
    if case["op"] == "step":
        nq, held = case["nq"], [h for h in held_lengths(case) if h >= 0]
        row = d // 2 + d // BLOCK
        pairs = sum(nq * h + nq * (nq + 1) / 2 for h in held) * Hq
        return {"bytes": int(2 * Hk * row * sum(h + nq for h in held) + len(held) * nq *
                             (Hq * (4 * d + 4) + 4 * Hk * d)), "flops": int(4 * d * pairs)}
    lens = lengths(case["n"], case["most"])
    T, pairs = sum(lens), Hq * sum(x * (x + 1) / 2 if case["causal"] else x * x for x in lens)
    if case["op"] == "fwd":
        return {"bytes": T * (4 * d * (Hq + Hk) + 4 * Hq), "flops": int(4 * d * pairs)}
    return {"bytes": T * (8 * d * (Hq + Hk) + 4 * Hq), "flops": int(10 * d * pairs)}


# -------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "step":
        return exact_step(case, st)
    return exact_fwd(case, st) if case["op"] == "fwd" else exact_bwd(case, st)


def exact_spans(st):
    offsets = st["seq_offsets"].tolist()
    return [(a, z) for a, z in zip(offsets, offsets[1:]) if z > a]


def exact_weights(case, st, a, z, h):
    """The scores' log-sum-exp and the weights of head h in the sequence of rows [a, z)."""
    kv = h // (case["Hq"] // case["Hk"])
    s = st["q"][a:z, h].double() @ st["k"][a:z, kv].double().T / case["d"] ** 0.5
    if case["causal"]:
        s.masked_fill_(torch.ones_like(s, dtype=torch.bool).triu_(1), -math.inf)
    lse = s.logsumexp(-1)
    return lse, (s - lse[:, None]).exp_(), kv


def exact_fwd(case, st):
    out, lse = st["out"].double(), st["lse"].double()
    for a, z in exact_spans(st):
        for h in range(case["Hq"]):
            lse[h, a:z], p, kv = exact_weights(case, st, a, z, h)
            out[a:z, h] = p @ st["v"][a:z, kv].double()
    return out, lse


def exact_bwd(case, st):
    dq, dk, dv = (st[x].double() for x in ("dq", "dk", "dv"))
    for a, z in exact_spans(st):
        for h in range(case["Hq"]):
            _, p, kv = exact_weights(case, st, a, z, h)
            q, k, v = (st[x][a:z, i].double() for x, i in (("q", h), ("k", kv), ("v", kv)))
            g = st["dout"][a:z, h].double()
            dv[a:z, kv] += p.T @ g
            dp = g @ v.T
            ds = p * (dp - (p * dp).sum(-1, keepdim=True)) / case["d"] ** 0.5
            dq[a:z, h] = ds @ k
            dk[a:z, kv] += ds.T @ q
    return dq, dk, dv


def exact_rows(rows, descale):
    """New rows [n, Hk, d] as the cache holds them, without the heads' descales, and their
    blocks' scales."""
    y = (rows.double() / descale.double()[:, None]).unflatten(-1, (-1, BLOCK))
    scale = (y.abs().amax(-1) / 7).clamp(max=448).float().to(torch.float8_e4m3fn)
    s = scale.double()[..., None]
    n = torch.where(s > 0, (y / s).round().clamp(-7, 7), torch.zeros_like(y))
    return (n * s).flatten(-2), scale


def exact_step(case, st):
    B, nq, Hq, Hk, d, page = (case[x] for x in ("B", "nq", "Hq", "Hk", "d", "page"))
    G, held = Hq // Hk, st["cache_lens"].tolist()
    out = torch.zeros((B, nq, Hq, d), dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq, nq), -math.inf, dtype=torch.float64, device="cuda")
    scales = {x: st[x + "_scale"].clone().view(torch.uint8) for x in "kv"}
    for b in range(B):
        if not st["new_lens"][b]:
            continue
        at = torch.arange(held[b] + nq, device="cuda")
        where = st["page_table"][b].long()[at // page], at % page
        kv = {}
        for x in "kv":
            new, new_scale = exact_rows(st[x][b], st[x + "_descale"])
            byte = st[x + "_cache"][where]
            n = torch.empty((*byte.shape[:-1], d), dtype=torch.float64, device="cuda")
            n[..., ::2], n[..., 1::2] = byte % 16, byte // 16
            s = scales[x][where].view(torch.float8_e4m3fn).double()
            old = (n - 8).unflatten(-1, (-1, BLOCK)) * s[..., None]
            kv[x] = torch.cat([old.flatten(-2)[:held[b]], new]) * st[x + "_descale"].double()[:, None]
            scales[x][where[0][held[b]:], where[1][held[b]:]] = new_scale.view(torch.uint8)
        for h in range(Hq):
            s = st["q"][b, :, h].double() @ kv["k"][:, h // G].T / d ** 0.5
            s.masked_fill_(at > held[b] + torch.arange(nq, device="cuda")[:, None], -math.inf)
            lse[b, h] = s.logsumexp(-1)
            out[b, :, h] = (s - lse[b, h][:, None]).exp() @ kv["v"][:, h // G]
    return out, lse, *(scales[x].view(torch.float8_e4m3fn) for x in "kv")
