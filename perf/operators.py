"""What is measured of the operators around the attention: the per-head norm
and rotation of queries and keys (forward and backward), the append to a paged
key/value cache, and the decode attention over that cache with a prefix that
the whole batch shares.

`run` computes a case through the framework's own calls where `own` is true
and in elementary torch operations otherwise; `exact` evaluates the
definition in 64 bits.
"""
import math
import random

import torch

own = False

EPS = 1e-6
THETA = 500000.0


def listed():
    return [
        # one decoding step of a small batch: what a layer adds to its latency
        rope_case("rope_step", B=16, S=1, Hq=32, Hk=8, d=128, fused=True),
        # the causal 8K layer's queries and keys, equal heads
        rope_case("rope_8k", B=1, S=8192, Hq=32, Hk=32, d=128),
        # packed documents: positions restart, q and k are views of one projection
        rope_case("rope_packed_64k", B=1, S=65536, Hq=16, Hk=16, d=128, fused=True, docs=8),
        # the training step's gradients at 8K
        rope_case("rope_bwd_8k", B=1, S=8192, Hq=32, Hk=32, d=128, bwd=True),
        # odd length, shared key heads, fp32, half of each head rotated in pairs
        rope_case("rope_bwd_f32_odd", B=2, S=1537, Hq=12, Hk=4, d=64, f32=True, rot=32,
                  pairs=True, fused=True, bwd=True),
        # the two 32K sequences of the long training shape
        rope_case("rope_bwd_32k", B=2, S=32768, Hq=16, Hk=16, d=128, fused=True, bwd=True),
        # one token for each of 64 running sequences
        append_case("append_step", B=64, S=1, Hq=32, Hk=8, d=128, page=16, held=900),
        # a prefill chunk of ragged prompts into an 8-bit cache
        append_case("append_chunk_e4m3", B=4, S=2048, Hq=32, Hk=8, d=128, page=64, held=5000,
                    e4m3=True, ragged=True),
        # one short conversation: latency
        decode_case("decode_short", B=1, nq=1, Hq=32, Hk=8, d=128, page=16, prefix=0, rest=700),
        # a running batch without a common prefix, lengths from a few tokens to 16K
        decode_case("decode_ragged", B=32, nq=1, Hq=32, Hk=8, d=128, page=16, prefix=0,
                    rest=16384),
        # a batch of answers under one 32K document
        decode_case("decode_prefix_32k", B=64, nq=1, Hq=32, Hk=8, d=128, page=64, prefix=32768,
                    rest=512),
        # four tokens of each sequence checked at once under a 128K prefix, 8-bit cache
        decode_case("decode_prefix_128k_e4m3", B=32, nq=4, Hq=32, Hk=8, d=128, page=64,
                    prefix=131072, rest=1024, e4m3=True),
    ]


def rope_case(name, *, B, S, Hq, Hk, d, fused=False, docs=0, f32=False, rot=None, pairs=False,
              bwd=False):
    return {"name": name, "op": "rope_bwd" if bwd else "rope", "B": B, "S": S, "Hq": Hq, "Hk": Hk,
            "d": d, "fused": fused, "docs": docs, "f32": f32, "rot": d if rot is None else rot,
            "pairs": pairs}


def append_case(name, *, B, S, Hq, Hk, d, page, held, e4m3=False, ragged=False, pairs=False):
    return {"name": name, "op": "append", "B": B, "S": S, "Hq": Hq, "Hk": Hk, "d": d,
            "page": page, "held": held, "e4m3": e4m3, "ragged": ragged, "rot": d, "pairs": pairs}


def decode_case(name, *, B, nq, Hq, Hk, d, page, prefix, rest, e4m3=False):
    return {"name": name, "op": "decode", "B": B, "nq": nq, "Hq": Hq, "Hk": Hk, "d": d,
            "page": page, "prefix": prefix, "rest": rest, "e4m3": e4m3}


def spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["rope", "rope_bwd", "append", "decode", "decode"])
    d = rng.choice([64, 128])
    Hk = rng.choice([1, 2, 4, 5, 8, 16])
    group = rng.choice([1, 2, 3, 4, 8]) if Hk < 16 else 1
    Hq = Hk * group
    if op in ("rope", "rope_bwd"):
        B, f32 = rng.randint(1, 4), rng.random() < 0.25
        S = spread(rng, 1, 65536 * 32 // (B * max(32, Hq + Hk) * (2 if f32 else 1)))
        return {k: v for k, v in rope_case(
            "", B=B, S=S, Hq=Hq, Hk=Hk, d=d, fused=rng.random() < 0.5,
            docs=rng.choice([0, 0, 3, 17]), f32=f32,
            rot=rng.choice([d, d, d // 2]), pairs=rng.random() < 0.3,
            bwd=op == "rope_bwd").items() if k != "name"}
    if op == "append":
        S = rng.choice([1, 1, 3, spread(rng, 2, 4096)])
        B = spread(rng, 1, max(1, min(128, 16384 // S)))
        return {k: v for k, v in append_case(
            "", B=B, S=S, Hq=Hq, Hk=Hk, d=d, page=rng.choice([16, 32, 48, 64, 128]),
            held=spread(rng, 1, 4000), e4m3=rng.random() < 0.5, ragged=rng.random() < 0.5,
            pairs=rng.random() < 0.3).items() if k != "name"}
    nq = rng.choice([1, 1, 1, 2, 4])
    B = spread(rng, 1, 128 // nq)
    prefix = rng.choice([0, 0, spread(rng, 1, 65536)])
    rest = spread(rng, 1, max(2, min(16384, 400000 // B)))
    return {k: v for k, v in decode_case(
        "", B=B, nq=nq, Hq=Hq, Hk=Hk, d=d, page=rng.choice([16, 32, 48, 64, 128]),
        prefix=prefix, rest=rest, e4m3=rng.random() < 0.5).items() if k != "name"}


# ------------------------------------------------------------------- inputs
def lengths(n, most, least=1):
    """n lengths between `least` and `most`, from short to long, the longest included."""
    return [least + round((most - least) * ((i + 1) / n) ** 2) for i in range(n)]


def own_lengths(case):
    """Keys of each sequence behind the prefix, the queries' own among them.  A batch of eight or
    more has one empty slot (-1)."""
    B, most = case["B"], max(case["rest"], case["nq"])
    return ([-1] if B >= 8 else []) + lengths(B - (B >= 8), most, case["nq"])


def new_lengths(case):
    return lengths(case["B"], case["S"]) if case["ragged"] else [case["S"]] * case["B"]


def generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * seed + 17)
    return g


def normal(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def frequencies(rot):
    return (THETA ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float().cuda()


def gain(g, d, scale=1.0):
    return (1.0 + 0.2 * torch.randn(d, generator=g, device="cuda")) * scale


def pages_of(rng, counts, page_count, longest):
    """A table [len(counts), longest] that deals `page_count` shuffled pages; unused entries -1."""
    order = list(range(page_count))
    rng.shuffle(order)
    rows, at = [], 0
    for n in counts:
        rows.append(order[at:at + n] + [-1] * (longest - n))
        at += n
    return rows, order[at:]


def filled_cache(g, pages, page, Hk, d, e4m3):
    """Keys and values as earlier steps left them: normed keys, values of unit size; E4M3 codes
    with one fixed scale per head."""
    shape = (pages, page, Hk, d)
    k, v = normal(g, shape, torch.bfloat16), normal(g, shape, torch.bfloat16)
    if not e4m3:
        return k, v, None, None
    kd = (0.01 + 0.01 * torch.rand(Hk, generator=g, device="cuda"))
    vd = (0.01 + 0.01 * torch.rand(Hk, generator=g, device="cuda"))
    code = lambda x, s: ((x.float() / s[:, None]).clamp(-448, 448)  # noqa: E731
                         .to(torch.float8_e4m3fn).view(torch.uint8))
    return code(k, kd), code(v, vd), kd, vd


def prepare(case, seed):
    g, rng = generator(seed), random.Random(seed)
    B, Hq, Hk, d = case["B"], case["Hq"], case["Hk"], case["d"]
    st = {"case": case}
    if case["op"] in ("rope", "rope_bwd"):
        S, t = case["S"], torch.float32 if case["f32"] else torch.bfloat16
        if case["fused"]:
            qkv = normal(g, (B, S, Hq + 2 * Hk, d), t, 2.0)
            st["q"], st["k"] = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hk]
        else:
            st["q"], st["k"] = normal(g, (B, S, Hq, d), t, 2.0), normal(g, (B, S, Hk, d), t, 2.0)
        st["positions"] = None
        if case["docs"]:
            cuts = sorted(rng.sample(range(1, S), min(case["docs"] - 1, S - 1))) if S > 1 else []
            starts = torch.zeros(S, dtype=torch.int64)
            for c in cuts:
                starts[c:] = c
            st["positions"] = ((torch.arange(S) - starts).to(torch.int32).cuda()
                               .expand(B, S).contiguous())
        st["q_weight"], st["k_weight"] = gain(g, d), gain(g, d)
        st["inv_freq"] = frequencies(case["rot"])
        if case["op"] == "rope_bwd":
            st["dq_out"], st["dk_out"] = normal(g, (B, S, Hq, d), t), normal(g, (B, S, Hk, d), t)
        return st
    page = case["page"]
    if case["op"] == "append":
        S, new = case["S"], new_lengths(case)
        held = [rng.randint(0, case["held"]) for _ in range(B)]
        longest = (case["held"] + S + page - 1) // page
        counts = [longest] * B
        rows, _ = pages_of(rng, counts, sum(counts) + 1, longest)
        (st["k_cache"], st["v_cache"], st["k_descale"],
         st["v_descale"]) = filled_cache(g, sum(counts) + 1, page, Hk, d, case["e4m3"])
        rng.shuffle(new)
        qkv = normal(g, (B, S, Hq + 2 * Hk, d), torch.bfloat16, 2.0)
        st["q"], st["k"], st["v"] = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hk], qkv[:, :, Hq + Hk:]
        st["q_out"] = torch.zeros((B, S, Hq, d), dtype=torch.bfloat16, device="cuda")
        st["q_weight"], st["k_weight"] = gain(g, d), gain(g, d)
        st["inv_freq"] = frequencies(case["rot"])
        st["page_table"] = torch.tensor(rows, dtype=torch.int32, device="cuda")
        st["cache_lens"] = torch.tensor(held, dtype=torch.int32, device="cuda")
        st["new_lens"] = torch.tensor(new, dtype=torch.int32, device="cuda")
        return st
    P, nq = case["prefix"], case["nq"]
    rest = own_lengths(case)
    rng.shuffle(rest)
    shared = (P + page - 1) // page
    whole = P // page
    counts = [0 if r < 0 else (P + r + page - 1) // page - whole for r in rest]
    longest = whole + max(counts)
    rows, left = pages_of(rng, counts, shared + sum(counts) + 1, max(counts))
    st["prefix_pages"] = torch.tensor(left[:shared], dtype=torch.int32, device="cuda") if P else None
    table = torch.full((B, longest), -1, dtype=torch.int32)
    table[:, whole:] = torch.tensor(rows, dtype=torch.int32)
    table[:, :whole] = torch.tensor(left[:whole], dtype=torch.int32)
    st["page_table"] = table.cuda()
    st["seq_lens"] = torch.tensor([0 if r < 0 else P + r for r in rest], dtype=torch.int32,
                                  device="cuda")
    (st["k_cache"], st["v_cache"], st["k_descale"],
     st["v_descale"]) = filled_cache(g, shared + sum(counts) + 1, page, Hk, d, case["e4m3"])
    st["q"] = normal(g, (B, nq, Hq, d), torch.bfloat16, 2.0)
    return st


# --------------------------------------------------------------- plain forms
def cos_sin(positions, inv_freq):
    """[..., rot / 2] in fp32, the angles themselves in 64 bits."""
    angle = positions.double()[..., None] * inv_freq.double()
    return angle.cos().float(), angle.sin().float()


def turn(x, cos, sin, rot, pairs):
    """x [B, S, H, d] fp32 with its first `rot` entries rotated by the angles [B, S, rot / 2]."""
    cos, sin = cos[:, :, None], sin[:, :, None]
    lo, hi = (x[..., 0:rot:2], x[..., 1:rot:2]) if pairs else (x[..., :rot // 2],
                                                               x[..., rot // 2:rot])
    a, b = lo * cos - hi * sin, hi * cos + lo * sin
    head = torch.stack([a, b], -1).flatten(-2) if pairs else torch.cat([a, b], -1)
    return torch.cat([head, x[..., rot:]], -1)


def normed(x, weight):
    x = x.float()
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight


def plain_positions(st):
    case = st["case"]
    if st["positions"] is not None:
        return st["positions"]
    return torch.arange(case["S"], device="cuda").expand(case["B"], case["S"])


def plain_rope(st):
    case = st["case"]
    cos, sin = cos_sin(plain_positions(st), st["inv_freq"])
    q = turn(normed(st["q"], st["q_weight"]), cos, sin, case["rot"], case["pairs"])
    k = turn(normed(st["k"], st["k_weight"]), cos, sin, case["rot"], case["pairs"])
    return q.to(st["q"].dtype), k.to(st["k"].dtype)


def plain_rope_grad(dy, x, weight, cos, sin, case):
    x, dy = x.float(), dy.float()
    g = turn(dy, cos, -sin, case["rot"], case["pairs"])
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    unit, gw = x * r, g * weight
    dx = r * (gw - unit * (gw * unit).mean(-1, keepdim=True))
    return dx, (g * unit).sum((0, 1, 2), dtype=torch.float64).float()


def plain_rope_bwd(st):
    case, t = st["case"], st["q"].dtype
    cos, sin = cos_sin(plain_positions(st), st["inv_freq"])
    dq, dqw = plain_rope_grad(st["dq_out"], st["q"], st["q_weight"], cos, sin, case)
    dk, dkw = plain_rope_grad(st["dk_out"], st["k"], st["k_weight"], cos, sin, case)
    return dq.to(t), dk.to(t), dqw, dkw


def stored(x, cache, descale):
    """x [n, Hk, d] fp32 as the cache holds it."""
    if descale is None:
        return x.to(cache.dtype)
    return ((x / descale[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))


def as_values(cache):
    """A cache's entries as the values that they stand for (before the heads' scales)."""
    return cache.view(torch.float8_e4m3fn) if cache.dtype == torch.uint8 else cache


def plain_append(st):
    case, page = st["case"], st["case"]["page"]
    at = st["cache_lens"][:, None].long() + torch.arange(case["S"], device="cuda")
    live = torch.arange(case["S"], device="cuda") < st["new_lens"][:, None]
    cos, sin = cos_sin(at, st["inv_freq"])
    q = turn(normed(st["q"], st["q_weight"]), cos, sin, case["rot"], case["pairs"])
    k = turn(normed(st["k"], st["k_weight"]), cos, sin, case["rot"], case["pairs"])
    slot = st["page_table"].long().gather(1, at // page) * page + at % page
    flat = slot[live]
    Hk, d = case["Hk"], case["d"]
    st["k_cache"].view(-1, Hk, d)[flat] = stored(k[live], st["k_cache"], st["k_descale"])
    st["v_cache"].view(-1, Hk, d)[flat] = stored(st["v"][live].float(), st["v_cache"],
                                                 st["v_descale"])
    st["q_out"][live] = q[live].to(st["q_out"].dtype)
    return st["q_out"], as_values(st["k_cache"]), as_values(st["v_cache"])


def widened(cache, pages, descale):
    """The pages' tokens in fp32: [..., pages * page, Hk, d]."""
    x = as_values(cache[pages.clamp(min=0).long()]).float().flatten(-4, -3)
    return x if descale is None else x * descale[:, None]


def plain_decode(st):
    case, page = st["case"], st["case"]["page"]
    B, nq, Hk, d, P = case["B"], case["nq"], case["Hk"], case["d"], case["prefix"]
    G = case["Hq"] // Hk
    q = st["q"].float().view(B, nq, Hk, G, d) / math.sqrt(d)
    first = P // page
    table = st["page_table"][:, first:]
    ko, vo = (widened(st[c], table, st[s]) for c, s in (("k_cache", "k_descale"),
                                                        ("v_cache", "v_descale")))
    at = first * page + torch.arange(ko.shape[1], device="cuda")
    last = st["seq_lens"][:, None] - nq + torch.arange(nq, device="cuda")
    seen = (at >= P) & (at <= last[..., None])
    score = torch.einsum("bnhgd,bkhd->bnhgk", q, ko)
    score = score.masked_fill(~seen[:, :, None, None], -math.inf)
    vo = vo.masked_fill(~seen.any(1)[..., None, None], 0.0)
    if P:
        kp, vp = (widened(st[c], st["prefix_pages"], st[s])[:P]
                  for c, s in (("k_cache", "k_descale"), ("v_cache", "v_descale")))
        score = torch.cat([torch.einsum("bnhgd,khd->bnhgk", q, kp), score], -1)
    live = (st["seq_lens"] > 0)[:, None, None, None]
    top = score.amax(-1, keepdim=True)
    top = top.masked_fill(top == -math.inf, 0.0)
    e = (score - top).exp()
    total = e.sum(-1, keepdim=True)
    out = torch.einsum("bnhgk,bkhd->bnhgd", e[..., P:], vo)
    if P:
        out = out + torch.einsum("bnhgk,khd->bnhgd", e[..., :P], vp)
    out = (out / total).masked_fill(~live[..., None] | (total == 0), 0.0)
    lse = (top + total.log())[..., 0].masked_fill(~live, -math.inf)
    return (out.reshape(B, nq, -1, d).to(st["q"].dtype),
            lse.reshape(B, nq, -1).transpose(1, 2).contiguous())


def run(st):
    case = st["case"]
    if own:
        import context_ring_attention_fwd_gb300 as pkg
        rope = {"interleaved": case.get("pairs", False), "eps": EPS}
        if case["op"] == "rope":
            return pkg.qk_norm_rope(st["q"], st["k"], st["q_weight"], st["k_weight"],
                                    st["inv_freq"], st["positions"], **rope)
        if case["op"] == "rope_bwd":
            return pkg.qk_norm_rope_bwd(st["dq_out"], st["dk_out"], st["q"], st["k"],
                                        st["q_weight"], st["k_weight"], st["inv_freq"],
                                        st["positions"], **rope)
        scales = {"k_descale": st["k_descale"], "v_descale": st["v_descale"]}
        if case["op"] == "append":
            q_out = pkg.paged_append(st["q"], st["k"], st["v"], st["k_cache"], st["v_cache"],
                                     st["page_table"], st["cache_lens"], st["new_lens"],
                                     st["q_weight"], st["k_weight"], st["inv_freq"],
                                     q_out=st["q_out"], **scales, **rope)
            return q_out, as_values(st["k_cache"]), as_values(st["v_cache"])
        return pkg.paged_attn_decode(st["q"], st["k_cache"], st["v_cache"], st["page_table"],
                                     st["seq_lens"], st["prefix_pages"], case["prefix"], **scales)
    plain = {"rope": plain_rope, "rope_bwd": plain_rope_bwd, "append": plain_append,
             "decode": plain_decode}
    return plain[case["op"]](st)


# ---------------------------------------------------------------------- work
def work(case):
    B, Hq, Hk, d = case["B"], case["Hq"], case["Hk"], case["d"]
    if case["op"] in ("rope", "rope_bwd"):
        n, e = B * case["S"] * (Hq + Hk) * d, 4 if case["f32"] else 2
        if case["op"] == "rope":
            return {"bytes": 2 * n * e + (4 * B * case["S"] if case["docs"] else 0) + 8 * d,
                    "flops": 8 * n}
        return {"bytes": 3 * n * e + (4 * B * case["S"] if case["docs"] else 0) + 16 * d,
                "flops": 16 * n}
    e = 1 if case["e4m3"] else 2
    if case["op"] == "append":
        t = sum(new_lengths(case))
        return {"bytes": t * d * (4 * Hq + 4 * Hk + 2 * Hk * e) + 8 * B,
                "flops": 8 * t * (Hq + Hk) * d}
    live = [r for r in own_lengths(case) if r >= 0]
    keys, rows = sum(live) + case["prefix"], len(live) * case["nq"] * Hq
    pairs = case["nq"] * Hq * (sum(live) - len(live) * (case["nq"] - 1) / 2)
    return {"bytes": int(2 * keys * Hk * d * e + rows * (4 * d + 4)),
            "flops": int(4 * d * (pairs + rows * case["prefix"]))}


# -------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] in ("rope", "rope_bwd"):
        return exact_rope(case, st)
    return exact_append(case, st) if case["op"] == "append" else exact_decode(case, st)


def exact_turned(x, weight, at, inv_freq, case):
    """Norm, then each pair as a complex number times exp(i angle)."""
    rot = case["rot"]
    y = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * weight.double()
    angle = at.double()[..., None, None] * inv_freq.double()
    unit = torch.polar(torch.ones_like(angle), angle)
    if case["pairs"]:
        z = torch.view_as_complex(y[..., :rot].reshape(*y.shape[:-1], rot // 2, 2).contiguous())
        head = torch.view_as_real(z * unit).flatten(-2)
    else:
        z = torch.complex(y[..., :rot // 2].contiguous(), y[..., rot // 2:rot].contiguous()) * unit
        head = torch.cat([z.real, z.imag], -1)
    return torch.cat([head, y[..., rot:]], -1)


def exact_rope(case, st):
    at = (st["positions"] if st["positions"] is not None else
          torch.arange(case["S"], device="cuda").repeat(case["B"], 1))
    if case["op"] == "rope":
        return tuple(exact_turned(st[x].double(), st[x + "_weight"], at, st["inv_freq"], case)
                     for x in "qk")
    grads = []
    for x in "qk":
        leaf = st[x].double().requires_grad_()
        weight = st[x + "_weight"].double().requires_grad_()
        y = exact_turned(leaf, weight, at, st["inv_freq"], case)
        grads.append(torch.autograd.grad(y, (leaf, weight), st["d" + x + "_out"].double()))
    return grads[0][0], grads[1][0], grads[0][1], grads[1][1]


def exact_append(case, st):
    new, held, page = st["new_lens"].tolist(), st["cache_lens"].tolist(), case["page"]
    q_out = st["q_out"].double()
    kc, vc = as_values(st["k_cache"]).double(), as_values(st["v_cache"]).double()
    for b in range(case["B"]):
        n = new[b]
        at = torch.arange(held[b], held[b] + n, device="cuda")
        q_out[b, :n], k = (exact_turned(st[x][b:b + 1, :n].double(), st[x + "_weight"], at[None],
                                        st["inv_freq"], case)[0] for x in "qk")
        v = st["v"][b, :n].double()
        if case["e4m3"]:
            k, v = k / st["k_descale"].double()[:, None], v / st["v_descale"].double()[:, None]
        where = st["page_table"][b].long()[at // page], at % page
        kc[where], vc[where] = k, v
    return q_out, kc, vc


def exact_decode(case, st):
    B, nq, Hq, Hk, d, P = (case[x] for x in ("B", "nq", "Hq", "Hk", "d", "prefix"))
    if 4.0 * d * B * nq * Hq * P > 4e12:
        return None
    G, page, lens = Hq // Hk, case["page"], st["seq_lens"].tolist()
    kc, vc = as_values(st["k_cache"]), as_values(st["v_cache"])
    ones = torch.ones(Hk, device="cuda")
    kd, vd = (ones if st[s] is None else st[s] for s in ("k_descale", "v_descale"))
    out = torch.zeros((B, nq, Hq, d), dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq, nq), -math.inf, dtype=torch.float64, device="cuda")
    places = [torch.arange(n, device="cuda") for n in lens]
    for h in range(Hk):
        if P:
            at = torch.arange(P, device="cuda")
            where = st["prefix_pages"].long()[at // page], at % page, h
            kp, vp = kc[where].double() * kd[h].double(), vc[where].double() * vd[h].double()
        for b in range(B):
            if not lens[b]:
                continue
            at = places[b][P:]
            where = st["page_table"][b].long()[at // page], at % page, h
            k, v = kc[where].double() * kd[h].double(), vc[where].double() * vd[h].double()
            if P:
                k, v = torch.cat([kp, k]), torch.cat([vp, v])
            for i in range(nq):
                n = max(lens[b] - nq + i + 1, P)
                if not n:
                    continue
                s = st["q"][b, i, h * G:(h + 1) * G].double() @ k[:n].T / d ** 0.5
                z = s.logsumexp(-1)
                lse[b, h * G:(h + 1) * G, i] = z
                out[b, i, h * G:(h + 1) * G] = (s - z[:, None]).exp() @ v[:n]
    return out, lse
