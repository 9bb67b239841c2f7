"""The paged cache in 4 bits: the append against the oracle's codes, and decode attention over it.

Tolerances.  Rows that are neither normed nor turned are quantised by operations that the format
defines to the bit, so codes and scales are equal.  A normed and turned row y is known to 2^-18 of
its largest entry (test_gpu_norm_rope.py), so a scale is within E4M3's half step, 2^-4 of it, of
max |y| / 7, and an entry within half a step of the scale held of y, each plus that error (a
block's largest entry is 7 (1 + 2^-4) steps at most, less than half a step above 7).
Decode: code times scale is exact in fp16 as an E4M3 code is, so test_gpu_paged_decode.py's
tolerances for 8 bits hold.
"""
import os

import numpy as np
import pytest
import torch

import context_ring_attention_fwd_gb300 as pkg
from oracle import serving
from test_gpu_paged_decode import CASES, Batch

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    if not os.path.exists(pkg.LIB_PATH):
        from context_ring_attention_fwd_gb300 import _build
        _build.build()
    pkg.lib()
    torch.cuda.set_device(0)
    yield
    assert pkg.cp_get_last_status() == 0


def _np(t):
    return t.detach().double().cpu().numpy()


def raw(t):
    return t.contiguous().view(torch.uint8).cpu().numpy()


def empty_cache(n_pages, page, Hk, d, head_major, seed):
    """Codes and scales of K and V, filled with junk."""
    g = torch.Generator().manual_seed(seed)
    made = []
    for n in (d // 2, d // 16):
        for _ in range(2):
            shape = (n_pages, Hk, page, n) if head_major else (n_pages, page, Hk, n)
            t = torch.randint(0, 256, shape, dtype=torch.uint8, generator=g).to(DEV)
            made.append(t.transpose(1, 2) if head_major else t)
    return made


def new_rows(B, S, Hq, Hk, d, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((B, S, Hq + 2 * Hk, d), generator=g)
    x = (x * torch.exp(spread * torch.randn((B, S, Hq + 2 * Hk, 1), generator=g))).bfloat16().to(DEV)
    return x[:, :, :Hq], x[:, :, Hq:Hq + Hk], x[:, :, Hq + Hk:]


def table_of(B, most, n_pages, seed):
    rng = np.random.default_rng(seed)
    return torch.tensor(rng.permutation(n_pages)[:B * most].reshape(B, most), dtype=torch.int32,
                        device=DEV)


@pytest.mark.parametrize("B,S,Hq,Hk,d,page,ragged,head_major,descaled", [
    (1, 1, 0, 1, 64, 1, False, False, False),
    (1, 1, 4, 1, 128, 16, False, False, True),
    (3, 5, 6, 3, 64, 7, True, True, True),
    (64, 1, 0, 8, 128, 16, False, True, False),
    (4, 130, 2, 5, 128, 48, True, False, True),
    (300, 3, 1, 1, 64, 16, True, False, False),
    (2, 700, 8, 8, 128, 64, True, True, False),
])
def test_rows_are_quantised_to_the_bit(B, S, Hq, Hk, d, page, ragged, head_major, descaled):
    held = 3 * page // 2
    most = (held + S) // page + 1
    n_pages = B * most + 2
    kc, vc, ks, vs = empty_cache(n_pages, page, Hk, d, head_major, 1)
    before = [raw(t) for t in (kc, vc, ks, vs)]
    table = table_of(B, most, n_pages, 2)
    rng = np.random.default_rng(3)
    lens = rng.integers(0, held + 1, B)
    new = rng.integers(0, S + 1, B) if ragged else np.full(B, S)
    q, k, v = new_rows(B, S, Hq, Hk, d, 4)
    dsc = [torch.tensor(rng.uniform(0.1, 3, Hk), dtype=torch.float32, device=DEV) if descaled
           else None for _ in range(2)]
    to_dev = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    scale_type = torch.float8_e4m3fn if head_major else torch.uint8
    q_out = pkg.paged_append(q if Hq else None, k, v, kc, vc, table, to_dev(lens),
                             to_dev(new) if ragged else None, k_descale=dsc[0], v_descale=dsc[1],
                             k_scale=ks.view(scale_type), v_scale=vs.view(scale_type))
    t = table.cpu().numpy()
    for x, cache, scales, c0, s0, dd in ((k, kc, ks, before[0], before[2], dsc[0]),
                                         (v, vc, vs, before[1], before[3], dsc[1])):
        codes, sc = serving.quantise4(x.float().cpu().numpy(), None if dd is None else dd.cpu().numpy())
        for b in range(B):
            for s in range(new[b]):
                at = lens[b] + s
                c0[t[b, at // page], at % page] = codes[b, s]
                s0[t[b, at // page], at % page] = sc[b, s]
        assert np.array_equal(raw(scales), s0)
        assert np.array_equal(raw(cache), c0)
    if Hq:
        for b in range(B):
            assert torch.equal(q_out[b, :new[b]], q[b, :new[b]])


def test_edges_of_the_format():
    """Zeros, ties, scales below E4M3's smallest and above its largest, NaN and infinity."""
    d, f = 64, float
    rows = torch.zeros((1, 8, 1, d))
    rows[0, 1, 0, :16] = torch.tensor([7, -7, 0.5, 1.5, -2.5, 3.4, -6.5, 6.5] + [0] * 8)
    rows[0, 2, 0, 16:32] = 2.0 ** -12          # scale 0: the codes are 8
    rows[0, 3, 0, 32:48] = torch.tensor([1e30, -1e30, 1, 448 * 3.5] + [0] * 12)
    rows[0, 4, 0, 48] = f("nan")
    rows[0, 5, 0, 0], rows[0, 5, 0, 1] = f("inf"), -1.0
    rows[0, 6] = torch.linspace(-3, 3, d)
    rows[0, 7, 0, :16] = 2.0 ** -7             # a subnormal scale
    x = rows.bfloat16().to(DEV)
    kc, vc, ks, vs = empty_cache(1, 8, 1, d, False, 1)
    zero = torch.zeros((1, 1), dtype=torch.int32, device=DEV)
    pkg.paged_append(None, x, x, kc, vc, zero, zero[0], k_scale=ks, v_scale=vs)
    assert torch.equal(kc, vc) and torch.equal(ks, vs)
    codes, scales = raw(kc)[0], raw(ks)[0]
    want_c, want_s = serving.quantise4(x.float().cpu().numpy()[0])
    fine = [0, 1, 2, 3, 6, 7]
    assert np.array_equal(codes[fine], want_c[fine]) and np.array_equal(scales[fine], want_s[fine])
    assert scales[4, 0, 3] == 0x7F and (scales[4, 0, :3] == 0).all()
    assert scales[5, 0, 0] == 0x7E and codes[5, 0, 0] == (15 | 8 << 4)
    assert np.isnan(serving.values4(codes, scales)[4, 0, 48:]).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rot,interleaved", [(16, False), (48, False), (64, False), (64, True),
                                             (32, True), (0, False), (None, False)])
def test_normed_and_turned_rows(d, rot, interleaved):
    """Blocks whose halves lie in different lanes, at far positions."""
    rot = d if rot is None else rot
    B, S, Hq, Hk, page = 2, 19, 3, 5, 16
    q, k, v = new_rows(B, S, Hq, Hk, d, 5, 0.3)
    g = torch.Generator().manual_seed(6)
    w = [(1 + 0.2 * torch.randn(d, generator=g)).to(DEV) for _ in range(2)]
    freq = torch.tensor(10000.0 ** (-np.arange(0, rot, 2) / max(rot, 1)), dtype=torch.float32)
    lens = torch.tensor([0, 1000], dtype=torch.int32, device=DEV)
    most = 1019 // page + 1
    table = table_of(B, most, B * most, 7)
    kc, vc, ks, vs = empty_cache(B * most, page, Hk, d, False, 8)
    dsc = torch.tensor([0.5, 1.0, 0.3, 2.0, 1.7], device=DEV)
    q_out = pkg.paged_append(q, k, v, kc, vc, table, lens, None, w[0], w[1],
                             freq.to(DEV) if rot else None, interleaved=interleaved, k_descale=dsc,
                             k_scale=ks, v_scale=vs)
    pos = lens.cpu().numpy()[:, None] + np.arange(S)
    t = table.cpu().numpy()
    pg, sl = t[np.arange(B)[:, None], pos // page], pos % page
    y, _ = serving.norm_rope(_np(k), _np(w[1]), 1e-6, freq.numpy(), pos, interleaved)
    err = 2.0 ** -18 * np.abs(y).max(-1, keepdims=True)
    codes, scales = raw(kc)[pg, sl], raw(ks)[pg, sl]
    got = serving.values4(codes, scales, dsc.cpu().numpy())
    step = serving.e4m3_values()[scales] * _np(dsc)[:, None]
    top = np.abs(y).reshape(B, S, Hk, -1, 16).max(-1) / 7
    assert np.all(np.abs(step - top) <= 2.0 ** -4 * top + err)
    assert np.all(np.abs(got - y) <= (0.5 + 2.0 ** -18) * step.repeat(16, -1) + err)
    want_c, want_s = serving.quantise4(v.float().cpu().numpy())
    assert np.array_equal(raw(vc)[pg, sl], want_c) and np.array_equal(raw(vs)[pg, sl], want_s)
    want_q = pkg.qk_norm_rope(q, None, w[0], None, freq.to(DEV) if rot else None,
                              torch.tensor(pos, dtype=torch.int32, device=DEV),
                              interleaved=interleaved)[0]
    assert torch.equal(q_out, want_q)


def test_places_outside_the_cache_are_not_written():
    d, page = 64, 4
    q, k, v = new_rows(3, 2, 0, 2, d, 9)
    cache = empty_cache(3, page, 2, d, False, 10)
    before = [raw(t) for t in cache]
    table = torch.tensor([[0, 7], [-1, 1], [2, 2]], dtype=torch.int32, device=DEV)
    lens = torch.tensor([4, 0, 7], dtype=torch.int32, device=DEV)  # bad pages; the table's end
    pkg.paged_append(None, k, v, cache[0], cache[1], table, lens, k_scale=cache[2],
                     v_scale=cache[3])
    assert pkg.cp_get_last_status() == pkg.STATUS_CODES["CP_ERR_CACHE"]
    for i, (t, b) in enumerate(zip(cache, before)):
        x = (k, v)[i % 2].float().cpu().numpy()
        b[2, 3] = serving.quantise4(x[2, 0])[i // 2]
        assert np.array_equal(raw(t), b)


class Batch4(Batch):
    """A filled cache in 4 bits; slots that no sequence owns hold NaN."""

    def __init__(self, lens, n_q, Hq, Hk, d, page, P=0, seed=0, head_major=False, scale=1.0,
                 descaled=True):
        super().__init__(lens, n_q, Hq, Hk, d, page, P, False, seed, head_major, scale)
        g = torch.Generator().manual_seed(seed + 1)
        self.kd, self.vd = (((0.2 + torch.rand(Hk, generator=g)) * (1 if x else scale)).to(DEV)
                            for x in range(2))
        if not descaled:
            self.kd.fill_(1), self.vd.fill_(1)
        self.descaled = descaled
        for x, dsc in (("k", self.kd), ("v", self.vd)):
            rows = _np(getattr(self, x))
            junk = np.isnan(rows[..., :1, 0])
            codes, scales = serving.quantise4(np.nan_to_num(rows), dsc.cpu().numpy())
            scales[np.broadcast_to(junk[..., None], scales.shape)] = 0x7F
            for name, c in ((x, codes), (x + "s", scales)):
                c = torch.tensor(c, device=DEV)
                if head_major:
                    c = c.transpose(1, 2).contiguous().transpose(1, 2)
                setattr(self, name, c)

    def run(self, **kw):
        return pkg.paged_attn_decode(self.q, self.k, self.v, self.table, self.lens, self.prefix,
                                     self.P, self.kd if self.descaled else None,
                                     self.vd if self.descaled else None, k_scale=self.ks,
                                     v_scale=self.vs, **kw)

    def value(self, c, desc):
        scales = self.ks if c is self.k else self.vs
        return serving.values4(raw(c), raw(scales), desc.cpu().numpy())


@pytest.mark.parametrize("lens,n_q,Hq,Hk,d,page,P,e4m3,hm", CASES)
def test_decode(lens, n_q, Hq, Hk, d, page, P, e4m3, hm):
    b = Batch4(lens, n_q, Hq, Hk, d, page, P, seed=len(lens) + page, head_major=hm, descaled=e4m3)
    b.check(*b.run())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("scale", [2.0 ** -7, 1.0, 24.0])
def test_decode_of_small_and_large_scores(d, scale):
    b = Batch4([37, 260, 1100, 64], 2, 12, 2, d, 16, seed=3, scale=scale)
    b.check(*b.run())


@pytest.mark.parametrize("Hq", [4, 12])
@pytest.mark.parametrize("fall", [False, True])
def test_decode_of_scores_that_rise_or_fall_along_the_keys(Hq, fall):
    """Scales from 2^-6 to 2^5 along the keys, all entries of one sign: scores that pass a row's
    reference again and again, or leave it behind by more than fp16 holds."""
    d, page, n = 64, 16, 900
    b = Batch4([n, 3], 1, Hq, 1, d, page, seed=21)
    b.q.abs_()
    t = b.table.cpu().numpy()[0]
    pos = np.arange(n)
    code = (8 + 88 * pos // n).astype(np.uint8)
    at = torch.tensor(t[pos // page], device=DEV).long(), torch.tensor(pos % page, device=DEV)
    b.k[at[0], at[1]] = 0xFF
    b.ks[at[0], at[1]] = torch.tensor(code[::-1].copy() if fall else code, device=DEV)[:, None, None]
    b.check(*b.run())


@pytest.mark.parametrize("n_q,P", [(1, 0), (3, 70)])
def test_the_split_and_its_join(n_q, P):
    """Sequences cut over many blocks, and short ones beside them."""
    b = Batch4([6001, 70 + n_q, 0, 9000, 333], n_q, 8, 2, 128, 64, P, seed=5, head_major=True)
    b.check(*b.run())


def test_a_nan_block_reaches_the_rows_that_see_it_alone():
    b = Batch4([40, 40], 1, 4, 2, 64, 16, seed=6)
    at = b.table[1, 1], 3
    b.ks[int(at[0]), at[1], 1, 2] = 0x7F
    out, lse = b.run()
    assert torch.isnan(out[1, 0, 2:]).all() and torch.isnan(lse[1, 2:]).all()
    assert not torch.isnan(out[0]).any() and not torch.isnan(out[1, 0, :2]).any()


def test_a_bad_page_makes_its_rows_nan():
    b = Batch4([40, 40], 1, 4, 2, 128, 16, seed=7)
    b.table[0, 2] = 1 << 20
    out, lse = b.run()
    assert pkg.cp_get_last_status() == pkg.STATUS_CODES["CP_ERR_CACHE"]
    assert torch.isnan(out[0]).all() and torch.isnan(lse[0]).all()
    b.table[0, 2] = b.table[1, 2]
    again, lse2 = b.run()
    assert torch.equal(out[1], again[1]) and torch.equal(lse[1], lse2[1])


def test_a_captured_step_follows_its_lengths():
    """Append and decode in one graph, replayed as the sequences grow, equals the eager steps."""
    B, Hq, Hk, d, page, steps = 5, 8, 2, 128, 16, 6
    most = 8
    lens = torch.tensor([0, 5, 30, 63, 100], dtype=torch.int32, device=DEV)
    table = table_of(B, most, B * most, 1)
    caches = [empty_cache(B * most, page, Hk, d, True, 2) for _ in range(2)]
    for c in caches:  # values, not NaN
        c[2].fill_(0x30), c[3].fill_(0x30)
    fresh = [new_rows(B, 1, Hq, Hk, d, 20 + i, 0.2) for i in range(steps)]
    q, k, v = (t.clone() for t in fresh[0])

    def step(q, k, v, c, lens):
        pkg.paged_append(None, k, v, c[0], c[1], table, lens, k_scale=c[2], v_scale=c[3])
        lens += 1
        return pkg.paged_attn_decode(q, c[0], c[1], table, lens, k_scale=c[2], v_scale=c[3])

    eager_lens, graph_lens = lens.clone(), lens.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(q, k, v, [t.clone() for t in caches[1]], lens.clone())
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = step(q, k, v, caches[1], graph_lens)
    for rows in fresh:
        want, wantl = step(*rows, caches[0], eager_lens)
        for to, x in zip((q, k, v), rows):
            to.copy_(x)
        graph.replay()
        assert torch.equal(out, want) and torch.equal(lse, wantl)
    assert all(torch.equal(a, b) for a, b in zip(*caches))


def test_offsets_past_32_bits():
    """A cache of 5 GB of codes: its last pages are appended to and attended."""
    Hk, d, page = 2, 128, 64
    n_pages = 5 * 2 ** 30 // (page * Hk * d // 2)
    kc, vc = (torch.empty((n_pages, page, Hk, d // 2), dtype=torch.uint8, device=DEV)
              for _ in range(2))
    # scales strided as far
    ks, vs = (torch.empty((n_pages, page, Hk, d // 2), dtype=torch.uint8, device=DEV)[..., :d // 16]
              for _ in range(2))
    table = torch.tensor([[n_pages - 1, n_pages - 3]], dtype=torch.int32, device=DEV)
    q, k, v = new_rows(1, 100, 4, Hk, d, 11, 0.2)
    zero = torch.zeros(1, dtype=torch.int32, device=DEV)
    pkg.paged_append(None, k, v, kc, vc, table, zero, k_scale=ks, v_scale=vs)
    out, lse = pkg.paged_attn_decode(q[:, -1:].contiguous(), kc, vc, table, zero + 100, k_scale=ks,
                                     v_scale=vs)
    near = [t[[n_pages - 1, n_pages - 3]].contiguous() for t in (kc, vc, ks, vs)]
    for t, x in zip(near, (0, 0, 1, 1)):
        rows = (k, v)[0 if t is near[0] or t is near[2] else 1].float().cpu().numpy()[0]
        assert np.array_equal(raw(t).reshape(-1, *t.shape[2:])[:100], serving.quantise4(rows)[x])
    table2 = torch.tensor([[0, 1]], dtype=torch.int32, device=DEV)
    again, lse2 = pkg.paged_attn_decode(q[:, -1:].contiguous(), near[0], near[1], table2,
                                        zero + 100, k_scale=near[2], v_scale=near[3])
    assert torch.equal(out, again) and torch.equal(lse, lse2)


def test_what_does_not_fit_is_refused():
    b = Batch4([20], 1, 4, 2, 64, 16, seed=8)
    kw = dict(k_scale=b.ks, v_scale=b.vs)
    args = (b.q, b.k, b.v, b.table, b.lens)
    with pytest.raises(TypeError, match="v_scale"):
        pkg.paged_attn_decode(*args, k_scale=b.ks)
    with pytest.raises(TypeError, match="uint8"):
        pkg.paged_attn_decode(b.q, b.k.view(torch.float8_e4m3fn), b.v, b.table, b.lens, **kw)
    with pytest.raises(TypeError, match="k_scale"):
        pkg.paged_attn_decode(*args, k_scale=b.ks.float(), v_scale=b.vs)
    with pytest.raises(ValueError, match="k_scale"):
        pkg.paged_attn_decode(*args, k_scale=b.ks[..., :2], v_scale=b.vs)
    with pytest.raises(ValueError, match="contiguous in its last"):
        pkg.paged_attn_decode(*args, k_scale=b.ks, v_scale=b.vs.repeat(1, 1, 1, 2)[..., ::2])
    with pytest.raises(ValueError, match="k_descale"):
        pkg.paged_attn_decode(*args, k_descale=torch.ones(3, device=DEV), **kw)
    with pytest.raises(pkg.CpError, match="ALIGN"):
        far = torch.zeros(b.ks.numel() + 4, dtype=torch.uint8, device=DEV)[4:].view(b.ks.shape)
        pkg.paged_attn_decode(*args, k_scale=far, v_scale=b.vs)
