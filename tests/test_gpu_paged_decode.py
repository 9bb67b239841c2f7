"""cp_paged_attn_decode against the fp64 oracle.

Tolerances.  Scores are fp32 sums of exact products (bf16 x bf16, or fp16 x
E4M3 code): with at most 128 terms the error of a score is below 2^-17 of
sum |q k| / sqrt(d), and of the logarithm's argument below twice that; the
running maxima, exponentials (2^-22) and sums add 2^-20 of the result's size
in units where l = 1.  So lse is within 2^-16 (A + 1), A the row's largest
sum |q k| / sqrt(d).  P is rounded to bf16 (2^-8 at most; to fp16, 2^-11, for
E4M3 caches) and divided by an exact sum: out is off by at most that share of
sum p |v|, plus the scores' part, 2^-15 (A + 1) sum p |v|, plus its own
rounding, 2^-8 of the value.
"""
import os

import numpy as np
import pytest
import torch

import context_ring_attention_fwd_gb300 as pkg
from oracle import serving

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


class Batch:
    """A filled cache with a table; slots that no sequence owns hold NaN."""

    def __init__(self, lens, n_q, Hq, Hk, d, page, P=0, e4m3=False, seed=0, head_major=False,
                 scale=1.0):
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        B = len(lens)
        self.P, self.n_q = P, n_q
        shared, whole = -(-P // page), P // page
        most = max(1, max(-(-max(lens) // page), shared))
        own = [0 if n == 0 else -(-n // page) - whole for n in lens]
        n_pages = shared + sum(own) + 2
        order = rng.permutation(n_pages)
        prefix, at = order[:shared], shared
        table = np.full((B, most), -1, dtype=np.int32)
        table[:, :whole] = prefix[:whole]
        written = torch.zeros((n_pages, page), dtype=torch.bool)
        for p in range(P):
            written[prefix[p // page], p % page] = True
        for b, n in enumerate(lens):
            table[b, whole:whole + own[b]] = order[at:at + own[b]]
            at += own[b]
            for p in range(P, n):
                written[table[b, p // page], p % page] = True
        shape = (n_pages, Hk, page, d) if head_major else (n_pages, page, Hk, d)
        self.kd = self.vd = None
        caches = []
        for x in range(2):
            c = torch.randn(shape, generator=g) * (1 if x else scale)
            if e4m3:
                dsc = (0.004 + 0.004 * torch.rand(Hk, generator=g)) * (1 if x else scale)
                by = dsc[None, :, None, None] if head_major else dsc[:, None]
                c = (c / by).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                junk = 0x7F
                setattr(self, "vd" if x else "kd", dsc.to(DEV))
            else:
                c, junk = c.to(torch.bfloat16), float("nan")
            c = c.to(DEV)
            c = c.transpose(1, 2) if head_major else c
            c[~written.to(DEV)] = junk
            caches.append(c)
        self.k, self.v = caches
        self.q = (torch.randn((B, n_q, Hq, d), generator=g) * scale).to(torch.bfloat16).to(DEV)
        self.table = torch.tensor(table, device=DEV)
        self.lens = torch.tensor(lens, dtype=torch.int32, device=DEV)
        self.prefix = torch.tensor(prefix, dtype=torch.int32, device=DEV) if P else None

    def run(self, **kw):
        return pkg.paged_attn_decode(self.q, self.k, self.v, self.table, self.lens, self.prefix,
                                     self.P, self.kd, self.vd, **kw)

    def value(self, c, desc):
        if c.dtype != torch.uint8:
            return _np(c)
        return _np(c.cpu().view(torch.float8_e4m3fn).float()) * _np(desc)[:, None]

    def check(self, out, lse, rows=None):
        k, v = self.value(self.k, self.kd), self.value(self.v, self.vd)
        pages = () if self.prefix is None else self.prefix.cpu().numpy()
        args = (self.table.cpu().numpy(), self.lens.tolist(), pages, self.P)
        q = _np(self.q)
        want, wantl = serving.paged_decode(q, k, v, *args)
        size, _ = serving.paged_decode(q, k, np.abs(v), *args)        # sum p |v|
        d = q.shape[-1]
        A = (np.abs(q).max(-1, keepdims=True) * np.nanmax(np.abs(k)) * np.sqrt(d)).max()
        rnd = 2.0 ** -11 if self.kd is not None else 2.0 ** -8
        got, gotl = _np(out), _np(lse)
        pick = slice(None) if rows is None else rows
        tol = (rnd + 2.0 ** -15 * (A + 1)) * size + 2.0 ** -8 * np.abs(want)
        assert np.all(np.abs(got - want)[pick] <= tol[pick])
        empty = np.isneginf(wantl)
        assert np.array_equal(np.isneginf(gotl)[pick], empty[pick])
        assert np.all(np.abs(np.where(empty, 0, gotl - np.where(empty, 0, wantl)))[pick]
                      <= 2.0 ** -16 * (A + 1))


CASES = [
    # lens, n_q, Hq, Hk, d, page, P, e4m3, head-major
    ([1], 1, 1, 1, 128, 16, 0, False, False),
    ([1], 1, 4, 1, 64, 1, 0, True, False),
    ([63, 64, 65, 0, 1, 200], 1, 8, 2, 128, 16, 0, False, False),
    ([63, 64, 65, 0, 1, 200], 1, 8, 2, 128, 16, 0, True, True),
    ([700], 1, 32, 8, 128, 16, 0, False, False),
    ([5, 300, 17], 1, 40, 2, 64, 48, 0, False, True),          # 20 rows: two row tiles
    ([5, 300, 17], 1, 5, 5, 64, 7, 0, True, False),
    ([130, 4, 0, 131], 4, 6, 2, 128, 32, 0, False, False),     # several queries
    ([3, 1, 90, 16], 16, 2, 2, 64, 5, 0, True, False),         # more queries than tokens
    ([100, 101, 0, 164, 500], 1, 8, 2, 128, 16, 100, False, False),
    ([100, 103, 0, 164, 500], 3, 8, 2, 128, 16, 100, True, False),
    ([128, 129, 131], 2, 16, 4, 64, 64, 128, False, True),
    ([77, 78, 0, 79], 4, 3, 1, 128, 3, 77, True, True),        # the last queries' own keys only
    ([40] * 30, 1, 6, 2, 64, 16, 33, False, False),            # 90 rows under the prefix
    ([9, 2000, 1, 640], 2, 4, 4, 128, 16, 0, False, False),
]


@pytest.mark.parametrize("lens,n_q,Hq,Hk,d,page,P,e4m3,hm", CASES)
def test_decode(lens, n_q, Hq, Hk, d, page, P, e4m3, hm):
    t = Batch(lens, n_q, Hq, Hk, d, page, P, e4m3, seed=len(lens) + P + Hq, head_major=hm)
    out, lse = t.run()
    assert pkg.cp_get_last_status() == 0
    t.check(out, lse)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("P", [0, 4000])
def test_long_rows_with_steep_scores(e4m3, P):
    """Thousands of keys, scores with a spread of tens: the maximum moves late and far."""
    t = Batch([P + 1, P + 3700], 1, 4, 1, 128, 16, P, e4m3, seed=3, scale=3.0)
    t.check(*t.run())


def test_the_split_does_not_matter_and_runs_are_equal():
    """One long sequence cut over the whole grid, with and without a part called the prefix."""
    t = Batch([6000], 1, 4, 1, 64, 16, 0, seed=5)
    a, la = t.run()
    for _ in range(2):
        b, lb = t.run()
        assert torch.equal(a, b) and torch.equal(la, lb)
    t.prefix, t.P = t.table[0, :200].contiguous(), 3190
    t.check(*t.run())


def test_strided_queries_and_a_wider_table():
    t = Batch([50, 80], 2, 4, 2, 64, 16, 0, seed=6)
    want = t.run()
    whole = torch.zeros((2, 2, 8, 64), dtype=torch.bfloat16, device=DEV)
    whole[:, :, 2:6] = t.q
    t.q = whole[:, :, 2:6]
    wide = torch.full((2, 40), -1, dtype=torch.int32, device=DEV)
    wide[:, 3:3 + t.table.shape[1]] = t.table
    t.table = wide[:, 3:3 + t.table.shape[1]]
    got = t.run()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    one = t.q[:1, :1, :1].expand(2, 2, 4, 64)
    t.q = one
    a = t.run()
    t.q = one.contiguous()
    b = t.run()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_a_later_draft_with_nan_or_inf_does_not_reach_earlier_queries():
    t = Batch([90, 33], 3, 4, 2, 64, 16, 0, seed=7)
    want, wantl = t.run()
    for val in (float("nan"), float("inf")):
        p = 89
        pg = int(t.table[0, p // 16])
        keep = t.v[pg, p % 16].clone()
        t.v[pg, p % 16] = val
        got, gotl = t.run()
        assert torch.equal(got[0, :2], want[0, :2]) and torch.equal(got[1], want[1])
        assert not got[0, 2].isfinite().any() and torch.equal(gotl[:, :, :2], wantl[:, :, :2])
        t.v[pg, p % 16] = keep


def test_a_row_of_nan_stays_alone():
    t = Batch([70, 30, 20], 1, 4, 2, 128, 16, 10, seed=8)
    want, wantl = t.run()
    t.q[1, 0, 2, 7] = float("nan")
    got, gotl = t.run()
    assert got[1, 0, 2].isnan().all() and gotl[1, 2].isnan().all()
    keep = torch.ones((3, 1, 4), dtype=torch.bool, device=DEV)
    keep[1, 0, 2] = False
    assert torch.equal(got[keep], want[keep])
    assert torch.equal(gotl.transpose(1, 2)[keep], wantl.transpose(1, 2)[keep])


@pytest.mark.parametrize("n_q", [1, 3])
@pytest.mark.parametrize("P", [0, 40])
def test_bad_pages_and_lengths_are_reported_and_stay_with_their_sequence(P, n_q):
    """The kernels' own bounds checks keep every access inside the cache."""
    lens = [P + 100, P + 60, P + 70, P + 90, P + 10]
    t = Batch(lens, n_q, 4, 2, 64, 16, P, seed=9)
    want, wantl = t.run()
    t.table[0, (P + 50) // 16] = t.k.shape[0]
    t.table[1, (P + 59) // 16] = -5                      # under the last queries
    t.lens[2] = -1
    t.lens[3] = t.table.shape[1] * 16 + 1
    got, gotl = t.run()
    assert pkg.cp_get_last_status() == pkg.STATUS_CODES["CP_ERR_CACHE"]
    assert pkg.cp_get_last_status() == 0
    for b in range(4):
        assert got[b, -1].isnan().all() and gotl[b, :, -1].isnan().all()
    assert torch.equal(got[4], want[4]) and torch.equal(gotl[4], wantl[4])
    if P:
        t = Batch(lens, n_q, 4, 2, 64, 16, P, seed=9)
        t.lens[4] = P - 1
        got, gotl = t.run()
        assert pkg.cp_get_last_status() == pkg.STATUS_CODES["CP_ERR_CACHE"]
        assert got[4].isnan().all() and torch.equal(got[:4], want[:4])
        t.lens[4] = 0
        t.prefix[1] = t.k.shape[0]
        got, gotl = t.run()
        assert pkg.cp_get_last_status() == pkg.STATUS_CODES["CP_ERR_CACHE"]
        assert got[:4].isnan().all() and (got[4] == 0).all() and gotl[4].isneginf().all()


def test_graph_replays_follow_the_lengths_and_streams_do_not_disturb_each_other():
    t = Batch([64, 300], 1, 8, 2, 128, 16, 0, seed=10)
    full = t.lens.clone()
    want = [t.run()]
    t.lens.copy_(torch.tensor([10, 65], dtype=torch.int32))
    want.append(t.run())
    t.lens.copy_(torch.tensor([0, 1], dtype=torch.int32))
    want.append(t.run())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = t.run()
    for lens, (a, b) in zip((full, torch.tensor([10, 65]), torch.tensor([0, 1])), want):
        t.lens.copy_(lens)
        graph.replay()
        assert torch.equal(out, a) and torch.equal(lse, b)
    t.lens.copy_(full)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for _ in range(4):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(t.run())
    torch.cuda.synchronize()
    for a, b in got:
        assert torch.equal(a, want[0][0]) and torch.equal(b, want[0][1])


def test_binding_refusals():
    t = Batch([20, 30], 1, 4, 2, 64, 16, 0, seed=11)
    args = [t.q, t.k, t.v, t.table, t.lens]
    for at, bad, error in [(0, t.q.float(), TypeError), (0, t.q[:1], ValueError),
                           (1, t.k.float(), TypeError), (2, t.v[:, :8], ValueError),
                           (3, t.table[:1], ValueError), (3, t.table.long(), TypeError),
                           (4, t.lens.cpu(), ValueError), (4, t.lens.float(), TypeError)]:
        a = list(args)
        a[at] = bad
        with pytest.raises(error):
            pkg.paged_attn_decode(*a)
    with pytest.raises(ValueError):
        pkg.paged_attn_decode(*args, t.table[0, :1].contiguous(), 17)
    with pytest.raises(pkg.CpError):
        pkg.paged_attn_decode(*args, None, 16)
    with pytest.raises(pkg.CpError) as e:
        pkg.paged_attn_decode(*args, workspace=torch.empty(512, dtype=torch.uint8, device=DEV))
    assert e.value.name == "CP_ERR_BUFFER"
    with pytest.raises(pkg.CpError):
        pkg.paged_attn_decode(t.q[:, :, :3], *args[1:])


@pytest.mark.parametrize("P,e4m3", [(0, False), (0, True), (20, False)])
def test_a_bad_page_of_the_last_keys_marks_the_queries_that_see_it(P, e4m3):
    """The last two of four queries' keys begin a page: the first two queries see none of it."""
    t = Batch([34, 50, 3], 4, 4, 2, 64, 16, 0, e4m3, seed=12) if not P else \
        Batch([34, 50], 4, 4, 2, 64, 16, P, e4m3, seed=12)
    want, wantl = t.run()
    assert pkg.cp_get_last_status() == 0
    for bad in (-1, t.k.shape[0]):
        t.table[0, 2] = bad                              # positions 32, 33 of 34
        got, gotl = t.run()
        assert pkg.cp_get_last_status() == pkg.STATUS_CODES["CP_ERR_CACHE"]
        assert got[0, 2:].isnan().all() and gotl[0, :, 2:].isnan().all()
        assert torch.equal(got[0, :2], want[0, :2]) and torch.equal(gotl[0, :, :2], wantl[0, :, :2])
        assert torch.equal(got[1:], want[1:]) and torch.equal(gotl[1:], wantl[1:])


@pytest.mark.parametrize("P", [0, 5])
@pytest.mark.parametrize("d", [64, 128])
def test_the_weights_keep_more_than_their_rounding_to_bf16(d, P):
    """Few keys of nearly equal small scores and values of either sign.  P is held as its upper
    half and a bf16 rounding of the rest, which is below 2^-7 of P: off by 2^-15 of P, and 2^-20
    for the bit that keeps the rest from 0.  With the scores' part and the output's own rounding
    that is all; P rounded once would be off by up to 2^-8 of sum p |v|."""
    lens = [P + 2 + b % 9 for b in range(60)]
    t = Batch(lens, 1, 8, 2, d, 16, P, seed=20 + P, scale=0.25)
    pkg.test_set_prefix_path(0)
    try:
        out, _ = t.run()
    finally:
        pkg.test_set_prefix_path(-1)
    q, k, v = _np(t.q), _np(t.k), _np(t.v)
    args = (t.table.cpu().numpy(), lens, () if t.prefix is None else t.prefix.cpu().numpy(), P)
    want, _ = serving.paged_decode(q, k, v, *args)
    size, _ = serving.paged_decode(q, k, np.abs(v), *args)
    A = np.linalg.norm(q, axis=-1).max() * np.nanmax(np.linalg.norm(k, axis=-1)) / np.sqrt(d)
    tol = (2.0 ** -15 + 2.0 ** -20 + 2.0 ** -15 * (A + 1)) * size + 2.0 ** -8 * np.abs(want)
    assert np.all(np.abs(_np(out) - want) <= tol)


@pytest.mark.parametrize("n", [1, 40, 700])
def test_infinite_values_of_seen_keys_stay_infinite(n):
    """out = sum p v with p > 0: +inf, -inf, or NaN where both meet, and no other column."""
    t = Batch([n, n], 1, 4, 2, 64, 16, 0, seed=13)
    want, wantl = t.run()
    inf = float("inf")
    at = [(int(t.table[0, p // 16]), p % 16) for p in sorted({0, n // 2, n - 1})]
    t.v[at[0][0], at[0][1], :, 3] = inf
    t.v[at[-1][0], at[-1][1], :, 9] = -inf
    t.v[at[0][0], at[0][1], :, 20] = inf
    t.v[at[-1][0], at[-1][1], :, 20] = inf if n == 1 else -inf
    got, gotl = t.run()
    assert torch.equal(gotl, wantl) and torch.equal(got[1], want[1])
    assert (got[0, :, :, 3] == inf).all() and (got[0, :, :, 9] == -inf).all()
    assert (got[0, :, :, 20] == inf).all() if n == 1 else got[0, :, :, 20].isnan().all()
    keep = [c for c in range(64) if c not in (3, 9, 20)]
    assert torch.equal(got[0][..., keep], want[0][..., keep])
