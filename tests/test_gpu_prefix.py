"""cp_paged_attn_decode with the prefix on its tcgen05 kernel: row counts around its 128- and 256-row tiles, prefixes around its
128-key tiles, items cut between CTAs and whole ones, against attention in 64
bits on the GPU.  Tolerances as derived in test_gpu_paged_decode.py, with the
largest product of norms in place of the largest sum of magnitudes (Cauchy's
inequality); a row's reference may lie 2^64 below its maximum, which changes
no relative error."""
import os

import numpy as np
import pytest
import torch

import context_ring_attention_fwd_gb300 as pkg

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
    pkg.test_set_prefix_path(1)
    yield
    pkg.test_set_prefix_path(-1)
    assert pkg.cp_get_last_status() == 0


class Case:
    def __init__(self, B, n_q, Hq, Hk, d, page, P, rest, e4m3, seed, scale=1.0, idle=()):
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.P = P
        lens = [0 if b in idle else P + int(rng.integers(0, rest + 1)) for b in range(B)]
        lens = [n if n else (1 if P == 0 and b not in idle else n) for b, n in enumerate(lens)]
        shared, whole = -(-P // page), P // page
        own = [0 if n == 0 else -(-n // page) - whole for n in lens]
        n_pages = shared + sum(own) + 2
        order = rng.permutation(n_pages)
        table = np.full((B, max(1, whole + max(own), shared)), -1, dtype=np.int32)
        table[:, :whole] = order[:whole]
        at, written = shared, torch.zeros((n_pages, page), dtype=torch.bool)
        pos = np.arange(P)
        written[order[pos // page], pos % page] = True
        for b, n in enumerate(lens):
            table[b, whole:whole + own[b]] = order[at:at + own[b]]
            at += own[b]
            pos = np.arange(P, n)
            written[table[b, pos // page], pos % page] = True
        self.kd = self.vd = None
        caches = []
        for x in range(2):
            c = torch.randn((n_pages, page, Hk, d), generator=g).to(DEV) * (1 if x else scale)
            if e4m3:
                dsc = ((0.004 + 0.004 * torch.rand(Hk, generator=g)) * (1 if x else scale)).to(DEV)
                c = (c / dsc[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                setattr(self, "vd" if x else "kd", dsc)
            else:
                c = c.to(torch.bfloat16)
            c[~written.to(DEV)] = 0x7F if e4m3 else float("nan")
            caches.append(c)
        self.k, self.v = caches
        self.q = (torch.randn((B, n_q, Hq, d), generator=g) * scale).to(torch.bfloat16).to(DEV)
        self.table = torch.tensor(table, device=DEV)
        self.lens = torch.tensor(lens, dtype=torch.int32, device=DEV)
        self.prefix = torch.tensor(order[:shared], dtype=torch.int32, device=DEV)

    def run(self, **kw):
        return pkg.paged_attn_decode(self.q, self.k, self.v, self.table, self.lens, self.prefix,
                                     self.P, self.kd, self.vd, **kw)

    def gathered(self, c, desc, pages, lo, hi):
        pos = torch.arange(lo, hi, device=DEV)
        x = c[pages.long()[pos // c.shape[1]], pos % c.shape[1]]
        if desc is not None:
            x = x.view(torch.float8_e4m3fn).float()
        x = x.double()
        return x if desc is None else x * desc.double()[:, None]

    def check(self, out, lse):
        B, n_q, Hq, d = self.q.shape
        Hk = self.k.shape[2]
        G = Hq // Hk
        kp, vp = (self.gathered(c, s, self.prefix, 0, self.P)
                  for c, s in ((self.k, self.kd), (self.v, self.vd)))
        rnd = 2.0 ** -11 if self.kd is not None else 2.0 ** -8
        for b, n in enumerate(self.lens.tolist()):
            if n == 0:
                assert (out[b] == 0).all() and lse[b].isneginf().all()
                continue
            k, v = (torch.cat([x, self.gathered(c, s, self.table[b], self.P, n)])
                    for x, c, s in ((kp, self.k, self.kd), (vp, self.v, self.vd)))
            q = self.q[b].double().view(n_q, Hk, G, d)
            sc = torch.einsum("ihgd,khd->ihgk", q, k) / d ** 0.5
            last = n - n_q + torch.arange(n_q, device=DEV)
            seen = torch.arange(n, device=DEV) <= last.clamp(min=self.P - 1)[:, None]
            sc = sc.masked_fill(~seen[:, None, None], -float("inf"))
            p = sc.softmax(-1)
            want = torch.einsum("ihgk,khd->ihgd", p, v)
            size = torch.einsum("ihgk,khd->ihgd", p, v.abs())
            A = (q.norm(dim=-1).max() * k.norm(dim=-1).max() / d ** 0.5).item()
            tol = (rnd + 2.0 ** -15 * (A + 1)) * size + 2.0 ** -8 * want.abs()
            err = (out[b].double().view(n_q, Hk, G, d) - want).abs()
            assert (err <= tol).all(), (b, (err - tol).max().item())
            z = sc.logsumexp(-1).permute(1, 2, 0).reshape(Hq, n_q)
            assert ((lse[b].double() - z).abs() <= 2.0 ** -16 * (A + 1)).all()


CASES = [
    # B, n_q, Hq, Hk, d, page, P, rest, e4m3, idle
    (33, 1, 1, 1, 128, 16, 1, 3, False, ()),
    (33, 1, 2, 2, 64, 16, 127, 3, True, (0,)),
    (32, 1, 8, 2, 128, 16, 128, 0, False, ()),                 # 128 rows, nothing behind
    (43, 1, 3, 1, 128, 48, 129, 10, False, (5, 42)),           # 129 rows
    (43, 3, 6, 3, 64, 7, 300, 10, False, ()),                  # 258 rows, odd pages
    (64, 1, 4, 1, 128, 64, 1000, 100, True, ()),               # 256 rows
    (100, 2, 12, 4, 128, 16, 777, 60, True, (7,)),             # 600 rows
    (100, 2, 12, 4, 64, 16, 777, 60, True, ()),
    (40, 1, 8, 8, 128, 32, 5000, 200, False, ()),              # cut between CTAs
    (40, 1, 32, 2, 64, 1, 2500, 200, False, ()),               # pages of one token
    (16, 16, 16, 16, 128, 128, 260, 40, True, ()),             # whole items, several per CTA
    (120, 4, 24, 8, 128, 16, 140, 5, False, ()),               # 1440 rows
]


@pytest.mark.parametrize("B,n_q,Hq,Hk,d,page,P,rest,e4m3,idle", CASES)
def test_prefix(B, n_q, Hq, Hk, d, page, P, rest, e4m3, idle):
    t = Case(B, n_q, Hq, Hk, d, page, P, rest, e4m3, B + P, idle=idle)
    before = pkg.launch_counts()[0]
    out, lse = t.run()
    assert pkg.launch_counts()[0] == before + 1       # the tcgen05 kernel ran
    assert pkg.cp_get_last_status() == 0
    t.check(out, lse)
    again = t.run()
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("rising", [False, True])
def test_references_that_have_to_move(e4m3, rising):
    """Scores that climb by hundreds along the prefix (every tile passes the guard), and scores
    with a spread of tens."""
    t = Case(40, 1, 4, 1, 128, 16, 1500, 20, e4m3, 4, scale=3.0)
    if rising:
        t.q[:] = t.q.abs()
        pos = torch.arange(t.P, device=DEV)
        ramp = 0.002 * pos[:, None, None]
        rows = (ramp.expand(t.P, 1, 128) / (t.kd[:, None] if e4m3 else 1.0))
        rows = rows.clamp(max=448).to(torch.float8_e4m3fn).view(torch.uint8) if e4m3 else \
            rows.to(torch.bfloat16)
        t.k[t.prefix.long()[pos // 16], pos % 16] = rows
    t.check(*t.run())


def test_a_row_of_nan_and_rows_of_any_size_stay_alone():
    for e4m3 in (False, True):
        t = Case(50, 1, 4, 1, 64, 16, 400, 20, e4m3, 6)
        want, wantl = t.run()
        t.q[3, 0, 1, 5] = float("nan")
        t.q[4, 0, 2, 5] = float("inf")
        got, gotl = t.run()
        assert got[3, 0, 1].isnan().all() and gotl[3, 1].isnan().all()
        keep = torch.ones((50, 1, 4), dtype=torch.bool, device=DEV)
        keep[3, 0, 1] = keep[4, 0, 2] = False
        assert torch.equal(got[keep], want[keep])
        t = Case(50, 1, 4, 1, 64, 16, 400, 20, e4m3, 6)
        t.q[7] *= 2.0 ** -60                            # scores of zero: the mean of v
        t.q[8] = 0
        t.check(*t.run())


def test_a_bad_page_reaches_every_used_row_and_is_reported():
    for e4m3 in (False, True):
        t = Case(50, 1, 4, 1, 128, 16, 400, 20, e4m3, 7, idle=(9,))
        t.prefix[11] = t.k.shape[0] + 3
        got, gotl = t.run()
        assert pkg.cp_get_last_status() == pkg.STATUS_CODES["CP_ERR_CACHE"]
        assert (got[9] == 0).all() and gotl[9].isneginf().all()
        keep = torch.arange(50, device=DEV) != 9
        assert got[keep].isnan().all() and gotl[keep].isnan().all()


def test_a_wait_that_runs_out_is_reported_and_marks_the_rows():
    """The test hook withholds one tile's signal; the bounded waits end and the parts that the
    CTA owed come out as NaN."""
    for e4m3 in (False, True):
        t = Case(50, 1, 4, 2, 128, 16, 700, 20, e4m3, 8)
        want = t.run()
        assert pkg.cp_get_last_status() == 0
        pkg.test_set_wait_fault(True, 20_000_000)
        try:
            got, gotl = t.run()
            assert pkg.cp_get_last_status() == pkg.STATUS_CODES["CP_ERR_TIMEOUT"]
        finally:
            pkg.test_set_wait_fault(False)
        assert got[:, :, :2].isnan().all() and gotl[:, :2].isnan().all()   # key head 0: CTA 0's
        assert torch.equal(got[:, :, 2:], want[0][:, :, 2:])
        again = t.run()
        assert pkg.cp_get_last_status() == 0
        assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])


def test_replayed_in_a_graph_with_other_lengths():
    t = Case(48, 1, 4, 1, 128, 16, 640, 100, False, 9)
    t.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = t.run()
    t.lens.copy_((t.lens - 1).clamp(min=t.P))
    t.lens[5] = 0
    graph.replay()
    t.check(out, lse)


@pytest.mark.parametrize("e4m3", [False, True])
def test_both_kernels_give_the_same_attention(e4m3):
    """The 16-row items and the tcgen05 kernel on one batch, and the rule's own choice on
    either side of its threshold."""
    t = Case(48, 1, 8, 4, 128, 16, 3000, 100, e4m3, 12)
    got = []
    for path in (0, 1):
        pkg.test_set_prefix_path(path)
        got.append(t.run())
        t.check(*got[-1])
    pkg.test_set_prefix_path(-1)
    before = pkg.launch_counts()[0]
    t.run()                                     # 6 * 3000 keys * 4 heads: 37 or 18 MB
    assert pkg.launch_counts()[0] == before
    big = Case(40, 1, 64, 8, 128, 64, 4000, 5, e4m3, 13)
    out = big.run()                             # 20 * 4000 keys * 8 heads: 328 or 164 MB
    assert pkg.launch_counts()[0] == before + 1
    big.check(*out)
    pkg.test_set_prefix_path(1)


@pytest.mark.parametrize("path", [0, 1])
@pytest.mark.parametrize("far", [-300.0, -20.0, 50.0])
def test_keys_that_score_minus_infinity_leave_the_others(path, far):
    """Keys of infinite entries lead the prefix over whole tiles and whole CTAs' shares of it:
    the heads that score them -inf attend the others, whatever those score, and the head that
    scores them +inf is NaN."""
    t = Case(40, 1, 4, 1, 128, 16, 20000, 4, False, 14)
    t.q[:, :, :, 0] = torch.tensor([-1.0, -2.0, 1.0, -0.5], device=DEV)
    t.q[:, :, :, 1] = 64.0
    pos = torch.arange(t.P, device=DEV)
    rows = t.k[t.prefix.long()[pos // 16], pos % 16]
    rows[:, 0, 0] = 0.0
    rows[:, 0, 1] = far * 128 ** 0.5 / 64.0            # moves every finite score by `far`
    rows[pos < 16992, 0, 0] = float("inf")
    t.k[t.prefix.long()[pos // 16], pos % 16] = rows
    own = t.k[:, :, :, 1]
    own[~own.isnan()] = far * 128 ** 0.5 / 64.0
    pkg.test_set_prefix_path(path)
    try:
        out, lse = t.run()
    finally:
        pkg.test_set_prefix_path(1)
    assert out[:, :, 2].isnan().all() and lse[:, 2].isnan().all()
    live = [0, 1, 3]
    t.q = t.q[:, :, live].contiguous()
    # the same attention without the keys that nobody sees, 1062 whole pages
    cut = Case.__new__(Case)
    cut.kd = cut.vd = None
    cut.q, cut.k, cut.v = t.q, t.k, t.v
    cut.prefix, cut.table = t.prefix[1062:].contiguous(), t.table[:, 1062:].contiguous()
    cut.P, cut.lens = t.P - 16992, t.lens - 16992
    cut.check(out[:, :, live], lse[:, live])


@pytest.mark.parametrize("e4m3,d,rows,page,wide", [
    (False, 128, 16, 64, False), (False, 128, 32, 64, True), (False, 64, 32, 64, False),
    (False, 64, 48, 64, True), (True, 128, 32, 64, False), (True, 128, 48, 64, True),
    (True, 64, 64, 64, False), (True, 64, 96, 64, True), (False, 128, 32, 60, False),
    (False, 128, 48, 60, True), (False, 64, 48, 60, False), (False, 64, 64, 60, True),
    (True, 128, 48, 60, False), (True, 128, 96, 60, True)])
def test_the_rule_takes_the_kernel_that_measured_faster(e4m3, d, rows, page, wide):
    """8 key heads under a 32K prefix, on both sides of the rule for each type and size of head,
    by TMA and by cp.async."""
    t = Case(rows // 4, 1, 32, 8, d, page, 32768, 30, e4m3, rows)
    pkg.test_set_prefix_path(-1)
    try:
        before = pkg.launch_counts()[0]
        out = t.run()
        assert pkg.launch_counts()[0] - before == int(wide)
    finally:
        pkg.test_set_prefix_path(1)
    t.check(*out)
