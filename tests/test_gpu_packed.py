"""cp_packed_attn_fwd and cp_packed_attn_bwd against the fp64 oracle.

Tolerances.  A score is a sum of d <= 128 exact products in fp32: its error is below 128 * 2^-23 =
2^-16 of A, the row's largest sum |q k| / sqrt(d), and its scaling and the exponent's argument add
2^-22 A; the exponential adds 2^-22 and a sum of n of them n 2^-24.  So with E = 2^-15 (A + 1) + n
2^-23 each P is known to E of itself before it is rounded to bf16 (2^-8 at most, which the row's
sum, formed in fp32, does not see), and lse to E.  out: (2^-8 + 2 E) sum p |v| (the other E for the
product's own n fp32 sums) and its own rounding, 2^-8 of the value.
Gradients, from the same out and lse as the oracle's: dv as out; dS = P (dP - D) is rounded to bf16,
2^-8 |dS|, and carries 2 E of P (sum |dO v| + sum |dO O|), the size of what cancels in it; dq and dk
sum that and are rounded once more.  E with the largest A of the call, since a key's gradient
mixes rows.
"""
import os

import numpy as np
import pytest
import torch

import context_ring_attention_fwd_gb300 as pkg
from oracle import packed
import packed_plan

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16 = torch.bfloat16


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


def int32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Prompts:
    """q, k, v as views of one projection's output; rows of no sequence hold NaN and infinities."""

    def __init__(self, lens, Hq, Hk, d, seed=0, lead=0, pad=5, scale=1.0, fused=True):
        g = torch.Generator().manual_seed(seed)
        self.ends = lead + np.concatenate([[0], np.cumsum(lens)]).astype(int)
        T = int(self.ends[-1]) + pad
        x = torch.randn((T, Hq + 2 * Hk, d), generator=g) * scale
        self.there = np.zeros(T, dtype=bool)
        self.there[lead:self.ends[-1]] = True
        x[~self.there] = float("nan")
        x[~self.there, :, ::3] = float("inf")
        x = x.to(BF16).to(DEV)
        self.q, self.k, self.v = x[:, :Hq], x[:, Hq:Hq + Hk], x[:, Hq + Hk:]
        if not fused:
            self.q, self.k, self.v = (t.contiguous() for t in (self.q, self.k, self.v))
        self.offsets = int32(self.ends)
        self.T, self.longest = T, max(lens) if len(lens) else 0
        self.shape = (T, Hq, d)
        self.dout = torch.randn(self.shape, generator=g)
        self.dout[~self.there] = float("nan")
        self.dout = self.dout.to(BF16).to(DEV)

    def forward(self, causal=True, **kw):
        T, Hq, d = self.shape
        out = torch.full(self.shape, -7.0, dtype=BF16, device=DEV)
        lse = torch.full((Hq, T), -7.0, device=DEV)
        got = pkg.packed_attn_fwd(self.q, self.k, self.v, self.offsets, causal, out=out, lse=lse,
                                  **kw)
        assert got[0] is out or got[0].data_ptr() == out.data_ptr()
        assert got[1].data_ptr() == lse.data_ptr()
        return out, lse

    def check(self, out, lse, causal=True):
        q, k, v = (np.where(self.there[:, None, None], _np(t), 0.0) for t in (self.q, self.k, self.v))
        want, wantl, A, spread = packed.attention(q, k, v, self.ends, causal)
        got, gotl = _np(out), _np(lse)
        here = self.there
        assert (got[~here] == -7).all() and (gotl[:, ~here] == -7).all()
        E = (2.0 ** -15 * (A + 1) + self.longest * 2.0 ** -23)[here]
        tol = (2.0 ** -8 + 2 * E[..., None]) * spread[here] + 2.0 ** -8 * np.abs(want[here])
        assert np.all(np.abs(got - want)[here] <= tol)
        assert np.all(np.abs(gotl - wantl)[:, here] <= E.T)

    def backward(self, out, lse, causal=True, fused=False, **kw):
        """Into tensors of their own, or into views of one projection's gradient."""
        T, Hq, d = self.shape
        Hk = self.k.shape[1]
        grad = torch.full((T, Hq + 2 * Hk, d), -7.0, dtype=BF16, device=DEV)
        to = [grad[:, :Hq], grad[:, Hq:Hq + Hk], grad[:, Hq + Hk:]]
        if not fused:
            to = [t.contiguous() for t in to]
        got = pkg.packed_attn_bwd(self.q, self.k, self.v, out, lse, self.dout, self.offsets,
                                  causal, dq=to[0], dk=to[1], dv=to[2], **kw)
        assert [g.data_ptr() for g in got] == [t.data_ptr() for t in to]
        return to

    def check_gradients(self, out, lse, grads, causal=True):
        zero = lambda t: np.where(self.there[:, None, None], _np(t), 0.0)  # noqa: E731
        q, k, v, o, g = (zero(t) for t in (self.q, self.k, self.v, out, self.dout))
        want, terms, fine = packed.attention_bwd(q, k, v, o, _np(lse), g, self.ends, causal)
        _, _, A, _ = packed.attention(q, k, v, self.ends, causal)
        here = self.there
        E = 2.0 ** -15 * (A.max(initial=0) + 1) + self.longest * 2.0 ** -23
        for i, (got, w) in enumerate(zip(grads, want)):
            got = _np(got)
            assert (got[~here] == -7).all()
            tol = (2.0 ** -8 + 2 * E) * terms[i] + 2.0 ** -8 * np.abs(np.nan_to_num(w))
            if i < 2:
                tol = tol + 2 * E * fine[i]
            assert np.all(np.abs(got - w)[here] <= tol[here]), ("dq", "dk", "dv")[i]


CASES = [
    # lens, Hq, Hk, d
    ([1], 1, 1, 128),
    ([1], 4, 1, 64),
    ([1, 1, 1], 8, 8, 64),
    ([16, 17, 15], 2, 1, 128),
    ([127, 128, 129], 2, 2, 128),          # a head to itself: 128 tokens to a tile
    ([255, 256, 257, 1], 1, 1, 64),
    ([31, 32, 33, 63, 64, 65], 8, 2, 128),  # 32 tokens to a tile
    ([100, 0, 0, 41, 0], 6, 2, 64),        # three heads: 126 rows of a tile; empty sequences
    ([0, 0], 4, 2, 128),
    ([300], 10, 2, 128),                   # five heads
    ([90, 7], 14, 2, 64),                  # seven
    ([513, 5], 8, 1, 128),                 # eight
    ([50, 20], 48, 1, 64),                 # 48: two tokens to a tile
    ([9, 30], 71, 1, 64),                  # one token to a tile
    ([13], 128, 1, 128),
    ([700, 130, 1, 385], 4, 4, 64),
    ([640], 32, 8, 128),
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens,Hq,Hk,d", CASES)
def test_forward(lens, Hq, Hk, d, causal):
    p = Prompts(lens, Hq, Hk, d, seed=len(lens) + Hq, lead=3 * (Hq % 2), pad=max(lens) % 7,
                fused=d == 128)
    p.check(*p.forward(causal), causal)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens,Hq,Hk,d", CASES)
def test_gradients(lens, Hq, Hk, d, causal):
    p = Prompts(lens, Hq, Hk, d, seed=len(lens) + Hq, lead=3 * (Hq % 2), pad=max(lens) % 7,
                fused=d == 128)
    out, lse = p.forward(causal)
    out[~torch.tensor(p.there)] = float("nan")
    p.check_gradients(out, lse, p.backward(out, lse, causal, fused=Hq % 4 == 0), causal)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens,Hq,Hk,d", [
    ([70, 9, 1], 16, 1, 64),      # two tokens to a warp's rows
    ([5, 40, 33], 32, 1, 128),    # one
    ([20, 3], 64, 1, 64),         # half a one
    ([17, 130, 64], 2, 1, 128),   # sixteen
])
def test_tokens_that_fill_a_warps_rows_or_do_not(lens, Hq, Hk, d, causal):
    p = Prompts(lens, Hq, Hk, d, seed=Hq, lead=2, pad=5, fused=True)
    out, lse = p.forward(causal)
    p.check(out, lse, causal)
    p.check_gradients(out, lse, p.backward(out, lse, causal, fused=True), causal)


def test_outputs_that_start_16_bytes_into_a_sector():
    p = Prompts([150, 40], 4, 2, 64, seed=5, pad=3)
    out, lse = p.forward()
    want = p.backward(out, lse)
    to = [torch.full((t.numel() + 8,), -7.0, dtype=BF16, device=DEV)[8:].view(t.shape)
          for t in want]
    assert all(t.data_ptr() % 32 == 16 for t in to)
    pkg.packed_attn_bwd(p.q, p.k, p.v, out, lse, p.dout, p.offsets, dq=to[0], dk=to[1], dv=to[2])
    assert all(torch.equal(a, b) for a, b in zip(to, want))


def test_gradients_are_differences():
    """Along a random direction in q, k and v the loss's slope, from the oracle's forward in 64
    bits, is the gradients' product with it: each gradient entry is known to 2^-7 of its size
    (the module's derivation) and they are independent enough for a tenth of the norm's."""
    p = Prompts([90, 50], 6, 2, 64, seed=11, lead=2)
    out, lse = p.forward()
    grads = [np.where(p.there[:, None, None], _np(t), 0.0) for t in p.backward(out, lse)]
    x = [np.where(p.there[:, None, None], _np(t), 0.0) for t in (p.q, p.k, p.v)]
    g = np.where(p.there[:, None, None], _np(p.dout), 0.0)
    rng = np.random.default_rng(12)
    for i in range(3):
        way = rng.standard_normal(x[i].shape)
        loss = []
        for sign in (1, -1):
            y = list(x)
            y[i] = x[i] + sign * 1e-5 * way
            loss.append(np.nansum(packed.attention(*y, p.ends, True)[0] * g))
        slope = (loss[0] - loss[1]) / 2e-5
        size = np.linalg.norm(grads[i] * way)
        assert abs(slope - (grads[i] * way).sum()) <= 2.0 ** -7 * size * 10


def test_gradients_do_not_change_from_run_to_run():
    p = Prompts([700, 30, 260], 8, 2, 128, seed=13)
    out, lse = p.forward()
    first = p.backward(out, lse)
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(first, p.backward(out, lse)))


def test_gradients_equal_the_ring_attentions():
    """Equal heads and one sequence: the ring's backward to a rounding or two."""
    p = Prompts([512], 4, 4, 128, seed=14, pad=0, fused=False)
    out, lse = p.forward()
    want = pkg.ring_attn_bwd(p.q[None], p.k[None], p.v[None], out[None], lse[None], p.dout[None])
    for a, b in zip(p.backward(out, lse), want):
        assert (a.float() - b[0].float()).abs().max() <= 2.0 ** -6 * b.float().abs().max()


def test_gradients_of_many_sequences():
    rng = np.random.default_rng(15)
    lens = rng.integers(0, 9, 3000)
    lens[1234] = 300
    p = Prompts(lens, 4, 2, 64, seed=16)
    out, lse = p.forward()
    p.check_gradients(out, lse, p.backward(out, lse))


def test_gradients_of_sequences_do_not_mix():
    p = Prompts([40, 75, 30], 6, 2, 128, seed=17)
    out, lse = p.forward()
    first = p.backward(out, lse)
    for x in (p.q, p.k, p.v, p.dout, out):
        x[:40] = float("nan")
        x[115:145] = float("inf")
    lse[:, :40] = float("nan")
    again = p.backward(out, lse)
    assert all(torch.equal(a[40:115], b[40:115]) for a, b in zip(first, again))


def test_bad_offsets_write_no_gradient():
    p = Prompts([3, 3, 14], 4, 2, 64, pad=0)
    out, lse = p.forward()
    p.offsets = int32([0, 5, 4, 20])
    grads = p.backward(out, lse)
    assert pkg.cp_get_last_status() == pkg.STATUS_CODES["CP_ERR_DOC_OFFSETS"]
    assert all((g == -7).all() for g in grads)


def test_a_captured_backward_follows_its_offsets():
    p = Prompts([100, 60, 40], 8, 2, 64, seed=18, pad=0)
    out, lse = p.forward()
    grads = p.backward(out, lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkg.packed_attn_fwd(p.q, p.k, p.v, p.offsets, out=out, lse=lse)
        pkg.packed_attn_bwd(p.q, p.k, p.v, out, lse, p.dout, p.offsets, dq=grads[0], dk=grads[1],
                            dv=grads[2])
    for c in [[0, 100, 160, 200], [0, 0, 10, 200], [0, 199, 199, 200]] * 2:
        p.offsets.copy_(int32(c))
        for g in grads:
            g.fill_(-7)
        graph.replay()
        want = p.backward(*p.forward())
        assert all(torch.equal(a, b) for a, b in zip(grads, want))


def test_a_wait_that_runs_out_in_the_backward_is_reported():
    p = Prompts([300], 4, 2, 128, seed=19)
    out, lse = p.forward()
    pkg.test_set_wait_fault(True, 200_000_000)
    try:
        p.backward(out, lse)
        assert pkg.cp_get_last_status() == pkg.STATUS_CODES["CP_ERR_TIMEOUT"]
    finally:
        pkg.test_set_wait_fault(False)
    p.check_gradients(out, lse, p.backward(out, lse))


def test_allocated_outputs_are_zero_where_no_sequence_is():
    p = Prompts([20, 9], 4, 2, 64, seed=20, lead=2)
    out, lse = pkg.packed_attn_fwd(p.q, p.k, p.v, p.offsets)
    grads = pkg.packed_attn_bwd(p.q, p.k, p.v, out, lse, p.dout, p.offsets)
    for t in (out, lse.T, *grads):
        assert (t[~torch.tensor(p.there)] == 0).all() and (t[p.ends[0]:p.ends[-1]] != 0).any()
    want = p.backward(*p.forward())
    assert all(torch.equal(a[2:31], b[2:31]) for a, b in zip(grads, want))


@pytest.mark.parametrize("scale", [0.02, 4.0, 12.0])
def test_forward_of_flat_and_peaked_rows(scale):
    """Scores from nothing to thousands: the reference moves, and far tails vanish."""
    p = Prompts([260, 390], 4, 2, 128, seed=3, scale=scale)
    p.check(*p.forward())


def test_scores_that_grow_along_the_keys():
    """Each key tile's largest score is far above the last one's: the guard's redo."""
    p = Prompts([900], 4, 1, 128, seed=4)
    ramp = torch.linspace(0, 60, 900, device=DEV)[:, None, None]
    p.q[:900] = 1.0
    p.k[:900] = (ramp * 0.5).expand(900, 1, 128).to(BF16)
    p.check(*p.forward())


def test_forward_equals_the_ring_attentions():
    """Equal heads and one sequence: P of the same scores against the same references.  The rows'
    sums of up to 512 of them are added in another order, which makes 2 * 512 * 2^-24 of each at
    most: lse differs by that, out by that and so by one step of bf16, 2^-7 of itself."""
    p = Prompts([512], 4, 4, 128, seed=5, pad=0, fused=False)
    out, lse = p.forward()
    want, wantl = pkg.ring_attn_fwd(p.q[None], p.k[None], p.v[None], 1, True)
    assert (lse - wantl[0]).abs().max() <= 2.0 ** -14
    assert ((out.float() - want[0].float()).abs() <= 2.0 ** -7 * want[0].float().abs()).all()


def test_many_sequences():
    """More sequences than the plan's shared memory holds, and many items of a CTA."""
    rng = np.random.default_rng(6)
    lens = rng.integers(0, 9, 5000)
    lens[4321] = 300
    p = Prompts(lens, 4, 2, 64, seed=7)
    p.check(*p.forward())


def test_sequences_do_not_see_one_another():
    """A sequence's rows are the same bits whatever the others hold, infinities and NaN among it."""
    p = Prompts([40, 75, 30], 8, 2, 128, seed=8)
    out, lse = p.forward()
    for x in (p.q, p.k, p.v):
        x[:40] = float("nan")
        x[115:145] = float("inf")
    again, lse2 = p.forward()
    assert torch.equal(out[40:115], again[40:115]) and torch.equal(lse[:, 40:115], lse2[:, 40:115])
    assert torch.isnan(again[:40]).all()


@pytest.mark.parametrize("offsets", [[0, 5, 4, 9], [-1, 3, 9, 9], [0, 3, 9, 21], [2, 1, 9, 9]])
def test_bad_offsets_write_nothing(offsets):
    p = Prompts([3, 3, 14], 4, 2, 64, pad=0)
    p.offsets = int32(offsets)
    out, lse = p.forward()
    assert pkg.cp_get_last_status() == pkg.STATUS_CODES["CP_ERR_DOC_OFFSETS"]
    assert (out == -7).all() and (lse == -7).all()
    p.offsets = int32([0, 3, 6, 20])
    p.check(*p.forward())


def test_a_captured_call_follows_its_offsets():
    p = Prompts([100, 60, 40], 8, 2, 64, seed=9, pad=0)
    cuts = [[0, 100, 160, 200], [0, 0, 10, 200], [0, 199, 199, 200], [0, 1, 2, 3]]
    out, lse = p.forward()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkg.packed_attn_fwd(p.q, p.k, p.v, p.offsets, out=out, lse=lse)
    for c in cuts * 2:
        p.offsets.copy_(int32(c))
        out.fill_(-7), lse.fill_(-7)
        graph.replay()
        want, wantl = p.forward()
        assert torch.equal(out, want) and torch.equal(lse, wantl)


def test_a_wait_that_runs_out_is_reported():
    p = Prompts([300], 4, 2, 128, seed=10)
    pkg.test_set_wait_fault(True, 200_000_000)
    try:
        p.forward()
        assert pkg.cp_get_last_status() == pkg.STATUS_CODES["CP_ERR_TIMEOUT"]
    finally:
        pkg.test_set_wait_fault(False)
    p.check(*p.forward())


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens,Hq,Hk,d", [
    ([1500], 2, 1, 128),             # few key tiles of many queries: cut into parts
    ([900, 40, 7], 14, 2, 64),       # beside tiles that are not
    ([400, 1100], 8, 1, 128),
])
def test_gradients_of_key_tiles_in_parts(lens, Hq, Hk, d, causal):
    """The parts are added up in one order, whichever ends last."""
    p = Prompts(lens, Hq, Hk, d, seed=21)
    out, lse = p.forward(causal)
    grads = p.backward(out, lse, causal)
    p.check_gradients(out, lse, grads, causal)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(grads, p.backward(out, lse, causal)))


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens,Hq,Hk,d", [
    ([3000], 2, 1, 128),             # few items of many keys: cut into parts
    ([2500, 40, 7], 3, 1, 64),       # tiles whose first rows see nothing of a part's keys
    ([1300, 1700], 8, 1, 128),
    ([1200] * 4, 2, 2, 64),
])
def test_forward_of_items_in_parts(lens, Hq, Hk, d, causal):
    """The parts are joined in one order, whichever ends last."""
    p = Prompts(lens, Hq, Hk, d, seed=22, scale=2.0)
    out, lse = p.forward(causal)
    p.check(out, lse, causal)
    for _ in range(3):
        again, lse2 = p.forward(causal)
        assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens,Hq,Hk,d", [
    ([300, 30], 1040, 260, 64),  # 10 streamed tiles, but two slots a key head
    ([200, 100], 16, 4, 128),    # 7
])
def test_gradients_where_no_tile_is_cut(lens, Hq, Hk, d, causal):
    p = Prompts(lens, Hq, Hk, d, seed=23)
    out, lse = p.forward(causal)
    p.check(out, lse, causal)
    p.check_gradients(out, lse, p.backward(out, lse, causal), causal)


PARTS = [
    # lens, Hq, Hk, d, of the forward: items, slots, causal or not
    ([1500] + [9] * 30, 21, 3, 64),     # seven heads; 72 items for 107 slots
    ([3000] + [20] * 25, 12, 4, 64),    # 61 for 80
    ([1600] + [5] * 60, 8, 8, 128),     # 67 for 40
    ([1091] + [13] * 5, 1, 1, 64),      # 10 for 126: parts are as short as they may be
    # of the backward
    ([2560] + [30] * 20, 32, 8, 64),    # 40 items for 64 slots
    ([2000] + [3] * 60, 28, 4, 128),    # seven heads; 76 for 128
    ([773], 2, 1, 128),                 # 7 for 28
]


class Guarded:
    """A workspace of exactly the stated size between two guards."""

    def __init__(self, need):
        self.all = torch.full((need + 3 * 4096,), 0xA5, dtype=torch.uint8, device=DEV)
        self.at = 4096 + -self.all.data_ptr() % 256
        self.need = need
        self.ws = self.all[self.at:self.at + need]

    def kept(self):
        return bool((self.all[:self.at] == 0xA5).all()
                    and (self.all[self.at + self.need:] == 0xA5).all())


def test_parts_take_every_branch_of_the_plan():
    for which in ("fwd", "bwd"):
        reached = set()
        for lens, Hq, Hk, d in PARTS:
            for causal in (True, False):
                slots, items, streamed, chunk, bound = packed_plan.cut(
                    which, lens, sum(lens) + 3, Hq, Hk, causal, torch.cuda.get_device_properties(
                        0).multi_processor_count)
                if chunk and packed_plan.parts(streamed, chunk):
                    reached.add(2 * items < slots)
        assert reached == {True, False}


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens,Hq,Hk,d", PARTS)
def test_parts_stay_in_the_workspace(lens, Hq, Hk, d, causal):
    p = Prompts(lens, Hq, Hk, d, seed=24, pad=3)
    args = (p.T, len(lens), Hq, Hk, d)
    fwd, bwd = (Guarded(f(*args)) for f in (pkg.cp_packed_attn_fwd_workspace_bytes,
                                            pkg.cp_packed_attn_bwd_workspace_bytes))
    out, lse = p.forward(causal, workspace=fwd.ws)
    assert fwd.kept()
    p.check(out, lse, causal)
    grads = p.backward(out, lse, causal, workspace=bwd.ws)
    assert bwd.kept()
    p.check_gradients(out, lse, grads, causal)


def test_parts_as_long_as_the_bound_has_them():
    """So much is streamed for so many items that the bound on the parts' number, not a block's
    share, sets their length."""
    lens, Hq, Hk, d = [10603, 10065, 7897] + [13] * 150, 1, 1, 64
    _, _, streamed, chunk, bound = packed_plan.cut("fwd", lens, sum(lens) + 3, Hq, Hk, False)
    assert bound and packed_plan.parts(streamed, chunk) > 200
    p = Prompts(lens, Hq, Hk, d, seed=25, pad=3)
    fwd = Guarded(pkg.cp_packed_attn_fwd_workspace_bytes(p.T, len(lens), Hq, Hk, d))
    out, lse = p.forward(False, workspace=fwd.ws)
    assert fwd.kept()
    p.check(out, lse, False)
