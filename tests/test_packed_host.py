"""Attention over packed prompts on the CPU: the oracle pinned by the ring attention's and by
differences, and what the calls refuse before any launch."""
import ctypes
import os

import numpy as np
import pytest
import torch

import context_ring_attention_fwd_gb300 as pkg
from oracle import packed, ref
import packed_plan

V = ctypes.c_void_p
FAKE, ODD = V(0x10000), V(0x10002)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(pkg.LIB_PATH):
        from context_ring_attention_fwd_gb300 import _build
        _build.build()
    return pkg.lib()


def rows(seed, T, Hq, Hk, d):
    rng = np.random.default_rng(seed)
    return [rng.standard_normal((T, H, d)) for H in (Hq, Hk, Hk)]


@pytest.mark.parametrize("causal", [True, False])
def test_the_oracle_is_the_ring_attentions_on_documents(causal):
    """Equal heads, no empty sequence, no padding: packed prompts are documents."""
    q, k, v = rows(0, 37, 3, 3, 16)
    offsets = [0, 1, 12, 37]
    out, lse, _, _ = packed.attention(q, k, v, offsets, causal)
    want, wantl = ref.attention(q[None], k[None], v[None], causal, offsets)
    assert np.abs(out - want[0]).max() < 1e-12 and np.abs(lse - wantl[0]).max() < 1e-12
    g = np.random.default_rng(1).standard_normal(q.shape)
    got, _, _ = packed.attention_bwd(q, k, v, out, lse, g, offsets, causal)
    for a, b in zip(got, ref.attention_bwd(q[None], k[None], v[None], g[None], causal, offsets)):
        assert np.abs(a - b[0]).max() < 1e-12


def test_grouped_heads_are_repeated_heads():
    """Hk key heads read by G heads each equal Hk G key heads that are copies; a shared head's
    gradient is the sum of its copies'."""
    q, k, v = rows(2, 29, 6, 2, 8)
    offsets = [3, 3, 17, 25]  # rows of no sequence at both ends, an empty sequence
    g = np.random.default_rng(3).standard_normal(q.shape)
    out, lse, _, _ = packed.attention(q, k, v, offsets, True)
    out3, lse3, _, _ = packed.attention(q, k.repeat(3, 1), v.repeat(3, 1), offsets, True)
    assert np.array_equal(np.isnan(out), np.isnan(out3)) and np.nanmax(np.abs(out - out3)) < 1e-14
    assert np.isnan(out[:3]).all() and np.isnan(out[25:]).all() and np.isnan(lse[:, :3]).all()
    got, _, _ = packed.attention_bwd(q, k, v, out, lse, g, offsets, True)
    many, _, _ = packed.attention_bwd(q, k.repeat(3, 1), v.repeat(3, 1), out, lse, g, offsets, True)
    assert np.nanmax(np.abs(got[0] - many[0])) < 1e-12
    for a, b in zip(got[1:], many[1:]):
        assert np.nanmax(np.abs(a - b.reshape(29, 2, 3, 8).sum(2))) < 1e-12


@pytest.mark.parametrize("causal", [True, False])
def test_the_gradients_are_differences(causal):
    q, k, v = rows(4, 23, 4, 2, 8)
    offsets = [0, 9, 9, 21]
    rng = np.random.default_rng(5)
    g = rng.standard_normal(q.shape)
    out, lse, _, _ = packed.attention(q, k, v, offsets, causal)
    grads, _, _ = packed.attention_bwd(q, k, v, out, lse, g, offsets, causal)
    loss = lambda *x: np.nansum(packed.attention(*x, offsets, causal)[0] * g)  # noqa: E731
    for i, grad in enumerate(grads):
        way = rng.standard_normal(grad.shape)
        x = [q, k, v]
        up, down = list(x), list(x)
        up[i], down[i] = x[i] + 1e-5 * way, x[i] - 1e-5 * way
        slope = (loss(*up) - loss(*down)) / 2e-5
        assert abs(slope - np.nansum(grad * way)) < 1e-7 * max(1, abs(slope))


def strides(*v):
    return (ctypes.c_int64 * len(v))(*v)


def fwd_args(**kw):
    a = dict(q=FAKE, qs=None, k=FAKE, ks=None, v=FAKE, vs=None, offsets=FAKE, out=FAKE, lse=FAKE,
             T=100, n=3, Hq=8, Hk=2, d=64, causal=1, ws=FAKE, bytes=1 << 40, stream=None)
    a.update(kw)
    return list(a.values())


BAD = [
    (dict(q=None), -1), (dict(k=None), -1), (dict(v=None), -1), (dict(offsets=None), -1),
    (dict(ws=None), -1),
    (dict(T=0), -2), (dict(n=0), -2), (dict(n=(1 << 20) + 1), -2), (dict(Hq=0), -2),
    (dict(Hk=0), -2), (dict(Hq=7), -2), (dict(causal=2), -2), (dict(T=1 << 28), -2),
    (dict(T=1 << 26, Hk=16, Hq=16), -2),
    (dict(d=96), -3), (dict(d=32), -3), (dict(Hq=258), -3),
    (dict(q=ODD), -4), (dict(k=ODD), -4), (dict(v=ODD), -4), (dict(offsets=ODD), -4),
    (dict(ws=V(0x10080)), -4), (dict(qs=strides(512, 60)), -4), (dict(qs=strides(8 * 64 + 8, 64)), -4),
    (dict(ks=strides(64, 64)), -4), (dict(vs=strides(0, 64)), -4), (dict(vs=strides(128, 0)), -4),
    (dict(ks=strides(-128, 64)), -4), (dict(qs=strides(1 << 40, 64)), -4),
    (dict(bytes=100), -6),
]


@pytest.mark.parametrize("change,want", BAD + [(dict(out=None), -1), (dict(lse=None), -1),
                                               (dict(out=ODD), -4), (dict(lse=ODD), -4)])
def test_forward_refuses_before_any_launch(lib, change, want):
    assert lib.cp_packed_attn_fwd(*fwd_args(**change)) == want


def bwd_args(**kw):
    a = dict(q=FAKE, qs=None, k=FAKE, ks=None, v=FAKE, vs=None, out=FAKE, lse=FAKE, dout=FAKE,
             offsets=FAKE, dq=FAKE, dqs=None, dk=FAKE, dks=None, dv=FAKE, dvs=None, T=100, n=3,
             Hq=8, Hk=2, d=64, causal=1, ws=FAKE, bytes=1 << 40, stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("change,want", BAD + [
    *((({x: None}), -1) for x in ("out", "lse", "dout", "dq", "dk", "dv")),
    *((({x: ODD}), -4) for x in ("out", "lse", "dout", "dq", "dk", "dv")),
    (dict(dqs=strides(64, 64)), -4), (dict(dks=strides(128, 8)), -4), (dict(dvs=strides(0, 0)), -4),
])
def test_backward_refuses_before_any_launch(lib, change, want):
    assert lib.cp_packed_attn_bwd(*bwd_args(**change)) == want


def test_views_of_a_projection_pass_the_checks(lib):
    """What fails next is the workspace's size."""
    for qs, ks in ((strides(12 * 64, 64), strides(12 * 64, 64)), (strides(8 * 128, 128), None)):
        assert lib.cp_packed_attn_fwd(*fwd_args(qs=qs, ks=ks, vs=ks, bytes=100)) == -6


def test_workspace_sizes():
    for f in (pkg.cp_packed_attn_fwd_workspace_bytes, pkg.cp_packed_attn_bwd_workspace_bytes):
        assert 0 < f(1, 1, 1, 1, 64) < f(1000, 5, 32, 8, 128) < f(100000, 5, 32, 8, 128)
        for bad in [(0, 1, 1, 1, 64), (1, 0, 1, 1, 64), (1, 1, 3, 2, 64), (1, 1, 2, 2, 80),
                    (1, 1, 258, 2, 64)]:
            assert f(*bad) == -1


def test_no_workspace_for_parts_where_nothing_is_cut():
    """Sums of parts take 128 KB a slot and key head at d = 128; what else there is (D, lists) is
    below 8 bytes a row and head and 1 KB."""
    bwd = pkg.cp_packed_attn_bwd_workspace_bytes
    for T, n, Hq, Hk in [(200, 6, 16, 4),      # 7 streamed tiles: they stay whole
                         (1000, 3, 1024, 1024),  # a slot for each key head: too few for a cut
                         (2000, 1, 600, 300)]:  # two
        assert bwd(T, n, Hq, Hk, 128) <= 8 * T * Hq + 1024
    assert bwd(2000, 1, 2, 1, 128) > 1 << 20   # where tiles are cut there is
    # the forward's, with two slots a key head
    assert pkg.cp_packed_attn_fwd_workspace_bytes(1200, 1, 170, 170, 128) <= 1 << 16


@pytest.mark.parametrize("which", ["fwd", "bwd"])
def test_the_plan_cuts_no_more_parts_than_there_are_slots(which):
    """By the plan's own rule, over random calls.  (The kernel sums its estimate of the streamed
    tiles in fp32: at most 2^10 terms to a thread and 2^5 + 5 additions behind them, each off by
    2^-24, and a term by a few: below 2^-13, where the rule adds 2^-10.)"""
    rng = np.random.default_rng(30)
    cut_calls = fullest = 0
    reached = set()
    for _ in range(4000):
        Hk = int(rng.choice([1, 2, 3, 4, 5, 8, 16, 24, 100]))
        Hq = Hk * int(rng.choice([1, 2, 3, 4, 7, 8, 16, 64, 128]))
        lens = np.concatenate([rng.integers(0, int(10 ** rng.uniform(1, 4.5)), rng.integers(1, 6)),
                               rng.integers(0, 40, rng.choice([0, 0, 5, 60, 400]))])
        T = int(lens.sum()) + int(rng.choice([0, 5, 3000]))
        if T == 0:
            continue
        causal = bool(rng.integers(2))
        slots, items, streamed, chunk, bound = packed_plan.cut(which, lens, T, Hq, Hk, causal)
        if chunk is None:
            continue
        n = packed_plan.parts(streamed, chunk)
        assert n <= slots, (lens, T, Hq, Hk, causal)
        if n:
            cut_calls += 1
            fullest = max(fullest, n / slots)
            reached.add((2 * items < slots, bound))
    assert cut_calls > 150 and fullest > 0.6
    # few items for the slots and many, the share and the bound (a backward of many items has
    # a share above its bound: 0.6 / 152 of what is streamed, the bound 2 / 512)
    want = {(True, True), (True, False), (False, False)} | ({(False, True)} if which == "fwd" else set())
    assert want <= reached


def test_host_tensors_are_refused():
    q = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        pkg.packed_attn_fwd(q, q, q, torch.tensor([0, 4], dtype=torch.int32))
