"""cp_paged_append against the fp64 oracle, on caches whose other slots must
stay as they were.

Tolerances: the norm and rotation in fp32 leave 2^-18 of the row's largest
entry (the derivation stands in test_gpu_norm_rope.py); then one rounding to
bf16, eps / 2 of the value, or to E4M3 after a division by the descale: 2^-4
of the value, at least half of the smallest code, 2^-10, times the descale.
Values are copied: exact in bf16 and one rounding in E4M3.
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


def freqs(rot, theta=10000.0):
    return torch.tensor(theta ** (-np.arange(0, rot, 2) / rot), dtype=torch.float32)


def values(cache, descale):
    if cache.dtype != torch.uint8:
        return _np(cache)
    return _np(cache.cpu().view(torch.float8_e4m3fn).float()) * _np(descale)[:, None]


def setup(B, S, Hq, Hk, d, page, e4m3, seed, head_major=False, held=40):
    g = torch.Generator().manual_seed(seed)
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, held + 1, B)
    most = (held + S + page - 1) // page
    n_pages = B * most + 3
    table = torch.tensor(rng.permutation(n_pages)[:B * most].reshape(B, most), dtype=torch.int32)
    shape = (n_pages, Hk, page, d) if head_major else (n_pages, page, Hk, d)
    caches = []
    for _ in range(2):
        c = torch.randn(shape, generator=g)
        c = (c * 100).to(torch.float8_e4m3fn).view(torch.uint8) if e4m3 else c.to(torch.bfloat16)
        c = c.to(DEV)
        caches.append(c.transpose(1, 2) if head_major else c)
    qkv = (2 * torch.randn((B, S, Hq + 2 * Hk, d), generator=g)).to(torch.bfloat16).to(DEV)
    q, k, v = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hk], qkv[:, :, Hq + Hk:]
    w = [(1 + 0.2 * torch.randn(d, generator=g)).to(DEV) for _ in range(2)]
    desc = [(0.01 + 0.02 * torch.rand(Hk, generator=g)).to(DEV) if e4m3 else None for _ in range(2)]
    return q, k, v, caches, table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV), w, desc


CASES = [
    # B, S, Hq, Hk, d, page, e4m3, rot, interleaved, head-major pages, ragged
    (1, 1, 1, 1, 128, 16, False, 128, False, False, False),
    (5, 1, 8, 2, 128, 16, False, 128, False, False, True),
    (5, 1, 8, 2, 128, 16, True, 128, False, True, True),
    (3, 7, 6, 3, 64, 5, False, 32, True, False, True),
    (3, 7, 6, 3, 64, 1, True, 64, False, False, True),
    (2, 50, 4, 4, 128, 48, True, 96, True, False, False),
    (2, 50, 0, 1, 128, 64, False, 0, False, True, True),
    (2, 700, 16, 8, 128, 32, True, 128, False, False, True),   # the wide units
    (2, 700, 16, 8, 64, 128, False, 64, False, False, True),
]


@pytest.mark.parametrize("B,S,Hq,Hk,d,page,e4m3,rot,il,hm,ragged", CASES)
def test_append(B, S, Hq, Hk, d, page, e4m3, rot, il, hm, ragged):
    q, k, v, (kc, vc), table, lens, (qw, kw), (kd, vd) = setup(B, S, Hq, Hk, d, page, e4m3,
                                                               S + Hq + page, hm)
    new = torch.tensor([(S * (i + 1)) // B if ragged else S for i in range(B)], dtype=torch.int32,
                       device=DEV)
    if B > 3:
        new[1] = 0
    k0, v0 = kc.clone(), vc.clone()
    f = freqs(rot) if rot else None
    q_out = None if Hq == 0 else torch.full((B, S, Hq, d), 9.0, dtype=torch.bfloat16, device=DEV)
    got = pkg.paged_append(q if Hq else None, k, v, kc, vc, table, lens, new if ragged else None,
                           qw, kw, None if f is None else f.to(DEV), 1e-6, il, kd, vd, q_out)
    assert pkg.cp_get_last_status() == 0
    at = lens.cpu().numpy()[:, None] + np.arange(S)
    fn = None if f is None else f.numpy()
    kk, _ = serving.norm_rope(_np(k), _np(kw), 1e-6, fn, at, il)
    half = torch.finfo(torch.bfloat16).eps / 2
    touched = torch.zeros(kc.shape[:2], dtype=torch.bool)
    t, n = table.cpu(), new.cpu()
    for cache, want, desc, inner in ((kc, kk, kd, 2.0 ** -18), (vc, _np(v), vd, 0.0)):
        val = values(cache, desc)
        for b in range(B):
            for s in range(int(n[b])):
                p = int(at[b, s])
                pg, sl = int(t[b, p // page]), p % page
                touched[pg, sl] = True
                w = want[b, s]
                tol = inner * np.abs(w).max(-1, keepdims=True)
                if e4m3:
                    dn = _np(desc)[:, None]
                    w = np.clip(w, -448 * dn, 448 * dn)
                    tol = tol + np.maximum(2.0 ** -4 * np.abs(w), 2.0 ** -10 * dn) * (1 + 2.0 ** -20)
                else:
                    tol = tol + (half * np.abs(w) if inner else 0.0)
                assert np.all(np.abs(val[pg, sl] - w) <= tol)
    assert torch.equal(kc.cpu()[~touched], k0.cpu()[~touched])
    assert torch.equal(vc.cpu()[~touched], v0.cpu()[~touched])
    if Hq:
        assert got is q_out
        qq, _ = serving.norm_rope(_np(q), _np(qw), 1e-6, fn, at, il)
        for b in range(B):
            m = int(n[b])
            tol = half * np.abs(qq[b, :m]) + 2.0 ** -18 * np.abs(qq[b, :m]).max(-1, keepdims=True)
            assert np.all(np.abs(_np(got[b, :m]) - qq[b, :m]) <= tol)
            assert (got[b, m:] == 9).all()


def test_equals_the_norm_and_rotation_call():
    q, k, v, (kc, vc), table, lens, (qw, kw), _ = setup(2, 6, 4, 2, 128, 16, False, 1)
    f = freqs(128).to(DEV)
    pos = (lens[:, None] + torch.arange(6, device=DEV, dtype=torch.int32)).contiguous()
    a, b = pkg.qk_norm_rope(q, k, qw, kw, f, pos)
    got = pkg.paged_append(q, k, v, kc, vc, table, lens, None, qw, kw, f)
    assert torch.equal(got, a)
    pg, sl = table.long().gather(1, pos.long() // 16), pos.long() % 16
    assert torch.equal(kc[pg, sl], b) and torch.equal(vc[pg, sl], v)


def test_codes_saturate_and_keep_nan():
    q, k, v, (kc, vc), table, lens, (qw, kw), (kd, vd) = setup(1, 2, 1, 1, 64, 4, True, 2)
    v = v.contiguous()
    v[0, 0, 0, :4] = torch.tensor([1e30, -1e30, float("inf"), float("nan")])
    pkg.paged_append(None, k, v, kc, vc, table, lens, None, None, kw, None, k_descale=kd,
                     v_descale=vd)
    p = int(lens[0])
    row = vc[table[0, p // 4].long(), p % 4, 0].cpu().view(torch.float8_e4m3fn).float()
    assert row[:3].tolist() == [448.0, -448.0, 448.0] and row[3].isnan()


def test_tokens_without_a_place_are_left_out_and_reported():
    """Bad pages and lengths: the kernel's own bounds checks skip the write."""
    q, k, v, (kc, vc), table, lens, (qw, kw), _ = setup(4, 3, 4, 2, 64, 8, False, 4, held=20)
    lens[:] = torch.tensor([4, 7, 1, 2], dtype=torch.int32)
    n_pages, most = kc.shape[0], table.shape[1]
    table[0, 0] = -1
    table[1, 0], table[1, 1] = n_pages, 2        # its first new token has no page, the next do
    lens[2] = most * 8 - 1                       # one fits, two are behind the table
    lens[3] = -1                                 # no position at all
    k0, v0 = kc.clone(), vc.clone()
    f = freqs(64).to(DEV)
    pkg.paged_append(q, k, v, kc, vc, table, lens, None, qw, kw, f)
    assert pkg.cp_get_last_status() == pkg.STATUS_CODES["CP_ERR_CACHE"]
    assert pkg.cp_get_last_status() == 0
    touched = torch.zeros(kc.shape[:2], dtype=torch.bool)
    touched[2, 0:2] = True
    touched[int(table[2, most - 1]), 7] = True
    for c, c0 in ((kc, k0), (vc, v0)):
        assert torch.equal(c.cpu()[~touched], c0.cpu()[~touched])
    assert torch.equal(vc[2, 0:2], v[1, 1:]) and torch.equal(vc[int(table[2, most - 1]), 7], v[2, 0])
    new = torch.tensor([4, 1, -2, 0], dtype=torch.int32, device=DEV)   # 4 > S, -2 < 0
    lens[:] = 0
    table[:] = torch.arange(4, dtype=torch.int32, device=DEV)[:, None]
    kc.copy_(k0), vc.copy_(v0)
    pkg.paged_append(q, k, v, kc, vc, table, lens, new, qw, kw, f)
    assert pkg.cp_get_last_status() == pkg.STATUS_CODES["CP_ERR_CACHE"]
    assert torch.equal(vc[0, :3], v[0]) and torch.equal(vc[1, :1], v[1, :1])
    assert torch.equal(vc[1, 1:], v0[1, 1:]) and torch.equal(vc[2:], v0[2:])


def test_graph_replays_follow_the_lengths_on_the_device():
    q, k, v, (kc, vc), table, lens, (qw, kw), _ = setup(3, 1, 4, 2, 128, 16, False, 6)
    f = freqs(128).to(DEV)
    q_out = torch.empty(q.shape, dtype=q.dtype, device=DEV)
    args = (q, k, v, kc, vc, table, lens, None, qw, kw, f)
    pkg.paged_append(*args, q_out=q_out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkg.paged_append(*args, q_out=q_out)
        lens += 1
    start = lens.clone()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(lens, start + 3)
    for i in range(3):
        p = (start + i).long()
        assert torch.equal(vc[table.long().gather(1, (p // 16)[:, None])[:, 0], p % 16], v[:, 0])


def test_binding_refusals():
    q, k, v, (kc, vc), table, lens, (qw, kw), _ = setup(2, 3, 4, 2, 64, 8, False, 7)
    f = freqs(64).to(DEV)
    ok = (q, k, v, kc, vc, table, lens, None, qw, kw, f)
    for at, bad, error in [(1, k.float(), TypeError), (3, kc.float(), TypeError),
                           (4, vc[:-1], ValueError), (5, table[:1], ValueError),
                           (5, table.long(), TypeError), (6, lens[:1], ValueError),
                           (6, lens.cpu(), ValueError), (2, v[:, :2], ValueError),
                           (0, q[:1], ValueError)]:
        args = list(ok)
        args[at] = bad
        with pytest.raises(error):
            pkg.paged_append(*args)
    with pytest.raises(ValueError):
        pkg.paged_append(*ok, k_descale=qw[:2])
    with pytest.raises(TypeError):                # E4M3 codes need their descales
        pkg.paged_append(q, k, v, kc.view(torch.uint8)[..., :64].contiguous(),
                         vc.view(torch.uint8)[..., :64].contiguous(), table, lens)


def test_a_cache_of_float8_tensors_is_that_of_its_codes():
    q, k, v, (kc, vc), table, lens, (qw, kw), (kd, vd) = setup(2, 3, 4, 2, 64, 8, True, 8)
    f = freqs(64).to(DEV)
    k8, v8 = kc.clone().view(torch.float8_e4m3fn), vc.clone().view(torch.float8_e4m3fn)
    a = pkg.paged_append(q, k, v, kc, vc, table, lens, None, qw, kw, f, k_descale=kd, v_descale=vd)
    pkg.paged_append(q, k, v, k8, v8, table, lens, None, qw, kw, f, k_descale=kd, v_descale=vd)
    assert torch.equal(k8.view(torch.uint8), kc) and torch.equal(v8.view(torch.uint8), vc)
    want = pkg.paged_attn_decode(a, kc, vc, table, lens + 3, k_descale=kd, v_descale=vd)
    got = pkg.paged_attn_decode(a, k8, v8, table, lens + 3, k_descale=kd, v_descale=vd)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    with pytest.raises(TypeError):
        pkg.paged_attn_decode(a, k8, vc, table, lens + 3, k_descale=kd, v_descale=vd)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("B,S", [(1600, 1), (4096, 1), (40, 100), (40, 700)])
def test_tokens_left_out_do_not_disturb_the_others(B, S, e4m3):
    """Thousands of tokens, several units a warp, a third of them on pages outside the cache, in
    runs and alone: every other slot and every query row is, bit for bit, that of a call whose
    table is sound."""
    q, k, v, (kc, vc), table, lens, (qw, kw), (kd, vd) = setup(B, S, 4, 4, 128, 8, e4m3, B, held=30)
    f = freqs(128).to(DEV)
    k0, v0, bad = kc.clone(), vc.clone(), table.clone()
    out = torch.rand(table.shape, generator=torch.Generator().manual_seed(S)) < 1 / 3
    out[::7] = True                                 # whole rows among them
    out = out.to(DEV)
    bad[out] = torch.where(torch.arange(B, device=DEV)[:, None] % 2 == 0, -1,
                           kc.shape[0]).expand_as(bad)[out].to(torch.int32)
    run = lambda t, a, b: pkg.paged_append(q, k, v, a, b, t, lens, None, qw, kw, f,  # noqa: E731
                                           k_descale=kd, v_descale=vd)
    want = run(table, kc, vc)
    assert pkg.cp_get_last_status() == 0
    lost = torch.zeros(kc.shape[0], dtype=torch.bool, device=DEV)
    lost[table.long()[out]] = True
    for _ in range(5):
        ka, va = k0.clone(), v0.clone()
        got = run(bad, ka, va)
        assert pkg.cp_get_last_status() == pkg.STATUS_CODES["CP_ERR_CACHE"]
        assert torch.equal(got, want)
        for a, whole, before in ((ka, kc, k0), (va, vc, v0)):
            assert torch.equal(a[~lost], whole[~lost]) and torch.equal(a[lost], before[lost])


@pytest.mark.parametrize("B,S", [(64, 1), (300, 2)])
@pytest.mark.parametrize("bad", [-2, 7])
def test_a_new_length_out_of_range_is_reported_for_any_row(B, S, bad):
    """The calls whose padding is walked: single tokens, and more rows than one scan takes."""
    q, k, v, (kc, vc), table, lens, (qw, kw), _ = setup(B, S, 32, 8, 128, 16, False, B)
    new = torch.full((B,), S, dtype=torch.int32, device=DEV)
    pkg.paged_append(q, k, v, kc, vc, table, lens, new, qw, kw)
    assert pkg.cp_get_last_status() == 0
    for row in (0, 1, B // 2, B - 1):
        new[:] = S
        new[row] = bad
        ka, va = kc.clone(), vc.clone()
        pkg.paged_append(q, k, v, ka, va, table, lens, new, qw, kw)
        assert pkg.cp_get_last_status() == pkg.STATUS_CODES["CP_ERR_CACHE"], row
        assert torch.equal(ka, kc) and torch.equal(va, vc)     # the nearer of 0 and S
