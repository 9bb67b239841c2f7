"""cp_qk_norm_rope and cp_qk_norm_rope_bwd against the fp64 oracle.

Tolerances.  The kernels hold everything in fp32 and round once at the store.
In units of 2^-24, an element's relative error before that is at most about:
the mean square 13 (a lane's chain of 8 + 5 additions), halved by the root,
7; rsqrt (2 ulp) 4; two products 2; the angle (rounded to 2^-25 half turns)
and its sine and cosine 8; the rotation 3: below 32 = 2^-19, relative to the
pair's magnitude, which the row's largest entry bounds up to sqrt 2, so
2^-18 of that.  The backward's dx adds the mean of g w u (13 + 4) and a
difference: 2^-17 of the magnitudes that enter it.  A rounding to the output
type is eps / 2 of the value.  The weights' gradients sum n rows: a lane's
chain, then fixed trees: (rows / 32 + 32) 2^-24 of the sum of |g u|, on top of
the 2^-18 of each term.
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


def make(B, S, Hq, Hk, d, dtype, seed, fused=False):
    g = torch.Generator().manual_seed(seed)
    qkv = (2 * torch.randn((B, S, Hq + 2 * Hk, d), generator=g)).to(dtype).to(DEV)
    q, k = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hk]
    if not fused:
        q, k = q.contiguous(), k.contiguous()
    w = [(1 + 0.2 * torch.randn(d, generator=g)).to(DEV) for _ in range(2)]
    return q, k, w[0], w[1], g


def close(got, want, scale, dtype):
    err = np.abs(_np(got) - want)
    tol = torch.finfo(dtype).eps / 2 * np.abs(want) + scale
    assert np.all(err <= tol), (err - tol).max()


def check_forward(y, x, w, eps, f, pos, il):
    want, _ = serving.norm_rope(_np(x), None if w is None else _np(w), eps,
                                None if f is None else f.cpu().numpy(), pos, il)
    close(y, want, 2.0 ** -18 * np.abs(want).max(-1, keepdims=True), x.dtype)


CASES = [
    # B, S, Hq, Hk, d, dtype, rot, interleaved, fused
    (1, 1, 1, 1, 128, torch.bfloat16, 128, False, False),
    (1, 1, 3, 1, 64, torch.bfloat16, 64, True, True),
    (2, 5, 7, 3, 64, torch.bfloat16, 32, False, True),
    (2, 5, 7, 3, 128, torch.bfloat16, 16, True, False),
    (1, 33, 32, 8, 128, torch.bfloat16, 128, False, True),
    (3, 7, 5, 5, 64, torch.float32, 64, False, True),
    (1, 9, 17, 2, 128, torch.float32, 96, True, True),
    (1, 4, 2, 2, 128, torch.float32, 128, False, False),
    (1, 700, 24, 8, 128, torch.bfloat16, 128, False, True),   # the wide units
    (1, 700, 24, 8, 64, torch.float32, 48, True, False),
    (2, 2500, 8, 8, 64, torch.bfloat16, 64, False, False),
    (1, 3, 4, 4, 128, torch.bfloat16, 0, False, False),        # no rotation
]


@pytest.mark.parametrize("B,S,Hq,Hk,d,dtype,rot,il,fused", CASES)
@pytest.mark.parametrize("far", [False, True])
def test_forward_and_backward(B, S, Hq, Hk, d, dtype, rot, il, fused, far):
    q, k, qw, kw, g = make(B, S, Hq, Hk, d, dtype, B * S + Hq, fused)
    f = freqs(rot) if rot else None
    fd = None if f is None else f.to(DEV)
    pos = None
    if far:   # anywhere an int32 reaches, negative ones too
        pos = torch.randint(-2 ** 31, 2 ** 31 - 1, (B, S), generator=g, dtype=torch.int64)
        pos = pos.to(torch.int32).to(DEV)
    at = np.tile(np.arange(S), (B, 1)) if pos is None else pos.cpu().numpy()
    eps = 1e-5
    before = q.clone(), k.clone()
    qo, ko = pkg.qk_norm_rope(q, k, qw, kw, fd, pos, eps, il)
    for y, x, w in ((qo, q, qw), (ko, k, kw)):
        check_forward(y, x, w, eps, f, at, il)
    dqo, dko = (torch.randn(t.shape, generator=g).to(dtype).to(DEV) for t in (qo, ko))
    dq, dk, dqw, dkw = pkg.qk_norm_rope_bwd(dqo, dko, q, k, qw, kw, fd, pos, eps, il)
    assert torch.equal(q, before[0]) and torch.equal(k, before[1])
    for dx, dw, dy, x, w in ((dq, dqw, dqo, q, qw), (dk, dkw, dko, k, kw)):
        fn = None if f is None else f.numpy()
        want, wantw = serving.norm_rope_bwd(_np(dy), _np(x), _np(w), eps, fn, at, il)
        gr = _np(dy) if fn is None else serving.rotate(
            _np(dy), -serving.angles(at, fn)[:, :, None], il)
        _, r = serving.norm_rope(_np(x), _np(w), eps, None, at)
        u, gw = _np(x) * r, gr * _np(w)
        top = lambda z: np.abs(z).max(-1, keepdims=True)  # noqa: E731
        mag = r * (top(gw) + top(u) * np.abs(gw * u).mean(-1, keepdims=True))
        close(dx, want, 2.0 ** -17 * mag, dtype)
        rows = B * S * x.shape[2]
        pair = np.abs(u).sum((0, 1, 2)) * top(gr).max()
        tol = (2.0 ** -18 + (rows / 32 + 32) * 2.0 ** -24) * pair
        assert np.all(np.abs(_np(dw) - wantw) <= tol)


def test_gradient_is_the_forward_difference():
    B, S, H, d = 1, 3, 2, 64
    q, k, qw, kw, g = make(B, S, H, H, d, torch.float32, 5)
    f = freqs(32).to(DEV)
    dqo, dko = (torch.randn((B, S, H, d), generator=g).to(DEV) for _ in range(2))
    dq, dk, dqw, dkw = pkg.qk_norm_rope_bwd(dqo, dko, q, k, qw, kw, f)

    def value(q_, k_, qw_, kw_):
        a, b = pkg.qk_norm_rope(q_, k_, qw_, kw_, f)
        return ((a.double() * dqo.double()).sum() + (b.double() * dko.double()).sum()).item()

    # Along a direction v a central difference of step h is off by h^2 times third derivatives
    # (of size |v|^3) and by the outputs' roundings over h.
    h = 2.0 ** -6
    args, grads = [q, k, qw, kw], [dq, dk, dqw, dkw]
    for i in range(4):
        v = torch.randn(args[i].shape, generator=g).to(DEV)
        v /= v.norm()
        hi, lo = ([a + s * h * v if j == i else a for j, a in enumerate(args)] for s in (1, -1))
        step = ((hi[i] - lo[i]).double() * v.double()).sum().item()
        diff = (value(*hi) - value(*lo)) / step
        want = (grads[i].double() * v.double()).sum().item()
        size = sum(t.double().norm().item() for t in (dqo, dko))
        assert abs(diff - want) <= h * h * size + 2.0 ** -20 * size / h


def test_parts_switched_off_in_place_and_queries_alone():
    q, k, qw, kw, g = make(2, 9, 6, 2, 128, torch.bfloat16, 11)
    f = freqs(128)
    at = np.tile(np.arange(9), (2, 1))
    qo, ko = pkg.qk_norm_rope(q, k, None, kw, f.to(DEV))          # q rotated only
    check_forward(qo, q, None, 1e-6, f, at, False)
    check_forward(ko, k, kw, 1e-6, f, at, False)
    only, none = pkg.qk_norm_rope(q, None, qw, None, f.to(DEV))
    both, _ = pkg.qk_norm_rope(q, k, qw, kw, f.to(DEV))
    assert none is None and torch.equal(only, both)
    dq, dk, dqw, dkw = pkg.qk_norm_rope_bwd(qo, ko, q, k, None, kw, f.to(DEV))
    assert dqw is None
    close(dq, serving.norm_rope_bwd(_np(qo), _np(q), None, 0, f.numpy(), at)[0],
          2.0 ** -18 * np.abs(_np(qo)).max(-1, keepdims=True), torch.bfloat16)
    same = pkg.qk_norm_rope_bwd(qo, None, q, None, None, None, f.to(DEV))
    assert torch.equal(same[0], dq) and same[1] is None
    here = q.clone()
    pkg.cp_qk_norm_rope(here, None, qw, None, f.to(DEV), None, here, None)
    assert torch.equal(here, both)
    copy, _ = pkg.qk_norm_rope(q, None)                           # neither: a copy
    assert torch.equal(copy, q)


def test_rows_of_zeros_of_huge_values_and_of_nan():
    q, k, qw, kw, g = make(1, 4, 2, 1, 64, torch.bfloat16, 12)
    q[0, 0] = 0
    q[0, 1] = 2.0 ** 60            # its squares fit, 2^120 times 64 entries
    q[0, 2, 0, 5] = float("nan")
    f = freqs(64).to(DEV)
    qo, ko = pkg.qk_norm_rope(q, k, qw, kw, f)
    assert torch.equal(qo[0, 0], torch.zeros_like(qo[0, 0]))
    check_forward(qo[:, 1:2], q[:, 1:2], qw, 1e-6, freqs(64), np.array([[1]]), False)
    assert qo[0, 2, 0].isnan().all() and not qo[0, 2, 1].isnan().any()
    assert not qo[0, 3].isnan().any() and not ko.isnan().any()


def test_broadcast_inputs_and_views_of_one_gradient():
    g = torch.Generator().manual_seed(3)
    B, S, Hq, Hk, d = 2, 6, 4, 2, 64
    one = torch.randn((1, 1, 1, d), generator=g).to(torch.bfloat16).to(DEV)
    q = one.expand(B, S, Hq, d)
    k = one.expand(B, S, Hk, d)
    w = torch.ones(d, device=DEV)
    f = freqs(64).to(DEV)
    got = pkg.qk_norm_rope(q, k, w, w, f)
    want = pkg.qk_norm_rope(q.contiguous(), k.contiguous(), w, w, f)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    dqo, dko = (torch.randn(t.shape, generator=g).to(torch.bfloat16).to(DEV) for t in want)
    plain = pkg.qk_norm_rope_bwd(dqo, dko, q, k, w, w, f)
    whole = torch.full((B, S, Hq + 2 * Hk, d), 7.0, dtype=torch.bfloat16, device=DEV)
    dw = torch.empty((2, d), device=DEV)
    pkg.cp_qk_norm_rope_bwd(dqo, dko, q, k, w, w, f, None, whole[:, :, :Hq],
                            whole[:, :, Hq:Hq + Hk], dw[0], dw[1])
    assert torch.equal(whole[:, :, :Hq], plain[0])
    assert torch.equal(whole[:, :, Hq:Hq + Hk], plain[1])
    assert (whole[:, :, Hq + Hk:] == 7).all()
    assert torch.equal(dw[0], plain[2]) and torch.equal(dw[1], plain[3])
    with pytest.raises(pkg.CpError) as e:
        pkg.cp_qk_norm_rope_bwd(dqo, dko, q, k, w, w, f, None, torch.empty_like(dqo)[:, :, :1]
                                .expand(B, S, Hq, d), whole[:, :, Hq:Hq + Hk], None, None)
    assert e.value.name == "CP_ERR_SHAPE"


def test_runs_are_equal_on_other_streams_and_in_replayed_graphs():
    q, k, qw, kw, g = make(1, 900, 16, 4, 128, torch.bfloat16, 21, True)
    f = freqs(128).to(DEV)
    qo, ko = pkg.qk_norm_rope(q, k, qw, kw, f)
    want = pkg.qk_norm_rope_bwd(qo, ko, q, k, qw, kw, f)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = pkg.qk_norm_rope_bwd(qo, ko, q, k, qw, kw, f)
    given = pkg.qk_norm_rope_bwd(qo, ko, q, k, qw, kw, f, stream=side)
    side.synchronize()
    for a in (again, given):
        assert all(torch.equal(x, y) for x, y in zip(a, want))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        a, b = pkg.qk_norm_rope(q, k, qw, kw, f)
        caught = pkg.qk_norm_rope_bwd(a, b, q, k, qw, kw, f)
    for t in caught:
        t.zero_()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(caught, want))


def test_binding_refusals():
    q, k, qw, kw, g = make(1, 4, 4, 2, 64, torch.bfloat16, 31)
    f = freqs(64).to(DEV)
    with pytest.raises(TypeError):
        pkg.qk_norm_rope(q.half(), k.half(), qw, kw, f)
    with pytest.raises(TypeError):
        pkg.qk_norm_rope(q, k.float(), qw, kw, f)
    with pytest.raises(TypeError):
        pkg.qk_norm_rope(q, k, qw.bfloat16(), kw, f)
    with pytest.raises(ValueError):
        pkg.qk_norm_rope(q, k, qw[:32], kw, f)
    with pytest.raises(ValueError):
        pkg.qk_norm_rope(q, k, qw, kw, f.cpu())
    with pytest.raises(ValueError):
        pkg.qk_norm_rope(q, k, qw, kw, f, torch.zeros(4, dtype=torch.int32, device=DEV))
    with pytest.raises(ValueError):
        pkg.qk_norm_rope(q, k[:, :3], qw, kw, f)
    with pytest.raises(ValueError):
        pkg.qk_norm_rope(q.transpose(2, 3), k, qw, kw, f)
    with pytest.raises(pkg.CpError):
        pkg.qk_norm_rope(q, k, qw, kw, f[:4])      # rot_dim 8


@pytest.mark.parametrize("il", [False, True])
def test_cosines_and_sines_are_those_of_the_exact_angle(il):
    """Rows of (1, 0) pairs, not normed, turn to the cosines and sines themselves.  The angle is
    off by 2^-27 pi from its rounding and 2^-32 pi from the position's product, cosine and sine by
    1 ulp (2^-24 below 1): 2.4e-8 + 6.0e-8."""
    d, S = 64, 20000
    g = torch.Generator().manual_seed(41)
    pos = torch.cat([torch.arange(S // 2), torch.randint(-2 ** 31, 2 ** 31 - 1, (S - S // 2,),
                                                         generator=g)])[None]
    pos = pos.to(torch.int32)
    x = torch.zeros((1, S, 1, d))
    x[..., slice(0, d, 2) if il else slice(0, d // 2)] = 1.0
    f = freqs(d)
    y, _ = pkg.qk_norm_rope(x.to(DEV), None, None, None, f.to(DEV), pos.to(DEV), interleaved=il)
    y = _np(y)[0, :, 0]
    c, s = (y[:, 0::2], y[:, 1::2]) if il else (y[:, :d // 2], y[:, d // 2:])
    angle = serving.angles(pos.numpy(), f.numpy())[0]
    bound = np.pi * (2.0 ** -27 + 2.0 ** -32) + 2.0 ** -24
    assert np.abs(c - np.cos(angle)).max() <= bound and np.abs(s - np.sin(angle)).max() <= bound
    # the quarter turns themselves: fp32 pi / 2 is 4.4e-8 from it, four of them 1.75e-7
    quarter = torch.tensor([np.pi / 2] * (d // 2), dtype=torch.float32)
    y, _ = pkg.qk_norm_rope(x[:, :9].to(DEV).contiguous(), None, None, None, quarter.to(DEV),
                            torch.arange(-4, 5, dtype=torch.int32, device=DEV)[None], interleaved=il)
    y = _np(y)[0, :, 0]
    c, s = (y[:, 0], y[:, 1]) if il else (y[:, 0], y[:, d // 2])
    assert np.abs(c - np.array([1, 0, -1, 0, 1, 0, -1, 0, 1])).max() <= 2e-7
    assert np.abs(s - np.array([0, 1, 0, -1, 0, 1, 0, -1, 0])).max() <= 2e-7


@pytest.mark.parametrize("S,Hq,Hk,d", [(64, 8, 2, 128), (1500, 16, 4, 64)])
def test_calls_in_a_row_share_a_workspace(S, Hq, Hk, d):
    """The gains' gradients are summed from the workspace that the call before used: each is of its
    own inputs, in single calls and in replays."""
    f = freqs(d).to(DEV)
    need = pkg.cp_qk_norm_rope_bwd_workspace_bytes(1, S, Hq, Hk, d)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    sets, outs, want = [], [], []
    for seed in range(8):
        q, k, qw, kw, g = make(1, S, Hq, Hk, d, torch.bfloat16, 100 + seed)
        dqo, dko = (torch.randn(t.shape, generator=g).to(t.dtype).to(DEV) for t in (q, k))
        sets.append((dqo, dko, q.contiguous(), k.contiguous(), qw, kw, f, None))
        outs.append([torch.empty_like(dqo), torch.empty_like(dko)]
                    + [torch.empty(d, device=DEV) for _ in range(2)])
        pkg.cp_qk_norm_rope_bwd(*sets[-1], *outs[-1], workspace=ws)
        torch.cuda.synchronize()
        want.append([t.clone() for t in outs[-1]])

    def all_of_them():
        for s, o in zip(sets, outs):
            pkg.cp_qk_norm_rope_bwd(*s, *o, workspace=ws)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        all_of_them()
    for once in [all_of_them] * 20 + [graph.replay] * 20:
        for o in outs:
            for t in o:
                t.zero_()
        once()
        for o, x in zip(outs, want):
            assert all(torch.equal(a, b) for a, b in zip(o, x))
