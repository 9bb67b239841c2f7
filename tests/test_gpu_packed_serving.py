"""The packed attention and the cache in 4 bits used together and with the operators around them,
and the calls at the edges of what they allow: host threads, graphs and streams side by side,
offsets past 32 bits.

Tolerances are those derived in test_gpu_packed.py, test_gpu_int4_cache.py, test_gpu_norm_rope.py
and test_gpu_paged_decode.py; where a step's output feeds the next, the oracle is fed that output.
"""
import os
import threading

import numpy as np
import pytest
import torch

import context_ring_attention_fwd_gb300 as pkg
from oracle import packed, serving
from test_gpu_int4_cache import empty_cache, raw
from test_gpu_packed import Prompts, int32

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


def freqs(rot, theta=10000.0):
    return torch.tensor(theta ** (-np.arange(0, rot, 2) / rot), dtype=torch.float32, device=DEV)


def test_prompts_are_prefilled_kept_in_4_bits_and_continued():
    """Packed prompts of different lengths through one layer of grouped heads: normed and turned
    by positions that restart, attended, appended to a cache in 4 bits, then continued for a few
    tokens each.  Every step against the oracle on what the step before left."""
    Hq, Hk, d, page, lens, steps = 6, 2, 64, 16, [33, 1, 70, 16], 3
    g = torch.Generator().manual_seed(1)
    p = Prompts(lens, Hq, Hk, d, seed=2, pad=0)
    w = [(1 + 0.2 * torch.randn(d, generator=g)).to(DEV) for _ in range(2)]
    f = freqs(d)
    pos = np.concatenate([np.arange(n) for n in lens])[None]
    q, k = (t[0] for t in pkg.qk_norm_rope(p.q[None], p.k[None], w[0], w[1], f,
                                           torch.tensor(pos, dtype=torch.int32, device=DEV)))
    for got, x, gain in ((q, p.q, w[0]), (k, p.k, w[1])):
        want, _ = serving.norm_rope(_np(x)[None], _np(gain), 1e-6, f.cpu().numpy(), pos)
        assert np.abs(_np(got) - want[0]).max() <= 2.0 ** -8 * np.abs(want).max()
    p.q, p.k = q, k
    p.check(*p.forward())
    # the cache: keys turned already, values as they are
    B, most = len(lens), 6
    n_pages = B * most + 1
    table = torch.tensor(np.random.default_rng(3).permutation(n_pages)[:B * most].reshape(B, most),
                         dtype=torch.int32, device=DEV)
    kc, vc, ks, vs = empty_cache(n_pages, page, Hk, d, True, 4)
    scales = dict(k_scale=ks, v_scale=vs)
    held = torch.zeros(B, dtype=torch.int32, device=DEV)
    for b, n in enumerate(lens):
        rows = slice(int(p.ends[b]), int(p.ends[b]) + n)
        pkg.paged_append(None, k[rows][None], p.v[rows][None], kc, vc, table[b:b + 1],
                         held[b:b + 1], **scales)
    held += int32(lens)
    t = table.cpu().numpy()
    for b, n in enumerate(lens):
        at = np.arange(n)
        rows = slice(int(p.ends[b]), int(p.ends[b]) + n)
        for x, cache, sc in ((k, kc, ks), (p.v, vc, vs)):
            codes, scale = serving.quantise4(x[rows].float().cpu().numpy())
            assert np.array_equal(raw(cache)[t[b, at // page], at % page], codes)
            assert np.array_equal(raw(sc)[t[b, at // page], at % page], scale)
    for step in range(steps):
        n_q = 1 + step % 2
        x = torch.randn((B, n_q, Hq + 2 * Hk, d), generator=g).to(BF16).to(DEV)
        q1 = pkg.paged_append(x[:, :, :Hq], x[:, :, Hq:Hq + Hk], x[:, :, Hq + Hk:], kc, vc, table,
                              held, None, w[0], w[1], f, **scales)
        held += n_q
        out, lse = pkg.paged_attn_decode(q1, kc, vc, table, held, **scales)
        keys, values = (serving.values4(raw(c), raw(s)) for c, s in ((kc, ks), (vc, vs)))
        args = (t, held.tolist())
        want, wantl = serving.paged_decode(_np(q1), np.nan_to_num(keys), np.nan_to_num(values), *args)
        size, _ = serving.paged_decode(_np(q1), np.nan_to_num(keys), np.abs(np.nan_to_num(values)),
                                       *args)
        seen = np.concatenate([keys[t[b, np.arange(n) // page], np.arange(n) % page].ravel()
                               for b, n in enumerate(held.tolist())])
        A = np.abs(_np(q1)).max() * np.abs(seen).max() * np.sqrt(d)
        tol = (2.0 ** -11 + 2.0 ** -15 * (A + 1)) * size + 2.0 ** -8 * np.abs(want)
        assert np.all(np.abs(_np(out) - want) <= tol)
        assert np.abs(_np(lse) - wantl).max() <= 2.0 ** -16 * (A + 1)


def test_the_gradient_runs_to_the_projection():
    """Norm and rotation, packed attention, and back, the gradients of q, k and v landing in views
    of one projection's gradient; each backward against the oracle on what it was given."""
    Hq, Hk, d, lens = 8, 2, 128, [50, 129, 7]
    g = torch.Generator().manual_seed(5)
    p = Prompts(lens, Hq, Hk, d, seed=6, pad=0)
    raw_q, raw_k = p.q, p.k
    w = [(1 + 0.2 * torch.randn(d, generator=g)).to(DEV) for _ in range(2)]
    f = freqs(d)
    pos = np.concatenate([np.arange(n) for n in lens])[None]
    pos_t = torch.tensor(pos, dtype=torch.int32, device=DEV)
    p.q, p.k = (t[0] for t in pkg.qk_norm_rope(raw_q[None], raw_k[None], w[0], w[1], f, pos_t))
    out, lse = p.forward()
    p.check(out, lse)
    grad = torch.zeros((p.T, Hq + 2 * Hk, d), dtype=BF16, device=DEV)
    dq, dk, dv = p.backward(out, lse)
    p.check_gradients(out, lse, (dq, dk, dv))
    grad[:, Hq + Hk:] = dv
    pkg.cp_qk_norm_rope_bwd(dq[None], dk[None], raw_q[None], raw_k[None], w[0], w[1], f, pos_t,
                            grad[None, :, :Hq], grad[None, :, Hq:Hq + Hk], None, None)
    for got, gy, x, gain in ((grad[:, :Hq], dq, raw_q, w[0]), (grad[:, Hq:Hq + Hk], dk, raw_k, w[1])):
        want, _ = serving.norm_rope_bwd(_np(gy)[None], _np(x)[None], _np(gain), 1e-6,
                                        f.cpu().numpy(), pos)
        assert np.abs(_np(got) - want[0]).max() <= 2.0 ** -7 * np.abs(want).max()


def layer_call(seed, lens, Hq, Hk, d):
    p = Prompts(lens, Hq, Hk, d, seed=seed)

    def call(**s):
        out, lse = pkg.packed_attn_fwd(p.q, p.k, p.v, p.offsets, **s)
        return (out, lse) + pkg.packed_attn_bwd(p.q, p.k, p.v, out, lse, p.dout, p.offsets, **s)
    return call


def test_threads_and_captures_side_by_side():
    """One host thread runs the backward eagerly, another captures and replays it, a third holds a
    capture open meanwhile: none disturbs the others, and all results are the single call's."""
    calls = [layer_call(7, [700, 90], 4, 1, 128), layer_call(8, [64] * 20, 8, 2, 64)]
    want = [c() for c in calls]
    torch.cuda.synchronize()
    bad, opened, finish = [], threading.Event(), threading.Event()

    def same(got, i):
        return all(torch.equal(a, b) for a, b in zip(got, want[i]))

    def eager():
        torch.cuda.set_device(0)
        s = torch.cuda.Stream()
        opened.wait(60)
        with torch.cuda.stream(s):
            for _ in range(20):
                got = calls[0]()
                s.synchronize()
                if not same(got, 0):
                    bad.append("eager")
        finish.set()

    def capture():
        torch.cuda.set_device(0)
        graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.stream(s):
            graph.capture_begin(capture_error_mode="thread_local")
            got = calls[1]()
            opened.set()
            finish.wait(60)  # the capture stays open while the other thread works
            graph.capture_end()
            for _ in range(5):
                graph.replay()
                s.synchronize()
                if not same(got, 1):
                    bad.append("captured")

    errors = []

    def guarded(f):
        def run():
            try:
                f()
            except Exception as e:  # noqa: BLE001 - reported below
                errors.append(repr(e))
                opened.set(), finish.set()
        return run

    threads = [threading.Thread(target=guarded(f)) for f in (capture, eager)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(120)
    assert not errors and not bad
    torch.cuda.synchronize()


def test_two_graphs_replayed_side_by_side():
    calls = [layer_call(9, [500, 30], 4, 2, 64), layer_call(10, [200, 200], 6, 2, 128)]
    want = [c() for c in calls]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for c in calls:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(c())
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(10):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for got, w in zip(outs, want):
        assert all(torch.equal(a, b) for a, b in zip(got, w))


@pytest.mark.parametrize("raw_stream", [False, True])
def test_a_call_on_another_stream_keeps_its_memory_to_itself(raw_stream):
    """stream= while that stream is behind: neither workspaces nor outputs are memory that the
    current stream takes meanwhile."""
    side = torch.cuda.Stream()
    given = side.cuda_stream if raw_stream else side
    p = Prompts([300, 41], 8, 2, 64, seed=11)
    out, lse = pkg.packed_attn_fwd(p.q, p.k, p.v, p.offsets)
    calls = {
        "fwd": (lambda **s: pkg.packed_attn_fwd(p.q, p.k, p.v, p.offsets, **s),
                pkg.cp_packed_attn_fwd_workspace_bytes(p.T, 2, 8, 2, 64)),
        "bwd": (lambda **s: pkg.packed_attn_bwd(p.q, p.k, p.v, out, lse, p.dout, p.offsets, **s),
                pkg.cp_packed_attn_bwd_workspace_bytes(p.T, 2, 8, 2, 64))}
    for name, (call, need) in calls.items():
        want = call()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
        got = call(stream=given)
        sizes = {need} | {t.numel() * t.element_size() for t in got}
        fills = [torch.full((n,), 0xA5, dtype=torch.uint8, device=DEV) for n in sizes
                 for _ in range(4)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), name
        assert all((t == 0xA5).all() for t in fills), name


def test_rows_past_32_bits():
    """q, out and their gradients of 2.4e9 entries each: the first and the last sequences, far
    behind 2^31, equal the same rows alone (but dk and dv, whose tiles a call of few sums up in
    parts and so in another order: those are held to the oracle)."""
    Hq, Hk, d, n, L = 64, 1, 128, 2930, 100
    T = n * L
    g = torch.Generator(device=DEV).manual_seed(12)
    q, dout = (torch.empty((T, Hq, d), dtype=BF16, device=DEV).normal_(generator=g) for _ in range(2))
    k, v = (torch.empty((T, Hk, d), dtype=BF16, device=DEV).normal_(generator=g) for _ in range(2))
    ends = torch.arange(0, T + 1, L, dtype=torch.int32, device=DEV)
    assert q.numel() > 2 ** 31
    out, lse = pkg.packed_attn_fwd(q, k, v, ends)
    grads = pkg.packed_attn_bwd(q, k, v, out, lse, dout, ends)
    for rows in (slice(0, 3 * L), slice(T - 3 * L, T)):
        alone, lse1 = pkg.packed_attn_fwd(q[rows], k[rows], v[rows], ends[:4])
        assert torch.equal(out[rows], alone) and torch.equal(lse[:, rows], lse1)
        few = pkg.packed_attn_bwd(q[rows], k[rows], v[rows], alone, lse1, dout[rows], ends[:4])
        assert torch.equal(grads[0][rows], few[0])
        p = Prompts([L] * 3, Hq, Hk, d, pad=0)
        p.q, p.k, p.v, p.dout = q[rows], k[rows], v[rows], dout[rows]
        p.check(alone, lse1)
        p.check_gradients(alone, lse1, [x[rows] for x in grads])
        p.check_gradients(alone, lse1, few)


def test_one_workspace_serves_calls_of_other_sizes_in_turn():
    a, b = Prompts([900, 3], 8, 1, 128, seed=13), Prompts([20] * 9, 6, 3, 64, seed=14)
    need = max(f(p.T, len(p.ends) - 1, p.q.shape[1], p.k.shape[1], p.q.shape[2])
               for p in (a, b) for f in (pkg.cp_packed_attn_fwd_workspace_bytes,
                                         pkg.cp_packed_attn_bwd_workspace_bytes))
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device=DEV)
    for p in (a, b, a):
        out, lse = p.forward(workspace=ws)
        p.check(out, lse)
        p.check_gradients(out, lse, p.backward(out, lse, workspace=ws))
    with pytest.raises(pkg.CpError, match="BUFFER"):
        b.forward(workspace=ws[:256])


def test_what_does_not_fit_is_refused():
    p = Prompts([20], 4, 2, 64, seed=15, pad=0)
    out, lse = p.forward()
    args = (p.q, p.k, p.v, p.offsets)
    with pytest.raises(TypeError, match="q must be"):
        pkg.packed_attn_fwd(p.q.float(), p.k, p.v, p.offsets)
    with pytest.raises(ValueError, match="three dimensions"):
        pkg.packed_attn_fwd(p.q[None], p.k, p.v, p.offsets)
    with pytest.raises(ValueError, match="k must have shape"):
        pkg.packed_attn_fwd(p.q, p.k[:10], p.v, p.offsets)
    with pytest.raises(ValueError, match="seq_offsets"):
        pkg.packed_attn_fwd(p.q, p.k, p.v, p.offsets[:1])
    with pytest.raises(TypeError, match="seq_offsets"):
        pkg.packed_attn_fwd(p.q, p.k, p.v, p.offsets.long())
    with pytest.raises(ValueError, match="out must be contiguous"):
        pkg.packed_attn_fwd(*args, out=torch.empty_like(out).transpose(0, 1).contiguous()
                            .transpose(0, 1))
    with pytest.raises(pkg.CpError, match="SHAPE"):
        pkg.packed_attn_fwd(p.q[:, :3], p.k, p.v, p.offsets)
    with pytest.raises(pkg.CpError, match="ALIGN"):       # one row for all tokens
        pkg.packed_attn_fwd(p.q, p.k[:1].expand(20, 2, 64), p.v, p.offsets)
    with pytest.raises(pkg.CpError, match="ALIGN"):       # one head for all
        pkg.packed_attn_fwd(p.q, p.k[:, :1].expand(20, 2, 64), p.v, p.offsets)
    with pytest.raises(ValueError, match="lse must have shape"):
        pkg.packed_attn_bwd(p.q, p.k, p.v, out, lse.T, p.q, p.offsets)
    with pytest.raises(pkg.CpError, match="ALIGN"):       # a gradient whose rows overlap
        pkg.packed_attn_bwd(p.q, p.k, p.v, out, lse, out, p.offsets,
                            dk=torch.zeros((20, 64), dtype=BF16, device=DEV)[:, None].expand(20, 2, 64))
