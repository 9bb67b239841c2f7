"""The norm, rotation, paged append and decode operators used together and with the ring
attention, and the calls at the edges of what they allow: layouts of the cache, the largest
batch, offsets past 32 bits, host threads and graphs side by side.

Tolerances are those derived in test_gpu_paged_decode.py, test_gpu_norm_rope.py and
test_gpu_bwd.py; where a step's bf16 output feeds the next, the oracle is fed that output.
"""
import os
import threading

import numpy as np
import pytest
import torch

import context_ring_attention_fwd_gb300 as pkg
from oracle import ref, serving

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


def normal(g, *shape):
    return torch.randn(shape, generator=g).to(BF16).to(DEV)


def test_a_layer_prefilled_appended_and_decoded_is_the_causal_layer():
    """A shared prompt is prefilled with the ring attention and appended; two continuations,
    of different lengths, are appended and decoded over it token by token and at last two tokens
    at once.  Every decoded row is causal attention over that sequence's whole history."""
    g = torch.Generator().manual_seed(1)
    H, d, page, P, steps = 4, 64, 16, 52, 7
    w = [(1 + 0.2 * torch.randn(d, generator=g)).to(DEV) for _ in range(2)]
    f = freqs(d)
    prompt = normal(g, 1, P, 3 * H, d)
    q, k, v = prompt[:, :, :H], prompt[:, :, H:2 * H], prompt[:, :, 2 * H:]
    qr, kr = pkg.qk_norm_rope(q, k, w[0], w[1], f)
    out, lse = pkg.ring_attn_fwd(qr, kr, v.contiguous(), 4, True)
    want, wantl = ref.attention(_np(qr), _np(kr), _np(v), True)
    assert np.abs(_np(out) - want).max() <= 2e-2 and np.abs(_np(lse) - wantl).max() <= 2e-2

    n_pages = 24
    kc, vc = (torch.full((n_pages, page, H, d), float("nan"), dtype=BF16, device=DEV)
              for _ in range(2))
    table = torch.full((3, 6), -1, dtype=torch.int32)
    shared = torch.tensor([17, 3, 9, 20], dtype=torch.int32)
    table[:, :4] = shared
    # the prompt goes in through one row; sequences 1 and 2 get their own copy of its last page
    lens = torch.tensor([0, 0, 0], dtype=torch.int32, device=DEV)
    one = table[:1].contiguous().to(DEV)
    again = pkg.paged_append(q, k, v, kc, vc, one, lens[:1], None, w[0], w[1], f)
    assert torch.equal(again, qr)
    for b, (last, more) in ((1, (5, 11)), (2, (6, 12))):
        table[b, 3], table[b, 4] = last, more
        kc[last], vc[last] = kc[20], vc[20]
    table = table.to(DEV)
    prefix = shared[:3].contiguous().to(DEV)             # whole pages: 48 of the 52 tokens
    hist = {b: [kr[0], v[0]] for b in (1, 2)}
    fresh = torch.tensor([0, 1, 1], dtype=torch.int32, device=DEV)   # row 0 is unused
    held = torch.tensor([0, P, P], dtype=torch.int32, device=DEV)
    for step in range(steps):
        n = 2 if step == steps - 1 else 1
        if step == 3:
            fresh[2] = 0                                 # sequence 2 pauses
        if step == 4:
            fresh[2] = 1
        new = normal(g, 3, n, 3 * H, d)
        q, k, v = new[:, :, :H], new[:, :, H:2 * H], new[:, :, 2 * H:]
        count = fresh * n
        q_out = torch.zeros((3, n, H, d), dtype=BF16, device=DEV)
        pkg.paged_append(q, k, v, kc, vc, table, held, count, w[0], w[1], f, q_out=q_out)
        at = held[:, None] + torch.arange(n, dtype=torch.int32, device=DEV)
        held = held + count
        seq = torch.where(count > 0, held, torch.zeros_like(held))
        out, lse = pkg.paged_attn_decode(q_out, kc, vc, table, seq, prefix, 48)
        assert pkg.cp_get_last_status() == 0
        k_rot = pkg.qk_norm_rope(k, None, w[1], None, f, at.contiguous())[0]
        for b in range(3):
            if int(count[b]) == 0:
                assert (out[b] == 0).all() and lse[b].isneginf().all()
                continue
            hist[b] = [torch.cat([hist[b][0], k_rot[b]]), torch.cat([hist[b][1], v[b]])]
            K, V = hist[b]
            L = K.shape[0]
            Q = torch.zeros((1, L, H, d), dtype=BF16, device=DEV)
            Q[0, L - n:] = q_out[b]
            want, wantl = ref.attention(_np(Q), _np(K)[None], _np(V)[None], True)
            assert np.abs(_np(out[b]) - want[0, L - n:]).max() <= 2e-2
            assert np.abs(_np(lse[b]) - wantl[0, :, L - n:]).max() <= 1e-3


def test_the_gradient_runs_through_rotation_and_ring_attention():
    """d(sum out * dout) through ring_attn_bwd and qk_norm_rope_bwd against the same chain in
    64 bits, packed documents with positions that restart."""
    g = torch.Generator().manual_seed(2)
    B, S, H, d = 1, 160, 2, 64
    docs = [0, 37, 96, 160]
    pos = np.concatenate([np.arange(b - a) for a, b in zip(docs, docs[1:])])[None]
    pos_d = torch.tensor(pos, dtype=torch.int32, device=DEV)
    qkv, dout = normal(g, B, S, 3 * H, d), normal(g, B, S, H, d)
    q, k, v = qkv[:, :, :H], qkv[:, :, H:2 * H], qkv[:, :, 2 * H:].contiguous()
    w = [(1 + 0.2 * torch.randn(d, generator=g)).to(DEV) for _ in range(2)]
    f = freqs(d)
    qr, kr = pkg.qk_norm_rope(q, k, w[0], w[1], f, pos_d)
    out, lse = pkg.ring_attn_fwd(qr, kr, v, 2, True, docs)
    dqr, dkr, dv = pkg.ring_attn_bwd(qr, kr, v, out, lse, dout, 2, True, docs)
    dq, dk, dqw, dkw = pkg.qk_norm_rope_bwd(dqr, dkr, q, k, w[0], w[1], f, pos_d)
    fn = f.cpu().numpy()
    rot = [serving.norm_rope(_np(x), _np(y), 1e-6, fn, pos)[0] for x, y in zip((q, k), w)]
    wq, wk, wv = ref.attention_bwd(rot[0], rot[1], _np(v), _np(dout), True, docs)
    want = [serving.norm_rope_bwd(gy, _np(x), _np(y), 1e-6, fn, pos)
            for gy, x, y in ((wq, q, w[0]), (wk, k, w[1]))]
    # the ring backward's bound, 2^-6 and 2^-10 of the largest gradient (test_gpu_bwd.py), and as
    # much again for the rounding of its bf16 operands qr and kr; through the norm it is scaled
    # by r |w|, as the gradient is
    for got, (gx, _) in zip((dq, dk), want):
        e = np.abs(_np(got) - gx)
        top = np.abs(gx).max()
        assert e.max() <= 2.0 ** -5 * top and e.mean() <= 2.0 ** -9 * top
    for got, (_, gw), gy in zip((dqw, dkw), want, (wq, wk)):
        # a sum over B S H rows of terms of size max|g| |u|, each off by its row's mean error
        assert np.abs(_np(got) - gw).max() <= B * S * H * 2.0 ** -9 * np.abs(gy).max() * 3
    assert np.abs(_np(dv) - wv).max() <= 2.0 ** -5 * np.abs(wv).max()


def filled(g, lens, Hq, Hk, d, page, n_pages, prefix_len=0, dtype=BF16, n_q=1):
    order = torch.randperm(n_pages, generator=g)
    most = -(-max(max(lens), prefix_len, 1) // page)
    whole, shared = prefix_len // page, -(-prefix_len // page)
    table = torch.full((len(lens), most), -1, dtype=torch.int32)
    table[:, :whole] = order[:whole]
    at = shared
    for b, n in enumerate(lens):
        need = max(0, -(-n // page) - whole)
        table[b, whole:whole + need] = order[at:at + need]
        at += need
    assert at <= n_pages
    q = normal(g, len(lens), n_q, Hq, d)
    return (q, table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV),
            order[:shared].to(torch.int32).to(DEV) if prefix_len else None)


@pytest.mark.parametrize("path", [0, 1])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("page", [8, 24, 256, 384])
def test_layouts_of_the_cache_give_one_result(path, e4m3, page):
    """Token-major, head-major, K and V of one allocation, pages with gaps, and strides that no
    tensor map describes: the same bits."""
    g = torch.Generator().manual_seed(page)
    Hq, Hk, d, P = 8, 2, 128, 500
    lens = [P + int(x) for x in torch.randint(0, 60, (20,), generator=g)]
    n_pages = 3 + sum(-(-n // page) - P // page for n in lens) + -(-P // page)
    q, table, seq, prefix = filled(g, lens, Hq, Hk, d, page, n_pages, P)
    k, v = (torch.randn((n_pages, page, Hk, d), generator=g).to(DEV) for _ in range(2))
    desc = None
    if e4m3:
        desc = torch.full((Hk,), 0.01, device=DEV)
        k, v = ((x / 0.01).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                for x in (k, v))
    else:
        k, v = k.to(BF16), v.to(BF16)

    def head_major(x):
        return x.transpose(1, 2).contiguous().transpose(1, 2)

    def apart(x, gap):          # rows of a wider allocation, `gap` more entries a token
        wide = torch.zeros((n_pages, page, Hk * d + gap), dtype=x.dtype, device=DEV)
        view = wide[:, :, :Hk * d].unflatten(2, (Hk, d))
        view.copy_(x)
        return view

    both = torch.stack([k, v], 1)                         # [pages, 2, page, Hk, d]
    layouts = [(k, v), (head_major(k), head_major(v)), (both[:, 0], both[:, 1]),
               (apart(k, d), apart(v, d)), (apart(k, 16), apart(v, 48)), (k, head_major(v))]
    pkg.test_set_prefix_path(path)
    try:
        want = None
        for kk, vv in layouts:
            got = pkg.paged_attn_decode(q, kk, vv, table, seq, prefix, P, desc, desc)
            assert pkg.cp_get_last_status() == 0
            if want is None:
                want = got
                assert not got[0].isnan().any()
            if path == 0 or not e4m3:
                assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
            else:   # S from E4M3 pairs of Q by TMA, from fp16 otherwise: two roundings of P apart
                assert (got[0].float() - want[0].float()).abs().max() <= 2.0 ** -7
                assert (got[1] - want[1]).abs().max() <= 2.0 ** -10
        # and the append fills every layout alike
        new = normal(g, 20, 1, 2 * Hk, d)
        filled_k = None
        for kk, vv in layouts:
            pkg.paged_append(None, new[:, :, :Hk], new[:, :, Hk:], kk, vv, table, seq - 1, None,
                             None, None, freqs(d), k_descale=desc, v_descale=desc)
            if filled_k is None:
                filled_k = kk.clone(), vv.clone()
            assert torch.equal(kk, filled_k[0]) and torch.equal(vv, filled_k[1])
    finally:
        pkg.test_set_prefix_path(-1)


def test_the_largest_batch():
    """4096 sequences of one or no key: the answer is that key's value."""
    g = torch.Generator().manual_seed(3)
    B, d = 4096, 64
    lens = [int(x) for x in torch.randint(0, 2, (B,), generator=g)]
    q, table, seq, _ = filled(g, lens, 1, 1, d, 2, B)
    k, v = normal(g, B, 2, 1, d), normal(g, B, 2, 1, d)
    out, lse = pkg.paged_attn_decode(q, k, v, table, seq)
    at = table[:, 0].clamp(min=0).long()
    live = seq > 0
    assert torch.equal(out[live, 0, 0], v[at, 0, 0][live]) and (out[~live] == 0).all()
    s = (q[:, 0, 0].double() * k[at, 0, 0].double()).sum(-1) / d ** 0.5
    assert ((lse[:, 0, 0].double() - s)[live].abs() <= 2.0 ** -18 * (1 + 64)).all()
    assert lse[~live].isneginf().all()
    with pytest.raises(pkg.CpError):
        pkg.paged_attn_decode(torch.cat([q, q[:1]]), k, v, torch.cat([table, table[:1]]),
                              torch.cat([seq, seq[:1]]))


@pytest.mark.parametrize("path", [0, 1])
def test_offsets_past_32_bits(path):
    """A cache of 5.9 G entries: the pages in use are its last ones, and equal a small cache's."""
    g = torch.Generator().manual_seed(4)
    Hk, d, page, P = 8, 128, 64, 200
    n_pages = 90000
    lens = [P + 1 + 3 * b for b in range(12)]
    q, table, seq, prefix = filled(g, lens, 32, Hk, d, page, 30, P)
    small_k, small_v = normal(g, 30, page, Hk, d), normal(g, 30, page, Hk, d)
    k = torch.empty((n_pages, page, Hk, d), dtype=BF16, device=DEV)
    v = torch.empty((n_pages, page, Hk, d), dtype=BF16, device=DEV)
    shift = n_pages - 30
    k[shift:], v[shift:] = small_k, small_v
    far = torch.where(table >= 0, table + shift, table)
    pkg.test_set_prefix_path(path)
    try:
        want = pkg.paged_attn_decode(q, small_k, small_v, table, seq, prefix, P)
        got = pkg.paged_attn_decode(q, k, v, far, seq, prefix + shift, P)
    finally:
        pkg.test_set_prefix_path(-1)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    new = normal(g, 12, 1, 2 * Hk, d)
    pkg.paged_append(None, new[:, :, :Hk], new[:, :, Hk:], k, v, far, seq - 1)
    pkg.paged_append(None, new[:, :, :Hk], new[:, :, Hk:], small_k, small_v, table, seq - 1)
    assert torch.equal(k[shift:], small_k) and torch.equal(v[shift:], small_v)


def test_rows_past_32_bits():
    """2.5 G entries of one broadcast token: its last rows equal those of a short call."""
    g = torch.Generator().manual_seed(5)
    S, H, d = 300000, 64, 128
    one = normal(g, 1, 1, H, d)
    w = torch.ones(d, device=DEV)
    f = freqs(d)
    out, _ = pkg.qk_norm_rope(one.expand(1, S, H, d), None, w, None, f)
    at = torch.arange(S - 5, S, dtype=torch.int32, device=DEV)[None]
    want, _ = pkg.qk_norm_rope(one.expand(1, 5, H, d), None, w, None, f, at)
    assert torch.equal(out[:, -5:], want)


def test_two_threads_and_two_graphs():
    """Two host threads on streams of their own, then two captured graphs replayed side by side:
    every result equals the single call's."""
    g = torch.Generator().manual_seed(6)
    cases = []
    for P in (0, 700):
        lens = [P + int(x) for x in torch.randint(1, 300, (9,), generator=g)]
        q, table, seq, prefix = filled(g, lens, 16, 4, 64, 16, 300, P, n_q=2)
        k, v = normal(g, 300, 16, 4, 64), normal(g, 300, 16, 4, 64)
        cases.append((q, k, v, table, seq, prefix, P))
    pkg.test_set_prefix_path(1)
    try:
        want = [pkg.paged_attn_decode(*c) for c in cases]
        bad = []

        def work(i):
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(30):
                    got = pkg.paged_attn_decode(*cases[i])
                    s.synchronize()
                    if not (torch.equal(got[0], want[i][0]) and torch.equal(got[1], want[i][1])):
                        bad.append(i)

        torch.cuda.synchronize()
        threads = [threading.Thread(target=work, args=(i,)) for i in (0, 1)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        assert not bad
        torch.cuda.synchronize()
        graphs, outs = [], []
        for c in cases:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                outs.append(pkg.paged_attn_decode(*c))
            graphs.append(graph)
        streams = [torch.cuda.Stream() for _ in graphs]
        for _ in range(10):
            for graph, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    graph.replay()
        torch.cuda.synchronize()
        for got, w in zip(outs, want):
            assert torch.equal(got[0], w[0]) and torch.equal(got[1], w[1])
    finally:
        pkg.test_set_prefix_path(-1)
    assert pkg.cp_get_last_status() == 0


def some_calls():
    """The four calls with small and large workspaces: (name, call, bytes of its workspace)."""
    g = torch.Generator().manual_seed(7)
    lens = [700 + int(x) for x in torch.randint(1, 90, (9,), generator=g)]
    q, table, seq, prefix = filled(g, lens, 16, 4, 64, 16, 300, 700, n_q=2)
    k, v = normal(g, 300, 16, 4, 64), normal(g, 300, 16, 4, 64)
    x, y = normal(g, 1, 900, 16, 128), normal(g, 1, 900, 4, 128)
    w, f = torch.ones(128, device=DEV), freqs(128)
    dx, dy = normal(g, *x.shape), normal(g, *y.shape)
    new = normal(g, 9, 2, 24, 64)
    need = pkg.cp_paged_attn_decode_workspace_bytes(9, 2, 16, 4, 64, 700)
    return [
        ("decode", lambda **s: pkg.paged_attn_decode(q, k, v, table, seq, prefix, 700, **s), need),
        ("forward", lambda **s: pkg.qk_norm_rope(x, y, w, w, f, **s), 1 << 16),
        ("backward", lambda **s: pkg.qk_norm_rope_bwd(dx, dy, x, y, w, w, f, **s),
         pkg.cp_qk_norm_rope_bwd_workspace_bytes(1, 900, 16, 4, 128)),
        ("append", lambda **s: (pkg.paged_append(new[:, :, :16], new[:, :, 16:20], new[:, :, 20:],
                                                 k, v, table, seq - 2, **s),), 1 << 16)]


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("path", [0, 1])
def test_a_call_on_another_stream_keeps_its_memory_to_itself(path, raw):
    """A call with stream= while that stream is behind, and while the current one is: neither
    its workspace nor its outputs are memory that the other stream's work holds."""
    side = torch.cuda.Stream()
    given = side.cuda_stream if raw else side
    pkg.test_set_prefix_path(path)
    try:
        for name, call, need in some_calls():
            want = call()
            torch.cuda.synchronize()
            # the side stream is behind: what the current one allocates now is its own
            with torch.cuda.stream(side):
                torch.cuda._sleep(20_000_000)
            got = call(stream=given)
            sizes = {need} | {t.numel() * t.element_size() for t in got}
            fills = [torch.full((n,), 0xA5, dtype=torch.uint8, device=DEV)
                     for n in sizes for _ in range(3)]
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want)), name
            assert all((t == 0xA5).all() for t in fills), name
            # the current stream is behind: its dropped blocks are not the call's yet
            del got, fills
            torch.cuda.synchronize()
            torch.cuda._sleep(20_000_000)
            for n in sizes:
                for _ in range(3):
                    torch.full((n,), 0x5A, dtype=torch.uint8, device=DEV)
            got = call(stream=given)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want)), name
            # the outputs, used here and dropped, are not the side stream's again until then
            torch.cuda._sleep(20_000_000)
            kept = [t.clone() for t in got]
            sizes = [t.numel() * t.element_size() for t in got]
            del got
            with torch.cuda.stream(side):
                for n in sizes:
                    for _ in range(3):
                        torch.full((n,), 0x5A, dtype=torch.uint8, device=DEV)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(kept, want)), name
    finally:
        pkg.test_set_prefix_path(-1)


def test_a_call_captured_beside_the_current_stream():
    """A capture whose calls are given a forked stream: replayed, it gives the single results."""
    calls = some_calls()[:3]
    want = [call() for _, call, _ in calls]
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        got = [call(stream=side) for _, call, _ in calls]
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(3):
        for r in got:
            for t in r:
                t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("path", [0, 1])
def test_an_expanded_page_table(path):
    """Sequences that share every page through one row of the table, as its copies give it."""
    g = torch.Generator().manual_seed(8)
    P = 100
    q, table, seq, prefix = filled(g, [P + 90], 8, 2, 64, 16, 20, P)
    k, v = normal(g, 20, 16, 2, 64), normal(g, 20, 16, 2, 64)
    q = normal(g, 40, 1, 8, 64)
    lens = (P + 1 + torch.arange(40, dtype=torch.int32, device=DEV) * 2).contiguous()
    wide = table.expand(40, table.shape[1])
    assert wide.stride(0) == 0
    pkg.test_set_prefix_path(path)
    try:
        want = pkg.paged_attn_decode(q, k, v, wide.contiguous(), lens, prefix, P)
        got = pkg.paged_attn_decode(q, k, v, wide, lens, prefix, P)
    finally:
        pkg.test_set_prefix_path(-1)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    new = normal(g, 40, 1, 4, 64)                    # to 40 slots of the shared pages
    ka, va = k.clone(), v.clone()
    pkg.paged_append(None, new[:, :, :2], new[:, :, 2:], k, v, wide, lens - 1)
    pkg.paged_append(None, new[:, :, :2], new[:, :, 2:], ka, va, wide.contiguous(), lens - 1)
    assert torch.equal(k, ka) and torch.equal(v, va)
    assert pkg.cp_get_last_status() == 0
