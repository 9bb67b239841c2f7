"""The ring attention's calls captured into graphs: every replay computes all work items from the
inputs as they are then.

Each shape has more work items than the GPU has multiprocessors, so that a block takes several.
Which block computes an item does not change its result: replays equal the single calls bit for
bit.
"""
import ctypes
import os

import pytest
import torch

import context_ring_attention_fwd_gb300 as pkg

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16 = torch.bfloat16
B, S, H = 1, 2048, 32
DOCS = [0, 300, 301, 1200, 2048]


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


def rows(seed, d, n=4):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return [torch.randn((B, S, H, d), generator=g, device=DEV).to(BF16) for _ in range(n)]


def offsets(docs):
    return pkg.doc_offsets_tensor(docs, torch.device(DEV, 0))


def noalloc(q, k, v, out, lse, docs):
    p = [ctypes.c_void_p(t.data_ptr()) for t in (q, k, v, out, lse)]
    st = pkg.lib().cp_ring_attn_fwd_noalloc(
        *p, B, S, H, q.shape[-1], 4, 1, ctypes.c_void_p(docs.data_ptr()),
        ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert st == 0


def forward_call(d):
    docs = offsets(DOCS)
    out, lse = torch.empty((B, S, H, d), dtype=BF16, device=DEV), torch.empty((B, H, S), device=DEV)

    def call(q, k, v, g):
        noalloc(q, k, v, out, lse, docs)
        return out, lse
    return call


def fp8_call(d):
    def call(q, k, v, g):
        return pkg.ring_attn_fwd_fp8(pkg.fp8_quantize_qkv(q, k, v), 2, True)
    return call


def step_call(d):
    o = torch.empty((B, S, H, d), device=DEV)
    m, l = (torch.empty((B, H, S), device=DEV) for _ in range(2))

    def call(q, k, v, g):
        pkg.cp_ring_step(q, k, v, o, m, l, 1, 0, 0, True)
        return o, m, l
    return call


def backward_call(d, docs=None):
    docs_t = None if docs is None else offsets(docs)
    grads = [torch.empty((B, S, H, d), dtype=BF16, device=DEV) for _ in range(3)]

    def call(q, k, v, g):
        out, lse = pkg.ring_attn_fwd(q, k, v, 2, True)
        pkg.cp_ring_attn_bwd(q, k, v, out, lse, g, *grads, 2, True, docs_t)
        return grads
    return call


CALLS = {"forward with documents": (forward_call, 128), "forward with documents, d = 64": (forward_call, 64),
         "forward in FP8": (fp8_call, 128), "one step": (step_call, 128),
         "backward": (backward_call, 128), "backward, d = 64": (backward_call, 64),
         "backward with documents": (lambda d: backward_call(d, DOCS), 128)}


def captured(call, x):
    side = torch.cuda.Stream()  # warm up on a stream, as a capture asks for
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(*x)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call(*x)
    return graph, got


@pytest.mark.parametrize("name", CALLS)
def test_replays_follow_the_inputs(name):
    make, d = CALLS[name]
    call = make(d)
    x = rows(1, d)
    graph, got = captured(call, x)
    for seed in (2, 3, 4):
        fresh = rows(seed, d)
        want = [t.clone() for t in make(d)(*fresh)]
        for to, t in zip(x, fresh):
            to.copy_(t)
        for t in got:
            t.fill_(7)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), seed


def test_replays_among_many_single_calls():
    """More single calls between and beside the replays than the library has claim counters."""
    call = forward_call(64)
    x = rows(5, 64)
    graph, got = captured(call, x)
    want = [t.clone() for t in forward_call(64)(*x)]
    o = torch.empty((1, 256, 2, 64), device=DEV)
    m, l = (torch.empty((1, 2, 256), device=DEV) for _ in range(2))
    small = [t[:, :256, :2].contiguous() for t in x[:3]]
    for _ in range(3):
        for _ in range(300):
            pkg.cp_ring_step(*small, o, m, l, 1, 0, 0, True)
        for t in got:
            t.fill_(7)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    single = backward_call(64)
    want_g = [t.clone() for t in single(*x)]
    side = torch.cuda.Stream()
    for _ in range(50):
        with torch.cuda.stream(side):
            graph.replay()
        got_g = single(*x)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got_g, want_g))
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def documents_call(d, docs, fp8=False):
    docs_t = offsets(docs)
    out, lse = torch.empty((B, S, H, d), dtype=BF16, device=DEV), torch.empty((B, H, S), device=DEV)

    def call(q, k, v, g):
        if fp8:
            pkg.cp_ring_attn_fwd_fp8(*pkg.fp8_quantize_qkv(q, k, v), out, lse, 2, True, docs_t)
        else:
            pkg.cp_ring_attn_fwd(q, k, v, out, lse, 2, True, docs_t)
        return out, lse
    return call


@pytest.mark.parametrize("fp8", [False, True])
def test_a_captured_call_has_scratch_of_its_own(fp8):
    """Calls whose scratch for documents is cached are captured, the cache grows, and replays run
    beside single calls with other documents."""
    d = 128
    x, fresh = rows(6, d), rows(7, d)
    call = documents_call(d, DOCS, fp8)
    graph, got = captured(call, x)
    # a longer sequence: more scratch than any call here before
    T = 65536
    y = [torch.randn((1, T, 1, 64), device=DEV).to(BF16) for _ in range(3)]
    pkg.ring_attn_fwd(*y, 64, True, [0, 5, T])
    for to, t in zip(x, fresh):
        to.copy_(t)
    other = documents_call(d, [0, 1024, 1500, 2048], fp8)
    want = [t.clone() for t in documents_call(d, DOCS, fp8)(*fresh)]
    want_other = [t.clone() for t in other(*fresh)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        with torch.cuda.stream(side):
            for t in got:
                t.fill_(7)
            graph.replay()
        got_other = other(*fresh)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert all(torch.equal(a, b) for a, b in zip(got_other, want_other))


def test_calls_with_documents_after_a_capture():
    """A capture in between leaves the other streams' calls as they were."""
    d = 64
    x = rows(8, d)
    call = documents_call(d, DOCS)
    want = [t.clone() for t in call(*x)]
    kept = documents_call(d, DOCS)  # its tensors are the graph's
    graph, got = captured(kept, x)
    for s in (torch.cuda.Stream(), torch.cuda.Stream()):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            again = call(*x)
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(again, want))
    for t in got:
        t.fill_(7)
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("docs", [None, DOCS])
def test_a_host_call_while_another_is_being_captured(docs):
    """The call from host buffers captured on one stream, and made on another while that capture is
    open: both give the single call's result, and the other stream is not drawn into the capture."""
    d, N = 64, 4
    x = [t.cpu().pin_memory() for t in rows(9, d, 3)]
    need = pkg.lib().cp_ring_attn_fwd_host_workspace_bytes(B, S, H, d, N, 2)
    docs_t = None if docs is None else offsets(docs)
    p = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731

    def buffers():
        return (torch.empty(need, dtype=torch.uint8, device=DEV),
                torch.zeros((B, S, H, d), dtype=BF16).pin_memory(),
                torch.zeros((B, H, S)).pin_memory())

    def call(ws, out, lse, stream):
        return pkg.lib().cp_ring_attn_fwd_host(*(p(t) for t in x), p(out), p(lse), B, S, H, d, N, 1,
                                               None if docs is None else p(docs_t), p(ws), need,
                                               ctypes.c_void_p(stream.cuda_stream))

    single, caught, beside = buffers(), buffers(), buffers()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    assert call(*single, s1) == 0
    s1.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s1):
        graph.capture_begin(capture_error_mode="thread_local")
        captured_status = call(*caught, s1)
        status = call(*beside, s2)
        graph.capture_end()
    assert captured_status == 0 and status == 0
    s2.synchronize()
    for a, b in zip(beside[1:], single[1:]):
        assert torch.equal(a, b)
    assert not caught[1].any()
    with torch.cuda.stream(s1):
        for _ in range(2):
            caught[1].zero_()
            graph.replay()
            s1.synchronize()
            for a, b in zip(caught[1:], single[1:]):
                assert torch.equal(a, b)
