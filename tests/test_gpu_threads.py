"""The library's per-device shared state under concurrent host threads.

The library keeps a few things per device for the process's life: the cached
scratch that launches with documents lease (the doc-scan word and the
cost-ranked slot order), the backward's second stream for its dQ launch, and
the host-buffer entry's copy streams.  Two host threads here drive every one
of those on their own streams at the same time, several calls each, and
every result must equal the same call made alone, bit for bit: a lease
handed to one thread while another's kernels still read it, or an event of
one call waited on by another, would show as a difference.
"""
import os
import threading

import pytest
import torch

import context_ring_attention_fwd_gb300 as pkg
from context_ring_attention_fwd_gb300 import inputs

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


def _case(seed, S, docs):
    B, H, d, N = 1, 2, 128, 4
    q, k, v = (t.to(DEV) for t in inputs.make_qkv(B, S, H, d, seed=seed, dtype=torch.bfloat16))
    dout = inputs.make_qkv(B, S, H, d, seed=seed + 1, dtype=torch.bfloat16)[0].to(DEV)
    return dict(q=q, k=k, v=v, dout=dout, N=N, docs=docs, S=S)


def _run(c, stream):
    """Forward with documents, backward, and the host-buffer entry, all on
    `stream`; returns host copies of every output."""
    q, k, v, N, docs = c["q"], c["k"], c["v"], c["N"], c["docs"]
    with torch.cuda.stream(stream):
        out, lse = pkg.ring_attn_fwd(q, k, v, N, True, docs, stream=stream)
        dq, dk, dv = pkg.ring_attn_bwd(q, k, v, out, lse, c["dout"], N, True, docs, stream=stream)
        ho, hl = pkg.ring_attn_fwd_host(q.cpu().pin_memory(), k.cpu().pin_memory(),
                                        v.cpu().pin_memory(), N, True, docs, stream=stream)
    stream.synchronize()
    return [t.cpu() for t in (out, lse, dq, dk, dv)] + [ho.clone(), hl.clone()]


def test_two_threads_share_the_library_state():
    cases = [_case(81, 2048, [0, 300, 301, 1500, 2048]), _case(82, 4096, [0, 2000, 4096])]
    alone = [_run(c, torch.cuda.Stream()) for c in cases]
    errors, results = [], [[None] * 4 for _ in cases]

    def worker(i):
        try:
            torch.cuda.set_device(0)
            st = torch.cuda.Stream()
            for rep in range(4):
                results[i][rep] = _run(cases[i], st)
        except Exception as e:  # noqa: BLE001 - reported below
            errors.append(repr(e))

    threads = [threading.Thread(target=worker, args=(i,)) for i in range(len(cases))]
    for t in threads:
        t.start()
    for t in threads:
        t.join(timeout=300)
    assert not errors, errors
    assert pkg.cp_get_last_status() == 0
    for i in range(len(cases)):
        for rep in range(4):
            got = results[i][rep]
            assert got is not None, (i, rep)
            for a, b in zip(got, alone[i]):
                assert torch.equal(a, b), (i, rep)


@pytest.mark.parametrize("raw", [False, True])
def test_a_given_stream_owns_what_the_call_allocates(raw):
    """stream= while that stream is behind: neither the outputs nor the workspaces and document
    offsets that a call makes itself are memory that the current stream can take meanwhile."""
    c = _case(83, 1024, [0, 300, 301, 1024])
    q, k, v, N, docs, dout = c["q"], c["k"], c["v"], c["N"], c["docs"], c["dout"]
    B, S, H, d = q.shape
    out, lse = pkg.ring_attn_fwd(q, k, v, N, True, docs)
    codes = pkg.fp8_quantize_qkv(q, k, v)
    docs_t = pkg.doc_offsets_tensor(docs, q.device)
    need = {"bwd": pkg.cp_ring_attn_bwd_workspace_bytes(B, S, H, d, N),
            "ring": pkg.cp_ring_emulated_workspace_bytes(B, S, H, d, 2),
            "all-to-all": pkg.cp_ulysses_workspace_bytes(B, S, H, d, 2)}

    def into(fn):
        def call(**s):
            o, l = torch.empty_like(out), torch.empty_like(lse)
            torch.cuda.synchronize()
            if s:
                with torch.cuda.stream(side):
                    torch.cuda._sleep(20_000_000)
            fn(q, k, v, o, l, 2, True, **s)
            return o, l
        return call

    side = torch.cuda.Stream()
    given = side.cuda_stream if raw else side
    calls = {"fwd": lambda **s: pkg.ring_attn_fwd(q, k, v, N, True, docs, **s),
             "bwd": lambda **s: pkg.ring_attn_bwd(q, k, v, out, lse, dout, N, True, docs, **s),
             "steps": lambda **s: pkg.ring_attn_composed(q, k, v, N, True, **s),
             "codes": lambda **s: pkg.fp8_quantize_qkv(q, k, v, **s),
             "fp8": lambda **s: pkg.ring_attn_fwd_fp8(codes, N, True, docs, **s),
             "schedule": lambda **s: (pkg.cp_ring_schedule_device(S, N, True, docs_t, **s),),
             "ring": into(pkg.cp_ring_attn_fwd_emulated),
             "all-to-all": into(pkg.cp_ulysses_attn_fwd)}
    for name, call in calls.items():
        want = call()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
        got = call(stream=given)
        sizes = {need.get(name, 1024)} | {t.numel() * t.element_size() for t in got}
        fills = [torch.full((n,), 0xA5, dtype=torch.uint8, device=DEV) for n in sizes
                 for _ in range(4)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), name
        assert all((t == 0xA5).all() for t in fills), name
        del got, fills
        torch.cuda.synchronize()
        if name in ("ring", "all-to-all"):
            continue                                   # their outputs are the caller's
        torch.cuda._sleep(20_000_000)
        for n in sizes:
            for _ in range(4):
                torch.full((n,), 0x5A, dtype=torch.uint8, device=DEV)
        got = call(stream=given)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), name
    assert pkg.cp_get_last_status() == 0
