"""Without a GPU: the oracle of the norm, rotation, append and decode operators
against closed forms and differences, and the calls' refusals."""
import ctypes
import os

import numpy as np
import pytest

import context_ring_attention_fwd_gb300 as pkg
from context_ring_attention_fwd_gb300 import _binding
from oracle import serving

V = ctypes.c_void_p
FAKE = V(0x10000)        # aligned, never dereferenced: checks fail first
ODD = V(0x10002)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(pkg.LIB_PATH):
        from context_ring_attention_fwd_gb300 import _build
        _build.build()
    return pkg.lib()


def freqs(rot, theta=10000.0):
    return (theta ** (-np.arange(0, rot, 2) / rot)).astype(np.float32)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_a_complex_product_and_keeps_relative_positions(interleaved):
    rng = np.random.default_rng(1)
    d, rot = 64, 48
    f = freqs(rot)
    x, z = rng.standard_normal((2, 1, 1, 1, d))
    ang = serving.angles(np.array([[11]]), f)[:, :, None]
    y = serving.rotate(x, ang, interleaved)
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2),
                                                                     slice(rot // 2, rot))
    want = (x[..., a] + 1j * x[..., b]) * np.exp(1j * 11.0 * f.astype(np.float64))
    assert np.abs(y[..., a] + 1j * y[..., b] - want).max() < 1e-13
    assert np.array_equal(y[..., rot:], x[..., rot:])
    # <R(p) x, R(p') z> depends on p - p' alone
    dots = [(serving.rotate(x, serving.angles(np.array([[p + 5]]), f)[:, :, None], interleaved)
             * serving.rotate(z, serving.angles(np.array([[p]]), f)[:, :, None], interleaved)).sum()
            for p in (0, 3, 1000)]
    assert np.ptp(dots) < 1e-10


def test_norm_has_unit_mean_square_and_its_gradient_is_the_differences():
    rng = np.random.default_rng(2)
    x = rng.standard_normal((1, 3, 2, 64)) * 3
    w, f = 1 + 0.3 * rng.standard_normal(64), freqs(32)
    pos = np.array([[4, 0, 9]])
    y, _ = serving.norm_rope(x, np.ones(64), 0.0, None, pos)
    assert np.abs((y * y).mean(-1) - 1).max() < 1e-12
    dy = rng.standard_normal(x.shape)
    dx, dw = serving.norm_rope_bwd(dy, x, w, 1e-3, f, pos, True)
    val = lambda x_, w_: (serving.norm_rope(x_, w_, 1e-3, f, pos, True)[0] * dy).sum()  # noqa: E731
    h = 1e-5
    for at in [(0, 0, 0, 0), (0, 1, 1, 31), (0, 2, 0, 63)]:
        e = np.zeros_like(x)
        e[at] = h
        assert abs((val(x + e, w) - val(x - e, w)) / (2 * h) - dx[at]) < 1e-8
    for c in (0, 17, 63):
        e = np.zeros(64)
        e[c] = h
        assert abs((val(x, w + e) - val(x, w - e)) / (2 * h) - dw[c]) < 1e-8


def rope_args(**kw):
    a = dict(q=FAKE, qs=None, k=FAKE, ks=None, qw=FAKE, kw=FAKE, eps=1e-6, f=FAKE, rot=64, il=0,
             pos=None, qo=FAKE, ko=FAKE, B=1, S=16, Hq=4, Hk=2, d=64, bf16=1, stream=None)
    a.update(kw)
    return list(a.values())


def strides(*s):
    return ctypes.cast((ctypes.c_int64 * 3)(*s), V)


@pytest.mark.parametrize("change,want", [
    (dict(q=None), -1), (dict(k=None), -1), (dict(qo=None), -1), (dict(ko=None), -1),
    (dict(f=None), -1), (dict(B=0), -2), (dict(S=0), -2), (dict(Hq=0), -2), (dict(Hk=-1), -2),
    (dict(rot=-16), -2), (dict(rot=80), -2), (dict(il=2), -2), (dict(bf16=2), -2),
    (dict(eps=-1.0), -2), (dict(eps=float("nan")), -2), (dict(eps=float("inf")), -2),
    (dict(S=1 << 30), -2), (dict(Hq=0x7fffffff), -2),
    (dict(d=96), -3), (dict(rot=8), -3), (dict(rot=24), -3),
    (dict(q=ODD), -4), (dict(ko=ODD), -4), (dict(qw=V(0x10001)), -4), (dict(pos=ODD), -4),
    (dict(qs=strides(0, 4, 64)), -4), (dict(ks=strides(0, -64, 64)), -4),
    (dict(qs=strides(0, 12, 64), bf16=1), -4),
])
def test_norm_rope_refuses_before_any_launch(lib, change, want):
    assert lib.cp_qk_norm_rope(*rope_args(**change)) == want


def bwd_args(**kw):
    a = dict(dqo=FAKE, dko=FAKE, q=FAKE, qs=None, k=FAKE, ks=None, qw=FAKE, kw=FAKE, eps=1e-6,
             f=FAKE, rot=64, il=0, pos=None, dq=FAKE, dqs=None, dk=FAKE, dks=None, dqw=FAKE,
             dkw=FAKE, B=1, S=16, Hq=4, Hk=2, d=64, bf16=1, ws=FAKE, n=1 << 30, stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("change,want", [
    (dict(dqo=None), -1), (dict(dk=None), -1), (dict(ws=None), -1), (dict(qw=None), -1),
    (dict(kw=None), -1), (dict(d=32), -3), (dict(dk=ODD), -4), (dict(ws=V(0x10008)), -4),
    (dict(dqs=strides(0, 256, 60)), -4),
    (dict(dqs=strides(0, 256, 0)), -2),            # heads on top of one another
    (dict(dks=strides(0, 64, 64)), -2),            # tokens on top of heads
    (dict(n=16), -6),
])
def test_norm_rope_bwd_refuses_before_any_launch(lib, change, want):
    assert lib.cp_qk_norm_rope_bwd(*bwd_args(**change)) == want


def test_norm_rope_bwd_workspace(lib):
    n = pkg.cp_qk_norm_rope_bwd_workspace_bytes(1, 1, 1, 0, 64)
    assert n > 0 and pkg.cp_qk_norm_rope_bwd_workspace_bytes(4, 8192, 32, 8, 128) >= n
    assert pkg.cp_qk_norm_rope_bwd_workspace_bytes(0, 1, 1, 1, 64) == -1
    assert pkg.cp_qk_norm_rope_bwd_workspace_bytes(1, 1, 1, 1, 80) == -1


def cache_struct(**kw):
    a = dict(k=0x10000, v=0x20000, k_strides=(16 * 2 * 64, 2 * 64, 64),
             v_strides=(16 * 2 * 64, 2 * 64, 64), k_descale=None, v_descale=None,
             page_table=0x30000, table_stride=8, n_pages=10, page_size=16, max_pages=8, Hk=2, d=64,
             elem_bytes=2)
    a.update(kw)
    a["k_strides"], a["v_strides"] = ((ctypes.c_int64 * 3)(*a[n]) for n in ("k_strides",
                                                                          "v_strides"))
    return _binding.PagedCacheStruct(**a)


BAD_CACHES = [
    (dict(k=None), -1), (dict(page_table=None), -1), (dict(elem_bytes=1), -1),
    (dict(n_pages=0), -2), (dict(page_size=0), -2), (dict(max_pages=0), -2), (dict(Hk=0), -2),
    (dict(table_stride=7), -2), (dict(page_size=1 << 28), -2),
    (dict(k_strides=(16 * 2 * 64, 64, 64)), -2), (dict(v_strides=(2 * 64, 2 * 64, 64)), -2),
    (dict(elem_bytes=4), -3), (dict(d=80), -3),
    (dict(k=0x10008), -4), (dict(k_strides=(16 * 2 * 64, 2 * 64, 60)), -4),
    (dict(elem_bytes=1, k_descale=0x10001, v_descale=0x10000), -4),
    (dict(elem_bytes=1, k_descale=0x10000, v_descale=0x10000,
          v_strides=(16 * 2 * 72, 2 * 72, 72)), -4),
]


def append_args(cache=None, **kw):
    a = dict(q=FAKE, qs=None, k=FAKE, ks=None, v=FAKE, vs=None, lens=FAKE, new=None, qw=None,
             kw=None, eps=1e-6, f=FAKE, rot=64, il=0, qo=FAKE, B=2, S=3, Hq=4, stream=None)
    a.update(kw)
    return [ctypes.byref(cache_struct(**(cache or {})))] + list(a.values())


@pytest.mark.parametrize("cache,want", BAD_CACHES)
def test_append_refuses_bad_caches(lib, cache, want):
    assert lib.cp_paged_append(*append_args(cache)) == want


@pytest.mark.parametrize("change,want", [
    (dict(k=None), -1), (dict(v=None), -1), (dict(lens=None), -1), (dict(q=None), -1),
    (dict(qo=None), -1), (dict(f=None), -1), (dict(B=0), -2), (dict(S=0), -2), (dict(Hq=-1), -2),
    (dict(rot=72), -2), (dict(eps=-1.0), -2), (dict(il=3), -2), (dict(B=1 << 30), -2),
    (dict(rot=8), -3), (dict(v=ODD), -4), (dict(new=ODD), -4), (dict(vs=strides(0, 4, 64)), -4),
])
def test_append_refuses_before_any_launch(lib, change, want):
    assert lib.cp_paged_append(*append_args(**change)) == want
    assert lib.cp_paged_append(None, *append_args(**change)[1:]) == -1


def test_paged_decode_is_attention_over_the_gathered_keys():
    """The decode oracle on an identity table equals the forward's causal oracle on its last
    rows, whatever part of the keys is called the prefix."""
    from oracle import ref
    rng = np.random.default_rng(9)
    L, H, d, ps, n = 23, 2, 16, 4, 3
    q, k, v = rng.standard_normal((3, 1, L, H, d))
    want, wantl = ref.attention(q, k, v, True)
    pages = -(-L // ps)
    kc, vc = np.zeros((2, pages, ps, H, d))
    kc.reshape(-1, H, d)[:L], vc.reshape(-1, H, d)[:L] = k[0], v[0]
    table = np.arange(pages)[None]
    for prefix in (0, 7, 20):
        out, lse = serving.paged_decode(q[:, L - n:], kc, vc, table, [L], table[0], prefix)
        assert np.abs(out - want[:, L - n:]).max() < 1e-12
        assert np.abs(lse - wantl[:, :, L - n:]).max() < 1e-12
    out, lse = serving.paged_decode(q[:, :3], kc, vc, table, [0])
    assert (out == 0).all() and np.isneginf(lse).all()


def decode_args(cache=None, **kw):
    a = dict(q=FAKE, qs=None, lens=FAKE, pages=None, P=0, out=FAKE, lse=FAKE, B=2, n_q=1, Hq=4,
             ws=FAKE, n=1 << 40, stream=None)
    a.update(kw)
    return [ctypes.byref(cache_struct(**(cache or {})))] + list(a.values())


@pytest.mark.parametrize("cache,want", BAD_CACHES)
def test_decode_refuses_bad_caches(lib, cache, want):
    assert lib.cp_paged_attn_decode(*decode_args(cache)) == want


@pytest.mark.parametrize("change,want", [
    (dict(q=None), -1), (dict(lens=None), -1), (dict(out=None), -1), (dict(lse=None), -1),
    (dict(ws=None), -1), (dict(P=5), -1), (dict(B=0), -2), (dict(B=4097), -2), (dict(n_q=0), -2),
    (dict(n_q=17), -2), (dict(Hq=3), -2), (dict(Hq=0), -2), (dict(P=-1), -2),
    (dict(P=129, pages=FAKE), -2),                        # more than max_pages * page_size
    (dict(q=ODD), -4), (dict(out=ODD), -4), (dict(ws=V(0x10010)), -4), (dict(lens=ODD), -4),
    (dict(qs=strides(0, 0, 60)), -4), (dict(n=1000), -6),
])
def test_decode_refuses_before_any_launch(lib, change, want):
    assert lib.cp_paged_attn_decode(*decode_args(**change)) == want
    assert lib.cp_paged_attn_decode(None, *decode_args(**change)[1:]) == -1


def test_decode_workspace(lib):
    f = pkg.cp_paged_attn_decode_workspace_bytes
    assert 0 < f(1, 1, 1, 1, 64) <= f(64, 4, 32, 8, 128) < f(64, 4, 32, 8, 128, 1000)
    for bad in [(0, 1, 1, 1, 64), (1, 17, 1, 1, 64), (1, 1, 3, 2, 64), (1, 1, 2, 2, 80),
                (4097, 1, 1, 1, 64)]:
        assert f(*bad) == -1


def test_the_library_is_built_where_the_extension_is_not(tmp_path, monkeypatch):
    """A failing extension leaves a linked libcpring.so behind, and its error is raised."""
    from context_ring_attention_fwd_gb300 import _build
    obj = tmp_path / "obj"
    src = tmp_path / "one.cpp"
    src.write_text('extern "C" int cp_one() { return 1; }\n')
    for name, value in (("OBJDIR", str(obj)), ("LIBDIR", str(tmp_path)), ("CSRC", str(tmp_path)),
                        ("LIB", str(tmp_path / "libcpring.so")), ("SOURCES", ["one.cpp"]),
                        ("EXT", str(tmp_path / "cpring_torch.so"))):
        monkeypatch.setattr(_build, name, value)

    (tmp_path / "cpring_torch.so").write_text("an older build's")

    def fails():
        raise RuntimeError("no headers")
    monkeypatch.setattr(_build, "_compile_ext", fails)
    with pytest.raises(RuntimeError, match="no headers"):
        _build.build()
    assert ctypes.CDLL(str(tmp_path / "libcpring.so")).cp_one() == 1
    assert not os.path.exists(tmp_path / "cpring_torch.so")


def test_one_row_of_pages_for_every_sequence_is_allowed(lib):
    """A row stride of 0 passes the cache's checks: what fails next is the workspace's size, and
    the append's heads."""
    assert lib.cp_paged_attn_decode(*decode_args(dict(table_stride=0), n=1000)) == -6
    assert lib.cp_paged_append(*append_args(dict(table_stride=0), Hq=-1)) == -2
    assert lib.cp_paged_append(*append_args(dict(table_stride=0), rot=8)) == -3
    for bad in (-1, 7):
        assert lib.cp_paged_attn_decode(*decode_args(dict(table_stride=bad), n=1000)) == -2


def test_strides_whose_extent_passes_64_bits_are_refused(lib):
    """2^40 entries between 2^31 - 1 pages, and the like for a gradient's rows."""
    far = dict(k_strides=(1 << 40, 2 * 64, 64), n_pages=0x7fffffff)
    assert lib.cp_paged_attn_decode(*decode_args(far, n=1000)) == -2
    assert lib.cp_paged_append(*append_args(far)) == -2
    assert lib.cp_qk_norm_rope_bwd(*bwd_args(dqs=strides(1 << 40, 256, 64), B=1 << 23, S=16, Hq=4,
                                             Hk=2, n=16)) == -2
