"""The cache in 4 bits on the CPU: the oracle's format pinned against torch's E4M3, and what the
calls refuse before any launch."""
import ctypes
import os

import numpy as np
import pytest
import torch

import context_ring_attention_fwd_gb300 as pkg
from oracle import serving
from test_serving_host import append_args, cache_struct, decode_args


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(pkg.LIB_PATH):
        from context_ring_attention_fwd_gb300 import _build
        _build.build()
    return pkg.lib()


def test_e4m3_of_the_oracle_is_torchs():
    codes = torch.arange(127, dtype=torch.uint8)
    assert np.array_equal(serving.e4m3_values(), codes.view(torch.float8_e4m3fn).double().numpy())
    rng = np.random.default_rng(0)
    v = serving.e4m3_values()
    x = np.concatenate([v, (v[1:] + v[:-1]) / 2, np.exp(rng.uniform(-9, 6.1, 4000))]).astype("f4")
    want = torch.tensor(x).clamp(max=448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(serving.e4m3_codes(x.astype(np.float64)), want)


def test_a_row_in_4_bits_by_hand():
    """Scale 1 where the largest is 7: entries are rounded to whole numbers, ties to even."""
    x = np.zeros((1, 32))
    x[0, :6] = [7, -7, 0.5, 1.5, -2.5, 3.4]
    x[0, 16:] = 0
    codes, scales = serving.quantise4(x)
    assert scales.tolist() == [[0x38, 0]]
    assert codes[0, :3].tolist() == [15 | 1 << 4, 8 | 10 << 4, 6 | 11 << 4]
    assert (codes[0, 3:] == 0x88).all()
    assert serving.values4(codes, scales)[0, :6].tolist() == [7, -7, 0, 2, -2, 3]


def test_an_entry_is_off_by_half_a_step_at_most():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((50, 3, 64)) * np.exp(rng.uniform(-3, 5, (50, 3, 1)))
    x = torch.tensor(x).bfloat16().double().numpy()
    desc = np.array([0.5, 1.25, 3.0])
    for dsc in (None, desc):
        codes, scales = serving.quantise4(x, dsc)
        step = serving.e4m3_values()[scales].repeat(16, -1)
        step = step if dsc is None else step * dsc[:, None]
        off = np.abs(serving.values4(codes, scales, dsc) - x)
        # E4M3's values lie 2^-9 apart below 2^-6, so there a scale is off by 2^-10 and 7 times it,
        # which the block's largest entry is brought to, by 7 * 2^-10
        small = 7 * 2.0 ** -10 * (1 if dsc is None else dsc[:, None])
        assert (off <= np.maximum(step / 2, small) * (1 + 2.0 ** -17)).all()
        assert off.max() > 0.4 * step.min()


def int4(**kw):
    """test_serving_host's cache (10 pages of 16 tokens, 2 heads of 64) in 4 bits."""
    a = dict(elem_bytes=-2, k_strides=(16 * 2 * 32, 2 * 32, 32), v_strides=(16 * 2 * 32, 2 * 32, 32),
             k_scale=0x50000, v_scale=0x60000, k_scale_strides=(16 * 2 * 4, 2 * 4, 4),
             v_scale_strides=(16 * 2 * 4, 2 * 4, 4))
    a.update(kw)
    for n in ("k_scale_strides", "v_scale_strides"):
        a[n] = (ctypes.c_int64 * 3)(*a[n])
    return a


@pytest.mark.parametrize("change,want", [
    (dict(k_scale=None), -1), (dict(v_scale=None), -1), (dict(k=None), -1),
    (dict(elem_bytes=0), -3), (dict(elem_bytes=-1), -3), (dict(d=32), -3),
    (dict(k_scale=0x50004), -4), (dict(k_scale_strides=(128, 8, 2)), -4),
    (dict(v_scale_strides=(-128, 8, 4)), -4), (dict(k_strides=(1024, 64, 24)), -4),
    (dict(k_descale=0x10001), -4),
    (dict(k_strides=(1024, 32, 32)), -2), (dict(v_scale_strides=(128, 4, 4)), -2),
    (dict(k_scale_strides=(64, 8, 4)), -2),
])
def test_bad_caches_in_4_bits_are_refused(lib, change, want):
    assert lib.cp_paged_append(*append_args(int4(**change))) == want
    assert lib.cp_paged_attn_decode(*decode_args(int4(**change))) == want


def test_a_cache_in_4_bits_passes_the_checks(lib):
    """What fails next is the workspace's size, and the append's rotation."""
    for change in ({}, dict(k_descale=0x10000, v_descale=0x10000),
                   dict(k_scale_strides=(128, 4, 64))):       # head-major scales
        assert lib.cp_paged_attn_decode(*decode_args(int4(**change), n=1000)) == -6
        assert lib.cp_paged_append(*append_args(int4(**change), rot=8)) == -3


def test_the_scales_of_other_caches_are_not_read(lib):
    cache = dict(k_scale=0x3, v_scale=0x5)
    assert lib.cp_paged_attn_decode(*decode_args(cache, n=1000)) == -6
    assert cache_struct(**cache).k_scale == 3


def test_tensors_of_another_type_are_refused():
    """Shapes and types are checked before the device is asked for anything else."""
    q = torch.zeros((1, 1, 2, 64), dtype=torch.bfloat16)
    t = torch.zeros((1, 1), dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        pkg.paged_attn_decode(q, t, t, t, t, k_scale=t, v_scale=t)
