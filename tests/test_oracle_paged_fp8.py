"""Pins of the 8-bit cache's oracle (oracle/paged_fp8.py): the number table and the rounding against torch's e4m3 type, the codes
against the definition's cases, and the way there and back against the bound of a rounding."""

import math

import numpy as np
import pytest
import torch

from oracle import paged_fp8 as p8


def test_table_is_torchs():
    theirs = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(p8.TABLE, theirs, equal_nan=True)


def test_rounding_is_torchs():
    """Every number of the format, every middle between two, and a step of fp64 beside each."""
    mid = (p8.TABLE[:126] + p8.TABLE[1:127]) / 2
    x = np.concatenate([p8.TABLE[:127], mid, np.nextafter(mid, 0), np.nextafter(mid, 1e9)])
    x = np.concatenate([x, -x])
    # (torch rounds from fp32: a step beside a middle has to be one there)
    near = np.concatenate([np.nextafter(mid.astype(np.float32), np.float32(0)), np.nextafter(mid.astype(np.float32), np.float32(1e9))])
    theirs = torch.tensor(near).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(p8.TABLE[p8.round_e4m3(near)], theirs)
    exact = np.concatenate([p8.TABLE[:127], mid])
    assert np.array_equal(p8.TABLE[p8.round_e4m3(exact)], torch.tensor(exact).to(torch.float8_e4m3fn).double().numpy())
    y = p8.TABLE[p8.round_e4m3(x)]
    assert (np.abs(y - x) <= np.maximum(2.0**-10, np.abs(x) * 2.0**-4)).all()


@pytest.mark.parametrize("row,code", [([0.0, -0.0], 0), ([1.0, 0.5], 120), ([-1.9921875, 1.0], 120), ([2.0, 0.0], 121),
                                      ([2.0**-73, 0.0], 47), ([2.0**-74, 0.0], 47), ([2.0**-133, 0.0], 47),
                                      ([2.0**127, 1.0], 247), ([math.inf, 1.0], 255), ([1.0, -math.inf], 255),
                                      ([math.nan, 0.0], 255)])
def test_codes(row, code):
    y, c = p8.quantise(np.array([row]))
    assert c[0] == code
    if code == 255:
        assert not y.any() and np.isnan(p8.values(y, c)).all()


def test_there_and_back():
    g = torch.Generator().manual_seed(1)
    x = (torch.randn((500, 64), generator=g) * torch.exp(4 * torch.randn((500, 1), generator=g))).to(torch.bfloat16)
    x = x.double().numpy()
    y, c = p8.quantise(x)
    back = p8.values(y, c)
    top = np.abs(x).max(-1, keepdims=True)
    assert (np.abs(back - x) <= np.maximum(2.0**-4 * np.abs(x), 2.0**-17 * top)).all()
    again, c2 = p8.quantise(back)  # the rows that a cache stands for are bf16 numbers, and stand for themselves
    assert np.array_equal(p8.values(again, c2), back)
    assert np.array_equal(torch.tensor(back).to(torch.bfloat16).double().numpy(), back)


def test_append_and_read():
    """Placement: the last keys of each sequence, per table; rows without a place, or of no sequence, are left."""
    r = np.random.default_rng(2)
    P, Hkv, d = 8, 2, 4
    table = np.array([[3, 0, 5], [1, 4, 2]])
    k_cache, v_cache = (r.integers(0, 100, (6, P, Hkv, d), dtype=np.uint8) for _ in range(2))
    codes = r.integers(100, 130, (6, Hkv, P, 2), dtype=np.uint8)
    old = k_cache.copy()
    cu = np.array([0, 3, 13])
    k, v = r.standard_normal((14, Hkv, d)), r.standard_normal((14, Hkv, d))
    lengths = [10, 9]
    p8.append(k, v, k_cache, v_cache, codes, table, lengths, cu)
    for i, (page, slot) in enumerate([(3, 7), (0, 0), (0, 1)]):
        y, c = p8.quantise(k[i])
        assert np.array_equal(k_cache[page, slot], y) and np.array_equal(codes[page, :, slot, 0], c)
    y, c = p8.quantise(v[4])  # the second sequence's second row: key 0 (its first has no place)
    assert np.array_equal(v_cache[1, 0], y) and np.array_equal(codes[1, :, 0, 1], c)
    assert np.array_equal(k_cache[5], old[5]) and np.array_equal(k_cache[3, :7], old[3, :7])
    kr, vr = np.full(k.shape, 7.0), np.full(v.shape, 7.0)
    p8.read(kr, vr, k_cache, v_cache, codes, table, lengths, cu)
    assert (kr[3] == 7.0).all() and (vr[13] == 7.0).all()
    seen = [0, 1, 2] + list(range(4, 13))
    assert np.array_equal(kr[seen], p8.values(*p8.quantise(k))[seen]) and np.array_equal(vr[seen], p8.values(*p8.quantise(v))[seen])
