"""Pins of the paged-cache oracle against the attention oracle and closed forms (CPU)."""

import numpy as np
import pytest

import oracle
from oracle import paged


def problem(seed, lk, lq, H=4, Hkv=2, d=8, P=4, packed=False):
    r = np.random.default_rng(seed)
    width = max(-(-max(n, 1) // P) for n in lk) + 1
    table = r.permutation(len(lk) * width).reshape(len(lk), width).astype(np.int32)
    k, v = r.normal(size=(len(lk) * width, P, Hkv, d)), r.normal(size=(len(lk) * width, P, Hkv, d))
    cu = np.cumsum([0] + list(lq)) if packed else None
    q = r.normal(size=(cu[-1], H, d)) if packed else r.normal(size=(len(lk), lq[0], H, d))
    return q, k, v, table, cu


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("lk,lq,packed", [([9, 5, 12], [3, 1, 4], True), ([7, 7], [2, 2], False), ([3, 0], [5, 2], True)])
def test_attention_is_the_attention_oracle_on_gathered_keys(lk, lq, packed, causal):
    q, k, v, table, cu = problem(1, lk, lq, packed=packed)
    for b, (o, lse, a) in enumerate(paged.attention(q, k, v, table, lk, 0.3, causal, cu)):
        x = paged.new_rows(q, b, cu).transpose(1, 0, 2)[None]
        kk = np.stack([paged.keys_of(k, table, lk[b], b, h) for h in range(2)])[None]
        vv = np.stack([paged.keys_of(v, table, lk[b], b, h) for h in range(2)])[None]
        if lk[b] == 0:
            assert (o == 0).all() and np.isneginf(lse).all()
            continue
        ro, rl = oracle.attention_forward(x, kk, vv, 0.3, causal=causal)
        assert np.allclose(o.transpose(1, 0, 2), ro[0], atol=1e-13)
        assert np.array_equal(np.isneginf(lse), np.isneginf(rl[0]))
        assert np.allclose(lse[np.isfinite(lse)], rl[0][np.isfinite(lse)], atol=1e-13)
        assert (a >= np.abs(o) - 1e-15).all()


@pytest.mark.parametrize("causal", [False, True])
def test_key_weights_sum_to_the_rows_that_see_a_key(causal):
    lk, lq = [9, 2, 5], [3, 4, 1]
    q, k, v, table, cu = problem(2, lk, lq, packed=True)
    att = paged.attention(q, k, v, table, lk, 0.4, causal, cu)
    w = paged.key_weights(q, k, table, lk, [x[1] for x in att], 0.4, causal, cu)
    for b in range(3):
        live = np.isfinite(att[b][1]).reshape(2, 2, -1).sum((1, 2))
        assert np.allclose(w[b].sum(1), live, atol=1e-12)
    uniform = paged.attention(q * 0, k, v, table, lk, 0.4, False, cu)
    w = paged.key_weights(q * 0, k, table, lk, [x[1] for x in uniform], 0.4, False, cu)
    for b in range(3):  # equal scores: each of the 2 n rows of a K/V head pays every key 1 / L
        assert np.allclose(w[b], 2 * lq[b] / lk[b], atol=1e-12)


def test_append_then_read():
    lk, lq = [6, 5], [2, 5]
    q, k, v, table, cu = problem(3, lk, lq, packed=True)
    w = np.ones((k.shape[0], 2, 4))
    new_k, new_v = np.random.default_rng(4).normal(size=(2, 7, 2, 8))
    before = k.copy()
    paged.append(new_k, new_v, k, v, table, lk, cu, w)
    for h in range(2):
        assert np.array_equal(paged.keys_of(k, table, 6, 0, h)[4:], new_k[:2, h])
        assert np.array_equal(paged.keys_of(k, table, 6, 0, h)[:4], paged.keys_of(before, table, 6, 0, h)[:4])
        assert np.array_equal(paged.keys_of(v, table, 5, 1, h), new_v[2:, h])
    assert w.sum() == w.size - 2 * 7


def test_evict_by_hand():
    table = np.array([[1, 0]], dtype=np.int32)
    k = np.arange(8.0).reshape(2, 4, 1, 1)
    v, w = -k, np.zeros((2, 1, 4))
    for j, x in enumerate([0.5, 2.0, float("nan"), 2.0, 0.5, 7.0]):  # key j: page table[0][j // 4], slot j % 4
        w[table[0][j // 4], 0, j % 4] = x
    kept, n = paged.evict(k, v, w, table, [6], 4, 1)
    assert kept[0, 0].tolist() == [0, 1, 3, 5] and n.tolist() == [4]  # of 0.5 and 0.5 the lower index; 5 is recent
    assert paged.keys_of(k, table, 4, 0, 0)[:, 0].tolist() == [4.0, 5.0, 7.0, 1.0]
    assert [w[1, 0, s] for s in range(4)] == [0.5, 2.0, 2.0, 7.0]
    kept, n = paged.evict(k, v, w, table, [3], 5, 0)
    assert kept[0, 0].tolist() == [0, 1, 2, -1, -1] and n.tolist() == [3]
