"""GPU parity of the 8-bit paged cache against the fp64 oracle (oracle/paged_fp8.py, and oracle/paged.py on the rows that a
cache stands for).

Every slot that no length reaches holds random bytes and codes, NaN among them; pages are shuffled and some belong to nobody.

Bounds, derived from the roundings on the way:
  append, read  exact: bytes, codes and bf16 rows are compared bit for bit;
  O    the probabilities are rounded (to bf16, or to three e5m2 numbers whose sum is as near; 2^-8 sum_j P |v|) and so is O
       (2^-8 |O|); 5% more for the fp32 sums, which also holds what is below 2^-24 of a row's largest P |v|;
  LSE  a score is an fp32 sum of d exact products: off by at most d 2^-23 c sum |q k|; q may be held as two e4m3 numbers, exact
       but for elements below 2^-14 of the row's largest, which are off by at most 2^-22 of that: sqrt(d) 2^-22 c |q| |k| in all;
       the sum of the exponentials adds 2^-18.
"""

import math

import numpy as np
import pytest
import torch

import exact_io_aware_38_gb300 as fa
from exact_io_aware_38_gb300 import build
from oracle import paged, paged_fp8 as p8
from test_gpu_paged import FIXED, HEADS, PACKED, Problem

pytestmark = pytest.mark.gpu

NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    fa.lib()
    assert torch.cuda.is_available(), "GPU tests need CUDA"


class Problem8(Problem):
    """A seeded batch over an 8-bit cache; k and v are the bf16 rows that its bytes and codes stand for."""

    def __init__(self, lk, lq, H=4, Hkv=2, d=128, page=16, seed=0, layout="phd", spread=0.7, **kw):
        super().__init__(lk, lq, H, Hkv, d, page, seed=seed, **kw)
        g = torch.Generator().manual_seed(500 + seed)
        for x, s in ((self.k, 0.2), (self.v, spread), (self.k_new, 0.2), (self.v_new, spread)):
            x *= torch.exp(s * torch.randn((*x.shape[:-1], 1), generator=g)).to(torch.bfloat16)
        self.layout, self.g = layout, g
        self.quantise()

    def quantise(self):
        """The bytes and codes of k and v (changed by a test, perhaps), and k and v as read back from them."""
        (ky, kc), (vy, vc) = (p8.quantise(self.np(x)) for x in (self.k, self.v))
        dead = ~self.live.numpy()
        r = np.random.default_rng(int(torch.randint(1 << 30, (1,), generator=self.g)))
        ky[dead], vy[dead] = r.integers(0, 256, (2, int(dead.sum()), *ky.shape[2:]), dtype=np.uint8)
        kc[dead], vc[dead] = r.choice([0, 1, 120, 130, 247, 255], (2, int(dead.sum()), ky.shape[2])).astype(np.uint8)
        self.codes = np.ascontiguousarray(np.stack([kc, vc], -1).transpose(0, 2, 1, 3))
        self.ky, self.vy = ky, vy
        for name, y, which in (("k", ky, 0), ("v", vy, 1)):
            x = torch.tensor(p8.cache_values(y, self.codes, which))
            x[~self.live] = NAN
            setattr(self, name, x.to(torch.bfloat16))
        self.ck, self.cv = self.bytes(ky), self.bytes(vy)
        self.ccodes = torch.tensor(self.codes).cuda()

    def bytes(self, y):
        """The cache on the GPU, its [page, slot, head, d] view over another order or with gaps between rows."""
        t = torch.tensor(y)
        if self.layout == "hpd":
            t = t.transpose(1, 2).contiguous().cuda().transpose(1, 2)
        elif self.layout == "gap":
            wide = torch.full((t.shape[0], t.shape[1] + 1, t.shape[2], t.shape[3] + 16), 127, dtype=torch.uint8)
            wide[:, :-1, :, :-16] = t
            t = wide.cuda()[:, :-1, :, :-16]
        else:
            t = t.cuda()
        return t.view(torch.float8_e4m3fn)

    @property
    def cache(self):
        return self.ck, self.cv, self.ccodes, self.ctable, self.clen

    def attend(self, causal, **kw):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        o, lse = fa.fwd_paged_fp8(self.cq, *self.cache, causal=causal, scale=self.scale, status=status, **self.tokens, **kw)
        torch.cuda.synchronize()
        assert int(status.item()) == 0, fa.fa_status_string(int(status.item()))
        return o, lse

    def score_error(self):
        kmax = np.nan_to_num(np.linalg.norm(self.np(self.k), axis=-1)).max()
        qmax = np.linalg.norm(self.np(self.q), axis=-1).max()
        return (self.d * 2.0**-23 + math.sqrt(self.d) * 2.0**-22) * self.scale * kmax * qmax


def raw(t):
    return t.view(torch.uint8).cpu().numpy()


# ------------------------------------------------------------------------------------------- append and read


def special_rows(x, seed):
    """Rows of every kind among x's: zeros, NaN, infinities, tiny and huge numbers, exact powers and ties."""
    r = np.random.default_rng(seed)
    flat = x.view(-1, x.shape[-1])
    for i in range(flat.shape[0]):
        kind = int(r.integers(0, 14))
        if kind == 0:
            flat[i] = 0.0
        elif kind == 1:
            flat[i, int(r.integers(x.shape[-1]))] = float(r.choice([math.inf, -math.inf, NAN]))
        elif kind == 2:
            flat[i] *= 2.0 ** float(r.integers(-100, -60))
        elif kind == 3:
            flat[i] *= 2.0 ** float(r.integers(60, 120))
        elif kind == 4:
            flat[i] = torch.tensor(2.0 ** r.integers(-12, 1, x.shape[-1])).to(x.dtype) * (1 + torch.tensor(r.integers(0, 16, x.shape[-1]) / 16)).to(x.dtype)
        elif kind == 5:
            flat[i] = 0.0
            flat[i, -1] = -(2.0**-133)
        elif kind == 6:
            flat[i, 0] = 2.0**127 * 1.9921875  # (its largest number)


def check_append(p, **kw):
    ky, vy, codes = p.ky.copy(), p.vy.copy(), p.codes.copy()
    p8.append(p.np(p.k_new), p.np(p.v_new), ky, vy, codes, p.table.numpy(), p.lk, p.cu)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    fa.paged_append_fp8(p.k_new.cuda(), p.v_new.cuda(), *p.cache, status=status, **p.tokens, **kw)
    assert int(status.item()) == 0
    for got, want in ((raw(p.ck), ky), (raw(p.cv), vy)):
        assert np.array_equal(p8.TABLE[got], p8.TABLE[want], equal_nan=True)  # (a zero's sign is free)
    assert np.array_equal(p.ccodes.cpu().numpy(), codes)


@pytest.mark.parametrize("heads", [(4, 2, 128), (1, 1, 64), (1, 1, 128), (5, 5, 64), (32, 32, 128), (17, 17, 128), (24, 24, 64)])
@pytest.mark.parametrize("packed", [False, True])
def test_append(packed, heads):
    if packed:
        p = Problem8([40, 3, 0, 200, 77], [40, 1, 0, 131, 5], *heads, page=16, packed=True, seed=1)
    else:
        p = Problem8([40, 11, 200], [5] * 3, *heads, page=32, seed=2)
    special_rows(p.k_new, 3)
    special_rows(p.v_new, 4)
    check_append(p)


@pytest.mark.parametrize("layout", ["hpd", "gap"])
def test_append_and_read_strided(layout):
    p = Problem8([90, 33], [7, 7], 2, 2, 128, page=8, seed=5, layout=layout)
    check_append(p)
    wide = torch.full((2, 2, 7, 128 + 8), 3.0, dtype=torch.bfloat16, device="cuda")  # [B, H, N, d] memory, gaps
    k, v = wide[..., :128].transpose(1, 2), torch.empty(2, 7, 2, 128, dtype=torch.bfloat16, device="cuda")
    rk, rv = fa.paged_read_fp8(k, v, *p.cache)
    assert rk is k and rv is v and (wide[..., 128:] == 3.0).all()
    want = [p8.values(*p8.quantise(p.np(x))) for x in (p.k_new, p.v_new)]
    assert np.array_equal(p.np(k), want[0]) and np.array_equal(p.np(v), want[1])


@pytest.mark.parametrize("heads", [(4, 2, 128), (1, 1, 64), (5, 5, 64), (32, 32, 128), (17, 17, 128), (24, 24, 64)])
@pytest.mark.parametrize("packed", [False, True])
def test_read(packed, heads):
    if packed:
        p = Problem8([40, 3, 0, 200, 77], [40, 1, 0, 131, 5], *heads, page=16, packed=True, seed=6)
    else:
        p = Problem8([40, 11, 200], [9] * 3, *heads, page=8, seed=7)
    special_rows(p.k, 8)
    special_rows(p.v, 9)
    p.quantise()
    k, v = torch.full_like(p.k_new, 7.0).cuda(), torch.full_like(p.v_new, 7.0).cuda()
    wk, wv = p.np(k), p.np(v)
    p8.read(wk, wv, p.ky, p.vy, p.codes, p.table.numpy(), p.lk, p.cu)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    fa.paged_read_fp8(k, v, *p.cache, status=status, **p.tokens)
    assert int(status.item()) == 0
    bf = lambda x: torch.tensor(x).to(torch.bfloat16).double().numpy()  # noqa: E731  (2^128 is bf16's infinity)
    assert np.array_equal(p.np(k), bf(wk), equal_nan=True) and np.array_equal(p.np(v), bf(wv), equal_nan=True)


@pytest.mark.parametrize("heads", [(1, 1, 64), (1, 1, 128), (2, 2, 64), (2, 2, 128), (3, 3, 64), (4, 4, 128), (6, 6, 64)])
@pytest.mark.parametrize("packed", [False, True])
def test_many_rows_of_few_heads(packed, heads):
    """Rows enough that a warp moves several: sequences of none to a few tokens, some with fewer keys than new tokens, one
    whose new tokens lie on no page of the cache."""
    r = np.random.default_rng(heads[2] + heads[0] + packed)
    B = 3001 if packed else 701
    lq = np.minimum(r.integers(0, 8, B) * (r.random(B) < 0.9), 6) if packed else np.full(B, 3)
    lq[-3:] = (9, 0, 2) if packed else 3
    assert lq.sum() > (8192 if packed else 2048)
    lk = lq + r.integers(0, 12, B) - (r.random(B) < 0.05)
    p = Problem8(np.maximum(lk, 0).tolist(), lq.tolist(), *heads, page=8, packed=packed, seed=12)
    lost = int(np.flatnonzero((lk > 8) & (lq > 0) & (lk - lq >= 8))[0])  # (its new tokens are all on its second page)
    p.ctable[lost, 1] = 1 << 20
    ky, vy, codes = p.ky.copy(), p.vy.copy(), p.codes.copy()
    new = p.np(p.k_new), p.np(p.v_new)
    cu = p.cu
    gone = {(lost, i) if cu is None else (int(cu[lost]) + i,) for i in range(int(lq[lost]))}
    keep = [x for x in p8.places(p.table.numpy(), p.lk, int(lq[0]), 8, cu) if x[0] not in gone]
    at = tuple(np.array([x[0] for x in keep]).T)
    page, slot = np.array([x[1] for x in keep]), np.array([x[2] for x in keep])
    for x, cache, which in ((new[0], ky, 0), (new[1], vy, 1)):
        cache[page, slot], c = p8.quantise(x[at])
        codes[page, :, slot, which] = c
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    fa.paged_append_fp8(p.k_new.cuda(), p.v_new.cuda(), *p.cache, status=status, **p.tokens)
    assert int(status.item()) == -6
    for got, want in ((raw(p.ck), ky), (raw(p.cv), vy)):
        assert np.array_equal(p8.TABLE[got], p8.TABLE[want], equal_nan=True)
    assert np.array_equal(p.ccodes.cpu().numpy(), codes)
    k, v = torch.full_like(p.k_new, 7.0).cuda(), torch.full_like(p.v_new, 7.0).cuda()
    wk, wv = p.np(k), p.np(v)
    for w, y, which in ((wk, ky, 0), (wv, vy, 1)):
        w[at] = p8.cache_values(y, codes, which)[page, slot]
    status.zero_()
    fa.paged_read_fp8(k, v, *p.cache, status=status, **p.tokens)
    assert int(status.item()) == -6
    assert np.array_equal(p.np(k), wk) and np.array_equal(p.np(v), wv)


def test_rows_without_a_place_are_reported():
    """More new tokens than keys, and keys past the table: those rows are left on both ways, the others move."""
    p = Problem8([3, 60], [5, 5], 2, 2, 64, page=16, seed=10)
    p.ctable = p.table[:, :3].contiguous().cuda()  # 48 slots: keys 55 .. 59 of the second have none
    ky, vy, codes = p.ky.copy(), p.vy.copy(), p.codes.copy()
    p8.append(p.np(p.k_new), p.np(p.v_new), ky, vy, codes, p.table.numpy()[:, :3], p.lk)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    fa.paged_append_fp8(p.k_new.cuda(), p.v_new.cuda(), *p.cache, status=status)
    assert int(status.item()) == -6 and np.array_equal(p8.TABLE[raw(p.ck)], p8.TABLE[ky], equal_nan=True)
    assert np.array_equal(p.ccodes.cpu().numpy(), codes)
    k, v = torch.full_like(p.k_new, 7.0).cuda(), torch.full_like(p.v_new, 7.0).cuda()
    status.zero_()
    fa.paged_read_fp8(k, v, *p.cache, status=status)
    assert int(status.item()) == -6 and (k[0, :2] == 7.0).all() and (v[1] == 7.0).all()
    assert np.array_equal(p.np(k)[0, 2:], p8.values(*p8.quantise(p.np(p.k_new)))[0, 2:])


def test_bad_pages_of_append_and_read():
    p = Problem8([30, 30], [4, 4], 2, 2, 128, page=16, seed=11)
    before = raw(p.ck).copy()
    for bad in (-1, p.pages, 1 << 20):
        p.ctable[0, 1] = bad  # (the new tokens of the first sequence lie there)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        fa.paged_append_fp8(p.k_new.cuda()[:1], p.v_new.cuda()[:1], p.ck, p.cv, p.ccodes, p.ctable[:1], p.clen[:1], status=status)
        assert int(status.item()) == -6 and np.array_equal(raw(p.ck), before)
        k, v = torch.full_like(p.k_new, 7.0).cuda(), torch.full_like(p.v_new, 7.0).cuda()
        status.zero_()
        fa.paged_read_fp8(k, v, *p.cache, status=status)
        assert int(status.item()) == -6 and (k[0] == 7.0).all() and (v[0] == 7.0).all() and (k[1] != 7.0).any()


# ------------------------------------------------------------------------------------------- attention


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("case", range(len(FIXED)))
def test_attend_fixed(case, heads, causal):
    lk, n = FIXED[case]
    p = Problem8(lk, [n] * len(lk), *heads, page=(16, 64, 8, 128, 32)[(case + heads[0]) % 5], seed=case)
    p.check_attend(*p.attend(causal), causal)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("case", range(len(PACKED)))
def test_attend_packed(case, heads, causal):
    lk, lq = PACKED[case]
    p = Problem8(lk, lq, *heads, page=(32, 256, 16)[case], packed=True, seed=20 + case)
    rows = p.q.shape[0]
    out = torch.full_like(p.cq, NAN)
    lse = torch.full((p.H, rows), 7.0, device="cuda")
    o, l = p.attend(causal, out=out, lse=lse)
    assert o is out and l is lse
    end = int(p.cu[-1])
    assert torch.isnan(o[end:].float()).all() and (l[:, end:] == 7.0).all()  # rows of no sequence stay as they were
    p.check_attend(o, l, causal)


@pytest.mark.parametrize("sms", [1, 2, 3, 7, 64, 400])
@pytest.mark.parametrize("n,heads", [(1, (4, 2, 128)), (3, (16, 2, 64)), (14, (8, 2, 128)), (40, (8, 2, 128)), (90, (6, 2, 64))])
def test_attend_any_division(n, heads, sms):
    """The same work divided among 1 to 400 CTAs: pieces of any length, more CTAs than key tiles included."""
    p = Problem8([1111, 250, 0, 1], [n] * 4, *heads, page=32, seed=n)
    p.check_attend(*p.attend(True, num_sms=sms), True)


@pytest.mark.parametrize("n,heads", [(1, (8, 2, 128)), (3, (8, 2, 64)), (7, (8, 2, 128)), (12, (8, 2, 64))])
@pytest.mark.parametrize("sms", [2, 3, 4, 5])
def test_attend_more_short_units_than_places(n, heads, sms):
    """8 units, of up to 8 tiles, on 2 to 10 places: undivided where they are nearly two a place; packed rows stay in place."""
    for packed in (False, True):
        p = Problem8([900, 130, 0, 128], [n, 1, n, 0] if packed else [n] * 4, *heads, page=32, packed=packed, seed=n)
        p.check_attend(*p.attend(True, num_sms=sms), True)


@pytest.mark.parametrize("B", [500, 600, 1300])
def test_attend_many_sequences(B):
    """More sequences than threads look for a CTA's share, many of them empty, in a packed batch with gaps."""
    r = np.random.default_rng(B)
    lk = r.integers(0, 250, B) * (r.random(B) < 0.4)
    lq = r.integers(0, 6, B) * (r.random(B) < 0.5)
    p = Problem8(lk.tolist(), lq.tolist(), 8, 2, 64, page=32, packed=True, seed=13)
    for sms in (1, 152):
        p.check_attend(*p.attend(True, num_sms=sms), True)


@pytest.mark.parametrize("B,heads", [(B, (65, 1, 64)) for B in (31, 64, 65, 96, 256, 321, 600)]
                         + [(97, (65, 1, 128)), (97, (130, 2, 128)), (70, (330, 5, 64))])
def test_read_back_of_many_sequences(B, heads):
    """More sequences than a warp that reads keys back looks at in a step, many of them empty or without new tokens."""
    r = np.random.default_rng(B)
    for packed in (False, True):
        lk = r.integers(0, 140, B) * (r.random(B) < 0.4)
        lq = r.integers(1, 4, B) * (r.random(B) < 0.5) if packed else np.full(B, 3)
        lq[B // 2] = 3
        p = Problem8(lk.tolist(), lq.tolist(), *heads, page=32, packed=packed, seed=14)
        for sms in (1, 152):
            p.check_attend(*p.attend(True, num_sms=sms), True)


@pytest.mark.parametrize("n", [1, 4, 70])
@pytest.mark.parametrize("layout", ["hpd", "gap"])
@pytest.mark.parametrize("d", [64, 128])
def test_attend_strided_cache_and_rows(d, layout, n):
    p = Problem8([259, 90], [n, n], 6, 2, d, page=16, seed=3, layout=layout)
    wide = torch.full((2, 6, n, d + 16), NAN, dtype=torch.bfloat16, device="cuda")  # [B, H, N, d] memory, gaps
    view = wide[..., :d].transpose(1, 2)
    view.copy_(p.cq)
    p.cq = view
    out = torch.full_like(wide, 3.0)
    o, lse = p.attend(True, out=out[..., :d].transpose(1, 2))
    assert (out[..., d:] == 3.0).all()
    p.check_attend(o, lse, True)


@pytest.mark.parametrize("n", [1, 3, 50])
@pytest.mark.parametrize("heads", [(96, 1, 64), (131, 1, 64), (128, 1, 128), (65, 1, 128), (96, 2, 64)])
def test_many_heads_per_kv_head(heads, n):
    p = Problem8([300, 77], [n, n], *heads, page=32, seed=14)
    p.check_attend(*p.attend(True), True)


@pytest.mark.parametrize("n,heads", [(48, (8, 2, 128)), (49, (8, 2, 128)), (32, (8, 2, 64)), (33, (8, 2, 64)), (84, (3, 1, 64)),
                                     (85, (3, 1, 64)), (36, (7, 1, 128)), (37, (7, 1, 128)), (4, (37, 1, 64)), (5, (37, 1, 64))])
def test_most_rows_of_one_way_and_least_of_the_other(n, heads):
    p = Problem8([700, 130, 0, n], [n] * 4, *heads, page=32, seed=n)
    for sms in (3, 152):
        p.check_attend(*p.attend(True, num_sms=sms), True)


@pytest.mark.parametrize("n,heads", [(1, (142, 2, 128)), (2, (142, 2, 64)), (2, (128, 1, 128)), (1, (256, 1, 64)), (1, (257, 1, 64)),
                                     (1, (390, 3, 64)), (2, (65, 1, 128))])
@pytest.mark.parametrize("sms", [1, 5, 152])
def test_parts_of_a_group_of_heads(n, heads, sms):
    """More than 64 heads on a K/V head: units of some of them, whole and divided, rows of other units left alone."""
    for packed in (False, True):
        p = Problem8([1111, 250, 0, 129], [n, 1, 0, n] if packed else [n] * 4, *heads, page=32, packed=packed, seed=n)
        out = torch.full_like(p.cq, 3.0)
        p.check_attend(*p.attend(True, num_sms=sms, out=out), True)
        if packed:
            assert (out[int(p.cu[-1]):] == 3.0).all()


def test_page_sizes_at_both_ends():
    for page, lk in ((8, [1000, 9]), (65536, [700, 0]), (1024, [1025, 1024])):
        for n in (1, 33):
            p = Problem8(lk, [n, n], 4, 2, 64, page=page, seed=15, extra_pages=0 if page > 10_000 else 2)
            p.check_attend(*p.attend(True), True)


@pytest.mark.parametrize("d", [64, 128])
def test_attend_extreme_scores(d):
    """Scores far apart in every direction: a row max that grows late and by a lot, one that never does, and keys that
    outweigh all others; a softmax is one-hot there, so O is one value row."""
    for n in (1, 6, 130):
        for sign in (1.0, -1.0):
            p = Problem8([900, 400], [n, n], 4, 2, d, page=16, seed=5, std=1.0, spread=0.0)
            grow = torch.linspace(-6.0, 6.0, 900)
            for b in range(2):
                j = torch.arange(p.lk[b])
                p.k[p.table[b][j // 16].long(), j % 16] *= (sign * grow[:p.lk[b]]).to(torch.bfloat16)[:, None, None]
            p.q = (p.q.float() * 8).to(torch.bfloat16)
            p.cq = p.q.cuda()
            p.quantise()
            p.check_attend(*p.attend(True), True)


@pytest.mark.parametrize("small,large", [(None, 60), (None, 115), (-60, 60), (-70, 100), (0, 113)])
@pytest.mark.parametrize("n,sms", [(1, None), (6, 1), (20, 3), (32, 1), (130, None)])
@pytest.mark.parametrize("where", ["first", "last", "all over"])
def test_row_sums_do_not_depend_on_the_values(where, n, sms, small, large):
    """Keys whose values are 2^large, others whose values are 2^small (or zeros), and ordinary ones between them: all of them count in the
    row sums by their scores alone. The large ones come before all others, behind them, or among them."""
    for d in (64, 128):
        p = Problem8([700, 390], [n, n], 4, 2, d, page=16, seed=36, spread=0.0)
        for b in range(2):
            L = p.lk[b]
            j = torch.arange(L)
            row = (p.table[b][j // 16].long(), j % 16)
            big = {"first": j < 9, "last": j >= L - n - 9, "all over": j % 41 == 3}[where]
            for at, by in (((j % 2 == 0) & ~big, 0.0 if small is None else 2.0**small), (big, 2.0**large)):
                p.v[row[0][at], row[1][at]] *= by
        p.quantise()
        p.check_attend(*p.attend(True, num_sms=sms), True)


@pytest.mark.parametrize("n", [1, 6, 130])
@pytest.mark.parametrize("d", [64, 128])
def test_values_of_very_different_sizes(d, n):
    """Keys that take most of the attention with values 2^-20 as large as the others' (or none at all), others with values of
    2^20: the sum of the exponentials and the product need another reference each."""
    p = Problem8([700, 260], [n, n], 4, 2, d, page=16, seed=21, spread=0.0)
    for b in range(2):
        j = torch.arange(p.lk[b])
        row = (p.table[b][j // 16].long(), j % 16)
        p.v[row[0][::7], row[1][::7]] *= 2.0**-20
        p.v[row[0][::5], row[1][::5]] = 0.0
        p.v[row[0][3::11], row[1][3::11]] *= 2.0**20
        p.k[row[0][::35], row[1][::35]] = p.q.view(-1, 4, d)[0, 0] * 2.0  # (a key that one head's rows look at)
        p.k[row[0][4::9], row[1][4::9]] = 0.0
    p.quantise()
    p.check_attend(*p.attend(True), True)
    p.v[p.live] = 0.0  # nothing but zeros: O is 0, LSE what it was
    p.quantise()
    o, lse = p.attend(True)
    p.check_attend(o, lse, True)


@pytest.mark.parametrize("n", [1, 6, 130])
def test_many_small_weights_beside_a_large_one(n):
    """One key holds half of the attention, thousands of others (with values of one sign) the rest: no share is too small."""
    L = 20_000
    p = Problem8([L], [n], 2, 1, 64, page=64, seed=22, spread=0.0)
    p.k[p.live] = 0.0
    p.v[p.live] = p.v[p.live].abs()
    p.q[:] = 1.0
    j = 12_345
    p.k[p.table[0, j // 64].long(), j % 64] = math.log(L) / (64 * p.scale)
    p.cq = p.q.cuda()
    p.quantise()
    p.check_attend(*p.attend(False), False)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,n", [(8, 1), (4, 4), (8, 4), (8, 8)])
@pytest.mark.parametrize("L", [1 << 18, (1 << 20) + 77])
def test_precision_of_one_long_piece(L, G, n, d):
    """One CTA goes through all keys of a head: the first weighs about as much as all the others, which are equal, each row's by another
    factor. Half of O is the first key's share, half the others'. Off by: 1.25 x 2^-9 of a probability, or 1.25 x 2^-23 where the largest
    is 2^7; 2^-8 for O in bf16; L / 32 sums in fp32, each off by up to 2^-23 of a sum that is half the last one in the mean; and
    L / 128 of a lane's row sum, each off by up to 2^-24 of one that may be near the last from the beginning."""
    P, rows = 4096, G * n
    pages = -(-L // P)
    one = int(np.flatnonzero(p8.TABLE == 1.0)[0])
    k, v = (torch.zeros(pages, P, 2, d, dtype=torch.uint8, device="cuda") for _ in range(2))
    k[..., 1] = one
    v[..., d // 2:] = one
    k[0, 0, :, 1], k[0, 0, :, 0] = 0, one
    v[0, 0, :, d // 2:], v[0, 0, :, :d // 2] = 0, one
    codes = torch.full((pages, 2, P, 2), 127, dtype=torch.uint8, device="cuda")
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None].contiguous()
    q = torch.zeros(1, n, 2, G, d, dtype=torch.float64)
    q[..., 0] = torch.tensor([math.log(L) + math.log(2) * (2 * i / rows - 1) for i in range(rows)]).view(1, n, 1, G)
    q = q.view(1, n, 2 * G, d).to(torch.bfloat16)
    e4 = torch.float8_e4m3fn
    o, lse = fa.fwd_paged_fp8(q.cuda(), k.view(e4), v.view(e4), codes, table, torch.tensor([L], dtype=torch.int32, device="cuda"),
                              scale=1.0, num_sms=1)
    x = q[0, :, :, 0].double()
    first, total = torch.exp(x), torch.exp(x) + (L - 1)
    small = torch.clamp(1.25 * 2.0**-23 * first / 2**7, min=1.25 * 2.0**-9)
    tol = (small + 2.0**-8 + L / 64 * 2.0**-23 + L / 128 * 2.0**-24)[..., None]
    o = o[0].double().cpu()
    for got, want in ((o[..., :d // 2], first / total), (o[..., d // 2:], (L - 1) / total)):
        assert ((got - want[..., None]).abs() <= tol * want[..., None]).all()
    assert ((lse[0].t().double().cpu() - torch.log(total)).abs() <= 2.0**-18 + 16 * 2.0**-22 + L / 128 * 2.0**-24).all()


def test_rows_and_keys_of_extreme_sizes():
    """q of 2^40 against keys of 2^-40 and the reverse, beside rows of zeros: the scores are ordinary numbers."""
    for n in (1, 5, 100):
        for e in (40, -40):
            p = Problem8([300, 131], [n, n], 4, 2, 128, page=16, seed=23)
            p.q = (p.q.float() * 2.0**e).to(torch.bfloat16)
            p.q[0, 0, 0] = 0.0
            p.k = (p.k.float() * 2.0**-e).to(torch.bfloat16)
            p.cq = p.q.cuda()
            p.quantise()
            p.check_attend(*p.attend(True), True)


def test_query_rows_with_outliers():
    """A channel 2^12 times the others, whose own products still count: keys are small in it."""
    for n in (1, 9, 80):
        p = Problem8([500], [n], 4, 2, 128, page=16, seed=24)
        p.q[..., 17] *= 2.0**12
        p.k[..., 17] = 0.0
        p.cq = p.q.cuda()
        p.quantise()
        ref = paged.attention(p.np(p.q), p.np(p.k), p.np(p.v), p.table.numpy(), p.lk, p.scale, True)
        o, lse = p.attend(True)
        ro, rl, a = ref[0]
        # an element is off by at most 2^-22 of the outlier: 2^-22 |q|_max c |k|_1, next to the fp32 sum's d 2^-23 c |q'| |k|
        q1 = p.np(p.q).copy()
        q1[..., 17] = 0.0
        kn = np.nan_to_num(p.np(p.k))
        tol = p.scale * (2.0**-22 * np.abs(p.np(p.q)).max() * np.abs(kn).sum(-1).max()
                         + 128 * 2.0**-23 * np.linalg.norm(q1, axis=-1).max() * np.linalg.norm(kn, axis=-1).max()) + 2.0**-18
        assert np.abs(p.np(lse)[0] - rl).max() <= tol
        assert (np.abs(p.np(o)[0] - ro) <= (1.05 * 2.0**-8 + 2 * tol) * (a + np.abs(ro))).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,sms", [(1, 152), (1, 3), (1, 1), (10, 152), (10, 3), (60, 152), (600, 152), (600, 5)])
@pytest.mark.parametrize("what", ["key", "value", "byte"])
def test_nan_is_seen_however_the_work_is_divided(what, n, sms, d):
    """A key or value of code 255 makes O (and LSE) of the rows that see it NaN, a NaN in a query row those of the row; the rest
    is as without. So does a key's byte of NaN."""
    L, j, bad_row = 1100, 700, n // 3
    p = Problem8([L, 300], [n, min(n, 300)], 8, 2, d, page=16, seed=31, packed=True)
    tol = p.score_error() + 2.0**-18
    ref = p.check_attend(*p.attend(True, num_sms=sms), True)
    page = p.ctable[0, j // 16].long()
    if what == "byte":
        p.ck.view(torch.uint8)[page, j % 16, 1, 5] = 127
    else:
        p.ccodes[page, 1, j % 16, 0 if what == "key" else 1] = 255
        (p.ck if what == "key" else p.cv).view(torch.uint8)[page, j % 16, 1] = 0
    p.cq[bad_row, 2, 7] = NAN
    o, lse = p.attend(True, num_sms=sms)
    end = int(p.cu[-1])
    bad = torch.zeros(end, 8, dtype=torch.bool, device="cuda")
    bad[bad_row, 2] = True
    bad[:n, 4:] = (torch.arange(n, device="cuda") + L - n >= j)[:, None]
    assert torch.isnan(o[:end][bad]).all() and torch.isnan(lse[:, :end].t()[bad]).all()
    ro, rl, a = np.concatenate([x[0] for x in ref]), np.concatenate([x[1].T for x in ref]), np.concatenate([x[2] for x in ref])
    good = ~bad.cpu().numpy()
    assert (np.abs(p.np(o)[:end] - ro) <= 1.05 * 2.0**-8 * (a + np.abs(ro)))[good].all()
    assert (np.abs(p.np(lse)[:, :end].T - rl) <= tol)[good].all()


def test_infinities_in_a_query_row():
    for n in (1, 70):
        p = Problem8([200], [n], 4, 2, 64, page=16, seed=32)
        ref = p.check_attend(*p.attend(True), True)
        p.cq[0, 0, 1, 3] = math.inf
        o, lse = p.attend(True)
        assert torch.isnan(o[0, 0, 1]).all() and torch.isnan(lse[0, 1, 0])
        keep = np.ones((n, 4), dtype=bool)
        keep[0, 1] = False
        ro, rl, a = ref[0]
        assert (np.abs(p.np(o)[0] - ro) <= 1.05 * 2.0**-8 * (a + np.abs(ro)))[keep].all()


@pytest.mark.parametrize("n", [1, 70, 200])
def test_infinity_that_makes_all_scores_minus_infinity(n):
    """NaN, or a row without keys; the other rows are as without it."""
    p = Problem8([200], [n], 4, 2, 64, page=16, seed=33)
    p.k[..., 3] = -1.0 - p.k[..., 3].abs()
    p.quantise()
    ref = p.check_attend(*p.attend(False), False)
    p.cq[0, 0, 1, 3] = math.inf
    o, lse = p.attend(False)
    got, at = o[0, 0, 1].float(), float(lse[0, 1, 0])
    assert (bool(torch.isnan(got).all()) and math.isnan(at)) or (bool((got == 0).all()) and at == -math.inf)
    keep = np.ones((n, 4), dtype=bool)
    keep[0, 1] = False
    ro, rl, a = ref[0]
    assert (np.abs(p.np(o)[0] - ro) <= 1.05 * 2.0**-8 * (a + np.abs(ro)))[keep].all()


def test_attend_shared_pages_and_bound():
    """Two sequences share their first pages; a bound above the longest length changes nothing, one below cuts."""
    for n in (2, 70):
        p = Problem8([200, 200], [n, n], 4, 2, 128, page=16, seed=6)
        p.table[1, :8] = p.table[0, :8]
        p.ctable = p.table.cuda()
        p.check_attend(*p.attend(True, max_seqlen_k=10_000), True)
        p.lk = [96, 96]
        p.check_attend(*p.attend(True, max_seqlen_k=96), True)


@pytest.mark.parametrize("n", [1, 70])
def test_attend_lengths_past_the_table_and_below_zero_are_clamped(n):
    p = Problem8([64, 64, 0], [n] * 3, 4, 2, 128, page=16, seed=7)
    p.ctable = p.table[:, :4].contiguous().cuda()
    p.clen = torch.tensor([1 << 30, 64, -5], dtype=torch.int32, device="cuda")
    p.check_attend(*p.attend(False), False)


@pytest.mark.parametrize("n", [1, 40])
def test_bad_page_is_reported_and_stays_in_bounds(n):
    for bad in (-1, 1 << 20):
        p = Problem8([100, 300], [n, n], 4, 2, 128, page=16, seed=8)
        good = p.attend(True)
        p.ctable[1, 3] = bad
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        o, lse = fa.fwd_paged_fp8(p.cq, *p.cache, causal=True, scale=p.scale, status=status)
        assert int(status.item()) == -6
        assert torch.equal(o[0], good[0][0]) and torch.equal(lse[0], good[1][0])  # the other sequence is sound


@pytest.mark.parametrize("n", [1, 40])
def test_cache_of_more_than_2_32_elements(n):
    """Pages at both ends of a cache whose offsets pass 32 bits: attention, reading and appending."""
    Hkv, d, P = 2, 128, 64
    pages = (1 << 32) // (P * Hkv * d) + 40
    p = Problem8([400], [n], 4, Hkv, d, page=P, seed=9)
    used = -(-400 // P)
    big = [torch.zeros((pages, P, Hkv, d), dtype=torch.uint8, device="cuda") for _ in range(2)]
    codes = torch.zeros((pages, Hkv, P, 2), dtype=torch.uint8, device="cuda")
    at = torch.tensor([pages - 1, 0, pages - 3, 1, pages // 2, pages - 2, 2], dtype=torch.int32)[:used]
    src = p.table[0, :used].long()
    for b, t in zip((*big, codes), (p.ck.view(torch.uint8), p.cv.view(torch.uint8), p.ccodes)):
        b[at.long().cuda()] = t[src.cuda()]
    ref = p.attend(True)
    p.ctable[0, :used] = at.cuda()
    p.ck, p.cv, p.ccodes = big[0].view(torch.float8_e4m3fn), big[1].view(torch.float8_e4m3fn), codes
    o, lse = p.attend(True)
    assert torch.equal(o, ref[0]) and torch.equal(lse, ref[1])
    fa.paged_append_fp8(p.k_new.cuda(), p.v_new.cuda(), *p.cache)
    k, v = torch.empty_like(p.k_new).cuda(), torch.empty_like(p.v_new).cuda()
    fa.paged_read_fp8(k, v, *p.cache)
    want = [p8.values(*p8.quantise(p.np(x))) for x in (p.k_new, p.v_new)]
    assert np.array_equal(p.np(k), want[0]) and np.array_equal(p.np(v), want[1])


def test_chunks_in_rounds_through_one_workspace():
    """A bound by which one sequence's keys take the whole workspace: the sequences go through it in turn."""
    for packed in (False, True):
        lq = [70, 1, 200] if packed else [70] * 3
        p = Problem8([300, 150, 1000], lq, 8, 2, 128, page=1024, seed=33, packed=packed)
        wide = torch.full((3, 1 << 10), -7, dtype=torch.int32)
        wide[:, :p.table.shape[1]] = p.table
        p.ctable = wide.cuda()
        assert (1 << 20) * 2 * 128 * 4 == 1 << 30  # by the table's width a sequence may have 2^20 keys
        p.check_attend(*p.attend(True), True)


@pytest.mark.parametrize("packed", [False, True])
def test_many_sequences_in_rounds_of_two(packed):
    """Nine sequences, two of which the workspace holds by the table's width: five rounds, the last of one sequence; packed, those of few
    tokens go another way, and one round has no tokens left."""
    lq = [70, 200, 1, 0, 65, 3, 129, 66, 90] if packed else [70] * 9
    p = Problem8([300, 200, 1000, 50, 65, 128, 131, 700, 90], lq, 16, 8, 128, page=1024, seed=35, packed=packed)
    wide = torch.full((9, 1 << 7), -7, dtype=torch.int32)
    wide[:, :p.table.shape[1]] = p.table
    p.ctable = wide.cuda()
    assert 2 * ((1 << 17) * 8 * 128 * 4) == 1 << 30
    p.check_attend(*p.attend(True), True)


@pytest.mark.parametrize("heads", [(8, 2, 128), (20, 1, 128), (5, 5, 64), (96, 1, 64), (130, 1, 64), (142, 2, 128)])
def test_prompts_beside_single_tokens(heads):
    """A packed batch in which two kernels share the sequences by their new tokens: none, one, at the limit between them,
    one past it, and prompts; a bound on the keys that makes the batch look large."""
    G = heads[0] // heads[1]
    limit = 4 * (16 // G if G <= 16 else 1) if G <= 64 else 4 // -(-G // 64)
    lq = [1, 300, 0, limit, limit + 1, 1, limit - 1, 90, 2, 0, 1]
    lk = [700, 300, 50, 129, 260, 0, 40, 500, 128, 0, 1]
    p = Problem8(lk, lq, *heads, page=16, seed=34, packed=True)
    wide = torch.full((len(lk), (1 << 26) // (len(lk) * heads[1] * heads[2] * 16) + 1), -7, dtype=torch.int32)
    wide[:, :p.table.shape[1]] = p.table
    p.ctable = wide.cuda()
    out = torch.full_like(p.cq, 3.0)
    for sms in (152, 7):
        o, lse = p.attend(True, num_sms=sms, out=out)
        p.check_attend(o, lse, True)
        assert (o[int(p.cu[-1]):] == 3.0).all()
    p.check_attend(*p.attend(False), False)


# ------------------------------------------------------------------------------------------- as they are used


@pytest.mark.parametrize("heads", [(8, 2, 128), (12, 12, 64)])
def test_prompt_chunks_then_captured_steps_then_reading(heads):
    """Prompts in two packed chunks, then single tokens in a captured graph whose lengths move on the device, then the whole
    sequences read back: outputs against the oracle on the rows that were appended."""
    H, Hkv, d = heads
    P, steps, prompts = 16, 5, [150, 40, 33]
    B = len(prompts)
    total = [n + steps for n in prompts]
    p = Problem8(total, [1] * B, H, Hkv, d, page=P, seed=41)
    p.ck.view(torch.uint8).random_(0, 256)
    p.cv.view(torch.uint8).random_(0, 256)
    p.ccodes.random_(0, 256)
    g = torch.Generator().manual_seed(42)
    bf = lambda *s: (1.3 * torch.randn(s, generator=g)).to(torch.bfloat16)  # noqa: E731
    ks, vs, qs = [bf(n, Hkv, d) for n in total], [bf(n, Hkv, d) for n in total], [bf(n, H, d) for n in total]
    scale = 1 / math.sqrt(d)
    kb, vb = ([torch.tensor(p8.values(*p8.quantise(x.double().numpy()))) for x in y] for y in (ks, vs))

    def want(b, lo, hi):  # rows lo .. hi of sequence b
        out = []
        for h in range(H):
            s = paged.head_scores(qs[b][lo:hi, h].double().numpy(), kb[b][:hi, h // (H // Hkv)].numpy(), scale, True)
            l = paged.row_lse(s)
            out.append((paged.row_probs(s, l) @ vb[b][:hi, h // (H // Hkv)].numpy(), l,
                        paged.row_probs(s, l) @ np.abs(vb[b][:hi, h // (H // Hkv)].numpy())))
        return [np.stack(x, 1) for x in zip(*out)]

    def check(o, lse, b, lo, hi):
        ro, rl, a = want(b, lo, hi)
        assert (np.abs(o.double().cpu().numpy() - ro) <= 1.05 * 2.0**-8 * (a + np.abs(ro))).all()
        assert np.abs(lse.double().cpu().numpy() - rl).max() < 1e-4

    at = [0] * B
    for share in (0.6, 1.0):
        to = [int(n * share) for n in prompts]
        cu = np.cumsum([0] + [t - f for f, t in zip(at, to)])
        tok = dict(cu_seqlens_q=torch.tensor(cu, dtype=torch.int32, device="cuda"), max_seqlen_q=max(t - f for f, t in zip(at, to)))
        cat = lambda x: torch.cat([y[f:t] for y, f, t in zip(x, at, to)]).cuda()  # noqa: E731
        p.clen.copy_(torch.tensor(to))
        fa.paged_append_fp8(cat(ks), cat(vs), *p.cache, **tok)
        o, lse = fa.fwd_paged_fp8(cat(qs), *p.cache, causal=True, max_seqlen_k=max(total), **tok)
        for b in range(B):
            check(o[cu[b]:cu[b + 1]], lse[:, cu[b]:cu[b + 1]].t(), b, at[b], to[b])
        at = to
    k1, v1, q1 = (torch.empty(B, 1, n, d, dtype=torch.bfloat16, device="cuda") for n in (Hkv, Hkv, H))
    out, lse = torch.empty_like(q1), torch.empty(B, H, 1, device="cuda")

    def step():
        p.clen.add_(1)
        fa.paged_append_fp8(k1, v1, *p.cache)
        fa.fwd_paged_fp8(q1, *p.cache, causal=True, max_seqlen_k=max(total), out=out, lse=lse)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        k1.zero_(), v1.zero_(), q1.zero_()
        step()  # (a warm-up, undone below)
    torch.cuda.current_stream().wait_stream(side)
    p.clen.sub_(1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(steps):
        for t, x in ((k1, ks), (v1, vs), (q1, qs)):
            t.copy_(torch.stack([y[n + i:n + i + 1] for y, n in zip(x, prompts)]))
        graph.replay()
        for b in range(B):
            check(out[b], lse[b].t(), b, prompts[b] + i, prompts[b] + i + 1)
    cu = np.cumsum([0] + total)
    tok = dict(cu_seqlens_q=torch.tensor(cu, dtype=torch.int32, device="cuda"), max_seqlen_q=max(total))
    k, v = (torch.empty(int(cu[-1]), Hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    fa.paged_read_fp8(k, v, *p.cache, **tok)
    assert torch.equal(k.cpu().double(), torch.cat(kb)) and torch.equal(v.cpu().double(), torch.cat(vb))


@pytest.mark.parametrize("n", [1, 40])
def test_two_captured_graphs_at_once_and_repeats(n):
    """Two graphs on two streams, each with a workspace of its own, give what single calls give, every time the same bits."""
    ps = [Problem8([900, 300, 5], [n] * 3, 8, 2, 128, page=16, seed=50 + i) for i in range(2)]
    refs = [p.attend(True) for p in ps]
    outs, graphs, streams = [], [], [torch.cuda.Stream() for _ in ps]
    for p in ps:
        nbytes = fa.fa_fwd_paged_fp8_workspace_bytes(fa.PagedProblem(
            3, 8, 2, 128, 16, p.pages, p.width, p.ctable.data_ptr(), p.clen.data_ptr(), n, p.width * 16, None, 0, 1, p.scale), 152)
        ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
        o, lse = torch.empty_like(p.cq), torch.empty(3, 8, n, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(3):
                fa.fwd_paged_fp8(p.cq, *p.cache, causal=True, scale=p.scale, out=o, lse=lse, workspace=ws, num_sms=152)
        outs.append((o, lse, ws))
        graphs.append(g)
    for _ in range(5):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for (o, lse, _), ref in zip(outs, refs):
        assert torch.equal(o, ref[0]) and torch.equal(lse, ref[1])


def test_another_stream():
    p = Problem8([500, 77], [3, 3], 8, 2, 128, page=16, seed=60)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    kn, vn = p.k_new.cuda(), p.v_new.cuda()
    torch.cuda.synchronize()
    fa.paged_append_fp8(kn, vn, *p.cache, stream=st)
    o, lse = fa.fwd_paged_fp8(p.cq, *p.cache, causal=True, scale=p.scale, stream=st.cuda_stream)
    k, v = fa.paged_read_fp8(torch.empty_like(kn), torch.empty_like(vn), *p.cache, stream=st)
    st.synchronize()
    p8.append(p.np(p.k_new), p.np(p.v_new), p.ky, p.vy, p.codes, p.table.numpy(), p.lk)
    p.k, p.v = (torch.tensor(p8.cache_values(y, p.codes, w)).to(torch.bfloat16) for w, y in enumerate((p.ky, p.vy)))
    p.check_attend(o, lse, True)
    assert np.array_equal(p.np(k), p8.values(*p8.quantise(p.np(p.k_new))))


def test_no_tokens_and_no_sequences():
    p = Problem8([50], [1], 4, 2, 64, page=16, seed=61)
    o, lse = fa.fwd_paged_fp8(p.cq[:, :0], *p.cache)
    assert o.shape == (1, 0, 4, 64) and lse.shape == (1, 4, 0)
    none = torch.empty(0, 1, 2, 64, dtype=torch.bfloat16, device="cuda")
    before = raw(p.ck).copy()
    fa.paged_append_fp8(none, none, p.ck, p.cv, p.ccodes, p.ctable[:0], p.clen[:0])
    fa.paged_read_fp8(none, none, p.ck, p.cv, p.ccodes, p.ctable[:0], p.clen[:0])
    assert np.array_equal(raw(p.ck), before)
