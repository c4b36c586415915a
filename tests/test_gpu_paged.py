"""GPU parity of the paged-cache operators against the fp64 oracle (oracle/paged.py).

Every slot that no length reaches holds NaN (keys, values and weights), pages are shuffled and some belong to nobody.

Bounds, derived from the roundings on the way (a rounding to bf16 is off by at most 2^-8 of the value, half a step):
  O    the probabilities are rounded to bf16 (2^-8 sum_j P |v|) and so is O (2^-8 |O|); 5% more for the fp32 sums;
  LSE  a score is an fp32 sum of d products of bf16 values, which are exact: off by at most d 2^-23 c sum |q k|
       (a tensor core's addition need not round to nearest: a whole step each); the sum of the exponentials adds 2^-18;
  W    each term exp(s - LSE) is off by the score's error and half a step of the given LSE, relatively, and the sum by
       2^-23 per 128 terms added in a row, bounded by 2^-16 here.
"""

import math

import numpy as np
import pytest
import torch

import exact_io_aware_38_gb300 as fa
from exact_io_aware_38_gb300 import build
from oracle import paged

pytestmark = pytest.mark.gpu

NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    fa.lib()
    assert torch.cuda.is_available(), "GPU tests need CUDA"


class Problem:
    """A seeded batch: host tensors, and their copies on the GPU."""

    def __init__(self, lk, lq, H=4, Hkv=2, d=128, page=16, packed=False, seed=0, std=1.5, layout="phd", spare=5,
                 extra_pages=3):
        g = torch.Generator().manual_seed(1000 + seed)
        self.lk, self.lq, self.H, self.Hkv, self.d, self.P, self.packed = list(lk), list(lq), H, Hkv, d, page, packed
        B = len(lk)
        used = [-(-n // page) for n in lk]
        self.width = max(max(used), 1) + 1
        self.pages = sum(used) + extra_pages
        order = torch.randperm(self.pages, generator=g).to(torch.int32)
        self.table = torch.full((B, self.width), -7, dtype=torch.int32)  # entries that no length reaches
        at = 0
        for b, n in enumerate(used):
            self.table[b, :n] = order[at:at + n]
            at += n
        bf = lambda *s, std=1.0: (torch.randn(s, generator=g) * std).to(torch.bfloat16)
        self.k, self.v = bf(self.pages, page, Hkv, d, std=std), bf(self.pages, page, Hkv, d)
        self.w = torch.exp(2 * torch.randn((self.pages, Hkv, page), generator=g))
        live = torch.zeros(self.pages, page, dtype=torch.bool)
        for b, n in enumerate(lk):
            j = torch.arange(n)
            live[self.table[b][j // page].long(), j % page] = True
        self.live = live
        self.k[~live], self.v[~live] = NAN, NAN
        self.w.transpose(1, 2)[~live] = NAN
        self.cu = np.cumsum([0] + list(lq)) if packed else None
        lead = (int(self.cu[-1]) + spare,) if packed else (B, lq[0])
        self.q = bf(*lead, H, d, std=std)
        self.k_new, self.v_new = bf(*lead, Hkv, d, std=std), bf(*lead, Hkv, d)
        self.scale = 1.0 / math.sqrt(d)
        dev = lambda t: t.cuda()
        self.ck, self.cv = (self.strided(t, layout) for t in (self.k, self.v))
        self.cw, self.ctable, self.cq = dev(self.w), dev(self.table), dev(self.q)
        self.clen = torch.tensor(self.lk, dtype=torch.int32, device="cuda")
        self.tokens = {}
        if packed:
            self.tokens = dict(cu_seqlens_q=torch.tensor(self.cu, dtype=torch.int32, device="cuda"),
                               max_seqlen_q=max(max(lq), 1))

    @staticmethod
    def strided(t, layout):
        """The cache on the GPU, its [page, slot, head, d] view over another order or with gaps between rows."""
        if layout == "hpd":
            return t.transpose(1, 2).contiguous().cuda().transpose(1, 2)
        if layout == "gap":
            wide = torch.full((t.shape[0], t.shape[1] + 1, t.shape[2], t.shape[3] + 8), NAN, dtype=t.dtype)
            wide[:, :-1, :, :-8] = t
            return wide.cuda()[:, :-1, :, :-8]
        return t.cuda()

    def np(self, t):
        return t.detach().double().cpu().numpy()

    def attend(self, causal, **kw):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        o, lse = fa.fwd_paged(self.cq, self.ck, self.cv, self.ctable, self.clen, causal=causal, scale=self.scale,
                              status=status, **self.tokens, **kw)
        torch.cuda.synchronize()
        assert int(status.item()) == 0, fa.fa_status_string(int(status.item()))
        return o, lse

    def score_error(self):
        """A bound on the error of any fp32 score: d 2^-23 c sum_k |q_k k_k|, the sum by its two norms."""
        kmax = np.nan_to_num(np.linalg.norm(self.np(self.k), axis=-1)).max()
        qmax = np.linalg.norm(self.np(self.q), axis=-1).max()
        return self.d * 2.0**-23 * self.scale * kmax * qmax

    def check_attend(self, o, lse, causal):
        o, lse = self.np(o), self.np(lse)
        ref = paged.attention(self.np(self.q), self.np(self.k), self.np(self.v), self.table.numpy(), self.lk, self.scale,
                              causal, self.cu)
        tol_lse = self.score_error() + 2.0**-18
        for b, (ro, rl, a) in enumerate(ref):
            ob = paged.new_rows(o, b, self.cu)
            lb = lse[b] if self.cu is None else lse[:, self.cu[b]:self.cu[b + 1]]
            assert np.isfinite(ob).all()
            over = np.abs(ob - ro) - 1.05 * 2.0**-8 * (a + np.abs(ro))
            assert over.max(initial=-1.0) <= 0, (b, np.abs(ob - ro).max(), over.max())
            empty = np.isneginf(rl)
            assert np.array_equal(np.isneginf(lb), empty) and (ob.transpose(1, 0, 2)[empty] == 0).all()
            err = np.abs(lb[~empty] - rl[~empty])
            assert err.max(initial=0.0) <= tol_lse, (b, err.max(), tol_lse)
        return ref


# (key lengths, new tokens): one token, lengths of 0 and 1, tile borders, more tokens than keys, odd sizes.
FIXED = [([100, 7, 0], 200), ([1], 1), ([0, 5], 1), ([127, 128, 129, 300], 1), ([777], 1), ([40, 3, 0], 5), ([300, 131], 37), ([513, 640], 130),
         ([700], 300)]
PACKED = [([9, 4, 131, 257, 128], [5, 0, 131, 200, 1]), ([640, 1000], [1, 333]), ([300, 2, 0, 70], [1, 5, 3, 64])]
HEADS = [(4, 2, 128), (8, 1, 128), (2, 2, 128), (7, 1, 128), (12, 4, 64), (3, 3, 64), (10, 2, 64)]


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("case", range(len(FIXED)))
def test_attend_fixed(case, heads, causal):
    lk, n = FIXED[case]
    p = Problem(lk, [n] * len(lk), *heads, page=(16, 64, 8, 128, 32)[(case + heads[0]) % 5], seed=case)
    p.check_attend(*p.attend(causal), causal)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("case", range(len(PACKED)))
def test_attend_packed(case, heads, causal):
    lk, lq = PACKED[case]
    p = Problem(lk, lq, *heads, page=(32, 256, 16)[case], packed=True, seed=20 + case)
    rows = p.q.shape[0]
    out = torch.full_like(p.cq, NAN)
    lse = torch.full((p.H, rows), 7.0, device="cuda")
    o, l = p.attend(causal, out=out, lse=lse)
    assert o is out and l is lse
    end = int(p.cu[-1])
    assert torch.isnan(o[end:].float()).all() and (l[:, end:] == 7.0).all()  # rows of no sequence stay as they were
    p.check_attend(o, l, causal)


@pytest.mark.parametrize("sms", [1, 2, 3, 7, 64, 400])
@pytest.mark.parametrize("n,heads", [(1, (4, 2, 128)), (3, (16, 2, 64)), (40, (8, 2, 128)), (90, (6, 2, 64))])
def test_attend_any_division(n, heads, sms):
    """The same work divided among 1 to 400 CTAs: pieces of any length, more CTAs than key tiles included."""
    p = Problem([1111, 250, 0, 1], [n] * 4, *heads, page=32, seed=n)
    p.check_attend(*p.attend(True, num_sms=sms), True)


def test_attend_many_sequences():
    """More sequences than threads look for a CTA's share, many of them empty, in a packed batch with gaps."""
    r = np.random.default_rng(12)
    lk = r.integers(0, 300, 500) * (r.random(500) < 0.6)
    lq = r.integers(0, 4, 500) * (r.random(500) < 0.7)
    p = Problem(lk.tolist(), lq.tolist(), 4, 2, 64, page=32, packed=True, seed=13)
    for sms in (1, 152):
        p.check_attend(*p.attend(True, num_sms=sms), True)


@pytest.mark.parametrize("rows", ["few", "many"])
def test_more_sequences_than_threads(rows):
    """Shares are found by threads that look at several sequences each, most of them without tokens or keys."""
    r = np.random.default_rng(14)
    lk = r.integers(0, 150, 1500) * (r.random(1500) < 0.2)
    lq = r.integers(0, 5 if rows == "few" else 70, 1500) * (r.random(1500) < 0.1)
    p = Problem(lk.tolist(), lq.tolist(), 4, 1, 64, page=16, packed=True, seed=18)
    for sms in (2, 152):
        o, lse = p.attend(True, num_sms=sms)
        p.check_attend(o, lse, True)
    w = torch.zeros_like(p.cw)
    fa.paged_key_weights(p.cq, p.ck, p.ctable, p.clen, lse, w, causal=True, scale=p.scale, **p.tokens)
    seen = int((~torch.isneginf(lse[:, :int(p.cu[-1])])).sum())  # every row that sees a key pays 1 in all
    assert abs(float(w.sum()) - seen) < 1e-3 * seen


@pytest.mark.parametrize("B", [577, 600, 1300])
def test_more_sequences_than_threads_of_the_largest_block(B):
    """40 rows per K/V head at d = 128: the block of the most warps, all of which have sequences to look at."""
    r = np.random.default_rng(B)
    lk = r.integers(0, 200, B) * (r.random(B) < 0.2)
    lq = r.integers(0, 6, B) * (r.random(B) < 0.2)
    lk[-1], lq[0], lq[-1] = 150, 5, 5
    p = Problem(lk.tolist(), lq.tolist(), 16, 2, 128, page=16, packed=True, seed=19)
    for sms in (1, 152):
        p.check_attend(*p.attend(True, num_sms=sms), True)


def test_packed_batch_with_a_wide_bound_on_its_lengths():
    """512 sequences whose new tokens are bounded by 2^20: append, attention and key weights."""
    r = np.random.default_rng(15)
    lq = r.integers(0, 3, 512)
    lk = lq + r.integers(0, 40, 512)
    lq[7], lk[7] = 200, 300
    p = Problem(lk.tolist(), lq.tolist(), 4, 2, 64, page=16, packed=True, seed=20)
    p.tokens["max_seqlen_q"] = 1 << 20
    k, v, w = p.np(p.k), p.np(p.v), p.np(p.w)
    paged.append(p.np(p.k_new), p.np(p.v_new), k, v, p.table.numpy(), p.lk, p.cu, w)
    fa.paged_append(p.k_new.cuda(), p.v_new.cuda(), p.ck, p.cv, p.ctable, p.clen, key_weights=p.cw, **p.tokens)
    assert np.array_equal(p.np(p.ck), k, equal_nan=True) and np.array_equal(p.np(p.cw), w, equal_nan=True)
    p.k, p.v, p.w = torch.tensor(k), torch.tensor(v), torch.tensor(w).float()
    p.check_attend(*p.attend(True), True)
    check_weights(p, True)


@pytest.mark.parametrize("n", [1, 4, 70])
@pytest.mark.parametrize("layout", ["hpd", "gap"])
@pytest.mark.parametrize("d", [64, 128])
def test_attend_strided_cache_and_rows(d, layout, n):
    p = Problem([259, 90], [n, n], 6, 2, d, page=16, seed=3, layout=layout)
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
    """Groups of heads past what one tile's rows take whole: divided groups, a prime count, one token a tile."""
    p = Problem([300, 77], [n, n], *heads, page=32, seed=14)
    o, lse = p.attend(True)
    p.check_attend(o, lse, True)
    check_weights(p, True)


def test_page_sizes_at_both_ends():
    for page, lk in ((8, [1000, 9]), (65536, [700, 0]), (1024, [1025, 1024])):
        for n in (1, 33):
            p = Problem(lk, [n, n], 4, 2, 64, page=page, seed=15, extra_pages=0 if page > 10_000 else 2)
            o, lse = p.attend(True)
            p.check_attend(o, lse, True)
            check_weights(p, True)


@pytest.mark.parametrize("n", [1, 40])
def test_interleaved_cache_and_fused_projection(n):
    """K and V as halves of one pool, q, k and v as slices of one projection: no tensor is contiguous."""
    H, Hkv, d, P = 6, 2, 128, 16
    p = Problem([90, 200], [n, n], H, Hkv, d, page=P, seed=16)
    pool = torch.empty((p.pages, 2, P, Hkv, d), dtype=torch.bfloat16, device="cuda")
    pool[:, 0], pool[:, 1] = p.ck, p.cv
    p.ck, p.cv = pool[:, 0], pool[:, 1]
    fused = torch.full((2, n, H + 2 * Hkv, d), NAN, dtype=torch.bfloat16, device="cuda")
    fused[:, :, :H], fused[:, :, H:H + Hkv], fused[:, :, H + Hkv:] = p.cq, p.k_new.cuda(), p.v_new.cuda()
    p.cq = fused[:, :, :H]
    fa.paged_append(fused[:, :, H:H + Hkv], fused[:, :, H + Hkv:], p.ck, p.cv, p.ctable, p.clen)
    k, v = p.np(p.k), p.np(p.v)
    paged.append(p.np(p.k_new), p.np(p.v_new), k, v, p.table.numpy(), p.lk)
    assert np.array_equal(p.np(p.ck), k, equal_nan=True) and np.array_equal(p.np(p.cv), v, equal_nan=True)
    p.k, p.v = torch.tensor(k), torch.tensor(v)
    p.check_attend(*p.attend(True), True)


def test_attend_extreme_scores():
    """Scores far apart in every direction: a row max that grows late and by a lot, one that never does, and keys that
    outweigh all others; a softmax is one-hot there, so O is one value row."""
    for n in (1, 6, 130):
        for sign in (1.0, -1.0):
            p = Problem([900, 400], [n, n], 4, 2, 128, page=16, seed=5, std=1.0)
            grow = torch.linspace(-6.0, 6.0, 900)
            for b in range(2):
                j = torch.arange(p.lk[b])
                p.k[p.table[b][j // 16].long(), j % 16] *= (sign * grow[:p.lk[b]]).to(torch.bfloat16)[:, None, None]
            p.q = (p.q.float() * 8).to(torch.bfloat16)
            p.cq, p.ck = p.q.cuda(), p.k.cuda()
            p.check_attend(*p.attend(True), True)


@pytest.mark.parametrize("n", [1, 6, 40])
def test_attend_large_values_behind_growing_scores(n):
    """Values of 2^100 and a key 2^30 times as heavy as those of the first tile behind it: O is finite and near 2^100,
    though the sum without a common maximum is not."""
    p = Problem([300], [n], 4, 2, 64, page=16, seed=17)
    p.k[p.live] = 0.0
    p.v[p.live] = 2.0**100
    j = 200
    p.q[:] = 1.0
    p.k[p.table[0, j // 16], j % 16] = 30 * math.log(2) / (64 * p.scale)
    p.cq, p.ck, p.cv = p.q.cuda(), p.k.cuda(), p.v.cuda()
    p.check_attend(*p.attend(False), False)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,sms", [(1, 152), (1, 3), (1, 1), (10, 152), (10, 3), (600, 152), (600, 5)])
def test_nan_key_or_query_is_seen_however_the_work_is_divided(n, sms, d):
    """A NaN in a key makes O and LSE of the rows that see it NaN, one in a query row those of the row; the rest is as
    without. Shares of clusters, of divided units and whole ones alike."""
    L, j, bad_row = 1100, 700, n // 3
    p = Problem([L, 300], [n, min(n, 300)], 8, 2, d, page=16, seed=31, packed=True)
    tol = p.score_error() + 2.0**-18
    ref = p.check_attend(*p.attend(True, num_sms=sms), True)
    p.ck[p.ctable[0, j // 16].long(), j % 16, 1, 5] = NAN
    p.cq[bad_row, 2, 7] = NAN
    o, lse = p.attend(True, num_sms=sms)
    end = int(p.cu[-1])
    bad = torch.zeros(end, 8, dtype=torch.bool, device="cuda")
    bad[:n, 4:] = (torch.arange(n, device="cuda") + L - n >= j)[:, None]
    bad[bad_row, 2] = True
    assert torch.isnan(o[:end][bad]).all() and torch.isnan(lse[:, :end].t()[bad]).all()
    ro, rl, a = np.concatenate([x[0] for x in ref]), np.concatenate([x[1].T for x in ref]), np.concatenate([x[2] for x in ref])
    good = ~bad.cpu().numpy()
    assert (np.abs(p.np(o)[:end] - ro) <= 1.05 * 2.0**-8 * (a + np.abs(ro)))[good].all()
    assert (np.abs(p.np(lse)[:, :end].T - rl) <= tol)[good].all()


def test_attend_shared_pages_and_bound():
    """Two sequences share their first pages; a bound above the longest length changes nothing, one below cuts."""
    p = Problem([200, 200], [2, 2], 4, 2, 128, page=16, seed=6)
    p.table[1, :8] = p.table[0, :8]
    p.ctable = p.table.cuda()
    p.check_attend(*p.attend(True, max_seqlen_k=10_000), True)
    p.lk = [96, 96]
    p.check_attend(*p.attend(True, max_seqlen_k=96), True)


def test_attend_lengths_past_the_table_and_below_zero_are_clamped():
    p = Problem([64, 64, 0], [1, 1, 1], 4, 2, 128, page=16, seed=7)
    p.ctable = p.table[:, :4].contiguous().cuda()
    p.clen = torch.tensor([1 << 30, 64, -5], dtype=torch.int32, device="cuda")
    p.check_attend(*p.attend(False), False)


@pytest.mark.parametrize("n", [1, 40])
def test_bad_page_is_reported_and_stays_in_bounds(n):
    for bad in (-1, 1 << 20):
        p = Problem([100, 300], [n, n], 4, 2, 128, page=16, seed=8)
        good = p.attend(True)
        p.ctable[1, 3] = bad
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        args = (p.ctable, p.clen)
        o, lse = fa.fwd_paged(p.cq, p.ck, p.cv, *args, causal=True, scale=p.scale, status=status)
        assert int(status.item()) == -6
        assert torch.equal(o[0], good[0][0]) and torch.equal(lse[0], good[1][0])  # the other sequence is sound
        status.zero_()
        fa.paged_key_weights(p.cq, p.ck, *args, good[1], p.cw, causal=True, scale=p.scale, status=status)
        assert int(status.item()) == -6
        status.zero_()
        fa.paged_evict(p.ck, p.cv, p.cw, *args, 90, recent=10, status=status)
        assert int(status.item()) == -6


@pytest.mark.parametrize("n", [1, 40])
def test_cache_of_more_than_2_31_elements(n):
    """Pages at both ends of a cache whose element offsets pass 32 bits."""
    H, Hkv, d, P = 4, 2, 128, 64
    pages = (1 << 31) // (P * Hkv * d) + 40
    p = Problem([400], [n], H, Hkv, d, page=P, seed=9)
    used = -(-400 // P)
    big = [torch.empty((pages, P, Hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    at = torch.tensor([pages - 1, 0, pages - 3, 1, pages // 2, pages - 2, 2], dtype=torch.int32)[:used]
    src = p.table[0, :used].long()
    for b, t in zip(big, (p.ck, p.cv)):
        b[at.long().cuda()] = t[src.cuda()]
    ref = p.attend(True)
    p.ctable[0, :used] = at.cuda()
    p.ck, p.cv = big
    o, lse = p.attend(True)
    assert torch.equal(o, ref[0]) and torch.equal(lse, ref[1])
    w = torch.zeros((pages, Hkv, P), device="cuda")
    fa.paged_key_weights(p.cq, p.ck, p.ctable, p.clen, lse, w, causal=True, scale=p.scale)
    assert abs(float(w.sum()) - n * H) < 1e-3 * n * H
    new = torch.randn((1, n, Hkv, d), device="cuda").to(torch.bfloat16)
    fa.paged_append(new, new, p.ck, p.cv, p.ctable, p.clen)
    j = torch.arange(400 - n, 400)
    assert torch.equal(p.ck[p.ctable[0, (j // P).cuda()].long(), (j % P).cuda()], new[0])


# ----------------------------------------------------------------------------- key weights


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("case", range(len(FIXED) + len(PACKED)))
def test_key_weights(case, heads, causal):
    page = (16, 64, 8, 128, 32)[(case + heads[0]) % 5]
    if case < len(FIXED):
        lk, n = FIXED[case]
        p = Problem(lk, [n] * len(lk), *heads, page=page, seed=40 + case)
    else:
        lk, lq = PACKED[case - len(FIXED)]
        p = Problem(lk, lq, *heads, page=page, packed=True, seed=40 + case)
    check_weights(p, causal)


def check_weights(p, causal, rel_sum=2.0**-16):
    att = paged.attention(p.np(p.q), p.np(p.k), p.np(p.v), p.table.numpy(), p.lk, p.scale, causal, p.cu)
    lses = [x[1].astype(np.float32) for x in att]
    if p.packed:
        lse = np.full((p.H, p.q.shape[0]), NAN, dtype=np.float32)  # rows of no sequence hold anything
        for b in range(len(p.lk)):
            lse[:, p.cu[b]:p.cu[b + 1]] = lses[b]
    else:
        lse = np.stack(lses)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = fa.paged_key_weights(p.cq, p.ck, p.ctable, p.clen, torch.tensor(lse).cuda(), p.cw, causal=causal,
                               scale=p.scale, status=status, **p.tokens)
    assert got is p.cw and int(status.item()) == 0
    add = paged.key_weights(p.np(p.q), p.np(p.k), p.table.numpy(), p.lk, lses, p.scale, causal, p.cu)
    w, w0 = p.np(p.cw), p.np(p.w)
    finite = [np.abs(x[np.isfinite(x)]).max(initial=0.0) for x in lses]
    rel = p.score_error() + max(finite) * 2.0**-24 + rel_sum
    for b, L in enumerate(p.lk):
        for j in range(L):
            at = (p.table[b][j // p.P].item(), slice(None), j % p.P)
            assert (np.abs(w[at] - w0[at] - add[b][:, j]) <= rel * add[b][:, j] + 2.0**-23 * w[at]).all(), (b, j)
    dead = ~p.live[:, None].expand(-1, p.Hkv, -1).numpy()
    assert np.isnan(w[dead]).all()  # the other slots stay as they were


def test_key_weights_of_many_rows_and_of_the_last_rows_only():
    """More query rows than one tile holds for every key; then only the last 16 tokens of the prompt."""
    p = Problem([700], [700], 8, 2, 128, page=64, seed=60)
    check_weights(p, True)
    full = p.q
    _, lse = p.attend(True)
    p.q, p.cq, p.lq, p.cw = full[:, -16:], p.cq[:, -16:], [16], p.w.cuda()
    check_weights(p, True)
    w = p.w.cuda()
    fa.paged_key_weights(p.cq, p.ck, p.ctable, p.clen, lse[:, :, -16:].contiguous(), w, causal=True, scale=p.scale)
    live = torch.isfinite(w)
    assert torch.allclose(w[live], p.cw[live], rtol=1e-4, atol=1e-5)


@pytest.mark.parametrize("n", [3, 90])
def test_key_weights_of_rows_without_weight(n):
    """Rows of LSE = -inf add nothing, whatever their q holds (a padded batch)."""
    p = Problem([300, 120], [n, n], 4, 2, 128, page=16, seed=61)
    _, lse = p.attend(True)
    dead = torch.zeros(2, n, dtype=torch.bool)
    dead[0, n // 2:], dead[1, 0] = True, True
    q = p.cq.clone()
    q[dead.cuda()] = NAN
    lse = lse.masked_fill(dead.cuda()[:, None], -math.inf)
    got = fa.paged_key_weights(q, p.ck, p.ctable, p.clen, lse, p.cw, causal=True, scale=p.scale)
    add = paged.key_weights(p.np(p.q), p.np(p.k), p.table.numpy(), p.lk, list(p.np(lse)), p.scale, True)
    rel = p.score_error() + 2.0**-20 + 2.0**-16
    for b, L in enumerate(p.lk):
        j = torch.arange(L)
        at = (p.table[b][j // 16].long(), slice(None), j % 16)
        w, w0 = p.np(got)[at], p.np(p.w)[at]
        assert (np.abs(w - w0 - add[b].T) <= rel * add[b].T + 2.0**-23 * w).all()


# ----------------------------------------------------------------------------- append and evict


@pytest.mark.parametrize("layout", ["phd", "hpd", "gap"])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("heads", [(2, 2, 128), (3, 3, 64), (1, 1, 128)])
def test_append(heads, packed, layout):
    lk, lq = ([9, 4, 131, 257], [5, 0, 131, 200]) if packed else ([70, 33, 20], [20] * 3)
    p = Problem(lk, lq, *heads, page=16, packed=packed, seed=70, layout=layout)
    k, v, w = p.np(p.k), p.np(p.v), p.np(p.w)
    paged.append(p.np(p.k_new), p.np(p.v_new), k, v, p.table.numpy(), lk, p.cu, w)
    for with_weights in (True, False):
        if not with_weights:
            p.cw.copy_(p.w)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        fa.paged_append(p.k_new.cuda(), p.v_new.cuda(), p.ck, p.cv, p.ctable, p.clen,
                        key_weights=p.cw if with_weights else None, status=status, **p.tokens)
        assert int(status.item()) == 0
        assert np.array_equal(p.np(p.ck), k, equal_nan=True) and np.array_equal(p.np(p.cv), v, equal_nan=True)
        assert np.array_equal(p.np(p.cw), w if with_weights else p.np(p.w), equal_nan=True)


@pytest.mark.parametrize("B", [31, 33, 500, 2100])
def test_append_of_many_packed_sequences(B):
    """One prompt among single tokens and sequences without any, more of them than one look at their ends covers."""
    r = np.random.default_rng(B)
    lq = (r.random(B) < 0.6).astype(int)
    lq[B // 3] = 300
    lk = lq + r.integers(0, 20, B)
    p = Problem(lk.tolist(), lq.tolist(), 2, 1, 64, page=8, packed=True, seed=72)
    k, v, w = p.np(p.k), p.np(p.v), p.np(p.w)
    paged.append(p.np(p.k_new), p.np(p.v_new), k, v, p.table.numpy(), lk, p.cu, w)
    fa.paged_append(p.k_new.cuda(), p.v_new.cuda(), p.ck, p.cv, p.ctable, p.clen, key_weights=p.cw, **p.tokens)
    assert np.array_equal(p.np(p.ck), k, equal_nan=True) and np.array_equal(p.np(p.cv), v, equal_nan=True)
    assert np.array_equal(p.np(p.cw), w, equal_nan=True)


@pytest.mark.parametrize("packed", [False, True])
def test_append_with_a_table_far_wider_than_the_lengths(packed):
    """512 sequences of 32 K/V heads with room for 131072 keys each: the places are what counts, not the table's width."""
    B, P, wide = 512, 16, 131072 // 16
    lq = [(b % 3 if packed else 1) for b in range(B)]
    p = Problem([n + b % 17 for b, n in enumerate(lq)], lq, 32, 32, 64, page=P, packed=packed, seed=73)
    k, v = p.np(p.k), p.np(p.v)
    paged.append(p.np(p.k_new), p.np(p.v_new), k, v, p.table.numpy(), p.lk, p.cu)
    table = torch.full((B, wide), -7, dtype=torch.int32)
    table[:, :p.width] = p.table
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    fa.paged_append(p.k_new.cuda(), p.v_new.cuda(), p.ck, p.cv, table.cuda(), p.clen, status=status, **p.tokens)
    assert int(status.item()) == 0
    assert np.array_equal(p.np(p.ck), k, equal_nan=True) and np.array_equal(p.np(p.cv), v, equal_nan=True)
    o, lse = fa.fwd_paged(p.cq, p.ck, p.cv, table.cuda(), p.clen, max_seqlen_k=18, causal=True, scale=p.scale, **p.tokens)
    p.k, p.v = torch.tensor(k), torch.tensor(v)
    p.check_attend(o, lse, True)


def test_append_places_outside_the_table_are_reported():
    """A length below the token count and one past the table's capacity: the tokens with a place are written."""
    p = Problem([16, 32], [4, 4], 2, 2, 128, page=16, seed=71)
    lens = [3, 50]  # tokens at -1 .. 2, and at 46 .. 49 of 48
    p.table[1, 2] = min(set(range(p.pages)) - set(p.table.flatten().tolist()))  # a page of nobody
    k, v = p.np(p.k), p.np(p.v)
    paged.append(p.np(p.k_new), p.np(p.v_new), k, v, p.table.numpy(), lens)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    fa.paged_append(p.k_new.cuda(), p.v_new.cuda(), p.ck, p.cv, p.table.cuda(),
                    torch.tensor(lens, dtype=torch.int32, device="cuda"), status=status)
    assert int(status.item()) == -6
    assert np.array_equal(p.np(p.ck), k, equal_nan=True) and np.array_equal(p.np(p.cv), v, equal_nan=True)


EVICT = [([100, 20, 0, 64], 64, 10), ([300], 1, 0), ([300], 1, 1), ([1000, 129], 128, 128), ([1500, 700], 600, 0),
         ([5000], 4000, 77), ([260, 2600], 255, 3), ([2500], 2499, 2000),
         ([2048, 1500, 40], 1499, 9), ([30, 2047], 1900, 1900), ([40] * 30 + [900], 300, 1)]


@pytest.mark.parametrize("weights", ["heavy", "ties", "odd"])
@pytest.mark.parametrize("heads", [(2, 2, 128), (3, 3, 64)])
@pytest.mark.parametrize("case", range(len(EVICT)))
def test_evict(case, heads, weights):
    lk, keep, recent = EVICT[case]
    p = Problem(lk, [1] * len(lk), *heads, page=(16, 8, 64, 32)[case % 4], seed=80 + case,
                layout=("phd", "hpd", "gap")[case % 3])
    g = torch.Generator().manual_seed(case)
    there = torch.isfinite(p.w)
    if weights == "ties":  # a handful of values, most of them 0 (of either sign)
        p.w = torch.where(there, torch.randint(-1, 3, p.w.shape, generator=g).float().clamp(min=-0.0), p.w)
    if weights == "odd":  # negative numbers, infinities, NaN and subnormal numbers among them
        pick = torch.tensor([NAN, math.inf, -math.inf, 1e-42, -1e-42, -3.0, 0.0, 2.0])
        p.w = torch.where(there, pick[torch.randint(0, 8, p.w.shape, generator=g)], p.w)
    p.cw = p.w.cuda()
    k, v, w = p.np(p.k), p.np(p.v), p.w.double().numpy().copy()
    kept, n = paged.evict(k, v, w, p.table.numpy(), lk, keep, recent)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got, lens = fa.paged_evict(p.ck, p.cv, p.cw, p.ctable, p.clen, keep, recent=recent, status=status)
    assert int(status.item()) == 0
    assert np.array_equal(got.cpu().numpy(), kept) and np.array_equal(lens.cpu().numpy(), n)
    assert np.array_equal(p.np(p.ck), k, equal_nan=True) and np.array_equal(p.np(p.cv), v, equal_nan=True)
    assert np.array_equal(p.np(p.cw), w, equal_nan=True)


@pytest.mark.parametrize("L", [20_000, 60_000, 140_000])
def test_evict_long(L):
    """Lengths that take clusters of 4 and 8 CTAs, and one past what a cluster's registers hold; many equal weights."""
    p = Problem([L, 70], [1, 1], 1, 1, 64, page=64, seed=95)
    p.w = torch.round(p.w * 4) / 4
    p.cw = p.w.cuda()
    k, v, w = p.np(p.k), p.np(p.v), p.w.double().numpy().copy()
    kept, n = paged.evict(k, v, w, p.table.numpy(), p.lk, L // 2, 100)
    got, lens = fa.paged_evict(p.ck, p.cv, p.cw, p.ctable, p.clen, L // 2, recent=100)
    assert np.array_equal(got.cpu().numpy(), kept) and lens.tolist() == n.tolist()
    assert np.array_equal(p.np(p.ck), k, equal_nan=True) and np.array_equal(p.np(p.cv), v, equal_nan=True)
    assert np.array_equal(p.np(p.cw), w, equal_nan=True)


def test_evict_does_not_look_at_the_rows_of_its_problem():
    """A packed step's problem serves its eviction after cu_seqlens_q is gone (here: an address that no GPU may read)."""
    import ctypes
    p = Problem([100, 30], [1, 1], 2, 2, 128, page=16, seed=99)
    k, v, w = p.np(p.k), p.np(p.v), p.w.double().numpy().copy()
    kept, n = paged.evict(k, v, w, p.table.numpy(), p.lk, 64, 10)
    host = (ctypes.c_int32 * 3)(5, 1, 0)
    prob = fa._paged(None, p.ck, p.cv, p.ctable, p.clen, None, None, None, False, 1.0)[0]
    prob.cu_seqlens_q, prob.rows_q, prob.seqlen_q = ctypes.addressof(host), 7, 1 << 30
    got = torch.empty((2, 2, 64), dtype=torch.int32, device="cuda")
    lens = torch.empty(2, dtype=torch.int32, device="cuda")
    st = fa._paged_view("k", p.ck, 4)
    assert fa.fa_paged_evict(prob, 64, 10, p.ck.data_ptr(), st, p.cv.data_ptr(), st, p.cw.data_ptr(), got.data_ptr(),
                             lens.data_ptr(), None, torch.cuda.current_stream().cuda_stream) == 0
    assert np.array_equal(got.cpu().numpy(), kept) and np.array_equal(lens.cpu().numpy(), n)
    assert np.array_equal(p.np(p.ck), k, equal_nan=True) and np.array_equal(p.np(p.cw), w, equal_nan=True)


# ----------------------------------------------------------------------------- together


def serve(p, q, k, v, keep, recent, budget):
    """One serving step through the public calls: append, attend, weigh, and evict past the budget."""
    fa.paged_append(k, v, p.ck, p.cv, p.ctable, p.clen, key_weights=p.cw)
    o, lse = fa.fwd_paged(q, p.ck, p.cv, p.ctable, p.clen, causal=True, scale=p.scale, max_seqlen_k=budget)
    fa.paged_key_weights(q, p.ck, p.ctable, p.clen, lse, p.cw, causal=True, scale=p.scale, max_seqlen_k=budget)
    kept, n = fa.paged_evict(p.ck, p.cv, p.cw, p.ctable, p.clen, keep, recent=recent, max_seqlen_k=budget)
    return o, lse, kept, n


@pytest.mark.parametrize("heads", [(4, 2, 128), (3, 3, 64)])
def test_a_run_of_all_operators(heads):
    """A prompt in two chunks and three tokens, evicted down to 96 keys after every step, against the oracle's run."""
    B, keep, recent, P = 2, 96, 20, 16
    p = Problem([400, 400], [1, 1], *heads, page=P, seed=90)
    p.k[:], p.v[:], p.w[:] = NAN, NAN, NAN
    p.ck, p.cv, p.cw = p.k.cuda(), p.v.cuda(), p.w.cuda()
    k, v = p.np(p.k), p.np(p.v)
    table = p.table.numpy()
    g = torch.Generator().manual_seed(91)
    have = [0, 0]
    for n in (150, 75, 1, 1, 1):
        bf = lambda h: torch.randn((B, n, h, p.d), generator=g).to(torch.bfloat16)
        q, kn, vn = bf(p.H), bf(p.Hkv), bf(p.Hkv)
        lens = [x + n for x in have]
        p.clen = torch.tensor(lens, dtype=torch.int32, device="cuda")
        o, lse, kept, new = serve(p, q.cuda(), kn.cuda(), vn.cuda(), keep, recent, 400)
        paged.append(p.np(kn), p.np(vn), k, v, table, lens)
        p.q, p.k, p.v, p.lk, p.lq = q, torch.tensor(k), torch.tensor(v), lens, [n] * B
        p.check_attend(o, lse, True)
        # The GPU's weights choose; the oracle then moves by the same choice (a near tie may fall either way).
        for b in range(B):
            for h in range(p.Hkv):
                idx = kept[b, h].cpu().numpy()
                m = min(lens[b], keep)
                assert (np.diff(idx[:m]) > 0).all() and (idx[m:] == -1).all()
                if lens[b] > keep:
                    assert (idx[m - recent:m] == np.arange(lens[b] - recent, lens[b])).all()
                for t in (k, v):
                    rows = paged.keys_of(t, table, lens[b], b, h)[idx[:m]]
                    for i in range(m):
                        t[table[b][i // P], i % P, h] = rows[i]
                got = np.stack([p.np(p.ck)[table[b][i // P], i % P, h] for i in range(m)])
                assert np.array_equal(got, paged.keys_of(k, table, m, b, h))
        have = [min(x, keep) for x in lens]
        assert new.tolist() == have


@pytest.mark.parametrize("sms", [152, 3])
def test_captured_and_replayed_step_follows_the_lengths(sms):
    """One decode step captured once, replayed with other lengths, rows and page tables in the same buffers, equals the
    eager calls; two graphs share the workspace (152 SMs: clusters, without one; 3: the work is divided)."""
    p = Problem([700, 1200], [1, 1], 8, 2, 128, page=16, seed=92)
    q, k, v = p.cq.clone(), p.k_new.cuda(), p.v_new.cuda()
    bound = p.width * p.P
    prob = fa._paged(q, p.ck, p.cv, p.ctable, p.clen, None, None, bound, True, p.scale)[0]
    ws = torch.empty(fa.fa_fwd_paged_workspace_bytes(prob, sms), dtype=torch.uint8, device="cuda")
    assert (ws.numel() > 0) == (sms == 3)
    state0 = [t.clone() for t in (p.ck, p.cv, p.cw)]

    def step():
        fa.paged_append(k, v, p.ck, p.cv, p.ctable, p.clen, key_weights=p.cw)
        o, lse = fa.fwd_paged(q, p.ck, p.cv, p.ctable, p.clen, causal=True, scale=p.scale, num_sms=sms, workspace=ws)
        fa.paged_key_weights(q, p.ck, p.ctable, p.clen, lse, p.cw, causal=True, scale=p.scale)
        kept, n = fa.paged_evict(p.ck, p.cv, p.cw, p.ctable, p.clen, 500, recent=50)
        return o, lse, kept, n

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = step()
        graphs.append((graph, outs))
    for lens in ([700, 1200], [33, 1100], [1, 600]):
        eager = []
        for mode in (None, 0, 1):
            for t, t0 in zip((p.ck, p.cv, p.cw), state0):
                t.copy_(t0)
            p.clen.copy_(torch.tensor(lens, dtype=torch.int32))
            q.copy_(p.cq * (1 if lens[0] != 33 else -1))
            if mode is None:
                got = step()
            else:
                graphs[mode][0].replay()
                got = graphs[mode][1]
            torch.cuda.synchronize()
            now = [t.clone() for t in got] + [p.ck.clone(), p.cv.clone(), p.cw.clone()]
            eager = eager or now
            for x, y in zip(now, eager):
                assert torch.equal(torch.nan_to_num(x.float(), 9.0), torch.nan_to_num(y.float(), 9.0))


def test_two_streams_at_once():
    """Calls of every kind on two streams without order between them, each with its own cache and workspace."""
    problems = [Problem([900, 300], [n, n], 8, 2, 128, page=16, seed=96 + n) for n in (1, 60)]
    refs, outs = [], []
    for p in problems:
        p.cw0, p.ck0, p.cv0 = p.cw.clone(), p.ck.clone(), p.cv.clone()

    def work(p):
        o, lse = fa.fwd_paged(p.cq, p.ck, p.cv, p.ctable, p.clen, causal=True, scale=p.scale)
        fa.paged_key_weights(p.cq, p.ck, p.ctable, p.clen, lse, p.cw, causal=True, scale=p.scale)
        kept, _ = fa.paged_evict(p.ck, p.cv, p.cw, p.ctable, p.clen, 200, recent=20)
        return o, lse, kept, p.ck.clone(), p.cv.clone(), p.cw.clone()

    for p in problems:
        refs.append(work(p))
        p.cw.copy_(p.cw0), p.ck.copy_(p.ck0), p.cv.copy_(p.cv0)
    torch.cuda.synchronize()
    for p in problems:
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(5):
                p.cw.copy_(p.cw0), p.ck.copy_(p.ck0), p.cv.copy_(p.cv0)
                last = work(p)
            outs.append(last)
    torch.cuda.synchronize()
    for ref, out in zip(refs, outs):
        for x, y in zip(ref, out):
            assert torch.equal(torch.nan_to_num(x.float(), 9.0), torch.nan_to_num(y.float(), 9.0))


def test_other_streams_and_back_to_back_calls():
    """Calls on a side stream with the tensors' work ordered by events, and many calls in a row without a wait."""
    p = Problem([513, 77], [1, 1], 8, 2, 128, page=16, seed=93)
    ref = p.attend(True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    outs = [fa.fwd_paged(p.cq, p.ck, p.cv, p.ctable, p.clen, causal=True, scale=p.scale,
                         stream=s if i % 2 else s.cuda_stream) for i in range(20)]
    with torch.cuda.stream(s):
        outs.append(fa.fwd_paged(p.cq, p.ck, p.cv, p.ctable, p.clen, causal=True, scale=p.scale))
    torch.cuda.synchronize()
    for o, lse in outs:
        assert torch.equal(o, ref[0]) and torch.equal(lse, ref[1])


@pytest.mark.parametrize("L,heads", [(1900, (4, 2, 128)), (6000, (24, 12, 64))])  # an eviction of one launch, and of two
def test_lengths_of_an_eviction_go_straight_into_the_next_call(L, heads):
    """Lengths written by an eviction and read by the next calls with no other kernel between, the old ones beside the new
    in one buffer: the same as with a wait after every call."""
    p = Problem([L, 700, 40], [1, 1, 1], *heads, page=16, seed=101)
    k, v = p.k_new.cuda(), p.v_new.cuda()
    first = [p.ck.clone(), p.cv.clone(), p.cw.clone()]
    lens = torch.zeros(3, 3, dtype=torch.int32, device="cuda")
    cont = [torch.randn(3, p.H, 256, p.d, device="cuda").to(torch.bfloat16) for _ in range(3)]

    def chain(n, wait):
        for t, t0 in zip((p.ck, p.cv, p.cw), first):
            t.copy_(t0)
        lens.zero_()
        lens[0] = torch.tensor(n, dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        outs = []

        def done(*x):
            outs.extend(x)
            if wait:
                torch.cuda.synchronize()

        done(*fa.paged_evict(p.ck, p.cv, p.cw, p.ctable, lens[0], 600, recent=30, seqlens_out=lens[1]))
        done(*fa.fwd(*cont, seqlens_k=lens[1]))
        done(*fa.paged_evict(p.ck, p.cv, p.cw, p.ctable, lens[1], 200, recent=10, seqlens_out=lens[2]))
        done(*fa.fwd_paged(p.cq, p.ck, p.cv, p.ctable, lens[2], causal=True, scale=p.scale))
        done(*fa.paged_evict(p.ck, p.cv, p.cw, p.ctable, lens[2], 100, recent=10, seqlens_out=lens[1]))
        fa.paged_append(k, v, p.ck, p.cv, p.ctable, lens[1], key_weights=p.cw)
        done(*fa.fwd_paged(p.cq, p.ck, p.cv, p.ctable, lens[1], causal=True, scale=p.scale))
        torch.cuda.synchronize()
        return [t.clone() for t in (*outs, p.ck, p.cv, p.cw)]

    for n in ([L, 700, 40], [650, 20, 1], [L // 2, 300, 7]):
        want = chain(n, True)
        for _ in range(30):
            for x, y in zip(chain(n, False), want):
                assert torch.equal(torch.nan_to_num(x.float(), 9.0), torch.nan_to_num(y.float(), 9.0))
