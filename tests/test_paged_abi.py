"""Host-side checks of the paged-cache entry points (no GPU): every refusal comes before any launch."""

import pytest
import torch

import exact_io_aware_38_gb300 as fa
from exact_io_aware_38_gb300 import build

A = 0x10000  # fake device address, never dereferenced


@pytest.fixture(scope="module", autouse=True)
def L():
    build.build()
    return fa.lib()


def problem(**kw):
    f = dict(B=2, H=8, Hkv=2, d=128, page_size=16, num_pages=50, max_pages=10, page_table=A, seqlens_k=A, seqlen_q=3,
             seqlen_k=160, cu_seqlens_q=None, rows_q=0, causal=1, scale=0.1)
    f.update(kw)
    return fa.PagedProblem(**f)


SQ = fa.Strides(8 * 128, 128, 3 * 8 * 128)
SN = fa.Strides(2 * 128, 128, 3 * 2 * 128)
SC = fa.Strides(2 * 128, 128, 16 * 2 * 128)


def attend(p=None, sms=152, q=A, sq=SQ, k=A, sk=SC, v=A, sv=SC, o=A, so=SQ, lse=A, ws=A, nbytes=1 << 30, status=None):
    return fa.fa_fwd_paged(p or problem(), sms, q, sq, k, sk, v, sv, o, so, lse, ws, nbytes, status, None)


def append(p=None, kn=A, skn=SN, vn=A, svn=SN, k=A, sk=SC, v=A, sv=SC, w=None, status=None):
    return fa.fa_paged_append(p or problem(), kn, skn, vn, svn, k, sk, v, sv, w, status, None)


def weights(p=None, sms=152, q=A, sq=SQ, k=A, sk=SC, lse=A, w=A, ws=A, nbytes=1 << 30, status=None):
    return fa.fa_paged_key_weights(p or problem(), sms, q, sq, k, sk, lse, w, ws, nbytes, status, None)


def evict(p=None, keep=64, recent=8, k=A, sk=SC, v=A, sv=SC, w=A, kept=A, out=2 * A, status=None):
    return fa.fa_paged_evict(p or problem(), keep, recent, k, sk, v, sv, w, kept, out, status, None)


@pytest.mark.parametrize("kw,rc", [
    (dict(B=0), -1), (dict(Hkv=0), -1), (dict(page_size=0), -1), (dict(num_pages=0), -1), (dict(max_pages=0), -1),
    (dict(seqlen_k=0), -1), (dict(seqlen_q=0), -1), (dict(page_table=None), -1), (dict(seqlens_k=None), -1),
    (dict(cu_seqlens_q=A, rows_q=0), -1), (dict(d=96), -2), (dict(page_size=24), -2), (dict(page_size=4), -2),
    (dict(page_size=1 << 17), -2), (dict(page_table=A + 2), -3), (dict(seqlens_k=A + 1), -3),
    (dict(cu_seqlens_q=A + 2, rows_q=9), -3),
    (dict(B=1 << 12, max_pages=1 << 20, seqlen_k=1 << 20), -2),  # B Hkv keys past 2^31
])
def test_problem_refusals(kw, rc):
    p = problem(**kw)
    assert attend(p) == rc and weights(p) == rc and append(p) == rc and evict(p) == rc


@pytest.mark.parametrize("kw,rc", [(dict(H=0), -1), (dict(H=7), -1), (dict(causal=2), -1), (dict(scale=0.0), -1),
                                   (dict(scale=float("nan")), -1)])
def test_problem_refusals_of_calls_with_queries(kw, rc):
    p = problem(**kw)
    assert attend(p) == rc and weights(p) == rc


def test_buffer_refusals():
    for call, names in ((attend, "q k v o lse"), (append, "kn vn k v"), (weights, "q k lse w"), (evict, "k v w kept out")):
        for n in names.split():
            assert call(**{n: None}) == -1, (call, n)
            assert call(**{n: A + 2}) == -3, (call, n)
        assert call(status=A + 2) == -3
    assert append(w=A + 2) == -3
    bad = [fa.Strides(0, 128, 8192), fa.Strides(256, 12, 8192), fa.Strides(256, 128, 0), fa.Strides(-256, 128, 8192)]
    for s in bad:
        assert attend(sq=s) == attend(sk=s) == attend(sv=s) == attend(so=s) == -1
        assert append(skn=s) == append(svn=s) == append(sk=s) == append(sv=s) == -1
        assert weights(sq=s) == weights(sk=s) == evict(sk=s) == evict(sv=s) == -1
    assert attend(sk=fa.Strides(256, 128, 1 << 39)) == -2


@pytest.mark.parametrize("call,size,kw", [
    (attend, "fa_fwd_paged_workspace_bytes", dict(max_pages=1000, seqlen_k=9000)),
    (attend, "fa_fwd_paged_workspace_bytes", dict(B=200)),
    (attend, "fa_fwd_paged_workspace_bytes", dict(seqlen_q=500)),
    (weights, "fa_paged_key_weights_workspace_bytes", dict(seqlen_q=500))])
def test_workspace_rules(call, size, kw):
    size = getattr(fa, size)
    p = problem(**kw)
    need = size(p, 152)
    assert need > 0 and need % 256 == 0
    assert size(problem(**{**kw, "seqlen_k": 160_000, "max_pages": 10_000}), 152) == need  # not by the lengths
    assert size(p, 0) == size(p, 1025) == size(problem(d=96), 152) == 0
    for sms, ws, nbytes, rc in ((0, A, 1 << 30, -1), (1025, A, 1 << 30, -1), (152, None, 1 << 30, -1),
                                (152, A, need - 1, -1), (152, A + 16, 1 << 30, -3)):
        assert call(p, sms=sms, ws=ws, nbytes=nbytes) == rc


def test_no_workspace():
    """Few rows over short keys are not divided, and key weights of few rows never are: the workspace may be null (the
    refusal is then the next one, an odd output pointer)."""
    assert fa.fa_fwd_paged_workspace_bytes(problem(), 152) == 0
    assert fa.fa_fwd_paged_workspace_bytes(problem(), 3) > 0  # more (sequence, head) units than CTAs
    assert fa.fa_paged_key_weights_workspace_bytes(problem(max_pages=9000, seqlen_k=100_000), 152) == 0
    assert attend(ws=None, nbytes=0, o=A + 2) == weights(ws=None, nbytes=0, w=A + 2) == -3


def test_evict_lengths_may_not_overlap():
    """The new lengths of a sequence may not lie over the old ones of any; side by side in one buffer they may."""
    p = problem(B=5, seqlens_k=2 * A)
    for off in (-16, -4, 0, 4, 16):
        assert evict(p, out=2 * A + off, k=None) == -1 and evict(p, out=2 * A + off, kept=A + 2) == -1
    for off in (-20, 20):
        assert evict(p, out=2 * A + off, kept=A + 2) == -3


def test_evict_heads_that_do_not_fit_a_grid():
    """16 blocks per sequence and K/V head stay below 2^31."""
    for B, rc in ((1 << 27, -2), ((1 << 27) - 1, -1)):
        assert evict(problem(B=B, H=1, Hkv=1, seqlen_k=1), keep=1, recent=0, k=None) == rc


def test_evict_has_no_rows():
    """An eviction's problem may be that of the step before it: whatever rows it tells of limit nothing (the refusal is
    the next one, a missing pointer)."""
    for kw in (dict(seqlen_q=1 << 30), dict(cu_seqlens_q=A, rows_q=1 << 30, seqlen_q=1 << 30)):
        assert evict(problem(**kw), k=None) == -1


def test_evict_budget_and_alias():
    for keep, recent in ((0, 0), (-1, 0), (5, 6), (5, -1)):
        assert evict(keep=keep, recent=recent) == -1
    assert evict(out=A) == -1  # the lengths it reads


def test_sizes_whose_indices_would_not_fit():
    """Key indices and places of kept keys, rounded up to what a CTA takes at a time, stay below 2^31."""
    wide = dict(B=1, H=1, Hkv=1, page_size=65536, max_pages=1 << 15)
    for seqlen_k, rc in (((1 << 31) - 1, -2), ((1 << 31) - (1 << 17), -2), ((1 << 31) - (1 << 17) - 1, -1)):
        p = problem(**wide, seqlen_k=seqlen_k)
        assert attend(p, q=None) == weights(p, q=None) == append(p, kn=None) == evict(p, k=None) == rc
    assert evict(problem(B=1, Hkv=1, H=1), keep=(1 << 31) - 1) == evict(problem(), keep=1 << 29) == -2


def test_append_takes_a_table_of_any_width():
    """The bound on the lengths limits the sizes, and an append has no use for a large one (the refusals are the next
    ones, a missing pointer)."""
    wide = dict(B=512, H=32, Hkv=32, page_size=16, num_pages=2000, max_pages=131072 // 16)
    sc = fa.Strides(32 * 128, 128, 16 * 32 * 128)
    assert append(problem(**wide, seqlen_k=1), sk=sc, sv=sc, kn=None) == -1


def test_packed_rows_are_limited_by_their_number_alone():
    """The bound on a packed batch's lengths sizes nothing: many sequences may stand beside one long prompt's bound."""
    p = problem(B=512, H=32, Hkv=8, cu_seqlens_q=A, rows_q=5000, seqlen_q=131072, seqlen_k=131072, max_pages=8192)
    assert fa.fa_fwd_paged_workspace_bytes(p, 152) > 0 and fa.fa_paged_key_weights_workspace_bytes(p, 152) > 0
    assert attend(p, q=None) == weights(p, q=None) == append(p, kn=None) == -1
    p = problem(B=512, H=32, Hkv=8, cu_seqlens_q=A, rows_q=1 << 20, seqlen_q=8, seqlen_k=1024)
    assert attend(p) == weights(p) == -2


def test_host_arrays_are_refused():
    """Arrays the kernels read must be device-accessible; this address is not (and there may be no GPU at all)."""
    import ctypes
    host = (ctypes.c_int32 * 64)()
    p = problem(page_table=ctypes.addressof(host), seqlens_k=ctypes.addressof(host))
    assert attend(p) == append(p) == weights(p) == evict(p) == -1


def test_binding_refuses():
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype)
    k = z(4, 16, 2, 64)
    table, lens = z(2, 3, dtype=torch.int32), z(2, dtype=torch.int32)
    good = dict(q=z(2, 1, 4, 64), k_cache=k, v_cache=k, page_table=table, seqlens_k=lens)
    for bad in (dict(), dict(page_table=table.long()), dict(seqlens_k=z(3, dtype=torch.int32)), dict(v_cache=z(4, 8, 2, 64)),
                dict(q=z(2, 1, 3, 64)), dict(q=z(2, 1, 4, 128)), dict(q=z(3, 1, 4, 64)), dict(q=z(2, 4, 64)),
                dict(out=z(2, 1, 4, 32)), dict(cu_seqlens_q=z(3, dtype=torch.int32))):
        with pytest.raises(ValueError):  # the first: these are CPU tensors
            fa.fwd_paged(**{**good, **bad})
    for keep, recent in ((0, 0), (3, 4), (3, -1)):
        with pytest.raises(ValueError):
            fa.paged_evict(k, k, z(4, 2, 16, dtype=torch.float32), table, lens, keep, recent=recent)
    for w in (z(4, 16, 2, dtype=torch.float32), z(4, 2, 16)):
        with pytest.raises(ValueError):
            fa.paged_evict(k, k, w, table, lens, 3)
    for call in (lambda s: fa.fwd_paged(**good, stream=s), lambda s: fa.paged_append(k[0], k[0], k, k, table, lens, stream=s),
                 lambda s: fa.paged_evict(k, k, z(4, 2, 16, dtype=torch.float32), table, lens, 3, stream=s)):
        with pytest.raises(ValueError, match="CUDA"):  # a stream beside CPU tensors
            call(0)


def test_stream_beside_keyword_arguments_in_any_order():
    """The device is that of the call's first tensor by name; CPU tensors get the refusal that names it."""
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype)
    k, w = z(4, 16, 2, 64), z(4, 2, 16, dtype=torch.float32)
    table, lens = z(2, 3, dtype=torch.int32), z(2, dtype=torch.int32)
    at = dict(page_table=table, seqlens_k=lens)
    for call in (lambda: fa.fwd_paged(causal=True, scale=0.5, **at, k_cache=k, v_cache=k, q=z(2, 1, 4, 64), stream=0),
                 lambda: fa.fwd_paged(cu_seqlens_q=None, stream=0, v_cache=k, k_cache=k, q=z(2, 1, 4, 64), **at),
                 lambda: fa.paged_append(**at, key_weights=None, k_cache=k, v_cache=k, v=k[:2], k=k[:2], stream=0),
                 lambda: fa.paged_key_weights(num_sms=3, **at, lse=w, key_weights=w, k_cache=k, q=z(2, 1, 4, 64), stream=0),
                 lambda: fa.paged_evict(keep=3, recent=1, **at, key_weights=w, v_cache=k, k_cache=k, stream=0)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(TypeError, match="q"):  # without the tensor: the call's own error
        fa.fwd_paged(causal=True, k_cache=k, v_cache=k, **at, stream=0)
    with pytest.raises(TypeError):
        fa.fwd_paged(stream=0)
