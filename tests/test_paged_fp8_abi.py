"""Host-side checks of the 8-bit cache's entry points (no GPU): every refusal comes before any launch."""

import pytest
import torch

import exact_io_aware_38_gb300 as fa
from exact_io_aware_38_gb300 import build
from test_paged_abi import A, SN, SQ, problem

SC = fa.Strides(2 * 128, 128, 16 * 2 * 128)  # (in bytes)


@pytest.fixture(scope="module", autouse=True)
def L():
    build.build()
    return fa.lib()


def attend(p=None, sms=152, q=A, sq=SQ, k=A, sk=SC, v=A, sv=SC, c=A, o=A, so=SQ, lse=A, ws=A, nbytes=1 << 40, status=None):
    return fa.fa_fwd_paged_fp8(p or problem(), sms, q, sq, k, sk, v, sv, c, o, so, lse, ws, nbytes, status, None)


def append(p=None, kn=A, skn=SN, vn=A, svn=SN, k=A, sk=SC, v=A, sv=SC, c=A, status=None):
    return fa.fa_paged_append_fp8(p or problem(), kn, skn, vn, svn, k, sk, v, sv, c, status, None)


def read(p=None, kn=A, skn=SN, vn=A, svn=SN, k=A, sk=SC, v=A, sv=SC, c=A, status=None):
    return fa.fa_paged_read_fp8(p or problem(), kn, skn, vn, svn, k, sk, v, sv, c, status, None)


@pytest.mark.parametrize("kw,rc", [
    (dict(B=0), -1), (dict(Hkv=0), -1), (dict(page_size=0), -1), (dict(num_pages=0), -1), (dict(max_pages=0), -1),
    (dict(seqlen_k=0), -1), (dict(seqlen_q=0), -1), (dict(page_table=None), -1), (dict(seqlens_k=None), -1),
    (dict(cu_seqlens_q=A, rows_q=0), -1), (dict(d=96), -2), (dict(page_size=24), -2), (dict(page_size=4), -2),
    (dict(page_size=1 << 17), -2), (dict(page_table=A + 2), -3), (dict(seqlens_k=A + 1), -3),
    (dict(cu_seqlens_q=A + 2, rows_q=9), -3),
    (dict(B=1 << 12, max_pages=1 << 20, seqlen_k=1 << 20), -2),  # B Hkv keys past 2^31
    (dict(B=1 << 22, seqlen_q=2), -2)])                         # rows past 2^31 elements
def test_problem_refusals(kw, rc):
    p = problem(**kw)
    assert attend(p) == rc and append(p) == rc and read(p) == rc


@pytest.mark.parametrize("kw,rc", [(dict(H=0), -1), (dict(H=7), -1), (dict(causal=2), -1), (dict(scale=0.0), -1),
                                   (dict(scale=float("inf")), -1)])
def test_problem_refusals_of_the_attention(kw, rc):
    assert attend(problem(**kw)) == rc and append(problem(**kw), c=None) == -1


def test_sequences_past_the_counters_of_the_attention():
    """2^26 sequences, times heads, of packed rows: few of them can have tokens. Append and reading take them (their next
    refusal is a misaligned pointer)."""
    kw = dict(Hkv=2, H=2, max_pages=1, page_size=8, seqlen_k=8, seqlen_q=1, cu_seqlens_q=A, rows_q=1 << 20)
    big, fits = problem(B=1 << 25, **kw), problem(B=(1 << 25) - 1, **kw)
    assert attend(big) == -2 and fa.fa_fwd_paged_fp8_workspace_bytes(big, 152) == 0
    assert attend(fits, lse=A + 2) == append(big, c=A + 2) == read(big, c=A + 2) == -3
    assert fa.fa_fwd_paged_fp8_workspace_bytes(fits, 152) > 0


def test_buffer_refusals():
    for call, names in ((attend, "q k v c o lse"), (append, "kn vn k v c"), (read, "kn vn k v c")):
        for n in names.split():
            assert call(**{n: None}) == -1, (call, n)
            assert call(**{n: A + 2}) == -3, (call, n)
        assert call(status=A + 2) == -3
        assert call(c=A + 8) == -3
        for s in (fa.Strides(0, 128, 8192), fa.Strides(256, 136, 8192), fa.Strides(264, 128, 8192), fa.Strides(256, 128, 8200),
                  fa.Strides(256, 128, 0), fa.Strides(-256, 128, 8192)):
            assert call(sk=s) == call(sv=s) == -1, (call, s.row, s.head, s.batch)
        assert call(sk=fa.Strides(256, 128, 1 << 39)) == -2
    for s in (fa.Strides(0, 128, 8192), fa.Strides(256, 12, 8192), fa.Strides(256, 128, 0)):
        assert attend(sq=s) == attend(so=s) == append(skn=s) == append(svn=s) == read(skn=s) == read(svn=s) == -1


def test_one_page_needs_no_page_stride():
    """(the refusal is then the next one: a misaligned pointer)"""
    p = problem(num_pages=1)
    s = fa.Strides(256, 128, 0)
    assert attend(p, sk=s, sv=s, lse=A + 2) == append(p, sk=s, sv=s, c=A + 2) == read(p, sk=s, sv=s, c=A + 2) == -3


def test_workspace_rules():
    for kw in (dict(max_pages=1000, seqlen_k=9000), dict(seqlen_q=500), dict(B=200, max_pages=1000, seqlen_k=9000)):
        p = problem(**kw)
        need = fa.fa_fwd_paged_fp8_workspace_bytes(p, 152)
        assert need > 0 and need % 256 == 0
        assert fa.fa_fwd_paged_fp8_workspace_bytes(p, 0) == fa.fa_fwd_paged_fp8_workspace_bytes(p, 1025) == 0
        for sms, ws, nbytes, rc in ((0, A, 1 << 40, -1), (1025, A, 1 << 40, -1), (152, None, 1 << 40, -1),
                                    (152, A, need - 1, -1), (152, A + 16, 1 << 40, -3)):
            assert attend(p, sms=sms, ws=ws, nbytes=nbytes) == rc
    assert fa.fa_fwd_paged_fp8_workspace_bytes(problem(d=96), 152) == 0


def test_workspace_of_chunks_stops_growing_with_the_sequences():
    """Keys and values read back for many rows take 1 GiB, or one sequence's."""
    size = lambda **kw: fa.fa_fwd_paged_fp8_workspace_bytes(problem(seqlen_q=500, max_pages=1 << 16, **kw), 152)  # noqa: E731
    assert size(seqlen_k=1000) < size(seqlen_k=2000) < size(seqlen_k=2000, B=4)
    assert size(seqlen_k=20_000, B=1000) <= size(seqlen_k=20_000, B=2000) < 1.2 * (1 << 30)
    one = 1_000_064 * 2 * 128 * 2 * 2  # its last 128-key tile included
    assert one <= size(seqlen_k=1_000_000, B=7) < one + (1 << 28)


def tensors(**kw):
    t = dict(q=torch.zeros(2, 3, 8, 128, dtype=torch.bfloat16), k=torch.zeros(2, 3, 2, 128, dtype=torch.bfloat16),
             k_cache=torch.zeros(5, 16, 2, 128, dtype=torch.float8_e4m3fn), scales=torch.zeros(5, 2, 16, 2, dtype=torch.uint8),
             table=torch.zeros(2, 4, dtype=torch.int32), lens=torch.zeros(2, dtype=torch.int32))
    t.update(kw)
    return t


@pytest.mark.parametrize("kw,match", [
    (dict(), "CUDA tensor"),  # all else is right: a CPU tensor is refused
    (dict(scales=torch.zeros(5, 16, 2, 2, dtype=torch.uint8)), "scales must be"),
    (dict(scales=torch.zeros(5, 2, 16, 2, dtype=torch.int8)), "scales must be"),
    (dict(scales=torch.zeros(5, 2, 2, 16, dtype=torch.uint8).transpose(2, 3)), "scales must be"),
    (dict(table=torch.zeros(2, 4, dtype=torch.int64)), "page_table"),
    (dict(lens=torch.zeros(3, dtype=torch.int32)), "seqlens_k"),
    (dict(q=torch.zeros(2, 3, 8, 64, dtype=torch.bfloat16), k=torch.zeros(2, 3, 2, 64, dtype=torch.bfloat16)), "new tokens"),
])
def test_helper_refusals(kw, match):
    t = tensors(**kw)
    with pytest.raises(ValueError, match=match):
        fa.fwd_paged_fp8(t["q"], t["k_cache"], t["k_cache"], t["scales"], t["table"], t["lens"])
    for call in (fa.paged_append_fp8, fa.paged_read_fp8):
        with pytest.raises(ValueError, match=match):
            call(t["k"], t["k"], t["k_cache"], t["k_cache"], t["scales"], t["table"], t["lens"])


def test_helper_refuses_rows_of_other_shapes():
    t = tensors()
    for call in (fa.paged_append_fp8, fa.paged_read_fp8):
        for k, v in ((t["k"], t["k"][:, :2]), (t["q"], t["q"])):  # (more heads than the cache)
            with pytest.raises(ValueError, match="one shape"):
                call(k, v, t["k_cache"], t["k_cache"], t["scales"], t["table"], t["lens"])
    with pytest.raises(ValueError, match="one shape"):
        fa.fwd_paged_fp8(t["q"], t["k_cache"], t["k_cache"][:, :8], t["scales"], t["table"], t["lens"])
