"""Bounded waits of the attention over an 8-bit cache, tested without a GPU fault: the test-only build of the library whose
producers never load K/V must make every consumer's wait run out. The kernels then record FA_ERR_DEVICE_TIMEOUT, let the
copies they issued land, release their tensor memory and return, and the GPU stays usable. Runs in a child process."""

import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

_CHILD = r'''
import ctypes, sys
import torch
sys.path.insert(0, ROOT)
import exact_io_aware_38_gb300 as fa
from exact_io_aware_38_gb300 import build

build.build()
real = fa.lib()
broken = ctypes.CDLL(build.build_withhold_kv_test_lib())
for name, (res, args) in fa._SIGS.items():
    f = getattr(broken, name)
    f.restype, f.argtypes = res, args
g = torch.Generator("cuda").manual_seed(1)
B, Hkv, G, P, L = 3, 2, 4, 32, 700
pages = B * -(-L // P)
table = torch.arange(pages, dtype=torch.int32, device="cuda").view(B, -1)
lens = torch.tensor([L, 300, 1], dtype=torch.int32, device="cuda")
for d in (64, 128):
    k, v = (torch.randn(pages, P, Hkv, d, generator=g, device="cuda").to(torch.float8_e4m3fn) for _ in range(2))
    codes = torch.full((pages, Hkv, P, 2), 127, dtype=torch.uint8, device="cuda")
    # 4, 12, 24, 64, 128 and 400 rows per K/V head; by clusters and divided
    for n, sms in ((1, None), (1, 4), (3, 4), (6, None), (16, 4), (32, None), (100, None)):
        q = torch.randn(B, n, Hkv * G, d, generator=g, device="cuda").to(torch.bfloat16)
        args = (q, k, v, codes, table, lens)
        want = fa.fwd_paged_fp8(*args, causal=True, num_sms=sms)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        fa._lib = broken
        fa.fwd_paged_fp8(*args, causal=True, status=status, num_sms=sms)
        torch.cuda.synchronize()
        fa._lib = real
        assert int(status.item()) == -5, (d, n, int(status.item()))
        got = fa.fwd_paged_fp8(*args, causal=True, num_sms=sms)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), (d, n)
print("CHILD_OK")
'''


def test_paged_fp8_bounded_waits_report_timeout_and_gpu_stays_usable():
    r = subprocess.run([sys.executable, "-c", f"ROOT = {ROOT!r}\n" + _CHILD], capture_output=True, text=True, timeout=600,
                       cwd=ROOT)
    assert r.returncode == 0 and "CHILD_OK" in r.stdout, (r.returncode, r.stdout[-2000:], r.stderr[-4000:])
