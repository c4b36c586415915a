"""Bounded waits of the paged-cache kernels, tested without a GPU fault: the test-only build of the library whose
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
rand = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)
B, Hkv, G, P, L = 3, 2, 4, 32, 700
pages = B * -(-L // P)
table = torch.arange(pages, dtype=torch.int32, device="cuda").view(B, -1)
lens = torch.tensor([L, 300, 1], dtype=torch.int32, device="cuda")
for d in (64, 128):
    k, v = rand(pages, P, Hkv, d), rand(pages, P, Hkv, d)
    w = torch.zeros(pages, Hkv, P, device="cuda")
    for n, sms in ((1, None), (1, 4), (100, None)):  # few rows by clusters and divided, many rows
        q = rand(B, n, Hkv * G, d)
        want = fa.fwd_paged(q, k, v, table, lens, causal=True, num_sms=sms)
        for call in ("attend", "weights"):
            status = torch.zeros(1, dtype=torch.int32, device="cuda")
            fa._lib = broken
            if call == "attend":
                fa.fwd_paged(q, k, v, table, lens, causal=True, status=status, num_sms=sms)
            else:
                fa.paged_key_weights(q, k, table, lens, want[1], w, causal=True, status=status, num_sms=sms)
            torch.cuda.synchronize()
            fa._lib = real
            assert int(status.item()) == -5, (d, n, call, int(status.item()))
            got = fa.fwd_paged(q, k, v, table, lens, causal=True, num_sms=sms)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), (d, n, call)
print("CHILD_OK")
'''


def test_paged_bounded_waits_report_timeout_and_gpu_stays_usable():
    r = subprocess.run([sys.executable, "-c", f"ROOT = {ROOT!r}\n" + _CHILD], capture_output=True, text=True, timeout=600,
                       cwd=ROOT)
    assert r.returncode == 0 and "CHILD_OK" in r.stdout, (r.returncode, r.stdout[-2000:], r.stderr[-4000:])
