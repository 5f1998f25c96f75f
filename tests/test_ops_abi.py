"""Argument validation of the balance loss, the 4-bit matrix-vector products and the paged cache, and the
cache's slot arithmetic: a host build of csrc/ops_api.cpp under AddressSanitizer and UndefinedBehaviorSanitizer
with stand-in launchers (tests/native/ops_check.cpp), and the binding's own refusals."""

import os
import shutil
import subprocess

import pytest
import torch

import mixed_precision_moe_amd as mx

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_validation_and_slots_under_asan_and_ubsan(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    exe = str(tmp_path / "ops_check")
    sources = [os.path.join(ROOT, "mixed_precision_moe_amd", "csrc", "ops_api.cpp"),
               os.path.join(ROOT, "tests", "native", "ops_check.cpp")]
    cmd = [cxx, "-std=c++17", "-g", "-O1", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
           "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I" + os.path.join(ROOT, "include"), *sources, "-o", exe]
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    assert r.returncode == 0, r.stdout
    r = subprocess.run([exe], stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True, timeout=120)
    assert r.returncode == 0 and "ops checks passed" in r.stdout, r.stdout


def test_host_tensors_are_refused():
    x = torch.zeros(1, 64, dtype=torch.bfloat16)
    q, s = torch.zeros(16, 32, dtype=torch.uint8), torch.zeros(16, 2, dtype=torch.uint8)
    with pytest.raises(ValueError, match="GPU tensor"):
        mx.fp4_matvec(x, q, s)
    with pytest.raises(ValueError, match="GPU tensor"):
        mx.fp4_expert_matvec(x, q[None], s[None], torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError, match="GPU tensor"):
        mx.balance_loss(torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32))
    with pytest.raises(ValueError, match="GPU tensor"):
        mx.PagedCache(2, 16, 1, 64, fmt=mx.FMT_MXFP4, v_dim=0,
                      storage=(torch.zeros(2, 16, 1, 32, dtype=torch.uint8), torch.zeros(2, 16, 1, 2, dtype=torch.uint8),
                               None, None))


@pytest.mark.parametrize("kw", [dict(k_dim=48), dict(heads=0), dict(page_size=0), dict(num_pages=-1), dict(fmt=9),
                                dict(fmt=mx.FMT_NVFP4, k_global_scale=0.0),
                                dict(fmt=mx.FMT_NVFP4, v_global_scale=float("nan"))])
def test_cache_shapes_are_refused(kw):
    args = dict(num_pages=4, page_size=16, heads=2, k_dim=64)
    args.update(kw)
    with pytest.raises(mx.Mxfp4Error):
        mx.PagedCache(**args)


def test_cache_storage_must_fit():
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)  # noqa: E731
    good = (u8(4, 16, 2, 64), u8(4, 16, 2, 2), u8(4, 16, 2, 32), u8(4, 16, 2, 1))
    for i in range(4):
        bad = list(good)
        bad[i] = bad[i][:, :15]
        with pytest.raises(ValueError, match=("k_q", "k_s", "v_q", "v_s")[i]):
            mx.PagedCache(4, 16, 2, 64, 32, storage=tuple(bad))
