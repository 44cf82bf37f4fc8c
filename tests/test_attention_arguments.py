"""What the attention entry points tell the kernels (CPU): api.cpp is linked with a launcher that only keeps its arguments."""

import ctypes
import os
import shutil
import subprocess

import pytest

from test_cache_abi import attention, cache
from test_host_sanitizers import CSRC, ROOT
from w4a4_bit_quantized_amd import binding

ERR_HIP = 5


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    path = str(tmp_path_factory.mktemp("record") / "libw4a4_record.so")
    stubs = [os.path.join(ROOT, "tests", "sanitize", f) for f in ("launch_stub.cpp", "record_attention.cpp")]
    cmd = ["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-Wl,-Bsymbolic", "-D__HIP_PLATFORM_AMD__", "-I",
           os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "include"), "-I", os.path.join(ROOT, "include"), "-I", CSRC,
           os.path.join(CSRC, "api.cpp"), os.path.join(CSRC, "lowrank_split.cpp"), *stubs, "-pthread", "-o", path]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-3000:]
    return binding.open_library(path)


def test_a_pool_of_no_pages_has_no_table(lib):
    """With no pages, page_table may be NULL or lie anywhere: whatever the lengths say, no entry of it is read."""
    lens = (ctypes.c_int32 * 2)(5, 100)
    at = ctypes.addressof(lens)
    assert attention(lib, lens=at) == ERR_HIP                             # 8 entries of 16 tokens a row: all are looked at
    assert lib.attention_table_entries() == 1 + 7 and lib.attention_max_len() == 128
    for tree in (None, (0x10000, 8, 3, 0x10000)):
        for table in (None, 0x10002):
            assert attention(lib, lens=at, table=table, c=cache(pages=0, k=None, v=None), tree=tree, window=3) == ERR_HIP
            assert lib.attention_table_entries() == 0 and lib.attention_max_len() == 0
