"""The paged 8-bit cache at the ends of what it accepts, without a GPU."""
import ctypes
import subprocess
import sys

import pytest

from block_sparse_long_pool_gb300 import binding, build
from test_paged_cpu import ATTN, PLAN

INVALID, UNSUPPORTED = binding.SPARSE_ERR_INVALID_ARG, binding.SPARSE_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


@pytest.mark.parametrize("max_blocks", [1 << 25, 2 ** 31 - 1])
def test_plan_refuses_tables_past_31_bits_of_tokens(lib, max_blocks):
    """2^25 blocks are 2^31 tokens: a length of 2^31 - 1 and one token more would not fit an int32
    length, and a block count of it, (length + 63) / 64, would wrap."""
    assert lib.sparse_page_plan(*{**PLAN, "max_blocks": max_blocks}.values()) == UNSUPPORTED
    assert "max_blocks" in lib.sparse_last_error().decode()


@pytest.mark.parametrize("scale", [2.4e38, -3.4e38, float("-inf")])
def test_attn_refuses_scales_that_overflow_in_base_2(lib, scale):
    """Times log2(e) they are infinite, which would make NaN of a score of zero."""
    assert lib.sparse_paged_decode_attn_f8(*{**ATTN, "sm": scale}.values()) == INVALID
    assert "scale" in lib.sparse_last_error().decode()


def test_only_the_paged_calls_need_the_module_that_marshals_them(monkeypatch, tmp_path):
    """It is built for one version of torch: without it (another torch) every other call loads."""
    build.build()
    monkeypatch.setattr(binding, "MARSHAL_PATH", str(tmp_path / "absent.so"))
    monkeypatch.setattr(binding, "_marshal", None)
    monkeypatch.setattr(binding, "_lib", None)
    assert binding.load().sparse_version() >= 100
    assert binding.status_string(binding.SPARSE_ERR_NO_PAGES)
    with pytest.raises(RuntimeError, match="absent.so is not built"):
        binding._passed("page_plan", 0, None)
    monkeypatch.undo()
    binding._load_marshal()
    assert binding._marshal is not None


def test_the_library_builds_without_torch(tmp_path):
    """A C program's user needs nvcc alone: linked here into a place of its own."""
    build.build()
    code = ("import sys; sys.modules['torch'] = None\n"
            "from block_sparse_long_pool_gb300 import build\n"
            f"build.LIB = {str(tmp_path / 'lib.so')!r}\n"
            "print(build.build())")
    r = subprocess.run([sys.executable, "-c", code], cwd=build.ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    assert r.stdout.strip() == str(tmp_path / "lib.so")
    assert ctypes.CDLL(r.stdout.strip()).sparse_version() >= 100
