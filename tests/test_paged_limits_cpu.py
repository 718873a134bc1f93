"""The paged 8-bit cache at the ends of what it accepts, without a GPU."""
import ctypes
import json
import os
import subprocess
import sys
import types

import numpy as np
import pytest
import torch

import paged_long as long
from block_sparse_long_pool_gb300 import binding, build
from block_sparse_long_pool_gb300 import workloads as wl
from test_paged_cpu import ATTN, PLAN

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bench  # noqa: E402

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


@pytest.mark.parametrize("n", [20032, 40000, 131072])
def test_the_bound_of_long_lists_shows_a_lost_or_repeated_tile(n):
    """What the attention's long lists are compared with: an answer with rounded weights passes, one
    with a tile of 64 tokens left out or counted twice does not, wherever it is."""
    rng = np.random.default_rng(n)
    K, V = rng.standard_normal((2, n, 128)) * 64 / 2 ** 7
    K, V = (torch.as_tensor(x * 32).to(torch.float8_e4m3fn).double().numpy() / 32 for x in (K, V))
    Q = torch.as_tensor(rng.standard_normal((2, 128))).to(torch.bfloat16).double().numpy()
    want = long.attend(Q, K, V)

    def answer(times):
        O, lse, _, _ = long.attend(Q, K, V, times=times)
        return torch.as_tensor(O).to(torch.bfloat16).double().numpy(), lse.astype(np.float32)

    long.assert_close(*answer(None), want)
    s = Q @ K.T / np.sqrt(128)
    p = np.exp(s - s.max(1, keepdims=True))
    rounded = (p * 4096).astype(np.float16).astype(np.float64) / 4096   # the weights of O; the sum keeps its own
    O = rounded @ V / p.sum(1, keepdims=True)
    long.assert_close(torch.as_tensor(O).to(torch.bfloat16).double().numpy(), want[1].astype(np.float32), want)
    blocks = -(-n // 64)
    for j in [0, 1, blocks - 2, *rng.integers(0, blocks - 1, 5).tolist()]:
        for count in (0.0, 2.0):
            times = np.ones(n)
            times[64 * j:64 * j + 64] = count
            with pytest.raises(AssertionError, match="of its bound"):
                long.assert_close(*answer(times), want)


def test_the_paged_case_says_what_its_cpu_baseline_is(monkeypatch):
    """The oracle has no paged cache: the line says that the baseline's is the contiguous bf16 one."""
    shape = wl.DecodeShape("tiny", B=1, H_q=2, H_kv=1, T=256, n_init=1, n_local=1, k=1, n_planted=1, n_new=1, seed=3)
    lay = types.SimpleNamespace(sh=shape, x=wl.single_layer(shape))
    plain = bench.single_layer_oracle(lay, 0.0)["sample"]
    assert "in fp64;" in plain
    lines = []
    monkeypatch.setattr(bench, "measured_peaks", lambda: (1000.0, "test"))
    monkeypatch.setattr(bench, "_PagedLayer", lambda sh, dev: types.SimpleNamespace(
        sh=shape, x=lay.x, step=None, attend=None, status=torch.zeros(1)))
    monkeypatch.setattr(bench, "_event_times", lambda *a: {"median_us": 1.0})
    monkeypatch.setattr(torch.cuda, "synchronize", lambda: None)
    monkeypatch.setattr(torch, "ones", lambda *a, **k: None)
    monkeypatch.setattr("builtins.print", lambda text, **k: lines.append(json.loads(text)))
    args = types.SimpleNamespace(steps=1, warmup=0, no_cpu_baseline=False, case_cpu_seconds=0.0)
    bench.run_paged_case(args, torch.device("cpu"))
    assert "contiguous bf16 cache" in lines[0]["cpu_baseline"]["sample"]
