"""Sizes at the edge of what the feed-forward operators' C interface can say, on
the CPU: no call here launches a kernel."""
import os
import re
import subprocess

import pytest
import torch

import mlp_step_gb300 as M
from mlp_step_gb300 import build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return M.load()


def test_binding_refuses_sizes_past_32_bits(lib):
    """Pitches and row counts that a 32-bit int cannot hold are refused: passed
    on by their low bits, 2^32 + 8 would be read as rows 8 values apart."""
    e = lambda *a: torch.empty_strided(*a, dtype=torch.bfloat16, device="meta")  # noqa: E731
    for pitch in (1 << 31, (1 << 32) + 8):
        with pytest.raises(ValueError, match="pitches"):
            M._mat(e((2, 8), (pitch, 1)), "x", 2, 8, -1)
    with pytest.raises(ValueError, match="pitches"):
        M._mat(e(((1 << 32) + 5, 1), (1, 1)), "x", (1 << 32) + 5, 1, -1)
    assert M._mat(e((2, 8), ((1 << 31) - 1, 1)), "x", 2, 8, -1)[1] == (1 << 31) - 1
    # a single row's pitch is never used
    assert M._mat(e((1, 8), (1 << 33, 1)), "x", 1, 8, -1)[1] == 16
    big = (1 << 32) + 32
    for f in (lambda: M.mlp_ckpt8_scale_cols(big), lambda: M.mlp_layernorm_workspace_bytes(big, 64),
              lambda: M.mlp_linear_workspace_bytes(64, big, 64, torch.float32),
              lambda: M.mlp_linear_bwd_workspace_bytes(64, 64, big, torch.float32),
              lambda: M.mlp_act_bwd_workspace_bytes(big, 64),
              lambda: M.mlp_stack_ckpt8_workspace_bytes(2, big, 512, 512)):
        with pytest.raises(ValueError, match="at most"):
            f()


def test_size_queries_beyond_the_widths(lib):
    """No arithmetic of a size query overflows: widths that the calls refuse need
    no workspace, and an INT_MAX columns' scale bytes are counted."""
    most, wide = (1 << 31) - 1, (1 << 24) + 1
    assert M.mlp_ckpt8_scale_cols(most) == 1 << 26
    assert M.mlp_ckpt8_scale_cols(most - 31) == (1 << 26) - 1
    for n in (wide, most):
        for dt in (torch.bfloat16, torch.float32):
            assert M.mlp_linear_workspace_bytes(64, n, 64, dt) == 0
            assert M.mlp_linear_workspace_bytes(64, 64, n, dt) == 0
            assert M.mlp_linear_bwd_workspace_bytes(64, n, 64, dt) == 0
            assert M.mlp_linear_bwd_workspace_bytes(64, 64, n, dt) == 0
        assert M.mlp_act_bwd_workspace_bytes(64, n) == 0
    # the widest that are taken
    w = 1 << 24
    assert M.mlp_act_bwd_workspace_bytes(64, w) == 2 * w * 4
    assert M.mlp_linear_workspace_bytes(64, 64, w, torch.float32) == 64 * w * 4
    assert M.mlp_linear_bwd_workspace_bytes(most, w, 64, torch.float32) > most * w * 4


PER_DEVICE = r"""
#include "per_device.cuh"
#include <cstdio>
#include <thread>
#include <vector>
int main() {
  static mlp::PerDevice cache;
  std::atomic<int> made[70] = {}, wrong{0};
  std::vector<std::thread> threads;
  for (int t = 0; t < 8; ++t)
    threads.emplace_back([&] {
      for (int i = 0; i < 7000; ++i) {
        const int dev = i % 70 - 1;  // -1 (no device) and 64.. are made every time
        const int n = cache.get(dev, [&] { ++made[dev + 1]; return 100 + dev; });
        if (n != 100 + dev) ++wrong;
      }
    });
  for (auto& t : threads) t.join();
  int too_often = 0;
  for (int dev = 0; dev < 64; ++dev) too_often += made[dev + 1] < 1 || made[dev + 1] > 8;
  // a failure is not kept
  mlp::PerDevice late;
  const int first = late.get(3, [] { return 0; }), then = late.get(3, [] { return 5; });
  printf("%d %d %d %d %d %d\n", wrong.load(), too_often, made[0].load(), made[69].load(), first, then);
}
"""


def test_what_belongs_to_a_device_is_kept_per_device(tmp_path):
    """Launchers keep occupancy and kernel attributes per device, from any thread:
    the cache itself, and that no launcher has a plain static of its own."""
    csrc = os.path.join(os.path.dirname(M.__file__), "csrc")
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(PER_DEVICE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", "-x", "c++", str(src), "-I", csrc, "-o",
                    str(exe)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()
    assert out == ["0", "0", "800", "800", "0", "5"]
    plain = re.compile(r"^\s+static (const )?(int|bool|cudaError_t)\s+\w+(\[\d+\])?\s*=[^;]*$|"
                       r"^\s+static (int|bool) \w+(\[\d+\])? = (0|false|-1|\{false.*)")
    for f in sorted(os.listdir(csrc)):
        if f.startswith("k_") or f in ("common.cuh", "linear_tc.cuh"):
            with open(os.path.join(csrc, f)) as lines:
                for i, line in enumerate(lines, 1):
                    assert not plain.match(line.rstrip()), "%s:%d %s" % (f, i, line)
