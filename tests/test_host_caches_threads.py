"""What the library looks up once per device may be looked up by any thread: eight threads at once under the thread sanitizer
(host code alone; without a GPU the lookups fail and are cached all the same)."""

import os
import subprocess

import pytest

from head_latent_attention_absorb_b200 import build as B

SOURCE = r"""
#include <thread>
#include <vector>
#include "common.cuh"
#include "tma_host.h"
__global__ void kernel() {}
int main() {
  static mla::PerDevice allowed;
  std::vector<std::thread> threads;
  for (int i = 0; i < 8; ++i)
    threads.emplace_back([] {
      mla::sm_count();
      mla::allow_smem(reinterpret_cast<const void*>(kernel), 1000, allowed);
      allowed.set(0, 1000);
      mla::allow_smem(reinterpret_cast<const void*>(kernel), 1000, allowed);
      mla::encode_tiled_fn();
    });
  for (auto& t : threads) t.join();
  return 0;
}
"""


def test_lookups_from_many_threads(tmp_path):
    src, exe = tmp_path / "threads.cu", tmp_path / "threads"
    src.write_text(SOURCE)
    sanitize = ["-Xcompiler", "-fsanitize=thread", "-ltsan"]
    plain = tmp_path / "plain.cu"
    plain.write_text("int main() { return 0; }\n")
    r = subprocess.run([B.NVCC, *sanitize, "-o", str(tmp_path / "plain"), str(plain)], capture_output=True)
    if r.returncode != 0 or subprocess.run([str(tmp_path / "plain")], capture_output=True).returncode != 0:
        pytest.skip("no thread sanitizer here")
    flags = [f for f in B.FLAGS if f != "-O3"]
    r = subprocess.run([B.NVCC, *B.ARCH, *flags, *sanitize, "-o", str(exe), str(src)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    # (races inside the CUDA runtime, which is not instrumented, are not looked at)
    env = dict(os.environ, TSAN_OPTIONS="ignore_noninstrumented_modules=1 halt_on_error=0")
    r = subprocess.run([str(exe)], capture_output=True, text=True, env=env, timeout=120)
    races = [line for line in r.stderr.splitlines() if "mla::" in line]
    assert not races, "\n".join(races[:8])
