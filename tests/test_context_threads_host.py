"""What calls from several threads leave in a context (no GPU): the launch count
of one whole call and one whole error text.  A small program hammers both from
four threads."""
import os
import shutil
import subprocess

from deepseek_sparse_attention_dsa_gb300 import build as dsa_build

PROGRAM = r"""
#include <cstdio>
#include <cstring>
#include <thread>
#include <vector>
#include "dsa_internal.h"
int main() {
  dsa_ctx ctx;
  const char *a = dsa::cuda_error_text(cudaErrorInvalidValue), *b = dsa::cuda_error_text(cudaErrorNotReady);
  if (!std::strstr(a, "cudaErrorInvalidValue: ") || !std::strstr(b, "cudaErrorNotReady: ")) return 1;
  if (dsa_last_launch_count(&ctx) != 0 || std::strcmp(dsa_last_cuda_error(&ctx), "")) return 2;
  std::atomic<int> bad{0};
  std::vector<std::thread> threads;
  for (int t = 0; t < 4; ++t)
    threads.emplace_back([&, t] {
      for (int i = 0; i < 20000; ++i) {
        {
          dsa::LaunchCount launched(&ctx);
          launched.n += 2;
        }
        if (dsa::cuda_status(&ctx, t & 1 ? cudaErrorInvalidValue : cudaErrorNotReady) != DSA_ERR_CUDA) ++bad;
        if (dsa::cuda_status(&ctx, cudaSuccess) != DSA_OK) ++bad;
        const char *text = dsa_last_cuda_error(&ctx);
        if (dsa_last_launch_count(&ctx) != 2 || (std::strcmp(text, a) && std::strcmp(text, b))) ++bad;
        // texts of codes that no thread has asked for yet
        const char *other = dsa::cuda_error_text(static_cast<cudaError_t>(100 + i % 300));
        if (!std::strstr(other, ": ")) ++bad;
      }
    });
  for (auto &t : threads) t.join();
  return bad ? 3 : 0;
}
"""


def test_threads_leave_one_calls_count_and_text(tmp_path):
    lib = dsa_build.build()
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(dsa_build._nvcc())))
    src, exe = tmp_path / "threads.cpp", tmp_path / "threads"
    src.write_text(PROGRAM)
    cmd = [shutil.which("g++") or "g++", "-std=c++17", "-O1", str(src), "-o", str(exe), "-I", dsa_build.INCLUDE,
           "-I", dsa_build.CSRC, "-isystem", os.path.join(cuda, "include"), lib, "-L", os.path.join(cuda, "lib64"), "-lcudart",
           "-pthread", "-Wl,-rpath," + os.path.dirname(lib), "-Wl,-rpath," + os.path.join(cuda, "lib64")]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, (r.returncode, r.stderr[-3000:])
