"""The waits of the tensor-core kernels end by themselves: on a barrier at which nothing arrives a wait gives up after
2^22 tries, sets the status bit and the abort flag of its CTA, and the flag of a pair's other CTA ends that one's
waits at once.  A kernel of two CTAs that does nothing else, compiled here against the kernels' own header."""
import ctypes
import os
import subprocess

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import quantized_expert_ffn_sigmoid_gb300 as cm  # noqa: E402
from quantized_expert_ffn_sigmoid_gb300 import build  # noqa: E402

SOURCE = r'''
#include "tcgen05.cuh"
using namespace colimoe;
__device__ unsigned long long now() { unsigned long long t; asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t)); return t; }
// out[CTA]: result of its wait, its nanoseconds, its flag
__global__ void __cluster_dims__(2, 1, 1) waits(uint32_t* status, long long* out, int arrive, int late_us) {
  __shared__ uint64_t bar;
  __shared__ volatile int abort_flag;
  const int rank = blockIdx.x;
  if (threadIdx.x == 0) {
    mbar_init(&bar, 1);
    abort_flag = 0;
    fence_barrier_init();
  }
  __syncthreads();
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
  if (threadIdx.x == 0) {
    const unsigned long long begin = now();
    if (rank == 0)
      for (int i = 0; i < 100000 && now() - begin < 1000ull * late_us; ++i) __nanosleep(10000);
    if (arrive) mbar_arrive(&bar);
    const unsigned long long t0 = now();
    const bool ok = gwait(&bar, 0, status, &abort_flag);
    if (!ok) abort_other(&abort_flag);
    out[3 * rank] = ok;
    out[3 * rank + 1] = (long long)(now() - t0);
    const bool again = gwait(&bar, 0, status, &abort_flag);   // at once
    out[3 * rank] += 2 * again;
  }
  __syncthreads();
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
  if (threadIdx.x == 0) out[3 * rank + 2] = abort_flag;
}
extern "C" int run(uint32_t* status, long long* out, int arrive, int late_us, cudaStream_t st) {
  waits<<<2, 32, 0, st>>>(status, out, arrive, late_us);
  return (int)cudaGetLastError();
}
'''


@pytest.fixture(scope="module")
def run(tmp_path_factory):
    d = tmp_path_factory.mktemp("waits")
    (d / "waits.cu").write_text(SOURCE)
    r = subprocess.run([build.nvcc(), *build.ARCH, "-O3", "-std=c++17", "-Xcompiler", "-fPIC", "-shared", "-I", build.CSRC, "-o", str(d / "waits.so"),
                        str(d / "waits.cu"), "-lcudart"], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    lib = ctypes.CDLL(os.path.join(d, "waits.so"))
    lib.run.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_void_p]

    def call(arrive, late_us):
        status, out = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.full((6,), -1, dtype=torch.int64, device="cuda")
        assert lib.run(status.data_ptr(), out.data_ptr(), arrive, late_us, torch.cuda.current_stream().cuda_stream) == 0
        torch.cuda.synchronize()
        return int(status[0]), out.view(2, 3).tolist()
    return call


def test_a_wait_that_is_met(run):
    status, (a, b) = run(1, 0)
    assert status == 0 and a[0] == b[0] == 3 and a[2] == b[2] == 0


def test_a_wait_that_runs_out_in_one_cta_ends_both(run):
    status, (a, b) = run(0, 700000)
    assert status == cm.STATUS_TIMEOUT and a[0] == b[0] == 0 and a[2] == b[2] == 1
    # below two seconds; the first CTA began 0.7 s later and was told, at once or before
    assert b[1] < 2e9 and a[1] < max(b[1] - 0.6e9, 1e7)
