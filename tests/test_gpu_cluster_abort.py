"""Split sums of the decode product over a 4-bit base: when one CTA of a cluster has given up a wait, no CTA
stores rows that its sums belong to.  The product asks cluster_unaborted, which is run here on clusters
whose CTAs raise the flag as told: no wait has to run out for it."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "adapter_gemm_segment_gb300", "csrc")

SOURCE = r"""
#include "common.cuh"
#include "tc_ptx.cuh"
using namespace lora;
__global__ void agree(const int* raise, int* out, int ctas) {
    __shared__ int flag[4];
    const int c = blockIdx.y;
    if (threadIdx.x == 0) flag[1] = raise[blockIdx.x * ctas + c];
    __syncthreads();
    ptx::cluster_sync();
    const bool ok = ptx::cluster_unaborted(&flag[1], ctas);
    out[(blockIdx.x * ctas + c) * blockDim.x + threadIdx.x] = ok;
    ptx::cluster_sync();
}
extern "C" int run(const int* raise, int* out, int clusters, int ctas, void* stream) {
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = dim3(clusters, ctas);
    cfg.blockDim = dim3(64);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = 1;
    at[0].val.clusterDim.y = ctas;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, agree, raise, out, ctas);
}
"""


@pytest.fixture(scope="module")
def agree(tmp_path_factory):
    d = tmp_path_factory.mktemp("cluster_abort")
    src, so = str(d / "agree.cu"), str(d / "agree.so")
    with open(src, "w") as f:
        f.write(SOURCE)
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    subprocess.run([nvcc, "-gencode", "arch=compute_103a,code=sm_103a", "-O2", "-std=c++17", "-Xcompiler", "-fPIC",
                    "--expt-relaxed-constexpr", "-I", CSRC, "-shared", "-o", so, src], check=True)
    return ctypes.CDLL(so).run


@pytest.mark.gpu
@pytest.mark.parametrize("ctas", [2, 3, 4, 8])
def test_one_abort_is_everyones(agree, ctas):
    torch.cuda.init()
    masks = list(range(1 << ctas))
    raise_ = torch.tensor([[(m >> c) & 1 for c in range(ctas)] for m in masks], dtype=torch.int32, device="cuda")
    out = torch.full((len(masks), ctas, 64), -1, dtype=torch.int32, device="cuda")
    rc = agree(ctypes.c_void_p(raise_.data_ptr()), ctypes.c_void_p(out.data_ptr()), len(masks), ctas,
               ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert rc == 0
    torch.cuda.synchronize()
    assert (out[0] == 1).all() and (out[1:] == 0).all()


def test_the_decode_product_asks_before_it_stores():
    with open(os.path.join(CSRC, "fp4_decode.cu")) as f:
        text = f.read()
    asked = text.index("good = cluster_unaborted(flags, a.splits)")
    assert text.index("cluster_sync();") < asked < text.index("if (warp >= 2 && good && store && recv)")
    assert text.count("good = cluster_unaborted(flags, a.splits)") == 2  # with pushed sums and with remote reads
