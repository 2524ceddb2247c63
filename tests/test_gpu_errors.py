"""A call that fails leaves no error behind for the next one."""
import ctypes

import pytest
import torch

from grouped_gemm_moe_gb300 import binding as B

from _parity import dev, ensure_built

pytestmark = pytest.mark.gpu


def test_a_failed_call_does_not_fail_the_next():
    """The status read synchronises, which a capturing stream refuses; the capture is dropped
    (the CUDA runtime is called directly: torch keeps state about its own captures)."""
    ensure_built()
    rt = ctypes.CDLL("libcudart.so." + torch.version.cuda.split(".")[0])
    x, gain = torch.ones(4, 64, device=dev()).to(torch.bfloat16), torch.ones(64, device=dev())
    want, _ = B.moe_norm_in(x, gain)
    ws = B.new_workspace(B.WORKSPACE_HEADER, dev())
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    handle, graph = ctypes.c_void_p(side.cuda_stream), ctypes.c_void_p()
    relaxed = 2
    assert rt.cudaStreamBeginCapture(handle, relaxed) == 0
    with torch.cuda.stream(side):
        with pytest.raises(B.MoEError) as e:
            B.moe_read_device_status(ws)
    left = rt.cudaPeekAtLastError()      # what the next launch, here or in torch, would report
    assert e.value.status == B.MOE_ERR_CUDA and B.load().moe_last_cuda_error() != 0
    assert rt.cudaStreamEndCapture(handle, ctypes.byref(graph)) != 0
    rt.cudaGetLastError()                # the test's own
    assert left == 0
    got, _ = B.moe_norm_in(x, gain)
    assert torch.equal(got, want)
