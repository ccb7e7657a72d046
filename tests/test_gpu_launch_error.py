"""A launch that CUDA refuses is reported by its own call and leaves nothing for the next one."""
import ctypes

import pytest
import torch

import continuous_softmax_attention_gb300 as csa
from continuous_softmax_attention_gb300 import _lib as L

pytestmark = pytest.mark.gpu


def test_a_refused_launch_is_reported_once():
    # While a stream that waits for the legacy stream is being captured, CUDA refuses launches on the legacy one.
    cudart = ctypes.CDLL("libcudart.so.%s" % torch.version.cuda.split(".")[0])
    refs, table = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.full((1, 2), -1, dtype=torch.int32, device="cuda")
    lens, counts, short = (torch.tensor([n], dtype=torch.int32, device="cuda") for n in (0, 3, 9))
    torch.cuda.synchronize()

    def reserve(stream):
        at = [ctypes.c_void_p(t.data_ptr()) for t in (refs, table, lens, counts, short)]
        return L.load().csa_cache_reserve(*at, 1, 4, 8, 2, stream)

    stream, graph = ctypes.c_void_p(), ctypes.c_void_p()
    assert cudart.cudaStreamCreate(ctypes.byref(stream)) == 0
    assert cudart.cudaStreamBeginCapture(stream, 0) == 0
    refused = reserve(None)
    cudart.cudaStreamEndCapture(stream, ctypes.byref(graph))  # the refused launch has ended the capture
    cudart.cudaGetLastError()
    assert cudart.cudaStreamDestroy(stream) == 0
    assert refused == L.CSA_ERR_CUDA
    assert reserve(None) == L.CSA_OK
    torch.cuda.synchronize()
    assert short.item() == 0 and lens.item() == 3 and csa.device_status() == 0
