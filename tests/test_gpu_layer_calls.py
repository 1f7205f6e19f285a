"""GPU tests of the layer's calls around launches that the host refuses."""
import ctypes

import pytest
import torch

import paged_mla_speculative_tree_gb300 as pkg
from tests.test_gpu_layer_ops import DEV, i32, i64, prefill_batch, rnd

pytestmark = pytest.mark.gpu

E_CUDA = -7  # MTV_E_CUDA


def product(n=64):
    """Outputs of whole 16 bytes, or (n = 63) not: the tensor-core kernel and the plain one."""
    x, w = rnd(1, (70, 2, 64), torch.bfloat16), rnd(2, (2, 64, n), torch.bfloat16)
    out = torch.empty((70, 2, n), dtype=torch.bfloat16, device=DEV)
    return lambda **kw: pkg.head_product(x, w, out, **kw), out


def attention():
    b = prefill_batch(3, [(40, 70)], 2, torch.bfloat16)
    out = torch.empty((43, 2, 128), dtype=torch.bfloat16, device=DEV)
    args = (b["q"], b["k_nope"], b["k_rope"], b["v"], i64(b["qo"]), i32(b["kv"]))
    return lambda **kw: pkg.prefill_run(*args, 40, 70, 0.07, out, **kw), out


def norms():
    q, out = rnd(4, (9, 4, 192), torch.bfloat16), torch.empty((9, 4, 64), dtype=torch.bfloat16, device=DEV)
    turns, positions = pkg.rope_freqs(64, 10000.0)[0].to(DEV), i64(list(range(9)))
    return lambda **kw: pkg.norm_rope_write(turns, positions, 1e-6, q_in=q, q_rope=out, **kw), out


@pytest.mark.parametrize("kind", [product, attention, norms])
def test_a_refused_launch_is_not_reported_by_the_next_call(kind):
    """A capture that something not allowed in it has ended takes no launches; the next call, elsewhere, is as ever."""
    runtime = ctypes.CDLL("libcudart.so.13")
    side = torch.cuda.Stream()
    handle, graph = ctypes.c_void_p(side.cuda_stream), ctypes.c_void_p()
    call, _ = kind()
    plain, out = product(63)
    assert call() == 0 and plain() == 0
    torch.cuda.synchronize()
    want = out.clone()
    out.zero_()
    torch.cuda.synchronize()
    assert runtime.cudaStreamBeginCapture(handle, 2) == 0  # relaxed
    try:
        assert runtime.cudaStreamSynchronize(handle) != 0
        rc = call(stream=side, check=False)
    finally:
        runtime.cudaStreamEndCapture(handle, ctypes.byref(graph))
        runtime.cudaGetLastError()
    assert rc == E_CUDA
    assert plain() == 0
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    assert call() == 0
    torch.cuda.synchronize()
