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


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("tokens,heads", [(0, 4), (0, 0), (5, 0)])
def test_norms_of_no_tokens_or_no_heads(tokens, heads, dtype):
    """Norms of both kinds given: nothing to do, or the latent rows alone."""
    turns = pkg.rope_freqs(64, 10000.0)[0].to(DEV)
    q, down = rnd(1, (tokens, heads, 192), dtype), rnd(2, (tokens, 576), dtype)
    qw, cw = rnd(3, (192,), dtype), rnd(4, (512,), dtype)
    q_nope, q_rope = torch.empty((tokens, heads, 128), dtype=dtype, device=DEV), torch.empty((tokens, heads, 64), dtype=dtype, device=DEV)
    pools = [torch.full((8, 576), 9.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    kw = dict(c_in=down[:, :512], c_weight=cw, k_in=down[:, 512:], out_cache_loc=torch.arange(tokens, device=DEV))
    positions = torch.arange(tokens, device=DEV)
    assert pkg.norm_rope_write(turns, positions, 1e-6, q_in=q, q_weight=qw, q_nope=q_nope, q_rope=q_rope, kv_pool=pools[0], **kw) == 0
    assert pkg.norm_rope_write(turns, positions, 1e-6, kv_pool=pools[1], **kw) == 0
    assert pkg.norm_rope_write(turns, positions, 1e-6, q_in=q, q_weight=qw, q_nope=q_nope, q_rope=q_rope) == 0
    assert torch.equal(pools[0], pools[1]) and (pools[0][tokens:] == 9).all()
    assert tokens == 0 or not (pools[0][:tokens] == 9).any(dim=1).all()
