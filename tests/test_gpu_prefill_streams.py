"""GPU tests of MlaPrefill called on another stream than torch's current one,
while that one is held up by a kernel that takes its time."""
import pytest
import torch

import paged_mla_speculative_tree_gb300 as pkg
from paged_mla_speculative_tree_gb300 import binding
from tests.test_gpu_layer_ops import i32, i64, prefill_batch

pytestmark = pytest.mark.gpu

HOLD = 200_000_000  # cycles: about a tenth of a second


@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("keys", [70, 4000])  # whole and split
@pytest.mark.parametrize("given", ["neither", "out", "lse"])
def test_new_outputs_are_zeroed_on_the_stream_of_the_call(given, keys, handle):
    b = prefill_batch(3, [(40, keys)], 2, torch.bfloat16)
    args = (b["q"], b["k_nope"], b["k_rope"], b["v"], i64(b["qo"]), i32(b["kv"]), 0.07)
    p = pkg.MlaPrefill(1, 40, 43, keys, 2)
    want = [t.clone() for t in p(*args)]
    other = torch.cuda.Stream()
    new = {"out": torch.zeros_like(want[0])} if given == "out" else {"lse": torch.zeros_like(want[1])} if given == "lse" else {}
    torch.cuda.synchronize()
    torch.cuda._sleep(HOLD)
    got = p(*args, stream=other.cuda_stream if handle else other, **new)
    other.synchronize()
    with torch.cuda.stream(other):
        early = [t.clone() for t in got]
    torch.cuda.synchronize()
    for w, g, e in zip(want, got, early):
        assert torch.equal(g, w) and torch.equal(e, w)


def test_default_stream_by_its_handles():
    b = prefill_batch(5, [(40, 70)], 2, torch.bfloat16)
    args = (b["q"], b["k_nope"], b["k_rope"], b["v"], i64(b["qo"]), i32(b["kv"]), 0.07)
    p = pkg.MlaPrefill(1, 40, 43, 70, 2)
    want = p(*args)
    for handle in (0, 1):
        got = p(*args, stream=handle)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def bad_batch():
    b = prefill_batch(7, [(40, 70)], 2, torch.bfloat16)
    return b["q"], b["k_nope"], b["k_rope"], b["v"], i64([0, 40]), i32([0, 999]), 0.07


def test_error_word_is_zeroed_before_a_call_on_any_stream():
    args, other = bad_batch(), torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(HOLD)
    p = pkg.MlaPrefill(1, 40, 43, 70, 2)
    p(*args, stream=other)
    torch.cuda.synchronize()
    assert p.device_error() == binding.DEVERR_INDPTR


def test_error_word_is_read_after_calls_on_all_streams():
    args, other = bad_batch(), torch.cuda.Stream()
    p = pkg.MlaPrefill(1, 40, 43, 70, 2)
    torch.cuda.synchronize()
    with torch.cuda.stream(other):
        torch.cuda._sleep(HOLD)
    p(*args, stream=other)
    assert p.device_error() == binding.DEVERR_INDPTR


def test_object_made_and_called_in_a_capture():
    b = prefill_batch(9, [(40, 4000)], 2, torch.bfloat16)
    args = (b["q"], b["k_nope"], b["k_rope"], b["v"], i64(b["qo"]), i32(b["kv"]), 0.07)
    want = pkg.MlaPrefill(1, 40, 43, 4000, 2)(*args)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p = pkg.MlaPrefill(1, 40, 43, 4000, 2)
        got = p(*args)
    for _ in range(2):
        graph.replay()
    assert p.device_error() == 0
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
