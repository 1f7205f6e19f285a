"""GPU tests of waits that give up inside the products and prompt attention, by
the test-only count in their dtype: at once, and after more and more of a
block's work.  The call ends, reports it, keeps to its outputs, waits for nothing
that cannot come, and the next call is right."""
import time

import pytest
import torch

import paged_mla_speculative_tree_gb300 as pkg
from paged_mla_speculative_tree_gb300 import binding
from tests.test_gpu_layer_ops import DEV, LAST, i32, i64, prefill_batch, rnd

pytestmark = pytest.mark.gpu

GIVE_UP = 0x100  # MTV_TEST_GIVE_UP
COUNTS = [1, 2, 3, 4, 6, 9, 13, 19, 28, 42, 63, 95, 142, 213, 255]
CODES = {torch.bfloat16: 0, torch.float16: 1}


def run_all(call, outs, want, err):
    """call(n) with every count; outs have to be as they are or, where nothing gave up, as wanted."""
    assert call(0) == 0  # what is loaded with the first call is not timed
    seen = 0
    for n in COUNTS + [1, 1]:
        for o in outs:
            o.fill_(7)
        torch.cuda.synchronize()
        start = time.monotonic()
        assert call(n) == 0
        torch.cuda.synchronize()
        took = time.monotonic() - start
        bits = int(err)
        # a drain that waits in vain takes a second
        assert took < 0.5, f"count {n}: {took:.2f} s, error word {bits}"
        assert bits in (0, binding.DEVERR_TIMEOUT)
        seen += bits != 0
        if not bits:
            assert all(torch.equal(o, w) for o, w in zip(outs, want)), f"count {n}"
        err.zero_()
    assert seen > 0
    for o in outs:
        o.fill_(7)
    assert call(0) == 0
    torch.cuda.synchronize()
    assert int(err) == 0 and all(torch.equal(o, w) for o, w in zip(outs, want))


@pytest.mark.parametrize("dense", ["n", "k"])
@pytest.mark.parametrize("tokens,heads,k,n", [(8, 64, 128, 512), (64, 64, 512, 128), (100, 200, 1024, 64), (1000, 16, 512, 160),
                                              (1024, 100, 512, 256), (2050, 70, 320, 256)])
def test_products_that_give_up(tokens, heads, k, n, dense):
    """One tile of tokens, several of them, and pairs of SMs (the last two)."""
    x = rnd(1, (tokens, heads, k), torch.bfloat16)
    w = rnd(2, (heads, k, n), torch.bfloat16) if dense == "n" else rnd(2, (heads, n, k), torch.bfloat16).transpose(1, 2)
    want = torch.empty((tokens, heads, n), dtype=torch.bfloat16, device=DEV)
    pkg.head_product(x, w, want)
    buf, err = torch.empty((tokens + 2, heads, n + 8), dtype=torch.bfloat16, device=DEV), i32([0])
    out = buf[:tokens, :, :n]

    def call(count):
        buf[tokens:], buf[:, :, n:] = 9, 9
        rc = binding.load().mla_head_product(x.data_ptr(), x.stride(0), x.stride(1), w.data_ptr(), *w.stride(), out.data_ptr(),
                                             out.stride(0), out.stride(1), tokens, heads, k, n, GIVE_UP * count, err.data_ptr(),
                                             torch.cuda.current_stream().cuda_stream)
        assert (buf[tokens:] == 9).all() and (buf[:, :, n:] == 9).all()
        return rc

    run_all(call, [out], [want], err)


@pytest.mark.parametrize("dtype", CODES)
@pytest.mark.parametrize("nsplit", [1, 3, 2 + LAST * 3])
@pytest.mark.parametrize("requests,heads", [([(300, 700)], 2), ([(60, 5000), (513, 513)], 3), ([(250, 130), (3, 3)], 80)])
def test_prompt_attention_that_gives_up(requests, heads, nsplit, dtype):
    b = prefill_batch(5, requests, heads, dtype, pad=0)
    rows = b["q"].shape[0]
    n, last = nsplit % LAST, nsplit // LAST
    size = n * max(last * 256, rows * heads) * 129 * 4
    ws = torch.empty(size, dtype=torch.uint8, device=DEV)
    qo, kv, err = i64(b["qo"]), i32(b["kv"]), i32([0])
    out, lse = torch.empty((rows, heads, 128), dtype=dtype, device=DEV), torch.empty((rows, heads), device=DEV)
    q, kn, kr, v = b["q"], b["k_nope"], b["k_rope"], b["v"]

    def call(count):
        ws.zero_()
        return binding.load().mla_prefill_run(
            q.data_ptr(), q.stride(0), q.stride(1), kn.data_ptr(), kn.stride(0), kn.stride(1), kr.data_ptr(), kr.stride(0),
            v.data_ptr(), v.stride(0), v.stride(1), qo.data_ptr(), kv.data_ptr(), len(requests), b["max_q"], b["max_kv"], rows,
            kn.shape[0], heads, CODES[dtype] + GIVE_UP * count, 0.07, 1, out.data_ptr(), out.stride(0), out.stride(1),
            lse.data_ptr(), nsplit, ws.data_ptr(), size, err.data_ptr(), torch.cuda.current_stream().cuda_stream)

    assert call(0) == 0
    want = [out.clone(), lse.clone()]
    run_all(call, [out, lse], want, err)


@pytest.mark.parametrize("nsplit", [1, 3, 9, 2 + LAST * 3])
def test_rows_of_prompt_attention_that_gave_up_are_left_or_nan(nsplit):
    """Each row is as it should be, as it was, or (with split keys) NaN: never made of what the workspace held."""
    b = prefill_batch(9, [(60, 3000), (300, 1700)], 2, torch.bfloat16, pad=0)
    heads, rows = 2, 360
    n, last = nsplit % LAST, nsplit // LAST
    ws = torch.empty(n * max(last * 256, rows * heads) * 129, dtype=torch.float32, device=DEV)
    qo, kv, err = i64(b["qo"]), i32(b["kv"]), i32([0])
    out, lse = torch.empty((rows, heads, 128), dtype=torch.bfloat16, device=DEV), torch.empty((rows, heads), device=DEV)
    q, kn, kr, v = b["q"], b["k_nope"], b["k_rope"], b["v"]

    def call(count):
        ws.fill_(3)
        out.fill_(7), lse.fill_(7)
        assert binding.load().mla_prefill_run(
            q.data_ptr(), q.stride(0), q.stride(1), kn.data_ptr(), kn.stride(0), kn.stride(1), kr.data_ptr(), kr.stride(0),
            v.data_ptr(), v.stride(0), v.stride(1), qo.data_ptr(), kv.data_ptr(), 2, 300, 3000, rows, kn.shape[0], heads,
            GIVE_UP * count, 0.07, 1, out.data_ptr(), out.stride(0), out.stride(1), lse.data_ptr(), nsplit, ws.data_ptr(),
            ws.numel() * 4, err.data_ptr(), torch.cuda.current_stream().cuda_stream) == 0
        torch.cuda.synchronize()

    call(0)
    want = out.clone(), lse.clone()
    missing = 0
    for count in COUNTS:
        call(count)
        good = (out == want[0]).all(dim=2) & (lse == want[1])
        left = (out == 7).all(dim=2) & (lse == 7)
        nan = out.isnan().all(dim=2) & lse.isnan()
        assert (good | left | nan).all(), f"count {count}"
        assert n > 1 or not nan.any()
        assert last or n == 1 or not left.any()
        missing += int((~good).sum())
    assert missing > 0 and int(err) == binding.DEVERR_TIMEOUT
