"""GPU tests of what the softmax weights of prompt attention lose to their
16-bit type, against oracle/layer_ops.py: the small ones of fp16 count, and the
output is divided by the sum of the weights as the product takes them, so that
their rounding cancels in what the values have in common.

With rounded weights p(1 + d) the output is off by sum p d (v - out), d at most
half a step u of the type: u times the oracle's spread, where a division by the
unrounded sum would leave u times the values' magnitudes."""
import math

import pytest
import torch

import paged_mla_speculative_tree_gb300 as pkg
from oracle import layer_ops as L
from tests.test_gpu_layer_ops import DEV, HALF, LAST, TYPES, half_step, i32, i64, prefill_batch, rnd

pytestmark = pytest.mark.gpu


def run(b, scale, nsplit=1):
    rows, heads, dtype = b["q"].shape[0], b["q"].shape[1], b["q"].dtype
    n, last = nsplit % LAST, nsplit // LAST
    size = n * (last * 256 if last else rows * heads) * 129 * 4 if n > 1 else 0
    out, lse = torch.empty((rows, heads, 128), dtype=dtype, device=DEV), torch.empty((rows, heads), device=DEV)
    err = i32([0])
    pkg.prefill_run(b["q"], b["k_nope"], b["k_rope"], b["v"], i64(b["qo"]), i32(b["kv"]), b["max_q"], b["max_kv"], scale, out, lse,
                    nsplit=nsplit, workspace=torch.empty(size, dtype=torch.uint8, device=DEV) if size else None, err=err)
    assert int(err) == 0
    return out, lse


def check(b, scale, nsplit, vmax):
    out, lse = run(b, scale, nsplit)
    ref = L.prefill(b["q"], b["k_nope"], b["k_rope"], b["v"], b["qo"], b["kv"], scale)
    keys, dtype = b["max_kv"], b["q"].dtype
    u, tiny = half_step(dtype)
    # scores: sums of 192 products, scaled and referred to the maximum; the exponential's own error
    score = 208 * 2.0 ** -23 * ref["smag"] + 2.0 ** -21
    sums = (keys + 8) * 2.0 ** -23
    bound = u * ref["out"].abs() + 1.05 * (u + score)[..., None] * ref["spread"] + 2 * sums * ref["mag"] + tiny
    if dtype == torch.float16:  # the largest weight is held as 2^7 at least, the smallest step is 2^-24
        bound += keys * 2.0 ** -32 * vmax
    real = ~ref["lse"].isnan().all(dim=1)
    over = ((out.double().cpu() - ref["out"]).abs() - bound)[real].max().item()
    assert over <= 0, f"beyond the bound by {over:.3e}"
    lse_bound = score + sums + 2.0 ** -22 * ref["lse"].abs()
    assert ((lse.double().cpu() - ref["lse"]).abs() <= lse_bound)[real].all()


def one_key_above_all(keys, at, dtype, seed):
    """Scores of 0 at one key and of -17.5 to -17 at all others, by the shared part; its value is 0, theirs are about 1."""
    b = prefill_batch(seed, [(2, keys)], 1, dtype, pad=0)
    b["q"].zero_()
    b["q"][:, :, 128] = 1
    b["k_rope"].zero_()
    b["k_rope"][:, 0] = (-17.5 + 0.5 * torch.rand(keys, generator=torch.Generator().manual_seed(seed))).to(dtype).to(DEV)
    b["k_rope"][at, 0] = 0
    b["v"].copy_((1 + rnd(seed, b["v"].shape, torch.float32, 0.25)).clamp(0, 2).to(dtype))
    b["v"][at] = 0
    return b


@pytest.mark.parametrize("nsplit", [1, 19, 3 + LAST])
@pytest.mark.parametrize("at", [0, 20_000])
@pytest.mark.parametrize("keys", [32_768, 131_072])
def test_small_fp16_weights_of_many_keys_count(keys, at, nsplit):
    check(one_key_above_all(keys, at, torch.float16, 3), 1.0, nsplit, 2.0)


def test_small_bf16_weights_of_many_keys_count():
    check(one_key_above_all(131_072, 0, torch.bfloat16, 5), 1.0, 1, 2.0)


@pytest.mark.parametrize("spread,scale", [(30.0, 192 ** -0.5), (1.5, 2.0), (1e-3, 192 ** -0.5)])
def test_fp16_weights_of_sharp_and_flat_scores(spread, scale):
    b = prefill_batch(7, [(140, 400)], 2, torch.float16, spread=spread)
    check(b, scale, 1, b["v"][:400].abs().max().item() * 2)


def test_fp16_weights_of_rising_scores():
    """The maximum grows within what a row's reference allows, and past it."""
    for top in (4.0, 40.0):
        b = prefill_batch(9, [(130, 700)], 1, torch.float16)
        b["q"][:, 0, 128] = 8.0
        b["k_rope"][:, 0] = torch.linspace(-top, top, 703, device=DEV).to(torch.float16)
        check(b, 192 ** -0.5, 1, b["v"][:700].abs().max().item() * 2)
        check(b, 192 ** -0.5, 4, b["v"][:700].abs().max().item() * 2)


@pytest.mark.parametrize("nsplit", [1, 3, 2 + LAST])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype", HALF)
def test_values_that_all_keys_share_come_out_as_they_are(dtype, causal, nsplit):
    """All values are the largest below 2 and every weight but one is a half and nearly half a step: what the weights'
    rounding takes away, half a step of theirs, is more than half a step of the output."""
    t = TYPES[dtype]
    u = half_step(t)[0]
    b = prefill_batch(11, [(1, 300)], 2, t, pad=0)
    b["q"].zero_(), b["k_nope"].zero_(), b["k_rope"].zero_()
    b["q"][:, :, 128], b["k_rope"][1:, 0] = 1, -1
    b["v"].fill_(2 - 2 * u)
    scale = -math.log(0.5 * (1 + 0.98 * u))
    out, lse = run(b, scale, nsplit)
    # sums of 300 values agree to 308 steps of 2^-23, a tenth of half a step of fp16
    assert (out == 2 - 2 * u).all()
    want = math.log(1 + 299 * 0.5 * (1 + 0.98 * u))
    assert (lse - want).abs().max() < 2.0 ** -20 + 308 * 2.0 ** -23


@pytest.mark.parametrize("nsplit", [1, 4, 3 + LAST * 2])
@pytest.mark.parametrize("requests", [[(140, 400)], [(257, 515)], [(3, 3), (129, 200), (1, 64), (5, 127)]])
@pytest.mark.parametrize("dtype", HALF)
def test_values_with_a_common_part(dtype, requests, nsplit):
    b = prefill_batch(13, requests, 2, TYPES[dtype])
    b["v"].copy_((3 + b["v"].float() * 0.05).to(TYPES[dtype]))
    check(b, 192 ** -0.5, nsplit, 4.0)
