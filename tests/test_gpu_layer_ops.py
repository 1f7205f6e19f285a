"""GPU tests of the attention layer's operators against oracle/layer_ops.py,
through the public entry points, within bounds counted from the roundings of
the computation: a stored value is off by half a step of its type, an fp32 sum
of n terms by n steps of 2^-23 of their magnitudes (the tensor cores' adders may
truncate), a softmax weight by its score's error and its own rounding."""
import math

import pytest
import torch

import paged_mla_speculative_tree_gb300 as pkg
from oracle import layer_ops as L
from oracle import step_ops as S
from paged_mla_speculative_tree_gb300 import binding

pytestmark = pytest.mark.gpu

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
HALF = ["bf16", "fp16"]


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def i64(v):
    return torch.tensor(v, dtype=torch.int64, device=DEV)


def rnd(seed, shape, dtype, scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(dtype)


def half_step(dtype):
    """(relative half step, half of the smallest subnormal) of a type."""
    return torch.finfo(dtype).eps / 2, torch.finfo(dtype).tiny * torch.finfo(dtype).eps / 2


def within(got, ref, bound, tag=""):
    got = got.double().cpu()
    assert torch.isfinite(got).all(), f"{tag}: not finite"
    over = ((got - ref).abs() - bound).max().item() if got.numel() else 0.0
    assert over <= 0, f"{tag}: beyond the bound by {over:.3e}"


# ------------------------------------------------------------- head product

def product_bound(ref, mag, k, dtype):
    u, tiny = half_step(dtype)
    s = (k + 8) * 2.0 ** -23 * mag
    return u * (ref.abs() + s) + s + tiny


def check_product(x, w, pad_tok=2, pad_dim=3, out=None):
    """Runs into a view of a buffer that has to stay as it was around it."""
    tokens, heads, k = x.shape
    n = w.shape[2]
    buf = torch.full((tokens + pad_tok, heads, n + pad_dim), 7.0, dtype=x.dtype, device=DEV)
    out = buf[:tokens, :, :n]
    pkg.head_product(x, w, out)
    torch.cuda.synchronize()
    ref, mag = L.head_product(x, w)
    within(out, ref, product_bound(ref, mag, k, x.dtype), f"{tuple(x.shape)} x {n}")
    assert (buf[tokens:] == 7).all() and (buf[:, :, n:] == 7).all()


@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("tokens,heads,k,n", [(1, 1, 8, 8), (1, 64, 128, 512), (8, 3, 128, 512), (16, 2, 512, 128),
                                              (17, 5, 64, 96), (127, 2, 200, 512), (129, 3, 512, 256), (300, 2, 96, 72),
                                              (257, 1, 1024, 64), (640, 7, 24, 1024), (33, 2, 520, 40), (1000, 4, 512, 160)])
@pytest.mark.parametrize("dense", ["n", "k"])
def test_head_product(tokens, heads, k, n, dtype, dense):
    t = TYPES[dtype]
    x = rnd(tokens + k, (tokens, heads, k + 64), t)[:, :, :k]
    w = rnd(n + k, (heads, k, n), t) if dense == "n" else rnd(n + k, (heads, n, k), t).transpose(1, 2)
    check_product(x, w, pad_dim=8)


@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("tokens,heads,k,n", [(1, 1, 1, 1), (5, 3, 7, 5), (70, 2, 33, 65), (130, 3, 1023, 1), (65, 2, 1, 1000)])
def test_head_product_of_odd_sizes_and_strides(tokens, heads, k, n, dtype):
    t = TYPES[dtype]
    x = rnd(k, (tokens, heads, k + 1), t)[:, :, 1:]
    w = rnd(n, (heads, k, 2 * n), t)[:, :, ::2]
    check_product(x, w)
    check_product(x.transpose(0, 1).contiguous().transpose(0, 1), w.contiguous())


@pytest.mark.parametrize("tokens,heads,n", [(1, 8, 256), (200, 3, 256), (1030, 5, 128)])
def test_head_product_of_rows_shared_by_the_heads(tokens, heads, n):
    rows = rnd(tokens, (tokens, 576), torch.bfloat16)
    x = rows[:, None, :512].expand(tokens, heads, 512)
    check_product(x, rnd(n, (heads, n, 512), torch.bfloat16, 0.05).transpose(1, 2), pad_dim=0)


@pytest.mark.parametrize("tokens,k,n", [(1, 128, 512), (130, 128, 512), (130, 512, 128), (60, 40, 24)])
def test_head_product_reads_nothing_beyond_its_operands(tokens, k, n):
    """NaN around x (columns, rows behind) and w (heads before and behind)."""
    x = torch.full((tokens + 140, 4, k + 8), math.nan, dtype=torch.bfloat16, device=DEV)
    x[:tokens, 1:3, :k] = rnd(1, (tokens, 2, k), torch.bfloat16)
    w = torch.full((4, k + 8, n + 8), math.nan, dtype=torch.bfloat16, device=DEV)
    w[1:3, :k, :n] = rnd(2, (2, k, n), torch.bfloat16)
    check_product(x[:tokens, 1:3, :k], w[1:3, :k, :n], pad_dim=8)
    v = torch.full((4, n + 8, k + 8), math.nan, dtype=torch.bfloat16, device=DEV)
    v[1:3, :n, :k] = w[1:3, :k, :n].transpose(1, 2)
    check_product(x[:tokens, 1:3, :k], v[1:3, :n, :k].transpose(1, 2), pad_dim=8)


@pytest.mark.parametrize("tokens,heads,k,n", [(3, 2, 7, 5), (129, 1, 65, 129), (40, 3, 1, 70), (200, 2, 130, 1), (257, 5, 513, 63),
                                              (3, 2, 7, 8), (129, 1, 65, 136), (40, 3, 1, 72), (257, 5, 513, 64)])
@pytest.mark.parametrize("dense", ["n", "k"])
def test_head_product_of_odd_sizes_in_aligned_rows(tokens, heads, k, n, dense):
    """Rows of whole 16 bytes that the operands and outputs only partly fill; NaN behind the operands."""
    up = lambda v: (v + 7) // 8 * 8 + 8  # noqa: E731
    x = torch.full((tokens, heads, up(k)), math.nan, dtype=torch.float16, device=DEV)
    x[:, :, :k] = rnd(k, (tokens, heads, k), torch.float16)
    w = torch.full((heads, k + 1, up(n)) if dense == "n" else (heads, n + 1, up(k)), math.nan, dtype=torch.float16, device=DEV)
    inner = rnd(n, (heads, k, n), torch.float16)
    w[:, :(k if dense == "n" else n), :(n if dense == "n" else k)] = inner if dense == "n" else inner.transpose(1, 2)
    view = w[:, :k, :n] if dense == "n" else w[:, :n, :k].transpose(1, 2)
    check_product(x[:, :, :k], view, pad_dim=up(n) - n)


def test_head_product_of_shared_weights_and_head_major_rows():
    """One weight for every head by its stride; operands and outputs with heads outside tokens."""
    x = rnd(1, (6, 150, 96), torch.bfloat16).transpose(0, 1)
    w = rnd(2, (1, 96, 200), torch.bfloat16).expand(6, 96, 200)
    out = torch.empty((6, 150, 200), dtype=torch.bfloat16, device=DEV).transpose(0, 1)
    pkg.head_product(x, w, out)
    ref, mag = L.head_product(x, w)
    within(out, ref, product_bound(ref, mag, 96, torch.bfloat16))


def test_calls_on_two_streams_at_once():
    """Products and split attention on two streams with buffers of their own, again and again."""
    jobs = []
    for i in range(2):
        b = prefill_batch(50 + i, [(40, 4000 + i)], 2, torch.bfloat16)
        p = pkg.MlaPrefill(1, 40, 43, 4001, 2)
        x, w = rnd(60 + i, (300, 8, 128), torch.bfloat16), rnd(70 + i, (8, 128, 512), torch.bfloat16)
        args = (b["q"], b["k_nope"], b["k_rope"], b["v"], i64(b["qo"]), i32(b["kv"]), 0.07)
        want = torch.empty((300, 8, 512), dtype=torch.bfloat16, device=DEV)
        pkg.head_product(x, w, want)
        jobs.append((p, args, [t.clone() for t in p(*args)], x, w, want, torch.cuda.Stream(), []))
    torch.cuda.synchronize()
    for _ in range(10):
        for p, args, _, x, w, want, stream, got in jobs:
            with torch.cuda.stream(stream):
                out = torch.empty_like(want)
                pkg.head_product(x, w, out)
                got.append((p(*args), out))
    torch.cuda.synchronize()
    for p, _, attention, _, _, want, _, got in jobs:
        assert p.nsplit > 1 and p.device_error() == 0
        for (out, lse), product in got:
            assert torch.equal(out, attention[0]) and torch.equal(lse, attention[1]) and torch.equal(product, want)


def test_head_product_keeps_rows_apart():
    """A row of NaN or infinity spoils its own outputs only."""
    x, w = rnd(5, (200, 2, 128), torch.bfloat16), rnd(6, (2, 128, 512), torch.bfloat16)
    out, again = torch.empty((200, 2, 512), dtype=torch.bfloat16, device=DEV), torch.empty((200, 2, 512), dtype=torch.bfloat16, device=DEV)
    pkg.head_product(x, w, out)
    y = x.clone()
    y[3], y[130, 1, 5] = math.nan, math.inf
    pkg.head_product(y, w, again)
    same = torch.ones((200, 2), dtype=torch.bool, device=DEV)
    same[3], same[130, 1] = False, False
    assert torch.equal(out[same], again[same])
    assert not torch.isfinite(again[~same].float()).any()


def test_head_product_writes_absorbed_queries_between_rotated_parts():
    """Into [tokens, heads, 576] rows whose last 64 are another call's."""
    x, w = rnd(7, (50, 64, 192), torch.bfloat16), rnd(8, (64, 256, 512), torch.bfloat16, 0.05)
    q = rnd(9, (50, 64, 576), torch.bfloat16)
    rope = q[:, :, 512:].clone()
    pkg.head_product(x[:, :, :128], w[:, :128], q[:, :, :512])
    ref, mag = L.head_product(x[:, :, :128], w[:, :128])
    within(q[:, :, :512], ref, product_bound(ref, mag, 128, torch.bfloat16))
    assert torch.equal(q[:, :, 512:], rope)


def test_head_product_without_tokens_or_heads():
    e = lambda *s: torch.empty(s, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    assert pkg.head_product(e(0, 4, 128), e(4, 128, 512), e(0, 4, 512)) == 0
    assert pkg.head_product(e(5, 0, 128), e(0, 128, 512), e(5, 0, 512)) == 0


# ------------------------------------------------------------------ prefill

def prefill_batch(seed, requests, heads, dtype, pad=3, spread=1.5):
    """requests: (queries, keys) each; rows and keys of no request are NaN."""
    new, length = [n for n, _ in requests], [k for _, k in requests]
    tq, tk = sum(new) + pad, sum(length) + pad
    q, kv = rnd(seed, (tq, heads, 192), dtype, spread), rnd(seed + 1, (tk, heads, 256), dtype)
    latent = rnd(seed + 2, (tk, 576), dtype)
    q[sum(new):], kv[sum(length):], latent[sum(length):] = math.nan, math.nan, math.nan
    ends = lambda v: [0] + torch.tensor(v, dtype=torch.int64).cumsum(0).tolist()  # noqa: E731
    return dict(q=q, k_nope=kv[:, :, :128], k_rope=latent[:, 512:], v=kv[:, :, 128:], qo=ends(new), kv=ends(length),
                max_q=max(new + [0]), max_kv=max(length + [0]))


def prefill_bounds(ref, keys, dtype):
    u, tiny = half_step(dtype)
    # scores: sums of 192 products, scaled and referred to the maximum; the exponential's own error
    score = 208 * 2.0 ** -23 * ref["smag"] + 2.0 ** -21
    weight = (u + score)[..., None] * 1.05
    # fp16 weights below 2^-24 of the reference become multiples of 2^-24
    out = u * ref["out"].abs() + weight * ref["mag"] + (keys + 8) * 2.0 ** -23 * ref["mag"] + keys * 2.0 ** -25 * 8 + tiny
    return out, score + (keys + 8) * 2.0 ** -24 + 2.0 ** -22 * ref["lse"].abs()


def check_prefill(b, dtype, scale=192 ** -0.5, causal=True, nsplit=1, lse=True):
    rows, heads = b["q"].shape[:2]
    out = torch.full((rows, heads, 128), 5.0, dtype=dtype, device=DEV)
    ls = torch.full((rows, heads), 5.0, device=DEV) if lse else None
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    ws = torch.full((nsplit * rows * heads * 129 * 4,), 255, dtype=torch.uint8, device=DEV) if nsplit > 1 else None
    pkg.prefill_run(b["q"], b["k_nope"], b["k_rope"], b["v"], i64(b["qo"]), i32(b["kv"]), b["max_q"], b["max_kv"], scale, out,
                    ls, causal=causal, nsplit=nsplit, workspace=ws, err=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    ref = L.prefill(b["q"], b["k_nope"], b["k_rope"], b["v"], b["qo"], b["kv"], scale, causal)
    real = ~ref["lse"].isnan().all(dim=1)
    assert (out.cpu()[~real] == 5).all()
    some = ref["lse"][real] > -math.inf
    bound, lse_bound = prefill_bounds({k: v[real] for k, v in ref.items()}, b["max_kv"], dtype)
    within(out.cpu()[real], ref["out"][real], bound, "out")
    assert (out.cpu()[real][~some] == 0).all()
    if lse:
        got = ls.cpu()
        assert (got[~real] == 5).all() and torch.equal(got[real] == -math.inf, ~some)
        within(got[real][some], ref["lse"][real][some], lse_bound[some], "lse")
    return out, ls


CASES = {
    "one": [(1, 1)],
    "one of many": [(1, 300)],
    "prompt": [(130, 130)],
    "tile": [(128, 128)],
    "two tiles": [(256, 256)],
    "behind a prefix": [(70, 333)],
    "odd": [(257, 515)],
    "ragged": [(3, 3), (0, 7), (129, 200), (1, 64), (64, 65), (0, 0), (5, 127)],
    "fewer keys": [(9, 4), (140, 130), (6, 0), (2, 2)],
    "short": [(2, 2)] * 9,
    "first rows without keys": [(300, 150), (600, 100), (257, 1)],
    "many blocks": [(700, 1000), (513, 513)],
}


@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("nsplit", [1, 3])
@pytest.mark.parametrize("name", CASES)
def test_prefill(name, nsplit, dtype):
    check_prefill(prefill_batch(len(name), CASES[name], 2, TYPES[dtype]), TYPES[dtype], nsplit=nsplit)


@pytest.mark.parametrize("nsplit", [1, 2, 64])
@pytest.mark.parametrize("name", ["odd", "ragged", "fewer keys"])
def test_prefill_of_all_keys(name, nsplit):
    check_prefill(prefill_batch(3, CASES[name], 3, torch.bfloat16), torch.bfloat16, causal=False, nsplit=nsplit)


@pytest.mark.parametrize("heads", [1, 5, 64])
def test_prefill_heads(heads):
    check_prefill(prefill_batch(11, [(33, 70), (90, 90)], heads, torch.bfloat16), torch.bfloat16)


@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("spread,scale", [(30.0, 192 ** -0.5), (1.5, 2.0), (1e-3, 192 ** -0.5), (1.5, 1e-6)])
def test_prefill_of_sharp_and_flat_scores(spread, scale, dtype):
    check_prefill(prefill_batch(13, [(140, 400)], 2, TYPES[dtype], spread=spread), TYPES[dtype], scale=scale)


def test_prefill_of_rising_and_falling_scores():
    """The running maximum moves at every step, or never after the first."""
    for sign in (1, -1):
        b = prefill_batch(17, [(130, 700)], 1, torch.bfloat16)
        ramp = torch.linspace(-40, 40, 703, device=DEV) * sign
        b["q"][:, 0, 128] = 8.0
        b["k_rope"][:, 0] = ramp.to(torch.bfloat16)
        b["k_rope"][700:] = math.nan
        check_prefill(b, torch.bfloat16)
        check_prefill(b, torch.bfloat16, nsplit=4)


def test_prefill_strides_and_no_lse():
    """Head-major queries, separate key and value buffers, outputs inside wider rows."""
    b = prefill_batch(19, [(40, 77), (100, 100)], 3, torch.bfloat16)
    b["q"] = b["q"].transpose(0, 1).contiguous().transpose(0, 1)
    b["v"] = b["v"].clone()
    b["k_rope"] = b["k_rope"].contiguous()
    want, _ = check_prefill(b, torch.bfloat16, lse=False)
    buf = torch.full((143, 3, 200), 5.0, dtype=torch.bfloat16, device=DEV)
    pkg.prefill_run(b["q"], b["k_nope"], b["k_rope"], b["v"], i64(b["qo"]), i32(b["kv"]), 100, 100, 192 ** -0.5,
                    buf[:, :, 64:192])
    assert torch.equal(buf[:, :, 64:192], want)
    assert (buf[:, :, :64] == 5).all() and (buf[:, :, 192:] == 5).all()


@pytest.mark.parametrize("nsplit", [1, 3])
def test_prefill_keeps_requests_apart(nsplit):
    """NaN and infinity in one request's keys and queries leave the others' rows."""
    requests = [(50, 100), (30, 45), (60, 61)]
    b = prefill_batch(23, requests, 2, torch.bfloat16)
    want, want_lse = check_prefill(b, torch.bfloat16, nsplit=nsplit)
    for what, value in (("v", math.nan), ("v", math.inf), ("k_nope", math.nan), ("k_rope", math.inf)):
        c = {**b, "v": b["v"].clone(), "k_nope": b["k_nope"].clone(), "k_rope": b["k_rope"].clone(), "q": b["q"].clone()}
        c[what][100:145] = value
        c["q"][50:80] = math.nan
        out, lse = torch.zeros_like(want), torch.zeros_like(want_lse)
        ws = torch.zeros(nsplit * 143 * 2 * 129 * 4, dtype=torch.uint8, device=DEV)
        pkg.prefill_run(c["q"], c["k_nope"], c["k_rope"], c["v"], i64(b["qo"]), i32(b["kv"]), 60, 100, 192 ** -0.5, out, lse,
                        nsplit=nsplit, workspace=ws)
        for rows in (slice(0, 50), slice(80, 140)):
            assert torch.equal(out[rows], want[rows]) and torch.equal(lse[rows], want_lse[rows])


def test_prefill_of_keys_and_values_shared_by_the_heads():
    """Head strides of zero: the heads' queries over the same keys and values."""
    b = prefill_batch(27, [(50, 90), (130, 140)], 4, torch.bfloat16)
    b["k_nope"] = b["k_nope"][:, :1].expand(-1, 4, -1)
    b["v"] = b["v"][:, :1].expand(-1, 4, -1)
    check_prefill(b, torch.bfloat16)


def test_prefill_is_the_same_each_time_and_alone_or_in_a_batch():
    b = prefill_batch(29, [(200, 500), (37, 90)], 2, torch.bfloat16)
    first, lse = check_prefill(b, torch.bfloat16)
    again, lse2 = check_prefill(b, torch.bfloat16)
    assert torch.equal(first, again) and torch.equal(lse, lse2)
    alone = {**b, "qo": [200, 237], "kv": [500, 590], "max_q": 37, "max_kv": 90}
    out, _ = check_prefill(alone, torch.bfloat16)
    assert torch.equal(out[200:237], first[200:237])


@pytest.mark.parametrize("nsplit", [1, 2])
@pytest.mark.parametrize("qo,kv", [([0, 20, 10, 40], [0, 20, 30, 60]), ([0, 10, 20, 60], [0, 20, 30, 60]),
                                   ([0, 10, 20, 40], [0, 30, 20, 60]), ([0, 10, 20, 40], [0, 20, 30, 999]),
                                   ([-5, 10, 20, 40], [0, 20, 30, 60]), ([0, 10, 20, 40], [-1, 20, 30, 60])])
def test_prefill_flags_bad_offsets(qo, kv, nsplit):
    """A request whose offsets do not hold is flagged and left; the others are done."""
    b = prefill_batch(31, [(40, 60)], 2, torch.bfloat16, pad=0)
    out, lse, err = torch.full((40, 2, 128), 5.0, dtype=torch.bfloat16, device=DEV), torch.full((40, 2), 5.0, device=DEV), i32([0])
    ws = torch.zeros(nsplit * 40 * 2 * 129 * 4, dtype=torch.uint8, device=DEV)
    pkg.prefill_run(b["q"], b["k_nope"], b["k_rope"], b["v"], i64(qo), i32(kv), 20, 40, 192 ** -0.5, out, lse, nsplit=nsplit,
                    workspace=ws, err=err)
    assert int(err) == binding.DEVERR_INDPTR
    ref = L.prefill(b["q"], b["k_nope"], b["k_rope"], b["v"], [0, 1], [0, 1], 1.0)  # shapes only
    for r in range(3):
        ok = 0 <= qo[r] <= qo[r + 1] <= 40 and 0 <= kv[r] <= kv[r + 1] <= 60 and qo[r + 1] - qo[r] <= 20 and kv[r + 1] - kv[r] <= 40
        if ok:
            ref = L.prefill(b["q"], b["k_nope"], b["k_rope"], b["v"], qo[r:r + 2], kv[r:r + 2], 192 ** -0.5)
            real = ~ref["lse"].isnan().all(dim=1)
            bound, _ = prefill_bounds({k: v[real] for k, v in ref.items()}, 40, torch.bfloat16)
            within(out.cpu()[real], ref["out"][real], bound, f"request {r}")


def test_prefill_keys_past_two_to_the_31_elements():
    """The last request's keys lie past 2^31 elements of their buffer."""
    heads, rows = 64, 140000
    kv = torch.empty((rows, heads, 256), dtype=torch.bfloat16, device=DEV)
    kv[-200:] = rnd(37, (200, heads, 256), torch.bfloat16)
    latent = rnd(38, (rows, 64), torch.bfloat16)
    q = rnd(39, (40, heads, 192), torch.bfloat16)
    out, lse = torch.empty((40, heads, 128), dtype=torch.bfloat16, device=DEV), torch.empty((40, heads), device=DEV)
    pkg.prefill_run(q, kv[:, :, :128], latent, kv[:, :, 128:], i64([0, 40]), i32([rows - 150, rows]), 40, 150, 0.07, out, lse)
    ref = L.prefill(q, kv[-150:, :, :128], latent[-150:], kv[-150:, :, 128:], [0, 40], [0, 150], 0.07)
    bound, _ = prefill_bounds(ref, 150, torch.bfloat16)
    within(out, ref["out"], bound)


@pytest.mark.parametrize("heads,rows,keys", [(2, 60, 5000), (3, 1, 9000), (64, 300, 300)])
def test_prefill_object_splits_and_captures(heads, rows, keys):
    """MlaPrefill's own split count; replays follow inputs and offsets changed in place."""
    b = prefill_batch(41, [(rows, keys)], heads, torch.bfloat16)
    p = pkg.MlaPrefill(2, rows, rows + 3, keys, heads)
    qo, kv = i64([0, rows, rows]), i32([0, keys, keys])
    args = (b["q"], b["k_nope"], b["k_rope"], b["v"], qo, kv, 192 ** -0.5)
    out, lse = p(*args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    got, got_lse = torch.zeros_like(out), torch.zeros_like(lse)
    with torch.cuda.graph(graph, stream=side):
        p(*args, out=got, lse=got_lse)
    graph.replay()
    assert torch.equal(got, out) and torch.equal(got_lse, lse)
    b["v"].mul_(-1)
    b["v"][keys:] = math.nan
    cut = keys - keys // 3
    kv.copy_(i32([0, cut, cut]))
    got.zero_()
    graph.replay()
    ref = L.prefill(b["q"], b["k_nope"], b["k_rope"], b["v"], [0, rows], [0, cut], 192 ** -0.5)
    bound, lse_bound = prefill_bounds({k: v[:rows] for k, v in ref.items()}, keys, torch.bfloat16)
    within(got[:rows], ref["out"][:rows], bound)
    some = ref["lse"][:rows] > -math.inf
    within(got_lse[:rows].cpu()[some], ref["lse"][:rows][some], lse_bound[some])
    assert (got[rows:] == 0).all() and p.device_error() == 0
    with pytest.raises(ValueError):
        p(b["q"], b["k_nope"], b["k_rope"], b["v"], i64([0, 1, 1, 1]), i32([0, 1, 1, 1]), 1.0)


def test_prefill_without_rows():
    e = lambda *s: torch.empty(s, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    assert pkg.prefill_run(e(0, 2, 192), e(4, 2, 128), e(4, 64), e(4, 2, 128), i64([0]), i32([0]), 0, 4, 1.0, e(0, 2, 128)) == 0
    out, lse = torch.full((2, 2, 128), 3.0, dtype=torch.bfloat16, device=DEV), torch.zeros((2, 2), device=DEV)
    pkg.prefill_run(rnd(1, (2, 2, 192), torch.bfloat16), e(0, 2, 128), e(0, 64), e(0, 2, 128), i64([0, 2]), i32([0, 0]), 2, 0, 1.0,
                    out, lse)
    assert (out == 0).all() and (lse == -math.inf).all()


# ---------------------------------------------------------- norms with rotation

def norm_case(seed, tokens, heads, nope, rope_dim, dtype, layout, q_norm=True, c_norm=True, pool=True, valid=None, strides=0,
              in_place=False, amplitude=1.0, eps=1e-6):
    """Runs norm_rope_write into buffers with room around the outputs and checks every value of them."""
    dim = nope + rope_dim
    size = torch.exp(rnd(seed, (tokens, heads, 1), torch.float32))
    q_in = (rnd(seed + 1, (tokens, heads, dim + strides), torch.float32) * size).to(dtype)[:, :, strides:]
    qw = (1 + rnd(seed + 2, (dim,), torch.float32, 0.2)).to(dtype) if q_norm else None
    down = rnd(seed + 3, (tokens, 576 + strides), dtype, 3.0)[:, strides:]
    cw = (1 + rnd(seed + 4, (512,), torch.float32, 0.2)).to(dtype) if c_norm else None
    turns, _ = pkg.rope_freqs(rope_dim, 10000.0)
    positions = torch.randint(0, 100000, (tokens,), generator=torch.Generator().manual_seed(seed)).to(DEV)
    n = tokens if valid is None else valid
    ref_in = q_in.double().cpu()
    # oracle
    half = layout == binding.ROPE_HALF
    q_ref = L.norm(q_in, qw, eps) if q_norm else ref_in
    turned, mag = S.rope(q_ref[..., nope:].numpy(), positions.tolist(), turns.tolist(), amplitude, half)
    turned, mag = torch.from_numpy(turned), torch.from_numpy(mag)
    u, tiny = half_step(dtype)
    rel = (dim / 2 + 16) * 2.0 ** -24
    # outputs
    if in_place:
        nope_buf = rope_buf = q_in
        q_nope, q_rope = (q_in[:, :, :nope] if q_norm and nope else None), q_in[:, :, nope:]
    else:
        nope_buf = torch.full((tokens, heads, nope + strides + 2), 9.0, dtype=dtype, device=DEV)
        rope_buf = torch.full((tokens, heads, 512 + rope_dim), 9.0, dtype=dtype, device=DEV)
        q_nope, q_rope = (nope_buf[:, :, :nope] if q_norm and nope else None), rope_buf[:, :, 512:]
    kw = {}
    if pool:
        slots = 2 * tokens + 3
        kv = torch.full((slots, 576), 9.0, dtype=torch.bfloat16, device=DEV)
        loc = torch.randperm(slots, generator=torch.Generator().manual_seed(seed))[:tokens].to(DEV)
        kw = dict(c_in=down[:, :512], c_weight=cw, k_in=down[:, 512:], out_cache_loc=loc, kv_pool=kv)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    pkg.norm_rope_write(turns.to(DEV), positions, eps, layout, amplitude, q_in=q_in, q_weight=qw, q_nope=q_nope, q_rope=q_rope,
                        num_valid=None if valid is None else i64([valid]), err=err, **kw)
    torch.cuda.synchronize()
    assert int(err) == 0
    within(q_rope[:n], turned[:n], (u * turned.abs() + (rel + 2.0 ** -22) * mag + tiny)[:n], "q_rope")
    if q_nope is not None:
        want = q_ref[..., :nope]
        within(q_nope[:n], want[:n], (u * want.abs() + rel * want.abs() + tiny)[:n], "q_nope")
    if in_place:
        assert torch.equal(q_in[n:].double().cpu(), ref_in[n:])
    else:
        assert (rope_buf[:, :, :512] == 9).all() and (rope_buf[n:] == 9).all()
        assert (nope_buf[:, :, nope if q_norm else 0:] == 9).all() and (nope_buf[n:] == 9).all()
    if pool:
        ub, tb = half_step(torch.bfloat16)
        lat = L.norm(down[:, :512], cw, eps) if c_norm else down[:, :512].double().cpu()
        within(kv[loc[:n], :512], lat[:n], (ub * lat.abs() + 272 * 2.0 ** -24 * lat.abs() + tb)[:n], "latent")
        key, kmag = S.rope(down[:, 512:].double().cpu().numpy(), positions.tolist(), turns.tolist(), amplitude, half)
        key, kmag = torch.from_numpy(key), torch.from_numpy(kmag)
        within(kv[loc[:n], 512:], key[:n], (ub * key.abs() + 2.0 ** -21 * kmag + tb)[:n], "key")
        rest = torch.ones(slots, dtype=torch.bool, device=DEV)
        rest[loc[:n]] = False
        assert (kv[rest] == 9).all()


LAYOUTS = [binding.ROPE_INTERLEAVED, binding.ROPE_HALF]


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens,heads", [(1, 1), (8, 64), (5, 7), (3, 130)])
def test_norm_rope_write(tokens, heads, dtype, layout):
    norm_case(tokens + heads, tokens, heads, 128, 64, TYPES[dtype], layout)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("q_norm,c_norm", [(False, True), (True, False), (False, False)])
def test_norm_rope_write_without_one_norm(q_norm, c_norm, dtype, layout):
    norm_case(3, 9, 20, 128, 64, TYPES[dtype], layout, q_norm=q_norm, c_norm=c_norm)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("nope,rope_dim", [(0, 64), (8, 16), (128, 2), (96, 32), (448, 64), (7, 10), (960, 64), (768, 256), (0, 2),
                                           (192, 24)])
def test_norm_rope_write_head_sizes(nope, rope_dim, layout):
    for dtype in TYPES.values():
        norm_case(nope + rope_dim, 4, 5, nope, rope_dim, dtype, layout, pool=rope_dim == 64)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("strides", [1, 2, 8])
def test_norm_rope_write_strides(strides, dtype, layout):
    norm_case(strides, 6, 9, 128, 64, TYPES[dtype], layout, strides=strides)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", TYPES)
def test_norm_rope_write_in_place_and_padded(dtype, layout):
    norm_case(2, 13, 33, 128, 64, TYPES[dtype], layout, valid=9, in_place=True)
    norm_case(4, 13, 33, 128, 64, TYPES[dtype], layout, valid=0)
    norm_case(5, 7, 3, 128, 64, TYPES[dtype], layout, q_norm=False, in_place=True, amplitude=1.3)


def test_norm_rope_write_small_and_large_values():
    """Rows of zeros, of tiny and of large values: eps carries the first, fp32 the squares of the rest."""
    for scale in (0.0, 1e-4, 1e4):
        c = rnd(1, (3, 576), torch.float32, 1.0) * scale
        pool = torch.zeros((3, 576), dtype=torch.bfloat16, device=DEV)
        turns, _ = pkg.rope_freqs(64, 10000.0)
        w = torch.ones(512, device=DEV)
        pkg.norm_rope_write(turns.to(DEV), i64([0, 1, 2]), 1e-6, c_in=c[:, :512], c_weight=w, k_in=c[:, 512:],
                            out_cache_loc=i64([2, 0, 1]), kv_pool=pool)
        ref = L.norm(c[:, :512], w, 1e-6)
        within(pool[i64([2, 0, 1]), :512], ref, ref.abs() * (2.0 ** -8 + 272 * 2.0 ** -24))


def test_norm_rope_write_flags_slots_and_leaves_them():
    for dtype in TYPES.values():
        c, q = rnd(1, (4, 576), dtype), rnd(2, (4, 2, 192), dtype)
        pool, err = torch.full((5, 576), 9.0, dtype=torch.bfloat16, device=DEV), i32([0])
        turns, _ = pkg.rope_freqs(64, 10000.0)
        out = torch.zeros((4, 2, 64), dtype=dtype, device=DEV)
        pkg.norm_rope_write(turns.to(DEV), i64([0, 1, 2, 3]), 1e-6, q_in=q, q_rope=out, c_in=c[:, :512],
                            c_weight=torch.ones(512, dtype=dtype, device=DEV), k_in=c[:, 512:], out_cache_loc=i64([-1, 3, 5, 1 << 40]),
                            kv_pool=pool, err=err)
        assert int(err) == binding.DEVERR_SLOT_RANGE
        assert (pool[[0, 1, 2, 4]] == 9).all() and not (pool[3] == 9).all()
        assert (out[0] == q[0, :, 128:]).all() and (out[1:] != 0).any(dim=2).all()


def test_norm_rope_write_of_one_kind_matches_rope_write():
    """Without weights it is rope_write, bit for bit."""
    for layout in LAYOUTS:
        q, c = rnd(1, (9, 8, 192), torch.bfloat16), rnd(2, (9, 576), torch.bfloat16)
        turns, pos = pkg.rope_freqs(64, 10000.0)[0].to(DEV), i64(list(range(0, 90000, 10000)))
        outs = [torch.zeros((9, 8, 64), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
        pools = [torch.zeros((16, 576), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
        loc = i64([3, 1, 4, 15, 9, 2, 6, 5, 8])
        pkg.rope_write(turns, pos, layout, q_in=q[:, :, 128:], q_out=outs[0], k_in=c[:, 512:], c_in=c[:, :512], out_cache_loc=loc,
                       kv_pool=pools[0])
        pkg.norm_rope_write(turns, pos, 0.0, layout, q_in=q, q_rope=outs[1], c_in=c[:, :512], k_in=c[:, 512:], out_cache_loc=loc,
                            kv_pool=pools[1])
        assert torch.equal(outs[0], outs[1]) and torch.equal(pools[0], pools[1])


# ------------------------------------------------------------- a run of them

def test_captured_layer_follows_its_inputs():
    """Norms, pool write, absorption and values in one graph: replays with other inputs, positions,
    slots and numbers of valid tokens give what calls one by one give."""
    bf, tokens, heads = torch.bfloat16, 37, 64
    turns = pkg.rope_freqs(64, 10000.0)[0].to(DEV)
    proj, down = rnd(1, (tokens, heads, 192), bf), rnd(2, (tokens, 576), bf)
    up, qw, cw = rnd(3, (heads, 256, 512), bf, 0.05), rnd(4, (192,), bf), rnd(5, (512,), bf)
    positions, loc, valid = i64(list(range(tokens))), i64(list(range(tokens, 0, -1))), i64([tokens])

    def step(pool, nope, q, values):
        pkg.norm_rope_write(turns, positions, 1e-6, q_in=proj, q_weight=qw, q_nope=nope, q_rope=q[:, :, 512:], c_in=down[:, :512],
                            c_weight=cw, k_in=down[:, 512:], out_cache_loc=loc, kv_pool=pool, num_valid=valid)
        pkg.head_product(nope, up[:, :128], q[:, :, :512])
        pkg.head_product(q[:, :, :512], up[:, 128:].transpose(1, 2), values)

    def buffers():
        return (torch.zeros((64, 576), dtype=bf, device=DEV), torch.zeros((tokens, heads, 128), dtype=bf, device=DEV),
                torch.zeros((tokens, heads, 576), dtype=bf, device=DEV), torch.zeros((tokens, heads, 128), dtype=bf, device=DEV))

    captured = buffers()
    step(*captured)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(*captured)
    for i, n in enumerate((tokens, 20, 0)):
        proj.copy_(rnd(10 + i, proj.shape, bf))
        down.copy_(rnd(20 + i, down.shape, bf))
        positions.add_(1000)
        loc.copy_(loc.roll(3))
        valid.fill_(n)
        want = buffers()
        for t in captured:
            t.zero_()
        graph.replay()
        step(*want)
        torch.cuda.synchronize()
        for a, b in zip(captured, want):
            assert torch.equal(a, b)


def test_absorbed_and_expanded_layers_agree():
    """One layer's attention both ways: norms, rotation and pool write, then
    absorbed queries through verify attention over the pool, and expanded keys
    through prefill attention; every stage within the oracle's bound for its
    own inputs, and the two results within the bound of their roundings."""
    bf, heads = torch.bfloat16, 64
    new, cached = [40, 17], [100, 0]
    total, slots = sum(new) + sum(cached), 256
    up = rnd(1, (heads, 256, 512), bf, 512 ** -0.5)  # 128 key rows, then 128 value rows a head
    down, proj = rnd(2, (total, 576), bf), rnd(3, (total, heads, 192), bf)
    qw, cw = (1 + rnd(4, (192,), torch.float32, 0.1)).to(bf), (1 + rnd(5, (512,), torch.float32, 0.1)).to(bf)
    turns, amplitude = pkg.rope_freqs(64, 10000.0)
    loc = torch.randperm(slots, generator=torch.Generator().manual_seed(1))[:total].to(DEV)
    positions = torch.cat([torch.arange(n + c) for n, c in zip(new, cached)]).to(DEV)
    pool = torch.zeros((slots, 576), dtype=bf, device=DEV)
    q = torch.zeros((total, heads, 192), dtype=bf, device=DEV)
    pkg.norm_rope_write(turns.to(DEV), positions, 1e-6, amplitude=amplitude, q_in=proj, q_weight=qw, q_nope=q[:, :, :128],
                        q_rope=q[:, :, 128:], c_in=down[:, :512], c_weight=cw, k_in=down[:, 512:], out_cache_loc=loc, kv_pool=pool)
    # the new tokens of each request are its last ones
    start = [0, new[0] + cached[0]]
    is_new = torch.zeros(total, dtype=torch.bool, device=DEV)
    for s, n, c in zip(start, new, cached):
        is_new[s + c:s + c + n] = True
    q = q[is_new].contiguous()
    kv_indptr, qo_indptr = i32([0, start[1], total]), i64([0, new[0], sum(new)])
    scale = 192 ** -0.5

    # expanded: every request's rows in one run, its latents to keys and values
    dense = torch.zeros((total, 576), dtype=bf, device=DEV)
    runs = torch.zeros((slots, 576), dtype=bf, device=DEV)
    pkg.kv_defrag(pool, runs, loc, kv_indptr, 2, total, i64(start), torch.empty_like(loc))
    dense = runs[:total]
    kv = torch.empty((total, heads, 256), dtype=bf, device=DEV)
    x = dense[:, None, :512].expand(total, heads, 512)
    pkg.head_product(x, up.transpose(1, 2), kv)
    ref, mag = L.head_product(x, up.transpose(1, 2))
    within(kv, ref, product_bound(ref, mag, 512, bf), "expansion")
    p = pkg.MlaPrefill(2, max(new), sum(new), total, heads)
    out, lse = p(q, kv[:, :, :128], dense[:, 512:], kv[:, :, 128:], qo_indptr, kv_indptr, scale)
    want = L.prefill(q, kv[:, :, :128], dense[:, 512:], kv[:, :, 128:], qo_indptr.tolist(), kv_indptr.tolist(), scale)
    bound, lse_bound = prefill_bounds(want, total, bf)
    within(out, want["out"], bound, "expanded attention")
    within(lse, want["lse"], lse_bound, "expanded lse")

    # absorbed: queries to the latent space, verify attention with a chain as its tree, latents to values
    qa = torch.empty((sum(new), heads, 576), dtype=bf, device=DEV)
    qa[:, :, 512:] = q[:, :, 128:]
    pkg.head_product(q[:, :, :128], up[:, :128], qa[:, :, :512])
    ref, mag = L.head_product(q[:, :, :128], up[:, :128])
    within(qa[:, :, :512], ref, product_bound(ref, mag, 128, bf), "absorption")
    prefix = torch.cat([loc[s:s + c] for s, c in zip(start, cached)])
    tree_loc = torch.cat([loc[s + c:s + c + n] for s, c, n in zip(start, cached, new)])
    prefix_indptr = i32([0, cached[0], sum(cached)])
    parents = i32([i - 1 for n in new for i in range(n)])
    mask = torch.zeros(sum(n * n for n in new), dtype=torch.uint8, device=DEV)
    mask_indptr = torch.zeros(3, dtype=torch.int64, device=DEV)
    binding.tree_mask_build(parents, qo_indptr, prefix_indptr, 2, max(new), binding.MASK_TREE_ONLY, mask, mask_indptr)
    m = pkg.MlaTreeVerify(2, max(new), sum(new), max(cached), mask_layout=binding.MASK_TREE_ONLY)
    latent, lse_a = m(qa, pool, prefix, prefix_indptr, tree_loc, qo_indptr, mask, mask_indptr, scale)
    values = torch.empty((sum(new), heads, 128), dtype=bf, device=DEV)
    pkg.head_product(latent, up[:, 128:].transpose(1, 2), values)
    ref, mag = L.head_product(latent, up[:, 128:].transpose(1, 2))
    within(values, ref, product_bound(ref, mag, 512, bf), "values")
    assert m.device_error() == 0 and p.device_error() == 0
    # both round the scores' operands to bf16 (expanded keys, absorbed queries): independent errors of 2^-8 at most
    # of each of 128 and 512 products, and weights, latents and values once each; their root sums of squares
    # are below 0.03 in the scores and 0.02 in outputs of about 0.1 to 1, of which the largest of 460,000 is within 8
    assert (lse - lse_a).abs().max() < 0.25
    assert (out.float() - values.float()).abs().max() < 0.16
    assert (out.float() - values.float()).square().mean().sqrt() < 0.02 * max(1.0, out.float().square().mean().sqrt().item())


# ----------------------------------------- prefill, the last blocks' keys split

LAST = 256  # one of nsplit's split blocks
# two results of values below 5 in bf16: the weights' and the output's half step each
TWICE = 4 * 5 * 2.0 ** -8


@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("n,blocks", [(2, 1), (3, 2), (9, 3), (64, 5), (2, 20), (1, 2)])
@pytest.mark.parametrize("name", ["two tiles", "odd", "ragged", "fewer keys", "first rows without keys"])
def test_prefill_with_the_last_blocks_split(name, n, blocks, dtype):
    check_prefill(prefill_batch(41, CASES[name], 2, TYPES[dtype]), TYPES[dtype], nsplit=n + LAST * blocks)


def test_prefill_of_all_keys_with_the_last_blocks_split():
    check_prefill(prefill_batch(43, CASES["odd"], 3, torch.bfloat16), torch.bfloat16, causal=False, nsplit=4 + LAST * 2)


def test_prefill_splits_the_last_blocks_only():
    """Blocks before the last are as without a split, and the workspace is used to its documented size."""
    b = prefill_batch(47, [(300, 700), (200, 600)], 2, torch.bfloat16)
    want, want_lse = check_prefill(b, torch.bfloat16)
    size = 3 * 3 * 256 * 129 * 4
    ws = torch.full((size + 256,), 77, dtype=torch.uint8, device=DEV)
    out, lse, err = torch.zeros_like(want), torch.zeros_like(want_lse), torch.zeros(1, dtype=torch.int32, device=DEV)
    run = lambda space: pkg.prefill_run(b["q"], b["k_nope"], b["k_rope"], b["v"], i64(b["qo"]), i32(b["kv"]), 300, 700,  # noqa: E731
                                        192 ** -0.5, out, lse, nsplit=3 + LAST * 3, workspace=space, err=err)
    run(ws[:size])
    assert int(err) == 0 and (ws[size:] == 77).all()
    # two blocks a head by its bound of 300 rows: the last three are those of the second request's rows
    assert torch.equal(out[:300], want[:300]) and torch.equal(lse[:300], want_lse[:300])
    ref = L.prefill(b["q"], b["k_nope"], b["k_rope"], b["v"], b["qo"], b["kv"], 192 ** -0.5, True)
    real = slice(300, 500)
    bound, lse_bound = prefill_bounds({k: v[real] for k, v in ref.items()}, 700, torch.bfloat16)
    within(out.cpu()[real], ref["out"][real], bound, "out")
    within(lse.cpu()[real], ref["lse"][real], lse_bound, "lse")
    with pytest.raises(pkg.MtvError):
        run(ws[:size - 1])


@pytest.mark.parametrize("nsplit", [2 + LAST, 5 + LAST * 4])
def test_prefill_with_the_last_blocks_split_flags_bad_offsets(nsplit):
    b = prefill_batch(53, [(10, 20), (10, 20), (20, 30)], 2, torch.bfloat16)
    out = torch.full((43, 2, 128), 5.0, dtype=torch.bfloat16, device=DEV)
    lse, err = torch.full((43, 2), 5.0, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    ws = torch.full((64 * 4 * 256 * 129,), 255, dtype=torch.uint8, device=DEV)
    pkg.prefill_run(b["q"], b["k_nope"], b["k_rope"], b["v"], i64([0, 10, 20, 40]), i32([0, 20, 40, 999]), 20, 40, 192 ** -0.5,
                    out, lse, nsplit=nsplit, workspace=ws, err=err)
    assert int(err) == binding.DEVERR_INDPTR
    assert (out[20:] == 5).all() and (lse[20:] == 5).all()
    want, want_lse = check_prefill({**b, "qo": b["qo"][:3], "kv": b["kv"][:3]}, torch.bfloat16)
    torch.testing.assert_close(out[:20], want[:20], rtol=0, atol=TWICE)  # the first requests are there


def test_prefill_object_splits_a_part_filled_wave():
    """A few blocks more than SMs over long keys, and a smaller batch in the same object."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    heads = sms + 3
    p = pkg.MlaPrefill(1, 20, 23, 2100, heads)
    assert p.nsplit % LAST > 1 and p.nsplit // LAST == 3
    b = prefill_batch(59, [(20, 2100)], heads, torch.bfloat16)
    want, want_lse = check_prefill(b, torch.bfloat16)
    out, lse = p(b["q"], b["k_nope"], b["k_rope"], b["v"], i64(b["qo"]), i32(b["kv"]), 192 ** -0.5)
    assert p.device_error() == 0
    assert torch.equal(out[:20, :sms], want[:20, :sms]) and torch.equal(lse[:20, :sms], want_lse[:20, :sms])
    few = slice(sms, heads)
    ref = L.prefill(b["q"][:, few], b["k_nope"][:, few], b["k_rope"], b["v"][:, few], b["qo"], b["kv"], 192 ** -0.5, True)
    bound, lse_bound = prefill_bounds({k: v[:20] for k, v in ref.items()}, 2100, torch.bfloat16)
    within(out.cpu()[:20, few], ref["out"][:20], bound, "out")
    within(lse.cpu()[:20, few], ref["lse"][:20], lse_bound, "lse")
    short = {**b, "qo": [0, 5], "kv": [0, 700]}
    got, _ = p(b["q"], b["k_nope"], b["k_rope"], b["v"], i64(short["qo"]), i32(short["kv"]), 192 ** -0.5)
    want, _ = check_prefill(short, torch.bfloat16)
    assert torch.equal(got[:5, :sms], want[:5, :sms])
    torch.testing.assert_close(got[:5, few], want[:5, few], rtol=0, atol=TWICE)


def test_prefill_with_the_last_blocks_split_in_a_graph():
    b = prefill_batch(61, [(300, 700)], 2, torch.bfloat16)
    eager, eager_lse = check_prefill(b, torch.bfloat16, nsplit=3 + LAST * 2)
    out, lse = torch.full_like(eager, 5.0), torch.full_like(eager_lse, 5.0)
    qo, kv = i64(b["qo"]), i32(b["kv"])
    ws = torch.full((3 * 2 * 256 * 129 * 4,), 255, dtype=torch.uint8, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(2):
            pkg.prefill_run(b["q"], b["k_nope"], b["k_rope"], b["v"], qo, kv, 300, 700, 192 ** -0.5, out, lse,
                            nsplit=3 + LAST * 2, workspace=ws)
    for _ in range(3):
        out.fill_(5.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager) and torch.equal(lse, eager_lse)


# ------------------------------------------------- products of pairs of SMs

PAIRED = [(130, 400, 264, 136), (200, 191, 320, 400), (24400, 4, 264, 256), (97500, 1, 512, 200)]  # five units a pair and more


@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("tokens,heads,k,n", PAIRED)
@pytest.mark.parametrize("dense", ["n", "k"])
def test_head_product_of_many_tokens(tokens, heads, k, n, dense, dtype):
    """NaN behind x and around w; outputs inside wider rows."""
    t = TYPES[dtype]
    x = torch.full((tokens + 5, heads, k + 8), math.nan, dtype=t, device=DEV)
    x[:tokens, :, :k] = rnd(tokens, (tokens, heads, k), t)
    shape = (heads, k, n) if dense == "n" else (heads, n, k)
    w = torch.full((heads, shape[1] + 8, shape[2] + 8), math.nan, dtype=t, device=DEV)
    w[:, :shape[1], :shape[2]] = rnd(n + k, shape, t)
    w = w[:, :shape[1], :shape[2]]
    check_product(x[:tokens, :, :k], w if dense == "n" else w.transpose(1, 2), pad_dim=8)


@pytest.mark.parametrize("dense", ["n", "k"])
def test_head_product_of_many_tokens_shared_by_the_heads(dense):
    rows = rnd(3, (2050, 576), torch.bfloat16)
    x = rows[:, None, :512].expand(2050, 50, 512)
    w = rnd(5, (50, 256, 512), torch.bfloat16, 0.05).transpose(1, 2)
    check_product(x, w if dense == "k" else w.contiguous(), pad_dim=0)


def test_head_product_of_many_tokens_again_and_in_a_graph():
    x, w = rnd(1, (1024, 100, 512), torch.bfloat16), rnd(2, (100, 512, 256), torch.bfloat16)
    first, again = torch.empty((2, 1024, 100, 256), dtype=torch.bfloat16, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    pkg.head_product(x, w, first, err=err)
    graph, side = torch.cuda.CUDAGraph(), torch.empty_like(first)
    with torch.cuda.graph(graph):
        pkg.head_product(x, w, again, err=err)
        pkg.head_product(x, w, side, err=err)
    for _ in range(3):
        again.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(first, again) and torch.equal(first, side) and int(err) == 0


def test_head_products_of_many_tokens_on_two_streams():
    x, w = rnd(1, (1024, 100, 512), torch.bfloat16), rnd(2, (100, 512, 256), torch.bfloat16)
    want = torch.empty((1024, 100, 256), dtype=torch.bfloat16, device=DEV)
    pkg.head_product(x, w, want)
    few = torch.empty((8, 100, 256), dtype=torch.bfloat16, device=DEV)
    pkg.head_product(x[:8], w, few)
    outs, fews = [torch.zeros_like(want) for _ in range(6)], [torch.zeros_like(few) for _ in range(6)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for i in range(6):
        with torch.cuda.stream(streams[i % 2]):
            pkg.head_product(x, w, outs[i])
            pkg.head_product(x[:8], w, fews[i])
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs) and all(torch.equal(o, few) for o in fews)


# --------------------------------- kernels that set up while the one before ends

@pytest.mark.parametrize("tokens,heads,dim", [(8, 64, 128), (300, 20, 512), (1024, 80, 512), (40, 3, 100)])
def test_products_in_a_row_read_what_the_call_before_wrote(tokens, heads, dim):
    """Each call's input is the output of the one before, or of a copy; in a row as with a wait after each."""
    ws = [rnd(70 + i, (heads, dim, dim), torch.bfloat16, dim ** -0.5) for i in range(4)]
    sources = [rnd(80 + i, (tokens, heads, dim), torch.bfloat16) for i in range(6)]
    x = torch.empty_like(sources[0])
    mids = [torch.empty_like(x) for _ in range(4)]

    def run(source, wait):
        x.copy_(source)
        at = x
        for w, mid in zip(ws, mids):
            pkg.head_product(at, w, mid)
            if wait:
                torch.cuda.synchronize()
            at = mid
        return at.clone()

    want = [run(s, True) for s in sources]
    got = [run(s, False) for s in sources * 3]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = [run(s, False) for s in sources]
    graph.replay()
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert torch.equal(g, want[i % 6])
    for g, w in zip(captured, want):
        assert torch.equal(g, w)


def test_a_layer_in_a_row_is_as_with_a_wait_after_each_call():
    """Norms, expansion and prompt attention with and without split keys, a new pass right behind the last."""
    heads, rows = 8, 40
    up = rnd(91, (heads, 256, 512), torch.bfloat16, 512 ** -0.5)
    q_in, c_in, k_in = rnd(92, (rows, heads, 192), torch.bfloat16), rnd(93, (rows, 512), torch.bfloat16), rnd(94, (rows, 64), torch.bfloat16)
    q_weight, c_weight = rnd(95, (192,), torch.bfloat16), rnd(96, (512,), torch.bfloat16)
    old = 1500
    pool = rnd(97, (old + rows, 576), torch.bfloat16)
    start = pool.clone()
    turns, amplitude = pkg.rope_freqs(64, 1e4)
    turns = turns.to(DEV)
    positions, loc = torch.arange(old, old + rows, device=DEV), torch.arange(old, old + rows, device=DEV)
    q = torch.empty_like(q_in)
    kv = torch.empty((old + rows, heads, 256), dtype=torch.bfloat16, device=DEV)
    qo, ko = i64([0, rows]), i32([0, old + rows])
    attention = pkg.MlaPrefill(1, rows, rows, old + rows, heads)
    assert attention.nsplit > 1

    def run(wait):
        step = torch.cuda.synchronize if wait else lambda: None
        pool.copy_(start)
        kv.fill_(math.nan), q.fill_(math.nan), step()
        pkg.norm_rope_write(turns, positions, 1e-6, amplitude=amplitude, q_in=q_in, q_weight=q_weight, q_nope=q[:, :, :128],
                            q_rope=q[:, :, 128:], c_in=c_in, c_weight=c_weight, k_in=k_in, out_cache_loc=loc, kv_pool=pool), step()
        pkg.head_product(pool[:, None, :512].expand(-1, heads, -1), up.transpose(1, 2), kv), step()
        out = torch.empty((rows, heads, 128), dtype=torch.bfloat16, device=DEV)
        lse = torch.empty((rows, heads), device=DEV)
        attention(q, kv[:, :, :128], pool[:, 512:], kv[:, :, 128:], qo, ko, 192 ** -0.5, out, lse), step()
        return out.clone(), lse.clone()

    want = run(True)
    for out, lse in [run(False) for _ in range(20)]:
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    assert torch.isfinite(want[0].float()).all()


def test_products_behind_a_fork_and_a_join_of_streams_in_a_graph():
    """The joining call waits for a kernel, a copy and a fill of other streams."""
    x, w = rnd(1, (8, 16, 128), torch.bfloat16), rnd(2, (16, 128, 128), torch.bfloat16, 0.1)
    big = rnd(3, (4000, 16, 128), torch.bfloat16)
    a, far = torch.zeros((4008, 16, 128), dtype=torch.bfloat16, device=DEV), torch.zeros((4008, 16, 128), dtype=torch.bfloat16, device=DEV)
    out, out2 = torch.zeros_like(a), torch.zeros_like(a)
    sides = [torch.cuda.Stream() for _ in range(3)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        a.zero_()
        for i, side in enumerate(sides):
            side.wait_stream(main)
            with torch.cuda.stream(side):
                if i == 0:
                    pkg.head_product(x, w, a[4000:])
                elif i == 1:
                    a[:4000].copy_(big)
                else:
                    far.fill_(0)
        for side in sides:
            main.wait_stream(side)
        pkg.head_product(a, w, out)
        sides[0].wait_stream(main)
        with torch.cuda.stream(sides[0]):
            pkg.head_product(out, w, far)
        main.wait_stream(sides[0])
        pkg.head_product(far, w, out2)
    for _ in range(5):
        out.zero_(), out2.zero_(), far.fill_(1)
        graph.replay()
    torch.cuda.synchronize()
    want = torch.empty_like(a)
    pkg.head_product(x, w, a[4000:])
    torch.cuda.synchronize()
    steps = [a.clone()]
    steps[0][:4000] = big
    for _ in range(3):
        pkg.head_product(steps[-1], w, want)
        torch.cuda.synchronize()
        steps.append(want.clone())
    assert torch.equal(out, steps[1]) and torch.equal(far, steps[2]) and torch.equal(out2, steps[3])


# ------------------------- prefill in blocks of 256 rows (few of them: of 128)

@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("name", ["two tiles", "odd", "ragged", "fewer keys", "first rows without keys", "many blocks"])
def test_prefill_of_more_blocks_than_half_of_the_sms(name, causal, dtype):
    heads = 78 if len(CASES[name]) == 1 else 30
    check_prefill(prefill_batch(67, CASES[name], heads, TYPES[dtype]), TYPES[dtype], causal=causal)


def test_prefill_in_blocks_of_128_and_of_256_rows():
    """A head's rows come out alike among few heads and among many."""
    b = prefill_batch(71, [(300, 500), (129, 700)], 80, torch.bfloat16)
    many, many_lse = check_prefill(b, torch.bfloat16)
    few = {**b, **{k: b[k][:, 7:10] for k in ("q", "k_nope", "v")}}
    out, lse = check_prefill(few, torch.bfloat16)
    assert torch.equal(out, many[:, 7:10]) and torch.equal(lse, many_lse[:, 7:10])
