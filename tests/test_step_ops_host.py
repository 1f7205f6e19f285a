"""Serving-step operators without a GPU: the oracle's pins, the host-side
frequency table, and every refusal of the C entries and of the binding."""
import ctypes
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

import paged_mla_speculative_tree_gb300 as pkg
from oracle import step_ops as S
from paged_mla_speculative_tree_gb300 import binding, build

FAKE = ctypes.c_void_p(0x100000)  # never dereferenced: checks fail first, or nothing is left to do


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


# ------------------------------------------------------------------- oracle

def test_page_oracle_rolls_back_and_keeps_every_page_once():
    rng = np.random.default_rng(3)
    rows, per = 9, 12
    held = [int(x) for x in rng.integers(0, per, rows)]
    ids = [int(x) for x in rng.permutation(rows * per)]
    table = [[ids.pop() if j < held[r] else -7 for j in range(per)] for r in range(rows)]
    lens = [h * 4 for h in held]
    grown = S.page_table_update([n + 9 if n < 4 * per - 9 else n for n in lens], 4, table, held, ids)
    back = S.page_table_update(lens, 4, *grown[:3])
    assert back[1] == held and back[2] == ids and not grown[3] and not back[3]
    in_use = [p for r in range(rows) for p in grown[0][r][:grown[1][r]]]
    assert sorted(in_use + grown[2]) == list(range(rows * per))


def test_page_oracle_hand_example():
    # row 0 releases pages 5, 6; row 1 grows by three: 5, 6 (pushed last first, so 5 is on top), then 9
    table, held, free, flagged = S.page_table_update([2, 10], 2, [[4, 5, 6, 0, 0], [1, 2, 0, 0, 0]], [3, 2], [8, 9])
    assert (table[1][:5], held, free, flagged) == ([1, 2, 5, 6, 9], [1, 5], [8], [])


def test_slot_map_oracle_hand_example():
    kv_ptr, kv, q_ptr, loc, pos = S.slot_map([[7, 2, 5], [0, 1, 3]], 2, [1, 0], [3, 0], [2, 3], [[-1, 0], [-1, -1, 1]])
    assert kv_ptr.tolist() == [0, 3, 3] and kv.tolist() == [0, 1, 2]
    assert q_ptr.tolist() == [0, 2, 5] and loc.tolist() == [3, 6, 14, 15, 4]
    assert pos.tolist() == [3, 4, 0, 0, 1]


def test_rope_oracle_keeps_norms_and_relative_positions():
    rng = np.random.default_rng(5)
    turns, _ = binding.rope_freqs(16, 10000.0)
    q, k = rng.standard_normal((1, 16)), rng.standard_normal((1, 16))
    for half in (False, True):
        at = lambda x, p: S.rope(x, [p], turns.tolist(), 1.0, half)[0][0]  # noqa: E731
        assert abs(at(q, 12345) @ at(k, 12300) - at(q, 45) @ at(k, 0)) < 1e-12
        np.testing.assert_allclose(S.rope(at(q, 999)[None], [999], turns.tolist(), 1.0, half, inverse=True)[0], q, atol=1e-13)


def test_logprob_oracle_against_log_softmax():
    g = torch.Generator().manual_seed(2)
    x = (torch.randn((5, 40), generator=g, dtype=torch.float64) * 3).float().double()
    x[2, 7:] = -math.inf
    inv = [1.0, 0.5, 2.0, 1.0, 3.0]
    got = S.token_logprobs(x.numpy(), np.float32(inv), [3, 0, 9, -1], [0, 1, 2, 3], 4)
    lp = torch.log_softmax(x * torch.tensor(inv, dtype=torch.float64)[:, None], dim=1)
    np.testing.assert_allclose(got["stats"][0] + got["stats"][1],
                               torch.logsumexp(x * torch.tensor(inv, dtype=torch.float64)[:, None], 1), atol=1e-12)
    np.testing.assert_allclose(got["top_logprobs"].T, lp.topk(4, dim=1).values, atol=1e-12)
    np.testing.assert_allclose(got["stats"][2], -(lp.exp() * lp.clamp(min=-1e3)).sum(1), atol=1e-12)
    assert got["logprobs"][2] == -math.inf and got["logprobs"][3] == 0.0
    np.testing.assert_allclose(got["logprobs"][:2], [lp[0, 3], lp[1, 0]], atol=1e-12)


# ---------------------------------------------------------- frequency table

def freqs(dim, base, kind, **kw):
    return binding.rope_freqs(dim, base, binding.RopeScaling(kind=kind, **kw))


def as_frequency(turns):
    return np.array([float(Fraction(int(t), 1 << 64)) * 2 * math.pi for t in turns])


@pytest.mark.parametrize("dim,base", [(2, 10000.0), (64, 10000.0), (64, 50000.0), (256, 1.5), (10, 500000.0)])
def test_freqs_plain(dim, base):
    turns, amp = pkg.rope_freqs(dim, base)
    assert amp == 1.0 and turns.shape == (dim // 2,)
    np.testing.assert_allclose(as_frequency(turns), base ** (-2.0 * np.arange(dim // 2) / dim), rtol=1e-14)


def test_freqs_scaled():
    dim, base = 64, 10000.0
    f = base ** (-2.0 * np.arange(dim // 2) / dim)
    turns, amp = freqs(dim, base, binding.ROPE_SCALE_LINEAR, factor=4.0)
    np.testing.assert_allclose(as_frequency(turns), f / 4, rtol=1e-14)
    assert amp == 1.0
    turns, amp = freqs(dim, base, binding.ROPE_SCALE_YARN, factor=40.0, original_len=4096.0, beta_fast=32.0, beta_slow=1.0)
    # 4096 f / 2 pi = 32 at i = 10.47, 1 at i = 22.5: kept below 10, divided from 23 on
    want = np.where(np.arange(32) <= 10, f, np.where(np.arange(32) >= 23, f / 40, np.nan))
    got = as_frequency(turns)
    for i in range(32):
        if np.isnan(want[i]):
            w = (i - 10) / 13
            want[i] = f[i] * (1 - w) + f[i] / 40 * w
    np.testing.assert_allclose(got, want, rtol=1e-13)
    assert amp == np.float32(0.1 * math.log(40.0) + 1)
    assert freqs(dim, base, binding.ROPE_SCALE_YARN, factor=40.0, original_len=4096.0, beta_fast=32.0, beta_slow=1.0,
                 amplitude=1.25)[1] == 1.25
    turns, amp = freqs(dim, base, binding.ROPE_SCALE_WAVELENGTH, factor=8.0, original_len=8192.0, low_turns=1.0, high_turns=4.0)
    n = 8192 * f / (2 * math.pi)
    blend = (1 - (n - 1) / 3) * f / 8 + (n - 1) / 3 * f
    np.testing.assert_allclose(as_frequency(turns), np.where(n > 4, f, np.where(n < 1, f / 8, blend)), rtol=1e-13)


def test_freqs_refusals(lib):
    buf, amp = (ctypes.c_uint64 * 128)(), ctypes.c_float()
    assert lib.mla_rope_freqs(64, 1e4, None, None, ctypes.byref(amp)) == -1
    assert lib.mla_rope_freqs(64, 1e4, None, buf, None) == -1
    for dim, base in [(0, 1e4), (3, 1e4), (258, 1e4), (-2, 1e4), (64, 1.0), (64, math.nan), (64, math.inf)]:
        assert lib.mla_rope_freqs(dim, base, None, buf, ctypes.byref(amp)) == -3
    ok = dict(factor=2.0, original_len=100.0, beta_fast=32.0, beta_slow=1.0, low_turns=1.0, high_turns=4.0)
    for bad in [dict(kind=4), dict(kind=-1), dict(kind=1, reserved=1), dict(kind=1, factor=0.5),
                dict(kind=1, factor=math.nan), dict(kind=2, original_len=0.0), dict(kind=2, beta_slow=0.0),
                dict(kind=2, beta_slow=33.0), dict(kind=3, low_turns=4.0), dict(kind=3, low_turns=0.0),
                dict(kind=1, amplitude=-1.0), dict(kind=1, amplitude=math.nan)]:
        s = binding.RopeScaling(**{**ok, **bad})
        assert lib.mla_rope_freqs(64, 1e4, ctypes.byref(s), buf, ctypes.byref(amp)) == -3, bad
    with pytest.raises(binding.MtvError):
        pkg.rope_freqs(7, 1e4)


# ----------------------------------------------------------------- refusals

def test_page_table_update_refusals(lib):
    def call(lens=FAKE, rows=4, page=16, table=FAKE, stride=8, per=8, held=FAKE, free=FAKE, cap=32, num=FAKE):
        return lib.mla_page_table_update(lens, rows, page, table, stride, per, held, free, cap, num, None, None)
    for kw in [dict(rows=-1), dict(page=0), dict(per=-1), dict(stride=7), dict(cap=-1), dict(cap=1 << 31)]:
        assert call(**kw) == -3, kw
    assert call(rows=8193) == -2
    assert call(rows=8192, per=1 << 18, stride=1 << 18) == -2  # 2^31 entries
    for kw in [dict(lens=None), dict(table=None), dict(held=None), dict(free=None), dict(num=None)]:
        assert call(**kw) == -1, kw
    assert call(rows=0) == 0


def test_slot_map_build_refusals(lib):
    def call(table=FAKE, stride=8, rows=4, per=8, pages=32, page=16, prefix=FAKE, bs=2, kvp=FAKE, kvcap=64, qop=FAKE, qcap=8):
        return lib.mla_slot_map_build(table, stride, rows, per, pages, page, None, prefix, None, None, bs, kvp, FAKE,
                                      kvcap, qop, FAKE, FAKE, qcap, None, None)
    for kw in [dict(bs=-1), dict(page=0), dict(stride=-1), dict(stride=7), dict(rows=-1), dict(per=-1), dict(pages=-1),
               dict(kvcap=-1), dict(qcap=-1)]:
        assert call(**kw) == -3, kw
    assert call(bs=8193) == -2
    for kw in [dict(table=None), dict(prefix=None), dict(kvp=None), dict(qop=None)]:
        assert call(**kw) == -1, kw


def test_rope_write_refusals(lib):
    def call(turns=FAKE, dim=64, amp=1.0, layout=0, inverse=0, pos=FAKE, tokens=4, dtype=0, q_in=FAKE, q_out=FAKE, heads=64,
             k=FAKE, c=FAKE, loc=FAKE, pool=FAKE, slots=8):
        return lib.mla_rope_write(turns, dim, amp, layout, inverse, pos, tokens, None, dtype, q_in, 64, 64, q_out, 64, 64,
                                  heads, k, 64, c, 512, loc, pool, slots, None, None)
    for kw in [dict(dim=0), dict(dim=3), dict(dim=258), dict(amp=math.nan), dict(amp=math.inf), dict(layout=2),
               dict(inverse=2), dict(tokens=-1), dict(heads=-1), dict(slots=-1), dict(dtype=3), dict(dtype=-1),
               dict(pool=ctypes.c_void_p(0x100008))]:
        assert call(**kw) == -3, kw
    assert call(dim=32) == -2 and call(tokens=1 << 31) == -2
    for kw in [dict(q_in=None), dict(q_out=None), dict(turns=None), dict(pos=None), dict(k=None), dict(c=None), dict(loc=None)]:
        assert call(**kw) == -1, kw
    assert call(tokens=0) == 0
    assert call(q_in=None, q_out=None, pool=None) == 0 and call(heads=0, pool=None) == 0


def test_token_logprobs_refusals(lib):
    def call(x=FAKE, dtype=0, rows=4, vocab=100, stride=100, tokens=FAKE, trows=None, n=4, lp=FAKE, stats=FAKE, k=2,
             tt=FAKE, tl=FAKE):
        return lib.mla_token_logprobs(x, dtype, rows, vocab, stride, None, tokens, trows, n, lp, stats, k, tt, tl, None, None)
    for kw in [dict(dtype=3), dict(dtype=-1), dict(rows=-1), dict(vocab=0), dict(vocab=(1 << 20) + 1), dict(stride=-1),
               dict(n=-1), dict(n=5), dict(k=-1), dict(k=33), dict(x=ctypes.c_void_p(0x100001))]:
        assert call(**kw) == -3, kw
    assert call(rows=1 << 31) == -2
    for kw in [dict(x=None), dict(stats=None), dict(tokens=None), dict(lp=None), dict(tt=None), dict(tl=None)]:
        assert call(**kw) == -1, kw
    assert call(rows=0, n=0) == 0


def test_binding_refuses_host_tensors_types_and_shapes():
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    i64 = lambda *s: torch.zeros(s, dtype=torch.int64)  # noqa: E731
    f32 = lambda *s: torch.zeros(s)  # noqa: E731
    with pytest.raises(TypeError, match="CUDA"):
        pkg.page_table_update(i32(2), 16, i32(2, 4), i32(2), i32(8), i32(1))
    with pytest.raises(ValueError, match="dense rows"):
        pkg.page_table_update(i32(2), 16, i32(4, 2).t(), i32(2), i32(8), i32(1))
    with pytest.raises(ValueError, match="one element"):
        pkg.page_table_update(i32(2), 16, i32(2, 4), i32(2), i32(8), i32(2))
    with pytest.raises(ValueError, match="num_pages"):
        pkg.slot_map_build(i32(2, 4), i32(2), i32(2), 16, i32(3), i64(8), i64(3), i64(4))
    with pytest.raises(ValueError, match="more requests"):
        pkg.slot_map_build(i32(2, 4), i32(3), i32(3), 16, i32(4), i64(8), i64(4), i64(4), num_pages=8)
    with pytest.raises(TypeError, match="CUDA"):
        pkg.slot_map_build(i32(2, 4), i32(2), i32(2), 16, i32(3), i64(8), i64(3), i64(4), num_pages=8)
    with pytest.raises(ValueError, match="neither"):
        pkg.rope_write(i64(32), i64(4))
    with pytest.raises(ValueError, match="go together"):
        pkg.rope_write(i64(32), i64(4), q_in=f32(4, 2, 64))
    with pytest.raises(TypeError, match="CUDA"):
        pkg.rope_write(i64(32), i64(4), q_in=f32(4, 2, 64), q_out=f32(4, 2, 64))
    with pytest.raises(TypeError, match="not one of"):
        pkg.rope_write(i64(32), i64(4), q_in=f32(4, 2, 64).double(), q_out=f32(4, 2, 64))
    with pytest.raises(TypeError, match="must be one of"):
        pkg.token_logprobs(f32(2, 9).double(), f32(3, 2))
    with pytest.raises(ValueError, match="dense rows"):
        pkg.token_logprobs(f32(9, 2).t(), f32(3, 2))
    with pytest.raises(ValueError, match="go together"):
        pkg.token_logprobs(f32(2, 9), f32(3, 2), tokens=i32(2))
    with pytest.raises(TypeError, match="CUDA"):
        pkg.token_logprobs(f32(2, 9), f32(3, 2))


def test_binding_refuses_log_probability_outputs_in_another_order():
    logits, f32 = torch.zeros((5, 9)), lambda *s: torch.zeros(s)  # noqa: E731
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError, match=r"stats must be \[3, rows\]"):
        pkg.token_logprobs(logits, f32(5, 3))
    with pytest.raises(ValueError, match=r"top_logprobs must be \[2, rows\]"):
        pkg.token_logprobs(logits, f32(3, 5), top_tokens=i32(2, 5), top_logprobs=f32(5, 2))
    for stats, top in [(f32(3, 5), f32(2, 5)), (f32(15), f32(10))]:  # up to the device, which is the host here
        with pytest.raises(TypeError, match="CUDA"):
            pkg.token_logprobs(logits, stats, top_tokens=i32(2, 5), top_logprobs=top)
