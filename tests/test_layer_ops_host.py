"""Operators of the attention layer without a GPU: the oracle's pins, the split
rule, and every refusal of the C entries and of the binding."""
import ctypes
import math

import pytest
import torch

import paged_mla_speculative_tree_gb300 as pkg
from oracle import layer_ops as L
from paged_mla_speculative_tree_gb300 import binding, build

FAKE = ctypes.c_void_p(0x100000)  # never dereferenced: checks fail first, or nothing is left to do


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


# ------------------------------------------------------------------- oracle

def test_prefill_oracle_against_attention_with_a_mask():
    g = torch.Generator().manual_seed(3)
    rnd = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    new, length = [3, 5, 2], [7, 5, 1]
    q, kn, kr, v = rnd(10, 2, 192), rnd(13, 2, 128), rnd(13, 64), rnd(13, 2, 128)
    got = L.prefill(q, kn, kr, v, [0, 3, 8, 10], [0, 7, 12, 13], 0.1)
    q0 = k0 = 0
    for n, m in zip(new, length):
        k = torch.cat([kn[k0:k0 + m], kr[k0:k0 + m, None].expand(m, 2, 64)], dim=2)
        mask = torch.ones(n, m, dtype=torch.bool).tril(m - n)
        want = torch.nn.functional.scaled_dot_product_attention(
            q[q0:q0 + n].transpose(0, 1), k.transpose(0, 1), v[k0:k0 + m].transpose(0, 1), attn_mask=mask, scale=0.1)
        some = mask.any(1)
        torch.testing.assert_close(got["out"][q0:q0 + n][some], want.transpose(0, 1)[some], rtol=1e-12, atol=1e-12)
        assert (got["out"][q0:q0 + n][~some] == 0).all() and (got["lse"][q0:q0 + n][~some] == -math.inf).all()
        q0, k0 = q0 + n, k0 + m
    assert int((got["lse"] == -math.inf).sum()) == 2  # the first query of the request with fewer keys than queries


def test_prefill_oracle_closed_form():
    q, kn = torch.zeros(2, 1, 192), torch.zeros(3, 1, 128)
    kr = torch.zeros(3, 64)
    q[:, 0, 128], kr[:, 0] = 2.0, torch.tensor([0.0, math.log(3) / 2, 5.0])
    v = torch.zeros(3, 1, 128)
    v[:, 0, 0] = torch.tensor([1.0, 9.0, 100.0])
    got = L.prefill(q, kn, kr, v, [0, 2], [0, 3], 1.0)  # the first query sees two keys of weights 1 : 3
    assert abs(got["out"][0, 0, 0] - 7.0) < 1e-6 and abs(got["lse"][0, 0] - math.log(4)) < 1e-6


def test_absorbed_and_expanded_oracles_agree():
    """Queries taken to the latent space score as they do against expanded keys."""
    g = torch.Generator().manual_seed(4)
    rnd = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    q, up, c = rnd(3, 2, 128), rnd(2, 128, 512), rnd(5, 512)
    absorbed = torch.einsum("thc,jc->thj", L.head_product(q, up)[0], c)
    keys = L.head_product(c[:, None].expand(5, 2, 512), up.transpose(1, 2))[0]
    torch.testing.assert_close(torch.einsum("thd,jhd->thj", q, keys), absorbed, rtol=1e-10, atol=1e-9)


def test_norm_oracle():
    x = torch.tensor([[3.0, 4.0], [0.0, 0.0]])
    got = L.norm(x, torch.tensor([1.0, 2.0]), 0.5)
    torch.testing.assert_close(got, torch.tensor([[3.0, 8.0], [0.0, 0.0]], dtype=torch.float64) / math.sqrt(13.0))


# --------------------------------------------------------------- split rule

def test_prefill_workspace_rule():
    one = pkg.prefill_workspace(152, 1, 8192, 8192, 8192, 64)
    assert one == (1, 0)  # queries enough for every SM: nothing to join
    for heads, rows, keys in ((8, 60, 32828), (4, 1, 100000), (64, 1, 4096), (1, 128, 1 << 20)):
        nsplit, size = pkg.prefill_workspace(152, 1, rows, keys, rows, heads)
        assert 1 <= nsplit <= 64
        assert size == (nsplit * rows * heads * 129 * 4 if nsplit > 1 else 0)
    assert pkg.prefill_workspace(152, 1, 1, 64, 1, 1) == (1, 0)  # no keys worth a split
    assert pkg.prefill_workspace(152, 0, 0, 0, 0, 0) == (1, 0)


def test_prefill_workspace_refusals(lib):
    n, size = ctypes.c_int(), ctypes.c_uint64()
    call = lambda *a: lib.mla_prefill_workspace(*a, ctypes.byref(n), ctypes.byref(size))  # noqa: E731
    assert call(0, 1, 8, 8, 8, 8) == -3
    assert call(152, -1, 8, 8, 8, 8) == -3
    assert call(152, 65536, 8, 8, 8, 8) == -3
    assert call(152, 1, -8, 8, 8, 8) == -3
    assert call(152, 1, 8, 1 << 31, 8, 8) == -3
    assert call(152, 1, 8, 8, 1 << 31, 8) == -3
    assert call(152, 1, 8, 8, 8, 65536) == -3
    assert lib.mla_prefill_workspace(152, 1, 8, 8, 8, 8, None, ctypes.byref(size)) == -1


# ------------------------------------------------------- refusals of the ABI

PRODUCT = dict(x=FAKE, x_tok=1024, x_head=128, w=FAKE, w_head=65536, w_k=512, w_n=1, out=FAKE, out_tok=36864, out_head=576,
               tokens=4, heads=8, k=128, n=512, dtype=0, err=None)


def product(lib, **kw):
    return lib.mla_head_product(*{**PRODUCT, **kw}.values(), None)


def test_head_product_refusals(lib):
    for kw in (dict(tokens=-1), dict(tokens=1 << 31), dict(heads=-1), dict(heads=65536), dict(k=0), dict(k=1025), dict(n=0),
               dict(n=1025), dict(dtype=2), dict(dtype=-1), dict(x=ctypes.c_void_p(0x100001))):
        assert product(lib, **kw) == -3, kw
    for name in ("x", "w", "out"):
        assert product(lib, **{name: None}) == -1
    assert product(lib, tokens=0, x=None, out=None) == 0
    assert product(lib, heads=0, w=None) == 0


PREFILL = dict(q=FAKE, q_tok=1536, q_head=192, kn=FAKE, k_tok=2048, k_head=256, kr=FAKE, kr_tok=576, v=FAKE, v_tok=2048,
               v_head=256, qo=FAKE, kv=FAKE, bs=1, max_q=8, max_kv=64, num_q=8, num_kv=64, heads=8, dtype=0, scale=1.0,
               causal=1, out=FAKE, o_tok=1024, o_head=128, lse=FAKE, nsplit=1, ws=None, ws_bytes=0, err=None)


def prefill(lib, **kw):
    return lib.mla_prefill_run(*{**PREFILL, **kw}.values(), None)


def test_prefill_refusals(lib):
    for kw in (dict(bs=-1), dict(bs=65536), dict(max_q=-1), dict(max_kv=-1), dict(max_q=1 << 31), dict(max_kv=1 << 31),
               dict(num_q=-1), dict(num_kv=1 << 31), dict(heads=65536), dict(dtype=2), dict(scale=0.0), dict(scale=-1.0),
               dict(scale=math.inf), dict(scale=math.nan), dict(scale=3e38), dict(causal=2), dict(nsplit=0), dict(nsplit=65)):
        assert prefill(lib, **kw) == -3, kw
    for name in ("q_tok", "q_head", "k_tok", "k_head", "kr_tok", "v_tok", "v_head", "o_tok", "o_head"):
        assert prefill(lib, **{name: PREFILL[name] + 4}) == -3, name
    for name in ("q", "kn", "kr", "v", "out"):
        assert prefill(lib, **{name: ctypes.c_void_p(0x100008)}) == -3, name
    for name in ("q", "kn", "kr", "v", "qo", "kv", "out"):
        assert prefill(lib, **{name: None}) == -1, name
    need = 2 * 8 * 8 * 129 * 4
    assert prefill(lib, nsplit=2) == -1
    assert prefill(lib, nsplit=2, ws=FAKE, ws_bytes=need - 1) == -4
    assert prefill(lib, nsplit=2, ws=ctypes.c_void_p(0x100010), ws_bytes=need) == -5
    for kw in (dict(bs=0, qo=None, kv=None), dict(max_q=0), dict(num_q=0, q=None, out=None), dict(heads=0)):
        assert prefill(lib, **kw) == 0, kw


NORM = dict(turns=FAKE, rope_dim=64, amplitude=1.0, layout=0, positions=FAKE, tokens=4, valid=None, dtype=0, eps=1e-6, q=FAKE,
            q_tok=1536, q_head=192, heads=8, nope=128, qw=FAKE, qn=FAKE, qn_tok=1024, qn_head=128, qr=FAKE, qr_tok=512,
            qr_head=64, c=FAKE, c_tok=576, cw=FAKE, k=FAKE, k_tok=576, loc=FAKE, pool=FAKE, slots=64, err=None)


def norm(lib, **kw):
    return lib.mla_norm_rope_write(*{**NORM, **kw}.values(), None)


def test_norm_rope_write_refusals(lib):
    for kw in (dict(rope_dim=0), dict(rope_dim=63), dict(rope_dim=258), dict(amplitude=math.inf), dict(layout=2),
               dict(tokens=-1), dict(dtype=3), dict(eps=-1e-6), dict(eps=math.nan), dict(heads=-1), dict(slots=-1),
               dict(nope=-1), dict(nope=961), dict(qn=None), dict(qw=None), dict(nope=0), dict(q=None, qr=None),
               dict(q=ctypes.c_void_p(0x100001)), dict(cw=ctypes.c_void_p(0x100001)), dict(pool=ctypes.c_void_p(0x100008)),
               dict(dtype=2, qr=ctypes.c_void_p(0x100002))):
        assert norm(lib, **kw) == -3, kw
    assert norm(lib, tokens=1 << 31) == -2
    assert norm(lib, rope_dim=32) == -2  # the pool's key part is 64 long
    for kw in (dict(q=None), dict(qr=None), dict(turns=None), dict(positions=None), dict(c=None), dict(k=None), dict(loc=None)):
        assert norm(lib, **kw) == -1, kw
    assert norm(lib, tokens=0, turns=None, positions=None) == 0
    assert norm(lib, heads=0, pool=None, turns=None) == 0


# --------------------------------------------------- refusals of the binding

def test_binding_wants_cuda_tensors():
    bf, z = torch.bfloat16, torch.zeros
    with pytest.raises(TypeError):
        pkg.head_product(z((2, 3, 8), dtype=bf), z((3, 8, 4), dtype=bf), z((2, 3, 4), dtype=bf))
    with pytest.raises(TypeError):
        pkg.head_product(z((2, 3, 8)), z((3, 8, 4)), z((2, 3, 4)))  # fp32 is not taken
    with pytest.raises(ValueError):
        pkg.head_product(z((3, 8), dtype=bf), z((3, 8, 4), dtype=bf), z((2, 3, 4), dtype=bf))
    ptr = lambda t: torch.zeros(2, dtype=t)  # noqa: E731
    with pytest.raises(TypeError):
        pkg.prefill_run(z((2, 3, 192), dtype=bf), z((2, 3, 128), dtype=bf), z((2, 64), dtype=bf), z((2, 3, 128), dtype=bf),
                        ptr(torch.int64), ptr(torch.int32), 2, 2, 1.0, z((2, 3, 128), dtype=bf))
    with pytest.raises(TypeError):
        pkg.prefill_run(z((2, 3, 192)), z((2, 3, 128)), z((2, 64)), z((2, 3, 128)), ptr(torch.int64), ptr(torch.int32), 2, 2,
                        1.0, z((2, 3, 128)))
    turns, pos = torch.zeros(32, dtype=torch.int64), torch.zeros(2, dtype=torch.int64)
    with pytest.raises(ValueError):
        pkg.norm_rope_write(turns, pos, 1e-6)
    with pytest.raises(ValueError):
        pkg.norm_rope_write(turns, pos, 1e-6, q_in=z((2, 3, 192), dtype=bf))
    with pytest.raises(TypeError):
        pkg.norm_rope_write(turns, pos, 1e-6, q_in=z((2, 3, 192), dtype=bf), q_rope=z((2, 3, 64), dtype=bf))
    with pytest.raises(TypeError):
        pkg.norm_rope_write(turns, pos, 1e-6, q_in=z((2, 3, 192), dtype=torch.float64), q_rope=z((2, 3, 64)))


def test_binding_refuses_what_is_no_tensor(lib):
    bf, z = torch.bfloat16, torch.zeros
    x, w, out = z((2, 3, 8), dtype=bf), z((3, 8, 4), dtype=bf), z((2, 3, 4), dtype=bf)
    for args in ((None, w, out), (x, None, out), (x, w, None), (x.tolist(), w, out), (x, w, out.float().numpy())):
        with pytest.raises(TypeError):
            pkg.head_product(*args)
    with pytest.raises(TypeError):
        pkg.head_product(x.to("meta"), w.to("meta"), out.to("meta"))
    turns, pos = torch.zeros(32, dtype=torch.int64), torch.zeros(2, dtype=torch.int64)
    with pytest.raises(TypeError):
        pkg.norm_rope_write(None, pos, 1e-6, q_in=x, q_rope=x)
    for fn, count in (("head_product", 5), ("prefill_run", 16), ("norm_rope_write", 17)):
        for n in (0, count - 1, count + 1):
            with pytest.raises(TypeError):
                getattr(binding._extension(), fn)(*[None] * n)


def test_extension_calls_the_library_that_ctypes_loaded(lib):
    binding._extension()
    with open("/proc/self/maps") as f:
        inodes = {line.split()[4] for line in f if "libmla_tree_verify" in line}
    assert len(inodes) == 1


def test_prefill_workspace_splits_a_part_filled_wave():
    def rule(bs, new, keys, heads):
        nsplit, size = pkg.prefill_workspace(152, bs, new, keys, bs * new, heads)
        n, last = nsplit % 256, nsplit // 256
        assert size == (n * 129 * 4 * (last * 256 if last else bs * new * heads) if n > 1 else 0)
        return n, last

    assert rule(2, 1000, 6760, 64) == (2, 56)       # 512 blocks, 3 waves and 56
    assert rule(1, 256, 8448, 160) == (16, 8)       # as many as the keys are worth
    assert rule(1, 2048, 2048, 64) == (1, 0)        # the heads' last blocks are short
    assert rule(1, 256, 1280, 160) == (1, 0)        # short keys
    assert rule(1, 256, 8448, 152) == (1, 0)        # a whole wave
    assert rule(1, 256, 8448, 152 + 76) == (2, 76)  # half a wave more
    assert rule(1, 256, 8448, 152 + 77) == (1, 0)
    assert rule(8, 256, 8448, 153) == (1, 0)        # many waves
    assert rule(1, 256, 100, 160) == (1, 0)         # fewer keys than queries


def test_prefill_refuses_split_counts(lib):
    need = 2 * 256 * 129 * 4
    assert prefill(lib, nsplit=2 + 256, ws=FAKE, ws_bytes=need - 1) == -4
    assert prefill(lib, nsplit=2 + 256) == -1
    for nsplit in (256, 65 + 256, 255, -255, -(1 << 31)):
        assert prefill(lib, nsplit=nsplit, ws=FAKE, ws_bytes=1 << 40) == -3, nsplit
    assert prefill(lib, nsplit=64 + 256 * 100, ws=FAKE, ws_bytes=64 * 8 * 256 * 129 * 4 - 1) == -4  # eight blocks are there


def test_prefill_workspace_prefers_smaller_blocks_to_two_parts():
    nsplit = lambda new, keys, heads: pkg.prefill_workspace(152, 1, new, keys, new, heads)[0]  # noqa: E731
    assert nsplit(256, 3256, 64) == 1    # blocks of 128 rows instead
    assert nsplit(128, 3256, 64) == 2    # no smaller blocks to take
    assert nsplit(256, 8192, 64) == 2    # long keys
    assert nsplit(256, 3256, 48) == 3
