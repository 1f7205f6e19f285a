"""The layer's calls without a GPU, beyond test_layer_ops_host.py."""
import pytest

from paged_mla_speculative_tree_gb300 import binding, build
from tests.test_layer_ops_host import prefill, product


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def test_test_count_of_waits_is_part_of_the_type(lib):
    for n in (1, 255):
        assert product(lib, dtype=1 + 256 * n, tokens=0) == 0 and prefill(lib, dtype=1 + 256 * n, bs=0) == 0
        assert product(lib, dtype=2 + 256 * n) == -3 and prefill(lib, dtype=2 + 256 * n) == -3
    for dtype in (256 * 256, -256, (1 << 31) - 256):
        assert product(lib, dtype=dtype, tokens=0) == -3 and prefill(lib, dtype=dtype, bs=0) == -3
