"""Where the sizes that the attention entry points take end; host checks alone."""
import pytest

from test_attention_abi import INVALID, WORKSPACE, _tree, lib  # noqa: F401


@pytest.mark.parametrize("width,ps", [(2 ** 27 - 1, 16), (2 ** 31 - 1, 1), (2 ** 23 - 15, 256), (1, 2 ** 31 - 1)])
def test_positions_close_to_31_bits(lib, width, ps):  # noqa: F811
    assert _tree(lib, width=width, ps=ps, bytes=8) == INVALID


@pytest.mark.parametrize("width,ps", [(2 ** 27 - 256, 16), (2 ** 31 - 4096, 1), (2 ** 23 - 16, 256)])
def test_the_largest_page_tables(lib, width, ps):  # noqa: F811
    assert _tree(lib, width=width, ps=ps, bytes=8) == WORKSPACE     # past the checks of sizes
