"""CPU checks of decode behind very long shared prefixes: what their parts ask of the workspace."""
import pytest

import paged_kv_block_gb300 as pkb
from paged_kv_block_gb300 import build as B
from tests.test_shared_prefix_host import BASE


@pytest.fixture(scope="module")
def lib():
    B.build()
    return pkb.lib()


def test_workspace_of_long_prefixes(lib):
    """Room for parts of at most 2^14 tiles of 128 keys, or a refusal."""
    size = lambda **kw: pkb.paged_decode_shared_workspace_size(  # noqa: E731
        pkb.DecodeParams(**{**BASE, **kw}), 1)
    part = 1 << 21
    assert size(max_seq_len=512) == size(max_seq_len=part) < size(max_seq_len=part + 1)
    tiles = lambda n: size(max_seq_len=n, batch=4096) - size(max_seq_len=n, batch=4)  # noqa: E731
    assert tiles(8 * part) >= tiles(part) + 7 * 2 * 4096 // 64 * 256 * 512
    assert size(max_seq_len=2 ** 31 - 1, batch=1 << 24, num_qo_heads=128) == 0
