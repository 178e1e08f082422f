"""The largest tables of 8-bit decode and of decode over a shared prefix: refusals and
sizes on the host, no GPU. Positions and their tiles are 32-bit in the kernels."""
import pytest

import paged_kv_cache_305_gb300 as pa
from paged_kv_cache_305_gb300 import build as pbuild
from test_fp8_oracle import _decode, _prefix

MOST = 2 ** 31 - 4096  # tokens of a table


@pytest.fixture(scope="module")
def lib():
    pbuild.build()
    return pa.load_library()


@pytest.mark.parametrize("call", [_decode, _prefix])
def test_tables_next_to_2_to_the_31_are_refused(lib, call):
    one = dict(S=1, Hq=1, Hkv=1, d=64, B=64, out=None)
    if call is _prefix:
        one.update(NG=1, NB=1000, mp=32, mg=1)
    for tokens in (MOST + 64, 2 ** 31 - 64):
        assert call(lib, MB=tokens // 64, **one) == -2
        assert "overflows" in pa.last_error()
    assert call(lib, MB=MOST // 64, **one) == -1  # accepted so far: the next check finds no output
    assert "NULL" in pa.last_error()


def test_workspaces_of_the_largest_tables(lib):
    f8, fp = pa.decode_fp8_workspace_bytes, pa.decode_shared_prefix_workspace_bytes
    assert 0 < f8(1, 1, 1, 64, MOST // 64, 64) < 2 ** 20
    assert f8(1, 1, 1, 64, MOST // 64 + 1, 64) == 0
    # two sequences behind a prefix of the whole table, cut into pieces of up to 8192 tokens:
    # 64 floats, their reference and sum for each row and piece, and those of the cuts
    for prefix in (2 ** 30, MOST - 64, MOST, 2 ** 31 - 1):
        n, chunks = fp(2, 1, 1, 1, 64, MOST // 64, 64, prefix, 2), -(-min(prefix, MOST) // 8192)
        assert 0 <= n - 2 * chunks * 66 * 4 < 2 ** 20, prefix
    assert fp(2, 1, 1, 1, 64, MOST // 64 + 1, 64, 64, 2) == 0
