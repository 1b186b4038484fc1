"""The ``appended`` array of the rotated append and of chunk attention: refused where it is not what the calls take (no GPU
needed)."""
import ctypes

import pytest
import torch

from tests.test_abi_host import ts  # noqa: F401
from tests.test_prompt_host import B, SHAPE, _append, _append_block, _chunk, _code, _i


@pytest.mark.parametrize("bad", [torch.zeros(B, dtype=torch.int64), torch.zeros(B + 1, dtype=torch.int32), torch.zeros(2 * B, dtype=torch.int32)[::2]])
def test_refused_tensors(ts, bad):  # noqa: F811
    assert _code(ts, lambda: _chunk(ts, appended=bad)) == SHAPE
    assert _code(ts, _append(ts, appended=bad)) == SHAPE
    assert _chunk(ts, appended=_i(B)).appended and _chunk(ts).appended is None


@pytest.mark.parametrize("other", ["prefix_len", "cu_len", "status", "new_prefix_len", "q_out"])
def test_refused_overlaps(ts, other):  # noqa: F811
    assert _append_block(ts, appended=other) == SHAPE


def test_blocks_are_as_the_header_has_them(ts):  # noqa: F811
    assert ts.ChunkParams.appended.offset == ctypes.sizeof(ts.ChunkParams) - 8 == 136
    assert ts.AppendParams.appended.offset == ctypes.sizeof(ts.AppendParams) - 8 == 184
