"""Sizes of the paged and window attention that no C int or packed word holds
are refused, on the CPU."""
import pytest
import torch

import decode_attention_static_gb300 as da
import paged_reference as R
from decode_attention_static_gb300 import build as da_build


@pytest.fixture(scope="module", autouse=True)
def _library():
    da_build.build_library()


def calls(**kw):
    """The three attentions on tensors that are refused later, for being on the host."""
    q, n = torch.zeros(2, 4, 64, dtype=torch.float16), torch.zeros(2, dtype=torch.int32)
    k, table, s = torch.zeros(6, 2, 16, 64, dtype=torch.float16), torch.zeros(2, 3, dtype=torch.int32), torch.ones(6, 2)
    window = dict(dict(window=4), **kw)
    yield lambda: da.decode_attn_paged_fwd(q, k, k, table, n, **kw)
    yield lambda: da.decode_attn_paged_q8_fwd(q, k.to(R.E4M3), k.to(R.E4M3), s, s, table, n, **kw)
    yield lambda: da.decode_attn_window_fwd(q, k[:2], k[:2], n, **window)


@pytest.mark.parametrize("value", [1 << 31, (1 << 32) + 1, 1 << 40, -(1 << 31) - 1, -(1 << 32) + 5])
@pytest.mark.parametrize("name", ["window", "sinks"])
def test_windows_past_32_bits_are_refused(name, value):
    """2^32 + 1 is not a window of one row, and 2^40 not one of none."""
    for call in calls(**{"window": 8, name: value}):
        with pytest.raises(ValueError, match=f"{name} = .* 32 bits"):
            call()


@pytest.mark.parametrize("value", [(1 << 31) - 1, 1, torch.tensor(7)])
def test_windows_of_32_bits_are_not(value):
    for call in calls(window=value, sinks=value):
        with pytest.raises(ValueError, match="CUDA"):
            call()
