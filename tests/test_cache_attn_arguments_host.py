"""Sizes of the paged and window attention that no C int or packed word holds
are refused, on the CPU."""
import pytest
import torch

import decode_attention_static_gb300 as da
import paged_reference as R
import test_paged_host as P
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


@pytest.mark.parametrize("fn", P.PAGED + ["decode_attn_window_fwd"])
def test_batches_and_heads_past_16_bits_are_refused(fn):
    """A sequence number and a head travel in 16 bits each."""
    lib, rows = da.load_library(), {"capacity": 64} if "window" in fn else {"max_pages": 4}
    assert P.call(lib, fn, B=65536, H=1, Hkv=1, **rows) == P.SHAPE
    assert P.call(lib, fn, B=1, H=65536, Hkv=65536, **rows) == P.SHAPE
    assert P.call(lib, fn, B=65535, H=1, Hkv=1, q=None, **rows) == P.NULL
    assert P.call(lib, fn, B=1, H=65535, Hkv=65535, q=None, **rows) == P.NULL
