"""Calls of the tree attention that its other tests do not make: an output over a
part of the query, and batches of more sequences than one pass of the division
looks at."""
import pytest
import torch

import decode_attention_static_gb300 as da
import paged_reference as R
from test_tree_attention_gpu import BOTH, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    da.build_library()
    da.load_library()


@BOTH
def test_output_over_a_part_of_the_query(eight):
    """CTAs read q while others write out: refused, and nothing is written."""
    case = Case([100, 40], [20, 12], 8, 2, 64, "f16", 16, eight).cuda()
    want = case.check()
    buffer = torch.zeros(32 * 3, 8, 64, dtype=torch.float16, device="cuda")
    buffer[32:64] = case.q
    case.q, keep = buffer[32:64], buffer.clone()
    for first in (31, 1, 63, 32, 33):
        with pytest.raises(da.DecodeAttnError) as e:
            case.call(out=buffer[first:first + 32])
        assert e.value.status == -2 and torch.equal(R.bits(buffer), R.bits(keep)), first
    for first in (0, 64):  # (right beside it is fine)
        assert torch.equal(R.bits(case.call(out=buffer[first:first + 32])), R.bits(want))


@BOTH
@pytest.mark.parametrize("idle", [0, 7])
@pytest.mark.parametrize("B", [33, 385, 600, 1500])
def test_many_sequences(B, idle, eight):
    """Batches around and past the numbers of threads that divide them; with idle, seven of eight own no token."""
    lens = [1 + 37 * b % 90 for b in range(B)]
    news = [0 if idle and b % 8 else 1 + b % 2 if lens[b] > 1 else 1 for b in range(B)]
    Case(lens, news, 2, 1, 64, "bf16", 16, eight, kind="chain", seed=B).cuda().check()


@BOTH
def test_one_long_sequence_among_idle_ones(eight):
    """Its unit is divided, wherever in the batch it stands."""
    for B, at in ((600, 0), (600, 599), (1500, 700)):
        lens, news = [5] * B, [0] * B
        lens[at], news[at] = 9000, 9
        Case(lens, news, 4, 1, 128, "f16", 64, eight, kind="chain", seed=at).cuda().check(f"{at} of {B}")
