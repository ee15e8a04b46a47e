"""Appending to 8-bit pages that come with scales from elsewhere, which are not
powers of two: bit for bit against the plain form, with values on the middle
between two e4m3 ones, where a quotient's last bit decides."""
import pytest
import torch

import decode_attention_static_gb300 as da
import test_paged_append_gpu as A

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    da.build_library()
    da.load_library()


PLACES = [([1, 1, 1, 1], [5, 15, 17, 250]), ([30, 3, 16, 1], [3, 30, 17, 9])]


def middles(shape, scale, gen):
    """scale times the middle of two neighbouring e4m3 values, in [2^-3, 2^6)."""
    odd = 2 * torch.randint(8, 16, shape, generator=gen) + 1
    sign = 2 * torch.randint(0, 2, shape, generator=gen) - 1
    return sign * odd * torch.exp2(torch.randint(-7, 2, shape, generator=gen).float()) * scale


@pytest.mark.parametrize("counts,positions", PLACES, ids=["tokens", "prompts"])
@pytest.mark.parametrize("page,D", [(16, 64), (16, 128), (64, 128), (256, 128)])
@pytest.mark.parametrize("times", [7, 13, 15, 51])
def test_quotients_are_rounded_once(times, page, D, counts, positions):
    """x / scale is exact here and lies in the middle; x times the reciprocal,
    rounded, would leave it."""
    scale, gen = times * 2.0 ** -6, torch.Generator().manual_seed(times)
    inp = A.Inputs(counts, positions, 2, 2, D, "f16", page, True, rope=False, with_q=False, seed=page)
    inp.ks[:], inp.vs[:] = scale, scale
    for name in ("k_new", "v_new"):
        x = middles(getattr(inp, name).shape, scale, gen)
        setattr(inp, name, x.half())
        assert torch.equal(getattr(inp, name).float(), x)
    A.check(inp, f"scale {scale}")


@pytest.mark.parametrize("counts,positions", PLACES, ids=["tokens", "prompts"])
def test_any_scale_grows_to_a_power_of_two(counts, positions):
    inp = A.Inputs(counts, positions, 4, 2, 128, "bf16", 32, True, seed=3)
    gen = torch.Generator().manual_seed(4)
    inp.ks, inp.vs = (torch.rand(inp.ks.shape, generator=gen) * 2.0 ** -6 + 2.0 ** -12 for _ in range(2))
    A.check(inp, "scales grow and stay")


@pytest.mark.parametrize("counts,positions", PLACES, ids=["tokens", "prompts"])
@pytest.mark.parametrize("scale", [2.0 ** 126, 2.0 ** 127, 1.5 * 2.0 ** 127])
def test_scales_at_the_end_of_the_range(scale, counts, positions):
    """Scales whose reciprocal is no normal number."""
    inp = A.Inputs(counts, positions, 2, 2, 64, "bf16", 16, True, rope=False, with_q=False, seed=6)
    inp.ks[:], inp.vs[:] = scale, scale
    inp.k_new, inp.v_new = ((x.float() * 1.2 * 2.0 ** 125).bfloat16() for x in (inp.k_new, inp.v_new))
    assert inp.k_new.isfinite().all() and inp.v_new.isfinite().all()
    A.check(inp, f"scale {scale}")
