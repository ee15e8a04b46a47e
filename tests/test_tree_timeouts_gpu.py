"""A copy of the tree attention that never comes, at any place of a long share: in
the first round of the ring, at its end and behind it, where the producer itself
waits for a slot that is not released. Every wait is bounded: rows become NaN,
the error bit is set, and the context and (zero-filled) the workspace serve on."""
import pytest
import torch

import decode_attention_static_gb300 as da
import paged_reference as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    da.build_library()
    da.load_library()


# sequences, their rows, drafts, query heads of a KV head, KV heads, head_dim
SHAPES = {
    "few rows, parts": (1, 16000, 3, 2, 16, 128),
    "256 rows, parts": (1, 16000, 64, 4, 16, 64),
    "more units than CTAs": (48, 700, 5, 4, 16, 128),
}


@pytest.mark.parametrize("eight", [False, True], ids=["16bit", "e4m3"])
@pytest.mark.parametrize("slot", [1, 7, 13])
@pytest.mark.parametrize("shape", SHAPES)
def test_a_copy_that_never_comes_late(shape, slot, eight):
    B, n, m, G, Hkv, D = SHAPES[shape]
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    tiles = B * Hkv * -(-n // 128)
    assert tiles // sms > 8  # (the first CTA has more than 16 copies)
    gen = torch.Generator(device="cuda").manual_seed(slot)
    page, most = 64, -(-n // 64)
    store = R.E4M3 if eight else torch.bfloat16
    k, v = (torch.randn(B * most, Hkv, page, D, generator=gen, device="cuda").to(store) for _ in range(2))
    scales = [torch.ones(B * most, Hkv, device="cuda") for _ in range(2)] if eight else []
    q = torch.randn(B * m, G * Hkv, D, generator=gen, device="cuda").to(torch.bfloat16)
    table = torch.arange(B * most, dtype=torch.int32, device="cuda").view(B, most)
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    start = torch.arange(B + 1, dtype=torch.int32, device="cuda") * m
    call = da.decode_attn_tree_q8_fwd if eight else da.decode_attn_tree_fwd
    ws = da.alloc_tree_workspace(G * Hkv, Hkv, D)

    def attend(err):
        return call(q, k, v, *scales, table, lens, token_start=start, workspace=ws, err_flag=err)

    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    clean = attend(err)
    assert int(err.item()) == 0 and torch.isfinite(clean).all()
    da.test_skip_slot(slot)
    try:
        out = attend(err)
        torch.cuda.synchronize()
    finally:
        da.test_skip_slot(-1)
    assert int(err.item()) == da.DA_DEVERR_TIMEOUT
    bad = out.isnan().view(B, m, Hkv, G, D).transpose(1, 2)
    assert bad[0, slot // 2 // -(-n // 128)].all()  # the unit in which the copy is
    whole = bad.flatten(2).all(dim=-1)  # [B, Hkv]: units are NaN as a whole, the others untouched
    assert torch.equal(whole, bad.flatten(2).any(dim=-1))
    assert int(whole.sum()) <= -(-B * Hkv // sms)  # (those of one CTA)
    ours, theirs = (x.view(B, m, Hkv, G, D).transpose(1, 2)[~whole] for x in (out, clean))
    assert torch.equal(R.bits(ours), R.bits(theirs))
    ws.zero_()
    err.zero_()
    assert torch.equal(R.bits(attend(err)), R.bits(clean)) and int(err.item()) == 0
