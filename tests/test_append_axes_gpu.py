"""The paged append with rotary positions of their own, bit for bit against the
plain form (tests/draft_reference.py)."""
import pytest
import torch

import decode_attention_static_gb300 as da
import draft_reference as Q
import paged_reference as R
import test_paged_append_gpu as T

pytestmark = pytest.mark.gpu
BOTH = T.BOTH
ROWS = 500


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    da.build_library()
    da.load_library()


class Inputs(T.Inputs):
    def __init__(self, counts, positions, H, Hkv, D, dtype, page, eight, axes=3, split="sections", rows=ROWS, **kw):
        super().__init__(counts, positions, H, Hkv, D, dtype, page, eight, **kw)
        gen = torch.Generator().manual_seed(axes + D)
        self.cos, self.sin = T.tables(rows, D)
        self.turns = torch.randint(0, rows, (axes, self.k_new.shape[0]), generator=gen).to(torch.int32)
        pair = torch.arange(D // 2)
        self.axis = {"none": None, "sections": pair * axes // (D // 2), "interleaved": pair % axes,
                     "odd": torch.randint(0, axes, (D // 2,), generator=gen)}[split]
        self.axis = None if self.axis is None else self.axis.to(torch.int32)

    def plain(self):
        c = [None if t is None else t.clone() for t in (self.k, self.v, self.ks, self.vs)]
        q = Q.append_axes(c[0], c[1], self.k_new, self.v_new, self.table, self.position, self.start, self.cos, self.sin,
                          self.turns, self.axis, self.q, c[2], c[3])
        return [*c, q]

    def call(self, q_out=None, err=None, dev=None):
        d = dev or self.cuda()
        args = (d["k_new"], d["v_new"], d["table"], d["position"], self.turns.cuda(), d["cos"], d["sin"])
        kw = dict(rope_axis=None if self.axis is None else self.axis.cuda(), token_start=d["start"], q=d["q"], q_out=q_out,
                  err_flag=err)
        if self.eight:
            q = da.kvcache_append_paged_q8_axes(d["k"], d["v"], d["ks"], d["vs"], *args, **kw)
        else:
            q = da.kvcache_append_paged_axes(d["k"], d["v"], *args, **kw)
        return [d["k"], d["v"], d["ks"], d["vs"], q]


@BOTH
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("axes,split", [(1, "none"), (1, "sections"), (2, "interleaved"), (3, "sections"), (3, "interleaved"),
                                        (4, "odd"), (4, "sections")])
@pytest.mark.parametrize("H,Hkv,D,page", [(4, 1, 64, 16), (16, 8, 128, 16), (5, 5, 128, 64), (32, 4, 64, 256)])
def test_one_token_each(H, Hkv, D, page, axes, split, dtype, eight):
    positions = [0, 1, page - 1, page, page + 1, 3 * page, 37, 700]
    for packed in (False, True):
        T.check(Inputs([1] * 8, positions, H, Hkv, D, dtype, page, eight, axes, split, seed=D + page, packed=packed))


@BOTH
@pytest.mark.parametrize("axes,split", [(1, "none"), (3, "sections"), (4, "odd")])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_prompts(page, D, axes, split, eight):
    counts = [1, page, 2 * page + 3, 0, page - 1, 5, 700]
    positions = [5, 0, page - 2, 9, 1, 2 * page - 1, 3]
    T.check(Inputs(counts, positions, 8, 2, D, "bf16", page, eight, axes, split, seed=page, lead=2, trail=3))
    T.check(Inputs(counts, positions, 3, 3, D, "f16", page, eight, axes, split, seed=page, with_q=False))


@BOTH
def test_tokens_positions_are_kvcache_append_paged(eight):
    """With every rope position the token's own, the plain append's bits."""
    inp = Inputs([3, 40, 1, 90], [5, 0, 63, 20], 8, 2, 128, "bf16", 16, eight, axes=2, split="odd")
    at = torch.cat([torch.arange(p, p + n) for p, n in ((5, 3), (0, 40), (63, 1), (20, 90))]).to(torch.int32)
    inp.turns = torch.stack([at, at])
    plain = T.Inputs.call(inp)
    for a, b in zip(inp.call(), plain):
        if a is not None:
            assert torch.equal(R.bits(a), R.bits(b))


@BOTH
def test_drafts_of_a_tree(eight):
    """Two drafts of one depth turn alike though they go to different rows."""
    inp = Inputs([4], [100], 4, 2, 64, "f16", 16, eight, axes=1, split="none")
    inp.turns = torch.tensor([[100, 101, 101, 102]], dtype=torch.int32)
    inp.q[2] = inp.q[1]
    q = inp.call()[4]
    assert torch.equal(R.bits(q[1]), R.bits(q[2]))
    T.check(inp)


@BOTH
@pytest.mark.parametrize("counts", [[1] * 6, [3, 40, 1, 0, 90, 17]])
def test_positions_outside_the_tables(counts, eight):
    """A token with a bad position is skipped whole, others are not."""
    inp = Inputs(counts, [5, 0, 63, 1, 20, 30], 8, 2, 128, "bf16", 16, eight, axes=3)
    last = inp.turns.shape[1] - 1
    for axis, t, bad in ((0, 1, -1), (2, 3, ROWS), (1, last, 1 << 30), (0, last // 2, -(1 << 31))):
        inp.turns[axis, t] = bad
    T.check(inp, flag=da.DA_DEVERR_POSITION)


@BOTH
def test_whole_pages_of_bad_positions(eight):
    inp = Inputs([50], [14], 4, 2, 64, "bf16", 16, eight, axes=1, split="none")
    inp.turns[0, 2:18] = -1
    T.check(inp, flag=da.DA_DEVERR_POSITION)


@BOTH
def test_bad_axes_count_as_the_first(eight):
    inp = Inputs([3, 20], [5, 0], 4, 2, 64, "f16", 16, eight, axes=2, split="odd")
    good = inp.axis.clone()
    inp.axis[3], inp.axis[31] = 2, -1
    good[3] = good[31] = 0
    got = inp.call(err=(err := torch.zeros(1, dtype=torch.int32, device="cuda")))
    assert int(err.item()) == da.DA_DEVERR_POSITION
    inp.axis = good
    T.same(got, inp.plain())


@BOTH
def test_sequences_outside_the_table(eight):
    """position_ids beyond the table skip a sequence; beyond the rope tables they do not."""
    inp = Inputs([3, 2, 4], [700, 20, 3], 4, 2, 64, "f16", 16, eight, axes=2, rows=64)
    T.check(inp)
    inp.position[1] = inp.table.shape[1] * 16 - 1
    T.check(inp, flag=da.DA_DEVERR_POSITION)
    inp.position[1] = -1
    T.check(inp, flag=da.DA_DEVERR_POSITION)
