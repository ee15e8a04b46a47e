"""Refusals of the entry points for drafted tokens and for pages, on the CPU: every
bad argument is turned away before anything touches a GPU (the pointers here
are never followed); and the tests' own plain forms on known values."""
import ctypes

import pytest
import torch

import decode_attention_static_gb300 as da
import draft_reference as Q
import paged_reference as R
from decode_attention_static_gb300 import build as da_build

A = 0x10000
NULL, SHAPE, UNSUPPORTED, WORKSPACE, CUDA, ALIGN, DTYPE = -1, -2, -3, -4, -5, -6, -7


@pytest.fixture(scope="module")
def lib():
    da_build.build_library()
    return da.load_library()


AXES = dict(k=A, v=2 * A, ks=A, vs=2 * A, k_new=A, v_new=A, q=A, q_out=A, cos=A, sin=A, rope_rows=4096, turns=A, axis=A, axes=3,
            table=A, pos=A, start=A, B=2, tokens=10, H=32, Hkv=8, D=128, pages=64, size=16, max_pages=8, dtype=1, err=None,
            stream=None)
TREE = dict(q=2 * A, k=A, v=A, ks=A, vs=A, table=A, kv_len=A, start=A, mask=A, words=1, B=2, tokens=10, H=32, Hkv=8, D=128,
            pages=64, size=16, max_pages=8, scale=0.1, out=A, ws=A, ws_bytes=1 << 30, dtype=1, err=None, stream=None)
RESIZE = dict(table=A, held=A, wanted=A, pool=A, B=4, pages=64, size=16, max_pages=8, err=None, stream=None)
FORK = dict(table=A, kv_len=A, parent=A, child=A, pool=A, copies=A, forks=2, B=4, pages=64, size=16, max_pages=8, err=None,
            stream=None)
COPY = dict(k=A, v=2 * A, ks=A, vs=2 * A, copies=A, n=3, layers=2, pages=64, Hkv=8, size=16, D=128, element=1, err=None,
            stream=None)
COMPACT = dict(k=A, v=2 * A, ks=A, vs=2 * A, table=A, keep=A, start=A, pos=A, B=2, kept=5, layers=2, Hkv=8, D=128, pages=64,
               size=16, max_pages=8, err=None, stream=None)
EVERY = {"kvcache_append_paged_axes": AXES, "kvcache_append_paged_q8_axes": AXES, "decode_attn_tree_fwd": TREE,
         "decode_attn_tree_q8_fwd": TREE, "kvcache_resize_paged": RESIZE, "kvcache_fork_paged": FORK,
         "kvcache_copy_pages": COPY, "kvcache_compact_paged": COMPACT, "kvcache_compact_paged_q8": COMPACT}


def call(lib, fn, **kw):
    base = dict(EVERY[fn])
    assert set(kw) <= set(base), set(kw) - set(base)
    base.update(kw)
    if "q8" not in fn and fn != "kvcache_copy_pages":
        base.pop("ks", None)
        base.pop("vs", None)
    return getattr(lib, fn)(*base.values())


def has(fn, name):
    return name in EVERY[fn] and ("q8" in fn or name not in ("ks", "vs"))


@pytest.mark.parametrize("fn", EVERY)
def test_sizes(lib, fn):
    if has(fn, "B"):
        assert call(lib, fn, B=-1) == SHAPE
    if has(fn, "Hkv"):
        assert call(lib, fn, Hkv=0) == SHAPE
        assert call(lib, fn, D=0) == SHAPE
        assert call(lib, fn, D=96) == UNSUPPORTED
        assert call(lib, fn, D=256) == UNSUPPORTED
    if has(fn, "dtype"):
        assert call(lib, fn, dtype=2) == DTYPE
        assert call(lib, fn, dtype=-1) == DTYPE
    for bad in (0, -16):
        assert call(lib, fn, size=bad) == SHAPE
    for bad in (1, 8, 24, 48, 512, 1 << 30):
        assert call(lib, fn, size=bad) == UNSUPPORTED
    assert call(lib, fn, pages=0) == SHAPE
    if has(fn, "max_pages"):
        assert call(lib, fn, max_pages=0) == SHAPE
        assert call(lib, fn, max_pages=(1 << 31) // 16) == SHAPE
    if has(fn, "layers"):
        assert call(lib, fn, layers=-1) == SHAPE
        assert call(lib, fn, layers=0) == 0


@pytest.mark.parametrize("fn", EVERY)
def test_pointers(lib, fn):
    wide = ("k", "v", "k_new", "v_new", "q", "q_out", "cos", "sin", "out", "ws", "axis")
    words = ("table", "kv_len", "pos", "turns", "held", "wanted", "pool", "parent", "child", "copies", "keep", "ks", "vs")
    for name in wide + words + ("start",):
        if not has(fn, name) or (name == "ws" and not torch.cuda.is_available()):
            continue
        optional = name in ("axis", "q", "start") and "append" in fn or name == "start" and "tree" in fn
        if not optional:
            assert call(lib, fn, **{name: None}) == (WORKSPACE if name == "ws" else NULL), name
        bad = 4 if name in wide else 2
        assert call(lib, fn, **{name: EVERY[fn][name] + bad}) == ALIGN, name
    assert call(lib, fn, err=A + 1) == ALIGN


@pytest.mark.parametrize("fn", ["kvcache_append_paged_axes", "kvcache_append_paged_q8_axes"])
def test_append_arguments(lib, fn):
    for bad in (0, -1, 5):
        assert call(lib, fn, axes=bad) == SHAPE
    assert call(lib, fn, tokens=-1) == SHAPE
    assert call(lib, fn, start=None) == SHAPE
    assert call(lib, fn, cos=None, sin=None, q=None, q_out=None) == NULL  # the tables are required
    assert call(lib, fn, rope_rows=0) == SHAPE
    assert call(lib, fn, B=0, tokens=0) == 0
    assert call(lib, fn, v=A) == SHAPE


@pytest.mark.parametrize("fn", ["decode_attn_tree_fwd", "decode_attn_tree_q8_fwd"])
def test_tree_arguments(lib, fn):
    assert call(lib, fn, H=30) == SHAPE
    assert call(lib, fn, H=24) == UNSUPPORTED
    assert call(lib, fn, H=128) == UNSUPPORTED
    assert call(lib, fn, B=70000) == SHAPE
    assert call(lib, fn, tokens=-1) == SHAPE
    assert call(lib, fn, start=None) == SHAPE
    assert call(lib, fn, B=0) == SHAPE
    assert call(lib, fn, B=0, tokens=0) == 0
    assert call(lib, fn, tokens=0) == 0
    for bad in (0, -1, 5):
        assert call(lib, fn, words=bad) == SHAPE
    assert call(lib, fn, mask=A + 4) == ALIGN
    assert call(lib, fn, out=2 * A) == SHAPE             # the output over the query
    assert call(lib, fn, pages=1 << 24) == SHAPE         # rows of the pools past 32 bits
    assert call(lib, fn, B=65535, tokens=65535, max_pages=1 << 26, Hkv=64, H=64) == SHAPE


def test_page_arguments(lib):
    big = (1 << 22) + 1
    for fn in ("kvcache_resize_paged", "kvcache_fork_paged"):
        assert call(lib, fn, pages=big) == SHAPE
        assert call(lib, fn, B=70000) == SHAPE
        assert call(lib, fn, B=65535, max_pages=1 << 16) == SHAPE
    assert call(lib, "kvcache_resize_paged", B=0) == 0
    assert call(lib, "kvcache_fork_paged", forks=0) == 0
    assert call(lib, "kvcache_fork_paged", forks=-1) == SHAPE
    assert call(lib, "kvcache_fork_paged", B=0) == SHAPE
    assert call(lib, "kvcache_copy_pages", n=0) == 0
    assert call(lib, "kvcache_copy_pages", n=-1) == SHAPE
    for bad in (0, 3, 4):
        assert call(lib, "kvcache_copy_pages", element=bad) == DTYPE
    assert call(lib, "kvcache_copy_pages", v=A) == SHAPE
    assert call(lib, "kvcache_copy_pages", vs=A) == SHAPE
    assert call(lib, "kvcache_copy_pages", ks=None) == NULL
    assert call(lib, "kvcache_copy_pages", n=1 << 20, layers=1 << 20) == SHAPE
    for fn in ("kvcache_compact_paged", "kvcache_compact_paged_q8"):
        assert call(lib, fn, kept=-1) == SHAPE
        assert call(lib, fn, kept=0) == 0
        assert call(lib, fn, B=0) == 0
        assert call(lib, fn, v=A) == SHAPE
        assert call(lib, fn, layers=(1 << 31) - 1, B=65535) == SHAPE
    assert lib.kvcache_pool_init(A, 0, None) == SHAPE
    assert lib.kvcache_pool_init(A, big, None) == SHAPE
    assert lib.kvcache_pool_init(None, 8, None) == NULL
    assert lib.kvcache_pool_init(A + 2, 8, None) == ALIGN


def test_workspace_size_rejects_bad_sizes(lib):
    bad = ctypes.c_size_t(-1).value
    for sizes in ((30, 8, 128), (32, 8, 96), (32, 0, 128)):
        assert lib.decode_attn_tree_workspace_size(*sizes) == bad
    with pytest.raises(da.DecodeAttnError):
        da.decode_attn_tree_workspace_size(30, 8, 128)


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-GPU error path")
@pytest.mark.parametrize("fn", EVERY)
def test_valid_call_without_gpu_reports_cuda_error(lib, fn):
    assert call(lib, fn) == CUDA


def arguments(device, eight):
    """Good arguments of every function of the binding."""
    store = R.E4M3 if eight else torch.float16
    i32 = dict(dtype=torch.int32, device=device)
    k = torch.zeros(6, 2, 16, 64, dtype=torch.float16, device=device).to(store)
    pool = dict(k_pages=k, v_pages=k.clone())
    scales = dict(k_scale=torch.ones(6, 2, device=device), v_scale=torch.ones(6, 2, device=device)) if eight else {}
    new, q = (torch.zeros(3, h, 64, dtype=torch.float16, device=device) for h in (2, 4))
    table, n = torch.arange(4, **i32).view(2, 2), torch.full((2,), 4, **i32)
    start, err = torch.tensor([0, 1, 3], **i32), torch.zeros(1, **i32)
    rope = torch.zeros(48, 64, device=device)
    state = Q.Pool(6, [4, 5], [1] * 4 + [0] * 2).tensor().to(device)
    q8 = "_q8" if eight else ""
    calls = {
        f"kvcache_append_paged{q8}_axes": dict(
            **pool, **scales, k_new=new, v_new=new, page_table=table, position_ids=n,
            rope_position_ids=torch.zeros(2, 3, **i32), rope_cos=rope, rope_sin=rope, rope_axis=torch.zeros(32, **i32),
            token_start=start, q=q, q_out=q.clone(), err_flag=err),
        f"decode_attn_tree{q8}_fwd": dict(
            q=q, **pool, **scales, page_table=table, kv_len=n, token_start=start,
            tree_mask=torch.ones(3, 1, dtype=torch.int64, device=device), out=q.clone(), err_flag=err),
        "kvcache_copy_pages": dict(**pool, **scales, copies=torch.full((3, 2), -1, **i32), err_flag=err),
        f"kvcache_compact_paged{q8}": dict(**pool, **scales, page_table=table, keep=torch.tensor([4, 5, 7], **i32),
                                           keep_start=start, position_ids=n, err_flag=err),
    }
    if not eight:
        calls["kvcache_resize_paged"] = dict(page_table=table, held_len=n, wanted_len=n, pool=state, page_size=16, err_flag=err)
        calls["kvcache_fork_paged"] = dict(page_table=table, kv_len=n, parent=torch.zeros(1, **i32),
                                           child=torch.ones(1, **i32), pool=state, page_size=16,
                                           copies=torch.zeros(3, 1, **i32), err_flag=err)
    return calls


@pytest.mark.parametrize("eight", [False, True], ids=["16bit", "e4m3"])
def test_binding_rejects_host_tensors(eight):
    for name, good in arguments("cpu", eight).items():
        with pytest.raises(ValueError, match="CUDA"):
            getattr(da, name)(**good)


@pytest.mark.gpu
@pytest.mark.parametrize("eight", [False, True], ids=["16bit", "e4m3"])
def test_binding_says_what_is_wrong(eight):
    """Every tensor argument in turn with a wrong type, shape, layout or device
    raises before the library is called; the same call with good ones runs."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    calls = arguments("cuda", eight)
    for fn, good in calls.items():
        if "tree" in fn:
            good["workspace"] = da.alloc_tree_workspace(4, 2, 64)
        getattr(da, fn)(**good)
        for name, x in good.items():
            if not isinstance(x, torch.Tensor):
                continue
            wrong = [x.cpu()]
            if name != "workspace":
                wrong.append(x.to(torch.float64 if x.dtype != torch.float64 else torch.float32))
            if name == "pool":
                wrong += [x[:-1], x[None]]
            elif name == "keep":
                wrong.append(x[None])
            elif name not in ("workspace", "err_flag", "copies", "parent", "child"):
                wrong.append(torch.cat([x, x, x]))  # (two rows of positions twice would be four axes)
            if name not in ("workspace", "err_flag") and x.dim() > 1 and x.shape[-1] > 1:
                wrong.append(x.transpose(-1, -2).contiguous().transpose(-1, -2) if x.shape[-2] > 1 else x[..., ::2])
            for bad in wrong:
                with pytest.raises((ValueError, TypeError)):
                    getattr(da, fn)(**{**good, name: bad})
    torch.cuda.synchronize()


def test_binding_refuses_mixed_pools():
    t = arguments("cpu", False)["kvcache_compact_paged"]
    with pytest.raises(TypeError):
        da.kvcache_compact_paged(**{**t, "k_pages": t["k_pages"].to(R.E4M3), "v_pages": t["v_pages"].to(R.E4M3)})
    with pytest.raises(ValueError, match="scales"):
        da.kvcache_compact_paged_q8(t["k_pages"], t["v_pages"], None, None, t["page_table"], t["keep"], t["keep_start"],
                                    t["position_ids"])


# ---------------------------------------------------------------------------
# The plain forms on known values


def test_plain_masks():
    assert Q.seen_rows(5, 3, None).int().tolist() == [[1, 1, 1, 0, 0], [1, 1, 1, 1, 0], [1, 1, 1, 1, 1]]
    assert Q.seen_rows(4, 3, [1, 3, 5]).int().tolist() == [[1, 1, 0, 0], [1, 1, 1, 0], [1, 1, 0, 1]]
    assert Q.words_of([1 << 63, 1 << 64 | 1], 2).tolist() == [[-(1 << 63), 0], [1, 1]]


def test_plain_tree_of_one_token_is_attention():
    gen = torch.Generator().manual_seed(0)
    q, k, v = (torch.randn(*s, generator=gen).double() for s in ((1, 4, 64), (2, 9, 64), (2, 9, 64)))
    out, _ = Q.attend_seen(q, k, v, Q.seen_rows(9, 1, [1]), 0.125, 2.0 ** -8)
    assert torch.equal(out[0], R.attend(q[0], k, v, 0.125)[0])
    # a token that sees one row gets it
    out, _ = Q.attend_seen(q, k[:, :1], v[:, :1], Q.seen_rows(1, 1, [1]), 0.125, 2.0 ** -8)
    assert torch.equal(out[0].view(2, 2, 64), v[:, :1].expand(2, 2, 64))


def test_plain_pages():
    pool = Q.Pool(6)
    table = [[-1] * 3 for _ in range(3)]
    Q.resize(table, [0, 0, 0], [33, 0, 16], pool, 16)
    assert table == [[5, 4, 3], [-1] * 3, [2, -1, -1]] and pool.free == 2 and pool.counts == [0, 0, 1, 1, 1, 1]
    lens = [33, 0, 16]
    assert Q.fork(table, lens, [0], [1], pool, 16) == [[3], [1], [1]]
    assert table[1] == [5, 4, 1] and pool.counts == [0, 1, 1, 1, 2, 2] and lens == [33, 33, 16] and pool.free == 1
    Q.resize(table, [33, 33, 16], [0, 16, 0], pool, 16)
    assert table == [[-1] * 3, [5, -1, -1], [-1] * 3] and pool.list[:pool.free] == [0, 1, 2, 3, 4]
    assert pool.counts == [0, 0, 0, 0, 0, 1] and not pool.errors
    Q.resize(table, [0, 16, 0], [48, 48, 16], pool, 16)
    assert pool.errors == {"full"} and table == [[4, 3, 2], [5, 1, 0], [-1] * 3]


def test_plain_compaction():
    pool = torch.arange(2 * 16).view(1, 2, 1, 16, 1).repeat(1, 1, 1, 1, 2)
    table = torch.tensor([[1, 0]])
    errors = Q.compact([pool, pool.clone()], table, torch.tensor([3, 6, 17]), [0, 3], [3], 16)
    assert not errors and pool[0, 1, 0, :7, 0].tolist() == [16, 17, 18, 19, 22, 1, 22]
    assert Q.compact([pool, pool.clone()], table, torch.tensor([3, 3]), [0, 2], [3], 16) == {"position"}


@pytest.mark.gpu
@pytest.mark.parametrize("eight", [False, True], ids=["16bit", "e4m3"])
def test_both_paths_of_the_binding(eight, monkeypatch):
    """The calls made in C++ and those made from Python do the same, and the C++ path takes them all."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from decode_attention_static_gb300 import _binding

    da_build.build_library()
    assert _binding._load_fast()
    taken = []

    class Counted:
        def __init__(self, module):
            self.module = module

        def __getattr__(self, name):
            def call(*args):
                r = getattr(self.module, name)(*args)
                taken.append(r is not NotImplemented)
                return r
            return call

    def run():
        gen = torch.Generator().manual_seed(0)
        got = []
        for fn, good in arguments("cuda", eight).items():
            for name in ("q", "k_new", "v_new", "k_pages", "v_pages", "rope_cos", "rope_sin"):
                if name in good:
                    good[name].copy_(torch.randn(good[name].shape, generator=gen).to(good[name].dtype))
            if "tree" in fn:
                good["workspace"] = da.alloc_tree_workspace(4, 2, 64)
            for drop in ("err_flag", "out", "q_out", "copies") if fn != "kvcache_copy_pages" else ("err_flag",):
                r = getattr(da, fn)(**{k: v for k, v in good.items() if k != drop})
                got += [t for t in good.values() if isinstance(t, torch.Tensor) and t is not good.get("workspace")]
                got += [r] if r is not None else []
                got = [t.clone() for t in got]
        return [R.bits(t.view(torch.uint8)) for t in got]

    monkeypatch.setattr(_binding, "_fast", Counted(_binding._fast))
    fast = run()
    assert all(taken) and len(taken) >= 13
    monkeypatch.setattr(_binding, "_fast", False)
    slow = run()
    assert len(fast) == len(slow)
    for f, s in zip(fast, slow):
        assert torch.equal(f, s)
