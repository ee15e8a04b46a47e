"""Refusals of the paged-cache and sliding-window entry points, on the CPU:
every bad argument is turned away before anything touches a GPU (the pointers
here are never followed)."""
import ctypes

import pytest
import torch

import decode_attention_static_gb300 as da
import paged_reference as R
from decode_attention_static_gb300 import build as da_build

A = 0x10000
NULL, SHAPE, UNSUPPORTED, ALIGN, DTYPE = -1, -2, -3, -6, -7


@pytest.fixture(scope="module")
def lib():
    da_build.build_library()
    return da.load_library()


APPEND = dict(k=A, v=2 * A, ks=A, vs=2 * A, k_new=A, v_new=A, q=A, q_out=A, cos=A, sin=A, rope_rows=4096, table=A, pos=A, start=A,
              B=2, tokens=10, H=32, Hkv=8, D=128, pages=64, size=16, max_pages=8, dtype=1, err=None, stream=None)
ATTN = dict(q=2 * A, k=A, v=A, ks=A, vs=A, table=A, kv_len=A, B=2, H=32, Hkv=8, D=128, pages=64, size=16, max_pages=8,
            window=0, sinks=0, scale=0.1, out=A, ws=A, ws_bytes=1 << 30, dtype=1, err=None, stream=None)
WINDOW = dict(q=2 * A, k=A, v=A, kv_len=A, B=2, H=32, Hkv=8, D=128, capacity=1024, window=64, sinks=4, scale=0.1, out=A, ws=A,
              ws_bytes=1 << 30, dtype=1, err=None, stream=None)


def call(lib, fn, **kw):
    base = dict(APPEND if "append" in fn else WINDOW if "window" in fn else ATTN)
    assert set(kw) <= set(base)
    base.update(kw)
    if "q8" not in fn:
        base.pop("ks", None)
        base.pop("vs", None)
    return getattr(lib, fn)(*base.values())


APPENDS = ["kvcache_append_paged", "kvcache_append_paged_q8"]
PAGED = ["decode_attn_paged_fwd", "decode_attn_paged_q8_fwd"]
EVERY = APPENDS + PAGED + ["decode_attn_window_fwd"]


@pytest.mark.parametrize("fn", EVERY)
def test_sizes_and_types(lib, fn):
    assert call(lib, fn, dtype=2) == DTYPE
    assert call(lib, fn, dtype=-1) == DTYPE
    assert call(lib, fn, B=-1) == SHAPE
    assert call(lib, fn, Hkv=0) == SHAPE
    assert call(lib, fn, D=0) == SHAPE
    assert call(lib, fn, D=96) == UNSUPPORTED
    assert call(lib, fn, D=256) == UNSUPPORTED
    for name in ("k", "v"):
        assert call(lib, fn, **{name: None}) == NULL
        assert call(lib, fn, **{name: A + 8}) == ALIGN
    assert call(lib, fn, err=A + 1) == ALIGN
    if fn != "decode_attn_window_fwd":
        for bad in (0, -16):
            assert call(lib, fn, size=bad) == SHAPE
        for bad in (1, 8, 24, 48, 512, 1 << 30):
            assert call(lib, fn, size=bad) == UNSUPPORTED
        assert call(lib, fn, pages=0) == SHAPE
        assert call(lib, fn, max_pages=0) == SHAPE
        assert call(lib, fn, max_pages=(1 << 31) // 16) == SHAPE
        assert call(lib, fn, max_pages=(1 << 31) // 16 - 32) == SHAPE
        assert call(lib, fn, table=None) == NULL
        assert call(lib, fn, table=A + 2) == ALIGN
    if "q8" in fn:
        for name in ("ks", "vs"):
            assert call(lib, fn, **{name: None}) == NULL
            assert call(lib, fn, **{name: A + 2}) == ALIGN


@pytest.mark.parametrize("fn", APPENDS)
def test_append_arguments(lib, fn):
    assert call(lib, fn, tokens=-1) == SHAPE
    assert call(lib, fn, start=None) == SHAPE             # 10 tokens of 2 sequences need token_start
    assert call(lib, fn, B=0) == SHAPE                    # tokens, but no sequence
    assert call(lib, fn, B=0, tokens=0) == 0
    assert call(lib, fn, tokens=0) == 0
    assert call(lib, fn, q=A, H=0) == SHAPE
    for name in ("k_new", "v_new", "pos"):
        assert call(lib, fn, **{name: None}) == NULL
    for name in ("cos", "sin"):                           # the tables come together, and q needs them
        assert call(lib, fn, **{name: None}) == NULL
    assert call(lib, fn, cos=None, sin=None) == NULL
    assert call(lib, fn, q_out=None) == NULL
    assert call(lib, fn, rope_rows=0) == SHAPE
    for name in ("k_new", "v_new", "q", "q_out", "cos", "sin"):
        assert call(lib, fn, **{name: A + 4}) == ALIGN
    for name in ("pos", "start"):
        assert call(lib, fn, **{name: A + 2}) == ALIGN
    assert call(lib, fn, v=A) == SHAPE                    # K and V in one array
    if "q8" in fn:
        assert call(lib, fn, vs=A) == SHAPE


@pytest.mark.parametrize("fn", PAGED + ["decode_attn_window_fwd"])
def test_attention_arguments(lib, fn):
    assert call(lib, fn, H=30) == SHAPE
    assert call(lib, fn, H=24) == UNSUPPORTED
    assert call(lib, fn, H=128) == UNSUPPORTED
    assert call(lib, fn, B=70000) == SHAPE
    assert call(lib, fn, window=-1) == SHAPE
    assert call(lib, fn, window=64, sinks=-1) == SHAPE
    for name in ("q", "kv_len", "out"):
        assert call(lib, fn, **{name: None}) == NULL
    for name in ("q", "out"):
        assert call(lib, fn, **{name: A + 2}) == ALIGN
    assert call(lib, fn, kv_len=A + 1) == ALIGN
    assert call(lib, fn, B=0, q=None, k=None) == 0
    assert call(lib, fn, out=2 * A) == SHAPE              # the output over the query
    if fn == "decode_attn_window_fwd":
        assert call(lib, fn, window=0) == SHAPE
        assert call(lib, fn, capacity=0) == SHAPE
        assert call(lib, fn, capacity=(1 << 31) - 1) == SHAPE
        assert call(lib, fn, B=65535, H=64, Hkv=64, capacity=1 << 30) == SHAPE  # more tiles than are numbered
    else:
        assert call(lib, fn, window=0, sinks=1) == SHAPE
        assert call(lib, fn, B=65535, H=64, Hkv=64, max_pages=1 << 26) == SHAPE


def test_workspace_size_rejects_bad_sizes(lib):
    bad = ctypes.c_size_t(-1).value
    assert lib.decode_attn_paged_workspace_size(30, 8, 128) == bad
    assert lib.decode_attn_paged_workspace_size(32, 8, 96) == bad
    assert lib.decode_attn_paged_workspace_size(32, 0, 128) == bad
    with pytest.raises(da.DecodeAttnError):
        da.decode_attn_paged_workspace_size(30, 8, 128)


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-GPU error path")
@pytest.mark.parametrize("fn", PAGED + ["decode_attn_window_fwd"])
def test_valid_call_without_gpu_reports_cuda_error(lib, fn):
    assert call(lib, fn) == -5


def tensors(eight=False):
    store = R.E4M3 if eight else torch.float16
    return dict(q=torch.zeros(2, 4, 64, dtype=torch.float16), k=torch.zeros(6, 2, 16, 64, dtype=torch.float16).to(store),
                new=torch.zeros(2, 2, 64, dtype=torch.float16), s=torch.zeros(6, 2),
                table=torch.zeros(2, 3, dtype=torch.int32), n=torch.zeros(2, dtype=torch.int32))


@pytest.mark.parametrize("eight", [False, True], ids=["16bit", "e4m3"])
def test_binding_rejects_host_tensors(eight):
    t = tensors(eight)
    pool = (t["k"], t["k"], t["s"], t["s"]) if eight else (t["k"], t["k"])
    with pytest.raises(ValueError, match="CUDA"):
        (da.kvcache_append_paged_q8 if eight else da.kvcache_append_paged)(*pool, t["new"], t["new"], t["table"], t["n"])
    with pytest.raises(ValueError, match="CUDA"):
        (da.decode_attn_paged_q8_fwd if eight else da.decode_attn_paged_fwd)(t["q"], *pool, t["table"], t["n"])
    with pytest.raises(ValueError, match="CUDA"):
        da.decode_attn_window_fwd(t["q"], t["k"][:2], t["k"][:2], t["n"], 4)


@pytest.mark.gpu
@pytest.mark.parametrize("eight", [False, True], ids=["16bit", "e4m3"])
def test_binding_says_what_is_wrong(eight):
    """Every tensor argument in turn with a wrong type, shape, layout or device
    raises before the library is called; the same call with good ones runs."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    t = {n: x.cuda() for n, x in tensors(eight).items()}
    f32 = dict(dtype=torch.float32, device="cuda")
    scales = dict(k_scale=t["s"], v_scale=t["s"].clone()) if eight else {}
    pool = dict(k_pages=t["k"], v_pages=t["k"].clone())
    append = dict(**pool, **scales, k_new=t["new"], v_new=t["new"], page_table=t["table"], position_ids=t["n"],
                  token_start=torch.arange(3, dtype=torch.int32, device="cuda"), rope_cos=torch.zeros(48, 64, **f32),
                  rope_sin=torch.zeros(48, 64, **f32), q=t["q"], q_out=t["q"].clone(),
                  err_flag=torch.zeros(1, dtype=torch.int32, device="cuda"))
    ws = da.alloc_paged_workspace(4, 2, 64)
    attend = dict(q=t["q"], **pool, **scales, page_table=t["table"], kv_len=t["n"], out=t["q"].clone(), workspace=ws,
                  err_flag=append["err_flag"])
    window = dict(q=t["q"], k_cache=t["new"][:, :, None], v_cache=t["new"][:, :, None], kv_len=t["n"], window=4,
                  out=t["q"].clone(), workspace=ws, err_flag=append["err_flag"])
    calls = [((da.kvcache_append_paged_q8 if eight else da.kvcache_append_paged), append),
             ((da.decode_attn_paged_q8_fwd if eight else da.decode_attn_paged_fwd), attend)]
    if not eight:
        calls.append((da.decode_attn_window_fwd, window))
    for fn, good in calls:
        fn(**good)
        for name, x in good.items():
            if not isinstance(x, torch.Tensor):
                continue
            wrong = [x.cpu()]
            if name != "workspace":
                other = torch.float64 if x.dtype != torch.float64 else torch.float32
                wrong.append(x.to(other))
            if name not in ("workspace", "err_flag"):
                wrong.append(torch.cat([x, x]))
                if x.dim() > 1:
                    wrong.append(x.transpose(-1, -2).contiguous().transpose(-1, -2) if x.shape[-2] > 1 else x[..., ::2])
            for bad in wrong:
                with pytest.raises((ValueError, TypeError)):
                    fn(**{**good, name: bad})
    torch.cuda.synchronize()


@pytest.mark.gpu
@pytest.mark.parametrize("eight", [False, True], ids=["16bit", "e4m3"])
def test_both_paths_of_the_binding(eight, monkeypatch):
    """The calls made in C++ and those made from Python do the same, on a stream
    of their own too, and the C++ path is there."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from decode_attention_static_gb300 import _binding

    da_build.build_library()
    assert _binding._load_fast()
    gen = torch.Generator().manual_seed(0)
    new, q = torch.randn(5, 2, 64, generator=gen).half().cuda(), torch.randn(5, 4, 64, generator=gen).half().cuda()
    tab = torch.arange(5, dtype=torch.int32, device="cuda")[:, None].contiguous()
    pos = torch.tensor([0, 3, 15, 7, 8], dtype=torch.int32, device="cuda")
    cos, sin = torch.rand(16, 64, generator=gen).cuda(), torch.rand(16, 64, generator=gen).cuda()
    ws, out = da.alloc_paged_workspace(4, 2, 64), torch.empty_like(q)
    taken = []

    def run():
        pool = [torch.full((6, 2, 16, 64), 0.5, device="cuda").to(R.E4M3 if eight else torch.float16) for _ in range(2)]
        pool += [torch.full((6, 2), 0.25, device="cuda") for _ in range(2)] if eight else []
        append = da.kvcache_append_paged_q8 if eight else da.kvcache_append_paged
        attend = da.decode_attn_paged_q8_fwd if eight else da.decode_attn_paged_fwd
        got = [append(*pool, new, new, tab, pos), append(*pool, new, new, tab, pos, rope_cos=cos, rope_sin=sin, q=q),
               append(*pool, new, new, tab, pos, rope_cos=cos, rope_sin=sin, q=q, q_out=out)]
        assert got[0] is None and got[2] is out
        got = [got[1], out.clone(), *pool]
        got.append(attend(q, *pool, tab, pos, workspace=ws))
        got.append(attend(q, *pool, tab, pos, window=3, sinks=1, scale=0.3, workspace=ws, out=out).clone())
        cache = torch.full((5, 2, 16, 64), 0.5, device="cuda").half()
        got.append(da.decode_attn_window_fwd(q, cache, new[:, :, None].repeat(1, 1, 16, 1), pos, 4, workspace=ws))
        return [t.view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()]).cpu() for t in got]

    class Counted:
        def __init__(self, module):
            self.module = module

        def __getattr__(self, name):
            def call(*args):
                r = getattr(self.module, name)(*args)
                taken.append(r is not NotImplemented)
                return r
            return call

    monkeypatch.setattr(_binding, "_fast", Counted(_binding._fast))
    fast = run()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        again = run()
    assert all(taken) and len(taken) == 12
    monkeypatch.setattr(_binding, "_fast", False)
    slow = run()
    for f, a, s in zip(fast, again, slow):
        assert torch.equal(f, s) and torch.equal(a, s)


def test_plain_forms_on_known_values():
    """The tests' own plain form: the e4m3 grid against torch's conversion, and
    scales at powers of two."""
    x = torch.randn(4000, generator=torch.Generator().manual_seed(0)) * torch.exp2(
        torch.randint(-14, 9, (4000,), generator=torch.Generator().manual_seed(1)).float())
    x = x.clamp(-448, 448)
    assert torch.equal(R.grid8(x.double()).float(), x.to(R.E4M3).float())
    for value, scale in ((448.0, 1.0), (448.5, 2.0), (7.0, 2.0 ** -6), (0.0, 2.0 ** -100), (1e-38, 2.0 ** -100)):
        assert R.block_scale(torch.tensor([value, 0.0])) == scale
    assert R.visible_rows(10, 3, 2).tolist() == [0, 1, 7, 8, 9]
    assert R.visible_rows(4, 9, 2).tolist() == [0, 1, 2, 3]
