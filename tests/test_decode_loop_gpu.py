"""The operators of a decode step chained as a serving loop runs them: length
update, append and attention in one captured graph, each kernel starting under
the one before it; and lengths that are written while the attention that
follows has already looked at them."""
import ctypes
import pathlib
import subprocess

import pytest
import torch

import cache_attn_split as S
import decode_attention_static_gb300 as da
import paged_reference as R
import test_paged_attention_gpu as T
from decode_attention_static_gb300 import build as da_build
from test_paged_append_gpu import tables

BOTH = pytest.mark.parametrize("eight", [False, True], ids=["16bit", "e4m3"])


def compile_helper(folder: pathlib.Path) -> pathlib.Path:
    out = folder / "late_lengths.so"
    subprocess.run([da_build.nvcc(), *da_build.ARCH, "-O2", "-std=c++17", "-shared", "-cudart", "static", "-Xcompiler",
                    "-fPIC", "-o", str(out), str(pathlib.Path(__file__).with_name("late_lengths.cu"))], check=True,
                   capture_output=True)
    return out


def test_the_helper_compiles(tmp_path):
    assert ctypes.CDLL(str(compile_helper(tmp_path))).late_lengths


@pytest.fixture(scope="module")
def late(tmp_path_factory):
    """late(kv_len, values): kv_len becomes values some 30 us after the next
    kernel on the stream may have started."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    da.build_library()
    fn = ctypes.CDLL(str(compile_helper(tmp_path_factory.mktemp("late")))).late_lengths
    fn.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_ulonglong, ctypes.c_void_p]
    seen = torch.zeros(1, dtype=torch.int32, device="cuda")

    def call(kv_len, values):
        assert fn(kv_len.data_ptr(), values.data_ptr(), values.numel(), seen.data_ptr(), 30000,
                  torch.cuda.current_stream().cuda_stream) == 0
    return call


# lengths that the call finds, those before it, KV heads
CHANGES = {
    "short to long": ([3000, 2500], [16, 20], 8),
    "long to short": ([16, 20], [3000, 2500], 8),
    "idle to busy": ([700] * 6, [0] * 6, 8),
    "one CTA a group to many": ([900, 30, 2000], [128] * 3, 8),
    "refused to valid": ([500, 60, 7], [-5, 1 << 30, 1 << 12], 4),
    "one more row": ([1024], [1023], 16),
    "teams to shares": ([3000] + [20] * 59, [60] * 60, 8),
    "shares to teams": ([60] * 60, [3000] + [20] * 59, 8),
    "teams of 1 to teams of 4": ([300] * 38 + [0] * 114, [100] * 152, 8),
    "teams of 4 to teams of 1": ([100] * 152, [300] * 38 + [0] * 114, 8),
    "more than one scan": ([3000] + [20] * 419, [60] * 420, 1),
}


def test_the_changes_change_the_way():
    def way(lens, Hkv):
        return S.ways([n if 0 <= n <= 8192 else 0 for n in lens], Hkv, 128, False)[0]

    for name, (new, old, Hkv) in CHANGES.items():
        if name not in ("one more row", "refused to valid", "idle to busy", "more than one scan"):
            assert way(new, Hkv) != way(old, Hkv), name


@pytest.mark.gpu
@BOTH
@pytest.mark.parametrize("name", CHANGES)
def test_lengths_written_under_the_prologue(name, eight, late):
    """The division is made from the lengths that a call reads before the kernel
    ahead of it is done, and made again where they were not final: the outputs
    are those of the final ones, bit for bit, whatever the earlier ones were."""
    new, old, Hkv = CHANGES[name]
    case = T.Case(new, 2 * Hkv, Hkv, 128, "bf16", 16, eight, seed=len(new), max_pages=200).cuda()
    ws, err = da.alloc_paged_workspace(2 * Hkv, Hkv, 128), torch.zeros(1, dtype=torch.int32, device="cuda")
    before, final = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (old, new))
    want = case.call(workspace=ws, err_flag=err).clone()
    R.assert_rows(want, case.ref, case.slack, name)
    out = torch.empty_like(want)

    def run():
        case.kv_len.copy_(before)
        late(case.kv_len, final)
        case.call(workspace=ws, err_flag=err, out=out)

    for _ in range(3):
        out.fill_(7.0)
        run()
        assert torch.equal(R.bits(out), R.bits(want)), f"{name}, call by call"
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        run()
    for _ in range(3):
        out.fill_(7.0)
        graph.replay()
        assert torch.equal(R.bits(out), R.bits(want)), f"{name}, in a graph"
    assert int(err.item()) == 0 and not ws[:4096].any()


@pytest.mark.gpu
@BOTH
@pytest.mark.parametrize("packed", [False, True], ids=["one token each", "idle slot"])
@pytest.mark.parametrize("dtype,H,Hkv,D,page,window,sinks", [("bf16", 16, 2, 128, 16, 0, 0), ("f16", 4, 4, 64, 32, 50, 3)])
def test_a_captured_decode_step(dtype, H, Hkv, D, page, window, sinks, packed, eight):
    """One graph holds a step: lengths up by one, append with the rotation,
    attention over the pages with the rotated query, positions up by one. The
    append and the attention are neighbours on the stream. Replayed 40 times with
    new values, every output and the cache at the end against the plain forms."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    da.build_library()
    gen, dt, steps = torch.Generator().manual_seed(page), T.TYPES[dtype], 40
    position, active = ([60, 133, 0], [1, 1, 0]) if packed else ([60, 1, 133], [1, 1, 1])
    tokens = sum(active)
    table, pool = R.deal_pages([p + a * steps for p, a in zip(position, active)], page, gen)
    cos, sin = tables(max(position) + steps, D)
    shape, store = (pool, Hkv, page, D), R.E4M3 if eight else dt
    cpu = [(torch.randn(shape, generator=gen) * (60 if eight else 1)).clamp(-448, 448).to(store) for _ in range(2)]
    cpu += [torch.exp2(torch.randint(-9, -4, (pool, Hkv), generator=gen).float()) for _ in range(2)] if eight else []
    start = torch.tensor([0, 1, 2, 2], dtype=torch.int32) if packed else None
    gpu = [t.cuda() for t in cpu]
    k_new, v_new = (torch.zeros(tokens, Hkv, D, dtype=dt, device="cuda") for _ in range(2))
    q = torch.zeros(tokens, H, D, dtype=dt, device="cuda")
    # the attention has a query for every slot; that of the last, idle one is not used
    rotated, out = torch.zeros(3, H, D, dtype=dt, device="cuda"), torch.zeros(3, H, D, dtype=dt, device="cuda")
    pos, up = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (position, active))
    kv_len, err = pos.clone(), torch.zeros(1, dtype=torch.int32, device="cuda")
    on_gpu = dict(token_start=None if start is None else start.cuda(), rope_cos=cos.cuda(), rope_sin=sin.cuda())
    tab, ws = table.cuda(), da.alloc_paged_workspace(H, Hkv, D)
    append = da.kvcache_append_paged_q8 if eight else da.kvcache_append_paged
    attend = da.decode_attn_paged_q8_fwd if eight else da.decode_attn_paged_fwd

    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        kv_len.add_(up)
        append(*gpu, k_new, v_new, tab, pos, q=q, q_out=rotated[:tokens], err_flag=err, **on_gpu)
        attend(rotated, *gpu, tab, kv_len, window=window, sinks=sinks, workspace=ws, out=out, err_flag=err)
        pos.add_(up)
    slots = [b for b in range(3) if active[b]]
    for step in range(steps):
        new = [R.randn((tokens, Hkv, D), dt, gen) for _ in range(2)] + [R.randn((tokens, H, D), dt, gen)]
        for dst, src in zip((k_new, v_new, q), new):
            dst.copy_(src)
        graph.replay()
        want_q = R.append(cpu[0], cpu[1], new[0], new[1], table, torch.tensor(position, dtype=torch.int32), start, cos,
                          sin, new[2], *(cpu[2:] if eight else (None, None)))
        position = [p + a for p, a in zip(position, active)]
        assert torch.equal(R.bits(rotated[:tokens]), R.bits(want_q))
        for b in slots:
            j = R.visible_rows(position[b], window, sinks)
            p = table[b].long()[j // page]
            rows = [t.view(torch.uint8 if eight else torch.int16)[p, :, j % page].view(store).double() for t in cpu[:2]]
            if eight:
                rows = [r * s[p].double()[..., None] for r, s in zip(rows, cpu[2:])]
            ref, slack = R.attend(rotated[b].cpu().double(), *(r.transpose(0, 1) for r in rows), D ** -0.5)
            R.assert_rows(out[b], ref, slack, f"step {step}, slot {b}")
        if packed:
            assert (out[2] == 0).all()
    assert int(err.item()) == 0 and pos.tolist() == position == kv_len.tolist()
    for got, want in zip(gpu, cpu):
        assert torch.equal(R.bits(got), R.bits(want))
