"""Attention with a sliding window and sinks (attn_window_fwd / attn_window_bwd) against
a plain 64-bit statement: lengths from one token, windows from one key, odd sizes, grouped
heads, offsets, padding that leaves rows empty or holds NaN, strided inputs, and the sink
tiles' split over the queries.  Bounds: tests/window_ref.py."""
import math

import pytest
import torch

import blockwise_attention_gb300 as ba
from tests import window_ref as ref

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def rand(shape, dtype, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def inputs(B, Hq, Hkv, Lq, Lk, d, dt, seed=0):
    return (rand((B, Hq, Lq, d), DT[dt], seed), rand((B, Hkv, Lk, d), DT[dt], seed + 1),
            rand((B, Hkv, Lk, d), DT[dt], seed + 2), rand((B, Hq, Lq, d), DT[dt], seed + 3))


def both(q, k, v, g, *, window, sinks, q_off=0, kpm=None, label=""):
    at = dict(window=window, sinks=sinks, q_off=q_off, key_padding_mask=kpm)
    seen = ref.visible(q.shape[2], k.shape[2], q_off, window, sinks, kpm, q.device)
    out, lse = ba.attn_window_fwd(q, k, v, **at)
    ref.check_forward(out, lse, q, k, v, seen, label=label)
    grads = ba.attn_window_bwd(q, k, v, out, g, lse, **at)
    assert grads[0].dtype == q.dtype
    ref.check_backward(grads, q, k, v, out, g, lse, seen, label=label)
    return out, lse, grads


@pytest.mark.parametrize("dt,d", [("bf16", 128), ("bf16", 64), ("f32", 64), ("f32", 128), ("bf16", 32), ("f32", 16)])
@pytest.mark.parametrize("L,window,sinks", [(1, 1, 0), (1, 5, 3), (2, 1, 1), (127, 64, 0), (129, 1, 0), (129, 128, 1),
                                            (256, 129, 4), (300, 300, 7), (301, 2, 130), (513, 200, 4), (640, 1000, 4),
                                            (640, 128, 640)])
def test_lengths_windows_sinks(dt, d, L, window, sinks):
    both(*inputs(1, 2, 1, L, L, d, dt), window=window, sinks=sinks, label=f"{dt} d={d} L={L} W={window} s={sinks}")


@pytest.mark.parametrize("dt,d", [("bf16", 128), ("bf16", 64), ("f32", 64)])
@pytest.mark.parametrize("Hq,Hkv", [(4, 4), (8, 2), (5, 1), (6, 3)])
def test_grouped_heads_many_tiles(dt, d, Hq, Hkv):
    both(*inputs(2, Hq, Hkv, 1111, 1111, d, dt, 10), window=257, sinks=4, label=f"groups {dt} {Hq}/{Hkv}")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("q_off,Lk", [(1, 301), (77, 377), (500, 800), (500, 640), (900, 300), (300, 0), (1000, 2)])
def test_chunks_behind_a_prefix(dt, q_off, Lk):
    """Queries at q_off .. q_off + 299; caches that end at, before and far before them."""
    both(*inputs(1, 4, 2, 300, Lk, 64, dt, 20), window=150, sinks=5, q_off=q_off, label=f"chunk {q_off} {Lk}")


@pytest.mark.parametrize("dt,d", [("bf16", 128), ("bf16", 64), ("f32", 64)])
@pytest.mark.parametrize("fill", [0.0, math.inf, math.nan])
def test_padding_empties_rows_and_hides_what_it_holds(dt, d, fill):
    """Left padding over the sinks and past the first windows, holes, a batch item wholly padded."""
    B, L = 4, 520
    q, k, v, g = inputs(B, 4, 2, L, L, d, dt, 30)
    kpm = torch.zeros((B, L), dtype=torch.uint8, device="cuda")
    kpm[0, :200] = 1
    kpm[1, 100:140] = 1
    kpm[1, 511:] = 1
    kpm[2] = 1
    kpm[3, ::3] = 1
    if fill:
        for b in range(B):
            k[b, :, kpm[b] == 1] = fill
            v[b, :, kpm[b] == 1] = fill
    out, lse, grads = both(q, k, v, g, window=50, sinks=4, kpm=kpm, label=f"pad {dt} {fill}")
    assert (lse[2] == -math.inf).all() and (grads[0][2] == 0).all() and (grads[1][2] == 0).all()


@pytest.mark.parametrize("dt,d", [("bf16", 128), ("f32", 32)])
def test_strided_inputs_and_any_alignment(dt, d):
    """Views of a packed projection, and rows that TMA cannot read (odd strides: the CUDA-core kernels)."""
    B, Hq, Hkv, L = 2, 4, 2, 333
    qkv = rand((B, L, Hq + 2 * Hkv, d), DT[dt], 40)
    q, k, v = (t.permute(0, 2, 1, 3) for t in qkv.split([Hq, Hkv, Hkv], dim=2))
    both(q, k, v, rand((B, L, Hq, d), DT[dt], 41).permute(0, 2, 1, 3), window=100, sinks=2, label="packed")
    odd = [rand((B, H, L, d + 3), DT[dt], 42 + i)[..., 1:d + 1] for i, H in enumerate((Hq, Hkv, Hkv, Hq))]
    both(*odd, window=100, sinks=2, label="odd strides")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_broadcast_inputs_and_empty_sides(dt):
    """Keys shared by the batch (stride 0), a cotangent of one value, and axes of length zero."""
    q, k, v, g = inputs(3, 4, 2, 150, 150, 64, dt, 45)
    both(q, k[:1].expand(3, -1, -1, -1), v[:1].expand(3, -1, -1, -1), g, window=60, sinks=2, label="batch shared")
    both(q, k, v, g[:1, :1, :1, :1].expand_as(g).contiguous(), window=60, sinks=2, label="one value")
    both(q, k[:, :1].expand(3, 2, 150, 64), v, g, window=60, sinks=2, label="head shared")
    for q0, k0 in ((q[:0], k[:0]), (q[:, :, :0], k), (q, k[:, :, :0])):
        out, lse = ba.attn_window_fwd(q0, k0, k0, window=9)
        dq, dk, dv = ba.attn_window_bwd(q0, k0, k0, out, out, lse, window=9)
        assert out.shape == q0.shape and (out == 0).all() and (lse == -math.inf).all()
        assert dq.shape == q0.shape and dk.shape == k0.shape and (dq == 0).all() and (dk == 0).all() and (dv == 0).all()


@pytest.mark.parametrize("dt,d", [("bf16", 64), ("f32", 64)])
def test_sink_tiles_split_over_long_sequences(dt, d):
    """A window far shorter than the sequence: the sinks' gradients come from many chunks."""
    q, k, v, g = inputs(1, 2, 1, 2900, 2900, d, dt, 50)
    _, _, first = both(q, k, v, g, window=64, sinks=140, label="sink split")
    again = ba.attn_window_bwd(q, k, v, *_saved(q, k, v, g, 64, 140), window=64, sinks=140)
    assert all(torch.equal(a, b) for a, b in zip(first, again))   # no atomics: equal bits


def _saved(q, k, v, g, window, sinks):
    out, lse = ba.attn_window_fwd(q, k, v, window=window, sinks=sinks)
    return out, g, lse


def test_wide_window_is_causal_attention():
    q, k, v, g = inputs(1, 2, 2, 700, 700, 128, "bf16", 60)
    out, lse = ba.attn_window_fwd(q, k, v, window=2 ** 31 - 1, sinks=2 ** 31 - 1)
    o2, l2 = ba.attn_block_fwd(q, k, v, causal=True)
    assert torch.equal(out, o2) and torch.equal(lse, l2)


def test_output_types_and_buffers():
    q, k, v, g = inputs(1, 4, 2, 200, 200, 64, "bf16", 70)
    seen = ref.visible(200, 200, 0, 50, 2, None, "cuda")
    out, lse = ba.attn_window_fwd(q, k, v, window=50, sinks=2, out_dtype=torch.float32)
    ref.check_forward(out, lse, q, k, v, seen, label="f32 out")
    out, lse = ba.attn_window_fwd(q, k, v, window=50, sinks=2)
    bufs = [torch.full(t.shape, math.nan, device="cuda") for t in (q, k, v)]
    ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    grads = ba.attn_window_bwd(q, k, v, out, g, lse, window=50, sinks=2, dq=bufs[0], dk=bufs[1], dv=bufs[2], workspace=ws)
    assert all(a is b for a, b in zip(grads, bufs))
    ref.check_backward(grads, q, k, v, out, g, lse, seen, label="f32 grads")


def test_gradient_against_differences():
    """Central differences of L = sum(out * g) along random directions, in fp32: step h, the
    loss rounded to about 2^-24 |terms| and the third derivative's h^2 term."""
    q, k, v, g = inputs(1, 4, 2, 150, 150, 32, "f32", 80)
    at = dict(window=40, sinks=3)
    out, lse = ba.attn_window_fwd(q, k, v, **at)
    grads = ba.attn_window_bwd(q, k, v, out, g, lse, **at)
    h = 2.0 ** -6
    for i in range(3):
        x = [q, k, v]
        u = rand(x[i].shape, torch.float32, 90 + i)
        u /= u.norm()
        lo, hi = list(x), list(x)
        hi[i], lo[i] = x[i] + h * u, x[i] - h * u
        f = [float((ba.attn_window_fwd(*y, **at)[0].double() * g.double()).sum()) for y in (hi, lo)]
        got, want = float((grads[i].double() * u.double()).sum()), (f[0] - f[1]) / (2 * h)
        # the loss's own error: n terms of relative 2^-20, in random sum sqrt(n); h^2 times a third derivative of order |grad|
        tol = 2.0 ** -20 * math.sqrt(g.numel()) / h + 4 * h * h * float(grads[i].norm())
        assert abs(got - want) <= tol, (i, got, want, tol)


def test_captured_and_replayed_on_a_side_stream():
    q, k, v, g = inputs(1, 8, 2, 900, 900, 64, "bf16", 100)
    at = dict(window=200, sinks=4)

    def step():
        out, lse = ba.attn_window_fwd(q, k, v, **at)
        return (out, lse, *ba.attn_window_bwd(q, k, v, out, g, lse, **at))

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got = step()
    q.copy_(q.flip(2))
    want2 = step()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want2))
    assert not torch.equal(want[0], want2[0])
    # outputs allocated by a call that names its stream belong to that stream
    out, lse = ba.attn_window_fwd(q, k, v, **at, stream=side)
    side.synchronize()
    assert torch.equal(out, want2[0])


def test_binding_refusals():
    q, k, v, g = inputs(1, 4, 2, 40, 40, 64, "bf16", 110)
    out, lse = ba.attn_window_fwd(q, k, v, window=8)
    for bad in (dict(window=0), dict(window=8, sinks=-1), dict(window=8, q_off=-1), dict(window=2 ** 31)):
        with pytest.raises(ValueError):
            ba.attn_window_fwd(q, k, v, **bad)
    with pytest.raises(ValueError):
        ba.attn_window_fwd(q[:, :3], k, v, window=8)   # 3 query heads over 2 key heads
    with pytest.raises(ValueError):
        ba.attn_window_fwd(q, k, v[:, :, :39], window=8)
    with pytest.raises(TypeError):
        ba.attn_window_fwd(q, k.float(), v.float(), window=8)
    with pytest.raises(ValueError):
        ba.attn_window_fwd(q, k, v, window=8, key_padding_mask=torch.zeros((1, 39), dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        ba.attn_window_bwd(q, k, v, out, g, lse, window=8, dk=torch.empty_like(q))
    with pytest.raises(ba.BlockAttnError):   # a workspace that is too small
        ba.attn_window_bwd(q, k, v, out, g, lse, window=8, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("dt,d", [("bf16", 128), ("bf16", 64), ("f32", 64), ("bf16", 32)])
@pytest.mark.parametrize("q_off,Lk", [(0, 300), (70, 512), (201, 500)])
def test_free_slots_behind_the_last_query(dt, d, q_off, Lk):
    """A chunk of 150 queries on a cache with free slots: NaN and infinities there have no effect."""
    q, k, v, g = inputs(2, 4, 2, 150, Lk, d, dt, 120)
    k[:, :, q_off + 150:], v[:, :, q_off + 150:] = math.nan, math.inf
    _, _, (_, dk, dv) = both(q, k, v, g, window=100, sinks=3, q_off=q_off, label=f"free slots {dt} {q_off}")
    assert (dk[:, :, q_off + 150:] == 0).all() and (dv[:, :, q_off + 150:] == 0).all()
