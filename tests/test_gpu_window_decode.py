"""Single-token attention of grouped heads over a window with sinks
(attn_window_decode_fwd) against a plain 64-bit statement: every head grouping, ragged and
empty sequences, garbage behind the lengths, strided caches, split ranges."""
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


def check(q, k, v, lengths, window, sinks, label="", **kw):
    S = k.shape[2]
    lens = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    out, lse = ba.attn_window_decode_fwd(q, k, v, window=window, sinks=sinks, lengths=lens, **kw)
    full = torch.full((q.shape[0],), S, device="cuda") if lens is None else lens
    ref.check_forward(out, lse, q, k, v, ref.visible_decode(full, S, window, sinks, "cuda"), label=label)
    return out, lse


@pytest.mark.parametrize("dt,d", [("bf16", 128), ("bf16", 64), ("f32", 128), ("f32", 64), ("bf16", 32), ("f32", 16)])
@pytest.mark.parametrize("Hq,Hkv", [(3, 3), (2, 1), (8, 2), (15, 3), (16, 2), (9, 1), (16, 1), (40, 1)])
def test_head_groups_and_ragged_lengths(dt, d, Hq, Hkv):
    S, lengths = 700, [700, 1, 0, 333, 17, 9000, -3]
    B = len(lengths)
    q, k, v = rand((B, Hq, 1, d), DT[dt], 1), rand((B, Hkv, S, d), DT[dt], 2), rand((B, Hkv, S, d), DT[dt], 3)
    for b, n in enumerate(lengths):   # slots behind a sequence are never read
        k[b, :, max(0, min(n, S)):] = math.nan
        v[b, :, max(0, min(n, S)):] = math.inf
    for window, sinks in ((1, 0), (130, 4), (130, 0), (5000, 7), (20, 320)):
        out, lse = check(q, k, v, lengths, window, sinks, f"{dt} {d} {Hq}/{Hkv} W={window} s={sinks}")
        assert (out[2] == 0).all() and (lse[2] == -math.inf).all()


@pytest.mark.parametrize("dt,d", [("bf16", 128), ("bf16", 64), ("f32", 64)])
@pytest.mark.parametrize("S,window", [(1, 1), (2, 2), (63, 64), (64, 64), (65, 65), (513, 513), (5000, 4097), (20000, 20000)])
def test_cache_sizes_and_splits(dt, d, S, window):
    check(rand((2, 8, 1, d), DT[dt], 4), rand((2, 2, S, d), DT[dt], 5), rand((2, 2, S, d), DT[dt], 6), None, window, 3,
          f"{dt} S={S} W={window}")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_empty_caches_batches_and_many_sequences(dt):
    q = rand((2, 4, 1, 64), DT[dt], 30)
    empty = rand((2, 2, 0, 64), DT[dt], 31)
    out, lse = ba.attn_window_decode_fwd(q, empty, empty, window=5, sinks=1)
    assert (out == 0).all() and (lse == -math.inf).all()
    out, lse = ba.attn_window_decode_fwd(q[:0], empty[:0], empty[:0], window=5)
    assert out.shape == (0, 4, 1, 64)
    B, S = 300, 90   # more sequences than the scan takes at a time, most of them short or empty
    lengths = [(b * 37) % 91 if b % 3 else 0 for b in range(B)]
    k, v = rand((1, 2, S, 64), DT[dt], 32).expand(B, -1, -1, -1), rand((B, 2, S, 64), DT[dt], 33)
    check(rand((B, 4, 1, 64), DT[dt], 34), k, v, lengths, 40, 3, "many")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_strided_cache_large_scores_and_out_types(dt):
    """A cache stored (B, S, H, d); scores up to about a hundred (the running maximum moves often)."""
    B, Hq, Hkv, S, d = 3, 8, 2, 1500, 64
    q = rand((B, Hq, 1, d), DT[dt], 7, 12.0)
    k, v = (rand((B, S, Hkv, d), DT[dt], 8 + i).permute(0, 2, 1, 3) for i in range(2))
    check(q, k, v, [1500, 77, 900], 700, 2, "strided")
    out, _ = check(q, k, v, [1500, 77, 900], 700, 2, "f32 out", out_dtype=torch.float32)
    assert out.dtype == torch.float32


def test_ascending_scores_move_the_maximum_every_tile():
    """Keys whose score grows along the cache by more than the lazy bound a tile, and falls."""
    d, S = 128, 2000
    q = torch.zeros((1, 4, 1, d), device="cuda", dtype=torch.bfloat16)
    q[..., 0] = 8.0
    for sign in (1.0, -1.0):
        k = rand((1, 1, S, d), torch.bfloat16, 10)
        k[..., 0] = (sign * torch.arange(S, device="cuda") / 8).to(torch.bfloat16)
        v = rand((1, 1, S, d), torch.bfloat16, 11)
        check(q, k, v, None, S, 0, f"ramp {sign}")


def test_is_the_last_row_of_the_prompt_form():
    q, k, v = rand((2, 8, 1, 64), torch.float32, 12), rand((2, 2, 900, 64), torch.float32, 13), rand((2, 2, 900, 64), torch.float32, 14)
    a = ba.attn_window_decode_fwd(q, k, v, window=200, sinks=4)
    b = ba.attn_window_fwd(q, k, v, window=200, sinks=4, q_off=899)
    assert (a[0] - b[0]).abs().max() <= 2e-6 and (a[1] - b[1]).abs().max() <= 2e-6


def test_captured_with_growing_lengths_and_two_streams():
    """One graph replayed as the sequences grow; two calls at once on two streams."""
    B, S, d = 4, 3000, 128
    q, k, v = rand((B, 8, 1, d), torch.bfloat16, 15), rand((B, 2, S, d), torch.bfloat16, 16), rand((B, 2, S, d), torch.bfloat16, 17)
    lens = torch.tensor([10, 500, 2000, 2990], dtype=torch.int32, device="cuda")
    at = dict(window=600, sinks=4, lengths=lens)
    ba.attn_window_decode_fwd(q, k, v, **at)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = ba.attn_window_decode_fwd(q, k, v, **at)
    for _ in range(3):
        lens += 3
        graph.replay()
        want = ba.attn_window_decode_fwd(q, k, v, **at)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [ba.attn_window_decode_fwd(q, k, v, **at, stream=s) for _ in range(4) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[0]) and torch.equal(l, want[1]) for o, l in outs)


def test_binding_refusals():
    q, k, v = rand((2, 4, 1, 64), torch.bfloat16, 18), rand((2, 2, 50, 64), torch.bfloat16, 19), rand((2, 2, 50, 64), torch.bfloat16, 20)
    lens = torch.tensor([3, 4], dtype=torch.int32, device="cuda")
    for bad in (dict(window=0), dict(window=4, sinks=-1), dict(window=4, lengths=lens.long()), dict(window=4, lengths=lens[:1])):
        with pytest.raises(ValueError):
            ba.attn_window_decode_fwd(q, k, v, **bad)
    with pytest.raises(ValueError):
        ba.attn_window_decode_fwd(q.expand(2, 4, 2, 64), k, v, window=4)
    with pytest.raises(ba.BlockAttnError):   # rows off a 16-byte boundary
        ba.attn_window_decode_fwd(q, *(torch.zeros((2, 2, 50, 65), dtype=torch.bfloat16, device="cuda")[..., 1:] for _ in "kv"),
                                  window=4)
