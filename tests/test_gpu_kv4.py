"""The KV cache held in 4 bits: kv4_append and kv4_read bit for bit against the format's
definition in 64 bits, attn_decode_kv4_fwd against plain 64-bit attention over the values
that the cache holds."""
import math

import pytest
import torch

import blockwise_attention_gb300 as ba
from tests import window_ref as ref

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
GRID = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
P_STEP = 2.0 ** -11 + 2.0 ** -20   # p in fp16 times 2^11: half a step, and what the smallest lose


def rand(shape, dtype, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def nearest(x, grid):
    """Index of the nearest grid value (ascending), ties to the even index, saturating; x >= 0 in double."""
    g = torch.tensor(grid, dtype=torch.double, device=x.device)
    hi = torch.searchsorted(g, x.contiguous()).clamp(1, len(grid) - 1)
    lo = hi - 1
    a, b = x - g[lo], g[hi] - x
    return torch.where((a < b) | ((a == b) & (lo % 2 == 0)), lo, hi)


E4M3 = [(m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)) for e in range(16) for m in range(8)][:127]


def quantise(x, exp):
    """codes (.., d), scale bytes (.., d / 16) and values (.., d), by the definition."""
    a = x.double().unflatten(-1, (-1, 16)) * 2.0 ** -exp
    a = torch.where(a.isnan(), torch.full_like(a, 1e300), a).clamp(-1e300, 1e300)
    sb = nearest(a.abs().amax(-1) / 6, E4M3)
    s = torch.tensor(E4M3, dtype=torch.double, device=x.device)[sb][..., None]
    c = torch.where(s > 0, nearest(a.abs() / s.clamp(min=1e-300), GRID), torch.zeros((), dtype=torch.long, device=x.device))
    val = torch.tensor(GRID, dtype=torch.double, device=x.device)[c] * s * 2.0 ** exp
    return c.flatten(-2), sb, torch.where(a < 0, -val, val).flatten(-2)


def codes_of(cache_codes):
    return torch.stack((cache_codes & 15, cache_codes >> 4), -1).flatten(-2).long()


@pytest.mark.parametrize("dt,d", [("bf16", 128), ("bf16", 64), ("f32", 128), ("f32", 64)])
@pytest.mark.parametrize("exps,std", [((0, 0), 1.0), ((-6, 5), 0.02), ((0, 0), 1e-3), ((0, 0), 3000.0), ((90, -90), 1.0)])
def test_append_and_read_are_the_format(dt, d, exps, std):
    B, H, T, S = 2, 3, 37, 50
    k, v = rand((B, H, T, d), DT[dt], 1, std), rand((B, H, T, d), DT[dt], 2, std)
    k[0, 0, 0] = 0
    k[0, 0, 1, :16] = 0
    cache = ba.KV4Cache.empty(B, H, S, d, k_exp=exps[0], v_exp=exps[1])
    ba.kv4_append(cache, k, v)
    for x, codes, scales, exp, got in zip((k, v), (cache.k_codes, cache.v_codes), (cache.k_scales, cache.v_scales), exps,
                                          ba.kv4_read(cache, T, dtype=torch.float32)):
        c, sb, val = quantise(x, exp)
        assert torch.equal(scales[:, :, :T].long(), sb)
        assert torch.equal(codes_of(codes[:, :, :T]) & 7, c)
        assert torch.equal(got.double(), val)
    for a, b in zip(ba.kv4_read(cache, T), ba.kv4_read(cache, T, dtype=torch.float32)):
        assert torch.equal(a.float(), b)   # bf16 holds them exactly


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_values_at_and_next_to_every_border(dt):
    """For every scale: each halfway point of the code grid, and the values on either side of it."""
    scale = torch.tensor(E4M3[8:126], dtype=torch.double)   # normal scales (their largest codes stay exact in bf16)
    mids = torch.tensor([(a + b) / 2 for a, b in zip(GRID, GRID[1:])], dtype=torch.double)
    rows = []
    for s in scale:
        x = (mids * s).to(DT[dt])
        up, down = torch.nextafter(x, torch.full_like(x, math.inf)), torch.nextafter(x, torch.zeros_like(x))
        block = torch.zeros(64, dtype=DT[dt])
        for i, part in enumerate((x, up, down)):
            block[16 * i] = 6 * s     # fixes the block's scale
            block[16 * i + 1:16 * i + 8] = part
            block[16 * i + 8:16 * i + 15] = -part
        # the scale's own border: maxima next to six times halfway points of the scale grid
        block[48] = 6 * s * (1 + 1 / 32)
        rows.append(block)
    x = torch.stack(rows).cuda()[None, None]
    cache = ba.KV4Cache.empty(1, 1, x.shape[2], 64)
    ba.kv4_append(cache, x, x)
    c, sb, val = quantise(x, 0)
    assert torch.equal(cache.k_scales.long(), sb) and torch.equal(codes_of(cache.k_codes) & 7, c)
    assert torch.equal(ba.kv4_read(cache, x.shape[2], dtype=torch.float32)[0].double(), val)


@pytest.mark.parametrize("exp", [0, -100, 100, -3])
def test_not_finite_and_huge_values_saturate(exp):
    x = rand((1, 1, 5, 64), torch.float32, 3) * 2.0 ** exp
    x[0, 0, 0, 5], x[0, 0, 1, 20], x[0, 0, 2, 40] = math.inf, -math.inf, math.nan
    x[0, 0, 3, 7], x[0, 0, 3, 33] = -3.4e38, 3.4e38
    x[0, 0, 4] *= -1e4
    cache = ba.KV4Cache.empty(1, 1, 5, 64, k_exp=exp, v_exp=exp)
    ba.kv4_append(cache, x, x)
    assert torch.equal(ba.kv4_read(cache, 5, dtype=torch.float32)[1].double(), quantise(x, exp)[2])


def test_append_starts_counts_and_leaves_the_rest():
    """Ragged chunks: rows behind counts and slots outside the cache are not written, others keep theirs."""
    B, H, T, S, d = 5, 2, 20, 60, 64
    fill = 0xA7
    new = lambda n: torch.full((B, H, S, n), fill, dtype=torch.uint8, device="cuda")  # noqa: E731
    cache = ba.KV4Cache(new(32), new(4), new(32), new(4))
    start = torch.tensor([0, 7, 50, -5, 100], dtype=torch.int32, device="cuda")
    counts = torch.tensor([20, 0, 30, 12, 20], dtype=torch.int32, device="cuda")
    k, v = rand((B, T, H, d), torch.bfloat16, 4).permute(0, 2, 1, 3), rand((B, T, H, d), torch.bfloat16, 5).permute(0, 2, 1, 3)
    ba.kv4_append(cache, k, v, start=start, counts=counts)
    want_c, want_s = new(32), new(4)
    c, sb, _ = quantise(v, 0)
    c = c + 8 * (v < 0)
    packed = (c[..., 0::2] | c[..., 1::2] << 4).to(torch.uint8)
    for b in range(B):
        for t in range(min(T, int(counts[b]))):
            slot = int(start[b]) + t
            if 0 <= slot < S:
                want_c[b, :, slot], want_s[b, :, slot] = packed[b, :, t], sb[b, :, t].to(torch.uint8)
    assert torch.equal(cache.v_scales, want_s)
    assert torch.equal(codes_of(cache.v_codes) & 7, codes_of(want_c) & 7)
    assert torch.equal(cache.v_codes[:, :, 55:][:2], want_c[:, :, 55:][:2])


def filled(B, H, S, d, seed, exps=(0, 0), std=1.0):
    cache = ba.KV4Cache.empty(B, H, S, d, k_exp=exps[0], v_exp=exps[1])
    k, v = rand((B, H, S, d), torch.float32, seed, std), rand((B, H, S, d), torch.float32, seed + 1, std)
    ba.kv4_append(cache, k * 2.0 ** exps[0], v * 2.0 ** exps[1])
    return cache


def check(q, cache, lengths, window, sinks, label, **kw):
    B, H, S, d = cache.shape
    k, v = (t.double() for t in ba.kv4_read(cache, S, dtype=torch.float32))
    lens = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    out, lse = ba.attn_decode_kv4_fwd(q, cache, lengths=lens, window=window, sinks=sinks, **kw)
    full = torch.full((B,), S, device="cuda") if lens is None else lens
    ref.check_forward(out, lse, q, k, v, ref.visible_decode(full, S, window, sinks, "cuda"), label=label, p_step=P_STEP)
    return out, lse


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(3, 3), (8, 2), (15, 3), (9, 1), (16, 1), (40, 1)])
def test_decode_groups_lengths_windows(d, Hq, Hkv):
    S, lengths = 900, [900, 1, 0, 333, 17, 9000, -3]
    B = len(lengths)
    cache = filled(B, Hkv, S, d, 6)
    for b, n in enumerate(lengths):   # slots behind a sequence are never read: NaN scales
        cache.k_scales[b, :, max(0, min(n, S)):] = 0x7f
        cache.v_scales[b, :, max(0, min(n, S)):] = 0x7f
    q = rand((B, Hq, 1, d), torch.bfloat16, 8)
    for window, sinks in ((0, 0), (0, 9), (1, 0), (130, 4), (5000, 7), (20, 320)):
        lens = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        out, lse = ba.attn_decode_kv4_fwd(q, cache, lengths=lens, window=window, sinks=sinks)
        k, v = ba.kv4_read(cache, S, dtype=torch.float32)
        ref.check_forward(out, lse, q, k, v, ref.visible_decode(lens, S, window, sinks, "cuda"), p_step=P_STEP,
                          label=f"{d} {Hq}/{Hkv} {window} {sinks}")
        assert (out[2] == 0).all() and (lse[2] == -math.inf).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("S", [1, 2, 15, 16, 17, 64, 65, 1000, 30000])
def test_decode_cache_sizes(d, S):
    check(rand((2, 8, 1, d), torch.bfloat16, 9), filled(2, 2, S, d, 10), None, 0, 0, f"S={S}")


@pytest.mark.parametrize("q_std,exps", [(1e-20, (0, 0)), (30.0, (0, 0)), (1e18, (-60, 3)), (1e-15, (50, -9))])
def test_decode_magnitudes(q_std, exps):
    """Queries far from one (they are scaled before their conversion) and scaled tensors."""
    check(rand((2, 4, 1, 128), torch.bfloat16, 11, q_std), filled(2, 2, 700, 128, 12, exps), [700, 55], 0, 0, f"{q_std} {exps}")


def test_decode_many_small_probabilities():
    """One key far above 60000 others that together weigh as much: p far below the largest keeps its part."""
    S, d = 60001, 64
    k = torch.zeros((1, 1, S, d), device="cuda")
    k[0, 0, 7, :] = 2.0
    cache = ba.KV4Cache.empty(1, 1, S, d)
    v = rand((1, 1, S, d), torch.float32, 13).abs()
    ba.kv4_append(cache, k, v)
    q = torch.full((1, 2, 1, d), 11.0 / 16, device="cuda", dtype=torch.bfloat16)   # score 11 = ln 60000
    check(q, cache, None, 0, 0, "small p", out_dtype=torch.float32)


def test_prompt_then_tokens_as_served():
    """Prompt written, chunk read back for the prompt form, then tokens appended and attended: as one path,
    eagerly and from one captured graph."""
    B, Hq, Hkv, d, P, S = 2, 8, 2, 128, 300, 340
    cache = ba.KV4Cache.empty(B, Hkv, S, d)
    k, v = rand((B, Hkv, S, d), torch.bfloat16, 14), rand((B, Hkv, S, d), torch.bfloat16, 15)
    ba.kv4_append(cache, k[:, :, :P], v[:, :, :P])
    pk, pv = ba.kv4_read(cache, P)
    q = rand((B, Hq, 50, d), torch.bfloat16, 16)
    out, lse = ba.attn_window_fwd(q, pk, pv, window=100, sinks=4, q_off=P - 50)
    ref.check_forward(out, lse, q, pk, pv, ref.visible(50, P, P - 50, 100, 4, None, "cuda"), label="prompt")
    lens = torch.full((B,), P, dtype=torch.int32, device="cuda")
    start = lens - 1
    nq, nk, nv = rand((B, Hq, 1, d), torch.bfloat16, 17), k[:, :, P:P + 1].clone(), v[:, :, P:P + 1].clone()

    def step():
        start.add_(1)
        lens.add_(1)
        ba.kv4_append(cache, nk, nv, start=start)
        return ba.attn_decode_kv4_fwd(nq, cache, lengths=lens, window=100, sinks=4)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for t in range(2, 12):
        nq.copy_(rand(nq.shape, torch.bfloat16, 20 + t))
        nk.copy_(k[:, :, P + t:P + t + 1])
        nv.copy_(v[:, :, P + t:P + t + 1])
        graph.replay()
        n = P + t
        assert int(lens[0]) == n
        ck, cv = ba.kv4_read(cache, n, dtype=torch.float32)
        seen = ref.visible_decode(lens, n, 100, 4, "cuda")
        ref.check_forward(*got, nq, ck, cv, seen, label=f"token {t}", p_step=P_STEP)


def test_empty_caches_chunks_and_sequences():
    cache = ba.KV4Cache.empty(2, 2, 0, 64)
    x = rand((2, 2, 3, 64), torch.bfloat16, 40)
    ba.kv4_append(cache, x, x)
    out, lse = ba.attn_decode_kv4_fwd(x[:, :, :1], cache)
    assert (out == 0).all() and (lse == -math.inf).all()
    cache = filled(2, 2, 9, 64, 41)
    before = [t.clone() for t in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales)]
    ba.kv4_append(cache, x[:, :, :0], x[:, :, :0])
    ba.kv4_append(cache, x, x, counts=torch.zeros(2, dtype=torch.int32, device="cuda"))
    ba.kv4_append(cache, x, x, start=torch.tensor([-3, 9], dtype=torch.int32, device="cuda"))
    assert all(torch.equal(a, b) for a, b in zip(before, (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales)))
    assert ba.kv4_read(cache, 0)[0].shape == (2, 2, 0, 64)
    many = filled(300, 1, 50, 64, 42)
    check(rand((300, 2, 1, 64), torch.bfloat16, 43), many, [(b * 7) % 51 for b in range(300)], 0, 0, "many sequences")


def test_long_chunks_with_any_strides():
    """Chunks of many rows into a cache stored (B, S, H, ..), starts that are not multiples of anything."""
    B, H, T, S, d = 2, 3, 500, 777, 128
    st = [torch.zeros((B, S, H, n), dtype=torch.uint8, device="cuda").permute(0, 2, 1, 3) for n in (64, 8, 64, 8)]
    cache = ba.KV4Cache(*st)
    k, v = (rand((B, T, H, d), torch.float32, 44 + i).permute(0, 2, 1, 3) for i in range(2))
    start = torch.tensor([277, 11], dtype=torch.int32, device="cuda")
    ba.kv4_append(cache, k, v, start=start)
    got = ba.kv4_read(cache, S, dtype=torch.float32)
    for x, y in zip((k, v), got):
        for b in range(B):
            n = int(start[b])
            assert torch.equal(y[b, :, n:n + T].double(), quantise(x[b], 0)[2])
            assert (y[b, :, :n] == 0).all() and (y[b, :, n + T:] == 0).all()


def test_binding_refusals():
    cache = ba.KV4Cache.empty(2, 2, 40, 64)
    x = rand((2, 2, 3, 64), torch.bfloat16, 30)
    for bad in (lambda: ba.kv4_append(cache, x, x[:, :, :2]), lambda: ba.kv4_append(cache, x[:, :1], x[:, :1]),
                lambda: ba.kv4_append(cache, x, x, start=torch.zeros(2, device="cuda")),
                lambda: ba.kv4_append(cache, x, x, counts=torch.zeros(3, dtype=torch.int32, device="cuda")),
                lambda: ba.KV4Cache(cache.k_codes, cache.k_scales, cache.v_codes[:, :, :39], cache.v_scales),
                lambda: ba.KV4Cache(cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales, k_exp=101),
                lambda: ba.attn_decode_kv4_fwd(x[:, :, :1].expand(2, 2, 2, 64), cache),
                lambda: ba.attn_decode_kv4_fwd(x[:1, :, :1], cache)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: ba.kv4_read(cache, 41), lambda: ba.kv4_read(cache, 10, first=31),
                lambda: ba.attn_decode_kv4_fwd(x[:, :, :1].float(), cache)):
        with pytest.raises(ba.BlockAttnError):
            bad()
