"""Per-head norm and rotation of queries and keys (qk_norm_rope_fwd / _bwd) against a plain
64-bit statement: types, head dimensions, groups, strides, positions, and the path norm ->
windowed attention -> its gradients.

Bounds (relative to the magnitudes that enter a result).  r: the fp32 sum of d squares is
off by at most d half steps, halved by the root, rsqrt by 2^-22; cos and sin by 2^-22 (the
angle's fraction rounded to fp32, times pi, and the functions' own 2 ulp); a handful of
roundings more.  Then one rounding to the output's type."""
import math

import pytest
import torch

import blockwise_attention_gb300 as ba
from tests import window_ref as ref

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5


def rand(shape, dtype, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def rotate(x, a):
    z = torch.view_as_complex(x.unflatten(-1, (-1, 2)).contiguous()) * torch.polar(torch.ones_like(a), a)
    return torch.view_as_real(z).flatten(-2)


def pairsum(x):   # |x_2c| + |x_2c+1| in both places
    return x.abs().unflatten(-1, (-1, 2)).sum(-1, keepdim=True).expand(*x.shape[:-1], x.shape[-1] // 2, 2).flatten(-2)


def exact(x, w, dy, positions, base, pos_scale=1.0):
    """y, its magnitude, and (dx, |dx| terms, dw, |dw| terms) in double."""
    B, H, T, d = x.shape
    m = torch.arange(T, device="cuda").double()[None] if positions is None else positions.double().reshape(-1, T)
    theta = torch.tensor([base ** (-2.0 * c / d) for c in range(d // 2)], dtype=torch.double, device="cuda")
    a = ((m * pos_scale)[:, None, :, None] * theta).expand(B, H, T, d // 2)
    x, w = x.double(), w.double()
    r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
    n = x * r
    y, ymag = rotate(n * w, a), pairsum(n * w)
    if dy is None:
        return y, ymag
    dz, dzmag = rotate(dy.double(), -a), pairsum(dy.double())
    dn, dnmag = dz * w, dzmag * w.abs()
    dx = r * (dn - n * (dn * n).mean(-1, keepdim=True))
    dxmag = r * (dnmag + n.abs() * (dnmag * n.abs()).mean(-1, keepdim=True))
    return y, ymag, dx, dxmag, (dz * n).sum((0, 1, 2)), (dzmag * n.abs()).sum((0, 1, 2))


def check(got, want, mag, rel, label):
    assert torch.isfinite(got).all(), label
    err = rel * mag
    tol = err + ref.HALF_STEP[got.dtype] * (want.abs() + err) + 1e-37
    bad = (got.double() - want).abs() > tol
    assert not bad.any(), (label, float(((got.double() - want).abs() - tol).max()), int(bad.sum()))


def both(q, k, wq, wk, dyq, dyk, positions=None, base=10000.0, pos_scale=1.0, label=""):
    at = dict(eps=EPS, positions=positions, base=base, pos_scale=pos_scale)
    ys = ba.qk_norm_rope_fwd(q, k, wq, wk, **at)
    *dxs, dwq, dwk = ba.qk_norm_rope_bwd(q, k, wq, wk, dyq, dyk, **at)
    d = q.shape[-1]
    rel = (d / 2 + 8) * 2.0 ** -24 + 2.0 ** -21
    for name, x, w, dy, y, dx, dw in zip("qk", (q, k), (wq, wk), (dyq, dyk), ys, dxs, (dwq, dwk)):
        if x.shape[1] == 0:
            assert (dw == 0).all()
            continue
        e = exact(x, w, dy, positions, base, pos_scale)
        assert y.is_contiguous() and y.dtype == x.dtype and dx.dtype == x.dtype and dw.dtype == torch.float32
        check(y, e[0], e[1], rel, f"{label} y{name}")
        check(dx, e[2], e[3], 2 * rel + d * 2.0 ** -24, f"{label} dx{name}")
        # a thread's chain is at most a few hundred rows here, the blocks' sums are in fp64
        check(dw, e[4], e[5], 2 * rel + 2.0 ** -15, f"{label} dw{name}")
    return ys, dxs


@pytest.mark.parametrize("dt,d", [("bf16", 128), ("bf16", 64), ("bf16", 32), ("bf16", 16), ("f32", 128), ("f32", 64), ("f32", 16)])
@pytest.mark.parametrize("B,Hq,Hkv,T", [(1, 1, 1, 1), (2, 3, 1, 17), (1, 8, 2, 333), (3, 5, 5, 64), (2, 2, 0, 9), (5, 0, 3, 1)])
@pytest.mark.parametrize("w_dt", ["same", "f32"])
def test_types_sizes_groups(dt, d, B, Hq, Hkv, T, w_dt):
    dtype, wd = DT[dt], DT[dt] if w_dt == "same" else torch.float32
    q, k = rand((B, Hq, T, d), dtype, 1, 2.0), rand((B, Hkv, T, d), dtype, 2, 0.1)
    if T > 2:
        q[..., 1, :], k[..., 2, :] = 0, 0   # rows of zeros: r = eps^-1/2
    both(q, k, rand((d,), wd, 3), rand((d,), wd, 4), rand(q.shape, dtype, 5), rand(k.shape, dtype, 6), label=f"{dt} {d}")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_strides_positions_and_fp32_gradients(dt):
    """The packed projection, far positions per sequence and shared, rows off 16 bytes, dy in fp32."""
    B, Hq, Hkv, T, d = 3, 6, 2, 50, 64
    qkv = rand((B, T, Hq + 2 * Hkv, d), DT[dt], 7)
    q, k = qkv[:, :, :Hq].permute(0, 2, 1, 3), qkv[:, :, Hq:Hq + Hkv].permute(0, 2, 1, 3)
    w = rand((d,), DT[dt], 8), rand((d,), DT[dt], 9)
    g = rand((B, T, Hq, d), torch.float32, 10).permute(0, 2, 1, 3), rand((B, Hkv, T, d), torch.float32, 11)
    own = torch.randint(0, 1 << 20, (B, T), device="cuda", dtype=torch.int32)
    for pos in (own, own[0], own[:1].expand(B, T), own.new_zeros((B, T + 3))[:, :T] + 7, None):
        both(q, k, *w, *g, positions=pos, base=500000.0, label="positions")
    both(q, k, *w, *g, positions=own, pos_scale=0.25, label="interpolated")
    odd = rand((B, Hq, T, d + 1), DT[dt], 12)[..., 1:], rand((B, Hkv, T, d + 1), DT[dt], 13)[..., :d]
    both(*odd, *w, *g, label="odd rows")


def test_many_rows_and_one_token_batches():
    d = 128
    w = rand((d,), torch.bfloat16, 14), rand((d,), torch.bfloat16, 15)
    for B, T in ((2, 4100), (300, 1)):
        q, k = rand((B, 4, T, d), torch.bfloat16, 16), rand((B, 2, T, d), torch.bfloat16, 17)
        pos = torch.randint(0, 100000, (B, T), device="cuda", dtype=torch.int32)
        both(q, k, *w, rand(q.shape, torch.bfloat16, 18), rand(k.shape, torch.bfloat16, 19), positions=pos, label=f"{B} {T}")


def test_unit_weights_are_norm_then_rope_apply():
    q, k = rand((2, 4, 100, 64), torch.float32, 20), rand((2, 2, 100, 64), torch.float32, 21)
    one = torch.ones(64, device="cuda")
    yq, yk = ba.qk_norm_rope_fwd(q, k, one, one, eps=EPS)
    for x, y in ((q, yq), (k, yk)):
        want = ba.rope_apply(x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS))
        assert (y - want).abs().max() <= 3e-6


def test_gradient_against_differences():
    """Central differences in fp32 of L = sum(y g): step h, the loss's rounding and an h^2 term."""
    q, k = rand((1, 2, 10, 32), torch.float32, 22), rand((1, 1, 10, 32), torch.float32, 23)
    w = [rand((32,), torch.float32, 24), rand((32,), torch.float32, 25)]
    g = rand(q.shape, torch.float32, 26), rand(k.shape, torch.float32, 27)
    grads = ba.qk_norm_rope_bwd(q, k, *w, *g, eps=EPS)
    h = 2.0 ** -7
    x = [q, k, *w]
    for i in range(4):
        u = rand(x[i].shape, torch.float32, 30 + i)
        u /= u.norm()
        f = []
        for sgn in (1, -1):
            z = list(x)
            z[i] = x[i] + sgn * h * u
            f.append(sum(float((y.double() * gy.double()).sum()) for y, gy in zip(ba.qk_norm_rope_fwd(*z, eps=EPS), g)))
        got, want = float((grads[i].double() * u.double()).sum()), (f[0] - f[1]) / (2 * h)
        tol = 2.0 ** -21 * math.sqrt(q.numel()) * 3 / h + 4 * h * h * float(grads[i].norm())
        assert abs(got - want) <= tol, (i, got, want, tol)


def test_layer_path_norm_attention_and_back():
    """As a training step of a layer runs it: norm and rotation of the packed projection, windowed
    attention, its gradients (fp32) into the norm's; and the same step captured and replayed."""
    B, Hq, Hkv, T, d = 1, 4, 2, 400, 64
    qkv = rand((B, T, Hq + 2 * Hkv, d), torch.bfloat16, 40)
    q, k, v = (t.permute(0, 2, 1, 3) for t in qkv.split([Hq, Hkv, Hkv], dim=2))
    w = rand((d,), torch.bfloat16, 41), rand((d,), torch.bfloat16, 42)
    g = rand((B, Hq, T, d), torch.bfloat16, 43)
    at = dict(window=100, sinks=4)

    def step():
        yq, yk = ba.qk_norm_rope_fwd(q, k, *w, eps=EPS)
        out, lse = ba.attn_window_fwd(yq, yk, v, **at)
        dyq, dyk, dv = ba.attn_window_bwd(yq, yk, v, out, g, lse, **at, grad_dtype=torch.float32)
        return (yq, yk, out, lse, dyq, dyk, dv, *ba.qk_norm_rope_bwd(q, k, *w, dyq, dyk, eps=EPS))

    yq, yk, out, lse, dyq, dyk, dv, dq, dk, dwq, dwk = first = step()
    seen = ref.visible(T, T, 0, 100, 4, None, "cuda")
    ref.check_forward(out, lse, yq, yk, v, seen, label="layer")
    ref.check_backward((dyq, dyk, dv), yq, yk, v, out, g, lse, seen, label="layer")
    rel = 2 * ((d / 2 + 8) * 2.0 ** -24 + 2.0 ** -21) + d * 2.0 ** -24
    for x, wt, dy, dx, dw in ((q, w[0], dyq, dq, dwq), (k, w[1], dyk, dk, dwk)):
        e = exact(x, wt, dy, None, 10000.0)
        check(dx, e[2], e[3], rel, "layer dx")
        check(dw, e[4], e[5], rel + 2.0 ** -15, "layer dw")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = step()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, first))


def test_empty_and_refusals():
    q, k = rand((2, 4, 8, 64), torch.bfloat16, 50), rand((2, 2, 8, 64), torch.bfloat16, 51)
    w = torch.ones(64, device="cuda", dtype=torch.bfloat16)
    e = ba.qk_norm_rope_bwd(q[:, :, :0], k[:, :, :0], w, w, q[:, :, :0], k[:, :, :0])
    assert (e[2] == 0).all() and (e[3] == 0).all()
    pos = torch.zeros(8, dtype=torch.int32, device="cuda")
    for bad in (lambda: ba.qk_norm_rope_fwd(q, k[:1], w, w), lambda: ba.qk_norm_rope_fwd(q, k, w[:32], w),
                lambda: ba.qk_norm_rope_fwd(q, k, w, w, positions=pos.long()), lambda: ba.qk_norm_rope_fwd(q, k, w, w, positions=pos[:7]),
                lambda: ba.qk_norm_rope_bwd(q, k, w, w, q[:, :2], k)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        ba.qk_norm_rope_fwd(q, k, w.half(), w.half())
    for bad in (dict(eps=-1.0), dict(eps=math.nan), dict(base=0.0), dict(pos_scale=-1.0)):
        with pytest.raises(ba.BlockAttnError):
            ba.qk_norm_rope_fwd(q, k, w, w, **bad)
    with pytest.raises(ba.BlockAttnError):   # d
        ba.qk_norm_rope_fwd(q[..., :48], k[..., :48], w[:48], w[:48])
