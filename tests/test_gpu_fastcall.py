"""The calls marshalled in C++ give what the same calls give through the Python binding, bit
for bit, and whatever they do not know goes on to the Python binding's checks."""
import pytest
import torch

import blockwise_attention_gb300 as ba
from blockwise_attention_gb300 import _lib

pytestmark = pytest.mark.gpu


def rnd(*shape, dtype=torch.bfloat16, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def tokens_first(B, H, T, d, **kw):
    """(B, H, T, d) as a view of (B, T, H, d)."""
    return rnd(B, T, H, d, **kw).transpose(1, 2)


def padding(B, L):
    m = torch.zeros(B, L + 5, dtype=torch.uint8, device="cuda")[:, :L]
    m[0, L // 2:] = 1
    return m


def cache_of(k, v, S):
    c = ba.KV4Cache.empty(k.shape[0], k.shape[1], S, k.shape[3], k_exp=1, v_exp=-1)
    return ba.kv4_append(c, k, v)


def window_fwd(dtype):
    q, k, v = rnd(2, 4, 37, 64, dtype=dtype), tokens_first(2, 2, 70, 64, dtype=dtype), tokens_first(2, 2, 70, 64, dtype=dtype, seed=1)
    return ba.attn_window_fwd(q, k, v, window=20, sinks=2, q_off=33, key_padding_mask=padding(2, 70), scale=0.2)


def window_bwd(dtype):
    q, k, v = tokens_first(2, 4, 70, 64, dtype=dtype), rnd(2, 2, 70, 64, dtype=dtype), rnd(2, 2, 70, 64, dtype=dtype, seed=1)
    out, lse = ba.attn_window_fwd(q, k, v, window=20, sinks=2)
    return ba.attn_window_bwd(q, k, v, out, rnd(2, 4, 70, 64, dtype=dtype, seed=2), lse, window=20, sinks=2)


def window_decode(dtype):
    q, k, v = rnd(3, 4, 1, 64, dtype=dtype), rnd(3, 2, 300, 64, dtype=dtype), rnd(3, 2, 300, 64, dtype=dtype, seed=1)
    lengths = torch.tensor([300, 0, 17], dtype=torch.int32, device="cuda")
    return ba.attn_window_decode_fwd(q, k, v, window=100, sinks=3, lengths=lengths)


def append(dtype):
    c = cache_of(tokens_first(2, 2, 40, 64, dtype=dtype), rnd(2, 2, 40, 64, dtype=dtype, seed=1), 50)
    start, counts = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([45, 3], [4, 0]))
    ba.kv4_append(c, rnd(2, 2, 9, 64, dtype=dtype, seed=3), rnd(2, 2, 9, 64, dtype=dtype, seed=4), start=start, counts=counts)
    return c.k_codes, c.k_scales, c.v_codes, c.v_scales


def read(dtype):
    return ba.kv4_read(cache_of(rnd(2, 2, 40, 128), rnd(2, 2, 40, 128, seed=1), 50), 45, first=2, dtype=dtype)


def decode_kv4(dtype):
    c = cache_of(rnd(2, 2, 40, 128), rnd(2, 2, 40, 128, seed=1), 50)
    lengths = torch.tensor([40, 7], dtype=torch.int32, device="cuda")
    return ba.attn_decode_kv4_fwd(rnd(2, 8, 1, 128), c, lengths=lengths, window=30, sinks=1, scale=0.1)


def positions(kind, B, T):
    p = torch.arange(B * (T + 3), dtype=torch.int32, device="cuda").view(B, T + 3)
    return {"none": None, "rows": p[:, :T], "one": p[0, :T], "shared": p[:1, :T].expand(B, T)}[kind]


def norm(kind):
    def run(dtype):
        q, k = tokens_first(3, 4, 19, 64, dtype=dtype), rnd(3, 2, 19, 64, dtype=dtype)
        wq, wk = rnd(64, dtype=torch.float32), rnd(64, dtype=torch.float32, seed=1)
        kw = dict(positions=positions(kind, 3, 19), base=5e5, pos_scale=0.5)
        dy = rnd(3, 4, 19, 64, dtype=torch.float32), rnd(3, 2, 19, 64, dtype=torch.float32, seed=1)
        return *ba.qk_norm_rope_fwd(q, k, wq, wk, **kw), *ba.qk_norm_rope_bwd(q, k, wq, wk, *dy, **kw)
    run.__name__ = f"norm_{kind}"
    return run


CALLS = [window_fwd, window_bwd, window_decode, append, read, decode_kv4, *map(norm, ("none", "rows", "one", "shared"))]


class Counted:
    """The module, with the answers of its functions counted."""

    def __init__(self, fast):
        self.fast, self.answers = fast, []

    def __getattr__(self, name):
        def call(*args):
            r = getattr(self.fast, name)(*args)
            self.answers.append((name, r is not None))
            return r
        return call


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("call", CALLS, ids=lambda f: f.__name__)
def test_same_bits_both_ways(call, dtype, monkeypatch):
    _lib.load()
    if _lib._fast is None:
        pytest.skip("the call marshalling could not be built")
    counted = Counted(_lib._fast)
    monkeypatch.setattr(_lib, "_fast", counted)
    fast = call(dtype)
    assert counted.answers and all(ok for _, ok in counted.answers), counted.answers
    monkeypatch.setattr(_lib, "_fast", None)
    slow = call(dtype)
    assert len(fast) == len(slow)
    for a, b in zip(fast, slow):
        assert a.shape == b.shape and a.dtype == b.dtype and a.device == b.device
        assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def test_on_the_current_stream_and_in_a_graph():
    q, k, v = rnd(2, 4, 1, 64), rnd(2, 2, 300, 64), rnd(2, 2, 300, 64, seed=1)
    want = ba.attn_window_decode_fwd(q, k, v, window=100)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out, lse = ba.attn_window_decode_fwd(q, k, v, window=100)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, lse = ba.attn_window_decode_fwd(q, k, v, window=100)
    q.copy_(rnd(2, 4, 1, 64, seed=9))
    g.replay()
    want = ba.attn_window_decode_fwd(q, k, v, window=100)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("change, error", [
    (dict(window=0), ValueError), (dict(window=1 << 31), ValueError), (dict(window=1.5), ValueError), (dict(sinks=-1), ValueError),
    (dict(lengths=torch.zeros(2, dtype=torch.int64)), ValueError), (dict(k=(2, 3, 300, 64)), ValueError),
    (dict(k=(1, 2, 300, 64)), ValueError), (dict(q=(2, 4, 2, 64)), ValueError), (dict(q=(2, 4, 64)), ValueError),
    (dict(q=(2, 4, 1, 80), k=(2, 2, 300, 80)), _lib.BlockAttnError),
])
def test_refusals_stay(change, error):
    q, k = rnd(*change.pop("q", (2, 4, 1, 64))), rnd(*change.pop("k", (2, 2, 300, 64)))
    if "lengths" in change:
        change["lengths"] = change["lengths"].cuda()
    with pytest.raises(error):
        ba.attn_window_decode_fwd(q, k, k, **{"window": 8, **change})


def test_dtypes_and_whole_floats_go_the_python_way():
    q, k = rnd(2, 4, 1, 64), rnd(2, 2, 300, 64)
    with pytest.raises(TypeError):
        ba.attn_window_decode_fwd(q, k.float(), k.float(), window=8)
    with pytest.raises(TypeError):
        ba.attn_window_decode_fwd(q.half(), k.half(), k.half(), window=8)
    a, b = ba.attn_window_decode_fwd(q, k, k, window=8.0, scale=1), ba.attn_window_decode_fwd(q, k, k, window=8, scale=1.0)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_threads_on_streams_of_their_own():
    """Host threads that call at once, each on its stream and with its own sizes and rotation base."""
    import threading
    n, want, got = 4, [], [None] * 4
    args = [(rnd(2, 4, 1, 64, seed=i), rnd(2, 2, 100 + 50 * i, 64, seed=i), rnd(64, dtype=torch.float32, seed=i)) for i in range(n)]

    def work(q, k, w, i):
        y, _ = ba.qk_norm_rope_fwd(q, k[:, :, :1], w, w, base=1000.0 * (i + 1))
        out, lse = ba.attn_window_decode_fwd(y, k, k, window=30 + i)
        c = ba.kv4_append(ba.KV4Cache.empty(2, 2, 64, 64), k[:, :, :64], k[:, :, :64])
        return out, lse, *ba.attn_decode_kv4_fwd(y, c)

    for i, a in enumerate(args):
        want.append(work(*a, i))
    torch.cuda.synchronize()

    def run(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(50):
                got[i] = work(*args[i], i)
        s.synchronize()
    threads = [threading.Thread(target=run, args=(i,)) for i in range(n)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    for w, g in zip(want, got):
        assert g is not None and all(torch.equal(a, b) for a, b in zip(w, g))


class Windowed(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v):
        out, lse = ba.attn_window_fwd(q, k, v, window=20, sinks=1)
        ctx.save_for_backward(q, k, v, out, lse)
        return out

    @staticmethod
    def backward(ctx, g):
        q, k, v, out, lse = ctx.saved_tensors
        return ba.attn_window_bwd(q, k, v, out, g.contiguous(), lse, window=20, sinks=1)


def test_parameters_autograd_and_inference_mode():
    q, k, v = (torch.nn.Parameter(rnd(1, H, 60, 64, dtype=torch.float32, seed=H)) for H in (4, 2, 2))
    Windowed.apply(q, k, v).square().sum().backward()
    out, lse = ba.attn_window_fwd(q.detach(), k.detach(), v.detach(), window=20, sinks=1)
    want = ba.attn_window_bwd(q.detach(), k.detach(), v.detach(), out, 2 * out, lse, window=20, sinks=1)
    assert all(torch.equal(a.grad, b) for a, b in zip((q, k, v), want))
    with torch.inference_mode():
        o2, l2 = ba.attn_window_fwd(q, k, v, window=20, sinks=1)
        assert o2.is_inference() and torch.equal(o2, out) and torch.equal(l2, lse)
