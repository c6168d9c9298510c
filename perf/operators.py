"""What the language-model operators of this library are timed on, and their plain forms.

Three families, as a decoder uses them next to the ring attention:

* queries and keys normalised per head and rotated to their positions, with the gradients;
* attention with a sliding window and a few first tokens that stay visible (sinks): prompts,
  training steps, and single tokens against a cache;
* a KV cache held in 4 bits (e2m1 codes, one e4m3 scale per 16 values): writing it, reading it
  back, and single-token attention over it.

``run`` computes an operator either in its plain form (elementary torch operations in 32 bits,
rounded once at the end) or, where ``own`` is set, by the library's entry point.  ``exact`` is
the definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


# --------------------------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------------------------

def _window(kind, name, B, Hq, Hkv, Lq, q_off, d, dtype, window, sinks, pad, packed=False):
    return dict(kind=kind, name=name, B=B, Hq=Hq, Hkv=Hkv, Lq=Lq, q_off=q_off, d=d, dtype=dtype, window=window,
                sinks=sinks, pad=pad, packed=packed)


def _decode(kind, name, B, Hq, Hkv, S, lo, hi, d, dtype, window, sinks):
    return dict(kind=kind, name=name, B=B, Hq=Hq, Hkv=Hkv, S=S, len_lo=lo, len_hi=hi, d=d, dtype=dtype, window=window,
                sinks=sinks)


def _fill(name, B, H, S, T, first, d, dtype, k_exp, v_exp):
    return dict(kind="kv4_fill", name=name, B=B, Hkv=H, S=S, T=T, first=first, d=d, dtype=dtype, k_exp=k_exp,
                v_exp=v_exp)


def _norm(kind, name, B, Hq, Hkv, T, d, dtype, base, far):
    return dict(kind=kind, name=name, B=B, Hq=Hq, Hkv=Hkv, T=T, d=d, dtype=dtype, base=base, far=far)


def listed():
    return [
        # a 16K prompt through a windowed layer, grouped heads read in place from the packed projection
        _window("window_fwd", "window_prefill_16k", 1, 32, 8, 16384, 0, 128, "bf16", 1024, 4, 0.0, True),
        # the last, ragged chunk of a chunked prefill of left-padded sequences, in fp32
        _window("window_fwd", "window_chunk_f32", 2, 8, 8, 765, 259, 64, "f32", 257, 3, 0.4),
        # a training step of a windowed layer (forward and gradients), grouped heads
        _window("window_train", "window_train_4k", 2, 16, 4, 4096, 0, 128, "bf16", 1024, 4, 0.0, True),
        # a training step on short, odd, left-padded sequences with a small window and no grouping
        _window("window_train", "window_train_odd", 2, 8, 8, 1001, 0, 64, "bf16", 200, 1, 0.3),
        # one sequence generating: the smallest call, where latency counts
        _decode("window_decode", "window_decode_1", 1, 32, 8, 8192, 8000, 8000, 128, "bf16", 1024, 4),
        # a full batch generating with a long window over ragged lengths
        _decode("window_decode", "window_decode_64", 64, 32, 8, 16384, 3000, 16384, 128, "bf16", 4096, 16),
        # prompts written into the 4-bit cache and read back, as a chunked prefill does
        _fill("kv4_fill_8k", 4, 16, 8192, 8192, 0, 128, "bf16", 0, 0),
        # a short odd chunk appended behind a prefix, fp32 values, scaled tensors
        _fill("kv4_fill_odd", 3, 5, 1500, 777, 123, 64, "f32", -3, 2),
        # one token appended and attended, one sequence
        _decode("kv4_step", "kv4_step_1", 1, 32, 8, 8192, 8191, 8191, 128, "bf16", 0, 0),
        # one token appended and attended, long ragged caches
        _decode("kv4_step", "kv4_step_64k", 8, 32, 8, 65536, 32768, 65536, 128, "bf16", 0, 0),
        # queries and keys of a prompt, forward and gradients, read from the packed projection
        _norm("norm_train", "qk_norm_rope_train_8k", 2, 16, 4, 8192, 128, "bf16", 10000.0, 0),
        # the single new token of every sequence of a batch, each at its own far position
        _norm("norm_fwd", "qk_norm_rope_token_64", 64, 32, 8, 1, 128, "bf16", 1000000.0, 60000),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["window_fwd", "window_train", "window_decode", "kv4_fill", "kv4_step", "norm_train", "norm_fwd"])
    d = rng.choice([64, 128])
    group = rng.choice([1, 2, 4, 8])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    Hq = group * Hkv
    if kind in ("window_fwd", "window_train"):
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        most = (8192 if kind == "window_fwd" else 4096) if dtype == "bf16" else 1024
        Lq = _log(rng, 1, most)
        B = max(1, min(rng.choice([1, 2, 3]), 40000000 // (Lq * Lq * Hq)))
        Hkv = max(1, min(Hkv, 1500000000 // (Lq * Lq * group * B)))
        q_off = rng.choice([0, 0, rng.randint(1, 300)]) if kind == "window_fwd" else 0
        window = _log(rng, 1, max(2, min(4096, Lq + q_off + 50)))
        pad = rng.choice([0.0, 0.0, rng.uniform(0.1, 0.6)])
        return _window(kind, "", B, group * Hkv, Hkv, Lq, q_off, d, dtype, window, rng.choice([0, 1, 4, 130]), pad,
                       rng.random() < 0.5)
    if kind in ("window_decode", "kv4_step"):
        S = _log(rng, 16, 32768)
        B = _log(rng, 1, max(1, min(48, 2500000 // (S * Hkv))))
        lo = rng.randint(1, S)
        dtype = "bf16" if kind == "kv4_step" else rng.choice(["bf16", "bf16", "f32"])
        window = _log(rng, 1, S) if kind == "window_decode" or rng.random() < 0.4 else 0
        return _decode(kind, "", B, Hq, Hkv, S, lo, rng.randint(lo, S), d, dtype, window, rng.choice([0, 1, 4, 16]))
    if kind == "kv4_fill":
        T = _log(rng, 1, 8192)
        first = rng.choice([0, rng.randint(0, 500)])
        return _fill("", rng.choice([1, 2, 3, 4]), rng.choice([1, 2, 5, 8, 16]), first + T + rng.randint(0, 100), T, first,
                     d, rng.choice(["bf16", "f32"]), rng.randint(-8, 8), rng.randint(-8, 8))
    T = _log(rng, 1, 8192)
    B = rng.choice([1, 2]) if T > 64 else _log(rng, 1, 64)
    return _norm(kind, "", B, Hq, Hkv, T, d, rng.choice(["bf16", "f32"]), rng.choice([10000.0, 500000.0]),
                 rng.choice([0, rng.randint(1, 1000000)]))


# --------------------------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------------------------

def _pads(case):
    """Left padding of each sequence: its first `pad[b]` key positions are padding."""
    L = case["q_off"] + case["Lq"]
    return [int(case["pad"] * L * (b + 1) / case["B"]) for b in range(case["B"])]


def _lengths(case):
    """Cache lengths, spread evenly over the case's range (shuffled by the seed in prepare)."""
    B, lo, hi = case["B"], case["len_lo"], case["len_hi"]
    return [lo + (hi - lo) * b // max(1, B - 1) for b in range(B)]


def _randn(g, shape, std=1.0):
    x = torch.randn(shape, generator=g, device="cuda")
    return x.mul_(std) if std != 1.0 else x


def _channels(g, H, d):
    """A gain for each channel of the keys: a few are several times the others, as in trained models."""
    gain = torch.exp(0.3 * torch.randn((H, 1, d), generator=g, device="cuda"))
    return gain * (1.0 + 5.0 * (torch.rand((H, 1, d), generator=g, device="cuda") < 0.03))


def _heads(g, B, H, T, d, dtype, packed, std=1.0):
    """(B, H, T, d): contiguous, or the view of a (B, T, H, d) buffer that a projection writes."""
    if packed:
        return _randn(g, (B, T, H, d), std).to(dtype).permute(0, 2, 1, 3)
    return _randn(g, (B, H, T, d), std).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    B, Hkv, d = case["B"], case["Hkv"], case["d"]
    st = {"case": case}
    if case["kind"] in ("window_fwd", "window_train"):
        Lq, Lk = case["Lq"], case["q_off"] + case["Lq"]
        st["q"] = _heads(g, B, case["Hq"], Lq, d, dt, case["packed"], 1.5)
        st["k"] = _heads(g, B, Hkv, Lk, d, dt, case["packed"])
        st["v"] = _heads(g, B, Hkv, Lk, d, dt, case["packed"])
        st["mask"] = None
        if case["pad"] > 0:
            pads = torch.tensor(_pads(case), device="cuda")
            st["mask"] = (torch.arange(Lk, device="cuda")[None, :] < pads[:, None]).to(torch.uint8)
        if case["kind"] == "window_train":
            st["dout"] = _randn(g, (B, case["Hq"], Lq, d)).to(dt)
    elif case["kind"] in ("window_decode", "kv4_step"):
        S = case["S"]
        order = torch.randperm(B, generator=g, device="cuda")
        st["lengths"] = torch.tensor(_lengths(case), device="cuda", dtype=torch.int32)[order].contiguous()
        st["q"] = _randn(g, (B, case["Hq"], 1, d), 1.5).to(dt)
        if case["kind"] == "window_decode":
            st["k"] = _randn(g, (B, Hkv, S, d)).to(dt)
            st["v"] = _randn(g, (B, Hkv, S, d)).to(dt)
        else:
            gain = _channels(g, Hkv, d)
            st["k_codes"], st["k_scales"] = _pack(_randn(g, (B, Hkv, S, d)).mul_(gain), 0)
            st["v_codes"], st["v_scales"] = _pack(_randn(g, (B, Hkv, S, d)), 0)
            st["k"] = (_randn(g, (B, Hkv, 1, d)) * gain).to(dt)
            st["v"] = _randn(g, (B, Hkv, 1, d)).to(dt)
            st["start"] = st["lengths"] - 1
    elif case["kind"] == "kv4_fill":
        S, T = case["S"], case["T"]
        st["k"] = (_randn(g, (B, Hkv, T, d)).mul_(_channels(g, Hkv, d)) * 2.0 ** case["k_exp"]).to(dt)
        st["v"] = (_randn(g, (B, Hkv, T, d)) * 2.0 ** case["v_exp"]).to(dt)
        st["start"] = torch.full((B,), case["first"], device="cuda", dtype=torch.int32)
        st["k_codes"] = torch.zeros((B, Hkv, S, d // 2), device="cuda", dtype=torch.uint8)
        st["v_codes"] = torch.zeros((B, Hkv, S, d // 2), device="cuda", dtype=torch.uint8)
        st["k_scales"] = torch.zeros((B, Hkv, S, d // 16), device="cuda", dtype=torch.uint8)
        st["v_scales"] = torch.zeros((B, Hkv, S, d // 16), device="cuda", dtype=torch.uint8)
    else:
        T, Hq = case["T"], case["Hq"]
        qkv = _randn(g, (B, T, Hq + 2 * Hkv, d), 2.0).to(dt)   # the packed projection of the layer's input
        st["q"] = qkv[:, :, :Hq].permute(0, 2, 1, 3)
        st["k"] = qkv[:, :, Hq:Hq + Hkv].permute(0, 2, 1, 3)
        st["wq"] = (1.0 + 0.2 * _randn(g, (d,))).to(dt)
        st["wk"] = (1.0 + 0.2 * _randn(g, (d,))).to(dt)
        st["positions"] = None
        if case["far"]:
            at = torch.randint(0, case["far"] + 1, (B, 1), generator=g, device="cuda")
            st["positions"] = (at + torch.arange(T, device="cuda")[None, :]).to(torch.int32)
        if case["kind"] == "norm_train":
            st["dyq"] = _randn(g, (B, Hq, T, d)).to(dt)
            st["dyk"] = _randn(g, (B, Hkv, T, d)).to(dt)
    return st


# --------------------------------------------------------------------------------------------
# plain forms: the 4-bit cache
# --------------------------------------------------------------------------------------------

def _pack(x, exp):
    """x (.., d) fp32 -> codes (.., d / 2) and scales (.., d / 16), both uint8.

    Per block of 16: scale = e4m3(max|x| 2^-exp / 6), code = e2m1(x 2^-exp / scale), both to the
    nearest, ties to even, saturating; element 2 i in the low half of byte i."""
    a = x.unflatten(-1, (-1, 16)) * 2.0 ** -exp
    scale = (a.abs().amax(-1, keepdim=True) / 6.0).clamp_(max=448.0).to(torch.float8_e4m3fn)
    s = scale.float()
    r = torch.where(s > 0, a.abs() / s, torch.zeros_like(a))
    code = (r > 0.25).to(torch.uint8)
    code += r >= 0.75
    code += r > 1.25
    code += r >= 1.75
    code += r > 2.5
    code += r >= 3.5
    code += r > 5.0
    code += (a < 0).to(torch.uint8) * 8
    code = code.flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), scale.squeeze(-1).view(torch.uint8)


def _unpack(codes, scales, exp):
    """The values (.., d) in fp32 that codes and scales stand for."""
    levels = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0],
                          device=codes.device)
    code = torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2)
    value = levels[code.int()].unflatten(-1, (-1, 16))
    return (value * (scales.view(torch.float8_e4m3fn).float() * 2.0 ** exp).unsqueeze(-1)).flatten(-2)


def _store(st, exps):
    """Pack st's k and v into the cache slots start[b] + t."""
    k, v = st["k"], st["v"]
    b = torch.arange(k.shape[0], device="cuda")[:, None]
    slot = st["start"].long()[:, None] + torch.arange(k.shape[2], device="cuda")[None, :]
    for x, codes, scales, exp in ((k, st["k_codes"], st["k_scales"], exps[0]), (v, st["v_codes"], st["v_scales"], exps[1])):
        c, s = _pack(x.float(), exp)
        codes[b, :, slot] = c.transpose(1, 2)
        scales[b, :, slot] = s.transpose(1, 2)


# --------------------------------------------------------------------------------------------
# plain forms: attention
# --------------------------------------------------------------------------------------------

def _hidden(case, mask, lengths, device="cuda"):
    """True where query and key do not meet: (B or 1, 1, 1, Lq, Lk)."""
    if lengths is None:
        p = case["q_off"] + torch.arange(case["Lq"], device=device)[None, :, None]
        j = torch.arange(case["q_off"] + case["Lq"], device=device)[None, None, :]
    else:
        p = lengths.long()[:, None, None] - 1
        j = torch.arange(case["S"], device=device)[None, None, :]
    h = j > p
    if case["window"] > 0:
        h = h | ((j <= p - case["window"]) & (j >= case["sinks"]))
    if mask is not None:
        h = h | (mask[:, None, :] != 0)
    return h[:, None, None]


def _attend(q, k, v, hidden):
    """q (B, Hkv, G, Lq, d), k, v (B, Hkv, 1, Lk, d), fp32 -> out, lse, the probabilities (in place of the scores)."""
    s = q @ k.transpose(-1, -2)
    s *= 1.0 / math.sqrt(q.shape[-1])
    s.masked_fill_(hidden, -math.inf)
    m = s.amax(-1, keepdim=True)
    seen = m > -math.inf
    s -= torch.where(seen, m, torch.zeros_like(m))
    s.exp_()
    l = s.sum(-1, keepdim=True)
    s /= torch.where(seen, l, torch.ones_like(l))
    return s @ v, (m + l.log()).squeeze(-1), s


def _grouped(x, case):
    return x.float().unflatten(1, (case["Hkv"], -1))


def _window_plain(st):
    case, dt = st["case"], st["q"].dtype
    q = _grouped(st["q"], case)
    k, v = st["k"].float().unsqueeze(2), st["v"].float().unsqueeze(2)
    out, lse, p = _attend(q, k, v, _hidden(case, st["mask"], None))
    res = {"out": out.flatten(1, 2).to(dt), "lse": lse.flatten(1, 2)}
    if case["kind"] == "window_train":
        g = _grouped(st["dout"], case)
        res["dv"] = (p.transpose(-1, -2) @ g).sum(2).to(dt)
        ds = g @ v.transpose(-1, -2)
        ds -= (g * out).sum(-1, keepdim=True)
        ds *= p
        ds *= 1.0 / math.sqrt(case["d"])
        res["dq"] = (ds @ k).flatten(1, 2).to(dt)
        res["dk"] = (ds.transpose(-1, -2) @ q).sum(2).to(dt)
    return res


def _decode_plain(st):
    case = st["case"]
    if case["kind"] == "kv4_step":
        _store(st, (0, 0))
        k = _unpack(st["k_codes"], st["k_scales"], 0)
        v = _unpack(st["v_codes"], st["v_scales"], 0)
    else:
        k, v = st["k"].float(), st["v"].float()
    # the G queries of a head group are the rows of one product
    q = _grouped(st["q"], case).squeeze(3).unsqueeze(2)
    out, lse, _ = _attend(q, k.unsqueeze(2), v.unsqueeze(2), _hidden(case, None, st["lengths"]))
    return {"out": out.squeeze(2).flatten(1, 2).unsqueeze(2).to(st["q"].dtype), "lse": lse.squeeze(2).flatten(1, 2).unsqueeze(2)}


# --------------------------------------------------------------------------------------------
# plain forms: norm and rotation
# --------------------------------------------------------------------------------------------

EPS = 1e-6


def _angles(case, positions):
    """cos and sin (B or 1, 1, T, d / 2), formed in 64 bits."""
    d = case["d"]
    theta = case["base"] ** (-torch.arange(0, d, 2, device="cuda", dtype=torch.float64) / d)
    m = torch.arange(case["T"], device="cuda")[None] if positions is None else positions
    a = m.double()[:, None, :, None] * theta
    return a.cos(), a.sin()


def _rotate(x, c, s):
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack((a * c - b * s, a * s + b * c), dim=-1).flatten(-2)


def _norm_plain(st):
    case, dt = st["case"], st["q"].dtype
    c, s = (t.float() for t in _angles(case, st["positions"]))
    res = {}

    def one(name, x, w, dy):
        x, w = x.float(), w.float()
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        n = x * r
        res["y" + name] = _rotate(n * w, c, s).to(dt)
        if dy is not None:
            dz = _rotate(dy.float(), c, -s)
            res["dw" + name] = (dz * n).double().sum((0, 1, 2)).float()
            dn = dz * w
            res["d" + name] = (r * (dn - n * (dn * n).mean(-1, keepdim=True))).to(dt)

    one("q", st["q"], st["wq"], st.get("dyq"))
    one("k", st["k"], st["wk"], st.get("dyk"))
    return res


# --------------------------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------------------------

def run(st):
    case = st["case"]
    kind = case["kind"]
    if not own:
        if kind in ("window_fwd", "window_train"):
            return _window_plain(st)
        if kind in ("window_decode", "kv4_step"):
            return _decode_plain(st)
        if kind == "kv4_fill":
            _store(st, (case["k_exp"], case["v_exp"]))
            a, b = case["first"], case["first"] + case["T"]
            return {"k": _unpack(st["k_codes"][:, :, a:b], st["k_scales"][:, :, a:b], case["k_exp"]).bfloat16(),
                    "v": _unpack(st["v_codes"][:, :, a:b], st["v_scales"][:, :, a:b], case["v_exp"]).bfloat16()}
        return _norm_plain(st)

    import blockwise_attention_gb300 as ba

    if kind in ("window_fwd", "window_train"):
        at = dict(window=case["window"], sinks=case["sinks"], q_off=case["q_off"], key_padding_mask=st["mask"])
        out, lse = ba.attn_window_fwd(st["q"], st["k"], st["v"], **at)
        if kind == "window_fwd":
            return {"out": out, "lse": lse}
        dq, dk, dv = ba.attn_window_bwd(st["q"], st["k"], st["v"], out, st["dout"], lse, **at)
        return {"out": out, "lse": lse, "dv": dv, "dq": dq, "dk": dk}
    if kind == "window_decode":
        out, lse = ba.attn_window_decode_fwd(st["q"], st["k"], st["v"], window=case["window"], sinks=case["sinks"],
                                             lengths=st["lengths"])
        return {"out": out, "lse": lse}
    if kind == "kv4_step":
        cache = ba.KV4Cache(st["k_codes"], st["k_scales"], st["v_codes"], st["v_scales"])
        ba.kv4_append(cache, st["k"], st["v"], start=st["start"])
        out, lse = ba.attn_decode_kv4_fwd(st["q"], cache, lengths=st["lengths"], window=case["window"], sinks=case["sinks"])
        return {"out": out, "lse": lse}
    if kind == "kv4_fill":
        cache = ba.KV4Cache(st["k_codes"], st["k_scales"], st["v_codes"], st["v_scales"], case["k_exp"], case["v_exp"])
        ba.kv4_append(cache, st["k"], st["v"], start=st["start"])
        k, v = ba.kv4_read(cache, case["T"], first=case["first"])
        return {"k": k, "v": v}
    at = dict(eps=EPS, base=case["base"], positions=st["positions"])
    yq, yk = ba.qk_norm_rope_fwd(st["q"], st["k"], st["wq"], st["wk"], **at)
    if kind == "norm_fwd":
        return {"yq": yq, "yk": yk}
    dq, dk, dwq, dwk = ba.qk_norm_rope_bwd(st["q"], st["k"], st["wq"], st["wk"], st["dyq"], st["dyk"], **at)
    return {"yq": yq, "dwq": dwq, "dq": dq, "yk": yk, "dwk": dwk, "dk": dk}


# --------------------------------------------------------------------------------------------
# the work of one pass
# --------------------------------------------------------------------------------------------

def _seen(p, window, sinks, pad):
    """Keys that the queries at positions p (array) see behind a left padding of `pad` keys."""
    lo = np.maximum(p - window + 1, 0)
    near = p + 1 - np.minimum(np.maximum(lo, pad), p + 1)
    return near + np.maximum(np.minimum(lo, sinks) - pad, 0)


def work(case):
    kind, B, d, e = case["kind"], case["B"], case["d"], SIZE[case["dtype"]]
    if kind in ("window_fwd", "window_train"):
        p = case["q_off"] + np.arange(case["Lq"])
        pairs = case["Hq"] * sum(int(_seen(p, case["window"], case["sinks"], pad).sum()) for pad in _pads(case))
        Lk = case["q_off"] + case["Lq"]
        q, kv = B * case["Hq"] * case["Lq"], B * case["Hkv"] * Lk
        moved = 2 * q * d * e + 2 * kv * d * e + 4 * q + (B * Lk if case["pad"] > 0 else 0)
        if kind == "window_fwd":
            return {"bytes": moved, "flops": 4 * d * pairs}
        return {"bytes": moved + 2 * q * d * e + 2 * kv * d * e, "flops": 14 * d * pairs}
    if kind in ("window_decode", "kv4_step"):
        n = np.array(_lengths(case))
        w = case["window"] if case["window"] > 0 else case["S"]
        keys = int(_seen(n - 1, w, case["sinks"] if case["window"] > 0 else 0, 0).sum())
        row = d * e if kind == "window_decode" else d // 2 + d // 16
        new = B * case["Hkv"] * 2 * d * e if kind == "kv4_step" else 0
        return {"bytes": 2 * keys * case["Hkv"] * row + 2 * B * case["Hq"] * d * e + 4 * B * case["Hq"] + new,
                "flops": 4 * d * keys * case["Hq"]}
    if kind == "kv4_fill":
        n = 2 * B * case["Hkv"] * case["T"]
        return {"bytes": n * (d * e + 2 * (d // 2 + d // 16) + 2 * d), "flops": 4 * n * d}
    n = B * (case["Hq"] + case["Hkv"]) * case["T"] * d
    if kind == "norm_fwd":
        return {"bytes": 2 * n * e, "flops": 8 * n}
    return {"bytes": 4 * n * e, "flops": 25 * n}


# --------------------------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------------------------

def _exact_rows(q, k, v, hidden, g):
    """One head's query rows against its keys in 64 bits: out, lse and, with g, the rows' dq and their shares of dk, dv."""
    sc = 1.0 / math.sqrt(q.shape[-1])
    s = (q @ k.T) * sc
    s = torch.where(hidden, torch.full_like(s, -math.inf), s)
    lse = torch.logsumexp(s, -1)
    p = torch.where(hidden, torch.zeros_like(s), torch.exp(s - torch.where(lse > -math.inf, lse, torch.zeros_like(lse))[:, None]))
    out = p @ v
    if g is None:
        return out, lse
    ds = p * (g @ v.T - (g * out).sum(-1, keepdim=True)) * sc
    return out, lse, ds @ k, ds.T @ q, p.T @ g


def _exact_window(st, case):
    B, Hq, Lq, d, W, sinks, off = (case[n] for n in ("B", "Hq", "Lq", "d", "window", "sinks", "q_off"))
    G, Lk = Hq // case["Hkv"], off + Lq
    train = case["kind"] == "window_train"
    new = lambda *shape: torch.zeros(shape, device="cuda", dtype=torch.float64)  # noqa: E731
    res = {"out": new(B, Hq, Lq, d), "lse": new(B, Hq, Lq)}
    if train:
        res |= {"dv": new(B, case["Hkv"], Lk, d), "dq": new(B, Hq, Lq, d), "dk": new(B, case["Hkv"], Lk, d)}
    step = 1024
    for b in range(B):
        for h in range(Hq):
            k, v = st["k"][b, h // G].double(), st["v"][b, h // G].double()
            for i in range(0, Lq, step):
                n = min(step, Lq - i)
                first = max(0, off + i - W + 1)
                near = torch.arange(first, off + i + n, device="cuda")
                j = torch.cat((torch.arange(0, min(sinks, first), device="cuda"), near))
                p = off + i + torch.arange(n, device="cuda")[:, None]
                hidden = (j > p) | ((j <= p - W) & (j >= sinks))
                if st["mask"] is not None:
                    hidden |= st["mask"][b, j] != 0
                got = _exact_rows(st["q"][b, h, i:i + n].double(), k[j], v[j], hidden,
                                  st["dout"][b, h, i:i + n].double() if train else None)
                res["out"][b, h, i:i + n], res["lse"][b, h, i:i + n] = got[0], got[1]
                if train:
                    res["dq"][b, h, i:i + n] = got[2]
                    res["dk"][b, h // G].index_add_(0, j, got[3])
                    res["dv"][b, h // G].index_add_(0, j, got[4])
    return res


_GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _exact_quantised(x, exp):
    """The values that a 4-bit cache holds for x (.., d), by nearest search over the two grids in 64 bits."""
    a = x.double().unflatten(-1, (-1, 16)) * 2.0 ** -exp
    bytes_ = torch.arange(127, device="cuda", dtype=torch.uint8)
    e4m3 = bytes_.view(torch.float8_e4m3fn).double()                        # 0 .. 448, ascending
    t = (a.abs().amax(-1) / 6.0).clamp(max=448.0)
    hi = torch.searchsorted(e4m3, t).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    down, up = t - e4m3[lo], e4m3[hi] - t
    pick = torch.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)   # ties to the even byte
    s = e4m3[pick].unsqueeze(-1)
    best = torch.zeros_like(a)
    near = a.abs()
    for i in range(1, 8):
        mid = 0.5 * (_GRID[i - 1] + _GRID[i]) * s
        up_ = (near > mid) if i % 2 else (near >= mid)                      # ties to the even code
        best = torch.where(up_ & (s > 0), _GRID[i] * s, best)
    return (torch.where(a < 0, -best, best) * 2.0 ** exp).flatten(-2)


def _exact_decode(st, case):
    B, Hq, d, W = case["B"], case["Hq"], case["d"], case["window"]
    G = Hq // case["Hkv"]
    out = torch.zeros((B, Hq, 1, d), device="cuda", dtype=torch.float64)
    lse = torch.zeros((B, Hq, 1), device="cuda", dtype=torch.float64)
    for b in range(B):
        n = int(st["lengths"][b])
        first = max(0, n - W) if W > 0 else 0
        j = torch.cat((torch.arange(0, min(case["sinks"], first), device="cuda"), torch.arange(first, n, device="cuda")))
        for h in range(case["Hkv"]):
            if case["kind"] == "kv4_step":
                k = _exact_values(st["k_codes"][b, h, j], st["k_scales"][b, h, j])
                v = _exact_values(st["v_codes"][b, h, j], st["v_scales"][b, h, j])
                k[j == n - 1] = _exact_quantised(st["k"][b, h], 0)
                v[j == n - 1] = _exact_quantised(st["v"][b, h], 0)
            else:
                k, v = st["k"][b, h, j].double(), st["v"][b, h, j].double()
            q = st["q"][b, h * G:(h + 1) * G, 0].double()
            o, l = _exact_rows(q, k, v, torch.zeros((G, len(j)), dtype=torch.bool, device="cuda"), None)
            out[b, h * G:(h + 1) * G, 0], lse[b, h * G:(h + 1) * G, 0] = o, l
    return {"out": out, "lse": lse}


def _exact_values(codes, scales):
    """codes (n, d / 2), scales (n, d / 16) -> values in 64 bits, by the fields of the two formats."""
    c = torch.stack((codes % 16, codes // 16), -1).flatten(-2).long()
    e, m = (c % 8) // 2, c % 2
    mag = torch.where(e == 0, 0.5 * m, (1.0 + 0.5 * m) * torch.pow(2.0, (e - 1).double()))
    b = scales.long()
    se, sm = b // 8, (b % 8).double()
    s = torch.where(se == 0, sm / 8.0 * 2.0 ** -6, (1.0 + sm / 8.0) * torch.pow(2.0, (se - 7).double()))
    return torch.where(c >= 8, -mag, mag).double() * s.repeat_interleave(16, dim=-1)


def _exact_norm(st, case):
    d, T, B = case["d"], case["T"], case["B"]
    theta = torch.tensor([case["base"] ** (-2.0 * c / d) for c in range(d // 2)], device="cuda", dtype=torch.float64)
    m = torch.arange(T, device="cuda").expand(B, T) if st["positions"] is None else st["positions"]
    z = torch.polar(torch.ones((), device="cuda", dtype=torch.float64), m.double()[:, None, :, None] * theta)
    res = {}
    for name in ("q", "k"):
        x, w = st[name].double(), st["w" + name].double()
        r = ((x * x).sum(-1, keepdim=True) / d + EPS) ** -0.5
        y = torch.view_as_complex((x * r * w).unflatten(-1, (-1, 2)).contiguous()) * z
        res["y" + name] = torch.view_as_real(y).flatten(-2)
        if case["kind"] == "norm_train":
            dy = torch.view_as_complex(st["dy" + name].double().unflatten(-1, (-1, 2)).contiguous())
            dz = torch.view_as_real(dy * z.conj()).flatten(-2)
            res["dw" + name] = (dz * x * r).sum((0, 1, 2))
            u = dz * w
            res["d" + name] = r * u - x * r ** 3 * (u * x).sum(-1, keepdim=True) / d
    return res


def exact(case, seed):
    st = prepare(case, seed)
    if case["kind"] in ("window_fwd", "window_train"):
        return _exact_window(st, case)
    if case["kind"] in ("window_decode", "kv4_step"):
        return _exact_decode(st, case)
    if case["kind"] == "kv4_fill":
        return {"k": _exact_quantised(st["k"], case["k_exp"]), "v": _exact_quantised(st["v"], case["v_exp"])}
    return _exact_norm(st, case)
