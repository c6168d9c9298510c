"""Plain 64-bit statements of the windowed attention and its gradients, and the
error bounds of the kernels (test-side only; torch in double on the inputs' device)."""
import math

import torch

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}   # largest relative rounding error


def visible(Lq, Lk, q_off, window, sinks, kpm=None, device="cpu"):
    """(B or 1, 1, Lq, Lk) bool: the pairs that meet.  window <= 0: no window."""
    p = q_off + torch.arange(Lq, device=device)[:, None]
    j = torch.arange(Lk, device=device)[None, :]
    m = j <= p
    if window > 0:
        m = m & ((j > p - window) | (j < sinks))
    m = m[None]
    if kpm is not None:
        m = m & (kpm[:, None, :Lk] == 0)
    return m[:, None]


def heads(x, Hq):
    """Key heads repeated for the query heads that read them, in double, masked garbage included."""
    return x.double().repeat_interleave(Hq // x.shape[1], dim=1)


def forward(q, k, v, seen, scale=None):
    """out, lse, p, and sum_j p_j |v_j| (all double); keys that no pair sees may hold anything."""
    Hq, d = q.shape[1], q.shape[3]
    sc = scale or 1.0 / math.sqrt(d)
    s = (q.double() @ heads(k, Hq).transpose(-1, -2)) * sc
    s = torch.where(seen, s, torch.full_like(s, -math.inf))
    lse = torch.logsumexp(s, -1)
    p = torch.where(seen, torch.exp(s - torch.where(lse > -math.inf, lse, torch.zeros_like(lse))[..., None]),
                    torch.zeros_like(s))
    vz = torch.where(seen.any(-2, keepdim=True).transpose(-1, -2), heads(v, Hq), torch.zeros((), dtype=torch.double,
                                                                                           device=q.device))
    return p @ vz, lse, p, p @ vz.abs()


def score_error(q, k, scale=None):
    """Bound of |s - s_exact| for fp32 sums of d products: d half steps of sum |q_c k_c|."""
    d = q.shape[-1]
    if k.shape[2] == 0:
        return 0.0
    sc = scale or 1.0 / math.sqrt(d)
    big = (q.double().abs().flatten(0, 2).amax(0) * torch.nan_to_num(k.double(), 0, 0, 0).abs().flatten(0, 2).amax(0)).sum()
    return float(d * 2.0 ** -24 * big * sc)


def check_forward(out, lse, q, k, v, seen, scale=None, label="", p_step=None):
    """p_step: the rounding of p before P V where it is not that of q's type.  fp32 kernels: the scores' error e moves every p by a factor in 1 +- (e + 2^-20)
    (the exponential, the running sums).  bf16 kernels round p once to bf16 before
    P V.  Then one rounding to out's type."""
    o, l, p, pa = forward(q, k, v, seen, scale)
    e = 2.0 * score_error(q, k, scale) + 2.0 ** -20
    if p_step is None:
        p_step = HALF_STEP[torch.bfloat16] if q.dtype == torch.bfloat16 else 0.0
    rel_p = e + p_step
    tol = rel_p * pa * 1.01 + HALF_STEP[out.dtype] * (o.abs() + rel_p * pa) + 1e-30
    bad = (out.double() - o).abs() > tol
    assert torch.isfinite(out).all(), f"{label}: non-finite out"
    assert not bad.any(), (label, float(((out.double() - o).abs() - tol).max()), int(bad.sum()))
    empty = l == -math.inf
    assert torch.equal(lse == -math.inf, empty), f"{label}: rows without keys"
    assert (out[empty] == 0).all()
    err = (lse.double() - l)[~empty].abs()
    lim = e + 2.0 ** -22 * l[~empty].abs()
    assert (err <= lim).all(), (label, float((err - lim).max()))


def check_backward(grads, q, k, v, out, dout, lse, seen, scale=None, label=""):
    """The gradients' formulas on the out and lse that the kernel was given.  p is off by
    a factor in 1 +- e as above (lse is an input); bf16 kernels round p and ds to bf16
    once each; sums in fp32 (n terms: at most n half steps of the sum of magnitudes,
    n <= a few thousand, covered by 2^-12); then one rounding to the gradient's type."""
    Hq, Hkv, d = q.shape[1], k.shape[1], q.shape[3]
    sc = scale or 1.0 / math.sqrt(d)
    z = torch.zeros((), dtype=torch.double, device=q.device)
    keys = seen.any(-2, keepdim=True).transpose(-1, -2)
    kd, vd = torch.where(keys, heads(k, Hq), z), torch.where(keys, heads(v, Hq), z)
    qd, g = q.double(), dout.double()
    rows = (lse > -math.inf)[..., None]
    p = torch.where(seen & rows, torch.exp((qd @ kd.transpose(-1, -2)) * sc - torch.where(rows, lse.double()[..., None], z)), z)
    D = (g * out.double()).sum(-1, keepdim=True)
    dp = g @ vd.transpose(-1, -2)
    ds = p * (dp - D)
    e = 2.0 * score_error(q, k, scale) + 2.0 ** -20
    half = HALF_STEP[torch.bfloat16] if q.dtype == torch.bfloat16 else 0.0
    sums = 2.0 ** -12 if q.dtype == torch.bfloat16 else 2.0 ** -18
    # error of ds: its rounding, p's factor, and the fp32 sums dp and D (d terms)
    mag = p * (g.abs() @ vd.abs().transpose(-1, -2) + (g * out.double()).abs().sum(-1, keepdim=True))
    ds_err = half * ds.abs() + (e + d * 2.0 ** -23) * mag
    fold = lambda x: x.unflatten(1, (Hkv, Hq // Hkv)).sum(2)  # noqa: E731
    want = {"dq": (sc * ds @ kd, sc * (ds_err + sums * mag) @ kd.abs()),
            "dk": (fold(sc * ds.transpose(-1, -2) @ qd), fold(sc * (ds_err + sums * mag).transpose(-1, -2) @ qd.abs())),
            "dv": (fold(p.transpose(-1, -2) @ g), fold((half + e + sums) * p.transpose(-1, -2) @ g.abs()))}
    for (name, (ref, tol)), got in zip(want.items(), grads):
        assert torch.isfinite(got).all(), (label, name, "non-finite")
        tol = tol + HALF_STEP[got.dtype] * (ref.abs() + tol) + 1e-30
        err = (got.double() - ref).abs()
        assert (err <= tol).all(), (label, name, float((err - tol).max()), float(err.max()), int((err > tol).sum()))


def visible_decode(lengths, S, window, sinks, device):
    """(B, 1, 1, S) bool: the slots that the newest token of each sequence sees."""
    n = lengths.long().clamp(0, S)[:, None]
    j = torch.arange(S, device=device)[None, :]
    m = j < n
    if window > 0:
        m = m & ((j >= n - window) | (j < sinks))
    return m[:, None, None]
