"""Plain 64-bit forms of the calls on packed sequences (torch, one sequence and one head at a time), with
how far a correct result in the calls' precision may be off, derived term by term."""
import math

import torch

D = 128
BF16 = torch.finfo(torch.bfloat16).eps / 2  # half a step, relative


def starts(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return at


def rope(x, pos, base, gain=None, eps=None):
    """x [T, H, 128] at positions pos [T], normed before where eps is given."""
    x = x.double()
    if eps is not None:
        x = x / (x.square().mean(-1, keepdim=True) + eps).sqrt()
        if gain is not None:
            x = x * gain.double()
    y = torch.empty_like(x)
    for i in range(D // 2):
        angle = pos.double() * base ** (-2.0 * i / D)
        c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
        y[..., 2 * i] = x[..., 2 * i] * c - x[..., 2 * i + 1] * s
        y[..., 2 * i + 1] = x[..., 2 * i] * s + x[..., 2 * i + 1] * c
    # fp32: the angle as half a circle's part (2^-25 pi), sine and cosine (2^-22), the norm (2^-21) and three
    # roundings, each relative to the pair's length; then one rounding to bf16
    pair = x.unflatten(-1, (D // 2, 2)).norm(dim=-1).repeat_interleave(2, -1)
    return y, BF16 * y.abs() + 2.0 ** -19 * pair


def visible(lq, lk, window, device):
    p = torch.arange(lk - lq, lk, device=device)[:, None]
    j = torch.arange(lk, device=device)
    return (j <= p) & (j > p - window)


def window_prefill(q, k, v, cu_q, cu_k, window, tau):
    """out [T, Hq, 128] and tolerance; rows of no sequence are NaN."""
    out = torch.full(q.shape, math.nan, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    G = q.shape[1] // k.shape[1]
    for (a, b), (c, d) in zip(zip(cu_q, cu_q[1:]), zip(cu_k, cu_k[1:])):
        if b == a:
            continue
        seen = visible(b - a, d - c, window, q.device)
        some = seen.any(1)
        out[a:b], tol[a:b] = 0.0, 0.0
        if not some.any():
            continue
        for h in range(q.shape[1]):
            qh, kh, vh = q[a:b, h].double(), k[c:d, h // G].double(), v[c:d, h // G].double()
            z = (tau * qh @ kh.T).masked_fill(~seen, -math.inf)[some]
            p = torch.softmax(z, -1)
            p = torch.where(seen[some], p, 0.0)
            rows = torch.arange(a, b, device=q.device)[some]
            vs = torch.where(seen.any(0)[:, None], vh, 0.0)  # (a key nobody sees may hold anything)
            o, mean = p @ vs, p @ vs.abs()
            # weights rounded to bf16; scores in fp32 (128 products) move them by e^(2 err) at most, the
            # exponent's own rounding by 2^-23 of its size (below 2^7 where a weight counts)
            size = (qh.abs() @ kh.abs().T).masked_fill(~seen, 0.0)[some].amax(1, keepdim=True)
            err = 2 * abs(tau) * D * 2.0 ** -24 * size + 2.0 ** -15
            out[rows, h], tol[rows, h] = o, BF16 * o.abs() + (BF16 + err) * mean * 1.02
    return out, tol


def prefill_packed(q, k, v, cu_q, cu_k, alpha, c, eps):
    out = torch.full(q.shape, math.nan, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    G = q.shape[1] // k.shape[1]
    for (a, b), (e, d) in zip(zip(cu_q, cu_q[1:]), zip(cu_k, cu_k[1:])):
        if b == a:
            continue
        seen = visible(b - a, d - e, 1 << 40, q.device)
        for h in range(q.shape[1]):
            qh, kh, vh = q[a:b, h].double(), k[e:d, h // G].double(), v[e:d, h // G].double()
            qn = qh / (qh.square().mean(-1, keepdim=True) + eps).sqrt()
            kn = kh / (kh.square().mean(-1, keepdim=True) + eps).sqrt()
            s = (alpha * qn @ kn.T).clamp(min=0.0).masked_fill(~seen, 0.0)
            vs = torch.where(seen.any(0)[:, None], vh, 0.0)
            w = s.square()
            den = c + w.sum(-1, keepdim=True)
            den = torch.where(den == 0, 1.0, den)
            o = w @ vs / den
            # weights rounded to bf16 (numerator and denominator); scores in fp32 off by 128 products of
            # rows of length sqrt(128), which counts twice in s^2
            moved = 2 * (s @ vs.abs()) / den * alpha * D * D * 2.0 ** -24
            out[a:b, h] = o
            tol[a:b, h] = BF16 * o.abs() + 2.04 * BF16 * (w @ vs.abs()) / den + 2 * moved + 1e-30
    return out, tol


def window_decode(q, k_win, v_win, pos, tau):
    B, Hkv, W, _ = k_win.shape
    G = q.shape[1] // Hkv
    out, tol = torch.zeros(q.shape, dtype=torch.float64, device=q.device), torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    for b, last in enumerate(pos):
        if last < 0:
            continue
        slots = torch.arange(max(0, last - W + 1), last + 1, device=q.device) % W
        for h in range(q.shape[1]):
            k, v = k_win[b, h // G][slots].double(), v_win[b, h // G][slots].double()
            p = torch.softmax(tau * (k @ q[b, h].double()), 0)
            size = (k.abs() @ q[b, h].double().abs()).max()
            out[b, h] = p @ v
            tol[b, h] = (2 * abs(tau) * D * 2.0 ** -24 * size + 2.0 ** -15) * (p @ v.abs())
    return out, tol


def assert_within(got, want, tol, what):
    got = got.double()
    assert got.shape == want.shape
    off = (got - want).abs()
    bad = ~(off <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outside; first at {bad.nonzero()[0].tolist()}: "
                           f"{got[bad][0].item()} for {want[bad][0].item()} +- {tol[bad][0].item()}")
