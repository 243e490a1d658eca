"""Timed cases of four operators on batches whose sequences have different lengths, with their
plain torch forms:

  rope    embla_rope_qkv             queries and keys of packed tokens normed per head and rotated at
                                     their positions, in one pass, the newest rows into the window rings
  window  embla_window_prefill       causal softmax attention of packed prompts over a window
  full    embla_prefill_packed       causal ReLU^2 attention of packed prompts
  decode  embla_window_decode_ragged one token per sequence over its ring, each at its own position

Shapes are the library's own: 16 query heads, 4 or 2 KV heads (groups of 4 or 8), head_dim 128,
windows of 128 keys (rings of up to 1,024), ReLU^2 weights with 5 % of the scores positive.  Packed
tokens lie one sequence behind the other, as rows of one projection [T, (Hq + 2 Hkv) 128].
"""
import math

import torch

own = False

D = 128
HQ = 16
BASE = 10000.0
ALPHA, C, EPS = 1.0, 1.0, 1e-6
TAU = D ** -0.5
DEV = "cuda"


# ----------------------------------------------------------------------------- cases

def listed():
    return [
        # one decode step of a batch of 8 far into their contexts: latency
        dict(name="rope-b8-t1", op="rope", hkv=4, lens="1,1,1,1,1,1,1,1", pos=32768, norm=False, window=128),
        # a few prompts of odd lengths, one of a single token, one empty, queries and keys normed
        dict(name="rope-ragged-5k", op="rope", hkv=2, lens="1021,3,2048,1,0,1999", pos=0, norm=True, window=128),
        # a batch of long prompts
        dict(name="rope-4x32k", op="rope", hkv=4, lens="32768,32768,32768,32768", pos=0, norm=True, window=128),
        # short prompts of a chat: latency
        dict(name="window-short", op="window", hkv=4, lens="17,1,130,0,64", window=128),
        # prompts of very different lengths
        dict(name="window-ragged-6k", op="window", hkv=4, lens="700,1,2500,129,0,1024,33,1777", window=128),
        # long prompts through the window layers
        dict(name="window-8x16k", op="window", hkv=4, lens=",".join(["16384"] * 8), window=128),
        # the largest ring, groups of 8
        dict(name="window-2x16k-w1024-g8", op="window", hkv=2, lens="16384,16011", window=1024),
        # prompts of very different lengths through a full layer
        dict(name="full-ragged-4k", op="full", hkv=4, lens="700,1,1500,129,0,1024,777"),
        # a few prompts, groups of 8
        dict(name="full-4x4k-g8", op="full", hkv=2, lens="4096,4000,3500,2900"),
        # one long prompt
        dict(name="full-1x16k", op="full", hkv=4, lens="16384"),
        # the step after: few sequences, latency
        dict(name="decode-b8", op="decode", hkv=4, lens="5,130,128,3000,20000,1,64,777", window=128),
        # a wide batch over the largest rings, groups of 8
        dict(name="decode-b96-w1024-g8", op="decode", hkv=2, window=1024,
             lens=",".join(str(1 + 97 * i * (i % 7)) for i in range(96))),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["rope", "window", "window", "full", "full", "decode"])
    hkv = rng.choice([2, 4])
    window = rng.choice([128, 128, _log(rng, 16, 1024)])
    if op == "decode":
        lens = [_log(rng, 1, 60000) for _ in range(_log(rng, 1, 96))]
        return dict(op=op, hkv=hkv, lens=",".join(map(str, lens)), window=window)
    batch = _log(rng, 1, 24)
    if op == "full":
        longest = _log(rng, 40, int(15000 / math.sqrt(batch)))
    else:
        longest = _log(rng, 4, (120000 if window < 200 else 30000) // batch)
    lens = [rng.choice([longest, _log(rng, 1, longest), _log(rng, 1, longest), rng.randrange(0, 3)])
            for _ in range(batch)]
    lens[rng.randrange(batch)] = longest
    case = dict(op=op, hkv=hkv, lens=",".join(map(str, lens)))
    if op == "rope":
        case.update(pos=rng.choice([0, rng.randrange(200000)]), norm=rng.random() < 0.5, window=window)
    if op == "window":
        case.update(window=window)
    return case


def _lens(case):
    return [int(x) for x in case["lens"].split(",")]


def _starts(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return at


# ----------------------------------------------------------------------------- inputs

def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEV)


def prepare(case, seed):
    op, hkv, lens = case["op"], case["hkv"], _lens(case)
    B, G = len(lens), HQ // hkv
    gen = torch.Generator(device=DEV).manual_seed(seed)
    st = dict(case=case)
    if op == "decode":
        W = case["window"]
        st["pos"] = torch.tensor([n - 1 for n in lens], dtype=torch.int32, device=DEV)
        st["q"] = (2.0 * _randn(gen, B, HQ, D)).bfloat16()
        st["k_win"] = _randn(gen, B, hkv, W, D).bfloat16()
        st["v_win"] = _randn(gen, B, hkv, W, D).bfloat16()
        st["out"] = torch.zeros(B, HQ, D, device=DEV)
    else:
        at = _starts(lens)
        T = at[-1]
        st["cu"] = torch.tensor(at, dtype=torch.int32, device=DEV)
        x = torch.empty(T, HQ + 2 * hkv, D, dtype=torch.bfloat16, device=DEV)
        x.copy_(_randn(gen, T, HQ + 2 * hkv, D))
        q, k, v = x[:, :HQ], x[:, HQ:HQ + hkv], x[:, HQ + hkv:]
        if op == "rope":
            # rows of different sizes, as tokens and heads have them
            q.mul_(torch.exp(0.5 * _randn(gen, T, HQ, 1)))
            k.mul_(torch.exp(0.5 * _randn(gen, T, hkv, 1)))
            W = case["window"]
            st["pos0"] = torch.tensor([case["pos"] + 61 * b for b in range(B)] if case["pos"] else [0] * B,
                                      dtype=torch.int32, device=DEV)
            st["q_gain"] = 1 + 0.2 * _randn(gen, D) if case["norm"] else None
            st["k_gain"] = 1 + 0.2 * _randn(gen, D) if case["norm"] else None
            st["q_out"] = torch.zeros(T, HQ, D, dtype=torch.bfloat16, device=DEV)
            st["k_out"] = torch.zeros(T, hkv, D, dtype=torch.bfloat16, device=DEV)
            st["k_win"] = torch.zeros(B, hkv, W, D, dtype=torch.bfloat16, device=DEV)
            st["v_win"] = torch.zeros(B, hkv, W, D, dtype=torch.bfloat16, device=DEV)
        elif op == "window":
            # what the rotation wrote, beside the projection's values
            q, k = (2.0 * q.float()).bfloat16(), k.contiguous()
        else:
            # scores D cos(q, k) positive for about 5 % of the keys of every head: the queries of a
            # KV head share a direction that the keys turn away from
            u = torch.nn.functional.normalize(_randn(gen, hkv, D), dim=-1)
            q.copy_(q.float() + 8.0 * u.repeat_interleave(G, 0))
            k.copy_(k.float() - 2.85 * u)
        if op != "rope":
            st["out"] = torch.zeros(T, HQ, D, dtype=torch.bfloat16, device=DEV)
        st.update(q=q, k=k, v=v)
    if own:
        import relu_sparse_kv_gb300 as E
        st["shape"] = E.Shape(B, HQ, hkv, D, 0, 0)
        if op == "full":
            need = E.embla_prefill_packed_workspace_size(st["shape"], st["k"].shape[0])
            st["workspace"] = torch.empty(max(need, 16), dtype=torch.uint8, device=DEV)
    return st


# ----------------------------------------------------------------------------- plain forms

def _where(s):
    """The sequence of every packed token and its place there."""
    cu = s["cu"].long()
    t = torch.arange(s["q"].shape[0], device=DEV)
    b = torch.bucketize(t, cu[1:], right=True)
    return b, t - cu[b]


def _turned(x, gain, pos):
    """Rows x [T, H, D], normed where there is a gain, and their pairs turned at pos."""
    f = x.float()
    if gain is not None:
        f = f / torch.sqrt(f.square().mean(-1, keepdim=True) + EPS) * gain
    i = torch.arange(D // 2, device=DEV, dtype=torch.float64)
    angle = pos.double()[:, None] * BASE ** (-2 * i / D)
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    a, b = f[..., 0::2], f[..., 1::2]
    return torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(2).bfloat16()


def _plain_rope(s):
    W = s["case"]["window"]
    b, i = _where(s)
    pos = s["pos0"].long()[b] + i
    s["q_out"].copy_(_turned(s["q"], s["q_gain"], pos))
    s["k_out"].copy_(_turned(s["k"], s["k_gain"], pos))
    cu = s["cu"].long()
    new = i >= (cu[1:] - cu[:-1])[b] - W
    s["k_win"][b[new], :, pos[new] % W] = s["k_out"][new]
    s["v_win"][b[new], :, pos[new] % W] = s["v"][new]


def _plain_window(s):
    W, hkv = s["case"]["window"], s["case"]["hkv"]
    T, G = s["q"].shape[0], HQ // hkv
    # queries in blocks of W tokens; a block sees keys of itself and the block before
    nb = -(-T // W)
    q, k, v = (torch.nn.functional.pad(x.float(), (0, 0, 0, 0, 0, nb * W - T)) for x in (s["q"], s["k"], s["v"]))
    q = q.view(nb, W, hkv, G, D).permute(0, 2, 3, 1, 4).reshape(nb, hkv, G * W, D)
    k, v = (torch.nn.functional.pad(x, (0, 0, 0, 0, W, 0)).view(nb + 1, W, hkv, D) for x in (k, v))
    k, v = (torch.cat([x[:-1], x[1:]], 1).permute(0, 2, 1, 3) for x in (k, v))
    b, _ = _where(s)
    seq = torch.nn.functional.pad(b, (W, nb * W - T), value=-1).view(nb + 1, W)
    mine, theirs = seq[1:, :, None], torch.cat([seq[:-1], seq[1:]], 1)[:, None]
    i, j = torch.arange(W, device=DEV)[:, None] + W, torch.arange(2 * W, device=DEV)
    seen = (mine == theirs) & (j <= i) & (j > i - W) | ((mine < 0) & (j == i))
    z = (q @ k.transpose(2, 3) * TAU).view(nb, hkv, G, W, 2 * W)
    z = z.masked_fill_(~seen[:, None, None], -math.inf)
    p = torch.exp_(z.sub_(z.amax(-1, keepdim=True)))
    total = p.sum(-1)
    o = (p.view(nb, hkv, G * W, 2 * W) @ v).view(nb, hkv, G, W, D) / total[..., None]
    s["out"].copy_(o.permute(0, 3, 1, 2, 4).reshape(nb * W, HQ, D)[:T])


def _normed(x):
    return x / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS)


def _plain_full(s):
    hkv, lens = s["case"]["hkv"], _lens(s["case"])
    G, L = HQ // hkv, max(lens)
    # sequences side by side, padded to the longest
    b, i = _where(s)
    B, T = len(lens), s["q"].shape[0]
    at = torch.full((B, L), T, device=DEV)
    at[b, i] = torch.arange(T, device=DEV)
    q, k, v = (torch.nn.functional.pad(x.float(), (0, 0, 0, 0, 0, 1))[at] for x in (s["q"], s["k"], s["v"]))
    q = _normed(q).view(B, L, hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, hkv, G * L, D)
    w = (q @ _normed(k).permute(0, 2, 3, 1)).mul_(ALPHA).clamp_(min=0.0).square_()
    t = torch.arange(L, device=DEV)
    w.view(B, hkv, G, L, L).mul_(t <= t[:, None])
    o = (w @ v.permute(0, 2, 1, 3)) / (w.sum(-1, keepdim=True) + C)
    o = o.view(B, hkv, G, L, D).permute(0, 3, 1, 2, 4).reshape(B, L, HQ, D)
    s["out"].copy_(o[b, i])


def _plain_decode(s):
    B, hkv, W, _ = s["k_win"].shape
    z = s["q"].float().view(B, hkv, HQ // hkv, D) @ s["k_win"].float().transpose(2, 3) * TAU
    late = torch.arange(W, device=DEV) > s["pos"][:, None]
    z = z.masked_fill(late[:, None, None], -math.inf)
    p = torch.exp(z - z.amax(-1, keepdim=True))
    s["out"].copy_((p @ s["v_win"].float() / p.sum(-1, keepdim=True)).view(B, HQ, D))


def run(s):
    op = s["case"]["op"]
    if own:
        import relu_sparse_kv_gb300 as E
        if op == "rope":
            E.embla_rope_qkv(s["shape"], s["cu"], s["pos0"], s["q"], s["k"], s["v"], s["q_out"], s["k_out"],
                             k_win=s["k_win"], v_win=s["v_win"], rope_base=BASE,
                             norm_eps=EPS if s["case"]["norm"] else None, q_gain=s["q_gain"], k_gain=s["k_gain"])
        elif op == "window":
            E.embla_window_prefill(s["shape"], s["cu"], s["q"], s["k"], s["v"], s["out"], window=s["case"]["window"])
        elif op == "full":
            E.embla_prefill_packed(s["shape"], s["cu"], s["q"], s["k"], s["v"], s["out"], alpha=ALPHA, c=C, eps=EPS,
                                   workspace=s["workspace"])
        else:
            E.embla_window_decode_ragged(s["shape"], s["q"], s["k_win"], s["v_win"], s["pos"], s["out"])
    else:
        plain = {"rope": _plain_rope, "window": _plain_window, "full": _plain_full, "decode": _plain_decode}
        plain[op](s)
    if op == "rope":
        return {n: s[n] for n in ("q_out", "k_out", "k_win", "v_win")}
    return {"out": s["out"]}


# ----------------------------------------------------------------------------- work

def work(case):
    op, hkv, lens = case["op"], case["hkv"], _lens(case)
    T = sum(lens)
    if op == "rope":
        late = sum(min(n, case["window"]) for n in lens)
        rows = 2 * T * (HQ + hkv) + 3 * late * hkv  # read and written; rings: k written, v read and written
        return {"bytes": rows * D * 2, "flops": T * (HQ + hkv) * D * (6 if case["norm"] else 3)}
    if op == "decode":
        seen = sum(min(n, case["window"]) for n in lens)
        return {"bytes": seen * hkv * D * 4 + len(lens) * HQ * D * 6, "flops": 4 * D * HQ * seen}
    rows = T * (2 * HQ + 2 * hkv)
    W = case["window"] if op == "window" else 1 << 30
    seen = sum(n * (n + 1) // 2 if n <= W else W * (W + 1) // 2 + (n - W) * W for n in lens)
    return {"bytes": rows * D * 2, "flops": 4 * D * HQ * seen}


# ----------------------------------------------------------------------------- 64 bits

def _exact_rope(s):
    got = {n: s[n].double() for n in ("q_out", "k_out", "k_win", "v_win")}
    W, at = s["case"]["window"], s["cu"].tolist()
    rate = torch.tensor([math.exp(-2 * i / D * math.log(BASE)) for i in range(D // 2)], dtype=torch.float64, device=DEV)
    for b, first in enumerate(s["pos0"].tolist()):
        lo, hi = at[b], at[b + 1]
        pos = torch.arange(first, first + hi - lo, device=DEV)
        turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV), pos.double()[:, None] * rate)[:, None]
        for x, gain, to in ((s["q"], s["q_gain"], "q_out"), (s["k"], s["k_gain"], "k_out")):
            x = x[lo:hi].double()
            if gain is not None:
                x = x * torch.rsqrt(x.pow(2).sum(-1, keepdim=True) / D + EPS) * gain.double()
            pairs = torch.view_as_complex(x.unflatten(-1, (D // 2, 2)).contiguous())
            got[to][lo:hi] = torch.view_as_real(pairs * turn).flatten(-2)
        keep = min(W, hi - lo)
        if keep:
            slots = pos[-keep:] % W
            got["k_win"][b][:, slots] = got["k_out"][hi - keep:hi].transpose(0, 1)
            got["v_win"][b][:, slots] = s["v"][hi - keep:hi].double().transpose(0, 1)
    return got


def _exact_prompt(s, lo, hi, window):
    """Outputs of one sequence, a few hundred queries at a time against the keys they see."""
    hkv, n = s["case"]["hkv"], hi - lo
    G = HQ // hkv
    relu2 = s["case"]["op"] == "full"
    got = torch.zeros(n, HQ, D, dtype=torch.float64, device=DEV)
    for t0 in range(0, n, 512):
        t1 = min(n, t0 + 512)
        j0 = max(0, t0 - window + 1)
        q = s["q"][lo + t0:lo + t1].double().view(t1 - t0, hkv, G, D)
        k, v = s["k"][lo + j0:lo + t1].double(), s["v"][lo + j0:lo + t1].double()
        z = torch.einsum("thgd,jhd->hgtj", q, k)
        ago = torch.arange(t0, t1, device=DEV)[:, None] - torch.arange(j0, t1, device=DEV)
        seen = (ago >= 0) & (ago < window)
        if relu2:
            rq, rk = ((x.square().mean(-1) + EPS).sqrt() for x in (q, k))
            z = z * ALPHA / rq.permute(1, 2, 0)[..., None] / rk.T[:, None, None]
            w = torch.where(seen, z.clamp(min=0.0) ** 2, 0.0)
            w = w / (C + w.sum(-1, keepdim=True))
        else:
            w = torch.softmax(torch.where(seen, z / math.sqrt(D), -math.inf), -1)
        got[t0:t1] = torch.einsum("hgtj,jhd->thgd", w, v).reshape(t1 - t0, HQ, D)
    return got


def exact(case, seed):
    with torch.no_grad():
        s = prepare(case, seed)
        op, hkv = case["op"], case["hkv"]
        if op == "rope":
            return _exact_rope(s)
        if op == "decode":
            out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
            for b, last in enumerate(s["pos"].tolist()):
                W = case["window"]
                slots = torch.arange(max(0, last - W + 1), last + 1, device=DEV) % W
                k, v = s["k_win"][b][:, slots].double(), s["v_win"][b][:, slots].double()
                q = s["q"][b].double().view(hkv, HQ // hkv, D)
                p = torch.softmax(torch.einsum("hgd,hjd->hgj", q, k) / math.sqrt(D), -1)
                out[b] = torch.einsum("hgj,hjd->hgd", p, v).reshape(HQ, D)
            return {"out": out}
        at = s["cu"].tolist()
        window = case.get("window", 1 << 30)
        return {"out": torch.cat([_exact_prompt(s, lo, hi, window) for lo, hi in zip(at, at[1:])])}
