"""Timed cases of four cache operators, with their plain torch forms:

  quantize   embla_quantize_kv_e4m3    bf16 K and V rows written into the 8-bit caches
  read       embla_dequantize_kv_e4m3  rows of the 8-bit caches read back as bf16
  full       embla_full_decode_shared  full-layer decode of a batch over one shared prefix
                                       and each sequence's own keys
  sparse     embla_sparse_decode_shared  sparse-layer decode over the selected keys of such
                                       a context

Shapes are the library's own: 16 query heads, 4 or 2 KV heads (groups of 4 or 8), head_dim
128, 1,024 selected + 128 recent keys, ReLU^2 weights with 5 % of the scores positive.
"""
import math

import torch

own = False

D = 128
TOPK, RECENT = 1024, 128
BINS = 2048
ALPHA, C, EPS = 1.0, 1.0, 1e-6
E4M3 = torch.float8_e4m3fn
DEV = "cuda"


# ----------------------------------------------------------------------------- cases

def listed():
    return [
        # one decode step's token of a batch of 8 into caches of 2 KV heads: latency
        dict(name="quantize-b8-t1", op="quantize", batch=8, hkv=2, tokens=1, pos=777, stride=1024),
        # a short odd chunk of one prompt, written behind what is there
        dict(name="quantize-b1-t1021", op="quantize", batch=1, hkv=4, tokens=1021, pos=1030, stride=2051),
        # a batch's whole prompts: 8 x 32,768 tokens
        dict(name="quantize-b8-t32k", op="quantize", batch=8, hkv=2, tokens=32768, pos=0, stride=32768),
        # a few hundred rows of one sequence
        dict(name="read-b1-t300", op="read", batch=1, hkv=2, tokens=300, pos=211, stride=2048),
        # a long prompt read back as the bf16 prefix that a batch will share
        dict(name="read-b1-t128k", op="read", batch=1, hkv=4, tokens=131072, pos=0, stride=131072),
        # four sequences behind a short shared prompt: latency counts
        dict(name="full-b4-p2k-n17", op="full", batch=4, hkv=4, prefix=2048, tokens=17),
        # groups of 8, a long prefix of odd length, few own tokens
        dict(name="full-b8-p32k-n129-g8", op="full", batch=8, hkv=2, prefix=32749, tokens=129),
        # an ordinary serving batch: 32 sequences behind a 32k prefix
        dict(name="full-b32-p32k-n300", op="full", batch=32, hkv=4, prefix=32768, tokens=300),
        # a wide batch (two blocks of 128 query rows) with longer own contexts
        dict(name="full-b64-p64k-n1k", op="full", batch=64, hkv=4, prefix=65536, tokens=1024),
        # sparse layers behind the same kinds of context
        dict(name="sparse-b4-p2k-n17", op="sparse", batch=4, hkv=4, prefix=2048, tokens=17),
        dict(name="sparse-b32-p32k-n300", op="sparse", batch=32, hkv=4, prefix=32768, tokens=300),
        dict(name="sparse-b64-p64k-n1k-g8", op="sparse", batch=64, hkv=2, prefix=65536, tokens=1024),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["quantize", "read", "full", "full", "sparse"])
    hkv = rng.choice([2, 4])
    if op in ("quantize", "read"):
        batch = _log(rng, 1, 16)
        tokens = _log(rng, 1, 524288 // (batch * hkv))
        pos = rng.randrange(0, 700)
        return dict(op=op, batch=batch, hkv=hkv, tokens=tokens, pos=pos,
                    stride=pos + tokens + rng.randrange(0, 300))
    batch = _log(rng, 2, 64)
    prefix = _log(rng, 500, 65536)
    return dict(op=op, batch=batch, hkv=hkv, prefix=prefix, tokens=_log(rng, 1, 1024))


def _sizes(case):
    """Units (sequence, KV head), query heads per KV head."""
    return case["batch"] * case["hkv"], 16 // case["hkv"]


# ----------------------------------------------------------------------------- inputs

def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEV)


def _relu2_inputs(case, seed):
    """Queries and keys whose scores D cos(q, k) are positive for about 5 % of the keys of
    every head (the queries of a KV head share a direction that the keys turn away from), no
    score within 1e-3 of zero and no group maximum within 5e-5 of an edge of the histogram's
    bins: keys nearer to one are drawn again, so counts do not hang on a rounding."""
    B, Hkv, P, n = case["batch"], case["hkv"], case["prefix"], case["tokens"]
    G = 16 // Hkv
    gen = torch.Generator(device=DEV).manual_seed(seed)
    u = torch.nn.functional.normalize(_randn(gen, Hkv, D), dim=-1)
    q = (_randn(gen, B, Hkv, G, D) + 8.0 * u[None, :, None]).bfloat16()
    qn = q.float() * torch.rsqrt(q.float().square().mean(-1, keepdim=True) + EPS)

    def keys_of(h, count):
        return (_randn(gen, count, D) - 2.85 * u[h]).bfloat16()

    def near(k, rows):  # rows [b, G, D] that read these keys
        kn = k.float() * torch.rsqrt(k.float().square().mean(-1, keepdim=True) + EPS)
        s = (rows.reshape(-1, D) @ kn.T).view(rows.shape[0], G, -1) * ALPHA
        sig = s.amax(1)
        low, high = _edges(sig)
        return ((s.abs() < 1e-3).any(1) | (sig - low < 5e-5) | (high - sig < 5e-5)).any(0)

    def draw_keys(h, count, rows):
        k = keys_of(h, count)
        bad = near(k, rows).nonzero().squeeze(1) if count else torch.zeros(0, dtype=torch.long)
        for _ in range(40):
            if bad.numel() == 0:
                break
            fresh = keys_of(h, bad.numel())
            k[bad] = fresh
            bad = bad[near(fresh, rows)]
        return k

    kp = torch.stack([draw_keys(h, P, qn[:, h]) for h in range(Hkv)])
    kc = torch.stack([draw_keys(h, n, qn[b:b + 1, h]) for b in range(B) for h in range(Hkv)])
    vp = _randn(gen, Hkv, P, D).bfloat16()
    vc = _randn(gen, B, Hkv, n, D).bfloat16()
    return q.view(B, 16, D), kp, vp, kc.view(B, Hkv, n, D), vc


def _edges(sig):
    """The edges of the histogram bin (the order key's top 11 bits: sign, exponent and two
    bits of the fraction) that each score lies in."""
    bits = sig.contiguous().view(torch.int32)
    toward = (bits & ~0x1FFFFF).view(torch.float32)
    away = ((bits & ~0x1FFFFF) + 0x200000).view(torch.float32)
    return torch.minimum(toward, away), torch.maximum(toward, away)


def prepare(case, seed):
    op, B, Hkv = case["op"], case["batch"], case["hkv"]
    gen = torch.Generator(device=DEV).manual_seed(seed)
    st = dict(case=case)
    if op in ("quantize", "read"):
        T, pos, stride = case["tokens"], case["pos"], case["stride"]
        # rows of different sizes, as layers and tokens have them
        k = (_randn(gen, B, Hkv, T, D) * torch.exp(_randn(gen, B, Hkv, T, 1))).bfloat16()
        v = (_randn(gen, B, Hkv, T, D) * torch.exp(_randn(gen, B, Hkv, T, 1))).bfloat16()
        st["k_codes"] = torch.zeros(B, Hkv, stride, D, dtype=torch.uint8, device=DEV)
        st["v_codes"] = torch.zeros(B, Hkv, stride, D, dtype=torch.uint8, device=DEV)
        st["k_scales"] = torch.ones(B, Hkv, stride, device=DEV)
        st["v_scales"] = torch.ones(B, Hkv, stride, device=DEV)
        if op == "quantize":
            st["k_rows"], st["v_rows"] = k, v
        else:
            for x, name in ((k, "k"), (v, "v")):
                codes, scales = _to_codes(x)
                st[name + "_codes"][:, :, pos:pos + T] = codes
                st[name + "_scales"][:, :, pos:pos + T] = scales
            st["k_rows"] = torch.zeros(B, Hkv, T, D, dtype=torch.bfloat16, device=DEV)
            st["v_rows"] = torch.zeros(B, Hkv, T, D, dtype=torch.bfloat16, device=DEV)
        ctx, cache = pos + T, stride
    else:
        P, n = case["prefix"], case["tokens"]
        N = P + n
        if op == "full":
            q, kp, vp, kc, vc = _relu2_inputs(case, seed)
            st["sel_scores"] = torch.zeros(B, Hkv, (N + 7) // 8 * 8, device=DEV)
            st["sel_hist"] = torch.zeros(B, Hkv, BINS, dtype=torch.int32, device=DEV)
            st["n_surv"] = torch.zeros(B, Hkv, dtype=torch.int32, device=DEV)
        else:
            q = _randn(gen, B, 16, D).bfloat16()
            kp, vp = _randn(gen, Hkv, P, D).bfloat16(), _randn(gen, Hkv, P, D).bfloat16()
            kc, vc = _randn(gen, B, Hkv, n, D).bfloat16(), _randn(gen, B, Hkv, n, D).bfloat16()
            idx = torch.zeros(B, Hkv, TOPK + RECENT, dtype=torch.int32, device=DEV)
            old = max(0, N - RECENT)
            top = min(old, TOPK)
            for b in range(B):
                idx[b, :, :top] = torch.rand(Hkv, old, generator=gen, device=DEV).topk(top).indices.sort().values
            idx[:, :, top:top + N - old] = torch.arange(old, N, device=DEV, dtype=torch.int32)
            st["idx"] = idx
            st["count"] = torch.full((B, Hkv), top + N - old, dtype=torch.int32, device=DEV)
        st.update(q=q, k_prefix=kp, v_prefix=vp, k_cache=kc, v_cache=vc,
                  out=torch.zeros(B, 16, D, device=DEV))
        ctx, cache = n, n
    if own:
        import relu_sparse_kv_gb300 as E
        st["shape"] = E.Shape(B, 16, Hkv, D, ctx, cache)
        if op == "full":
            need = E.embla_full_decode_shared_workspace_size(st["shape"], case["prefix"])
            st["workspace"] = torch.empty(max(need, 16), dtype=torch.uint8, device=DEV)
    return st


# ----------------------------------------------------------------------------- plain forms

def _to_codes(x):
    """Rows of bf16 as E4M3 codes and one scale per row: the largest magnitude maps to 448."""
    f = x.float()
    amax = f.abs().amax(-1, keepdim=True)
    codes = torch.where(amax > 0, f * 448.0 / amax, 0.0).to(E4M3).view(torch.uint8)
    scales = torch.where(amax > 0, amax / 448.0, 1.0).squeeze(-1)
    return codes, scales


def _plain_quantize(s):
    pos, T = s["case"]["pos"], s["case"]["tokens"]
    codes, scales = _to_codes(s["k_rows"])
    s["k_codes"][:, :, pos:pos + T] = codes
    s["k_scales"][:, :, pos:pos + T] = scales
    codes, scales = _to_codes(s["v_rows"])
    s["v_codes"][:, :, pos:pos + T] = codes
    s["v_scales"][:, :, pos:pos + T] = scales


def _plain_read(s):
    pos, T = s["case"]["pos"], s["case"]["tokens"]
    k = s["k_codes"][:, :, pos:pos + T].view(E4M3).float() * s["k_scales"][:, :, pos:pos + T, None]
    v = s["v_codes"][:, :, pos:pos + T].view(E4M3).float() * s["v_scales"][:, :, pos:pos + T, None]
    s["k_rows"].copy_(k.bfloat16())
    s["v_rows"].copy_(v.bfloat16())


def _normed(x):
    f = x.float()
    return f / torch.sqrt(f.square().mean(-1, keepdim=True) + EPS)


def _plain_full(s):
    B, Hkv, P, n = (s["case"][k] for k in ("batch", "hkv", "prefix", "tokens"))
    G, N = 16 // Hkv, P + n
    q = _normed(s["q"]).view(B, Hkv, G, D)
    qt = q.transpose(0, 1).reshape(Hkv, B * G, D)
    sp = (qt @ _normed(s["k_prefix"]).transpose(1, 2)).view(Hkv, B, G, P).transpose(0, 1)
    so = q @ _normed(s["k_cache"]).transpose(2, 3)
    score = torch.cat([sp, so], -1) * ALPHA
    w = score.clamp(min=0.0).square()
    wp = w[..., :P].transpose(0, 1).reshape(Hkv, B * G, P)
    num = (wp @ s["v_prefix"].float()).view(Hkv, B, G, D).transpose(0, 1)
    num = num + w[..., P:] @ s["v_cache"].float()
    s["out"].copy_((num / (w.sum(-1, keepdim=True) + C)).reshape(B, 16, D))
    sigma = score.amax(2)
    s["n_surv"].copy_((sigma > 0).sum(-1))
    s["sel_scores"][..., :N] = sigma
    bits = sigma.view(torch.int32).long()
    order = torch.where(bits < 0, -1 - bits, bits + (1 << 31)) >> 21
    order = (order + torch.arange(B * Hkv, device=DEV).view(B, Hkv, 1) * BINS).view(-1)
    s["sel_hist"].copy_(torch.bincount(order, minlength=B * Hkv * BINS).view(B, Hkv, BINS))


def _plain_sparse(s):
    B, Hkv, P, n = (s["case"][k] for k in ("batch", "hkv", "prefix", "tokens"))
    j = s["idx"].long()
    g = torch.arange(Hkv, device=DEV).view(1, Hkv, 1)
    b = torch.arange(B, device=DEV).view(B, 1, 1)
    shared = (j < P)[..., None]
    jp, jo = j.clamp(max=P - 1), (j - P).clamp(min=0)
    k = torch.where(shared, s["k_prefix"][g, jp], s["k_cache"][b, g, jo]).float()
    v = torch.where(shared, s["v_prefix"][g, jp], s["v_cache"][b, g, jo]).float()
    q = s["q"].float().view(B, Hkv, 16 // Hkv, D)
    z = q @ k.transpose(2, 3) * D ** -0.5
    past = torch.arange(j.shape[-1], device=DEV) >= s["count"][..., None]
    z = z.masked_fill(past[:, :, None], -math.inf)
    p = torch.exp(z - z.amax(-1, keepdim=True))
    s["out"].copy_((p @ v / p.sum(-1, keepdim=True)).reshape(B, 16, D))


def run(s):
    op = s["case"]["op"]
    if own:
        import relu_sparse_kv_gb300 as E
        if op == "quantize":
            E.embla_quantize_kv_e4m3(s["shape"], s["case"]["pos"], s["k_rows"], s["v_rows"], s["k_codes"],
                                     s["k_scales"], s["v_codes"], s["v_scales"])
        elif op == "read":
            E.embla_dequantize_kv_e4m3(s["shape"], s["case"]["pos"], s["k_codes"], s["k_scales"],
                                       s["v_codes"], s["v_scales"], s["k_rows"], s["v_rows"])
        elif op == "full":
            E.embla_full_decode_shared(s["shape"], s["case"]["prefix"], s["q"], s["k_prefix"], s["v_prefix"],
                                       s["k_cache"], s["v_cache"], s["out"], s["n_surv"], s["sel_scores"],
                                       s["sel_hist"], alpha=ALPHA, c=C, eps=EPS, workspace=s["workspace"])
        else:
            E.embla_sparse_decode_shared(s["shape"], s["case"]["prefix"], s["q"], s["k_prefix"], s["v_prefix"],
                                         s["k_cache"], s["v_cache"], s["idx"], s["count"], s["out"])
    else:
        plain = {"quantize": _plain_quantize, "read": _plain_read, "full": _plain_full, "sparse": _plain_sparse}
        plain[op](s)
    if op == "quantize":
        return {"k_codes": s["k_codes"].view(E4M3), "k_scales": s["k_scales"],
                "v_codes": s["v_codes"].view(E4M3), "v_scales": s["v_scales"]}
    if op == "read":
        return {"k_rows": s["k_rows"], "v_rows": s["v_rows"]}
    if op == "full":
        return {"out": s["out"], "n_surv": s["n_surv"], "sel_scores": s["sel_scores"], "sel_hist": s["sel_hist"]}
    return {"out": s["out"]}


# ----------------------------------------------------------------------------- work

def work(case):
    units, G = _sizes(case)
    op, B, Hkv = case["op"], case["batch"], case["hkv"]
    if op in ("quantize", "read"):
        rows = 2 * units * case["tokens"]  # K and V
        return {"bytes": rows * (D * 2 + D + 4), "flops": rows * D * 2}
    P, n = case["prefix"], case["tokens"]
    N = P + n
    qo = B * 16 * D * (2 + 4)
    if op == "full":
        # every K row once; V rows that some reading head weighs above zero (5 % per head)
        live_p, live_o = 1 - 0.95 ** (B * G), 1 - 0.95 ** G
        rows = Hkv * P * (1 + live_p) + units * n * (1 + live_o)
        return {"bytes": rows * D * 2 + qo + units * (N * 4 + BINS * 4 + 4),
                "flops": 2 * B * 16 * D * N * 1.05}
    count = min(N, TOPK + RECENT)
    # prefix rows that some sequence selects, once; own rows; the indices
    own_rows = min(n, RECENT) + max(0, n - RECENT) * min(1.0, TOPK / max(1, N - RECENT))
    of_prefix = (count - own_rows) / P
    rows = Hkv * P * (1 - (1 - min(1.0, of_prefix)) ** B) + units * own_rows
    return {"bytes": rows * D * 4 + qo + units * (count * 4 + 4), "flops": 4 * B * 16 * D * count}


# ----------------------------------------------------------------------------- 64 bits

def _round_e4m3(y):
    """The nearest E4M3 value (ties to even) of each y, |y| <= 448: three fraction bits, the
    smallest exponent -6."""
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step  # torch.round takes ties to even


def exact(case, seed):
    with torch.no_grad():
        s = prepare(case, seed)
        op, B, Hkv = case["op"], case["batch"], case["hkv"]
        if op in ("quantize", "read"):
            pos, T = case["pos"], case["tokens"]
            if B * Hkv * case["stride"] * D > 1 << 28:
                return None
            got = {}
            for name in ("k", "v"):
                codes, scales = s[name + "_codes"].view(E4M3).double(), s[name + "_scales"].double()
                if op == "read":
                    got[name + "_rows"] = codes[:, :, pos:pos + T] * scales[:, :, pos:pos + T, None]
                    continue
                x = s[name + "_rows"].double()
                top = x.abs().max(-1).values
                codes[:, :, pos:pos + T] = _round_e4m3(x * 448 / top[..., None])
                scales[:, :, pos:pos + T] = top / 448
                got[name + "_codes"], got[name + "_scales"] = codes, scales
            return got
        P, n, G = case["prefix"], case["tokens"], 16 // Hkv
        out = torch.zeros(B, 16, D, dtype=torch.float64, device=DEV)
        if op == "sparse":
            for b in range(B):
                for g in range(Hkv):
                    j = s["idx"][b, g, :int(s["count"][b, g])].long()
                    k = torch.cat([s["k_prefix"][g], s["k_cache"][b, g]])[j].double()
                    v = torch.cat([s["v_prefix"][g], s["v_cache"][b, g]])[j].double()
                    z = s["q"][b, g * G:(g + 1) * G].double() @ k.T / math.sqrt(D)
                    out[b, g * G:(g + 1) * G] = torch.softmax(z, -1) @ v
            return {"out": out}
        n_surv = torch.zeros_like(s["n_surv"])
        sel = s["sel_scores"].double()
        hist = torch.zeros_like(s["sel_hist"])
        edges = _bin_starts()
        for g in range(Hkv):
            kp, vp = s["k_prefix"][g].double(), s["v_prefix"][g].double()
            for b in range(B):
                k = torch.cat([kp, s["k_cache"][b, g].double()])
                v = torch.cat([vp, s["v_cache"][b, g].double()])
                q = s["q"][b, g * G:(g + 1) * G].double()
                z = ALPHA * (q @ k.T) / torch.outer((q.pow(2).mean(-1) + EPS).sqrt(),
                                                    (k.pow(2).mean(-1) + EPS).sqrt())
                w = torch.relu(z) ** 2
                out[b, g * G:(g + 1) * G] = (w @ v) / (C + w.sum(-1))[:, None]
                best = z.max(0).values
                n_surv[b, g] = (best > 0).sum()
                sel[b, g, :P + n] = best
                at = torch.bucketize(best.float(), edges, right=True) - 1
                hist[b, g] = torch.bincount(at, minlength=BINS)
        return {"out": out, "n_surv": n_surv, "sel_scores": sel, "sel_hist": hist}


def _bin_starts():
    """The smallest score of every histogram bin (finite ones; the NaN bins keep infinities)."""
    key = torch.arange(BINS, dtype=torch.int64) << 21
    bits = torch.where(key >= 1 << 31, key - (1 << 31), (1 << 32) - 1 - key)
    bits = torch.where(bits >= 1 << 31, bits - (1 << 32), bits).to(torch.int32)
    start = bits.view(torch.float32)
    low = torch.where(torch.arange(BINS) < BINS // 2, -math.inf, math.inf)
    return torch.where(torch.isnan(start), low, start).to(DEV)
