"""embla_quantize_kv_e4m3 / embla_dequantize_kv_e4m3 against the format's definition in 64 bits.

Codes are compared as values and exactly: code_d is the E4M3 value nearest to 448 x_d / a (ties to
even), which 64-bit arithmetic decides (its quotient is within 2^-52 of the exact one, and a
quotient that is not a tie is at least 2^-13 away from one).  Scales are the fp32 nearest to a / 448.
What is read back is the bf16 of the fp32 product scale * value, exactly."""
import pytest
import torch

import relu_sparse_kv_gb300 as E

pytestmark = pytest.mark.gpu
D = 128
E4M3 = torch.float8_e4m3fn


def definition(x):
    """Rows x (bf16) -> (values of the codes, scales), in 64 bits."""
    f = x.double()
    fine = torch.isfinite(f)
    a = torch.where(fine, f.abs(), 0.0).amax(-1, keepdim=True)
    y = torch.where(a > 0, f * 448.0 / a, 0.0)
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6, max=448.0))) - 3)
    v = torch.where(fine, torch.round(y / step) * step, float("nan"))
    # a / 448 in 64 bits, then fp32: a has 8 bits, so a / 448 is never near a tie of fp32
    return v, torch.where(a > 0, a / 448.0, 1.0).squeeze(-1).float()


def buffers(B, Hkv, ncap, fill=0x5A):
    mk = lambda: torch.full((B, Hkv, ncap, D), fill, dtype=torch.uint8, device="cuda")
    ms = lambda: torch.full((B, Hkv, ncap), -7.0, device="cuda")
    return mk(), ms(), mk(), ms()


def check(B, Hkv, G, ncap, pos, k, v):
    T = k.shape[2]
    kc, ks, vc, vs = buffers(B, Hkv, ncap)
    E.embla_quantize_kv_e4m3(E.Shape(B, G * Hkv, Hkv, D, 0, ncap), pos, k, v, kc, ks, vc, vs)
    torch.cuda.synchronize()
    inside = torch.zeros(ncap, dtype=torch.bool, device="cuda")
    inside[pos:pos + T] = True
    for x, c, s in ((k, kc, ks), (v, vc, vs)):
        want, scale = definition(x)
        got = c[:, :, inside].view(E4M3).double()
        same = (got == want) | (torch.isnan(got) & torch.isnan(want))
        assert same.all(), (~same).sum()
        assert torch.equal(s[:, :, inside], scale)
        assert (c[:, :, ~inside] == 0x5A).all() and (s[:, :, ~inside] == -7.0).all()


@pytest.mark.parametrize("B,Hkv,G,ncap,pos,T", [
    (1, 4, 4, 1, 0, 1), (8, 2, 8, 300, 299, 1), (3, 2, 8, 1037, 500, 37), (1, 1, 4, 129, 1, 128),
    (2, 4, 4, 4096, 0, 4096), (33, 4, 4, 70, 3, 66),
])
def test_quantize_rows(B, Hkv, G, ncap, pos, T):
    g = torch.Generator(device="cuda").manual_seed(B * 100 + T)
    rnd = lambda: (torch.randn(B, Hkv, T, D, device="cuda", generator=g) *
                   torch.exp(4 * torch.randn(B, Hkv, T, 1, device="cuda", generator=g))).bfloat16()
    check(B, Hkv, G, ncap, pos, rnd(), rnd())


def test_every_pair_of_significands_rounds_as_the_definition():
    """Rows whose largest element has each 8-bit significand against elements of every 8-bit
    significand from the largest's exponent down past E4M3's smallest subnormal: every tie and
    every near-tie that bf16 rows can form."""
    a = (torch.arange(128, 256, device="cuda").float() / 128)  # 1 .. 1.99
    x = (torch.arange(128, 256, device="cuda").float()[None] / 128 *
         torch.exp2(-torch.arange(0, 21, device="cuda").float())[:, None]).reshape(-1)  # 21 * 128
    per = D - 1
    n = -(-x.numel() // per)
    x = torch.nn.functional.pad(x, (0, n * per - x.numel())).view(1, n, per).expand(128, n, per)
    rows = torch.cat([a[:, None, None].expand(128, n, 1), x], -1)
    rows = torch.where(rows <= a[:, None, None], rows, -rows / 2)  # the first stays the largest
    rows = rows.reshape(1, 1, 128 * n, D)
    k, v = rows.bfloat16(), (-rows * 2.0 ** 40).bfloat16()
    assert torch.equal(k.float(), rows)
    check(1, 1, 4, 128 * n, 0, k, v)


def test_zero_tiny_huge_infinite_and_nan_rows():
    x = torch.zeros(1, 1, 12, D, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(2)
    z = torch.randn(1, 1, 12, D, device="cuda", generator=g)
    x[:, :, 1] = -0.0
    x[:, :, 2, 5] = 2.0 ** -133             # the smallest bf16
    x[:, :, 3] = z[:, :, 3] * 2.0 ** -128   # subnormals
    x[:, :, 4] = z[:, :, 4] * 2.0 ** -108   # around the switch to division
    x[:, :, 5] = z[:, :, 5] * 2.0 ** -110
    x[:, :, 6] = z[:, :, 6].clamp(-3, 3) * 2.0 ** 126
    x[:, :, 7] = z[:, :, 7].clamp(-3, 3) * 2.0 ** 126
    x[:, :, 7, 3] = float("inf")
    x[:, :, 8] = z[:, :, 8]
    x[:, :, 8, 0], x[:, :, 8, 127], x[:, :, 8, 64] = float("nan"), float("-inf"), float("inf")
    x[:, :, 9] = float("nan")
    x[:, :, 10] = z[:, :, 10] * 2.0 ** -127
    x[:, :, 10, 1] = float("inf")
    x[:, :, 11] = z[:, :, 11]
    k = x.bfloat16()
    check(1, 1, 4, 12, 0, k, k.flip(2).contiguous())


def test_rows_past_32_bit_offsets():
    """Codes of the second plane and of late rows lie past 2^31 bytes, the bf16 rows read back past
    2^32 bytes."""
    B, Hkv, T, ncap = 1, 2, 33, (1 << 24) + 100
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(B, Hkv, T, D, device="cuda", generator=g).bfloat16()
    codes = [torch.empty(B, Hkv, ncap, D, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.empty(B, Hkv, ncap, device="cuda") for _ in range(2)]
    pos = ncap - T
    sh = E.Shape(B, 4 * Hkv, Hkv, D, 0, ncap)
    E.embla_quantize_kv_e4m3(sh, pos, x, x, codes[0], scales[0], codes[1], scales[1])
    back = [torch.zeros(B, Hkv, ncap, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    E.embla_dequantize_kv_e4m3(sh, pos, codes[0], scales[0], codes[1], scales[1], *back, n_rows=T)
    torch.cuda.synchronize()
    v, s = definition(x)
    for c, sc, b in zip(codes, scales, back):
        assert torch.equal(c[:, :, pos:].view(E4M3).double(), v) and torch.equal(sc[:, :, pos:], s)
        assert torch.equal(b[:, :, :T].float(), (v.float() * s[..., None]).bfloat16().float())
        assert (b[:, :, T:T + 50] == 0).all()


@pytest.mark.parametrize("B,Hkv,G,ncap,pos,T,stride", [
    (1, 4, 4, 1, 0, 1, 1), (8, 2, 8, 300, 299, 1, 7), (3, 2, 8, 1037, 500, 37, 37), (1, 1, 4, 129, 1, 128, 200),
    (2, 4, 4, 4096, 0, 4096, 4096),
])
def test_read_back(B, Hkv, G, ncap, pos, T, stride):
    g = torch.Generator(device="cuda").manual_seed(7 * B + T)
    rc = lambda: torch.randint(0, 256, (B, Hkv, ncap, D), device="cuda", generator=g, dtype=torch.int32).to(torch.uint8)
    rs = lambda: torch.exp(8 * torch.randn(B, Hkv, ncap, device="cuda", generator=g))
    kc, vc, ks, vs = rc(), rc(), rs(), rs()  # every code, NaN ones too
    ks[:, :, pos] = float("inf")
    kr = torch.full((B, Hkv, stride, D), 3.0, dtype=torch.bfloat16, device="cuda")
    vr = kr.clone()
    E.embla_dequantize_kv_e4m3(E.Shape(B, G * Hkv, Hkv, D, 0, ncap), pos, kc, ks, vc, vs, kr, vr, n_rows=T)
    torch.cuda.synchronize()
    for c, s, r in ((kc, ks, kr), (vc, vs, vr)):
        want = (c[:, :, pos:pos + T].view(E4M3).float() * s[:, :, pos:pos + T, None]).bfloat16()
        assert torch.equal(r[:, :, :T].float().nan_to_num(nan=1.5), want.float().nan_to_num(nan=1.5))
        assert (r[:, :, T:] == 3.0).all()


def test_read_back_into_rows_on_sixteen_bytes_only():
    B, Hkv, T = 2, 2, 77
    g = torch.Generator(device="cuda").manual_seed(11)
    kc = torch.randint(0, 256, (B, Hkv, T, D), device="cuda", generator=g, dtype=torch.int32).to(torch.uint8)
    ks = torch.rand(B, Hkv, T, device="cuda", generator=g)
    raw = torch.zeros(2, B * Hkv * T * D + 16, dtype=torch.bfloat16, device="cuda")
    rows = []
    for r in raw:
        start = (16 - r.data_ptr()) % 32 // 2
        rows.append(r[start:start + B * Hkv * T * D].view(B, Hkv, T, D))
        assert rows[-1].data_ptr() % 32 == 16
    E.embla_dequantize_kv_e4m3(E.Shape(B, 16, Hkv, D, 0, T), 0, kc, ks, kc, ks, *rows)
    torch.cuda.synchronize()
    want = (kc.view(E4M3).float() * ks[..., None]).bfloat16().float().nan_to_num(nan=1.5)
    assert all(torch.equal(r.float().nan_to_num(nan=1.5), want) for r in rows)


def test_round_trip_error_and_idempotence():
    """scale * decode(code) is within 2^-4 |x| + 2^-10 scale (half a step of E4M3, normal or
    subnormal) of x, plus the bf16 rounding of what is read back (2^-8 of it), and the fp32
    roundings of scale and product (2^-23)."""
    B, Hkv, T = 2, 2, 777
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(B, Hkv, T, D, device="cuda", generator=g).bfloat16()
    sh = E.Shape(B, 8 * Hkv, Hkv, D, 0, T)
    kc, ks, vc, vs = buffers(B, Hkv, T)
    E.embla_quantize_kv_e4m3(sh, 0, x, x, kc, ks, vc, vs)
    kr, vr = torch.empty_like(x), torch.empty_like(x)
    E.embla_dequantize_kv_e4m3(sh, 0, kc, ks, vc, vs, kr, vr)
    torch.cuda.synchronize()
    assert torch.equal(kr, vr) and torch.equal(kc, vc) and torch.equal(ks, vs)
    err = (kr.double() - x.double()).abs()
    lim = x.double().abs() * 2.0 ** -4 + ks.double()[..., None] * 2.0 ** -10
    assert (err <= lim + kr.double().abs() * (2.0 ** -8 + 2.0 ** -23)).all()


def test_quantized_token_is_read_by_the_decode_after_it_on_one_stream():
    """The appended token's codes, written by the call before, reach the 8-bit decode: the same
    result as a cache that held them all along."""
    B, Hkv, G, n = 2, 2, 8, 1000
    g = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g).bfloat16()
    shape = E.Shape(B, G * Hkv, Hkv, D, n, n)
    q, k, v = r(B, G * Hkv, D), r(B, Hkv, n, D), r(B, Hkv, n, D)
    whole = buffers(B, Hkv, n)
    E.embla_quantize_kv_e4m3(shape, 0, k, v, *whole)
    out_a, out_b = torch.empty(B, G * Hkv, D, device="cuda"), torch.empty(B, G * Hkv, D, device="cuda")
    ns_a = torch.empty(B, Hkv, dtype=torch.int32, device="cuda")
    ns_b = torch.empty_like(ns_a)
    E.embla_full_decode_e4m3(shape, q, *whole, out_b, ns_b)
    kt, vt = k[:, :, n - 1:].contiguous(), v[:, :, n - 1:].contiguous()
    for _ in range(5):
        step = [t.clone() for t in whole]
        step[0][:, :, n - 1], step[1][:, :, n - 1], step[2][:, :, n - 1], step[3][:, :, n - 1] = 0, 0, 0, 0
        E.embla_quantize_kv_e4m3(shape, n - 1, kt, vt, *step)
        E.embla_full_decode_e4m3(shape, q, *step, out_a, ns_a)
        torch.cuda.synchronize()
        assert torch.equal(out_a, out_b) and torch.equal(ns_a, ns_b)
    assert E.embla_device_check() == 0


def test_on_a_side_stream_and_in_a_graph():
    B, Hkv, T, ncap = 2, 4, 50, 64
    g = torch.Generator(device="cuda").manual_seed(9)
    k = torch.randn(B, Hkv, T, D, device="cuda", generator=g).bfloat16()
    sh = E.Shape(B, 16, Hkv, D, 0, ncap)
    bufs = buffers(B, Hkv, ncap)
    back = torch.zeros(B, Hkv, T, D, dtype=torch.bfloat16, device="cuda")
    back2 = torch.zeros_like(back)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        E.embla_quantize_kv_e4m3(sh, 7, k, k, *bufs)
        E.embla_dequantize_kv_e4m3(sh, 7, *bufs, back, back2)
    for seed in (1, 2):
        k.copy_(torch.randn(B, Hkv, T, D, device="cuda", generator=g).bfloat16() * seed)
        graph.replay()
        torch.cuda.synchronize()
        v, s = definition(k)
        assert torch.equal(back.float(), (v.float() * s[..., None]).bfloat16().float())
        assert torch.equal(back, back2)


def test_refusals_on_device_tensors():
    B, Hkv, T, ncap = 1, 2, 4, 8
    sh = E.Shape(B, 8 * Hkv, Hkv, D, 0, ncap)
    bufs = buffers(B, Hkv, ncap)
    x = torch.zeros(B, Hkv, T, D, dtype=torch.bfloat16, device="cuda")
    for pos in (-1, 5, 8):
        with pytest.raises(E.EmblaError) as err:
            E.embla_quantize_kv_e4m3(sh, pos, x, x, *bufs)
        assert err.value.status == 1
        with pytest.raises(E.EmblaError):
            E.embla_dequantize_kv_e4m3(sh, pos, *bufs, x, x)
    with pytest.raises(E.EmblaError):
        E.embla_dequantize_kv_e4m3(sh, 0, *bufs, x, x, n_rows=5)  # more rows than k_rows holds
    with pytest.raises(ValueError):
        E.embla_quantize_kv_e4m3(sh, 0, x.transpose(1, 2).contiguous(), x, *bufs)
    with pytest.raises(ValueError):
        E.embla_quantize_kv_e4m3(sh, 0, x.transpose(2, 3), x, *bufs)
    torch.cuda.synchronize()
    assert all((b == f).all() for b, f in zip(bufs, (0x5A, -7.0, 0x5A, -7.0)))
