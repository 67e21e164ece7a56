"""The 8-bit floating-point linear layers on the GPU against 64-bit arithmetic.

Codes and scales are exact (compared bit for bit).  Products are compared with
the 64-bit product of what the codes stand for, within the tolerance that
fp8_reference derives from the arithmetic.
"""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import fp8_reference as ref  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from video_vae_decode_b200 import qvae
    qvae.lib()
    return qvae


def rows(m, k, seed, extra=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((m, k + extra), generator=g) * torch.exp(torch.randn((m, 1), generator=g))
    x = x * torch.where(torch.rand((1, k + extra), generator=g) < 0.02, 20.0, 1.0)
    return x.to(torch.bfloat16).cuda()[:, :k]


def matrix(shape, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * torch.exp(torch.randn(shape[:-1] + (1,), generator=g) * 0.5)
            * shape[-1] ** -0.5).to(torch.bfloat16).cuda()


def code_bits(values):
    """e4m3 bytes of exact code values (float64), every NaN as 0x7F, zeros without sign."""
    b = values.float().to(torch.float8_e4m3fn).view(torch.uint8)
    b = torch.where(torch.isnan(values), torch.full_like(b, 0x7F), b)
    return torch.where(b == 0x80, torch.zeros_like(b), b)


def plain_bits(codes):
    b = torch.where((codes & 0x7F) == 0x7F, torch.full_like(codes, 0x7F), codes)
    return torch.where(b == 0x80, torch.zeros_like(b), b)


def by_row(codes):
    """[M, 128 kb] of codes [kb, M, 128]."""
    return codes.permute(1, 0, 2).reshape(codes.shape[1], -1)


def scale_bytes(words, kb):
    """[M, kb] bytes of scale words [kg, M]."""
    m = words.shape[1]
    return words.contiguous().view(torch.uint8).view(words.shape[0], m, 4).permute(1, 0, 2).reshape(m, -1)[:, :kb]


def unpack(w):
    """(codes [E, 128 nblk, 128 Kb], scale bytes [E, nblk, Kb]) of packed weights, undoing tiles and swizzle."""
    nblk, kb, kg = -(-w.N // 128), -(-w.K // 128), -(-w.K // 512)
    t = w.wq.view(w.E, nblk, kb, 128, 8, 16)
    r = torch.arange(128, device=t.device)
    g = torch.arange(8, device=t.device)
    t = t[:, :, :, r[:, None], g[None, :] ^ (r[:, None] % 8)]
    return (t.permute(0, 1, 3, 2, 4, 5).reshape(w.E, nblk * 128, kb * 128),
            w.w_scale.view(w.E, nblk, kg * 4)[:, :, :kb], w.w_scale.view(w.E, nblk, kg * 4)[:, :, kb:])


def check_product(out, y, s, K):
    err = (out.double() - y).abs()
    tol = ref.tolerance(y, s, K)
    bad = ~(err <= tol)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} outputs off, worst {float((err / tol.clamp(min=1e-300)).max())} of the tolerance"


# ------------------------------------------------------------- quantisers

@pytest.mark.parametrize("m,k,extra", [(1, 1, 0), (1, 128, 0), (3, 127, 0), (5, 130, 0), (33, 512, 8), (31, 520, 3),
                                       (70, 1000, 24), (257, 1176, 0), (2, 8192, 0), (1030, 96, 32)])
def test_activation_codes_and_scales_are_exact(q, m, k, extra):
    x = rows(m, k, m * 7 + k, extra)
    x[:, :1] *= 0.0                                       # zeros among the values
    if m > 2:
        x[1] = 0.0                                        # a row of zeros
        x[2] *= 2.0 ** -120                               # and one of tiny values
    codes, words = q.fp8_quant_act(x)
    want, byte = ref.quantise(x, 1)
    assert torch.equal(scale_bytes(words, byte.shape[1]).long(), byte)
    assert torch.equal(plain_bits(by_row(codes)), code_bits(want))
    assert (scale_bytes(words, words.shape[0] * 4)[:, byte.shape[1]:] == 1).all()
    assert q.qvae_get_error() == 0


def test_activation_codes_of_every_bf16_value(q):
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16)
    x = bits.view(torch.bfloat16).cuda()
    x = torch.where(torch.isfinite(x.float()), x, torch.zeros_like(x)).view(512, 128)
    for y in (x, x.flatten()[torch.randperm(65536, generator=torch.Generator().manual_seed(1)).cuda()].view(64, 1024)):
        codes, words = q.fp8_quant_act(y.contiguous())
        want, byte = ref.quantise(y, 1)
        assert torch.equal(scale_bytes(words, byte.shape[1]).long(), byte)
        assert torch.equal(plain_bits(by_row(codes)), code_bits(want))


def test_activation_groups_with_infinities_and_nan(q):
    x = rows(6, 300, 3)
    x[1, 5], x[2, 130], x[3, 299] = float("inf"), float("nan"), float("-inf")
    codes, words = q.fp8_quant_act(x)
    want, byte = ref.quantise(x, 1)
    assert (byte == 255).sum() == 3
    assert torch.equal(scale_bytes(words, 3).long(), byte)
    # the group's codes are NaN, the padding of its last block included
    assert torch.equal(plain_bits(by_row(codes)), code_bits(want))


@pytest.mark.parametrize("m,k,extra", [(1, 1, 0), (4, 129, 0), (65, 1024, 16), (9, 1000, 0), (40, 333, 5)])
def test_activation_codes_of_silu_mul(q, m, k, extra):
    h = rows(m, 2 * k, m + k, extra)
    if m > 2:
        h[1, :k] = -100.0                                 # exp(-gate) beyond fp32
        h[2, :k] = 90.0
    codes, words = q.fp8_quant_act(h, silu_mul=True)
    v = ref.silu_mul(h)
    # computed in fp32: a value next to a border of the codes may take either neighbour.  exp, the sum, the
    # divide and the product are off by at most (|gate| + 4) 2^-22 of the value; half a step of the code more
    amax = ref.blocks(v, 1).abs().amax(3).amax(1)
    byte = scale_bytes(words, amax.shape[1]).long()
    rel = (h[:, :k].double().abs() + 4) * 2.0 ** -22
    scale = torch.exp2(byte.double() - 127)
    assert ((amax * (1 - 2.0 ** -14) <= 448 * scale) & ((byte == 1) | (amax * (1 + 2.0 ** -14) > 224 * scale))).all()
    got = by_row(codes).view(torch.float8_e4m3fn).double().view(m, -1, 128) * scale[:, :, None]
    got = got.view(m, -1)
    assert (got[:, k:] == 0).all()
    s = scale.repeat_interleave(128, 1)[:, :k]
    half = torch.exp2(torch.floor(torch.log2(torch.clamp(v.abs() / s, min=2.0 ** -6))) - 4) * s
    # a value below a power of two may be rounded on the finer or the coarser side of it.  Where 1 + exp(-gate) is
    # above 2^126 (gate < -87.33) its reciprocal is below fp32's normal numbers and counts as 0; what is lost is at most
    # |gate| exp(gate) |up| <= 87.33 * 2^-126 |up| < 2^-119 |up| there (x exp(-x) falls for x > 1)
    lost = torch.where(h[:, :k] < -87.3, 2.0 ** -119, 0.0) * h[:, k:2 * k].double().abs()
    assert bool(((got[:, :k] - v).abs() <= half * (1 + 2.0 ** -8) + rel * v.abs() + 2.0 ** -149 + lost).all())


@pytest.mark.parametrize("up", [1.0, 2.0 ** 40, 2.0 ** 126])
@pytest.mark.parametrize("gate", [-80.0, -87.0, -87.5, -88.0, -88.5, -89.0, -3.0e38])
def test_silu_mul_of_gates_whose_exponential_is_next_to_the_largest_number(q, gate, up):
    # exp(-gate) is an fp32 number down to gate = -88.72: gate / (1 + exp(-gate)) is one, and so is its product with up.
    # Below it exp(-gate) is infinite in fp32 and the formula gives 0
    m, k = 3, 300
    h = torch.empty((m, 2 * k), dtype=torch.bfloat16, device="cuda")
    h[:, :k] = gate
    h[:, k:] = rows(m, k, 5).clamp(-3.9, 3.9) * up
    codes, words = q.fp8_quant_act(h, silu_mul=True)
    byte = scale_bytes(words, 3)
    scale = torch.exp2(byte.double() - 127)
    got = (by_row(codes).view(torch.float8_e4m3fn).double().view(m, -1, 128) * scale[:, :, None]).view(m, -1)
    if gate <= -89.0:
        assert (got == 0).all() and (byte == 1).all()
        return
    v = ref.silu_mul(h)
    assert float(v.abs().max()) > 2.0 ** -126
    s = scale.repeat_interleave(128, 1)[:, :k]
    half = torch.exp2(torch.floor(torch.log2(torch.clamp(v.abs() / s, min=2.0 ** -6))) - 4) * s
    rel = (abs(gate) + 4) * 2.0 ** -22                    # as in test_activation_codes_of_silu_mul
    assert ((got[:, :k] - v).abs() <= half * (1 + 2.0 ** -8) + rel * v.abs() + 2.0 ** -149).all()
    p = q.fp8_quantize_weights(matrix((64, k), 6))        # quantised by the product: the same codes
    q.qvae_set_linear_tiling(16, 1, 1)
    try:
        one, two = q.linear_fp8_fused(h, p, silu_mul=True), q.linear_fp8(codes, words, p)
        assert torch.equal(one.view(torch.int16), two.view(torch.int16))
    finally:
        q.qvae_set_linear_tiling()
    assert q.qvae_get_error() == 0


@pytest.mark.parametrize("e,n,k", [(1, 1, 1), (1, 128, 128), (2, 130, 200), (1, 1000, 1176), (3, 64, 515), (1, 257, 127)])
def test_packed_weights_are_exact(q, e, n, k):
    w = matrix((e, n, k), e + n + k)
    w[0, 0] *= 2.0 ** 30
    if n > 128:
        w[-1, 128:] = 0.0
    p = q.fp8_quantize_weights(w if e > 1 else w[0])
    assert (p.E, p.N, p.K) == (e, n, k)
    codes, byte, pads = unpack(p)
    assert (pads == 1).all()
    for i in range(e):
        want, wb = ref.quantise(w[i], 128)
        assert torch.equal(byte[i].long(), wb)
        assert torch.equal(plain_bits(codes[i]), code_bits(want))


# --------------------------------------------------------------- products

SIZES = [(1, 1, 1), (1, 128, 128), (1, 2048, 2048), (2, 130, 96), (7, 1000, 1176), (16, 512, 4096), (17, 384, 640),
         (33, 257, 511), (64, 64, 8192), (77, 1000, 1176), (100, 96, 33), (128, 128, 513), (129, 200, 384), (200, 640, 129),
         (240, 256, 256), (241, 384, 256), (300, 1024, 1024), (512, 512, 512), (999, 330, 700), (1500, 1152, 64),
         (4097, 136, 160)]


@pytest.mark.parametrize("m,n,k", SIZES, ids=lambda v: str(v))
@pytest.mark.parametrize("bias", [False, True])
def test_linear_matches_the_exact_product(q, m, n, k, bias):
    x, w = rows(m, k, m + n + k), matrix((n, k), m + 2 * n)
    b = matrix((1, n), 5)[0] * 8 if bias else None
    p = q.fp8_quantize_weights(w)
    out = q.linear_fp8(*q.fp8_quant_act(x), p, b)
    assert q.qvae_get_error() == 0
    y, s = ref.linear(ref.act_values(x), ref.weight_values(w), b)
    check_product(out, y, s, k)
    again = q.linear_fp8_fused(x, p, b)
    assert q.qvae_get_error() == 0
    check_product(again, y, s, k)


def test_scales_of_every_block_reach_their_products(q):
    # one block's scale differs by a lot from the others': a wrong byte or row cannot hide
    m, n, k = 150, 400, 1300
    x, w = rows(m, k, 1), matrix((n, k), 2)
    g = torch.Generator().manual_seed(3)
    for r in range(m):
        for b in range(11):
            x[r, b * 128:(b + 1) * 128] *= 2.0 ** int(torch.randint(-12, 13, (1,), generator=g))
    for i in range(4):
        for b in range(11):
            w[i * 128:(i + 1) * 128, b * 128:(b + 1) * 128] *= 2.0 ** int(torch.randint(-12, 13, (1,), generator=g))
    y, s = ref.linear(ref.act_values(x), ref.weight_values(w))
    p = q.fp8_quantize_weights(w)
    for lo, hi in ((0, 150), (3, 4), (5, 21), (0, 100)):
        check_product(q.linear_fp8_fused(x[lo:hi], p), y[lo:hi], s[lo:hi], k)
    assert q.qvae_get_error() == 0


def test_linear_of_extreme_scales(q):
    x, w = rows(40, 384, 4), matrix((200, 384), 5)
    y, s = ref.linear(ref.act_values(x), ref.weight_values(w))
    for a, b in ((-100, 100), (100, -100), (60, 40), (-40, -60)):
        xs, ws = (x.float() * 2.0 ** a).to(torch.bfloat16), (w.float() * 2.0 ** b).to(torch.bfloat16)
        ya, sa = ref.linear(ref.act_values(xs), ref.weight_values(ws))
        assert torch.equal(ya, y * 2.0 ** (a + b))          # nothing left the formats' ranges
        check_product(q.linear_fp8_fused(xs, q.fp8_quantize_weights(ws)), ya, sa, 384)


@pytest.mark.parametrize("m", [1, 16, 40, 300])
def test_rows_and_channels_with_nan_stay_apart(q, m):
    x, w = rows(m, 300, 9), matrix((300, 300), 10)
    x[0, 17] = float("nan")
    if m > 1:
        x[m - 1, 290] = float("inf")
    w[140, 3] = float("inf")                                # its block: channels 128..255
    out = q.linear_fp8_fused(x, q.fp8_quantize_weights(w))
    y, s = ref.linear(ref.act_values(x), ref.weight_values(w))
    assert torch.isnan(out[0]).all() and torch.isnan(out[m - 1]).all() and torch.isnan(out[:, 128:256]).all()
    assert torch.equal(torch.isnan(out), torch.isnan(y))
    fine = ~torch.isnan(y)
    err, tol = (out.double() - y).abs()[fine], ref.tolerance(y, s, 300)[fine]
    assert (err <= tol).all()


def test_zero_rows_and_zero_weights_give_the_bias(q):
    x, w = rows(20, 256, 1), matrix((128, 256), 2)
    b = matrix((1, 128), 3)[0]
    x[4] = 0
    out = q.linear_fp8_fused(x, q.fp8_quantize_weights(w), b)
    assert torch.equal(out[4], b)
    out = q.linear_fp8_fused(x, q.fp8_quantize_weights(torch.zeros_like(w)), b)
    assert torch.equal(out, b.expand(20, 128))
    assert (q.linear_fp8_fused(x, q.fp8_quantize_weights(torch.zeros_like(w))) == 0).all()


@pytest.mark.parametrize("m,n,k,ldo", [(5, 100, 200, 104), (50, 100, 200, 111), (130, 256, 256, 320), (300, 257, 64, 257),
                                       (600, 512, 128, 520)])
def test_only_the_rows_and_columns_of_out_are_written(q, m, n, k, ldo):
    x, w = rows(m, k, 1, 40), matrix((n, k), 2)
    p = q.fp8_quantize_weights(w)
    guard = 64
    buf = torch.full(((m + 2 * guard) * ldo,), 7.5, dtype=torch.bfloat16, device="cuda")
    off = guard * ldo // 8 * 8
    out = buf[off:off + m * ldo].view(m, ldo)[:, :n]
    got = q.linear_fp8_fused(x, p, out=out)
    assert got.data_ptr() == out.data_ptr() and q.qvae_get_error() == 0
    y, s = ref.linear(ref.act_values(x), ref.weight_values(w))
    check_product(out, y, s, k)
    out.fill_(7.5)
    assert (buf == 7.5).all()


def test_rows_that_do_not_start_on_16_bytes(q):
    buf = rows(50, 1111, 8)
    x = buf[:, :1003]                                       # odd row stride
    w = matrix((96, 1003), 3)
    p = q.fp8_quantize_weights(w)
    assert torch.equal(q.linear_fp8_fused(x, p), q.linear_fp8_fused(x.contiguous(), p))
    one = torch.zeros(50 * 1003 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(50, 1003)
    one.copy_(x)
    out = torch.zeros(50 * 96 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(50, 96)
    assert torch.equal(q.linear_fp8_fused(one, p, out=out), q.linear_fp8_fused(x.contiguous(), p))
    h = rows(30, 2 * 205, 4)                                # the up half of a row starts anywhere
    p = q.fp8_quantize_weights(matrix((64, 205), 5))
    wide = torch.zeros((30, 416), dtype=torch.bfloat16, device="cuda")
    wide[:, :410] = h
    assert torch.equal(q.linear_fp8_fused(h, p, silu_mul=True), q.linear_fp8_fused(wide[:, :410], p, silu_mul=True))


# ---------------------------------------------------------------- grouped

def spans(counts, before=0):
    o = [before]
    for c in counts:
        o.append(o[-1] + c)
    return o


GROUPS = [
    ([5], 0, 0), ([0, 3, 0], 0, 0), ([1, 1, 1, 1], 0, 0), ([16, 0, 17, 1, 0, 33], 2, 3), ([0, 0, 0], 0, 5),
    ([300, 5, 0, 127, 128, 129], 0, 0), ([1] * 70, 0, 0), ([0] * 40 + [9] + [0] * 90, 1, 1), ([241, 0, 480, 239], 7, 9),
    ([700, 1], 0, 0),
]


@pytest.mark.parametrize("counts,before,behind", GROUPS, ids=lambda v: str(v)[:24])
@pytest.mark.parametrize("n,k", [(128, 128), (200, 333), (384, 1024)])
def test_grouped_matches_each_experts_product(q, counts, before, behind, n, k):
    e, o = len(counts), spans(counts, before)
    m = o[-1] + behind
    x, w, b = rows(m, k, m + n), matrix((e, n, k), n), matrix((e, n), 3)
    p = q.fp8_quantize_weights(w)
    offsets = torch.tensor(o, dtype=torch.int32, device="cuda")
    for bias in (None, b):
        out = torch.full((m, n), 3.25, dtype=torch.bfloat16, device="cuda")
        two = out.clone()
        q.linear_fp8_grouped_fused(x, offsets, p, bias, out=out)
        q.linear_fp8_grouped(*q.fp8_quant_act(x), offsets, p, bias, out=two)
        assert q.qvae_get_error() == 0
        for t in (out, two):
            assert (t[:before] == 3.25).all() and (t[o[-1]:] == 3.25).all()
            for i in range(e):
                lo, hi = o[i], o[i + 1]
                if hi > lo:
                    y, s = ref.linear(ref.act_values(x[lo:hi]), ref.weight_values(w[i]), None if bias is None else bias[i])
                    check_product(t[lo:hi], y, s, k)


def test_grouped_rows_equal_the_single_layer(q):
    # one expert's rows give what its matrix alone gives, whatever stands beside them
    counts = [40, 0, 100, 3]
    x, w = rows(143, 512, 1), matrix((4, 256, 512), 2)
    o = torch.tensor(spans(counts), dtype=torch.int32, device="cuda")
    out = q.linear_fp8_grouped_fused(x, o, q.fp8_quantize_weights(w))
    for i, c in enumerate(counts):
        lo = sum(counts[:i])
        if c:
            y, s = ref.linear(ref.act_values(x[lo:lo + c]), ref.weight_values(w[i]))
            check_product(out[lo:lo + c], y, s, 512)
            one = q.linear_fp8_fused(x[lo:lo + c], q.fp8_quantize_weights(w[i]))
            check_product(one, y, s, 512)


@pytest.mark.parametrize("offsets", [[-5, 10, 20, 1000], [30, 20, 10, 0], [0, 1 << 30, -(1 << 30), 40], [50, 50, 50, 50]])
def test_offsets_out_of_range_stay_inside_the_rows(q, offsets):
    m, n, k = 40, 130, 200
    x, w = rows(m, k, 1), matrix((3, n, k), 2)
    buf = torch.full((m + 64, n), 3.25, dtype=torch.bfloat16, device="cuda")
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    q.linear_fp8_grouped_fused(x, off, q.fp8_quantize_weights(w), out=buf[32:32 + m])
    assert q.qvae_get_error() == 0
    assert (buf[:32] == 3.25).all() and (buf[32 + m:] == 3.25).all()
    if offsets == [-5, 10, 20, 1000]:                       # clipped to 0, 10, 20, 40
        for i, (lo, hi) in enumerate(((0, 10), (10, 20), (20, 40))):
            y, s = ref.linear(ref.act_values(x[lo:hi]), ref.weight_values(w[i]))
            check_product(buf[32 + lo:32 + hi], y, s, k)
    if offsets[0] == 50:
        assert (buf == 3.25).all()


def test_many_experts(q):
    e = 1024
    g = torch.Generator().manual_seed(0)
    counts = torch.randint(0, 3, (e,), generator=g).tolist()
    o = spans(counts)
    x, w = rows(o[-1], 96, 1), matrix((e, 64, 96), 2)
    out = q.linear_fp8_grouped_fused(x, torch.tensor(o, dtype=torch.int32, device="cuda"), q.fp8_quantize_weights(w))
    assert q.qvae_get_error() == 0
    who = torch.repeat_interleave(torch.arange(e), torch.tensor(counts)).cuda()
    wv = torch.stack([ref.weight_values(t) for t in w])[who]
    xv = ref.act_values(x)
    y = torch.einsum("mk,mnk->mn", xv, wv)
    s = torch.einsum("mk,mnk->mn", xv.abs(), wv.abs())
    check_product(out, y, s, 96)


# ------------------------------------------- a feed-forward of experts, use

def feed_forward(q, x, offsets, p1, p2, **kw):
    h = q.linear_fp8_grouped_fused(x, offsets, p1, **kw)
    return h, q.linear_fp8_grouped_fused(h, offsets, p2, silu_mul=True, **kw)


@pytest.mark.parametrize("counts", [[1, 0, 2, 1], [16, 1, 0, 15], [100, 0, 301, 20]])
def test_feed_forward_of_experts(q, counts):
    e, d, inner = len(counts), 320, 200
    o = spans(counts)
    x, w1, w2 = rows(o[-1], d, 1), matrix((e, 2 * inner, d), 2), matrix((e, d, inner), 3)
    offsets = torch.tensor(o, dtype=torch.int32, device="cuda")
    h, out = feed_forward(q, x, offsets, q.fp8_quantize_weights(w1), q.fp8_quantize_weights(w2))
    assert q.qvae_get_error() == 0
    for i in range(e):
        lo, hi = o[i], o[i + 1]
        if hi == lo:
            continue
        y, s = ref.linear(ref.act_values(x[lo:hi]), ref.weight_values(w1[i]))
        check_product(h[lo:hi], y, s, d)
        # the second product from the hidden rows as stored, so that one rounding is not counted twice; a code next to a
        # border may take either neighbour (2^-3 of its value): where none does the product's own tolerance holds
        v = ref.act_values(ref.silu_mul(h[lo:hi]))
        y, s = ref.linear(v, ref.weight_values(w2[i]))
        tol = ref.tolerance(y, s, inner) + 2.0 ** -3 * v.abs().amax(1, keepdim=True) * ref.weight_values(w2[i]).abs().amax(1)
        assert ((out[lo:hi].double() - y).abs() <= tol).all()


def test_graph_replay_streams_and_shared_weights(q):
    counts = [30, 0, 4, 66]
    offsets = torch.tensor(spans(counts), dtype=torch.int32, device="cuda")
    xs = [rows(100, 256, s) for s in range(3)]
    p1 = q.fp8_quantize_weights(matrix((4, 384, 256), 2))
    p2 = q.fp8_quantize_weights(matrix((4, 256, 192), 3))
    want = [feed_forward(q, x, offsets, p1, p2)[1] for x in xs]
    torch.cuda.synchronize()
    x = xs[0].clone()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        out = feed_forward(q, x, offsets, p1, p2)[1]
    for i in (1, 2, 0, 0):
        x.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i])
    # other offsets in the captured buffer
    offsets.copy_(torch.tensor([0, 10, 60, 60, 100], dtype=torch.int32))
    direct = feed_forward(q, x, offsets, p1, p2)[1]
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, direct)
    offsets.copy_(torch.tensor(spans(counts), dtype=torch.int32))
    torch.cuda.synchronize()
    # the same weights on several streams at once, each call with buffers of its own
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = [[feed_forward(q, xs[i], offsets, p1, p2, stream=streams[i])[1] for i in range(3)] for _ in range(10)]
    torch.cuda.synchronize()
    assert q.qvae_get_error() == 0
    for r in got:
        for i in range(3):
            assert torch.equal(r[i], want[i])


def test_weights_and_inputs_written_just_before_the_call(q):
    # what a call reads may come from the launch right before it
    w = [matrix((256, 512), s) for s in range(2)]
    p = [q.fp8_quantize_weights(t) for t in w]
    x = rows(24, 512, 4)
    want = [q.linear_fp8_fused(x, t) for t in p]
    codes, words = q.fp8_quant_act(x)
    live = q.Fp8Weights(p[0].wq.clone(), p[0].w_scale.clone(), 1, 256, 512)
    for i in range(20):
        live.w_scale.copy_(p[i % 2].w_scale)
        live.wq.copy_(p[i % 2].wq)
        assert torch.equal(q.linear_fp8_fused(x, live), want[i % 2])
        live.w_scale.copy_(p[1 - i % 2].w_scale)
        live.wq.copy_(p[1 - i % 2].wq)
        check = q.linear_fp8(codes, words, live)
        assert (check.double() - want[1 - i % 2].double()).abs().max() <= 0.02 * want[1 - i % 2].abs().max()
    assert q.qvae_get_error() == 0


def test_empty_calls(q):
    p = q.fp8_quantize_weights(matrix((2, 64, 96), 1))
    x = torch.empty((0, 96), dtype=torch.bfloat16, device="cuda")
    o = torch.zeros(3, dtype=torch.int32, device="cuda")
    assert q.linear_fp8_grouped_fused(x, o, p).shape == (0, 64)
    assert q.linear_fp8_grouped(*q.fp8_quant_act(x), o, p).shape == (0, 64)
    x = rows(10, 96, 1)
    out = torch.full((10, 64), 2.0, dtype=torch.bfloat16, device="cuda")
    q.linear_fp8_grouped_fused(x, o, p, out=out)
    assert (out == 2.0).all()


def test_binding_refusals(q):
    p = q.fp8_quantize_weights(matrix((2, 64, 96), 1))
    one = q.fp8_quantize_weights(matrix((64, 96), 1))
    x = rows(4, 96, 1)
    o = torch.tensor([0, 1, 4], dtype=torch.int32, device="cuda")
    for call in (lambda: q.linear_fp8_fused(x, p),                                            # experts without offsets
                 lambda: q.linear_fp8_fused(x[:, :95], one), lambda: q.linear_fp8_fused(x.float(), one),
                 lambda: q.linear_fp8_fused(x, one, silu_mul=True),
                 lambda: q.linear_fp8_fused(x, one, bias=torch.zeros(63, dtype=torch.bfloat16, device="cuda")),
                 lambda: q.linear_fp8_fused(x, one, bias=torch.zeros(64, device="cuda")),
                 lambda: q.linear_fp8_fused(x, one, out=torch.zeros((3, 64), dtype=torch.bfloat16, device="cuda")),
                 lambda: q.linear_fp8_fused(x, one, out=torch.zeros((4, 64), device="cuda")),
                 lambda: q.linear_fp8_fused(x, one, out=torch.zeros((64, 4), dtype=torch.bfloat16, device="cuda").t()),
                 lambda: q.linear_fp8_grouped_fused(x, o.long(), p), lambda: q.linear_fp8_grouped_fused(x, o[:2], p),
                 lambda: q.linear_fp8_grouped_fused(x, o.cpu(), p), lambda: q.linear_fp8_grouped_fused(x, None, p),
                 lambda: q.linear_fp8_grouped_fused(x, o, p, bias=torch.zeros(64, dtype=torch.bfloat16, device="cuda")),
                 lambda: q.linear_fp8(q.fp8_quant_act(x)[0], q.fp8_quant_act(x)[1][:, :3], one),
                 lambda: q.Fp8Weights(one.wq[:-1], one.w_scale, 1, 64, 96), lambda: q.Fp8Weights(one.wq, one.w_scale[:2], 1, 64, 96),
                 lambda: q.linear_fp8_fused(x.cpu(), one), lambda: q.Fp8Weights(one.wq, one.w_scale.cpu(), 1, 64, 96)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(q.QvaeError) as e:
        q.linear_fp8_fused(x, one, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    assert e.value.status == q.QVAE_ERR_ARG
    words = torch.empty(2048, dtype=torch.uint8, device="cuda")
    with pytest.raises(q.QvaeError) as e:
        q.linear_fp8_fused(x, one, workspace=words[8:])
    assert e.value.status == q.QVAE_ERR_ALIGN


# ---------------------------------------------------------------- tilings

@pytest.mark.parametrize("mode", [1, 2])
@pytest.mark.parametrize("nt", [16, 48, 112, 128, 208, 240])
@pytest.mark.parametrize("ctas", [0, 2])
def test_every_tiling_gives_the_same_products(q, mode, nt, ctas):
    if mode == 1 and nt > 128:
        pytest.skip("single CTAs take at most 128 rows")
    try:
        q.qvae_set_linear_tiling(nt, mode, 1, ctas)
        for m, n, k in ((1, 128, 128), (37, 300, 700), (300, 129, 1100), (500, 520, 96)):
            x, w, b = rows(m, k, m), matrix((n, k), n), matrix((1, n), 3)[0]
            out = q.linear_fp8_fused(x, q.fp8_quantize_weights(w), b)
            assert q.qvae_get_error() == 0
            y, s = ref.linear(ref.act_values(x), ref.weight_values(w), b)
            check_product(out, y, s, k)
        counts = [100, 0, 1, 17, 260, 0, 33]
        o = spans(counts, 3)
        x, w = rows(o[-1] + 2, 600, 1), matrix((7, 300, 600), 2)
        out = torch.full((o[-1] + 2, 300), 3.25, dtype=torch.bfloat16, device="cuda")
        q.linear_fp8_grouped_fused(x, torch.tensor(o, dtype=torch.int32, device="cuda"), q.fp8_quantize_weights(w), out=out)
        assert q.qvae_get_error() == 0
        assert (out[:3] == 3.25).all() and (out[o[-1]:] == 3.25).all()
        for i in range(7):
            if counts[i]:
                y, s = ref.linear(ref.act_values(x[o[i]:o[i + 1]]), ref.weight_values(w[i]))
                check_product(out[o[i]:o[i + 1]], y, s, 600)
    finally:
        q.qvae_set_linear_tiling()


@pytest.mark.parametrize("mode,split", [(1, 2), (1, 3), (1, 5), (1, 8), (2, 2), (2, 3), (2, 4)])
@pytest.mark.parametrize("nt", [16, 64, 128, 240])
def test_tiles_split_along_k(q, nt, mode, split):
    if mode == 1 and nt > 128:
        pytest.skip("single CTAs take at most 128 rows")
    try:
        q.qvae_set_linear_tiling(nt, mode, split)
        for m, n, k in ((1, 128, 2048), (1, 300, 4096), (16, 257, 1100), (37, 300, 2000), (100, 129, 4444), (230, 300, 1500)):
            if -(-m // nt) <= 2 or nt > 16:
                assert q.qvae_get_linear_tiling(0, m, n, k) == {"NT": nt, "mode": mode, "split": min(split, -(-k // 256))}
            x, w, b = rows(m, k, m), matrix((n, k), n), matrix((1, n), 3)[0]
            p = q.fp8_quantize_weights(w)
            out = q.linear_fp8_fused(x, p, b)
            assert q.qvae_get_error() == 0
            y, s = ref.linear(ref.act_values(x), ref.weight_values(w), b)
            check_product(out, y, s, k)
            assert torch.equal(out, q.linear_fp8_fused(x, p, b))      # the same bits every time
            odd = torch.empty((m, n + 3), dtype=torch.bfloat16, device="cuda")[:, 1:n + 1]
            assert torch.equal(out, q.linear_fp8_fused(x, p, b, out=odd))
        counts = [3, 0, 1, 17, 0, 20]
        o = spans(counts, 3)
        x, w = rows(o[-1] + 2, 2100, 1), matrix((6, 300, 2100), 2)
        out = torch.full((o[-1] + 2, 300), 3.25, dtype=torch.bfloat16, device="cuda")
        q.linear_fp8_grouped_fused(x, torch.tensor(o, dtype=torch.int32, device="cuda"), q.fp8_quantize_weights(w), out=out)
        assert q.qvae_get_error() == 0
        assert (out[:3] == 3.25).all() and (out[o[-1]:] == 3.25).all()
        for i in range(6):
            if counts[i]:
                y, s = ref.linear(ref.act_values(x[o[i]:o[i + 1]]), ref.weight_values(w[i]))
                check_product(out[o[i]:o[i + 1]], y, s, 2100)
    finally:
        q.qvae_set_linear_tiling()


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("split", [0, 1, 4])
@pytest.mark.parametrize("m,n,k,extra", [(1, 128, 128, 0), (1, 300, 2048, 0), (3, 200, 8, 8), (7, 136, 1176, 16),
                                         (16, 384, 1000, 0), (16, 128, 4096, 0), (5, 257, 264, 0)])
def test_few_rows_quantised_by_the_product(q, m, n, k, extra, split, silu):
    # one launch: the same codes and scales as the quantiser, so the sums differ by their order at most
    x, w, b = rows(m, (2 if silu else 1) * k, m + n, extra), matrix((n, k), k), matrix((1, n), 3)[0]
    if m > 4:
        x[1] = 0.0
        x[2, k - 1] = float("nan")
    p = q.fp8_quantize_weights(w)
    two = q.linear_fp8(*q.fp8_quant_act(x, silu_mul=silu), p, b)
    try:
        q.qvae_set_linear_tiling(16, 1, split)
        one = q.linear_fp8_fused(x, p, b, silu_mul=silu)
        same = q.linear_fp8(*q.fp8_quant_act(x, silu_mul=silu), p, b)   # the same tiling, quantised before
        assert torch.equal(one.view(torch.int16), same.view(torch.int16))
        many = rows(60, (2 if silu else 1) * k, 1, extra)               # several spans of 16 rows
        assert torch.equal(q.linear_fp8_fused(many, p, b, silu_mul=silu),
                           q.linear_fp8(*q.fp8_quant_act(many, silu_mul=silu), p, b))
        o = torch.tensor([0, 20, 20, 21, 60], dtype=torch.int32, device="cuda")
        pe = q.fp8_quantize_weights(matrix((4, n, k), 8))
        assert torch.equal(q.linear_fp8_grouped_fused(many, o, pe, silu_mul=silu),
                           q.linear_fp8_grouped(*q.fp8_quant_act(many, silu_mul=silu), o, pe))
    finally:
        q.qvae_set_linear_tiling()
    assert q.qvae_get_error() == 0
    assert torch.equal(torch.isnan(one), torch.isnan(two))
    if not silu:
        fine = [i for i in range(m) if not (m > 4 and i == 2)]
        y, s = ref.linear(ref.act_values(x[fine]), ref.weight_values(w), b)
        check_product(one[fine], y, s, k)


@pytest.mark.parametrize("m,n,k,split", [(1, 4096, 4096, 0), (2, 6000, 4096, 2), (2, 128, 8192, 2), (4, 4096, 8192, 0), (1, 18944, 4096, 0),
                                         (2, 2048, 16384, 8)])
def test_few_rows_of_many_experts_and_large_layers(q, m, n, k, split):
    # what the variants keep in shared memory besides their ring: the table of 1024 experts, codes of a long part of K
    x = rows(m, k, 1)
    try:
        q.qvae_set_linear_tiling(16 if split else 0, 1 if split else 0, split)
        w = matrix((n, k), 2)
        p = q.fp8_quantize_weights(w)
        y, s = ref.linear(ref.act_values(x), ref.weight_values(w))
        check_product(q.linear_fp8_fused(x, p), y, s, k)
        many = q.Fp8Weights(p.wq.repeat(1024) if n * k < 1 << 21 else p.wq, p.w_scale.repeat(1024) if n * k < 1 << 21 else p.w_scale,
                            1024 if n * k < 1 << 21 else 1, n, k)
        if many.E > 1:
            o = torch.full((1025,), m, dtype=torch.int32, device="cuda")
            o[:700] = 0
            check_product(q.linear_fp8_grouped_fused(x, o, many), y, s, k)
        assert q.qvae_get_error() == 0
    finally:
        q.qvae_set_linear_tiling()


@pytest.mark.parametrize("seed", range(40))
def test_random_layers(q, seed):
    g = torch.Generator().manual_seed(1000 + seed)
    r = lambda lo, hi: int(torch.randint(lo, hi + 1, (1,), generator=g))
    size = lambda hi: min(hi, max(1, int(2 ** (float(torch.rand(1, generator=g)) * torch.tensor(float(hi)).log2()))))
    m, n, k, e, pad = size(900), size(700), size(2500), r(1, 6), r(0, 9)
    silu, bias, grouped = r(0, 1) == 1, r(0, 1) == 1, r(0, 1) == 1
    x = rows(m, (2 if silu else 1) * k, seed, pad)
    w, b = matrix((e, n, k), seed), matrix((e, n), seed + 1) if bias else None
    wide = torch.full((m, n + r(0, 5)), 3.25, dtype=torch.bfloat16, device="cuda")
    out = wide[:, :n]
    codes, words = q.fp8_quant_act(x, silu_mul=silu)
    byte = scale_bytes(words, -(-k // 128)).double()
    xv = (by_row(codes).view(torch.float8_e4m3fn).double().view(m, -1, 128) * torch.exp2(byte - 127)[:, :, None]).view(m, -1)[:, :k]
    if not silu:
        assert torch.equal(xv, ref.act_values(x))
    if grouped:
        cuts = sorted(r(0, m) for _ in range(e + 1))
        p, o = q.fp8_quantize_weights(w), torch.tensor(cuts, dtype=torch.int32, device="cuda")
        q.linear_fp8_grouped_fused(x, o, p, b, silu_mul=silu, out=out)
        parts = [(i, cuts[i], cuts[i + 1]) for i in range(e)]
        assert (out[:cuts[0]] == 3.25).all() and (out[cuts[-1]:] == 3.25).all()
    else:
        q.linear_fp8_fused(x, q.fp8_quantize_weights(w[0]), None if b is None else b[0], silu_mul=silu, out=out)
        parts = [(0, 0, m)]
    assert q.qvae_get_error() == 0
    assert (wide[:, n:] == 3.25).all()
    for i, lo, hi in parts:
        if hi > lo:
            y, s = ref.linear(xv[lo:hi], ref.weight_values(w[i]), None if b is None else b[i])
            check_product(out[lo:hi], y, s, k)


@pytest.mark.parametrize("m,n,k", [(600000, 4096, 128), (1, 128, 1 << 20), (3, 1 << 20, 40), (1 << 20, 24, 136)])
def test_sizes_beyond_32_bits_and_longest(q, m, n, k):
    gen = torch.Generator(device="cuda").manual_seed(m)
    x = torch.randn((m, k), generator=gen, device="cuda").to(torch.bfloat16)
    w = (torch.randn((n, k), generator=gen, device="cuda") * k ** -0.5).to(torch.bfloat16)
    out = q.linear_fp8_fused(x, q.fp8_quantize_weights(w))
    assert q.qvae_get_error() == 0
    wv = ref.weight_values(w)
    for lo in sorted({0, m // 2, max(0, m - 40)}):      # the first, middle and last rows
        y, s = ref.linear(ref.act_values(x[lo:lo + 40]), wv)
        check_product(out[lo:lo + 40], y, s, k)


def test_more_columns_than_32_bits_count_are_refused(q):
    x = torch.empty((1, 2 ** 32 + 128), dtype=torch.bfloat16, device="cuda")
    for call in (lambda: q.fp8_quant_act(x), lambda: q.fp8_quant_act(x, silu_mul=True), lambda: q.fp8_quantize_weights(x),
                 lambda: q.fp8_quantize_weights(x.view(-1, 1))):
        with pytest.raises(q.QvaeError) as e:
            call()
        assert e.value.status == q.QVAE_ERR_SHAPE


FIRST_CALL = """
import torch
from video_vae_decode_b200 import qvae as q
x = torch.randn(200, 512, device="cuda").to(torch.bfloat16)
w = q.fp8_quantize_weights(torch.randn(3, 256, 512, device="cuda").to(torch.bfloat16))
o = torch.tensor([0, 3, 100, 200], dtype=torch.int32, device="cuda")
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    y = q.linear_fp8_grouped_fused(x, o, w)
    z = q.linear_fp8_grouped_fused(x[:3], torch.clamp(o, max=3), w)
g.replay()
torch.cuda.synchronize()
assert torch.equal(y, q.linear_fp8_grouped_fused(x, o, w))
assert torch.equal(z, q.linear_fp8_grouped_fused(x[:3], torch.clamp(o, max=3), w))
assert q.qvae_get_error() == 0
print("ok")
"""


def test_first_call_of_a_process_inside_a_capture(q):
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    res = subprocess.run([sys.executable, "-c", FIRST_CALL], cwd=root, capture_output=True, text=True, timeout=300)
    assert res.returncode == 0 and res.stdout.strip() == "ok", res.stderr[-2000:]


# -------------------------------------------- exact sums, far offsets, company

@pytest.mark.parametrize("m", [1, 3, 20, 130])
@pytest.mark.parametrize("k", [1 << 20, (1 << 20) - 77, 300001])
def test_every_block_of_a_long_row_counts_once(q, m, k):
    # One channel of each 128-block is not zero, and its products with output n are 2^0 .. 2^7 of eight blocks of n's:
    # the sum 255 * 2^r of row r is exact in fp32 and in bf16, so a block that is missing, counted twice or scaled by
    # another's byte shows.  128 outputs have 1024 blocks in a pass; the passes go through all of them.
    n, kb = 128, -(-k // 128)
    b = torch.arange(kb)
    last = torch.clamp(k - b * 128, max=128)
    at = (b * 128 + (b * 37 + 5) % last).cuda()             # the channel of each block
    a = ((b * 7) % 21 - 10).cuda()                          # its power of two: the scales differ from block to block
    x = torch.zeros((m, k), dtype=torch.bfloat16, device="cuda")
    r = (torch.arange(m) % 5).cuda()
    x[:, at] = torch.exp2((a[None, :] + r[:, None]).float()).to(torch.bfloat16)
    assert torch.equal((x != 0).sum(1), torch.full((m,), kb, device="cuda"))
    codes = q.fp8_quant_act(x)
    for first in range(0, kb, 8 * n):
        mine = b[first:first + 8 * n].cuda()
        w = torch.zeros((n, k), dtype=torch.bfloat16, device="cuda")
        # blocks next to one another belong to different outputs: those at the edge of a part of K too
        out, bit = (mine - first) % n, (mine - first) // n
        w[out, at[mine]] = torch.exp2((bit - a[mine]).float()).to(torch.bfloat16)
        want = torch.zeros(n, dtype=torch.float64, device="cuda").index_add_(0, out, torch.exp2(bit.double()))
        want = torch.exp2(r.double())[:, None] * want
        p = q.fp8_quantize_weights(w)
        assert torch.equal(q.linear_fp8(*codes, p).double(), want)
        assert torch.equal(q.linear_fp8_fused(x, p).double(), want)


def check_sharp(out, y, s, K):
    """check_product where its tolerance is well below the outputs."""
    assert float(ref.tolerance(y, s, K).median()) < 0.05 * float(y.abs().median())
    check_product(out, y, s, K)


def test_codes_beyond_32_bits(q):
    m, n, k = 300000, 40, 8192                              # 2.46e9 codes and values of x
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((m, k), generator=gen, device="cuda", dtype=torch.bfloat16)
    w = matrix((n, k), 2)
    out = q.linear_fp8_fused(x, q.fp8_quantize_weights(w))
    for lo in (0, m // 2, (1 << 31) // k - 20, m - 40):     # also around the 2^31st value
        y, s = ref.linear(ref.act_values(x[lo:lo + 40]), ref.weight_values(w))
        check_sharp(out[lo:lo + 40], y, s, k)


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("m", [9, 50000])
def test_rows_far_apart(q, m, silu):
    # rows whose first values are more than 2^32 values behind the first row's, on 16 bytes and not
    n, k, ldx = 72, 264, (1 << 29) + 9 if m == 9 else 100008
    buf = torch.empty((m - 1) * ldx + 2 * k, dtype=torch.bfloat16, device="cuda")
    x = torch.as_strided(buf, (m, (2 if silu else 1) * k), (ldx, 1))
    dense = rows(m, x.shape[1], 3)
    x.copy_(dense)
    p = q.fp8_quantize_weights(matrix((n, k), 4))
    out = q.linear_fp8_fused(x, p, silu_mul=silu)
    assert torch.equal(out, q.linear_fp8_fused(dense, p, silu_mul=silu))
    if not silu:
        y, s = ref.linear(ref.act_values(dense[-9:]), ref.weight_values(matrix((n, k), 4)))
        check_sharp(out[-9:], y, s, k)


@pytest.mark.parametrize("counts", [[1, 0, 2, 1], [16, 1, 0, 15], [100, 0, 301, 20]])
def test_second_product_of_a_feed_forward_is_that_of_its_codes(q, counts):
    e, d, inner = len(counts), 320, 200
    o = spans(counts)
    x, w1, w2 = rows(o[-1], d, 1), matrix((e, 2 * inner, d), 2), matrix((e, d, inner), 3)
    offsets = torch.tensor(o, dtype=torch.int32, device="cuda")
    h, out = feed_forward(q, x, offsets, q.fp8_quantize_weights(w1), q.fp8_quantize_weights(w2))
    codes, words = q.fp8_quant_act(h, silu_mul=True)        # tested by itself
    byte = scale_bytes(words, -(-inner // 128)).double()
    v = (by_row(codes).view(torch.float8_e4m3fn).double().view(o[-1], -1, 128) * torch.exp2(byte - 127)[:, :, None])
    v = v.view(o[-1], -1)[:, :inner]
    for i in range(e):
        lo, hi = o[i], o[i + 1]
        if hi > lo:
            y, s = ref.linear(v[lo:hi], ref.weight_values(w2[i]))
            check_sharp(out[lo:hi], y, s, inner)


def company(q):
    """Calls of every kind of launch: what each writes, from inputs of its own."""
    from video_vae_decode_b200 import synth

    def linear(m, n, k, silu=False):
        x, p = rows(m, (2 if silu else 1) * k, m), q.fp8_quantize_weights(matrix((n, k), n))
        return lambda: q.linear_fp8_fused(x, p, silu_mul=silu)

    def kind(size):
        t = q.qvae_get_linear_tiling(0, *size)
        return t["mode"], t["split"] > 1

    t = synth.draw_custom(synth.LayerShape(128, 128, 96, 96, T=2), seed=3, outliers=True)
    cx, cb = t.x.cuda(), t.bias.cuda()
    packed, s_w = q.quantize_weights(t.w.cuda())

    def conv():
        xq, s_a = q.act_absmax_quant(cx)
        return q.causal_conv3d_w8a8(xq, s_a, packed, s_w, cb, 128)

    ge = rows(64, 1024, 2)
    gp, go = q.fp8_quantize_weights(matrix((8, 512, 1024), 3)), torch.tensor([0, 3, 3, 20, 21, 40, 50, 63, 64], dtype=torch.int32, device="cuda")
    # how many clusters a device holds decides which sizes are split over pairs
    sizes = [(363, 1964, 11014), (200, 2304, 8192), (469, 1500, 6706), (349, 720, 16341), (16, 8192, 4096), (300, 4096, 4096),
             (16, 1152, 8192), (77, 1000, 1176)]
    assert {(1, True), (1, False), (2, False)} <= {kind(s) for s in sizes}
    return [linear(*s) for s in sizes] + [linear(1, 4096, 8192, True), lambda: q.linear_fp8_grouped_fused(ge, go, gp), conv]


def test_every_kind_of_launch_beside_every_other(q):
    # clusters, pairs and convolutions that wait for their SMs, their TMEM and one another, on four streams
    jobs = company(q)
    want = [job() for job in jobs]
    torch.cuda.synchronize()
    g = torch.Generator().manual_seed(7)
    streams = [torch.cuda.Stream() for _ in range(4)]
    got = []
    for _ in range(12):
        for s in streams:
            i = int(torch.randint(0, len(jobs), (1,), generator=g))
            with torch.cuda.stream(s):
                got.append((i, jobs[i]()))
    torch.cuda.synchronize()
    for i, out in got:
        assert torch.equal(out, want[i]), i


def test_calls_of_several_threads(q):
    import threading

    jobs = company(q)
    want = [job() for job in jobs]
    torch.cuda.synchronize()
    wrong, done = [], []

    def work(k):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                outs = [((k + r) % len(jobs), jobs[(k + r) % len(jobs)]()) for r in range(16)]
                torch.cuda.current_stream().synchronize()
                wrong.extend(i for i, out in outs if not torch.equal(out, want[i]))
            done.append(k)
        except Exception as e:  # (an assertion of the main thread's shows it)
            wrong.append(repr(e))

    threads = [threading.Thread(target=work, args=(k,)) for k in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(120)
    torch.cuda.synchronize()
    assert not wrong and len(done) == 4, wrong
