"""The 8-bit floating-point linear layers without a GPU: the plain 64-bit form
against torch's own e4m3, sizes, and every argument that the entry points
refuse (before anything is launched)."""
import ctypes
import os
import sys
import types

import pytest
import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import fp8_reference as ref  # noqa: E402
from video_vae_decode_b200 import qvae

FAKE = ctypes.c_void_p(0x10000)          # aligned, never dereferenced
FAKE_ODD = ctypes.c_void_p(0x10008)      # not on 16 bytes
FAKE_BYTE = ctypes.c_void_p(0x10001)     # not on an element of bf16
BF16 = ("w", "x", "out", "bias")         # tensors that may start at any element


def off(name):
    return FAKE_BYTE if name in BF16 else FAKE_ODD
OK, ARG, SHAPE, ALIGN = qvae.QVAE_OK, qvae.QVAE_ERR_ARG, qvae.QVAE_ERR_SHAPE, qvae.QVAE_ERR_ALIGN


def test_reference_codes_are_torchs_e4m3():
    u = torch.cat([torch.linspace(-448, 448, 20001), torch.linspace(-0.05, 0.05, 20001)]).to(torch.float32)
    want = u.to(torch.float8_e4m3fn).double()
    assert torch.equal(ref.e4m3(u.double()), want)
    every = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    every = every[torch.isfinite(every)].sort().values
    ties = (every[1:] + every[:-1]) / 2                     # exact in float32
    assert torch.equal(ref.e4m3(ties), ties.float().to(torch.float8_e4m3fn).double())


@pytest.mark.parametrize("amax,e", [(448.0, 0), (448.0 * (1 + 2.0 ** -40), 1), (449.0, 1), (1.0, -8), (1.75, -8), (1.76, -7),
                                    (0.0, -126), (2.0 ** -133, -126), (448 * 2.0 ** -126, -126), (449 * 2.0 ** -126, -125),
                                    (3.3895313892515355e38, 120)])
def test_reference_scale_is_the_least_power_of_two(amax, e):
    got = int(ref.exponents(torch.tensor([amax], dtype=torch.float64))[0])
    assert got == e
    assert amax <= 448 * 2.0 ** got and (got == -126 or amax > 448 * 2.0 ** (got - 1))


def test_sizes():
    assert qvae.qvae_fp8_packed_weight_bytes(1, 128, 128) == 16384
    assert qvae.qvae_fp8_packed_weight_bytes(3, 129, 1) == 3 * 2 * 16384
    assert qvae.qvae_fp8_weight_scale_bytes(3, 129, 513) == 3 * 2 * 2 * 4
    assert qvae.qvae_fp8_code_bytes(5, 129) == 5 * 256
    assert qvae.qvae_fp8_scale_bytes(5, 513) == 5 * 2 * 4
    assert qvae.qvae_fp8_workspace_bytes(5, 129) == 1280 + 256
    assert qvae.qvae_fp8_workspace_bytes(0, 129) == 0
    for bad in ((0, 128, 128), (1, 0, 128), (1, 128, 0), (1025, 128, 128), (1, 1 << 20, 1 << 20), (-1, 128, 128)):
        assert qvae.qvae_fp8_packed_weight_bytes(*bad) == 0
        assert qvae.qvae_fp8_weight_scale_bytes(*bad) == 0
    assert qvae.qvae_fp8_code_bytes((1 << 30) + 1, 128) == 0 and qvae.qvae_fp8_code_bytes(-1, 128) == 0


def weights(E=1, N=128, K=128, w=FAKE, wq=FAKE, ws=FAKE):
    return qvae.lib().qvae_fp8_quantize_weights(E, N, K, w, wq, ws, None)


def test_weight_argument_checks():
    assert weights(w=None) == ARG and weights(wq=None) == ARG and weights(ws=None) == ARG
    assert weights(N=-1) == ARG and weights(N=0) == SHAPE and weights(K=0) == SHAPE and weights(E=0) == SHAPE
    assert weights(E=1025) == SHAPE and weights(N=(1 << 20) + 1) == SHAPE
    assert weights(E=1024, N=128 * 128, K=128 * 128) == SHAPE           # 2^24 blocks
    assert weights(w=FAKE_BYTE) == ALIGN and weights(wq=FAKE_ODD) == ALIGN and weights(ws=FAKE_ODD) == ALIGN


def act(M=4, K=128, op=0, x=FAKE, ldx=None, xq=FAKE, xs=FAKE):
    ldx = (2 * K if op == 1 else K) if ldx is None else ldx
    return qvae.lib().qvae_fp8_quant_act(M, K, op, x, ldx, xq, xs, None)


def test_activation_argument_checks():
    assert act(M=0, x=None) == OK                                       # nothing to do
    assert act(x=None) == ARG and act(xq=None) == ARG and act(xs=None) == ARG
    assert act(M=-1) == ARG and act(K=0) == SHAPE and act(M=(1 << 30) + 1) == SHAPE
    assert act(op=2) == ARG and act(op=-1) == ARG
    assert act(ldx=127) == ARG and act(op=1, ldx=255) == ARG
    assert act(ldx=1 << 62) == SHAPE
    assert act(x=FAKE_BYTE) == ALIGN and act(xq=FAKE_ODD) == ALIGN and act(xs=FAKE_ODD) == ALIGN


def product(M=4, N=128, K=128, xq=FAKE, xs=FAKE, wq=FAKE, ws=FAKE, bias=None, out=FAKE, ldo=None, E=None, offsets=FAKE):
    ldo = N if ldo is None else ldo
    L = qvae.lib()
    if E is None:
        return L.qvae_linear_fp8(M, N, K, xq, xs, wq, ws, bias, out, ldo, None)
    return L.qvae_linear_fp8_grouped(E, M, N, K, xq, xs, offsets, wq, ws, bias, out, ldo, None)


@pytest.mark.parametrize("E", [None, 3])
def test_product_argument_checks(E):
    assert product(E=E, M=0, xq=None, out=None, offsets=None) == OK
    for name in ("xq", "xs", "wq", "ws", "out"):
        assert product(E=E, **{name: None}) == ARG
        assert product(E=E, **{name: off(name)}) == ALIGN
    assert product(E=E, bias=FAKE_BYTE) == ALIGN
    assert product(E=E, M=-1) == ARG and product(E=E, N=0) == SHAPE and product(E=E, K=0) == SHAPE
    assert product(E=E, M=(1 << 30) + 1) == SHAPE
    assert product(E=E, ldo=127) == ARG and product(E=E, ldo=1 << 62) == SHAPE


def test_grouped_argument_checks():
    assert product(E=3, offsets=None) == ARG and product(E=3, offsets=ctypes.c_void_p(0x10002)) == ALIGN
    assert product(E=0) == SHAPE and product(E=1025) == SHAPE and product(E=-1) == ARG


def fused(M=4, N=128, K=128, op=0, x=FAKE, ldx=None, wq=FAKE, ws=FAKE, bias=None, out=FAKE, ldo=None, work=FAKE,
          work_bytes=None, E=None, offsets=FAKE):
    ldx = (2 * K if op == 1 else K) if ldx is None else ldx
    ldo = N if ldo is None else ldo
    work_bytes = qvae.qvae_fp8_workspace_bytes(max(M, 0), K) if work_bytes is None else work_bytes
    L = qvae.lib()
    if E is None:
        return L.qvae_linear_fp8_fused(M, N, K, op, x, ldx, wq, ws, bias, out, ldo, work, work_bytes, None)
    return L.qvae_linear_fp8_grouped_fused(E, M, N, K, op, x, ldx, offsets, wq, ws, bias, out, ldo, work, work_bytes, None)


@pytest.mark.parametrize("M", [1, 4, 300])
@pytest.mark.parametrize("E", [None, 3])
def test_fused_argument_checks(E, M):
    assert fused(E=E, M=0, x=None, out=None, work=None, offsets=None) == OK
    for name in ("x", "wq", "ws", "out", "work"):
        assert fused(E=E, M=M, **{name: None}) == ARG
        assert fused(E=E, M=M, **{name: off(name)}) == ALIGN
    assert fused(E=E, M=M, work_bytes=qvae.qvae_fp8_workspace_bytes(M, 128) - 1) == ARG
    assert fused(E=E, M=M, bias=FAKE_BYTE) == ALIGN
    assert fused(E=E, M=M, op=3) == ARG and fused(E=E, M=M, ldx=127) == ARG and fused(E=E, M=M, op=1, ldx=255) == ARG
    assert fused(E=E, M=M, ldo=127) == ARG and fused(E=E, M=M, N=0) == SHAPE and fused(E=E, M=-M) == ARG
    assert fused(E=E, M=M, ldx=1 << 62) == SHAPE and fused(E=E, M=M, ldo=1 << 62) == SHAPE
    assert fused(E=E, M=M) == ARG and fused(E=E, M=M, op=1, ldo=256) == ARG  # in place
    if E:
        assert fused(E=E, M=M, offsets=None) == ARG
        assert fused(E=E, M=M, offsets=ctypes.c_void_p(0x10002)) == ALIGN


def test_binding_refuses_tensors_that_are_not_on_a_gpu():
    x = torch.zeros((4, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        qvae.fp8_quant_act(x)
    with pytest.raises(ValueError):
        qvae.fp8_quantize_weights(x)
    with pytest.raises(ValueError):
        qvae.Fp8Weights(torch.zeros(16384, dtype=torch.uint8), torch.zeros(4, dtype=torch.uint8), 1, 128, 128)


def test_binding_checks_of_layouts():
    cpu = -1                                                            # what a CPU tensor says its device is
    x = torch.zeros((4, 256), dtype=torch.bfloat16)
    assert qvae._rows(x[:, :128], 128, cpu, "x") == (4, 256)
    assert qvae._rows(x[:1, :128], 128, cpu, "x") == (1, 128)           # one row: its stride says nothing
    for bad in (x[:, ::2], x.t(), x[0].expand(4, 256), x[0], x.half()):
        with pytest.raises(ValueError):
            qvae._rows(bad, bad.shape[-1], cpu, "x")
    with pytest.raises(ValueError):
        qvae._rows(x, 128, cpu, "x")
    with pytest.raises(ValueError):
        qvae._buffer(torch.zeros(3, dtype=torch.int64), torch.int32, 3, cpu, "offsets")
    with pytest.raises(ValueError):
        qvae._buffer(torch.zeros(3, dtype=torch.int32), torch.int32, 4, cpu, "offsets")


def test_footprint_argument_checks():
    out = (ctypes.c_int32 * 3)()
    L = qvae.lib()
    assert L.qvae_get_linear_footprint(0, 4, 128, 128, 1, None) == ARG
    assert L.qvae_get_linear_footprint(-1, 4, 128, 128, 1, out) == ARG
    assert L.qvae_get_linear_footprint(0, 4, 0, 128, 1, out) == SHAPE
    assert L.qvae_get_linear_footprint(0, 4, 128, 128, 1, out) == OK


def footprints():
    """What the CTAs of products take, automatic and forced tilings, single and grouped."""
    sizes = [(m, n, k) for m in (1, 3, 16, 60, 100, 230, 480, 700, 5000) for n in (64, 300, 2048)
             for k in (100, 600, 1500, 4096, 16384)]
    tilings = [(0, 0, 0)] + [(nt, mode, split) for mode in (1, 2) for nt in (16, 32, 48, 112, 128, 224, 240)
                             for split in (1, 2, 3, 4, 8)]
    seen = {}
    try:
        for t in tilings:
            qvae.qvae_set_linear_tiling(*t)
            for m, n, k in sizes:
                for e in (0, 6, 1024):
                    for fused in (False, True):
                        f = qvae.qvae_get_linear_footprint(e, m, n, k, fused)
                        seen.setdefault((f["smem"], f["tmem_cols"], f["cluster"]), (t, m, n, k, e, fused))
    finally:
        qvae.qvae_set_linear_tiling()
    return seen


def test_clusters_that_can_share_an_sm_fit_its_tensor_memory():
    # Clusters wait for one another's CTAs, and a CTA for its TMEM: two clusters that each hold columns on one SM and
    # wait for them on another would wait for ever.  An SM has 228 KB of shared memory (1 KB of each CTA is the
    # system's) and 512 columns.
    seen = footprints()
    clusters = [f for f in seen if f[2] > 1]
    assert len(clusters) > 20 and any(f[1] == 512 for f in clusters)
    room = 228 * 1024
    assert min(f[0] for f in clusters) + 1024 > room / 3                 # never three on an SM
    for a in clusters:
        for b in clusters:
            if a[0] + b[0] + 2 * 1024 <= room:
                assert a[1] + b[1] <= 512, (a, seen[a], b, seen[b])
    for f in seen:
        assert f[0] <= 232448 and f[1] in (32, 64, 128, 256, 512), (f, seen[f])


def test_sizes_beyond_32_bits_are_refused_not_cut():
    big = 2 ** 32 + 128                                                 # its lower 32 bits are a size in range
    for bad in ((big, 1, 128), (1, big, 128), (1, 128, big)):
        assert qvae.qvae_fp8_packed_weight_bytes(*bad) == 0 and qvae.qvae_fp8_weight_scale_bytes(*bad) == 0
        with pytest.raises(qvae.QvaeError):
            qvae.qvae_get_linear_tiling(bad[0], 4, bad[1], bad[2])
        with pytest.raises(qvae.QvaeError):
            qvae.qvae_get_linear_footprint(bad[0], 4, bad[1], bad[2])
    assert qvae.qvae_fp8_code_bytes(4, big) == 0 and qvae.qvae_fp8_scale_bytes(4, big) == 0
    assert qvae.qvae_fp8_workspace_bytes(4, big) == 0
    for bad in ((2 ** 32 + 16, 0, 0, 0), (0, 2 ** 32 + 1, 0, 0), (0, 0, 2 ** 32 + 2, 0), (0, 0, 0, -2 ** 32 - 1)):
        with pytest.raises(qvae.QvaeError):
            qvae.qvae_set_linear_tiling(*bad)
    qvae.qvae_set_linear_tiling()


def test_scale_words_of_another_number_of_rows_are_refused():
    # enough words, but word (g, m) of 6 rows is not where that of 4 rows is (CPU tensors: refused before any launch)
    weights = types.SimpleNamespace(E=1, N=128, K=600, device=-1)
    xq = torch.zeros((5, 4, 128), dtype=torch.uint8)
    for words in (torch.zeros((2, 6), dtype=torch.int32), torch.zeros((2, 3), dtype=torch.int32)):
        with pytest.raises(ValueError, match="x_scale"):
            qvae._product(None, "qvae_linear_fp8", xq, words, weights, None, None, None)


# Clusters of 1..8 CTAs that a B200 holds at a time, with one and with two CTAs to an SM, as it answered (without a device
# the library plans with these).
HELD = ((148, 74, 45, 33, 26, 22, 15, 15), (296, 148, 93, 71, 56, 45, 37, 33))


@pytest.mark.skipif(torch.cuda.is_available(), reason="plans for the device that is there")
def test_the_device_holds_all_clusters_of_a_split():
    # a split has one tile to a cluster and counts on all of them running at once
    sizes = [(200, 2048, 8192), (200, 2304, 8192), (87, 384, 11776), (16, 1152, 8192), (1, 2048, 2048), (300, 4096, 4096)]
    g = torch.Generator().manual_seed(1)
    for _ in range(3000):
        sizes.append(tuple(int(2 ** (float(torch.rand(1, generator=g)) * h)) for h in (11, 14, 15)))
    splits = 0
    for m, n, k in sizes:
        t, f = qvae.qvae_get_linear_tiling(0, m, n, k), qvae.qvae_get_linear_footprint(0, m, n, k, False)
        if t["split"] > 1:
            splits += 1
            clusters = -(-m // t["NT"]) * -(-n // (128 * t["mode"]))
            assert f["cluster"] == t["split"] * t["mode"]
            two = 2 * (f["smem"] + 1024) <= 228 * 1024
            assert clusters <= HELD[two][f["cluster"] - 1], (m, n, k, t, f)
    assert splits > 500
