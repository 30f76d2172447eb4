"""The stand-alone operators without a GPU: refusals on the host before any
launch, calls with no rows, and pins of their oracle."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import operators as orc

OK, INVALID, TOO_LARGE = 0, 1, 9
P = 0x10000  # a non-null address that no refused call may touch


@pytest.fixture(scope="module")
def bq():
    from bit_quantized_moe_top_b200 import build
    build.build()
    import bit_quantized_moe_top_b200 as m
    return m


def _norm(bq, **kw):
    base = dict(tokens=4, width=64, dtype=bq.BF16, residual_dtype=bq.BF16, branch=P, branch_stride=64, branch_rows=4,
                residual=P, residual_stride=64, residual_scale=1.0, branch_scale=1.0, pre_weight=P, eps=1e-6,
                residual_out=P, residual_out_stride=64, h=P, h_stride=64)
    base.update(kw)
    return bq._lib().moe_block_norm(ctypes.byref(bq.BlockNormArgs(**base)), None)


@pytest.mark.parametrize("kw", [
    dict(tokens=-1), dict(width=0), dict(dtype=2), dict(dtype=7), dict(residual_dtype=1), dict(residual_dtype=3),
    dict(branch=None, residual=None), dict(residual_out=None, h=None, pre_weight=None), dict(h=None),
    dict(pre_weight=None), dict(branch=None, post_weight=P), dict(branch=None, gate=P), dict(branch=None, pairs=2),
    dict(pairs=-1), dict(pairs=9, inv_pos=P, pair_weights=P), dict(pairs=2), dict(pairs=2, inv_pos=P),
    dict(branch_rows=3), dict(branch_stride=-1), dict(residual_stride=-1), dict(gate=P, gate_channel_stride=2),
    dict(gate=P, gate_token_stride=-1), dict(residual_out_stride=63), dict(h_stride=0), dict(eps=-1.0),
    dict(eps=float("nan")), dict(weight_offset=float("inf")), dict(residual_scale=float("nan")),
    dict(branch_scale=float("inf")),
])
def test_block_norm_refusals(bq, kw):
    assert _norm(bq, **kw) == INVALID


def test_block_norm_limits(bq):
    assert bq._lib().moe_block_norm(None, None) == INVALID
    wide = dict(width=16392, branch_stride=16392, residual_stride=16392, residual_out_stride=16392, h_stride=16392)
    assert _norm(bq, **wide) == TOO_LARGE
    assert _norm(bq, tokens=0, branch_rows=0) == OK


def _quant(bq, x=P, ldx=64, xr=4, dt=0, src=None, rows=4, K=64, q=P, ldq=64, s=P):
    return bq._lib().moe_quantize_rows(x, ldx, xr, dt, src, rows, K, q, ldq, s, None)


@pytest.mark.parametrize("kw", [dict(rows=-1), dict(xr=-1), dict(K=0), dict(dt=2), dict(dt=-1), dict(ldx=-1),
                                dict(ldq=63), dict(rows=3), dict(x=None), dict(q=None), dict(s=None)])
def test_quantize_refusals(bq, kw):
    assert _quant(bq, **kw) == INVALID


def test_quantize_limits(bq):
    assert _quant(bq, K=16385, ldx=16385, ldq=16385) == TOO_LARGE
    assert _quant(bq, rows=0, xr=0, x=None, q=None, s=None) == OK
    assert _quant(bq, rows=0, xr=4, src=P) == OK


def _mm(bq, int8, x=P, ldx=64, w=P, ldw=64, ldwe=64 * 32, off=P, rows=8, E=2, K=64, N=32, y=P, ldy=32, yd=0, dt=0,
        xs=P, ws=P):
    if int8:
        return bq._lib().moe_int8_matmul(x, ldx, xs, w, ldw, ldwe, ws, off, rows, E, K, N, y, ldy, yd, None)
    return bq._lib().moe_grouped_matmul(x, ldx, w, ldw, ldwe, off, rows, E, K, N, dt, y, ldy, yd, None)


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("kw", [dict(rows=-1), dict(E=0), dict(K=0), dict(N=0), dict(N=-4), dict(yd=3), dict(yd=-1),
                                dict(off=None), dict(ldx=-1), dict(ldw=-1), dict(ldwe=-1), dict(ldy=31), dict(x=None),
                                dict(w=None), dict(y=None)])
def test_product_refusals(bq, int8, kw):
    assert _mm(bq, int8, **kw) == INVALID


def test_product_limits(bq):
    for int8 in (False, True):
        assert _mm(bq, int8, E=257) == TOO_LARGE
        assert _mm(bq, int8, rows=0, x=None, y=None) == OK
    assert _mm(bq, True, K=131072, ldx=131072, ldw=131072) == TOO_LARGE
    assert _mm(bq, True, xs=None) == INVALID
    assert _mm(bq, True, ws=None) == INVALID
    assert _mm(bq, False, dt=2) == INVALID


def test_binding_refuses_host_and_mismatched_tensors(bq):
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(2, 32, 64, dtype=torch.bfloat16)
    off = torch.zeros(3, dtype=torch.int32)
    for call in (lambda: bq.moe_grouped_matmul(x, w, off),
                 lambda: bq.moe_int8_matmul(x.to(torch.int8), torch.ones(4), w.to(torch.int8), torch.ones(2, 32), off),
                 lambda: bq.moe_int8_matmul(x, torch.ones(4), w, torch.ones(2, 32), off),
                 lambda: bq.moe_quantize_rows(x), lambda: bq.moe_block_norm(x, x, w_pre=w[0, 0]),
                 lambda: bq.moe_block_norm()):
        with pytest.raises(bq.MoEError) as ei:
            call()
        assert ei.value.status == INVALID


# ---- pins of the oracle ----

def test_oracle_norm_by_hand():
    # rows (3, 4): mean square 12.5; a unit residual of the same row doubles it
    v = np.array([[3.0, 4.0]])
    r, h = orc.block_norm(v, v, w_pre=np.array([1.0, 2.0]), eps=0.0)
    assert np.allclose(r, [[6.0, 8.0]]) and np.allclose(h, [[6 / np.sqrt(50), 16 / np.sqrt(50)]])
    r, _ = orc.block_norm(v, v, w_post=np.array([1.0, 1.0]), gate=np.array([[0.0]]), gate_sigmoid=True,
                          residual_scale=2.0, branch_scale=3.0, eps=0.0)
    assert np.allclose(r, 2 * v + 1.5 * v / np.sqrt(12.5))


def test_oracle_combine_and_offsets():
    rows = np.array([[1.0], [10.0], [100.0]])
    got = orc.combine_rows(rows, np.array([[2, 0], [-1, 1], [3, -7]]), np.array([[0.5, 2.0], [9.0, 0.1], [1.0, 1.0]]))
    assert np.allclose(got, [[52.0], [1.0], [0.0]])
    assert orc.group_ranges([0, 3, 2, 99, -5], 7, 4) == [(0, 3), (3, 3), (3, 7), (7, 7)]


def test_oracle_quantizer_ties_and_empty_rows():
    # max 254: x/2 exactly, so odd values are ties and go to the even code
    codes, scales = orc.quantize_rows(np.array([[254.0, 1.0, 3.0, -5.0], [0, 0, 0, 0], [1, np.inf, 0, 0]]),
                                      [0, 1, 2, -1, 3])
    assert codes[0].tolist() == [127, 0, 2, -2] and scales[0] == 2.0
    assert not codes[1:].any() and scales[1] == 0 and np.isnan(scales[2]) and scales[3] == scales[4] == 0


def test_fp32_quotient_rounds_like_the_exact_one():
    """round(fp32(127 x) / fp32 a) equals the rounding of the exact quotient for
    every pair of fp16 significands (an fp32 quotient never crosses a tie)."""
    a = np.arange(1024, 2048, dtype=np.int64)
    for top in a[::7]:
        x = np.arange(0, top + 1, dtype=np.int64)
        got = np.rint((np.float32(127) * x.astype(np.float32)) / np.float32(top)).astype(np.int64)
        q, r = np.divmod(127 * x, top)
        want = q + ((2 * r > top) | ((2 * r == top) & (q % 2 == 1)))
        assert np.array_equal(got, want)


def test_oracle_grouped_brute_force():
    rng = np.random.default_rng(3)
    x, w = rng.normal(size=(7, 5)), rng.normal(size=(3, 4, 5))
    y, covered = orc.grouped_matmul(x, w, [1, 3, 3, 6])
    assert covered.tolist() == [False, True, True, True, True, True, False]
    for r, e in ((1, 0), (2, 0), (3, 2), (5, 2)):
        for n in range(4):
            assert abs(y[r, n] - sum(x[r, k] * w[e, n, k] for k in range(5))) < 1e-12


def test_pointers_off_their_elements_are_refused(bq):
    """A base that is no multiple of its element's size never reaches a kernel."""
    for name in ("branch", "residual", "residual_out", "h", "pre_weight", "post_weight", "gate"):
        assert _norm(bq, **{name: P + 1}) == INVALID
    assert _norm(bq, residual_dtype=bq.FP32, residual=P + 2, residual_out=P) == INVALID
    assert _quant(bq, x=P + 1) == INVALID
    lib = bq._lib()
    for x, w, y, yd in ((P + 1, P, P, bq.BF16), (P, P + 1, P, bq.BF16), (P, P, P + 1, bq.BF16), (P, P, P + 2, bq.FP32)):
        assert lib.moe_grouped_matmul(x, 64, w, 64, 0, None, 4, 1, 64, 32, bq.BF16, y, 32, yd, None) == INVALID
    assert lib.moe_int8_matmul(P, 64, P, P, 64, 0, P, None, 4, 1, 64, 32, P + 2, 32, bq.FP32, None) == INVALID


@pytest.mark.parametrize("off", [1, 2, 3])
def test_words_off_their_boundary_are_refused(bq, off):
    """Indices, offsets and scales of 4 bytes too: a misaligned one would fault on the device."""
    lib, Q = bq._lib(), P + off
    for name in ("inv_pos", "pair_weights"):
        kw = {"pairs": 2, "inv_pos": P, "pair_weights": P, name: Q}
        assert _norm(bq, **kw) == INVALID
    assert _quant(bq, src=Q) == INVALID
    assert _quant(bq, s=Q) == INVALID
    for int8 in (False, True):
        assert _mm(bq, int8, off=Q) == INVALID
    assert _mm(bq, True, xs=Q) == INVALID
    assert _mm(bq, True, ws=Q) == INVALID


def test_product_extents(bq):
    lib = bq._lib()
    big = (1 << 29) + 1
    for rows, K, N in ((big, 64, 32), (4, (1 << 24) + 1, 32), (4, 64, big)):
        assert lib.moe_grouped_matmul(P, K, P, K, 0, None, rows, 1, K, N, bq.BF16, P, N, bq.BF16, None) == TOO_LARGE
        assert lib.moe_int8_matmul(P, K, P, P, K, 0, P, None, rows, 1, K, N, P, N, bq.BF16, None) == TOO_LARGE


def test_binding_refuses_without_a_device(bq):
    """The calls on torch tensors take CUDA tensors only, name the call in their errors, and check their types."""
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    for name, call in (("moe_block_norm", lambda: bq.moe_block_norm(x, x)),
                       ("moe_block_norm", lambda: bq.moe_block_norm()),
                       ("moe_quantize_rows", lambda: bq.moe_quantize_rows(x)),
                       ("moe_int8_matmul", lambda: bq.moe_int8_matmul(x.to(torch.int8), torch.ones(4), x.to(torch.int8),
                                                                      torch.ones(4))),
                       ("moe_grouped_matmul", lambda: bq.moe_grouped_matmul(x, x))):
        with pytest.raises(bq.MoEError, match=name) as ei:
            call()
        assert ei.value.status == INVALID
    for call in (lambda: bq.moe_quantize_rows(3), lambda: bq.moe_block_norm("x"),
                 lambda: bq.moe_grouped_matmul(None, x)):
        with pytest.raises(TypeError):
            call()
