"""GPU parity of the stand-alone operators against their fp64 oracle.

Tolerances, derived from the arithmetic:

* one rounding to the output type: half a step, ``finfo.eps / 2`` relative (and
  half the smallest subnormal);
* fp32 steps: 2^-24 relative each. The norms sum squares over chains of at most
  32 terms per thread, 5 shuffles and 32 warps, enter through a square root
  (half the relative error) and take about ten more operations: 96 * 2^-24 of
  the terms' magnitudes covers them;
* 16-bit products: K fp32 additions whose partial sums stay below sum |x w|,
  truncated to 24 bits in the worst case: K * 2^-23 * sum |x w|;
* 8-bit products: the int32 sum is exact; its conversion and two
  multiplications: 3 * 2^-24.

Most products use small whole numbers, whose sums are exact in fp32 in any
order: the outputs must then be the exact values, rounded once.
"""
import numpy as np
import pytest
import torch

from oracle import operators as orc
from product_forms import FORMS

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
U = 2.0 ** -24


@pytest.fixture(scope="module")
def bq():
    from bit_quantized_moe_top_b200 import build
    build.build()
    import bit_quantized_moe_top_b200 as m
    return m


def f64(t):
    return t.detach().double().cpu().numpy()


def half_step(dtype, ref):
    fi = torch.finfo(dtype)
    return fi.eps / 2 * np.abs(ref) + fi.smallest_normal * fi.eps / 2


def check(got, ref, tol, what):
    g = f64(got)
    assert g.shape == ref.shape
    bad = ~(np.abs(g - ref) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} outside, worst {np.nanmax(np.abs(g - ref) / np.maximum(tol, 1e-300)):.3g} x tolerance"


def rnd(gen, shape, std, dtype):
    return (torch.randn(shape, generator=gen, dtype=torch.float32) * std).to(dtype).cuda()


def ints(gen, shape, lo, hi, dtype):
    return torch.randint(lo, hi + 1, shape, generator=gen).to(dtype).cuda()


def seeded(*key):
    return torch.Generator().manual_seed(sum((i + 1) * 7919 ** i * int(k) for i, k in enumerate(key)) % (1 << 62))


# ---------------------------------------------------------------------------
# norms around a block
# ---------------------------------------------------------------------------

def norm_case(bq, T, K, dtype, res, k=0, gate="none", post=True, pre=True, sig=False, scale=1.5, rscale=0.75,
              offset=0.0, pad=0, drop=False, shift=0):
    gen = seeded(T, K, k, len(gate), pad)
    dt, rt = DT[dtype], DT[res]

    def mat(rows, std, t):
        return rnd(gen, (rows, K + pad + shift), std, t)[:, shift:shift + K]

    rows = T * max(k, 1) + 3 if k else T
    y, r = mat(rows, 0.7, dt), mat(T, 1.0, rt)
    inv = pw = None
    if k:
        inv = torch.randint(0, rows, (T, k), generator=gen).to(torch.int32)
        if drop:
            inv[::2, -1] = -1
            inv[0, :] = rows
        inv = inv.cuda()
        pw = torch.softmax(torch.randn(T, k, generator=gen), 1).cuda()
    w_pre = rnd(gen, (K,), 0.2, dt) + 1 if pre else None
    w_post = rnd(gen, (K,), 0.2, dt) + 1 if post else None
    g = {"none": None, "channel": (K,), "token": (T, 1), "element": (T, K)}[gate]
    g = None if g is None else (mat(T, 1.0, dt) if gate == "element" else rnd(gen, g, 1.0, dt))
    kw = dict(w_pre=w_pre, w_post=w_post, gate=g, gate_sigmoid=sig, residual_scale=rscale, branch_scale=scale,
              eps=1e-5, weight_offset=offset, inv_pos=inv, pair_weights=pw)
    return y, r, kw


def norm_reference(r, y, kw):
    c = {k: (f64(v) if isinstance(v, torch.Tensor) else v) for k, v in kw.items()}
    ref, h = orc.block_norm(f64(r), f64(y), c["w_pre"], c["w_post"], c["gate"], c["gate_sigmoid"], c["residual_scale"],
                            c["branch_scale"], c["eps"], c["weight_offset"], c["inv_pos"], c["pair_weights"])
    # magnitudes of the terms of r': the same formula with every term positive
    b = np.abs(f64(y)) if c["inv_pos"] is None else orc.combine_rows(np.abs(f64(y)), c["inv_pos"], np.abs(c["pair_weights"]))
    if c["w_post"] is not None:
        v = f64(y) if c["inv_pos"] is None else orc.combine_rows(f64(y), c["inv_pos"], c["pair_weights"])
        b = b / np.sqrt((v * v).mean(1, keepdims=True) + c["eps"]) * (abs(c["weight_offset"]) + np.abs(c["w_post"]))
    if c["gate"] is not None:
        b = b * (1.0 if c["gate_sigmoid"] else np.abs(c["gate"]))
    mag = np.abs(c["residual_scale"] * f64(r)) + abs(c["branch_scale"]) * b
    tol_r = 96 * U * mag
    tol_h = None
    if h is not None:
        inv = 1 / np.sqrt((ref * ref).mean(1, keepdims=True) + c["eps"])
        tol_h = (tol_r + 96 * U * np.abs(ref)) * inv * (abs(c["weight_offset"]) + np.abs(c["w_pre"]))
    return ref, h, tol_r, tol_h


@pytest.mark.parametrize("T,K,dtype,res,opt", [
    (1, 64, "bf16", "bf16", {}),
    (1, 4096, "bf16", "fp32", dict(k=8)),
    (3, 8, "fp16", "fp16", dict(gate="token", sig=True)),
    (5, 7, "bf16", "bf16", dict(gate="element")),
    (33, 1, "fp16", "fp32", {}),
    (17, 2048, "bf16", "bf16", dict(k=2, gate="channel", drop=True)),
    (9, 2056, "fp16", "fp32", dict(gate="element", sig=True, offset=1.0)),
    (13, 4096, "fp16", "fp16", dict(k=6, gate="token", sig=True)),
    (4, 7168, "bf16", "fp32", dict(k=8, drop=True, post=False)),
    (2, 16384, "bf16", "bf16", dict(gate="channel")),
    (2, 16383, "fp16", "fp16", dict(gate="channel", sig=True)),
    (6, 2051, "fp16", "fp16", dict(gate="element", pad=5)),
    (6, 512, "bf16", "bf16", dict(pad=8, pre=False)),
    (6, 512, "bf16", "fp32", dict(pad=3, k=3)),
    (6, 512, "bf16", "bf16", dict(pad=7, shift=1)),
    (300, 96, "bf16", "bf16", dict(post=False, k=1)),
])
def test_block_norm(bq, T, K, dtype, res, opt):
    y, r, kw = norm_case(bq, T, K, dtype, res, **opt)
    ref, h, tol_r, tol_h = norm_reference(r, y, kw)
    got_r, got_h = bq.moe_block_norm(r, y, **kw)
    torch.cuda.synchronize()
    check(got_r, ref, tol_r + half_step(DT[res], ref), "residual")
    if h is None:
        assert got_h is None
    else:
        check(got_h, h, tol_h + half_step(DT[dtype], h), "h")


@pytest.mark.parametrize("T,K,dtype,res,opt", [
    (300, 4096, "bf16", "bf16", dict(k=2, gate="channel", drop=True)),
    (301, 2048, "fp16", "fp32", dict(gate="token", sig=True)),
    (310, 256, "bf16", "fp32", {}),
    (304, 512, "bf16", "bf16", dict(k=3, gate="element")),
    (303, 512, "fp16", "fp16", dict(gate="element", sig=True)),
    (299, 1000, "bf16", "bf16", dict(k=2)),
    (297, 7000, "bf16", "fp32", dict(k=6, gate="token", drop=True)),
    (297, 8192, "fp16", "fp16", dict(k=1)),
    (298, 14336, "bf16", "fp32", dict(k=2, gate="channel")),
    (298, 8200, "fp16", "fp16", dict(gate="element")),
    (300, 97, "bf16", "bf16", dict(k=2, gate="element")),
    (297, 2051, "fp16", "fp32", dict(k=2, gate="channel", drop=True)),
    (297, 6001, "bf16", "bf16", dict(k=8, gate="element", sig=True)),
    (297, 9001, "fp16", "fp16", dict(k=2, gate="element")),
    (297, 8999, "bf16", "fp32", dict(pad=2, gate="channel")),
    (297, 4100, "bf16", "bf16", dict(post=False, pad=3, shift=5)),
    (30, 9001, "bf16", "bf16", dict(k=2, shift=3, pad=4)),
])
def test_block_norm_row_shapes(bq, T, K, dtype, res, opt):
    """More rows than run at one time, and every way in which rows may lie."""
    test_block_norm(bq, T, K, dtype, res, opt)


def test_block_norm_forms(bq):
    """Plain pre-norm, no residual, in place, outputs into strided views, and rows of zeros."""
    y, r, kw = norm_case(bq, 5, 256, "bf16", "bf16")
    none, h = bq.moe_block_norm(r, w_pre=kw["w_pre"], eps=1e-5)
    ref = orc.rms_norm(f64(r), f64(kw["w_pre"]), 1e-5, 0.0)
    assert none is None
    check(h, ref, 96 * U * np.abs(ref) + half_step(torch.bfloat16, ref), "plain norm")
    only, _ = bq.moe_block_norm(None, y, w_post=kw["w_post"], eps=1e-5)
    ref = orc.rms_norm(f64(y), f64(kw["w_post"]), 1e-5, 0.0)
    check(only, ref, 96 * U * np.abs(ref) + half_step(torch.bfloat16, ref), "post norm alone")
    want_r, want_h = bq.moe_block_norm(r, y, **kw)
    inplace, hy = r.clone(), y.clone()
    a, b = bq.moe_block_norm(inplace, hy, residual_out=inplace, h_out=hy, **kw)
    assert a is inplace and torch.equal(inplace, want_r) and torch.equal(hy, want_h)
    big = torch.full((5, 300), 7.0, dtype=torch.bfloat16, device="cuda")
    bq.moe_block_norm(r, y, residual_out=big[:, 20:276], **kw)
    assert torch.equal(big[:, 20:276], want_r) and bool((big[:, :20] == 7).all()) and bool((big[:, 276:] == 7).all())
    zero, hz = bq.moe_block_norm(torch.zeros_like(r), torch.zeros_like(y), **kw)
    assert not zero.any() and not hz.any()
    empty_r, empty_h = bq.moe_block_norm(r[:0], y[:0], **{**kw, "gate": None})
    assert empty_r.shape == (0, 256) and empty_h.shape == (0, 256)


@pytest.mark.parametrize("T,K,post", [(1, 4096, True), (300, 256, False), (7, 2051, True)])
def test_block_norm_without_branch_rows(bq, T, K, post):
    """No expert had a row: every pair is dropped, and the branch adds nothing."""
    y, r, kw = norm_case(bq, T, K, "bf16", "bf16", k=3, gate="channel", post=post)
    kw["inv_pos"] = (torch.arange(3 * T, dtype=torch.int32).reshape(T, 3) - 1).cuda()
    none = y[:0].clone()
    got_r, got_h = bq.moe_block_norm(r, none, **kw)
    ref, h, tol_r, tol_h = norm_reference(r, none, kw)
    check(got_r, ref, tol_r + half_step(torch.bfloat16, ref), "residual")
    check(got_h, h, tol_h + half_step(torch.bfloat16, h), "h")


def test_block_norm_broadcast_rows(bq):
    """One residual row for every token (stride 0)."""
    y, r, kw = norm_case(bq, 9, 128, "fp16", "fp16")
    one = r[:1].expand(9, 128)
    ref, h, tol_r, tol_h = norm_reference(one, y, kw)
    got_r, got_h = bq.moe_block_norm(one, y, **kw)
    check(got_r, ref, tol_r + half_step(torch.float16, ref), "residual")
    check(got_h, h, tol_h + half_step(torch.float16, h), "h")


def test_block_norm_nan_stays_in_its_row(bq):
    y, r, kw = norm_case(bq, 40, 128, "bf16", "bf16")
    want_r, want_h = bq.moe_block_norm(r, y, **kw)
    y[7, 3] = float("nan")
    r[21, 0] = float("inf")
    got_r, got_h = bq.moe_block_norm(r, y, **kw)
    keep = [t for t in range(40) if t not in (7, 21)]
    assert torch.equal(got_r[keep], want_r[keep]) and torch.equal(got_h[keep], want_h[keep])
    assert bool(got_h[7].isnan().all()) and bool(got_h[21, 0].isnan())


# ---------------------------------------------------------------------------
# 8-bit rows
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("M,K,dtype,gather,pad", [
    (1, 64, "bf16", False, 0), (5, 1, "fp16", False, 0), (7, 2048, "bf16", True, 0), (33, 100, "fp16", True, 0),
    (3, 2056, "bf16", False, 0), (4, 7168, "fp16", True, 8), (2, 16384, "bf16", False, 0), (2, 16383, "fp16", False, 1),
    (300, 72, "bf16", True, 3),
])
def test_quantize_rows(bq, M, K, dtype, gather, pad):
    gen = seeded(M, K, pad)
    x = rnd(gen, (M, K + pad), 1.0, DT[dtype])[:, :K]
    # ties: the largest value a power of two, the others whole multiples of 1/254 of it where they exist
    x[0] = torch.randint(-127, 128, (K,), generator=gen).to(DT[dtype]).cuda() / 2
    x[0, 0] = 127.0
    src = None
    if gather:
        src = torch.randint(0, M, (2 * M + 1,), generator=gen).to(torch.int32)
        src[1] = -1
        src[-1] = M
        src = src.cuda()
    q, s = bq.moe_quantize_rows(x, src)
    want_q, want_s = orc.quantize_rows(f64(x), None if src is None else src.cpu().numpy())
    assert np.array_equal(q.cpu().numpy(), want_q)
    assert np.array_equal(s.cpu().numpy(), want_s.astype(np.float32))


@pytest.mark.parametrize("M,K,dtype,gather,pad", [
    (300, 4096, "bf16", False, 0), (301, 14336, "fp16", True, 0), (297, 512, "bf16", True, 0), (300, 4104, "fp16", False, 8),
    (298, 9001, "bf16", False, 0), (310, 16383, "fp16", False, 1), (400, 255, "bf16", True, 2), (303, 1024, "fp16", False, 3),
])
def test_quantize_row_shapes(bq, M, K, dtype, gather, pad):
    test_quantize_rows(bq, M, K, dtype, gather, pad)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_quantize_rows_ties(bq, dtype):
    """Rows of every finite magnitude up to their largest one, whose odd part is
    small, so that many quotients are half-integers; and scales near both ends of
    the type's range."""
    dt = DT[dtype]
    values = torch.arange(0x7c00 if dtype == "fp16" else 0x7f80, dtype=torch.int16).view(dt).double()
    lowest = float(values[1])
    tops = [lowest * m for m in (1, 3, 127, 254, 255, 1000)] + [m * 2.0 ** e for m in (1, 1.5, 1.25, 1.875, 127 / 64, 127 / 128 + 1)
                                                            for e in (-10, 0, 5)] + [float(values[-1]), float(values[-2])]
    if dtype == "bf16":
        tops += [1.5 * 2.0 ** e for e in (-126, -120, -65, -64, -63, 64, 127)]
    for top in tops:
        top = float(torch.tensor(top, dtype=torch.float64).to(dt).double())
        below = values[(values <= top) & (values > top / 300)]
        row = torch.cat([below[-8000:], -below[-8000:], torch.tensor([top, 0.0], dtype=torch.float64)])
        q, s = bq.moe_quantize_rows(row.to(dt).cuda()[None])
        want_q, want_s = orc.quantize_rows(row.numpy()[None])
        assert np.array_equal(q.cpu().numpy(), want_q), top
        assert np.array_equal(s.cpu().numpy(), want_s.astype(np.float32)), top


def test_quantize_rows_extremes(bq):
    rows = [[0.0] * 16, [float("nan")] + [1.0] * 15, [float("-inf")] + [1.0] * 15,
            [torch.finfo(torch.float16).max] * 8 + [-65504.0] * 8, [2.0 ** -24] * 4 + [0.0] * 12, [-0.0] * 15 + [1.0]]
    for dt in (torch.float16, torch.bfloat16):
        x = torch.tensor(rows, dtype=torch.float32).to(dt).cuda()
        q, s = bq.moe_quantize_rows(x)
        want_q, want_s = orc.quantize_rows(f64(x))
        assert np.array_equal(q.cpu().numpy(), want_q)
        assert np.array_equal(s.cpu().numpy(), want_s.astype(np.float32), equal_nan=True)
    x = torch.full((3, 8), 2.0 ** -130, dtype=torch.bfloat16).cuda()  # subnormal in fp32
    assert bool((bq.moe_quantize_rows(x)[0] == 127).all())


# ---------------------------------------------------------------------------
# products grouped by expert
# ---------------------------------------------------------------------------

def split(counts, lead=0):
    o = np.cumsum([lead] + list(counts))
    return torch.tensor(o, dtype=torch.int32).cuda()


def product(bq, op, x, w, off, out_dtype, xs=None, ws=None, out=None):
    if op == "int8":
        return bq.moe_int8_matmul(x, xs, w, ws, off, out_dtype=out_dtype, out=out)
    return bq.moe_grouped_matmul(x, w, off, out_dtype=out_dtype, out=out)


def operands(op, gen, R, E, N, K, pad=0, shift=0):
    """Whole-number operands whose sums are exact in fp32, and power-of-two scales."""
    lo, hi, dt = (-127, 127, torch.int8) if op == "int8" else (-8, 8, DT[op])
    x = ints(gen, (R, K + pad + shift), lo, hi, dt)[:, shift:shift + K]
    w = ints(gen, (E, N, K + pad + shift), lo, hi, dt)[:, :, shift:shift + K]
    if op != "int8":
        return x, w, None, None
    xs = 2.0 ** torch.randint(-3, 4, (R,), generator=gen).float().cuda()
    ws = 2.0 ** torch.randint(-3, 4, (E, N), generator=gen).float().cuda()
    return x, w, xs, ws


def run_exact(bq, op, out, counts, N, K, lead=0, tail=0, pad=0, shift=0, dense=False, ypad=0):
    E, R = len(counts), lead + sum(counts) + tail
    gen = seeded(R, E, N, K, pad, len(out), len(op))
    x, w, xs, ws = operands(op, gen, R, E, N, K, pad, shift)
    off = None if dense else split(counts, lead)
    y = torch.full((R, N + ypad), 77.0, dtype=DT[out], device="cuda")
    got = product(bq, op, x, w, off, DT[out], xs, ws, y[:, :N])
    assert bq.moe_op_sync_status() == 0
    ref, covered = orc.grouped_matmul(f64(x), f64(w), None if dense else off.cpu().numpy(),
                                      None if xs is None else f64(xs), None if ws is None else f64(ws))
    # int8 sums may pass 2^24: one fp32 rounding, then the output's
    want = torch.from_numpy(ref).to(torch.float32).to(DT[out])
    want[~torch.from_numpy(covered)] = 77.0
    same = torch.equal(got.cpu(), want)
    if not same:
        d = (got.cpu() != want).nonzero()
        raise AssertionError(f"{len(d)} of {want.numel()} differ, first {d[:4].tolist()}: "
                             f"{[(float(got[tuple(i)]), float(want[tuple(i)])) for i in d[:4]]}")
    assert bool((y[:, N:] == 77.0).all())


@pytest.mark.parametrize("op", ["bf16", "fp16", "int8"])
@pytest.mark.parametrize("counts,N,K,opt", [
    ([1], 128, 64, dict(dense=True)),
    ([1], 1, 16, dict(dense=True)),
    ([2], 100, 2048, dict(dense=True)),
    ([31], 129, 144, dict(dense=True)),
    ([33], 256, 512, dict(dense=True)),
    ([300], 257, 96, dict(dense=True)),
    ([1, 0, 2, 0], 64, 128, {}),
    ([0, 0, 0], 64, 128, dict(tail=5)),
    ([3, 129, 0, 64, 1], 384, 272, dict(lead=2, tail=7)),
    ([255, 256, 257, 1], 130, 80, {}),
    ([127, 128, 513], 640, 1008, dict(lead=1)),
    ([16] * 40, 72, 64, {}),
    ([5, 40], 96, 160, dict(pad=16)),
    ([5, 40], 96, 160, dict(pad=3)),
    ([5, 40], 90, 75, {}),
    ([70, 40], 96, 160, dict(pad=15, shift=1)),
    ([20, 30], 200, 64, dict(ypad=3)),
    ([20, 600], 200, 64, dict(ypad=56)),
])
def test_products_exact(bq, op, counts, N, K, opt):
    run_exact(bq, op, "fp32", counts, N, K, **opt)


@pytest.mark.parametrize("op", ["bf16", "int8"])
@pytest.mark.parametrize("counts,N,K,opt", [
    ([1], 2816, 2048, dict(dense=True)),
    ([16], 512, 4096, dict(dense=True)),
    ([17], 1024, 8192, dict(dense=True)),
    ([100], 640, 2048, dict(dense=True)),
    ([128], 1024, 4096, dict(dense=True)),
    ([250], 4096, 512, dict(dense=True)),
    ([500], 4000, 256, dict(dense=True)),
    ([760], 4096, 128, dict(dense=True)),
    ([1290], 4096, 64, dict(dense=True)),
    ([2100], 1500, 64, dict(dense=True)),
    ([90, 1, 0, 2, 3], 256, 2048, dict(lead=1, tail=2)),
    ([1, 1, 1, 77], 512, 4096, {}),
    ([33, 15, 16, 17, 0, 49], 128, 1024, {}),
    ([900, 0, 5, 3], 1100, 128, dict(tail=3)),
    ([64] * 9, 384, 640, {}),
])
def test_products_tile_forms(bq, op, counts, N, K, opt):
    """Sizes over the range in which the tiles' width and the split of K change."""
    run_exact(bq, op, "fp32", counts, N, K, **opt)
    run_exact(bq, op, "bf16", counts, N, K, **opt)


@pytest.mark.parametrize("op,counts,N,K", [f[:4] for f in FORMS])
def test_every_form_of_the_products(bq, op, counts, N, K):
    """Every tile width, split of K and sharing of the last turn that some size takes, into 32 and 16 bits."""
    if torch.cuda.get_device_properties(0).multi_processor_count != 148:
        pytest.skip("the forms are listed for 148 SMs")
    run_exact(bq, op, "fp32", counts, N, K)
    run_exact(bq, op, "bf16" if op == "int8" else op, counts, N, K)


@pytest.mark.parametrize("seed", range(12))
def test_products_random_shapes(bq, seed):
    rng = np.random.default_rng(100 + seed)
    E = int(rng.choice([1, 2, 7, 32]))
    counts = (rng.integers(0, 3, E) * np.exp(rng.uniform(0, 5, E))).astype(int).tolist()
    op = ["bf16", "fp16", "int8"][seed % 3]
    N, K = int(np.exp(rng.uniform(3, 7))), int(np.exp(rng.uniform(3, 7.5))) // 16 * 16 + 16
    run_exact(bq, op, "fp32", counts, N, K, lead=int(rng.integers(0, 3)), tail=int(rng.integers(1, 4)))


@pytest.mark.parametrize("op,out", [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "fp16"), ("int8", "bf16"),
                                    ("int8", "fp16")])
@pytest.mark.parametrize("counts,N,K", [([1], 256, 320), ([40, 0, 3, 270], 200, 144), ([9, 33], 131, 64)])
def test_products_rounded_once(bq, op, out, counts, N, K):
    run_exact(bq, op, out, counts, N, K, dense=len(counts) == 1)


@pytest.mark.parametrize("op", ["bf16", "int8"])
def test_products_many_experts(bq, op):
    rng = np.random.default_rng(5)
    counts = rng.integers(0, 7, 256)
    counts[rng.integers(0, 256, 80)] = 0
    counts[17] = 300
    run_exact(bq, op, "fp32", counts.tolist(), 96, 64, lead=3, tail=1)


@pytest.mark.parametrize("dtype,counts,N,K", [("bf16", [1], 512, 4096), ("fp16", [30, 2, 0, 200], 300, 2048),
                                              ("bf16", [700], 256, 1024)])
def test_grouped_matmul_gaussian(bq, dtype, counts, N, K):
    gen = seeded(N, K)
    x, w = rnd(gen, (sum(counts), K), 1.0, DT[dtype]), rnd(gen, (len(counts), N, K), 0.02, DT[dtype])
    off = split(counts)
    got = bq.moe_grouped_matmul(x, w, off, out_dtype=torch.float32)
    rounded = bq.moe_grouped_matmul(x, w, off)
    ref, _ = orc.grouped_matmul(f64(x), f64(w), off.cpu().numpy())
    mag, _ = orc.grouped_matmul(np.abs(f64(x)), np.abs(f64(w)), off.cpu().numpy())
    tol = K * 2.0 ** -23 * mag
    check(got, ref, tol, "fp32")
    check(rounded, ref, tol + half_step(DT[dtype], np.abs(ref) + tol), dtype)


@pytest.mark.parametrize("R,N,K", [(8, 512, 8192), (600, 4096, 8192), (300, 1024, 8192), (200, 256, 8191), (3, 200, 7168)])
def test_grouped_matmul_long_sums(bq, R, N, K):
    """The error of fp32 outputs does not grow with K. Accumulators truncate, 32
    times in 512 values of K, by at most 2^-23 of a partial sum each time, whose
    size is on average two thirds of the last: 32 * 2^-23 * 2 / 3 of a chunk's
    sum. Chunks are independent, so the whole output has the same relative error,
    and sqrt(chunks) roundings of 2^-24 more. Without chunks it would be 16 times
    as much at K = 8192."""
    gen = seeded(R, N, K)
    x, w = rnd(gen, (R, K), 1.0, torch.float16), rnd(gen, (1, N, K), 0.02, torch.float16)
    got = bq.moe_grouped_matmul(x, w, out_dtype=torch.float32).double()
    ref = x.double() @ w[0].double().t()
    assert float((got - ref).norm() / ref.norm()) <= 32 * 2.0 ** -23 * 2 / 3 + U * (K / 512) ** 0.5


@pytest.mark.parametrize("R,N,K", [(8, 512, 8192), (300, 1024, 8192), (3, 200, 7168)])
def test_grouped_matmul_long_sums_of_a_split(bq, R, N, K):
    """fp32 outputs where four CTAs split K, each summing some 2048 values of it. A
    chunk's 32 truncations take half a unit of 2^-23 each, on average 0.36 * 2^-23 of
    a partial sum that is two thirds of the chunk's: 32 * 0.36 * 2^-23 * 2 / 3, and
    the roundings to nearest of the chunks. 2048 values in one go: four times that."""
    gen = seeded(R, N, K)
    x, w = rnd(gen, (R, K), 1.0, torch.float16), rnd(gen, (1, N, K), 0.02, torch.float16)
    got = bq.moe_grouped_matmul(x, w, out_dtype=torch.float32).double()
    ref = x.double() @ w[0].double().t()
    assert float((got - ref).norm() / ref.norm()) <= 32 * 0.36 * 2.0 ** -23 * 2 / 3 + U * (K / 512) ** 0.5


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("R,N,K", [(2048, 2048, 14336), (16, 512, 131072), (200, 512, 14335)])
def test_16_bit_outputs_are_rounded_sums(bq, dtype, R, N, K):
    """How many 16-bit outputs are not the 64-bit value rounded once. A sum that is
    off by e rounds otherwise with probability e / step. Accumulators truncate 64
    times in 1024 values of K, each time by half a unit of 2^-23 on average, which is
    0.36 * 2^-23 of a partial sum between two powers of two, whose size is on average
    two thirds of its chunk's; chunks are independent and are added to nearest: e is
    64 * 0.36 * 2^-23 * 2 / 3 + 2^-24 sqrt(K / 1024) of the outputs' size. Twice the
    mean of e / step leaves room for the count's own spread. (All of K in one
    accumulator: 14 times as much at K = 14336.)"""
    gen = seeded(R, N, K, len(dtype), ord(dtype[0]))
    x, w = rnd(gen, (R, K), 1.0, DT[dtype]), rnd(gen, (1, N, K), 0.02, DT[dtype])
    got = bq.moe_grouped_matmul(x, w).double()
    ref = x.double() @ w[0].double().t()
    fi = torch.finfo(DT[dtype])
    step = torch.exp2(torch.floor(torch.log2(ref.abs().clamp_min(fi.smallest_normal)))) * fi.eps
    off = ((got - ref).abs() > step / 2).double().mean()
    e = (64 * 0.36 * 2.0 ** -23 * 2 / 3 + U * (K / 1024) ** 0.5) * ref.square().mean().sqrt()
    assert float(off) <= 2 * float((e / step).clamp_max(1.0).mean()) + 4 / ref.numel()


@pytest.mark.parametrize("out", ["fp16", "fp32"])
@pytest.mark.parametrize("R,N,K", [(64, 256, 131072), (300, 1024, 65536), (1100, 2048, 32768), (3, 200, 131071), (400, 512, 65535)])
def test_grouped_matmul_sums_do_not_drift(bq, out, R, N, K):
    """Positive terms, where truncation always takes away: 64 times in 1024 values
    of K at most 2^-23 of a partial sum, which is no larger than the chunk's: 64 *
    2^-23 of the output at any K; and K / 512 + 4 additions to nearest, 2^-24 of a
    partial output each. In one go it would be up to K / 16 * 2^-23."""
    gen = seeded(R, N, K)
    x = (torch.rand(R, K, generator=gen) + 0.5).half().cuda()
    w = (torch.rand(1, N, K, generator=gen) / 1024).half().cuda()
    got = bq.moe_grouped_matmul(x, w, out_dtype=DT[out]).double()
    ref = x.double() @ w[0].double().t()
    tol = (64 * 2.0 ** -23 + (K / 512 + 4) * U) * ref
    fi = torch.finfo(DT[out])
    half = torch.exp2(torch.floor(torch.log2(ref + tol))) * fi.eps / 2
    worst = float(((got - ref).abs() - half).max() / tol.min())
    assert bool(((got - ref).abs() <= half + tol).all()), worst


@pytest.mark.parametrize("out", ["bf16", "fp32"])
def test_int8_matmul_scales(bq, out):
    gen = seeded(11)
    counts, N, K = [3, 0, 61], 160, 1024
    x, w = ints(gen, (64, K), -128, 127, torch.int8), ints(gen, (3, N, K), -128, 127, torch.int8)
    xs, ws = torch.rand(64, generator=gen).cuda(), torch.rand(3, N, generator=gen).cuda()
    off = split(counts)
    got = bq.moe_int8_matmul(x, xs, w, ws, off, out_dtype=DT[out])
    ref, _ = orc.grouped_matmul(f64(x), f64(w), off.cpu().numpy(), f64(xs), f64(ws))
    check(got, ref, 3 * U * np.abs(ref) * 1.01 + half_step(DT[out], ref) * 1.01, out)


@pytest.mark.parametrize("rows,N,K", [(2, 64, 131071), (40, 256, 131056)])
def test_int8_largest_sums(bq, rows, N, K):
    """Every product 128 * 128: the sum comes within 2^14 of the int32 range."""
    x = torch.full((rows, K), -128, dtype=torch.int8, device="cuda")
    w = torch.full((1, N, K), -128, dtype=torch.int8, device="cuda")
    y = bq.moe_int8_matmul(x, torch.ones(rows, device="cuda"), w, torch.ones(1, N, device="cuda"),
                           out_dtype=torch.float32)
    assert bool((y == float(np.float32(K * 16384))).all())


@pytest.mark.parametrize("op", ["bf16", "int8"])
def test_products_bad_offsets_stay_inside(bq, op):
    """Offsets that descend or leave the range act as their running maximum clamped to the rows."""
    gen = seeded(4)
    x, w, xs, ws = operands(op, gen, 50, 4, 64, 64)
    for o in ([0, 30, 10, 40, 50], [-9, 5, 5, 2 ** 31 - 1, 3], [50, 0, 0, 0, 0], [-1, -2, -3, -4, -5],
              [0, 10, 60, 70, 2 ** 30]):
        off = torch.tensor(o, dtype=torch.int32).cuda()
        y = torch.full((50, 64), 77.0, device="cuda")
        product(bq, op, x, w, off, torch.float32, xs, ws, y)
        ref, covered = orc.grouped_matmul(f64(x), f64(w), o, None if xs is None else f64(xs),
                                          None if ws is None else f64(ws))
        ref[~covered] = 77.0
        assert bq.moe_op_sync_status() == 0
        assert np.array_equal(f64(y), ref)


@pytest.mark.parametrize("counts", [[5, 6, 7], [40, 3, 200]])
def test_products_nan_stays_with_its_rows(bq, counts):
    """A NaN or infinity in one row, or in another expert's weights, reaches no other output."""
    gen = seeded(8, counts[0])
    R, N, K = sum(counts), 160, 96
    x, w, _, _ = operands("bf16", gen, R + 4, 3, N, K)
    off = split(counts)
    clean = bq.moe_grouped_matmul(x, w, off, out_dtype=torch.float32)
    x2, w2 = x.clone(), w.clone()
    x2[2, 5] = float("nan")
    x2[R:] = float("inf")         # rows of no expert
    w2[1] = float("nan")          # a whole expert
    w2[2, N - 1, K - 1] = float("inf")
    got = bq.moe_grouped_matmul(x2, w2, off, out_dtype=torch.float32)
    a, b = counts[0], counts[0] + counts[1]
    keep = [r for r in range(a) if r != 2]
    assert torch.equal(got[keep], clean[keep]) and bool(got[2].isnan().all()) and bool(got[a:b].isnan().all())
    assert torch.equal(got[b:R, :N - 1], clean[b:R, :N - 1])
    q = torch.zeros(R, 64, dtype=torch.int8, device="cuda")
    xs = torch.ones(R, device="cuda")
    xs[1] = float("nan")
    y = bq.moe_int8_matmul(q, xs, torch.zeros(3, 32, 64, dtype=torch.int8, device="cuda"), torch.ones(3, 32, device="cuda"),
                           off, out_dtype=torch.float32)
    assert bool(y[1].isnan().all()) and int(y.isnan().sum()) == 32


@pytest.mark.parametrize("op", ["bf16", "int8"])
def test_products_weight_strides(bq, op):
    """Experts taken from a larger stack: every second one, and a slice of the channels."""
    gen = seeded(21)
    x, w, xs, ws = operands(op, gen, 90, 6, 256, 128)
    off = split([30, 20, 40])
    part = w[::2, 64:224]
    sc = None if ws is None else ws[::2, 64:224].contiguous()
    got = product(bq, op, x, part, off, torch.float32, xs, sc)
    want = product(bq, op, x, part.contiguous(), off, torch.float32, xs, sc)
    ref, _ = orc.grouped_matmul(f64(x), f64(part), off.cpu().numpy(), None if xs is None else f64(xs),
                                None if sc is None else f64(sc))
    assert torch.equal(got, want) and np.array_equal(f64(got), ref)


@pytest.mark.parametrize("op", ["bf16", "int8"])
@pytest.mark.parametrize("R", [24, 700])
def test_products_repeat_bitwise(bq, op, R):
    gen = seeded(R)
    x = rnd(gen, (R, 512), 1.0, torch.bfloat16)
    w = rnd(gen, (4, 384, 512), 1.0, torch.bfloat16)
    off = split([R // 4, R // 2, 0, R // 4])
    if op == "int8":
        x, xs = bq.moe_quantize_rows(x)
        w, ws = bq.moe_quantize_rows(w.reshape(-1, 512))
        w, ws = w.reshape(4, 384, 512), ws.reshape(4, 384)
    else:
        xs = ws = None
    first = product(bq, op, x, w, off, torch.float32, xs, ws)
    for _ in range(5):
        assert torch.equal(product(bq, op, x, w, off, torch.float32, xs, ws), first)


FAR = 2 ** 30 + 256  # elements between rows: the third row lies beyond 2^31


@pytest.fixture
def far_rows():
    """Three rows of a matrix that spans more than 2^31 elements, at column c."""
    raw = torch.empty(2 * (2 * FAR + 4096), dtype=torch.uint8, device="cuda")
    yield lambda c, width, dtype: raw.view(dtype).as_strided((3, width), (FAR, 1), c)
    del raw
    torch.cuda.empty_cache()


def test_rows_beyond_2_31_elements(bq, far_rows):
    gen = seeded(41)
    put = lambda c, t: far_rows(c, t.shape[1], t.dtype).copy_(t)
    y, r, kw = norm_case(bq, 3, 256, "bf16", "bf16", k=1, gate="element")
    y = y[:3].contiguous()
    kw["inv_pos"] = torch.tensor([[2], [0], [1]], dtype=torch.int32).cuda()
    want = bq.moe_block_norm(r, y, **kw)
    kw["gate"] = put(0, kw["gate"])
    got = bq.moe_block_norm(put(256, r), put(512, y), residual_out=far_rows(768, 256, torch.bfloat16),
                            h_out=far_rows(1024, 256, torch.bfloat16), **kw)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    src = torch.tensor([2, 0, 1], dtype=torch.int32).cuda()
    want = bq.moe_quantize_rows(r, src)
    got = bq.moe_quantize_rows(far_rows(256, 256, torch.bfloat16), src, codes=far_rows(4000, 256, torch.int8))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("op", ["fp16", "int8"])
@pytest.mark.parametrize("shift", [0, 1])  # bulk copies, ordinary loads
def test_products_beyond_2_31_elements(bq, far_rows, op, shift):
    gen = seeded(42, shift)
    x, w, xs, ws = operands(op, gen, 3, 1, 160, 256)
    want = product(bq, op, x, w, None, torch.float32, xs, ws)
    far = far_rows(64 + shift, 256, x.dtype).copy_(x)
    y = far_rows(1024, 160, torch.float16)
    got = product(bq, op, far, w, None, torch.float16, xs, ws, y)
    assert torch.equal(got, want.half())
    # experts that far apart: the third one's rows
    x, w, xs, ws = operands(op, gen, 7, 3, 1, 256)
    off = split([2, 0, 5])
    want = product(bq, op, x, w, off, torch.float32, xs, ws)
    rows = far_rows(64 + shift, 256, x.dtype)
    rows.copy_(w[:, 0])
    apart = rows[:, None, :]
    got = product(bq, op, x, apart, off, torch.float32, xs, ws)
    assert torch.equal(got, want)
    assert bq.moe_op_sync_status() == 0


def test_refusals_on_the_device(bq):
    x = torch.zeros(8, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(2, 32, 64, dtype=torch.bfloat16, device="cuda")
    off = split([4, 4])
    for call in (lambda: bq.moe_grouped_matmul(x, w),                               # two experts without offsets
                 lambda: bq.moe_grouped_matmul(x, w, off.long()),
                 lambda: bq.moe_grouped_matmul(x, w, off[:2]),
                 lambda: bq.moe_grouped_matmul(x, w.half(), off),
                 lambda: bq.moe_grouped_matmul(x, w[:, :, :32], off),
                 lambda: bq.moe_grouped_matmul(x.t(), w, off),
                 lambda: bq.moe_grouped_matmul(x, w.cpu(), off),
                 lambda: bq.moe_grouped_matmul(x, w, off, out=torch.zeros(8, 31, device="cuda")),
                 lambda: bq.moe_grouped_matmul(x.float(), w.float(), off),
                 lambda: bq.moe_int8_matmul(x.to(torch.int8), torch.ones(7, device="cuda"), w.to(torch.int8),
                                            torch.ones(2, 32, device="cuda"), off),
                 lambda: bq.moe_int8_matmul(x.to(torch.int8), torch.ones(8, device="cuda"), w.to(torch.int8),
                                            torch.ones(2, 31, device="cuda"), off),
                 lambda: bq.moe_quantize_rows(x.float()),
                 lambda: bq.moe_block_norm(x, x[:4]),
                 lambda: bq.moe_block_norm(x, x, w_pre=torch.ones(64, device="cuda")),
                 lambda: bq.moe_block_norm(x, x, inv_pos=torch.zeros(8, 2, dtype=torch.int32, device="cuda")),
                 lambda: bq.moe_block_norm(x.half(), x)):
        with pytest.raises(bq.MoEError) as ei:
            call()
        assert ei.value.status == 1
    wide = torch.zeros(2, 16392, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(bq.MoEError) as ei:
        bq.moe_quantize_rows(wide)
    assert ei.value.status == 9
    assert bq.moe_op_sync_status() == 0


def test_block_norm_refused_forms(bq):
    x = torch.zeros(8, 64, dtype=torch.bfloat16, device="cuda")
    for kw in (dict(gate=torch.ones(8, 1, 64, dtype=torch.bfloat16, device="cuda")),
               dict(gate=torch.ones((), dtype=torch.bfloat16, device="cuda")),
               dict(gate=torch.ones(1, 64, dtype=torch.bfloat16, device="cuda")),
               dict(h_out=torch.zeros_like(x)),
               dict(residual_out=x[:, :32]),
               dict(residual_out=x.expand(8, 64).float())):
        with pytest.raises(bq.MoEError) as ei:
            bq.moe_block_norm(x, x, **kw)
        assert ei.value.status == 1


def test_written_tensors_raise_their_version(bq):
    """What a call writes into a given tensor is a change in place: a backward pass that saved it notices."""
    x = torch.randn(8, 64, device="cuda").bfloat16()
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    W = torch.zeros(32, 64, dtype=torch.bfloat16, device="cuda")
    r, h, y = torch.empty_like(x), torch.empty_like(x), torch.empty(8, 32, dtype=torch.bfloat16, device="cuda")
    q, s = torch.empty(8, 64, dtype=torch.int8, device="cuda"), torch.empty(8, device="cuda")
    z = torch.empty(8, 32, device="cuda")
    before = [t._version for t in (x, r, h, y, q, s, z)]
    bq.moe_block_norm(x, x, w_pre=w, residual_out=r, h_out=h)
    bq.moe_quantize_rows(x, codes=q, scales=s)
    bq.moe_grouped_matmul(x, W, out=y)
    bq.moe_int8_matmul(q, s, W.to(torch.int8), torch.ones(32, device="cuda"), out=z)
    assert [t._version - b for t, b in zip((x, r, h, y, q, s, z), before)] == [0, 1, 1, 1, 1, 1, 1]
    a = torch.ones(8, 32, dtype=torch.bfloat16, device="cuda", requires_grad=True)
    loss = (a * y).sum()
    bq.moe_grouped_matmul(x, W, out=y)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    with torch.inference_mode():
        out = torch.empty(8, 32, dtype=torch.bfloat16, device="cuda")
        bq.moe_grouped_matmul(x, W, out=out)
    bq.moe_grouped_matmul(x, W, out=out)  # an inference tensor has no version
    assert torch.equal(out, y)


@pytest.mark.parametrize("op", ["bf16", "int8"])
@pytest.mark.parametrize("R,N,K,pad", [
    (700, 2048, 2048, 0),    # CTA pairs
    (8, 256, 4096, 0),       # K split over a cluster
    (100, 128, 2048, 3),     # ordinary loads
])
def test_products_wait_limit_then_recovery(bq, op, R, N, K, pad):
    """With a limit of 1 ns the first wait between roles that is not over yet gives
    up: the call returns, the status says so once, and the next call is right."""
    gen = seeded(R, N, K)
    x, w, xs, ws = operands(op, gen, R, 1, N, K, pad)
    want = product(bq, op, x, w, None, torch.float32, xs, ws)
    assert bq.moe_op_sync_status() == 0
    bq.moe_op_set_wait_limit(1)
    try:
        seen = []
        for _ in range(5):
            product(bq, op, x, w, None, torch.float32, xs, ws)
            seen.append(bq.moe_op_sync_status())
            if seen[-1] == 8:
                break
    finally:
        bq.moe_op_set_wait_limit(0)
    assert seen[-1] == 8 and set(seen) <= {0, 8}, seen
    assert bq.moe_op_sync_status() == 0
    for _ in range(3):
        assert torch.equal(product(bq, op, x, w, None, torch.float32, xs, ws), want)
    assert bq.moe_op_sync_status() == 0


def test_every_stream_is_told_of_a_timeout(bq):
    """An answer about one stream takes no other stream's timeout away."""
    gen = seeded(31)
    x, w, _, _ = operands("bf16", gen, 700, 1, 2048, 2048)
    mine, other, idle = (torch.cuda.Stream() for _ in range(3))
    call = lambda st: bq.moe_grouped_matmul(x, w, stream=st.cuda_stream)
    torch.cuda.synchronize()
    for st in (mine, other, idle):
        want = call(st)
        bq.moe_op_sync_status(st.cuda_stream)
    assert all(bq.moe_op_sync_status(st.cuda_stream) == 0 for st in (mine, other, idle))
    bq.moe_op_set_wait_limit(1)
    try:
        for _ in range(5):
            call(mine)
            mine.synchronize()
            if bq.moe_op_sync_status(other.cuda_stream) == 8:
                break
    finally:
        bq.moe_op_set_wait_limit(0)
    # the stream whose call it was, the others, and the current one: each once
    for st in (mine.cuda_stream, idle.cuda_stream, torch.cuda.current_stream().cuda_stream):
        assert bq.moe_op_sync_status(st) == 8
    for st in (mine, other, idle, torch.cuda.current_stream()):
        assert bq.moe_op_sync_status(st.cuda_stream) == 0
    assert torch.equal(call(mine), want)
    assert bq.moe_op_sync_status(mine.cuda_stream) == 0
    # a stream whose first product comes after a timeout is not told of it
    late = torch.cuda.Stream(priority=-1)
    call(late)
    assert bq.moe_op_sync_status(late.cuda_stream) == 0


def test_timeout_of_a_replayed_product(bq):
    """Captured on one stream, replayed on another: both are told."""
    gen = seeded(32)
    x, w, _, _ = operands("int8", gen, 8, 1, 256, 4096)[:4]
    xs, ws = torch.ones(8, device="cuda"), torch.ones(1, 256, device="cuda")
    bq.moe_int8_matmul(x, xs, w, ws)
    here, there = torch.cuda.current_stream(), torch.cuda.Stream()
    with torch.cuda.stream(there):
        bq.moe_int8_matmul(x, xs, w, ws)
    for st in (here, there):
        bq.moe_op_sync_status(st.cuda_stream)
        assert bq.moe_op_sync_status(st.cuda_stream) == 0
    g = torch.cuda.CUDAGraph()
    bq.moe_op_set_wait_limit(1)
    try:
        with torch.cuda.graph(g):
            bq.moe_int8_matmul(x, xs, w, ws)
    finally:
        bq.moe_op_set_wait_limit(0)
    told = 0
    for _ in range(5):
        with torch.cuda.stream(there):
            g.replay()
        told = bq.moe_op_sync_status(there.cuda_stream)
        if told:
            break
    assert told == 8 and bq.moe_op_sync_status(here.cuda_stream) == 8
    assert bq.moe_op_sync_status(there.cuda_stream) == bq.moe_op_sync_status(here.cuda_stream) == 0


# ---------------------------------------------------------------------------
# streams, graphs and the calls together
# ---------------------------------------------------------------------------

def chain(bq, s):
    """A block with 8-bit gate/up and 16-bit down experts: norm, gathered
    quantisation, grouped products, SwiGLU, and the combining norm."""
    _, h = bq.moe_block_norm(s["res"], w_pre=s["w1n"])
    q, qs = bq.moe_quantize_rows(h, s["perm"])
    gu = bq.moe_int8_matmul(q, qs, s["w1q"], s["w1s"], s["off"], out_dtype=torch.float32)
    n = gu.shape[1] // 2
    z = (torch.nn.functional.silu(gu[:, :n]) * gu[:, n:]).to(torch.bfloat16)
    o = bq.moe_grouped_matmul(z, s["w2"], s["off"])
    return bq.moe_block_norm(s["res"], o, w_post=s["w2n"], w_pre=s["w3n"], branch_scale=0.5, inv_pos=s["inv"],
                             pair_weights=s["pw"]), (h, gu, z, o)


def chain_state(bq, T, E, k, K, N, seed):
    gen = seeded(T, E, k, K, N, seed)
    s = {"res": rnd(gen, (T, K), 1.0, torch.bfloat16)}
    logits = torch.randn(T, E, generator=gen).cuda()
    s["idx"] = torch.empty(T, k, dtype=torch.int32, device="cuda")
    s["pw"] = torch.empty(T, k, dtype=torch.float32, device="cuda")
    s["counts"] = torch.empty(E, dtype=torch.int32, device="cuda")
    s["off"] = torch.empty(E + 1, dtype=torch.int32, device="cuda")
    bq.moe_route_topk_noalloc(logits, k, s["idx"], s["pw"], s["counts"], s["off"])
    order = torch.argsort(s["idx"].flatten().long(), stable=True)
    s["perm"] = (order // k).to(torch.int32)
    inv = torch.empty_like(order)
    inv[order] = torch.arange(T * k, device="cuda")
    s["inv"] = inv.reshape(T, k).to(torch.int32)
    w1 = rnd(gen, (E * 2 * N, K), 0.05, torch.bfloat16)
    q, qs = bq.moe_quantize_rows(w1)
    s["w1q"], s["w1s"] = q.reshape(E, 2 * N, K), qs.reshape(E, 2 * N)
    s["w2"] = rnd(gen, (E, K, N), 0.05, torch.bfloat16)
    for name in ("w1n", "w2n", "w3n"):
        s[name] = rnd(gen, (K,), 0.1, torch.bfloat16) + 1
    return s


@pytest.mark.parametrize("T", [1, 5, 300])
def test_operators_together(bq, T):
    s = chain_state(bq, T, 8, 2, 256, 128, 1)
    (r, h), (h0, gu, z, o) = chain(bq, s)
    assert bq.moe_op_sync_status() == 0
    # each step against the oracle on the step's own inputs
    q, qs = orc.quantize_rows(f64(h0), s["perm"].cpu().numpy())
    ref, covered = orc.grouped_matmul(q, f64(s["w1q"]), s["off"].cpu().numpy(), qs, f64(s["w1s"]))
    assert covered.all()
    check(gu, ref, 5 * U * np.abs(ref), "gate/up")
    ref, _ = orc.grouped_matmul(f64(z), f64(s["w2"]), s["off"].cpu().numpy())
    mag, _ = orc.grouped_matmul(np.abs(f64(z)), np.abs(f64(s["w2"])), s["off"].cpu().numpy())
    tol = 128 * 2.0 ** -23 * mag
    check(o, ref, tol + half_step(torch.bfloat16, np.abs(ref) + tol), "down")
    kw = dict(w_pre=s["w3n"], w_post=s["w2n"], gate=None, gate_sigmoid=False, residual_scale=1.0, branch_scale=0.5,
              eps=1e-6, weight_offset=0.0, inv_pos=s["inv"], pair_weights=s["pw"])
    ref, rh, tol_r, tol_h = norm_reference(s["res"], o, kw)
    check(r, ref, tol_r + half_step(torch.bfloat16, ref), "residual")
    check(h, rh, tol_h + half_step(torch.bfloat16, rh), "h")


def test_layer_output_into_the_norm(bq):
    """The quantised layer's own output as the branch, on the layer's routing."""
    import moe_synth as ms
    from moe_testlib import make_blocks, make_layer
    cfg = ms.make_config("tiny")
    blocks = make_blocks(cfg, "cuda")
    L = make_layer(cfg, blocks, max_tokens=16)
    res, logits = ms.make_inputs(cfg, 16, "cuda")
    w = torch.ones(cfg.K, dtype=torch.bfloat16, device="cuda")
    _, X = bq.moe_block_norm(res, w_pre=w)
    Y = L.forward(X, logits, cfg.top_k)
    kw = dict(w_pre=w, w_post=w, gate=None, gate_sigmoid=False, residual_scale=1.0, branch_scale=1.0, eps=1e-6,
              weight_offset=0.0, inv_pos=None, pair_weights=None)
    r, h = bq.moe_block_norm(res, Y, w_pre=w, w_post=w)
    assert L.sync_status() == 0
    ref, rh, tol_r, tol_h = norm_reference(res, Y, kw)
    check(r, ref, tol_r + half_step(torch.bfloat16, ref), "residual")
    check(h, rh, tol_h + half_step(torch.bfloat16, rh), "h")
    L.close()


def test_operators_on_other_streams(bq):
    """The same calls on two side streams at once give what they give alone."""
    states = [chain_state(bq, T, 8, 2, 256, 128, 2) for T in (40, 90)]
    torch.cuda.synchronize()
    want = [chain(bq, s)[0] for s in states]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in states]
    got = []
    for _ in range(3):
        for st, s in zip(streams, states):
            with torch.cuda.stream(st):
                got.append(chain(bq, s)[0])
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert torch.equal(g[0], want[i % 2][0]) and torch.equal(g[1], want[i % 2][1])


def test_operators_on_a_given_stream(bq):
    """Outputs made for a call on another stream belong to that stream: freed and
    asked for again on the current one they do not come back while it may write."""
    s = chain_state(bq, 200, 8, 2, 256, 128, 6)
    (want_r, want_h), (h, gu, z, o) = chain(bq, s)
    want_q, want_qs = bq.moe_quantize_rows(h, s["perm"])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    st = side.cuda_stream
    for _ in range(3):
        _, h1 = bq.moe_block_norm(s["res"], w_pre=s["w1n"], stream=st)
        q, qs = bq.moe_quantize_rows(h1, s["perm"], stream=st)
        gu1 = bq.moe_int8_matmul(q, qs, s["w1q"], s["w1s"], s["off"], out_dtype=torch.float32, stream=st)
        o1 = bq.moe_grouped_matmul(z, s["w2"], s["off"], stream=st)
        r, hh = bq.moe_block_norm(s["res"], o1, w_post=s["w2n"], w_pre=s["w3n"], branch_scale=0.5, inv_pos=s["inv"],
                                  pair_weights=s["pw"], stream=st)
        del h1
        scratch = torch.full_like(h, 9.0)
        torch.cuda.synchronize()
        assert torch.equal(q, want_q) and torch.equal(qs, want_qs) and torch.equal(gu1, gu) and torch.equal(o1, o)
        assert torch.equal(r, want_r) and torch.equal(hh, want_h) and bool((scratch == 9.0).all())
    assert bq.moe_op_sync_status(st) == 0


def test_operators_captured(bq):
    """Two captured chains, replayed together with new inputs in their buffers."""
    states = [chain_state(bq, T, 8, 2, 256, 128, 3) for T in (24, 200)]
    for s in states:
        chain(bq, s)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for s in states:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(chain(bq, s)[0])
        graphs.append(g)
    for seed in (4, 5):
        fresh = [chain_state(bq, s["res"].shape[0], 8, 2, 256, 128, seed) for s in states]
        for s, f in zip(states, fresh):
            for name in s:
                s[name].copy_(f[name])
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        graphs[0].replay()
        with torch.cuda.stream(side):
            graphs[1].replay()
        torch.cuda.synchronize()
        got = [(o[0].clone(), o[1].clone()) for o in outs]
        for s, g in zip(fresh, got):
            want = chain(bq, s)[0]
            assert torch.equal(g[0], want[0]) and torch.equal(g[1], want[1])
    assert bq.moe_op_sync_status() == 0


FIRST_CALLS = """
import threading
import torch
import bit_quantized_moe_top_b200 as bq

torch.manual_seed(0)
x = torch.randn(40, 256, device="cuda").bfloat16()
w = torch.randn(2, 128, 256, device="cuda").bfloat16()
one = torch.ones(256, dtype=torch.bfloat16, device="cuda")
off = torch.tensor([0, 15, 40], dtype=torch.int32, device="cuda")
torch.cuda.synchronize()


def calls(x):
    _, h = bq.moe_block_norm(x, w_pre=one)
    q, s = bq.moe_quantize_rows(h)
    wq, ws = bq.moe_quantize_rows(w.reshape(-1, 256))
    y = bq.moe_int8_matmul(q, s, wq.reshape(2, 128, 256), ws.reshape(2, 128), off)
    return [h, q, s, y, bq.moe_grouped_matmul(h, w, off), bq.moe_grouped_matmul(h[:, 1:], w[:, :, 1:], off)]


def captured():
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = calls(x)
    g.replay()
    return [out]


def threads():
    out = [None] * 4

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            out[i] = calls(x)
            torch.cuda.current_stream().synchronize()

    ts = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    return out


first = MODE()
torch.cuda.synchronize()
want = calls(x)
torch.cuda.synchronize()
for got in first:
    assert all(torch.equal(a, b) for a, b in zip(got, want))
assert bq.moe_op_sync_status() == 0
print("the same")
"""


@pytest.mark.parametrize("mode", ["captured", "threads"])
def test_first_calls_of_a_process(bq, mode):
    """Nothing has to be called once beforehand: the first calls may be captured, or made by several threads at once."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS.replace("MODE", mode)], cwd=root, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "the same" in r.stdout, r.stderr[-2000:]
