"""MX4 (MXFP4) quantiser, grouped product and the layer on MX4 experts, against the definitions in 64
bits (tests/mx4_reference.py).

Bars.  Codes, scales and rounded values: equal.  Products whose partial sums all fit fp32 (small
whole-number data with block scales of one size): equal, whatever the order of the sums.  Other
products: every term is exact, a sum of K terms makes at most K roundings of 2^-24 relative each to
a partial sum no larger than the sum of the terms' magnitudes S, so |err| <= K 2^-24 S, plus half a
step of the output type.  An activation adds its own few roundings (16 x 2^-24 relative allowed:
exp 1 ulp, an addition, a division, a product) on top of what it makes of the sum's error.
"""
import ctypes

import numpy as np
import pytest
import torch

import moe_inputs as mi
import sparse_moe_expert_router_amd as moe
from tests import mx4_reference as ref

DEV = "cuda"
gpu = pytest.mark.gpu
FAKE = 1 << 20
ACTS = {"none": moe.ACT_NONE, "swiglu": moe.ACT_SWIGLU, "relu2": moe.ACT_RELU2}
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def say(*a):
    print(*a, flush=True)


def f64(t):
    return t.detach().double().cpu().numpy()


# ------------------------------------------------------------------------------------------
# without a GPU

def test_reference_rounds_ties_to_the_even_code():
    v = np.zeros((1, 64))
    v[0, :16] = [4, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, 6.9, 7.99, -.25, -.75, -5, -0., 0.1, 0.26]
    q, s = ref.quantize(v)
    assert s.tolist() == [[127, 0]]                         # floor(log2 7.99) - 2 = 0; an all-zero block
    want = [4, 0, 1, 1, 2, 2, 4, 4, 6, 6, 0, -1, -4, 0, 0, .5]
    assert ref.decode(q, s)[0, :16].tolist() == want
    assert (q[0, 5] & 15) == 8 and (q[0, 6] >> 4) == 8     # the sign of -0.25 -> -0 and of -0 is kept


def test_packer_matches_the_reference():
    w = torch.randn((3, 5, 128), generator=torch.Generator().manual_seed(1)) * 0.02
    w[0, 0, :32] = 0
    w[0, 1, 3] = 100.0
    q, s = mi.pack_mx4(w)
    rq, rs = ref.quantize(w.double().numpy())
    assert np.array_equal(s.numpy(), rs)
    np.testing.assert_array_equal(ref.decode(q.numpy(), s.numpy()), ref.decode(rq, rs))


def test_quantize_argument_checks():
    L = moe.lib()
    def q(v=FAKE, xt=1, rows=4, cols=128, codes=FAKE, s=FAKE, values=None):
        return L.moe_quantize_rows_mx4(v, xt, rows, cols, codes, s, values, None)
    for bad in (dict(v=None), dict(v=FAKE + 8), dict(xt=2), dict(xt=3), dict(xt=-1), dict(rows=0),
                dict(rows=(1 << 24) + 1), dict(cols=32), dict(cols=96), dict(cols=16448), dict(codes=None),
                dict(codes=FAKE + 4), dict(s=None), dict(s=FAKE + 1), dict(values=FAKE + 2)):
        assert q(**bad) == moe.EINVAL, bad


def test_matmul_argument_checks():
    L = moe.lib()
    def mm(x=FAKE, xs=None, xt=1, xr=8, K=128, perm=FAKE, k=2, rows=16, w=FAKE, ws=FAKE, E=4, N=48, off=FAKE, act=2,
           out=FAKE, os=None, ot=1):
        return L.moe_matmul_mx4(x, xs, xt, xr, K, perm, k, rows, w, ws, E, N, off, act, out, os, ot, None)
    for bad in (dict(x=None), dict(x=FAKE + 4), dict(xt=3), dict(xt=-1), dict(xs=FAKE), dict(xt=2), dict(xt=2, xs=FAKE + 1),
                dict(xr=0), dict(xr=(1 << 21) + 1), dict(K=32), dict(K=96), dict(K=16448), dict(k=0), dict(k=65),
                dict(rows=0), dict(rows=(1 << 21) + 1), dict(w=None), dict(w=FAKE + 2), dict(ws=None), dict(E=0),
                dict(E=513), dict(N=0), dict(N=65537), dict(N=47, act=0), dict(act=3), dict(act=-1), dict(off=None),
                dict(off=FAKE + 4), dict(perm=FAKE + 4), dict(perm=None), dict(perm=None, k=1), dict(out=None),
                dict(out=FAKE + 8), dict(os=FAKE), dict(ot=2), dict(ot=3)):
        assert mm(**bad) == moe.EINVAL, bad
    # MX4 results need MX4 rows and whole blocks of 32 output columns
    assert mm(ot=2, os=FAKE, N=64) == moe.EUNSUPPORTED
    assert mm(xt=2, xs=FAKE, ot=2, os=FAKE, N=48) == moe.EUNSUPPORTED
    assert mm(xt=2, xs=FAKE, ot=2, os=FAKE, N=96, act=0) == moe.EUNSUPPORTED
    assert mm(rows=1 << 20, N=(1 << 14) + 2) == moe.EUNSUPPORTED         # rows * N > 2^34


def test_layer_argument_checks():
    L = moe.lib()
    def fwd(E=8, d=256, dff=512, k=2, act=0, flags=0, S=0, ws_bytes=1024):
        s = moe.Experts(moe.W_MX4, E, d, dff, FAKE, FAKE, FAKE, FAKE, S)
        return L.moe_layer_forward(FAKE, 1, 4, FAKE, None, ctypes.byref(s), k, act, flags, FAKE, None, None, FAKE,
                                   ws_bytes, None)
    PM = moe.F_PREFILL_MX4
    for ok in (dict(), dict(flags=PM), dict(act=1), dict(act=1, flags=PM), dict(S=2)):
        assert fwd(**ok) == moe.EWORKSPACE, ok                 # accepted up to the workspace
    assert fwd(dff=96) == moe.EINVAL
    assert fwd(act=2) == moe.EINVAL                            # the bare product is no layer
    assert fwd(flags=PM | moe.F_PREFILL_I8) == moe.EINVAL
    assert fwd(flags=moe.F_PREFILL_I8) == moe.EUNSUPPORTED
    assert fwd(flags=moe.F_PREFILL_FP8) == moe.EUNSUPPORTED
    assert fwd(flags=moe.F_ZERO_SKIP) == moe.EUNSUPPORTED
    q8 = moe.Experts(moe.W_Q8_0, 8, 256, 512, FAKE, FAKE, FAKE, FAKE, 0)
    assert L.moe_workspace_bytes(4, 2, ctypes.byref(q8), 0, PM) == 0     # MX4 rows need MX4 weights
    mx = moe.Experts(moe.W_MX4, 8, 256, 512, FAKE, FAKE, FAKE, FAKE, 0)
    assert L.moe_workspace_bytes(4, 2, ctypes.byref(mx), 0, 0) > L.moe_workspace_bytes(4, 2, ctypes.byref(mx), 0, PM) > 0
    assert L.moe_read_intermediates(4, 2, ctypes.byref(mx), 0, PM, 1, FAKE, 1 << 30, FAKE, None, None,
                                    None) == moe.EUNSUPPORTED
    assert L.moe_repack_experts(ctypes.byref(mx), 0, ctypes.byref(mx), None) == moe.EINVAL


def test_binding_refuses_wrong_tensors():
    x = torch.zeros((4, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        moe.quantize_rows_mx4(x)                               # not on a GPU
    with pytest.raises(TypeError):
        moe.quantize_rows_mx4(x.half())
    with pytest.raises(TypeError):
        moe.quantize_rows_mx4([1.0])
    with pytest.raises(ValueError):
        moe.quantize_rows_mx4(torch.zeros((2, 2, 64)))
    with pytest.raises(ValueError):
        moe.matmul_mx4(x, torch.zeros((4, 64), dtype=torch.uint8), torch.zeros((4, 4), dtype=torch.uint8))


# ------------------------------------------------------------------------------------------
# quantiser

def edge_rows():
    """Blocks at the edges: zeros, ties at several scales, signed zeros, the smallest and largest
    values, powers of two and their neighbours, NaN and infinities."""
    t = torch.zeros((24, 64))
    ties = torch.tensor([.25, .75, 1.25, 1.75, 2.5, 3.5, 5., 7.])
    for i, e in enumerate((0, -30, 30, -120, -126, 100, 120)):
        t[i, :8] = torch.ldexp(ties, torch.tensor(e))
        t[i, 8:16] = -t[i, :8]
        t[i, 32:40] = torch.ldexp(ties.flip(0) * 0.9999, torch.tensor(e))
    t[7, :4] = torch.tensor([1e-45, -1e-45, 1e-40, 1.1754944e-38])
    t[8, :3] = torch.tensor([3.4028235e38, -3.4028235e38, 1e38])
    t[9, 5] = float("nan")
    t[10, 40] = float("inf")
    t[11, 0] = -float("inf")
    t[11, 32:] = 1.0
    t[12, :32] = -0.0
    t[13] = torch.arange(64) - 31.5
    t[14, :32] = 2.0 ** torch.arange(-16, 16)
    t[15, 0] = 7.9999995
    t[16, 0] = 8.0
    t[17, 0] = 2.0 ** -125
    t[18, 0] = 2.0 ** -124
    t[19, 0] = 2.0 ** -126
    return t


def check_quantize(v):
    q, s, val = moe.quantize_rows_mx4(v, want_values=True)
    q2, s2 = moe.quantize_rows_mx4(v)
    torch.cuda.synchronize()
    assert torch.equal(q, q2) and torch.equal(s, s2)
    rq, rs = ref.quantize(f64(v))
    assert np.array_equal(s.cpu().numpy(), rs)
    assert np.array_equal(q.cpu().numpy(), rq)
    np.testing.assert_array_equal(f64(val), ref.decode(rq, rs))


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_quantize_edges(dtype):
    check_quantize(edge_rows().to(dtype).to(DEV))


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,cols", [(1, 64), (1, 2816), (3, 704), (37, 192), (1, 16384), (257, 64)])
def test_quantize_random(rows, cols, dtype):
    g = torch.Generator(device=DEV).manual_seed(rows * 7 + cols)
    v = torch.randn((rows, cols), generator=g, device=DEV) * torch.exp(3 * torch.randn((rows, cols), generator=g, device=DEV))
    check_quantize(v.to(dtype))


# ------------------------------------------------------------------------------------------
# product

def make_w(E, N, K, seed, spread):
    """Random codes; scales 2^(0 .. -spread)."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    w = torch.randint(0, 256, (E, N, K // 2), generator=g, device=DEV, dtype=torch.int32).to(torch.uint8)
    s = (127 - torch.randint(0, spread + 1, (E, N, K // 32), generator=g, device=DEV, dtype=torch.int32)).to(torch.uint8)
    return w, s


def make_x(kind, rows, K, seed, spread, whole):
    """(argument, scales, float64 values): whole numbers up to 4 (or MX4 rows), or Gaussian."""
    g = torch.Generator(device=DEV).manual_seed(seed + 99)
    if kind == "mx4":
        q, s = make_w(1, rows, K, seed + 5, spread)
        return q[0], s[0], ref.decode(q[0].cpu(), s[0].cpu())
    x = torch.randn((rows, K), generator=g, device=DEV)
    if whole:
        x = torch.round(2 * x).clamp(-4, 4)
    x = x.to(torch.bfloat16 if kind == "bf16" else torch.float32)
    return x, None, f64(x)


def make_groups(E, rows, seed, how):
    """Ascending offsets over `rows` rows."""
    r = np.random.default_rng(seed)
    if how == "one":                                            # everything in one group
        c = np.zeros(E, np.int64)
        c[E // 2] = rows
    elif how == "short":                                        # rows behind the last group
        c = np.bincount(r.integers(0, E, rows - rows // 4), minlength=E)
    elif how == "hot":
        c = np.bincount(np.minimum(r.geometric(0.3, rows) - 1, E - 1), minlength=E)
    else:
        c = np.bincount(r.integers(0, E, rows), minlength=E)
    return np.concatenate([[0], np.cumsum(c)]).astype(np.int32)


def run_product(kind, E, N, K, rows, act, out_dtype, how="even", gather=True, k=3, spread=1, whole=True, seed=0):
    """A call and its reference: (out, y before the activation, S, offsets)."""
    w, ws = make_w(E, N, K, seed, spread)
    T = max(1, -(-rows // k)) if gather else rows
    x, xs, xv = make_x(kind, T, K, seed, spread, whole)
    off = make_groups(E, rows, seed, how)
    r = np.random.default_rng(seed + 3)
    perm = r.permutation(T * k)[:rows].astype(np.int32) if gather else None
    src = perm // k if gather else np.arange(rows)
    cols = N // 2 if act == "swiglu" else N
    out = torch.full((rows, cols), -77.0, dtype=out_dtype, device=DEV)
    say(f"product {kind} E={E} N={N} K={K} rows={rows} {act} {out_dtype} {how} gather={gather}")
    got = moe.matmul_mx4(x, w, ws, x_scales=xs, offsets=torch.from_numpy(off).to(DEV),
                         perm=None if perm is None else torch.from_numpy(perm).to(DEV), k=k if gather else 1,
                         act=ACTS[act], out_dtype=out_dtype, out=out)
    torch.cuda.synchronize()
    assert got is out
    y, S = ref.product(xv, ref.decode(w.cpu(), ws.cpu()), off, src)
    assert (f64(out)[off[-1]:] == -77.0).all()                  # rows of no group stay as they were
    return f64(out)[:off[-1]], y[:off[-1]], S[:off[-1]]


SHAPES = [  # E, N, K, rows, how
    (1, 1, 64, 1, "even"), (1, 16, 64, 1, "even"), (8, 48, 64, 5, "even"), (4, 96, 192, 33, "even"),
    (5, 130, 704, 77, "even"), (128, 64, 320, 64, "even"), (3, 258, 128, 300, "hot"), (512, 32, 64, 700, "even"),
    (2, 514, 256, 129, "one"), (6, 34, 448, 41, "short"), (130, 36, 64, 1000, "hot"), (4, 320, 2816, 40, "even"),
    (2, 64, 16384, 3, "even"),
]


@gpu
@pytest.mark.parametrize("kind", ["mx4", "bf16", "f32"])
@pytest.mark.parametrize("E,N,K,rows,how", SHAPES, ids=["E%d-N%d-K%d-r%d-%s" % s for s in SHAPES])
def test_product_exact_sums(kind, E, N, K, rows, how):
    """Data whose every partial sum fits 24 bits: the fp32 result is the exact one, bit for bit.
    Terms are multiples of 2^-4 (codes' halves, scales 2^0 or 2^-1 on either side) of at most 36, so
    sums of up to 16384 of them stay below 2^20 = 2^24 x 2^-4."""
    got, y, _ = run_product(kind, E, N, K, rows, "none", torch.float32, how, gather=rows % 2 == 1, seed=E + N + K)
    assert np.abs(y).max() < 2 ** 20
    np.testing.assert_array_equal(got, y)


@gpu
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("act", ["none", "swiglu", "relu2"])
@pytest.mark.parametrize("kind", ["mx4", "bf16", "f32"])
@pytest.mark.parametrize("E,N,K,rows", [(4, 96, 192, 33), (3, 258, 704, 150), (8, 34, 1024, 9)])
def test_product_bounds(kind, act, out_dtype, E, N, K, rows):
    """Gaussian rows and scales over 2^0 .. 2^-6, each activation and output type, to the derived bound."""
    got, y, S = run_product(kind, E, N, K, rows, act, out_dtype, spread=6, whole=False, seed=N + rows)
    err = K * 2.0 ** -24 * S
    want = ref.activate(y, act)
    if act == "relu2":
        bound = 2 * np.maximum(y, 0) * err + err ** 2
    elif act == "swiglu":
        g, u = y[:, :N // 2], y[:, N // 2:]
        eg, eu = err[:, :N // 2], err[:, N // 2:]
        bound = 1.1 * eg * (np.abs(u) + eu) + np.abs(g) * eu    # |silu'| <= 1.1, |silu(g)| <= |g|
    else:
        bound = err
    bound = bound + (16 * 2.0 ** -24 + HALF[out_dtype]) * (np.abs(want) + bound) + 1e-35
    worst = float((np.abs(got - want) / bound).max())
    say("  worst error / bound:", worst)
    assert worst <= 1
    assert np.linalg.norm(got - want) <= (2e-6 if out_dtype == torch.float32 else HALF[out_dtype]) * np.linalg.norm(want)


@gpu
@pytest.mark.parametrize("act,N", [("swiglu", 128), ("swiglu", 192), ("relu2", 96), ("none", 320), ("none", 32)])
def test_product_mx4_result_is_its_fp32_result_quantised(act, N):
    E, K, rows = 5, 320, 201
    w, ws = make_w(E, N, K, N, 3)
    x, xs, _ = make_x("mx4", rows, K, 5, 3, False)
    off = torch.from_numpy(make_groups(E, rows, 1, "hot")).to(DEV)
    kw = dict(x_scales=xs, offsets=off, act=ACTS[act])
    y = moe.matmul_mx4(x, w, ws, out_dtype=torch.float32, **kw)
    q, s = moe.matmul_mx4(x, w, ws, out_dtype=torch.uint8, **kw)
    cols = y.shape[1]
    if cols % 64:                                               # the quantiser takes whole 64s
        y = torch.nn.functional.pad(y, (0, 64 - cols % 64))
    rq, rs = moe.quantize_rows_mx4(y)
    torch.cuda.synchronize()
    assert torch.equal(q, rq[:, :cols // 2]) and torch.equal(s, rs[:, :cols // 32])


@gpu
@pytest.mark.parametrize("kind", ["mx4", "bf16", "f32"])
def test_product_nan_and_infinity_stay_in_their_rows(kind):
    """A NaN block of x, a NaN scale of one weight row and (bf16) an infinite value reach the outputs
    that use them and no other; the padding of short tiles is not read as data."""
    E, N, K, rows = 2, 48, 192, 21
    w, ws = make_w(E, N, K, 3, 1)
    x, xs, xv = make_x(kind, rows, K, 3, 1, True)
    off = np.array([0, 11, 21], np.int32)
    ws[1, 7, 2] = 255
    if kind == "mx4":
        xs[4, 1] = 255
    else:
        x[4, 40] = float("nan")
    want, _ = ref.product(xv, ref.decode(w.cpu(), ws.cpu()), off, np.arange(rows))
    want[4] = np.nan
    got = moe.matmul_mx4(x, w, ws, x_scales=xs, offsets=torch.from_numpy(off).to(DEV), out_dtype=torch.float32)
    torch.cuda.synchronize()
    assert np.isnan(want[11:, 7]).all() and np.isfinite(np.delete(want, 4, 0)[:10]).all()
    np.testing.assert_array_equal(f64(got), want)


@gpu
@pytest.mark.parametrize("kind", ["mx4", "bf16", "f32"])
def test_product_bad_indexes_stay_in_bounds(kind):
    """Permutation entries outside the pairs are clamped into the rows of x; offsets outside
    [0, rows] are clamped; the results are those of the clamped values."""
    E, N, K, rows, T, k = 3, 32, 128, 20, 7, 3
    w, ws = make_w(E, N, K, 8, 1)
    x, xs, xv = make_x(kind, T, K, 8, 1, True)
    perm = np.arange(rows).astype(np.int32)
    perm[3], perm[9] = -5, 10 ** 8
    off = np.array([-4, 6, 13, 1000], np.int32)
    src = np.clip(perm // k, 0, T - 1)
    want, _ = ref.product(xv, ref.decode(w.cpu(), ws.cpu()), np.clip(off, 0, rows), src)
    got = moe.matmul_mx4(x, w, ws, x_scales=xs, offsets=torch.from_numpy(off).to(DEV),
                         perm=torch.from_numpy(perm).to(DEV), k=k, out_dtype=torch.float32)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(f64(got), want)


@gpu
def test_product_of_one_group_without_offsets():
    for kind in ("mx4", "bf16", "f32"):
        w, ws = make_w(1, 80, 256, 2, 1)
        x, xs, xv = make_x(kind, 150, 256, 2, 1, True)
        got = moe.matmul_mx4(x, w[0], ws[0], x_scales=xs, out_dtype=torch.float32)
        torch.cuda.synchronize()
        np.testing.assert_array_equal(f64(got), xv @ ref.decode(w[0].cpu(), ws[0].cpu()).T)


@gpu
@pytest.mark.parametrize("kind", ["mx4", "bf16", "f32"])
def test_product_at_the_ends_of_the_scales(kind):
    """Scale bytes from 1 to 253, and 0 and 254 with codes that stay in range, against rows that bring
    the products back: every sum here has one nonzero term per block pair, exact in fp32."""
    K, N = 256, 48
    w = torch.zeros((1, N, K // 2), dtype=torch.uint8)
    ws = torch.full((1, N, K // 32), 127, dtype=torch.uint8)
    e = torch.linspace(-126, 126, N).round().int()
    w[0, :, 0], ws[0, :, 0] = 0x02, (e + 127).to(torch.uint8)          # 1 x 2^e at column 0
    w[0, 0, 0], ws[0, 0, 0] = 0x02, 254                                # 2^127
    w[0, 1, 0], ws[0, 1, 0] = 0x07, 0                                  # 6 x 2^-127, normal in fp32
    x = torch.zeros((3, K))
    x[:, 0] = torch.tensor([1.0, -1.5, 2.0]) * torch.tensor([1.0, 2.0 ** -10, 2.0 ** 10])
    xs = None
    if kind == "mx4":
        q, s = ref.quantize(x.double().numpy())
        x, xs = torch.from_numpy(q).to(DEV), torch.from_numpy(s).to(DEV)
        xv = ref.decode(q, s)
    else:
        xv = x.double().numpy()
        x = x.to(torch.bfloat16 if kind == "bf16" else torch.float32).to(DEV)
    want = xv @ ref.decode(w[0], ws[0]).T
    got = f64(moe.matmul_mx4(x, w.to(DEV), ws.to(DEV), x_scales=xs, out_dtype=torch.float32))
    normal = (np.abs(want) >= 2.0 ** -126) & (np.abs(want) < 2.0 ** 128)
    assert normal.sum() > 120
    np.testing.assert_array_equal(got[normal], want[normal])
    assert np.abs(got[np.abs(want) < 2.0 ** -126]).max() <= 2.0 ** -126   # below: flushed or kept


@gpu
@pytest.mark.parametrize("kind", ["mx4", "bf16"])
def test_product_past_32_bit_offsets(kind):
    """Outputs of over 2^32 bytes, and weights of over 2^32 bytes: the last rows and the last group."""
    K = 64
    rows, N = 1 << 19, 2304                                             # 4.8 GB of fp32
    w, ws = make_w(2, N, K, 1, 1)
    x, xs, xv = make_x(kind, rows, K, 1, 1, True)
    off = torch.tensor([0, 1000, rows], dtype=torch.int32, device=DEV)
    got = moe.matmul_mx4(x, w, ws, x_scales=xs, offsets=off, out_dtype=torch.float32)
    at = np.r_[0:3, 998:1003, rows // 2:rows // 2 + 3, rows - 5:rows]
    wv = ref.decode(w.cpu(), ws.cpu())
    want = np.stack([xv[r] @ wv[0 if r < 1000 else 1].T for r in at])
    np.testing.assert_array_equal(f64(got[torch.from_numpy(at).to(DEV)]), want)
    del got, x
    K, N, E = 16384, 8192, 70                                           # 4.7 GB of codes
    w = torch.zeros((E, N, K // 2), dtype=torch.uint8, device=DEV)
    ws = torch.full((E, N, K // 32), 127, dtype=torch.uint8, device=DEV)
    w1, ws1 = make_w(1, N, K, 2, 1)
    w[-1], ws[-1] = w1[0], ws1[0]
    x, xs, xv = make_x(kind, 3, K, 3, 1, True)
    off = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    off[-1] = 3
    got = moe.matmul_mx4(x, w, ws, x_scales=xs, offsets=off, out_dtype=torch.float32)
    np.testing.assert_array_equal(f64(got), xv @ ref.decode(w1[0].cpu(), ws1[0].cpu()).T)


@gpu
def test_product_on_a_side_stream_of_its_own_inputs():
    """Two products at once on two streams, each with its own inputs and outputs."""
    E, N, K, rows = 8, 512, 1024, 400
    args, want = [], []
    for i, kind in enumerate(("mx4", "bf16")):
        w, ws = make_w(E, N, K, i, 3)
        x, xs, _ = make_x(kind, rows, K, i, 3, False)
        args.append((x, w, ws, xs, torch.from_numpy(make_groups(E, rows, i, "even")).to(DEV)))
        x, w, ws, xs, off = args[-1]
        want.append(moe.matmul_mx4(x, w, ws, x_scales=xs, offsets=off))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in args]
    got = [[], []]
    for _ in range(6):
        for i, s in enumerate(streams):
            x, w, ws, xs, off = args[i]
            with torch.cuda.stream(s):
                got[i].append(moe.matmul_mx4(x, w, ws, x_scales=xs, offsets=off))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(g, want[i]) for g in got[i])


@gpu
def test_refusals_on_the_gpu():
    w, ws = make_w(2, 64, 128, 0, 1)
    x = torch.zeros((4, 128), dtype=torch.bfloat16, device=DEV)
    off = torch.tensor([0, 2, 4], dtype=torch.int32, device=DEV)
    ok = dict(offsets=off)
    assert moe.matmul_mx4(x, w, ws, **ok).shape == (4, 64)
    for bad in (dict(offsets=None), dict(offsets=off.long()), dict(offsets=off[:2].contiguous()), dict(offsets=off.cpu()),
                dict(ok, perm=off.long()), dict(ok, perm=off[:, None]), dict(ok, x_scales=ws), dict(ok, out_dtype=torch.float16),
                dict(ok, out=torch.zeros((4, 63), dtype=torch.bfloat16, device=DEV)),
                dict(ok, out=torch.zeros((64, 4), dtype=torch.bfloat16, device=DEV).T)):
        with pytest.raises((TypeError, ValueError)):
            moe.matmul_mx4(x, w, ws, **bad)
    for bad in (dict(ok, act=7), dict(ok, k=3), dict(ok, out_dtype=torch.uint8)):
        with pytest.raises(moe.MoeError):
            moe.matmul_mx4(x, w, ws, **bad)
    with pytest.raises(ValueError):
        moe.matmul_mx4(x[:, ::2], w, ws, **ok)                 # strided, and too short
    with pytest.raises(ValueError):
        moe.quantize_rows_mx4(x.T)
    with pytest.raises(moe.MoeError):
        moe.quantize_rows_mx4(x[:, :96].contiguous())          # not a multiple of 64
    with pytest.raises(moe.MoeError):
        moe.quantize_rows_mx4(x[:0])                           # no rows
    with pytest.raises(moe.MoeError):
        moe.matmul_mx4(x.view(-1)[4:388].view(3, 128), w[0], ws[0])   # 8 bytes off a 16-byte boundary


# ------------------------------------------------------------------------------------------
# the layer on MX4 experts

def layer_case(T, E, k, d, dff, act, S=0, xtype=mi.X_BF16):
    w = mi.workload("tiny", T=T, E=E, k=k, d_model=d, d_ff=dff, act=act, fmt=mi.FMT_MX4, xtype=xtype, n_shared=S)
    lay = mi.make_layer(w, 0, DEV)
    return w, lay, mi.make_x(w, 0, device=DEV)


LAYERS = [(1, 8, 2, 256, 512, mi.ACT_SWIGLU, 0), (5, 8, 3, 192, 128, mi.ACT_SWIGLU, 1), (37, 40, 4, 320, 192, mi.ACT_RELU2, 0),
          (70, 6, 6, 128, 64, mi.ACT_SWIGLU, 2), (300, 16, 2, 256, 192, mi.ACT_RELU2, 1)]
LAYER_IDS = ["T%d-E%d-k%d-d%d-f%d-act%d-S%d" % c for c in LAYERS]


def reference_layer(lay, x, idx, wts, act):
    ex = lay["experts"]
    E, S = ex["E"], ex["n_shared"]
    gu = ref.decode(ex["gate_up"].cpu(), ex["gate_up_scales"].cpu())
    dn = ref.decode(ex["down"].cpu(), ex["down_scales"].cpu())
    xv, out = f64(x), np.zeros((x.shape[0], ex["d_model"]))
    for t in range(x.shape[0]):
        for j, e in enumerate(list(idx[t]) + [E + s for s in range(S)]):
            h = ref.activate(gu[e] @ xv[t], "swiglu" if act == mi.ACT_SWIGLU else "relu2")
            out[t] += (wts[t, j] if j < idx.shape[1] else 1.0) * (dn[e] @ h)
    return out


@gpu
@pytest.mark.parametrize("xtype", [mi.X_BF16, mi.X_F32])
@pytest.mark.parametrize("case", LAYERS, ids=LAYER_IDS)
def test_layer_matches_the_definition(case, xtype):
    """Exact x and h: the error is that of fp32 sums of at most 512 terms and of the activation, so a
    row is within 1e-4 of its largest output (the bar of the other exact-product decode paths)."""
    T, E, k, d, dff, act, S = case
    w, lay, x = layer_case(T, E, k, d, dff, act, S, xtype)
    out, idx, wts = moe.layer_forward(x, lay["w_router"], lay["bias"], lay["experts"], k, act, want_routing=True)
    st = moe.layer_forward_static(x, lay["w_router"], lay["bias"], lay["experts"], k, act)
    ex = moe.experts_forward(x, idx, wts, lay["experts"], act)
    torch.cuda.synchronize()
    assert torch.equal(out, st) and torch.equal(out, ex)
    want = reference_layer(lay, x, idx.cpu().numpy(), f64(wts), act)
    err = np.abs(f64(out) - want).max(1) / np.abs(want).max(1)
    say("  rel err", float(err.max()))
    assert err.max() < 1e-4


@gpu
@pytest.mark.parametrize("case", LAYERS, ids=LAYER_IDS)
def test_prefill_layer_is_the_run_of_its_operators(case):
    """route, permute, quantise, product with the activation into MX4 rows, product, combine: the
    operators called one by one give the layer's output (the combine's fp32 sums apart)."""
    T, E, k, d, dff, act, S = case
    w, lay, x = layer_case(T, E, k, d, dff, act, S)
    ex = lay["experts"]
    out, idx, wts = moe.layer_forward(x, lay["w_router"], lay["bias"], ex, k, act, moe.F_PREFILL_MX4, want_routing=True)
    ri, rw = moe.route(x, lay["w_router"], lay["bias"], k)
    counts, off, perm, inv = moe.permute(ri, E)
    q, s = moe.quantize_rows_mx4(x)
    gu, gus, dn, dns = (ex[n] for n in ("gate_up", "gate_up_scales", "down", "down_scales"))
    hq, hs = moe.matmul_mx4(q, gu[:E], gus[:E], x_scales=s, offsets=off, perm=perm, k=k, act=act, out_dtype=torch.uint8)
    y = moe.matmul_mx4(hq, dn[:E], dns[:E], x_scales=hs, offsets=off, out_dtype=torch.float32)
    shared = []
    for e in range(E, E + S):
        hq, hs = moe.matmul_mx4(q, gu[e], gus[e], x_scales=s, act=act, out_dtype=torch.uint8)
        shared.append(moe.matmul_mx4(hq, dn[e], dns[e], x_scales=hs, out_dtype=torch.float32))
    torch.cuda.synchronize()
    assert torch.equal(ri, idx) and torch.equal(rw, wts)
    yp = f64(y)[inv.cpu().numpy()].reshape(T, k, d)
    want = (yp * f64(wts)[:, :, None]).sum(1) + sum(f64(v) for v in shared)
    mag = (np.abs(yp) * f64(wts)[:, :, None]).sum(1) + sum(np.abs(f64(v)) for v in shared)
    assert (np.abs(f64(out) - want) <= (k + S + 1) * 2.0 ** -23 * mag).all()


@gpu
def test_prefill_layer_near_the_exact_layer():
    """4-bit rounding of x and h moves the output by a bounded share: a value is off by at most 1/4 of
    its size or 1/8 of its block's largest (half a step), about 0.1 of its norm, at both roundings.
    Catches a wrong operand, not a rounding."""
    w, lay, x = layer_case(64, 16, 4, 512, 512, mi.ACT_SWIGLU)
    args = (x, lay["w_router"], lay["bias"], lay["experts"], 4, mi.ACT_SWIGLU)
    a, b = f64(moe.layer_forward(*args)), f64(moe.layer_forward(*args, moe.F_PREFILL_MX4))
    assert 0.01 < np.linalg.norm(a - b) / np.linalg.norm(a) < 0.5


@gpu
@pytest.mark.parametrize("name,T,act", [("gemma_decode", 8, mi.ACT_SWIGLU), ("gemma_prefill", 300, mi.ACT_SWIGLU),
                                        ("nemotron_latent", 4, mi.ACT_RELU2)])
def test_full_size_layers(name, T, act):
    """Whole layers of the benchmarked shapes on a few of their tokens: exact x and h to the decode bar;
    with MX4 rows, h within its rounding of the exact one (at most 1 step of the block, 2 where a value
    above 6 saturates), and the output that of the rounded h (fp32 sums: 1e-5 of the largest output)."""
    w = mi.workload(name, T=T, fmt=mi.FMT_MX4)
    lay = mi.make_layer(w, 0, DEV)
    x, ex, k = mi.make_x(w, 0, device=DEV), lay["experts"], w.k
    out, idx, wts = moe.layer_forward(x, lay["w_router"], lay["bias"], ex, k, act, want_routing=True)
    outq = moe.layer_forward(x, lay["w_router"], lay["bias"], ex, k, act, moe.F_PREFILL_MX4)
    _, off, perm, inv = moe.permute(idx, w.E)
    q, qs = moe.quantize_rows_mx4(x)
    hq, hs = moe.matmul_mx4(q, ex["gate_up"], ex["gate_up_scales"], x_scales=qs, offsets=off, perm=perm, k=k, act=act,
                            out_dtype=torch.uint8)
    torch.cuda.synchronize()
    hv = ref.decode(hq.cpu(), hs.cpu())[inv.cpu().numpy()].reshape(T, k, -1)
    step = np.ldexp(1.0, hs.cpu().numpy().astype(int) - 127).repeat(32, 1)[inv.cpu().numpy()].reshape(T, k, -1)
    xv, xqv = f64(x), ref.decode(q.cpu(), qs.cpu())
    a = "swiglu" if act == mi.ACT_SWIGLU else "relu2"
    for t in sorted({0, T // 2, T - 1}):
        want, wantq = np.zeros(w.d_model), np.zeros(w.d_model)
        for j, e in enumerate(idx[t].tolist()):
            gu = ref.decode(ex["gate_up"][e].cpu(), ex["gate_up_scales"][e].cpu())
            dn = ref.decode(ex["down"][e].cpu(), ex["down_scales"][e].cpu())
            want += float(wts[t, j]) * (dn @ ref.activate(gu @ xv[t], a))
            h = ref.activate(gu @ xqv[t], a)
            assert (np.abs(hv[t, j] - h) <= 2 * step[t, j] * (1 + 1e-5)).all()
            small = np.abs(h) <= 6 * step[t, j]
            assert (np.abs(hv[t, j] - h)[small] <= step[t, j][small] * (1 + 1e-5)).all()
            wantq += float(wts[t, j]) * (dn @ hv[t, j])
        assert np.abs(f64(out[t]) - want).max() <= 1e-4 * np.abs(want).max()
        assert np.abs(f64(outq[t]) - wantq).max() <= 1e-5 * np.abs(wantq).max()


@gpu
def test_intermediates_of_mx4_experts():
    T, E, k, d, dff = 9, 8, 2, 128, 192
    w, lay, x = layer_case(T, E, k, d, dff, mi.ACT_SWIGLU)
    ex = lay["experts"]
    ws = moe.alloc_workspace(moe.workspace_bytes(T, k, ex, mi.ACT_SWIGLU))
    out, idx, _ = moe.layer_forward(x, lay["w_router"], lay["bias"], ex, k, mi.ACT_SWIGLU, ws=ws, want_routing=True)
    h = moe.read_intermediates(T, k, ex, mi.ACT_SWIGLU, 0, ws)
    torch.cuda.synchronize()
    gu, xv = ref.decode(ex["gate_up"].cpu(), ex["gate_up_scales"].cpu()), f64(x)
    for p, e in enumerate(idx.cpu().numpy().reshape(-1)):
        want = ref.activate(gu[e] @ xv[p // k], "swiglu")
        assert np.abs(f64(h)[p] - want).max() <= 1e-5 * np.abs(want).max()


# ------------------------------------------------------------------------------------------
# streams, graphs, repetition

@gpu
@pytest.mark.parametrize("kind", ["mx4", "bf16", "f32"])
def test_product_repeats_and_replays_bit_for_bit(kind):
    """The same call three times, on another stream, and captured in a graph that is replayed with
    eager work between the replays and new inputs in place."""
    E, N, K, rows = 6, 200, 448, 90
    w, ws = make_w(E, N, K, 4, 5)
    x, xs, _ = make_x(kind, rows, K, 4, 5, False)
    off = torch.from_numpy(make_groups(E, rows, 2, "even")).to(DEV)
    def call(out=None):
        return moe.matmul_mx4(x, w, ws, x_scales=xs, offsets=off, act=moe.ACT_SWIGLU, out_dtype=torch.float32, out=out)
    first = call()
    assert all(torch.equal(call(), first) for _ in range(2))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = call()
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(other, first)
    out = torch.zeros_like(first)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(out)
    for i in range(4):
        if i == 2:
            x.copy_(x.flip(0))
            if xs is not None:
                xs.copy_(xs.flip(0))
        want = call()
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), i


@gpu
def test_layer_replays_in_a_graph():
    w, lay, x = layer_case(40, 8, 2, 256, 192, mi.ACT_SWIGLU, 1)
    for flags in (0, moe.F_PREFILL_MX4):
        ws = moe.alloc_workspace(moe.workspace_bytes(40, 2, lay["experts"], mi.ACT_SWIGLU, flags))
        args = (x, lay["w_router"], lay["bias"], lay["experts"], 2, mi.ACT_SWIGLU, flags)
        want = moe.layer_forward(*args)
        out = torch.zeros_like(want)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            moe.layer_forward(*args, out=out, ws=ws)
        for _ in range(4):
            out.zero_()
            ws.fill_(255)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want)
            assert torch.equal(moe.layer_forward(*args), want)
